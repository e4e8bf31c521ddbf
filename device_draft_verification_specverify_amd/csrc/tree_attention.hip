// tree_attention.hip -- attention of drafted tree nodes over a paged prefix and
// their ancestors (gfx950, matrix cores).
//
// Keys of a request are numbered 0 .. len + n - 1: the cached prefix, then the
// tree's nodes. Rows are (node, query head of the group) pairs of one key head.
// One pass over the keys with a running maximum m and sum l of the softmax.
//
// Both products are taken transposed. S^T = K Q^T leaves each lane the scores of
// ONE row (column lane % 32 of the 32x32 accumulator), so the running maximum,
// sum and rescaling are per-lane scalars; and the lane's scores, in order, are
// already the second operand of O^T = V^T P^T if V's keys are read in the same
// order: k index 8 h + j of a 16-key step (h = lane / 32) is key 4 h + j for
// j < 4 and 8 + 4 h + j - 4 for the rest, which is how the accumulator holds
// them. V^T fragments come from the row-major tile by the transposing LDS read
// (4 keys x 16 columns per 16 lanes).

#include "tree_common.h"

namespace {

using namespace svtree;

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

#define LDS_PTR(p) ((__attribute__((address_space(3))) void*)(p))
#define GLOBAL_PTR(p) ((const __attribute__((address_space(1))) void*)(p))

template <int DT>
struct Elem;
template <>
struct Elem<SV_BF16> {
  typedef __bf16 type;
  typedef bf16x8 vec;
  static __device__ __forceinline__ bool wild(uint32_t bits) { return (~bits & 0x7F80u) == 0; }
  static __device__ __forceinline__ f32x16 mfma(s16x8 a, vec b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(vec, a), b, c, 0, 0, 0);
  }
};
template <>
struct Elem<SV_F16> {
  typedef _Float16 type;
  typedef f16x8 vec;
  static __device__ __forceinline__ bool wild(uint32_t bits) { return (~bits & 0x7C00u) == 0; }
  static __device__ __forceinline__ f32x16 mfma(s16x8 a, vec b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(vec, a), b, c, 0, 0, 0);
  }
};

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

struct AttnArgs {
  const char* q;
  const char* k_tree;
  const char* k_cache;
  int64_t v_tree, v_cache;  // byte distance of the values from the keys
  int64_t q_t, q_h, n_t, n_h, c_page, c_token, c_h, o_t, o_h;  // bytes
  const int32_t* table;
  const int32_t* prefix_len;
  const int32_t* node_start;
  const uint64_t* anc;
  char* out;
  float* lse;
  int32_t* err;
  int64_t B, T, table_stride, num_pages, max_keys;
  int Hq, Hkv, G, D, max_nodes, words, page_shift;
  float scale_log2;
  // workspace
  int64_t* first_tile;  // [B + 1] tiles in front of each request
  float* part;          // [workers * 2][M][DP + 2]: sums, then m and l
  int tile_keys, tile_rows, width;
};

__device__ const u32x4 zero_piece = {0, 0, 0, 0};

// Tiles of request b, and its sizes.
struct Req {
  int64_t first;
  int32_t n, len, tiles, row_tiles;
};
__device__ __forceinline__ Req request(const AttnArgs& a, int64_t b) {
  Req r;
  const Nodes nd = nodes_of(a.node_start, b, a.T, a.max_nodes);
  r.first = nd.first;
  r.n = nd.n < 0 ? 0 : nd.n;
  const int64_t len = a.prefix_len[b];
  r.len = int32_t(len < 0 ? 0 : len > a.max_keys ? a.max_keys : len);
  r.tiles = (r.len + r.n + a.tile_keys - 1) / a.tile_keys;
  r.row_tiles = (r.n * a.G + a.tile_rows - 1) / a.tile_rows;
  return r;
}
__device__ __forceinline__ int64_t tiles_of(const AttnArgs& a, const Req& r) {
  return int64_t(r.tiles) * r.row_tiles * a.Hkv;
}

// Worker w's share of `total` tiles starts here.
__device__ __forceinline__ int64_t share_start(int64_t total, int workers, int64_t w) {
  const int64_t q = total / workers, rem = total % workers;
  return w * q + (w < rem ? w : rem);
}
__device__ __forceinline__ int64_t worker_of(int64_t total, int workers, int64_t tile) {
  const int64_t q = total / workers, rem = total % workers;
  const int64_t big = rem * (q + 1);
  return tile < big ? tile / (q + 1) : rem + (tile - big) / q;
}

// Where the 16-byte piece c of row r of a tile lies (in pieces of its row): 16
// rows that are read at one column, and 4 rows read over 64 bytes, fall on
// different banks.
template <int CPR>
__device__ __forceinline__ int swizzle(int r) {
  if constexpr (CPR == 8) return (((r >> 1) & 1) << 2) | ((r >> 2) & 3);
  else return ((r & 3) << 2) | ((r >> 2) & 3);
}

// 64 bits of a row's mask from node x on; what is in front of node 0 is the
// prefix, which every row sees. No branches: per-score branches around values
// in accumulation registers were compiled into wrong code.
__device__ __forceinline__ uint64_t window(uint64_t m0, uint64_t m1, int x) {
  const uint64_t none = x >= 128 ? 0 : m1 >> (x & 63);
  const uint64_t both = (m0 >> (x & 63)) | ((m1 << 1) << (63 - (x & 63)));
  const int before = (-x) & 63;
  const uint64_t some = (m0 << before) | ((uint64_t(1) << before) - 1);
  return x <= -64 ? ~uint64_t(0) : x < 0 ? some : x < 64 ? both : none;
}

// 16 bytes a lane from global memory straight into LDS at `to` (the wavefront's
// lanes in order). Written out because the compiler puts a wait for all such
// loads in front of every later LDS read; the loop below counts them itself.
__device__ __forceinline__ void load_lds16(const char* from, uint32_t to) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
               :
               : "s"(to), "v"(from)
               : "memory", "m0");
}

// This wavefront's loads but the newest N have landed and its LDS reads are
// done; then the workgroup meets.
template <int N>
__device__ __forceinline__ void wait_and_meet() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" : : "n"(N) : "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" : : : "memory");
}

constexpr int kTablePart = 1024;  // page ids held in LDS at a time

// RW wavefronts along the rows (32 each), KW along a tile's keys (KB each), a
// ring of S tiles.
template <int DT, int DP, int RW, int KW, int KB, int S>
__global__ __launch_bounds__(64 * RW * KW) void attention_kernel(AttnArgs a) {
  using E = Elem<DT>;
  using elem = typename E::type;
  constexpr int NT = 64 * RW * KW;
  constexpr int KT = KW * KB;
  constexpr int CPR = DP / 8;
  constexpr int M = 32 * RW;
  constexpr int NB = KB / 32;
  constexpr int ND = DP / 32;
  constexpr int UNITS = KT * CPR / NT;
  constexpr int STEP = DP / 16 < 8 ? DP / 16 : 8;  // fragments of K read at once
  static_assert(KT * CPR % NT == 0, "whole rounds of 16-byte pieces");
  constexpr int STAGE = 2 * KT * DP * 2;  // bytes of a tile's keys and values
  constexpr int LOADS = 2 * UNITS;        // of a thread for a tile
  static_assert((KW - 1) * RW * ND * 16 * 64 * 4 <= S * STAGE, "the merge fits the tile");
  __shared__ __align__(1024) char tile[S * STAGE];
  __shared__ int32_t ids[kTablePart];
  __shared__ float merge_ml[KW][RW][2][32];
  __shared__ int64_t scan[NT / 64 + 1];
  __shared__ int64_t found[2];
  const int tid = int(threadIdx.x), lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int rw = wv % RW, kw = wv / RW;
  const int col = lane & 31, half = lane >> 5;

  // This worker's share: neighbours in the order of tiles share an XCD's L2
  // (workgroups go round robin over the 8 XCDs).
  const int workers = int(gridDim.x);
  const int64_t w = workers % 8 == 0 ? (blockIdx.x % 8) * (workers / 8) + blockIdx.x / 8
                                     : blockIdx.x;
  int64_t total = 0;
  for (int64_t o = tid; o < a.B; o += NT) total += tiles_of(a, request(a, o));
  for (int d = 32; d >= 1; d /= 2) total += __shfl_xor(total, d);
  if (lane == 0) scan[wv] = total;
  __syncthreads();
  total = 0;
  for (int k = 0; k < NT / 64; ++k) total += scan[k];
  __syncthreads();
  int64_t at = share_start(total, workers, w);
  const int64_t end = share_start(total, workers, w + 1);
  if (at >= end && w != 0) return;

  // the request that holds tile `at`; worker 0 writes down where all begin
  int64_t base = 0;
  for (int64_t o = 0; o < a.B; o += NT) {
    int64_t mine = o + tid < a.B ? tiles_of(a, request(a, o + tid)) : 0;
    int64_t s = mine;
    for (int d = 1; d < 64; d *= 2) {
      const int64_t y = __shfl_up(s, d);
      if (lane >= d) s += y;
    }
    if (lane == 63) scan[wv] = s;
    __syncthreads();
    int64_t before = base;
    for (int k = 0; k < wv; ++k) before += scan[k];
    int64_t all = base;
    for (int k = 0; k < NT / 64; ++k) all += scan[k];
    const int64_t lo = before + s - mine;
    if (w == 0 && o + tid < a.B) a.first_tile[o + tid] = lo;
    if (at >= lo && at < lo + mine) {
      found[0] = o + tid;
      found[1] = lo;
    }
    base = all;
    __syncthreads();
    if (w != 0 && base > at) break;
  }
  if (w == 0 && tid == 0) a.first_tile[a.B] = total;
  if (w == 0) {  // wrong requests are reported once
    int bits = 0;
    for (int64_t o = tid; o < a.B; o += NT) {
      const int64_t len = a.prefix_len[o];
      if (len < 0 || len > a.max_keys) bits |= SV_ERR_LENGTH;
      if (nodes_of(a.node_start, o, a.T, a.max_nodes).n < 0) bits |= SV_ERR_TREE;
    }
    if (bits) set_error(a.err, bits);
  }
  if (at >= end) return;
  int64_t b = found[0];
  int64_t b_first = found[1];
  Req rq = request(a, b);

  // This lane's places in a stage. K: row col, piece 2 ks + half; V: 4 keys from
  // 4 half on at 4 columns. Pieces are swizzled by their row, rows a multiple of
  // 16 apart alike, and stages begin at multiples of 1024, so the ks-th piece
  // and the db-th 32 columns are one exclusive or away.
  const uint32_t k_off = (kw * KB + col) * (DP * 2) + ((half ^ swizzle<CPR>(col)) * 16);
  const int v_row = 4 * half + ((lane & 15) >> 2);
  const uint32_t v_off = KT * DP * 2 + (kw * KB + v_row) * (DP * 2) +
                         (((((lane >> 4) & 1) * 2 + ((lane & 3) >> 1)) ^ swizzle<CPR>(v_row)) * 16) +
                         (lane & 1) * 8;
  const uint32_t tile_at = __builtin_amdgcn_readfirstlane(
      uint32_t(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) char*)tile)));
  while (at < end) {
    while (at >= b_first + tiles_of(a, rq)) {
      b_first += tiles_of(a, rq);
      rq = request(a, ++b);
    }
    const int item = int((at - b_first) / rq.tiles);  // (key head, row tile)
    const int t0 = int((at - b_first) - int64_t(item) * rq.tiles);
    const int t1 = int(rq.tiles - t0 < end - at ? rq.tiles : t0 + (end - at));
    const int h = item / rq.row_tiles, rt = item - h * rq.row_tiles;
    const int n = rq.n, len = rq.len, keys = len + n;
    const int32_t* const table = a.table + b * a.table_stride;

    // this lane's row
    const int r = rt * M + rw * 32 + col;
    const bool row_ok = r < n * a.G;
    const int node = row_ok ? r / a.G : 0;
    const int hq = h * a.G + (row_ok ? r - node * a.G : 0);
    const bool wave_ok = rt * M + rw * 32 < n * a.G;
    uint64_t see0 = 0, see1 = 0;
    typename E::vec qf[DP / 16];
    if (wave_ok) {
      const char* qp = a.q + (rq.first + node) * a.q_t + hq * a.q_h;
#pragma unroll
      for (int s = 0; s < DP / 16; ++s) {
        const int d = 16 * s + 8 * half;
        u32x4 x = {0, 0, 0, 0};
        if (d < a.D) x = *reinterpret_cast<const u32x4*>(qp + d * 2);
        qf[s] = __builtin_bit_cast(typename E::vec, x);
      }
      if (a.anc) {
        const uint64_t* m = a.anc + (rq.first + node) * a.words;
        see0 = m[0];
        if (a.words > 1) see1 = m[1];
      } else {
        see0 = node >= 63 ? ~uint64_t(0) : (uint64_t(2) << node) - 1;
        see1 = node < 64 ? 0 : node >= 127 ? ~uint64_t(0) : (uint64_t(2) << (node - 64)) - 1;
      }
      // bits behind the tree are none of its nodes
      see0 &= n >= 64 ? ~uint64_t(0) : (uint64_t(1) << n) - 1;
      see1 &= n >= 128 ? ~uint64_t(0) : n <= 64 ? 0 : (uint64_t(1) << (n - 64)) - 1;
    }
    f32x16 acc[ND];
#pragma unroll
    for (int i = 0; i < ND; ++i) acc[i] = f32x16{0};
    float m = -INFINITY, l = 0.0f;
    int wild = 0;

    // Page ids of the share, a part at a time; bad ones become -1.
    int ids_from = 0, ids_to = 0;  // pages held
    auto fetch_ids = [&](int t) {
      const int need = min(min(t * KT + KT, len) - 1, len - 1) >> a.page_shift;
      if (len == 0 || t * KT >= len || need < ids_to) return;
      __syncthreads();  // the ids before are read
      ids_from = (t * KT) >> a.page_shift;
      const int last = (min(t1 * KT, len) - 1) >> a.page_shift;
      ids_to = min(ids_from + kTablePart, last + 1);
      for (int i = tid; i < ids_to - ids_from; i += NT) {
        int32_t id = table[ids_from + i];
        if (id < 0 || id >= a.num_pages) {
          set_error(a.err, SV_ERR_PAGE);
          id = -1;
        }
        ids[i] = id;
      }
      __syncthreads();
    };
    // Starts a tile's keys and values on their way into stage t % S. Branches
    // only where the whole workgroup takes them; lanes choose between addresses.
    const char* const zero = reinterpret_cast<const char*>(&zero_piece);
    const char* const k_head = a.k_cache + h * a.c_h;
    const char* const k_node = a.k_tree + rq.first * a.n_t + h * a.n_h;
    const int64_t c_page = a.c_page, c_token = a.c_token, v_cache = a.v_cache;
    const int in_page = (1 << a.page_shift) - 1, page_shift = a.page_shift;
    auto fetch = [&](int t) {
      fetch_ids(t);
      const uint32_t stage = tile_at + uint32_t(t % S) * STAGE;
      const int key0 = t * KT + tid / CPR;
      const bool inside = t * KT + KT <= len;  // cached keys only
      int32_t id[UNITS];
#pragma unroll
      for (int u = 0; u < UNITS; ++u) {
        const int key = key0 + u * (NT / CPR);
        const int at_id = (key >> page_shift) - ids_from;
        id[u] = ids[inside || key < len ? at_id : 0];
      }
#pragma unroll
      for (int u = 0; u < UNITS; ++u) {
        const int row = u * (NT / CPR) + tid / CPR;
        // rounds of 16 rows and more repeat the order of pieces
        const int c = (tid % CPR) ^ swizzle<CPR>(NT / CPR % 16 == 0 ? tid / CPR : row);
        const int key = t * KT + row;
        const char* kp = k_head + c * 16 + uint32_t(id[u]) * uint64_t(c_page) +
                         uint32_t(key & in_page) * uint64_t(c_token);
        bool some = id[u] >= 0;
        const char* vp = kp + v_cache;
        if (!inside) {
          const char* np = k_node + c * 16 + int64_t(key - len) * a.n_t;
          const char* nv = np + a.v_tree;
          some = key < len ? some : key < keys;
          kp = key < len ? kp : np;
          vp = key < len ? vp : nv;
        }
        some = some && (DP == a.D || c * 8 < a.D);
        kp = some ? kp : zero;
        vp = some ? vp : zero;
        const uint32_t to = stage + (u * NT + wv * 64) * 16;
        load_lds16(kp, to);
        load_lds16(vp, to + KT * DP * 2);
      }
    };
#pragma unroll
    for (int i = 0; i < S - 1; ++i)
      if (t0 + i < t1) fetch(t0 + i);

    for (int t = t0; t < t1; ++t) {
      // tile t is here; everyone is done with tile t - 1, whose stage is next
      if (S >= 4 && t1 - t > 2) wait_and_meet<2 * LOADS>();
      else if (S >= 3 && t1 - t > 1) wait_and_meet<LOADS>();
      else wait_and_meet<0>();
      if (t + S - 1 < t1) fetch(t + S - 1);
      char* const tv = tile + (t % S) * STAGE + KT * DP * 2;
      const uint32_t stage = tile_at + uint32_t(t % S) * STAGE;
      // Nodes' values that are infinite or NaN would reach the rows that do not
      // see them as 0 * inf: they become zeros here and are added at the end.
      if (t * KT + KT > len) {
        bool mine = false;
#pragma unroll
        for (int u = 0; u < UNITS; ++u) {
          const int unit = u * NT + tid;
          const int key = t * KT + unit / CPR;
          if (key >= len && key < keys) {
            u32x4* at16 = reinterpret_cast<u32x4*>(tv + unit * 16);
            u32x4 x = *at16;
            bool any = false;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t lo = E::wild(x[i]) ? 0xFFFFu : 0, hi = E::wild(x[i] >> 16) ? ~0xFFFFu : 0;
              any = any || lo || hi;
              x[i] &= ~(lo | hi);
            }
            if (any) *at16 = x;
            mine = mine || any;
          }
        }
        wild |= __syncthreads_or(mine);
      }
      if (wave_ok) {
        // Fragments are read ahead of the products that take them, 8 at a time
        // (the barriers keep the compiler from pulling each read down to its
        // use, where its latency would show).
        f32x16 s[NB];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          s[nb] = f32x16{0};
#pragma unroll
          for (int k8 = 0; k8 < DP / 16; k8 += STEP) {
            s16x8 kf[STEP];
#pragma unroll
            for (int i = 0; i < STEP; ++i)
              kf[i] = *reinterpret_cast<__attribute__((address_space(3))) const s16x8*>(
                  ((stage + k_off) ^ ((k8 + i) * 32)) + nb * 32 * (DP * 2));
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < STEP; ++i) s[nb] = E::mfma(kf[i], qf[k8 + i], s[nb]);
          }
        }
        // V^T of a half block of keys: columns d of this lane, keys in the order
        // of the scores
        s16x8 vf[2][STEP / 2];
        auto read_v = [&](int half_block, int db0, s16x8* to) {
#pragma unroll
          for (int i = 0; i < STEP / 2; ++i) {
            const uint32_t at = (stage + v_off) ^ ((db0 + i) * 64);
            const uint32_t rows = half_block * 16 * (DP * 2);
            const s16x4 x0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (__attribute__((address_space(3))) s16x4*)(at + rows));
            const s16x4 x1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (__attribute__((address_space(3))) s16x4*)((at ^ 32) + rows + 8 * (DP * 2)));
            to[i] = __builtin_shufflevector(x0, x1, 0, 1, 2, 3, 4, 5, 6, 7);
          }
        };
        read_v(0, 0, vf[0]);
        __builtin_amdgcn_sched_barrier(0);
        const int key0 = t * KT + kw * KB + 4 * half;
        if (t * KT + KT > len) {
          const uint64_t see = window(see0, see1, key0 - len);
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const uint32_t bit = uint32_t(see >> (nb * 32)) & (1u << (8 * (i / 4) + i % 4));
              s[nb][i] = bit ? s[nb][i] : -INFINITY;
            }
        }
        float top = -INFINITY;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int i = 0; i < 16; ++i) top = fmaxf(top, s[nb][i]);
        top *= a.scale_log2;
        top = fmaxf(top, __shfl_xor(top, 32));
        if (__any(top > m)) {
          const float to = fmaxf(m, top);
          const float f = to == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m - to);
          l *= f;
#pragma unroll
          for (int i = 0; i < ND; ++i) acc[i] *= f;
          m = to;
        }
        const float ref = m == -INFINITY ? 0.0f : m;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            s[nb][i] = __builtin_amdgcn_exp2f(fmaf(s[nb][i], a.scale_log2, -ref));
            l += s[nb][i];
          }
        // V is read one step (a half block of keys, STEP / 2 blocks of columns)
        // ahead of its products
        constexpr int PER = ND / (STEP / 2), STEPS = 2 * NB * PER;
#pragma unroll
        for (int st = 0; st < STEPS; ++st) {
          const int hb = st / PER, db0 = st % PER * (STEP / 2);
          if (st + 1 < STEPS) read_v((st + 1) / PER, (st + 1) % PER * (STEP / 2), vf[(st + 1) % 2]);
          typename E::vec pf;
#pragma unroll
          for (int j = 0; j < 8; ++j) pf[j] = elem(s[hb / 2][8 * (hb % 2) + j]);
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int i = 0; i < STEP / 2; ++i)
            acc[db0 + i] = E::mfma(vf[st % 2][i], pf, acc[db0 + i]);
        }
      }
    }
    __syncthreads();
    l += __shfl_xor(l, 32);

    if constexpr (KW > 1) {
      // the wavefronts along the keys join in LDS
      if (half == 0) {
        merge_ml[kw][rw][0][col] = m;
        merge_ml[kw][rw][1][col] = l;
      }
      float* const box = reinterpret_cast<float*>(tile);
      if (kw > 0) {
        float* o = box + ((kw - 1) * RW + rw) * (ND * 16 * 64);
#pragma unroll
        for (int i = 0; i < ND; ++i)
#pragma unroll
          for (int j = 0; j < 16; ++j) o[(i * 16 + j) * 64 + lane] = acc[i][j];
      }
      __syncthreads();
      if (kw == 0) {
        float to = m;
#pragma unroll
        for (int k = 1; k < KW; ++k) to = fmaxf(to, merge_ml[k][rw][0][col]);
        const float ref = to == -INFINITY ? 0.0f : to;
        float f = __builtin_amdgcn_exp2f(m - ref);
        l *= f;
#pragma unroll
        for (int i = 0; i < ND; ++i) acc[i] *= f;
#pragma unroll
        for (int k = 1; k < KW; ++k) {
          f = __builtin_amdgcn_exp2f(merge_ml[k][rw][0][col] - ref);
          l += f * merge_ml[k][rw][1][col];
          const float* o = box + ((k - 1) * RW + rw) * (ND * 16 * 64);
#pragma unroll
          for (int i = 0; i < ND; ++i)
#pragma unroll
            for (int j = 0; j < 16; ++j) acc[i][j] = fmaf(f, o[(i * 16 + j) * 64 + lane], acc[i][j]);
        }
        m = to;
      }
      __syncthreads();
    }

    if (wild && kw == 0) {
      // The wild values of the nodes among this share's keys, for the rows that
      // see them (rare, so scores are simply taken again).
      for (int x = max(t0 * KT - len, 0); x < min(t1 * KT - len, n); ++x) {
        const bool see = row_ok && ((x < 64 ? see0 >> (x & 63) : see1 >> (x & 63)) & 1);
        const char* kp = a.k_tree + (rq.first + x) * a.n_t + h * a.n_h;
        const elem* kx = reinterpret_cast<const elem*>(kp);
        const elem* qx = reinterpret_cast<const elem*>(a.q + (rq.first + node) * a.q_t + hq * a.q_h);
        const uint16_t* vx = reinterpret_cast<const uint16_t*>(kp + a.v_tree);
        float dot = 0.0f;
#pragma unroll 1
        for (int d = 0; d < a.D; ++d) dot = fmaf(float(qx[d]), float(kx[d]), dot);
        // a weight that underflows is still one
        const float px = fmaxf(__builtin_amdgcn_exp2f(fmaf(dot, a.scale_log2, -m)), 1e-30f);
#pragma unroll
        for (int i = 0; i < ND; ++i)
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const int d = i * 32 + 8 * (j / 4) + 4 * half + j % 4;
            const uint16_t raw = d < a.D ? vx[d] : 0;
            const float sum = fmaf(px, float(__builtin_bit_cast(elem, raw)), acc[i][j]);
            acc[i][j] = see & E::wild(raw) ? sum : acc[i][j];
            __builtin_amdgcn_sched_barrier(0);  // few registers rather than many loads at once
          }
      }
    }

    if (kw == 0 && row_ok) {
      if (t0 == 0 && t1 == rq.tiles) {
        const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
        char* op = a.out + (rq.first + node) * a.o_t + hq * a.o_h;
#pragma unroll
        for (int i = 0; i < ND; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int d = i * 32 + 8 * j + 4 * half;
            if (d < a.D) {
              typedef elem e4 __attribute__((ext_vector_type(4)));
              e4 x;
#pragma unroll
              for (int k = 0; k < 4; ++k) x[k] = elem(acc[i][4 * j + k] * inv);
              *reinterpret_cast<e4*>(op + d * 2) = x;
            }
          }
        if (a.lse && half == 0)
          a.lse[(rq.first + node) * a.Hq + hq] =
              l > 0.0f || l != l ? (m + __builtin_amdgcn_logf(l)) * kLn2 : -INFINITY;
      } else {
        // a share of the keys: slot 0 of the worker if it began inside the
        // item (its first), slot 1 if it ends inside (its last)
        float* p = a.part + ((w * 2 + (t0 > 0 ? 0 : 1)) * M + rw * 32 + col) * int64_t(DP + 2);
#pragma unroll
        for (int i = 0; i < ND; ++i)
#pragma unroll
          for (int j = 0; j < 16; ++j) p[i * 32 + 8 * (j / 4) + 4 * half + j % 4] = acc[i][j];
        if (half == 0) {
          p[DP] = m;
          p[DP + 1] = l;
        }
      }
    }
    // Loads are counted in order among themselves only: no store stays behind.
    asm volatile("s_waitcnt vmcnt(0)" : : : "memory");
    at += t1 - t0;
  }
}

// Joins the shares of items that several workers had: a wavefront per row
// (node, query head); rows of whole items end at once.
template <int DT>
__global__ __launch_bounds__(256) void join_kernel(AttnArgs a, int workers) {
  using elem = typename Elem<DT>::type;
  const int lane = int(threadIdx.x) & 63;
  const int64_t row = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 6);
  if (row >= a.T * a.Hq) return;
  const int64_t i = row / a.Hq;
  const int hq = int(row - i * a.Hq);
  // the request of row i (node_start ascends where it is right)
  int64_t lo = 0, hi = a.B;
  while (hi - lo > 1) {
    const int64_t mid = (lo + hi) / 2;
    if (a.node_start[mid] <= i) lo = mid;
    else hi = mid;
  }
  const Req rq = request(a, lo);
  if (i < rq.first || i >= rq.first + rq.n) return;
  const int64_t total = a.first_tile[a.B];
  const int h = hq / a.G;
  const int r = int(i - rq.first) * a.G + hq - h * a.G;
  const int rt = r / a.tile_rows;
  const int64_t t0 = a.first_tile[lo] + (int64_t(h) * rq.row_tiles + rt) * rq.tiles;
  const int64_t w0 = worker_of(total, workers, t0);
  const int64_t w1 = worker_of(total, workers, t0 + rq.tiles - 1);
  if (w0 == w1) return;
  const int64_t step = int64_t(a.tile_rows) * (a.width + 2);
  const float* p = a.part + int64_t(r % a.tile_rows) * (a.width + 2);
  // w0's share is its last segment when it starts in front of the item or at it
  auto at = [&](int64_t w) { return p + (w * 2 + (w == w0 ? 1 : 0)) * step; };
  float m = -INFINITY;
  for (int64_t w = w0 + lane; w <= w1; w += 64) m = fmaxf(m, at(w)[a.width]);
  for (int d = 32; d >= 1; d /= 2) m = fmaxf(m, __shfl_xor(m, d));
  const float ref = m == -INFINITY ? 0.0f : m;
  float l = 0.0f, x[4] = {0, 0, 0, 0};
  const int d0 = lane * 4;
  for (int64_t w = w0; w <= w1; ++w) {
    const float* o = at(w);
    const float f = __builtin_amdgcn_exp2f(o[a.width] - ref);
    l = fmaf(f, o[a.width + 1], l);
    if (d0 < a.D)
      for (int k = 0; k < 4; ++k) x[k] = fmaf(f, o[d0 + k], x[k]);
  }
  const bool some = l > 0.0f || l != l;
  const float inv = some ? 1.0f / l : 0.0f;
  if (d0 < a.D) {
    elem* op = reinterpret_cast<elem*>(a.out + i * a.o_t + hq * a.o_h);
    for (int k = 0; k < 4; ++k) op[d0 + k] = elem(x[k] * inv);
  }
  if (a.lse && lane == 0) a.lse[row] = some ? (m + __builtin_amdgcn_logf(l)) * kLn2 : -INFINITY;
}

// Which kernel: rows of the largest tree in wavefronts of 32 rows, and the rest
// of a workgroup along the keys.
struct Variant {
  int rw, kw, kb, width, workers;
};
Variant variant_of(int64_t rows, int64_t D) {
  Variant v;
  v.width = D <= 64 ? 64 : D <= 128 ? 128 : 256;
  v.rw = rows <= 32 ? 1 : rows <= 64 ? 2 : rows <= 128 || v.width == 256 ? 4 : 8;
  if (v.width == 256) {
    v.kw = v.rw == 1 ? 2 : v.rw == 2 ? 2 : 1;
    v.kb = 32;
  } else {
    v.kw = v.rw == 1 ? 4 : 8 / v.rw;
    v.kb = v.rw == 8 ? 64 : 32;
  }
  v.workers = 256;
  return v;
}

template <int DT, int DP, int RW, int KW, int KB, int S>
void launch_one(const Variant& v, const AttnArgs& a, hipStream_t st) {
  hipLaunchKernelGGL((attention_kernel<DT, DP, RW, KW, KB, S>), dim3(unsigned(v.workers)),
                     dim3(64 * RW * KW), 0, st, a);
}

template <int DT, int DP>
void launch(const Variant& v, const AttnArgs& a, hipStream_t st) {
  if constexpr (DP == 256) {
    if (v.rw == 1) launch_one<DT, DP, 1, 2, 32, 2>(v, a, st);
    else if (v.rw == 2) launch_one<DT, DP, 2, 2, 32, 2>(v, a, st);
    else launch_one<DT, DP, 4, 1, 32, 4>(v, a, st);
  } else {
    constexpr int X = 128 / DP;  // stages of half the size, twice as many
    if (v.rw == 1) launch_one<DT, DP, 1, 4, 32, 2 * X>(v, a, st);
    else if (v.rw == 2) launch_one<DT, DP, 2, 4, 32, 2 * X>(v, a, st);
    else if (v.rw == 4) launch_one<DT, DP, 4, 2, 32, 4>(v, a, st);
    else launch_one<DT, DP, 8, 1, 64, 4>(v, a, st);
  }
}

template <int DT>
void launch_width(const Variant& v, const AttnArgs& a, hipStream_t st) {
  if (v.width == 64) launch<DT, 64>(v, a, st);
  else if (v.width == 128) launch<DT, 128>(v, a, st);
  else launch<DT, 256>(v, a, st);
  const int64_t rows = a.T * a.Hq;
  hipLaunchKernelGGL((join_kernel<DT>), dim3(unsigned((rows + 3) / 4)), dim3(256), 0, st, a,
                     v.workers);
}

bool sizes_ok(int64_t B, int64_t T, int64_t Hq, int64_t Hkv, int64_t D, int64_t max_nodes) {
  const int64_t k31 = int64_t(1) << 31;
  return B >= 1 && B < k31 && T >= 0 && T < k31 && Hq >= 1 && Hkv >= 1 && Hq < k31 && Hkv < k31 &&
         Hq % Hkv == 0 && D >= 8 && D <= SV_MAX_HEAD_DIM && D % 8 == 0 && max_nodes >= 1 &&
         max_nodes <= SV_MAX_TREE_NODES && max_nodes * (Hq / Hkv) <= (1 << 16) &&
         B * Hkv <= (1 << 24) && T * Hq < k31;
}

}  // namespace

extern "C" {

size_t specverify_tree_attention_workspace_size(int64_t B, int64_t T, int64_t Hq, int64_t Hkv,
                                                int64_t D, int64_t max_nodes) {
  if (!sizes_ok(B, T, Hq, Hkv, D, max_nodes)) return 0;
  const Variant v = variant_of(max_nodes * (Hq / Hkv), D);
  return align256(size_t(B + 1) * 8) +
         align256(size_t(v.workers) * 2 * (32 * v.rw) * (v.width + 2) * sizeof(float));
}

int specverify_tree_attention(
    const void* q, const void* k_tree, const void* v_tree, const void* k_cache,
    const void* v_cache, int dtype, int64_t B, int64_t T, int64_t Hq, int64_t Hkv, int64_t D,
    int64_t max_nodes, int64_t q_stride_t, int64_t q_stride_h, int64_t n_stride_t,
    int64_t n_stride_h, int64_t c_stride_page, int64_t c_stride_token, int64_t c_stride_h,
    int64_t num_pages, int64_t page_size, const int32_t* block_table, int64_t max_pages,
    int64_t table_stride, const int32_t* prefix_len, const int32_t* node_start,
    const uint64_t* ancestors, float scale, void* out, int64_t o_stride_t, int64_t o_stride_h,
    float* lse, int32_t* device_error, void* workspace, size_t workspace_bytes, void* stream) {
  if (!k_cache || !v_cache || !block_table || !prefix_len || !node_start) return SV_EINVAL;
  if (T > 0 && (!q || !k_tree || !v_tree || !out)) return SV_EINVAL;
  if (!sizes_ok(B, T, Hq, Hkv, D, max_nodes)) return SV_EINVAL;
  const int64_t k31 = int64_t(1) << 31;
  if (!pow2(page_size) || page_size >= k31 || max_pages < 1 || max_pages >= k31 ||
      max_pages * page_size + max_nodes > k31 - (1 << 12) || num_pages < 1 || num_pages >= k31 ||
      table_stride < max_pages)
    return SV_EINVAL;
  const int64_t strides[] = {q_stride_t, q_stride_h, n_stride_t, n_stride_h, c_stride_page,
                             c_stride_token, c_stride_h, o_stride_t, o_stride_h};
  for (int64_t s : strides)
    if (s < 0) return SV_EINVAL;
  if (!(scale > 0.0f) || !std::isfinite(scale)) return SV_EINVAL;
  if (dtype != SV_BF16 && dtype != SV_F16) return SV_EDTYPE;
  for (int64_t s : strides)
    if (s % 8 != 0) return SV_EALIGN;
  if (!aligned16(q) || !aligned16(k_tree) || !aligned16(v_tree) || !aligned16(k_cache) ||
      !aligned16(v_cache) || !aligned16(out))
    return SV_EALIGN;
  int status = SV_OK;
  if (!workspace_ok(workspace, workspace_bytes,
                    specverify_tree_attention_workspace_size(B, T, Hq, Hkv, D, max_nodes),
                    &status))
    return status;
  if (T == 0) return SV_OK;
  const Variant v = variant_of(max_nodes * (Hq / Hkv), D);
  AttnArgs a{};
  a.q = static_cast<const char*>(q);
  a.k_tree = static_cast<const char*>(k_tree);
  a.k_cache = static_cast<const char*>(k_cache);
  a.v_tree = static_cast<const char*>(v_tree) - a.k_tree;
  a.v_cache = static_cast<const char*>(v_cache) - a.k_cache;
  a.q_t = q_stride_t * 2;
  a.q_h = q_stride_h * 2;
  a.n_t = n_stride_t * 2;
  a.n_h = n_stride_h * 2;
  a.c_page = c_stride_page * 2;
  a.c_token = c_stride_token * 2;
  a.c_h = c_stride_h * 2;
  a.o_t = o_stride_t * 2;
  a.o_h = o_stride_h * 2;
  a.table = block_table;
  a.prefix_len = prefix_len;
  a.node_start = node_start;
  a.anc = ancestors;
  a.out = static_cast<char*>(out);
  a.lse = lse;
  a.err = device_error;
  a.B = B;
  a.T = T;
  a.table_stride = table_stride;
  a.num_pages = num_pages;
  a.max_keys = max_pages * page_size;
  a.Hq = int(Hq);
  a.Hkv = int(Hkv);
  a.G = int(Hq / Hkv);
  a.D = int(D);
  a.max_nodes = int(max_nodes);
  a.words = int((max_nodes + 63) / 64);
  a.page_shift = log2_of(page_size);
  a.scale_log2 = scale * kLog2e;
  a.first_tile = static_cast<int64_t*>(workspace);
  a.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + align256(size_t(B + 1) * 8));
  a.tile_keys = v.kw * v.kb;
  a.tile_rows = 32 * v.rw;
  a.width = v.width;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  if (dtype == SV_BF16) launch_width<SV_BF16>(v, a, st);
  else launch_width<SV_F16>(v, a, st);
  return launch_status();
}

}  // extern "C"
