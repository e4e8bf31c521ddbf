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
//
// What bounds it, heads of 128 in bf16: for few rows memory, with a ring of tiles
// in LDS kept full over the ends of items (64 single tokens over 1000 to 16000 keys
// 407 us, 5.5 TB/s; 64 chains of 9 over 301 to 8011 keys 231 us, 4.8 TB/s); for
// many rows each wavefront's own chain of fetches, LDS reads, products and
// exponentials (16 trees of 64 nodes, 256 rows an item: 197 us, 3.0 TB/s and 0.56
// PFLOP/s; per 64 keys fetch 0.6 us, K Q 0.5, softmax 0.4, P V 0.64, barrier 0.6);
// for a few hundred keys latency (one token over 100 keys, one tile, 12 us; over
// 500 keys, four tiles, 17.5 us: 10 us whatever the keys, 1.8 us a tile).

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
  struct Split* split;  // [workers], and all tiles in one more's start
  float* part;          // [workers * 2][M][DP + 4]: sums, then m and l
  int tile_keys, tile_rows, whole;
};

// An item (request, key head, row tile) that a worker began inside of: its tiles
// count from `start` in the order of all tiles.
struct Split {
  int64_t start, first;  // first: the request's first row
  int32_t tiles;         // 0: none
  int32_t h, row0, rows; // rows of the item, from row0 on, of `rows` in all
};

__device__ const u32x4 zero_piece = {0, 0, 0, 0};

// Tiles of request b, and its sizes.
struct Req {
  int64_t first;
  int32_t n, len, tiles, row_tiles;
};
__device__ __forceinline__ Req request(const AttnArgs& a, int64_t b, int* bits = nullptr) {
  Req r;
  const Nodes nd = nodes_of(a.node_start, b, a.T, a.max_nodes);
  r.first = nd.first;
  r.n = nd.n < 0 ? 0 : nd.n;
  const int64_t len = a.prefix_len[b];
  r.len = int32_t(len < 0 ? 0 : len > a.max_keys ? a.max_keys : len);
  if (bits) *bits |= (nd.n < 0 ? SV_ERR_TREE : 0) | (r.len != len ? SV_ERR_LENGTH : 0);
  r.tiles = (r.len + r.n + a.tile_keys - 1) / a.tile_keys;
  r.row_tiles = (r.n * a.G + a.tile_rows - 1) / a.tile_rows;
  return r;
}
// The kernel's arguments where they are seldom used: read again at each such
// place, or some hundred of them would be held in scalar registers throughout
// and push out what the loop over the tiles uses. (The pointer to them is taken
// once, in the kernel: elsewhere there is none.)
typedef const __attribute__((address_space(4))) AttnArgs* Args;
__device__ __forceinline__ Args again(Args p) {
  asm volatile("" : "+s"(p));
  return p;
}

// The same for an index that the whole workgroup has: by scalar loads.
template <typename T>
__device__ __forceinline__ const __attribute__((address_space(4))) T* constant(const T* p) {
  return reinterpret_cast<const __attribute__((address_space(4))) T*>(
      reinterpret_cast<uintptr_t>(p));
}
__device__ __forceinline__ Req uniform_request(Args a, int64_t b) {
  const auto* start = constant(a->node_start) + b;
  const int64_t lo = start[0], hi = start[1], len = constant(a->prefix_len)[b];
  const bool good = lo >= 0 && hi >= lo && hi <= a->T && hi - lo <= a->max_nodes;
  Req r;
  r.first = good ? lo : 0;
  r.n = good ? int32_t(hi - lo) : 0;
  r.len = int32_t(len < 0 ? 0 : len > a->max_keys ? a->max_keys : len);
  r.tiles = (r.len + r.n + a->tile_keys - 1) / a->tile_keys;
  r.row_tiles = (r.n * a->G + a->tile_rows - 1) / a->tile_rows;
  return r;
}
// Work is shared out in places: an item (request, key head, row tile) takes one
// for each of its tiles and kItemPlaces more for what it costs besides (rows
// loaded, wavefronts joined, results written).
// Where no request can have many tiles and every item has a worker, items are not
// split (`whole`): one place each, and nothing to join (calls, both sides timed
// together: 32 requests of up to 600 tokens 24 us so, 30 us split; one token over
// 500 keys 20 and 22 us; 256 requests, with 8 items a worker, 170 us so, 147 us
// split).
constexpr int kWorkers = 256;  // one to a CU
constexpr int kItemPlaces = 3;
constexpr int kWholeTiles = 6;
__device__ __forceinline__ int item_places(int whole, int tiles) {
  return whole ? 1 : tiles + kItemPlaces;
}
__device__ __forceinline__ int64_t places_of(int whole, int heads, const Req& r) {
  return int64_t(item_places(whole, r.tiles)) * r.row_tiles * heads;
}

__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ int64_t uniform(int64_t x) {
  return int64_t(uint64_t(uint32_t(uniform(int(x >> 32)))) << 32 | uint32_t(uniform(int(x))));
}

// Worker w's share of `total` tiles starts here.
__device__ __forceinline__ int64_t share_start(int64_t total, int workers, int64_t w) {
  const int64_t q = total / workers, rem = total % workers;
  return w * q + (w < rem ? w : rem);
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
               : "s"(__builtin_amdgcn_readfirstlane(to)), "v"(from)
               : "memory", "m0");
}

__device__ __forceinline__ void load_lds4(const int32_t* from, uint32_t to) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off"
               :
               : "s"(__builtin_amdgcn_readfirstlane(to)), "v"(from)
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

__device__ __forceinline__ void meet() {
  asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" : : : "memory");
}

// Where the fetching side stands among the items.
struct Cursor {
  int64_t at, b, b_first;  // the next place, its request, that one's first place
  Req rq;
};

// A share of an item's tiles, prepared while the one before is fetched.
struct Seg {
  int64_t start, first;
  int64_t head, node, table;  // the request's keys of this head, its nodes', its pages
  int32_t n, len, h, rt, t0, t1, tiles;
};

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
  // blocks of 32 columns that the wavefronts along the keys join at a time
  constexpr int BOX = (KW > 1 ? KW - 1 : 1) * RW * 16 * 64 * 4;
  constexpr int JOIN = STAGE / BOX < ND ? STAGE / BOX : ND;
  static_assert(KW == 1 || (JOIN >= 1 && ND % JOIN == 0), "the join fits a stage");
  __shared__ __align__(1024) char tile[S * STAGE];
  __shared__ float merge_ml[KW][RW][2][32];
  __shared__ int64_t scan[NT / 64];
  __shared__ Seg segs[S + 2];
  __shared__ Cursor cursors[2];
  __shared__ int32_t id_box[NT / 64][2][64];
  __shared__ int wild_seg;
  const Args args = (Args)__builtin_amdgcn_kernarg_segment_ptr();
  const int tid = int(threadIdx.x), lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int rw = wv % RW, kw = wv / RW;
  const int col = lane & 31, half = lane >> 5;

  // This worker's share: neighbours in the order of tiles share an XCD's L2
  // (workgroups go round robin over the 8 XCDs).
  const int workers = int(gridDim.x);
  const int64_t w = workers % 8 == 0 ? (blockIdx.x % 8) * (workers / 8) + blockIdx.x / 8
                                     : blockIdx.x;
  if (tid == 0) {
    a.split[w].tiles = 0;
    wild_seg = -1;
  }
  // All tiles, and those in front of this thread's request (of the last round).
  int64_t total = 0, mine = 0, lo = 0;
  Req own{};
  for (int64_t o = 0; o < a.B; o += NT) {
    int bits = 0;
    if (o + tid < a.B) own = request(a, o + tid, &bits);
    mine = o + tid < a.B ? places_of(a.whole, a.Hkv, own) : 0;
    if (w == 0 && bits) set_error(a.err, bits);
    int64_t s = mine;
    for (int d = 1; d < 64; d *= 2) {
      const int64_t y = __shfl_up(s, d);
      if (lane >= d) s += y;
    }
    if (o) __syncthreads();
    if (lane == 63) scan[wv] = s;
    __syncthreads();
    lo = total + s - mine;
    for (int k = 0; k < NT / 64; ++k) {
      if (k < wv) lo += scan[k];
      total += scan[k];
    }
  }
  const int64_t at = uniform(share_start(total, workers, w));
  const int64_t end = uniform(share_start(total, workers, w + 1));
  if (!sv_ok(workers == kWorkers && w < workers && at <= end && end <= total)) return;
  if (w == 0 && tid == 0) a.split[workers].start = total;
  if (at >= end) return;
  // the request that holds tile `at`: more than NT of them are gone through again
  int64_t base = 0;
  for (int64_t o = 0; o < a.B; o += NT) {
    if (a.B > NT) {
      if (o + tid < a.B) own = request(a, o + tid);
      mine = o + tid < a.B ? places_of(a.whole, a.Hkv, own) : 0;
      int64_t s = mine;
      for (int d = 1; d < 64; d *= 2) {
        const int64_t y = __shfl_up(s, d);
        if (lane >= d) s += y;
      }
      __syncthreads();
      if (lane == 63) scan[wv] = s;
      __syncthreads();
      lo = base + s - mine;
      for (int k = 0; k < NT / 64; ++k) {
        if (k < wv) lo += scan[k];
        base += scan[k];
      }
    }
    if (at >= lo && at < lo + mine) cursors[0] = Cursor{at, o + tid, lo, own};
    if (base > at) break;
  }
  __syncthreads();

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
  // ---- the fetching side: S - 1 tiles ahead, over the ends of items
  int f_t = 0, f_t1 = 0, f_len = 0, f_keys = 0, f_batch = 0, f_tiles = S;
  int prepared = 0, f_seg = 0;  // shares prepared, the next one to fetch
  int turn = 0;                 // which cursor holds
  bool more = true;
  const char *f_head = nullptr, *f_node = nullptr;
  const int32_t* f_table = nullptr;
  const char* const zero = reinterpret_cast<const char*>(&zero_piece);
  const int64_t c_page = a.c_page, c_token = a.c_token, v_cache = a.v_cache;
  const int in_page = (1 << a.page_shift) - 1, page_shift = a.page_shift;
  const uint32_t num_pages = uint32_t(a.num_pages);
  const bool full = DP == a.D;
  constexpr int WROWS = 64 / CPR;  // rows of a wavefront's load
  // The pieces of a row come in the same order for every round of 16 rows and
  // more, so a lane's part of the addresses is one offset.
  constexpr bool SAME = NT / CPR % 16 == 0;
  const int lane_row = lane / CPR;
  // The rows of a wavefront's load lie in one page, so its page ids are UNITS a
  // tile. A register holds those of BATCH tiles, one a lane; the next BATCH (box
  // 0) and the first of the next share (box 1) are on their way to LDS meanwhile.
  const bool one_page = (WROWS >> page_shift) <= 1;
  constexpr int BATCH = 64 / UNITS;
  static_assert(BATCH >= S && UNITS <= 64, "a batch of page ids lands before its use");
  int32_t ids = 0;
  const uint32_t id_at = uniform(int(reinterpret_cast<uintptr_t>(
      (__attribute__((address_space(3))) char*)&id_box[wv][0][0])));
  // this lane's page id in the batch of tiles from t on (the prefix's last at most)
  auto id_place = [&](const int32_t* table, int t, int len) __attribute__((always_inline)) {
    const int key = (t + lane / UNITS) * KT + lane % UNITS * (NT / CPR) + wv * WROWS;
    const int at = (key < len ? key : len - 1) >> page_shift;
    return table + (sv_ok(at >= 0 && at < a.max_keys >> page_shift) ? at : 0);
  };
  auto take_ids = [&](int box) __attribute__((always_inline)) {
    ids = id_box[wv][box][lane];
    asm volatile("s_waitcnt lgkmcnt(0)" : "+v"(ids) : : "memory");
  };

  // Finds the next share of this worker, with its first page ids on their way.
  auto prepare = [&]() __attribute__((always_inline)) {
    const Args s = again(args);
    const Cursor& cursor = cursors[turn];
    int64_t at = uniform(cursor.at), b = uniform(cursor.b), b_first = uniform(cursor.b_first);
    Req rq{uniform(cursor.rq.first), uniform(cursor.rq.n), uniform(cursor.rq.len),
           uniform(cursor.rq.tiles), uniform(cursor.rq.row_tiles)};
    Seg sg;
    do {
      if (at >= end) {
        more = false;
        return;
      }
      while (at >= b_first + places_of(s->whole, s->Hkv, rq)) {
        b_first += places_of(s->whole, s->Hkv, rq);
        rq = uniform_request(s, ++b);
      }
      const int64_t into = at - b_first;
      const int size = item_places(s->whole, rq.tiles);
      const int item = int(into / size);  // (key head, row tile)
      const int p0 = int(into - int64_t(item) * size);
      const int p1 = int(size - p0 < end - at ? size : p0 + (end - at));
      sg.start = at - p0;
      sg.t0 = min(p0, rq.tiles);
      sg.t1 = s->whole ? rq.tiles : min(p1, rq.tiles);
      sg.h = item / rq.row_tiles;
      sg.rt = item - sg.h * rq.row_tiles;
      at += p1 - p0;
    } while (sg.t0 == sg.t1);
    if (!sv_ok(b < s->B && sg.h >= 0 && sg.h < s->Hkv && sg.rt < rq.row_tiles && sg.t0 < sg.t1 &&
               sg.t1 <= rq.tiles && rq.first + rq.n <= s->T)) {
      more = false;
      return;
    }
    sg.first = rq.first;
    sg.n = rq.n;
    sg.len = rq.len;
    sg.tiles = rq.tiles;
    sg.head = int64_t(s->k_cache + sg.h * s->c_h);
    sg.node = int64_t(s->k_tree + rq.first * s->n_t + sg.h * s->n_h);
    const int32_t* table = s->table + b * s->table_stride;
    sg.table = int64_t(table);
    if (one_page && rq.len > 0) load_lds4(id_place(table, sg.t0, rq.len), id_at + 256);
    turn ^= 1;
    if (tid == 0) {
      segs[prepared % (S + 2)] = sg;
      cursors[turn] = Cursor{at, b, b_first, rq};
    }
    ++prepared;
  };
  // Starts the next tile's keys and values on their way into a stage; false when
  // the share is at its end.
  auto fetch_next = [&](int to_stage) __attribute__((always_inline)) {
    const bool fresh = f_t == f_t1;
    if (fresh) {
      if (!more) return false;
      const Seg& sg = segs[f_seg % (S + 2)];
      ++f_seg;
      f_t = uniform(sg.t0);
      f_t1 = uniform(sg.t1);
      f_len = uniform(sg.len);
      f_keys = f_len + uniform(sg.n);
      f_head = reinterpret_cast<const char*>(uniform(sg.head));
      f_node = reinterpret_cast<const char*>(uniform(sg.node));
      f_table = reinterpret_cast<const int32_t*>(uniform(sg.table));
      f_batch = f_t;
      if (one_page && f_len > 0) {
        // its ids are older than the tiles of the share before but the first
        if (f_tiles < S) asm volatile("s_waitcnt vmcnt(0)" : : : "memory");
        take_ids(1);
        if (f_t + BATCH < f_t1) load_lds4(id_place(f_table, f_t + BATCH, f_len), id_at);
      }
      f_tiles = f_t1 - f_t;
    }
    const int t = f_t++;
    if (!sv_ok(to_stage < S && t * KT < f_keys && f_seg <= prepared)) return false;
    const uint32_t stage = tile_at + uint32_t(to_stage) * STAGE + wv * 1024;
    if (t - f_batch == BATCH) {
      f_batch = t;
      if (one_page && f_len > 0) {
        take_ids(0);
        if (t + BATCH < f_t1) load_lds4(id_place(f_table, t + BATCH, f_len), id_at);
      }
    }
    const int id0 = (t - f_batch) * UNITS;
    bool quick = one_page && t * KT + KT <= f_len;
    if (quick) {
      const bool here = lane >= id0 && lane < id0 + UNITS;
      quick = !__any(here && uint32_t(ids) >= num_pages);
    }
    if (quick) {
#pragma unroll
      for (int u = 0; u < UNITS; ++u) {
        const int row0 = u * (NT / CPR) + wv * WROWS;
        const int c = (lane % CPR) ^ swizzle<CPR>(SAME ? wv * WROWS + lane_row : row0 + lane_row);
        const char* base =
            f_head + uint32_t(__builtin_amdgcn_readlane(ids, id0 + u)) * uint64_t(c_page) +
            uint32_t((t * KT + row0) & in_page) * uint64_t(c_token);
        const char* kp = base + (lane_row * c_token + c * 16);
        const char* vp = kp + v_cache;
        if (!full) {
          const bool some = c * 8 < a.D;
          kp = some ? kp : zero;
          vp = some ? vp : zero;
        }
        load_lds16(kp, stage + u * NT * 16);
        load_lds16(vp, stage + u * NT * 16 + KT * DP * 2);
      }
    } else {
      // the end of the prefix, the tree's nodes, pages of fewer rows than a
      // wavefront loads, bad pages: lane by lane
      const Args s = again(args);
      int32_t page[UNITS];
#pragma unroll
      for (int u = 0; u < UNITS; ++u) {
        const int key = t * KT + u * (NT / CPR) + wv * WROWS + lane_row;
        page[u] = -1;
        if (one_page) page[u] = __builtin_amdgcn_readlane(ids, id0 + u);
        else if (f_len > 0) page[u] = f_table[(key < f_len ? key : f_len - 1) >> page_shift];
      }
#pragma unroll
      for (int u = 0; u < UNITS; ++u) {
        const int row = u * (NT / CPR) + wv * WROWS + lane_row;
        const int c = (lane % CPR) ^ swizzle<CPR>(row);
        const int key = t * KT + row;
        const char* cp = f_head + uint32_t(page[u]) * uint64_t(c_page) +
                         uint32_t(key & in_page) * uint64_t(c_token);
        const char* np = f_node + int64_t(key - f_len) * s->n_t;
        const bool cached = key < f_len, good = uint32_t(page[u]) < num_pages;
        const bool some = c * 8 < s->D && (cached ? good : key < f_keys);
        if (cached && !good) set_error(s->err, SV_ERR_PAGE);
        const char* kp = (cached ? cp : np) + c * 16;
        const char* vp = kp + (cached ? v_cache : s->v_tree);
        load_lds16(some ? kp : zero, stage + u * NT * 16);
        load_lds16(some ? vp : zero, stage + u * NT * 16 + KT * DP * 2);
      }
    }
    if (fresh) prepare();
    return true;
  };

  // ---- the computing side
  int t = 0, t1 = 0, seg = 0;
  int len = 0, n = 0, keys = 0;
  int hq = 0, node = 0, wild = 0;
  bool row_ok = false, wave_ok = false;
  uint64_t see0 = 0, see1 = 0;
  u32x4 qf[DP / 16];
  f32x16 acc[ND];
  float m = -INFINITY, l = 0.0f;

  // The rows of share `which`: this lane's part of them to registers, and its mask.
  uint64_t next_see0 = 0, next_see1 = 0;
  auto load_rows = [&](int which) __attribute__((always_inline)) {
    const Args s = again(args);
    const Seg& sg = segs[which % (S + 2)];
    const int n = uniform(sg.n), h = uniform(sg.h), row0 = uniform(sg.rt) * M + rw * 32;
    if (row0 >= n * s->G) return;
    const int r = row0 + col < n * s->G ? row0 + col : 0;
    const int node = r / s->G;
    const int64_t i = uniform(sg.first) + node;
    if (!sv_ok(node < n && i < s->T)) return;
    const char* qp = s->q + i * s->q_t + (h * s->G + r - node * s->G) * s->q_h;
#pragma unroll
    for (int k = 0; k < DP / 16; ++k) {
      const int d = 16 * k + 8 * half;
      qf[k] = *reinterpret_cast<const u32x4*>(d < s->D ? qp + d * 2 : zero);
    }
    if (s->anc) {
      const uint64_t* words = s->anc + i * s->words;
      next_see0 = words[0];
      next_see1 = s->words > 1 ? words[1] : 0;
    } else {
      next_see0 = node >= 63 ? ~uint64_t(0) : (uint64_t(2) << node) - 1;
      next_see1 = node < 64 ? 0 : node >= 127 ? ~uint64_t(0) : (uint64_t(2) << (node - 64)) - 1;
    }
  };

  // They are asked for when a share ends, and here before its results are
  // written: where the loop over tiles began with them on their way, the
  // compiler would wait for every load in it.
  auto rows_here = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int k = 0; k < DP / 16; ++k) asm volatile("" : "+v"(qf[k]));
    asm volatile("" : "+v"(next_see0), "+v"(next_see1));
  };

  prepare();
  meet();
  if (more) load_rows(0);
  rows_here();
  asm volatile("s_waitcnt vmcnt(0)" : : : "memory");  // the first page ids
  int fetched = 0, done = 0;
#pragma unroll 1
  for (int i = 0; i < S - 1; ++i) {
    if (fetch_next(i)) ++fetched;
    meet();
  }
  int st_now = 0, st_next = S - 1;  // stages of this tile and of the one to fetch
  for (; done < fetched; ++done) {
    // this tile is here; everyone is done with the one before, whose stage is next
    if (S >= 4 && fetched - done > 2) wait_and_meet<2 * LOADS>();
    else if (S >= 3 && fetched - done > 1) wait_and_meet<LOADS>();
    else wait_and_meet<0>();

    if (t == t1) {
      const Args s = again(args);
      const Seg& sg = segs[seg % (S + 2)];
      t = uniform(sg.t0);
      t1 = uniform(sg.t1);
      len = uniform(sg.len);
      n = uniform(sg.n);
      const int h = uniform(sg.h), rt = uniform(sg.rt);
      keys = len + n;
      ++seg;
      const int r = rt * M + rw * 32 + col;
      row_ok = r < n * s->G;
      node = row_ok ? r / s->G : 0;
      hq = h * s->G + (row_ok ? r - node * s->G : 0);
      wave_ok = rt * M + rw * 32 < n * s->G;
      // bits behind the tree are none of its nodes
      see0 = next_see0 & (n >= 64 ? ~uint64_t(0) : (uint64_t(1) << n) - 1);
      see1 = next_see1 &
             (n >= 128 ? ~uint64_t(0) : n <= 64 ? 0 : (uint64_t(1) << (n - 64)) - 1);
#pragma unroll
      for (int i = 0; i < ND; ++i) acc[i] = f32x16{0};
      m = -INFINITY;
      l = 0.0f;
      wild = 0;
    }
    if (fetch_next(st_next)) ++fetched;
    char* const tv = tile + st_now * STAGE + KT * DP * 2;
    const uint32_t stage = tile_at + uint32_t(st_now) * STAGE;
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
      if (mine) wild_seg = seg;
      meet();
      wild = wild_seg == seg;
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
          for (int i = 0; i < STEP; ++i) s[nb] = E::mfma(kf[i], __builtin_bit_cast(typename E::vec, qf[k8 + i]), s[nb]);
        }
      }
      // V^T of a half block of keys: columns d of this lane, keys in the order
      // of the scores
      s16x8 vf[2][STEP / 2];
      auto read_v = [&](int half_block, int db0, s16x8* to) __attribute__((always_inline)) {
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
        // The weights are rounded to the storage type here, the product's operands
        // being of 16 bits: each is off by at most half a step of it (2^-8 in bf16),
        // an output by that times sum p |v|. Their sum l keeps the float32 ones.
        // A second product for what the rounding takes away would add half to the
        // matrix work of a tile.
        typename E::vec pf;
#pragma unroll
        for (int j = 0; j < 8; ++j) pf[j] = elem(s[hb / 2][8 * (hb % 2) + j]);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < STEP / 2; ++i)
          acc[db0 + i] = E::mfma(vf[st % 2][i], pf, acc[db0 + i]);
      }
    }
    ++t;
    if (t == t1) {
      if (fetched - done > 1) load_rows(seg);
      const Args s = again(args);
      const Seg& sg = segs[(seg - 1) % (S + 2)];
      const int t0 = uniform(sg.t0), h = uniform(sg.h);
      const int64_t first = uniform(sg.first);
      const bool whole = t0 == 0 && t1 == uniform(sg.tiles);
      l += __shfl_xor(l, 32);

      if constexpr (KW > 1) {
        // The wavefronts along the keys join in this tile's stage (the others are
        // being filled), JOIN blocks of columns at a time; each adds up the blocks
        // i with i % KW = kw, and writes those out.
        if (half == 0) {
          merge_ml[kw][rw][0][col] = m;
          merge_ml[kw][rw][1][col] = l;
        }
        float* const box = reinterpret_cast<float*>(tile + st_now * STAGE) + lane;
        float mine = 1.0f, f[KW];
#pragma unroll
        for (int i0 = 0; i0 < ND; i0 += JOIN) {
          meet();
          if (i0 == 0) {
            float to = -INFINITY;
#pragma unroll
            for (int k = 0; k < KW; ++k) to = fmaxf(to, merge_ml[k][rw][0][col]);
            const float ref = to == -INFINITY ? 0.0f : to;
            mine = __builtin_amdgcn_exp2f(m - ref);
            l = 0.0f;
#pragma unroll
            for (int k = 0; k < KW; ++k) {
              f[k] = __builtin_amdgcn_exp2f(merge_ml[k][rw][0][col] - ref);
              l = fmaf(f[k], merge_ml[k][rw][1][col], l);
            }
            m = to;
          }
#pragma unroll
          for (int i = 0; i < JOIN; ++i) {
            const int owner = (i0 + i) % KW;
            if (kw == owner) continue;
            float* o = box + ((i * (KW - 1) + (kw < owner ? kw : kw - 1)) * RW + rw) * (16 * 64);
#pragma unroll
            for (int j = 0; j < 16; ++j) o[j * 64] = acc[i0 + i][j];
          }
          meet();
#pragma unroll
          for (int i = 0; i < JOIN; ++i) {
            const int owner = (i0 + i) % KW;
            if (kw != owner) continue;
            acc[i0 + i] *= mine;
#pragma unroll
            for (int k = 0; k < KW; ++k) {
              if (k == owner) continue;
              const float* o = box + ((i * (KW - 1) + (k < owner ? k : k - 1)) * RW + rw) * (16 * 64);
#pragma unroll
              for (int j = 0; j < 16; ++j) acc[i0 + i][j] = fmaf(f[k], o[j * 64], acc[i0 + i][j]);
            }
          }
        }
      }

      if (wild) {
        // The wild values of the nodes among this share's keys, for the rows that
        // see them (rare, so scores are simply taken again).
        for (int x = max(t0 * KT - len, 0); x < min(t1 * KT - len, n); ++x) {
          const bool see = row_ok && ((x < 64 ? see0 >> (x & 63) : see1 >> (x & 63)) & 1);
          const char* kp = s->k_tree + (first + x) * s->n_t + h * s->n_h;
          const elem* kx = reinterpret_cast<const elem*>(kp);
          const elem* qx =
              reinterpret_cast<const elem*>(s->q + (first + node) * s->q_t + hq * s->q_h);
          const uint16_t* vx = reinterpret_cast<const uint16_t*>(kp + s->v_tree);
          float dot = 0.0f;
#pragma unroll 1
          for (int d = 0; d < s->D; ++d) dot = fmaf(float(qx[d]), float(kx[d]), dot);
          // a weight that underflows is still one
          const float px = fmaxf(__builtin_amdgcn_exp2f(fmaf(dot, s->scale_log2, -m)), 1e-30f);
#pragma unroll
          for (int i = 0; i < ND; ++i)
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const int d = i * 32 + 8 * (j / 4) + 4 * half + j % 4;
              const uint16_t raw = d < s->D ? vx[d] : 0;
              const float sum = fmaf(px, float(__builtin_bit_cast(elem, raw)), acc[i][j]);
              acc[i][j] = (see & E::wild(raw)) ? sum : acc[i][j];
              __builtin_amdgcn_sched_barrier(0);  // few registers rather than many loads at once
            }
        }
      }

      rows_here();
      if (row_ok && sv_ok(first + node < s->T && hq < s->Hq)) {
        if (whole) {
          const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
          char* op = s->out + (first + node) * s->o_t + hq * s->o_h + 8 * half;
#pragma unroll
          for (int i = 0; i < ND; ++i) {
            if (i % KW != kw) continue;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              if (i * 32 + 8 * j >= s->D) continue;  // D is a multiple of 8
              typedef elem e4 __attribute__((ext_vector_type(4)));
              e4 x;
#pragma unroll
              for (int k = 0; k < 4; ++k) x[k] = elem(acc[i][4 * j + k] * inv);
              *reinterpret_cast<e4*>(op + (i * 32 + 8 * j) * 2) = x;
            }
          }
          if (s->lse && half == 0 && kw == 0)
            s->lse[(first + node) * s->Hq + hq] =
                l > 0.0f || l != l ? (m + __builtin_amdgcn_logf(l)) * kLn2 : -INFINITY;
        } else {
          // a share of the keys: slot 0 of the worker if it began inside the
          // item (its first), slot 1 if it ends inside (its last)
          float* p = s->part + ((w * 2 + (t0 > 0 ? 0 : 1)) * M + rw * 32 + col) * int64_t(DP + 4);
#pragma unroll
          for (int i = 0; i < ND; ++i) {
            if (i % KW != kw) continue;
#pragma unroll
            for (int j = 0; j < 4; ++j)
              *reinterpret_cast<f32x4*>(p + i * 32 + 8 * j + 4 * half) =
                  f32x4{acc[i][4 * j], acc[i][4 * j + 1], acc[i][4 * j + 2], acc[i][4 * j + 3]};
          }
          if (half == 0 && kw == 0) {
            p[DP] = m;
            p[DP + 1] = l;
          }
        }
      }
      if (t0 > 0 && tid == 0)
        s->split[w] = Split{sg.start, first, sg.tiles, h, sg.rt * M, n * s->G};
    }
    st_now = st_now + 1 == S ? 0 : st_now + 1;
    st_next = st_next + 1 == S ? 0 : st_next + 1;
  }
}

// Joins the shares of items that several workers had. The worker that comes
// second in an item stands for it; every workgroup counts those items' rows for
// itself, a unit is as many rows as it takes at once (DP / 4 lanes each), and
// units go round robin. Bound by the trips to memory one after another, so AHEAD
// shares are asked for at once: 16 items of 136 rows in 17 shares each 8.2 us, 128
// items of 256 rows (35 MB of shares) 10.8 us. (A workgroup for each possible unit,
// most of them without work, and a share at a time: 16.2 and 15.7 us.)
constexpr int kJoiners = 2048;
template <int DT, int DP>
__global__ __launch_bounds__(kWorkers) void join_kernel(AttnArgs a) {
  using elem = typename Elem<DT>::type;
  constexpr int LANES = DP / 4, ROWS = kWorkers / LANES, AHEAD = 4;
  __shared__ Split item;
  __shared__ int item_second, item_unit, wave_units[kWorkers / kWave];
  const int tid = int(threadIdx.x), lane = tid % kWave;
  const Split own = a.split[tid];
  const int64_t total = a.split[kWorkers].start;
  const bool stands = own.tiles > 0 && share_start(total, kWorkers, tid - 1) <= own.start;
  const int units = stands ? (min(own.rows - own.row0, a.tile_rows) + ROWS - 1) / ROWS : 0;
  int upto = units;
  for (int d = 1; d < kWave; d *= 2) {
    const int y = __shfl_up(upto, d);
    if (lane >= d) upto += y;
  }
  if (lane == kWave - 1) wave_units[tid / kWave] = upto;
  __syncthreads();
  int all = 0;
  for (int k = 0; k < kWorkers / kWave; ++k) {
    if (k < tid / kWave) upto += wave_units[k];
    all += wave_units[k];
  }
  for (int u = int(blockIdx.x); u < all; u += int(gridDim.x)) {
    if (u >= upto - units && u < upto) {
      item = own;
      item_second = tid;
      item_unit = u - (upto - units);
    }
    __syncthreads();
    const Split sp = item;
    const int second = item_second;
    const int in_tile = item_unit * ROWS + tid / LANES, r = sp.row0 + in_tile;
    __syncthreads();
    if (in_tile >= a.tile_rows || r >= sp.rows) continue;
    const int64_t step = int64_t(a.tile_rows) * (DP + 4);
    const float* p = a.part + int64_t(in_tile) * (DP + 4);
    const int d0 = tid % LANES * 4;
    // the first one's share is its last segment, the others' their first
    float m = -INFINITY, l = 0.0f;
    f32x4 x = {0, 0, 0, 0};
    const auto has = [&](int w) {
      return w < kWorkers && share_start(total, kWorkers, w) < sp.start + sp.tiles;
    };
    // an infinite sum stays so however little its share weighs, as within a share
    const auto weighed = [](f32x4 v, float f) {
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = fabsf(v[k]) == INFINITY ? v[k] : v[k] * f;
      return v;
    };
    const auto add = [&](f32x4 y, float mw, float lw) {
      const float to = fmaxf(m, mw), ref = to == -INFINITY ? 0.0f : to;
      const float f = __builtin_amdgcn_exp2f(m - ref), g = __builtin_amdgcn_exp2f(mw - ref);
      l = l * f + lw * g;
      x = weighed(x, f) + weighed(y, g);
      m = to;
    };
    const auto share_of = [&](int w) { return p + (w * 2 + (w < second ? 1 : 0)) * step; };
    int w = second - 1;
    for (; has(w + AHEAD - 1); w += AHEAD) {
      f32x4 y[AHEAD];
      float mw[AHEAD], lw[AHEAD];
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        const float* o = share_of(w + i);
        y[i] = *reinterpret_cast<const f32x4*>(o + d0);
        mw[i] = o[DP];
        lw[i] = o[DP + 1];
      }
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) add(y[i], mw[i], lw[i]);
    }
    for (; has(w); ++w) {
      const float* o = share_of(w);
      add(*reinterpret_cast<const f32x4*>(o + d0), o[DP], o[DP + 1]);
    }
    const int node = r / a.G;
    const int hq = sp.h * a.G + r - node * a.G;
    if (!sv_ok(sp.first + node < a.T && hq < a.Hq && w <= kWorkers)) continue;
    const bool some = l > 0.0f || l != l;
    const float inv = some ? 1.0f / l : 0.0f;
    if (d0 < a.D) {
      typedef elem e4 __attribute__((ext_vector_type(4)));
      e4 y;
      for (int k = 0; k < 4; ++k) y[k] = elem(x[k] * inv);
      *reinterpret_cast<e4*>(a.out + (sp.first + node) * a.o_t + hq * a.o_h + d0 * 2) = y;
    }
    if (a.lse && d0 == 0)
      a.lse[(sp.first + node) * a.Hq + hq] =
          some ? (m + __builtin_amdgcn_logf(l)) * kLn2 : -INFINITY;
  }
}

// Which kernel: rows of the largest tree in wavefronts of 32 rows, and the rest
// of a workgroup along the keys. Fewer rows leave some wavefronts without
// products, more than a workgroup has would read the keys once more.
//   up to 64 rows: 64 single tokens, heads of 64, 224 us, 253 us with the kernel of
//     128 rows (heads of 128 alike, 414 and 408 us; a kernel of 32 rows for them
//     took 416 us)
//   up to 128: 32 trees of 32 nodes 157 us, 165 us with the kernel of 256 rows; 178
//     us with tiles of 64 keys (32 a wavefront), 193 us without wavefronts along
//     the keys; heads of 64: 93 and 113 us
//   more: 16 trees of 64 nodes 222 us, 243 us in two tiles of 128 rows
// Heads wider than 128 (registers for 4 wavefronts): 64 rows 110 us, 125 us with the
// kernel of 128 rows; 16 rows 187 and 200 us, 269 us with one of 32.
// (Each pair was timed together, some before later steps made both sides faster;
// the head of this file has the present times.)
struct Variant {
  int rw, kw, kb, width;
};
Variant variant_of(int64_t rows, int64_t D) {
  Variant v;
  v.width = D <= 64 ? 64 : D <= 128 ? 128 : 256;
  if (v.width == 256) {
    v.rw = rows <= 64 ? 2 : 4;
    v.kw = 4 / v.rw;
    v.kb = 32;
  } else {
    v.rw = rows <= 64 ? 2 : rows <= 128 ? 4 : 8;
    v.kw = 8 / v.rw;
    v.kb = v.rw == 2 ? 32 : 64;
  }
  return v;
}

template <int DT, int DP, int RW, int KW, int KB, int S>
void launch_one(const Variant& v, const AttnArgs& a, hipStream_t st) {
  hipLaunchKernelGGL((attention_kernel<DT, DP, RW, KW, KB, S>), dim3(unsigned(kWorkers)),
                     dim3(64 * RW * KW), 0, st, a);
}

template <int DT, int DP>
void launch(const Variant& v, const AttnArgs& a, hipStream_t st) {
  if constexpr (DP == 256) {
    if (v.rw == 2) launch_one<DT, DP, 2, 2, 32, 2>(v, a, st);
    else launch_one<DT, DP, 4, 1, 32, 4>(v, a, st);
  } else {
    constexpr int X = 128 / DP;  // stages of half the size, twice as many
    if (v.rw == 2) launch_one<DT, DP, 2, 4, 32, 2 * X>(v, a, st);
    else if (v.rw == 4) launch_one<DT, DP, 4, 2, 64, 2 * X>(v, a, st);
    else launch_one<DT, DP, 8, 1, 64, 4>(v, a, st);
  }
}

template <int DT, int DP>
void launch_both(const Variant& v, const AttnArgs& a, hipStream_t st) {
  launch<DT, DP>(v, a, st);
  if (a.whole) return;
  hipLaunchKernelGGL((join_kernel<DT, DP>), dim3(kJoiners), dim3(kWorkers), 0, st, a);
}

template <int DT>
void launch_width(const Variant& v, const AttnArgs& a, hipStream_t st) {
  if (v.width == 64) launch_both<DT, 64>(v, a, st);
  else if (v.width == 128) launch_both<DT, 128>(v, a, st);
  else launch_both<DT, 256>(v, a, st);
}

bool sizes_ok(int64_t B, int64_t T, int64_t Hq, int64_t Hkv, int64_t D, int64_t max_nodes) {
  const int64_t k31 = int64_t(1) << 31;
  return B >= 1 && B < k31 && T >= 0 && T < k31 && Hq >= 1 && Hkv >= 1 && Hq < k31 && Hkv < k31 &&
         Hq % Hkv == 0 && D >= 8 && D <= SV_MAX_HEAD_DIM && D % 8 == 0 && max_nodes >= 1 &&
         max_nodes <= SV_MAX_TREE_NODES && max_nodes * (Hq / Hkv) <= (1 << 16) &&
         B * Hkv <= (1 << 24) && T * Hq < k31;
}

}  // namespace

#ifdef SV_DEVICE_CHECKS
bool sv_add_tree_attention_checks(uint32_t* count, int reset) { return sv_add_checks(count, reset); }
#endif

extern "C" {

size_t specverify_tree_attention_workspace_size(int64_t B, int64_t T, int64_t Hq, int64_t Hkv,
                                                int64_t D, int64_t max_nodes) {
  if (!sizes_ok(B, T, Hq, Hkv, D, max_nodes)) return 0;
  const Variant v = variant_of(max_nodes * (Hq / Hkv), D);
  return align256(size_t(kWorkers + 1) * sizeof(Split)) +
         align256(size_t(kWorkers) * 2 * (32 * v.rw) * (v.width + 4) * sizeof(float));
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
      max_pages * page_size + max_nodes > k31 - (1 << 14) || num_pages < 1 || num_pages >= k31 ||
      table_stride < max_pages || !stride_ok(table_stride))
    return SV_EINVAL;
  const int64_t strides[] = {q_stride_t, q_stride_h, n_stride_t, n_stride_h, c_stride_page,
                             c_stride_token, c_stride_h, o_stride_t, o_stride_h};
  for (int64_t s : strides)
    if (!stride_ok(s)) return SV_EINVAL;
  if (!(scale > 0.0f) || !std::isfinite(scale * kLog2e)) return SV_EINVAL;
  if (dtype != SV_BF16 && dtype != SV_F16) return SV_EDTYPE;
  for (int64_t s : strides)
    if (s % 8 != 0) return SV_EALIGN;
  if (!aligned16(q) || !aligned16(k_tree) || !aligned16(v_tree) || !aligned16(k_cache) ||
      !aligned16(v_cache) || !aligned16(out))
    return SV_EALIGN;
  const int64_t out_sizes[] = {T, Hq}, out_strides[] = {o_stride_t, o_stride_h};
  if (!apart(2, out_sizes, out_strides, D)) return SV_EINVAL;
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
  a.split = static_cast<Split*>(workspace);
  a.part = reinterpret_cast<float*>(static_cast<char*>(workspace) +
                                    align256(size_t(kWorkers + 1) * sizeof(Split)));
  a.tile_keys = v.kw * v.kb;
  a.tile_rows = 32 * v.rw;
  const int64_t items = B * Hkv * ((max_nodes * (Hq / Hkv) + a.tile_rows - 1) / a.tile_rows);
  a.whole = max_pages * page_size + max_nodes <= kWholeTiles * int64_t(a.tile_keys) &&
            items <= kWorkers;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  if (dtype == SV_BF16) launch_width<SV_BF16>(v, a, st);
  else launch_width<SV_F16>(v, a, st);
  return launch_status();
}

}  // extern "C"
