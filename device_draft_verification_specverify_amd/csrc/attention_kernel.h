// attention_kernel.h -- attention over a paged cache by matrix cores (gfx950): of
// drafted tree nodes over their prefix and ancestors, and of chunks of new tokens
// over all that is cached up to each of them.
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
//
// Chunks of many rows, of heads up to 128, have a kernel whose 8 wavefronts are two
// halves: while one half is at the products of a tile the other is at its softmax, so
// that the matrix cores and the exponentials have work at the same time. A prompt of
// 8192 tokens, 32 heads of 128: 563 us, 0.98 PFLOP/s; 274 tokens behind 100003 and
// 131072: 504 us, 0.90 PFLOP/s. A tile of 64 keys takes a wavefront some 3700 cycles,
// of them 2 x 1100 the two halves' products, and an item some 22000 besides (rows
// loaded and written, masked tiles at its end), which is what bounds chunks of some
// hundred tokens behind nothing.
#pragma once

#include <type_traits>

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
  // chunks (below): query heads of a row tile at most, parts of a key head's query
  // heads, whole tokens of a row tile, and the rows that requests taken here have
  int GS, parts, tokens, rows_from, rows_to;
  int item_places;  // what an item costs besides its tiles, in tiles
  // workspace
  struct Split* split;  // [workers], and all tiles in one more's start
  float* part;          // [workers * 2][M][DP + 4]: sums, then m and l
  int tile_keys, tile_rows, whole;
};

// An item (request, key head, row tile) that a worker began inside of: its tiles
// count from `start` in the order of all tiles.
struct Split {
  int64_t start, first;  // first: the request's first row (chunks: the item's first)
  int32_t tiles;         // 0: none
  int32_t h, row0, rows; // rows of the item, from row0 on, of `rows` in all (chunks: the
                         // first query head, query heads, rows)
};

__device__ const u32x4 zero_piece = {0, 0, 0, 0};

// Tiles of request b, and its sizes.
struct Req {
  int64_t first;
  int32_t n, len, tiles, row_tiles;
};

// Chunks (CHUNK): the new tokens' keys are in the pages, too, and token i sees the
// keys up to its own, len + i. A row tile holds the rows of whole tokens, `tokens`
// of them, so what it sees ends at one key for all but the diagonal, and its tiles
// are a closed formula.

// What a request with n tokens behind `len` keys has of rows; none if that goes
// beyond its block table or another launch takes requests of so many rows.
__device__ __forceinline__ Req chunk_request(int64_t max_keys, int G, int tile_keys, int tokens,
                                             int rows_from, int rows_to, Req r, int64_t len) {
  const int64_t most = max_keys - r.n;
  r.len = int32_t(len < 0 ? 0 : len > most ? (most < 0 ? 0 : most) : len);
  if (most < 0 || r.n * G < rows_from || r.n * G > rows_to) r.n = 0;
  r.tiles = (r.len + r.n + tile_keys - 1) / tile_keys;
  r.row_tiles = (r.n + tokens - 1) / tokens;
  return r;
}

// Tiles that row tile i has.
__device__ __forceinline__ int chunk_tiles(int tile_keys, int tokens, const Req& r, int i) {
  const int upto = r.n - i * tokens < tokens ? r.n : (i + 1) * tokens;
  return (r.len + upto + tile_keys - 1) / tile_keys;
}

// sum over i < n of floor((a i + b) / 2^s): the sum of a i + b without what each leaves.
// What they leave repeats after 2^s / g of them, g the largest power of two in a up to
// 2^s, and is each of b mod g, b mod g + g, ... once in a period; the rest of a period is
// gone through. (With Euclid's divisions a
// worker took 10700 cycles to find its place, with this 7500.)
__device__ __forceinline__ int64_t floor_sum(int64_t n, int s, uint32_t a, uint32_t b) {
  const uint32_t m = 1u << s, low = (a & (0u - a)) | m, g = low & (0u - low);
  const int period_log = s - (31 - __builtin_clz(g));
  const int64_t period = int64_t(1) << period_log;
  int64_t left = (n >> period_log) *
                 (period * (b & (g - 1)) + int64_t(g) * (period * (period - 1) / 2));
  const int rest = int(n & (period - 1));
  for (int i = 0; i < rest; ++i) left += (a * uint32_t(i) + b) & (m - 1);
  return (int64_t(a) * (n * (n - 1) / 2) + int64_t(b) * n - left) >> s;
}

// Tiles of the first k row tiles, of row_tiles at most.
__device__ __forceinline__ int64_t chunk_tile_sum(int tile_keys, int tokens, const Req& r, int k) {
  if (k == 0) return 0;
  const int full = k < r.row_tiles ? k : k - 1;
  return floor_sum(full, 31 - __builtin_clz(tile_keys), tokens, r.len + tokens + tile_keys - 1) +
         (full < k ? r.tiles : 0);
}
template <bool CHUNK>
__device__ __forceinline__ Req request(const AttnArgs& a, int64_t b, int* bits = nullptr) {
  Req r;
  const Nodes nd = nodes_of(a.node_start, b, a.T, a.max_nodes);
  r.first = nd.first;
  r.n = nd.n < 0 ? 0 : nd.n;
  const int64_t len = a.prefix_len[b];
  if constexpr (CHUNK) {
    r = chunk_request(a.max_keys, a.G, a.tile_keys, a.tokens, a.rows_from, a.rows_to, r, len);
    if (bits)
      *bits |= (nd.n < 0 ? SV_ERR_TREE : 0) |
               (r.len != len || nd.n > a.max_keys ? SV_ERR_LENGTH : 0);
    return r;
  }
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
template <bool CHUNK>
__device__ __forceinline__ Req uniform_request(Args a, int64_t b) {
  const auto* start = constant(a->node_start) + b;
  const int64_t lo = start[0], hi = start[1], len = constant(a->prefix_len)[b];
  const bool good = lo >= 0 && hi >= lo && hi <= a->T && hi - lo <= a->max_nodes;
  Req r;
  r.first = good ? lo : 0;
  r.n = good ? int32_t(hi - lo) : 0;
  if constexpr (CHUNK)
    return chunk_request(a->max_keys, a->G, a->tile_keys, a->tokens, a->rows_from, a->rows_to, r,
                         len);
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
// The same for chunks: of the first k row tiles of one part of a key head's rows.
__device__ __forceinline__ int64_t chunk_places(const AttnArgs& a, const Req& r, int k) {
  return a.whole ? k
                 : int64_t(a.item_places) * k + chunk_tile_sum(a.tile_keys, a.tokens, r, k);
}
template <bool CHUNK>
__device__ __forceinline__ int64_t all_places(const AttnArgs& a, const Req& r) {
  if constexpr (CHUNK)
    return chunk_places(a, r, r.row_tiles) * (a.Hkv * a.parts);
  else
    return places_of(a.whole, a.Hkv, r);
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
  int32_t head, rt, place; // chunks: that place's part of the heads, row tile, and how far in
};

// A share of an item's tiles, prepared while the one before is fetched.
struct Seg {
  int64_t start, first;
  int64_t head, node, table;  // the request's keys of this head, its nodes', its pages
  int32_t n, len, h, rt, t0, t1, tiles;
  int32_t token0, heads, rows;  // chunks: the item's first token, query heads (h: the first), rows
};

// RW wavefronts along the rows (32 each), KW along a tile's keys (KB each), a
// ring of S tiles. DC > 0: the wavefronts take turns (below), with DC columns of
// the DP that a tile holds.
template <int DT, int DP, int RW, int KW, int KB, int S, bool CHUNK, int DC = 0>
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
  constexpr int SEGS = S + (DC ? 4 : 2);
  __shared__ Seg segs[SEGS];
  __shared__ Cursor cursors[2];
  __shared__ int32_t id_box[NT / 64][2][64];
  __shared__ int wild_seg;
  __shared__ int wild_of[DC ? SEGS : 1];  // the same of each share on its way
  const Args args = (Args)__builtin_amdgcn_kernarg_segment_ptr();
  const int tid = int(threadIdx.x), lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int rw = wv % RW, kw = wv / RW;
  const int col = lane & 31, half = lane >> 5;

  // This worker's share: neighbours in the order of tiles share an XCD's L2
  // (workgroups go round robin over the 8 XCDs).
  constexpr int workers = kWorkers;
  const int64_t w = workers % 8 == 0 ? (blockIdx.x % 8) * (workers / 8) + blockIdx.x / 8
                                     : blockIdx.x;
  if (tid == 0) {
    a.split[w].tiles = 0;
    wild_seg = -1;
    if constexpr (DC)
      for (int i = 0; i < SEGS; ++i) wild_of[i] = -1;
  }
  // All tiles, and those in front of this thread's request (of the last round).
  int64_t total = 0, mine = 0, lo = 0;
  Req own{};
  for (int64_t o = 0; o < a.B; o += NT) {
    int bits = 0;
    if (o + tid < a.B) own = request<CHUNK>(a, o + tid, &bits);
    mine = o + tid < a.B ? all_places<CHUNK>(a, own) : 0;
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
  if (!sv_ok(int(gridDim.x) == workers && w < workers && at <= end && end <= total)) return;
  if (w == 0 && tid == 0) a.split[workers].start = total;
  if (at >= end) return;
  // the request that holds tile `at`: more than NT of them are gone through again
  int64_t base = 0;
  for (int64_t o = 0; o < a.B; o += NT) {
    if (a.B > NT) {
      if (o + tid < a.B) own = request<CHUNK>(a, o + tid);
      mine = o + tid < a.B ? all_places<CHUNK>(a, own) : 0;
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
    if (at >= lo && at < lo + mine) {
      cursors[0] = Cursor{at, o + tid, lo, own, 0, 0, 0};
      if constexpr (CHUNK) cursors[1].at = chunk_places(a, own, own.row_tiles);
    }
    if (base > at) break;
  }
  __syncthreads();
  if constexpr (CHUNK) {
    // Its part of the heads and its row tile, the one that begins last of those that
    // begin no later: every thread tries one (512 at a time), for a sum takes long.
    const Req rq = cursors[0].rq;
    const int64_t each = cursors[1].at, into = at - cursors[0].b_first;
    int head = int(double(into) / double(each));  // to one less or more
    if (head * each > into) --head;
    if ((head + 1) * each <= into) ++head;
    const int64_t within = into - head * each;
    for (int k0 = 0; k0 < rq.row_tiles; k0 += NT) {
      const int k = k0 + tid;
      if (k >= rq.row_tiles) break;
      const int64_t begins = chunk_places(a, rq, k);
      const int64_t places = a.whole ? 1 : chunk_tiles(a.tile_keys, a.tokens, rq, k) + a.item_places;
      if (begins <= within && within < begins + places) {
        cursors[0].head = head;
        cursors[0].rt = k;
        cursors[0].place = int32_t(within - begins);
      }
    }
    __syncthreads();
  }

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
    int head = 0, rt = 0, place = 0;
    if constexpr (CHUNK) {
      head = uniform(cursor.head);
      rt = uniform(cursor.rt);
      place = uniform(cursor.place);
      const int heads = s->Hkv * s->parts;
      do {
        if (at >= end) {
          more = false;
          return;
        }
        while (rt == rq.row_tiles) {  // (also of requests without rows)
          rt = 0;
          if (rq.row_tiles == 0 || ++head == heads) {
            head = 0;
            rq = uniform_request<CHUNK>(s, ++b);
          }
        }
        sg.tiles = chunk_tiles(s->tile_keys, s->tokens, rq, rt);
        const int size = s->whole ? 1 : sg.tiles + s->item_places;
        const int64_t left = end - at;
        const int upto = size - place < left ? size : place + int(left);
        sg.start = at - place;
        sg.t0 = min(place, sg.tiles);
        sg.t1 = s->whole ? sg.tiles : min(upto, sg.tiles);
        sg.h = head;
        sg.rt = rt;
        at += upto - place;
        place = upto;
        if (upto == size) {
          place = 0;
          ++rt;
        }
      } while (sg.t0 == sg.t1);
      if (!sv_ok(b < s->B && sg.h >= 0 && sg.h < heads && sg.rt < rq.row_tiles && sg.t0 < sg.t1 &&
                 sg.t1 <= sg.tiles && rq.first + rq.n <= s->T)) {
        more = false;
        return;
      }
      const int kv = sg.h / s->parts, part = sg.h - kv * s->parts;
      sg.token0 = sg.rt * s->tokens;
      sg.heads = min(s->GS, s->G - part * s->GS);
      sg.rows = min(s->tokens, rq.n - sg.token0) * sg.heads;
      sg.h = kv * s->G + part * s->GS;
      sg.head = int64_t(s->k_cache + kv * s->c_h);
      sg.node = 0;
    } else {
      do {
        if (at >= end) {
          more = false;
          return;
        }
        while (at >= b_first + places_of(s->whole, s->Hkv, rq)) {
          b_first += places_of(s->whole, s->Hkv, rq);
          rq = uniform_request<CHUNK>(s, ++b);
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
      sg.tiles = rq.tiles;
      sg.head = int64_t(s->k_cache + sg.h * s->c_h);
      sg.node = int64_t(s->k_tree + rq.first * s->n_t + sg.h * s->n_h);
    }
    sg.first = rq.first;
    sg.n = rq.n;
    sg.len = rq.len;
    const int32_t* table = s->table + b * s->table_stride;
    sg.table = int64_t(table);
    const int cached = CHUNK ? rq.len + rq.n : rq.len;
    if (one_page && cached > 0) load_lds4(id_place(table, sg.t0, cached), id_at + 256);
    turn ^= 1;
    if (tid == 0) {
      segs[prepared % SEGS] = sg;
      cursors[turn] = Cursor{at, b, b_first, rq, head, rt, place};
    }
    ++prepared;
  };
  // Starts the next tile's keys and values on their way into a stage; false when
  // the share is at its end.
  auto fetch_next = [&](int to_stage) __attribute__((always_inline)) {
    const bool fresh = f_t == f_t1;
    if (fresh) {
      if (!more) return false;
      const Seg& sg = segs[f_seg % SEGS];
      ++f_seg;
      f_t = uniform(sg.t0);
      f_t1 = uniform(sg.t1);
      f_len = uniform(sg.len) + (CHUNK ? uniform(sg.n) : 0);
      f_keys = f_len + (CHUNK ? 0 : uniform(sg.n));
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
        const char* np = CHUNK ? nullptr : f_node + int64_t(key - f_len) * s->n_t;
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
  int all_see = 0, last = 0;  // chunks: keys that all rows of the item see, this row's last
  u32x4 qf[DP / 16];
  f32x16 acc[ND];
  float m = -INFINITY, l = 0.0f;

  // The rows of share `which`: this lane's part of them to registers, and its mask.
  uint64_t next_see0 = 0, next_see1 = 0;
  auto load_rows = [&](int which) __attribute__((always_inline)) {
    const Args s = again(args);
    const Seg& sg = segs[which % SEGS];
    if constexpr (CHUNK) {
      const int rows = uniform(sg.rows), heads = uniform(sg.heads), row0 = rw * 32;
      if (row0 >= rows) return;
      const int r = row0 + col < rows ? row0 + col : 0;
      const int token = r / heads;
      const int64_t i = uniform(sg.first) + uniform(sg.token0) + token;
      const int hq = uniform(sg.h) + r - token * heads;
      if (!sv_ok(i < s->T && hq < s->Hq)) return;
      const char* qp = s->q + i * s->q_t + hq * s->q_h;
#pragma unroll
      for (int k = 0; k < DP / 16; ++k) {
        const int d = 16 * k + 8 * half;
        qf[k] = *reinterpret_cast<const u32x4*>(d < s->D ? qp + d * 2 : zero);
      }
      return;
    }
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

  // Zeros for the wild values of keys first .. keys - 1 among tile t's at tv; thread
  // `who` of THREADS; whether there were any of its part.
  auto tame_some = [&](char* tv, int tile_t, int who, auto threads, int first, int keys)
                       __attribute__((always_inline)) {
    constexpr int THREADS = decltype(threads)::value;
    bool mine = false;
#pragma unroll
    for (int u = 0; u < KT * CPR / THREADS; ++u) {
      const int unit = u * THREADS + who;
      const int key = tile_t * KT + unit / CPR;
      if (key >= first && key < keys) {
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
    return mine;
  };
  auto tame = [&](char* tv, int who, int first, int keys) __attribute__((always_inline)) {
    return tame_some(tv, t, tid, std::integral_constant<int, NT>{}, first, keys);
  };

  // What was zeroed, for the rows that see it (rare, so scores are simply taken again).
  auto add_wild = [&](const Seg& sg) __attribute__((always_inline)) {
    const Args s = again(args);
    const int t0 = uniform(sg.t0), t1 = uniform(sg.t1), h = uniform(sg.h);
    const int64_t first = uniform(sg.first);
    // The wild values of the nodes among this share's keys, for the rows that
    // see them (rare, so scores are simply taken again).
    const int32_t* pages = reinterpret_cast<const int32_t*>(uniform(sg.table));
    const int x0 = CHUNK ? all_see - len : 0;
    for (int x = max(t0 * KT - len, x0); x < min(t1 * KT - len, n); ++x) {
      const bool see = row_ok && (CHUNK ? x <= node : (x < 64 ? see0 >> (x & 63) : see1 >> (x & 63)) & 1);
      const char* kp;
      if constexpr (CHUNK) {
        const int at = len + x;
        const int32_t id = pages[sv_ok(at < a.max_keys) ? at >> page_shift : 0];
        if (uint32_t(id) >= num_pages) continue;
        kp = reinterpret_cast<const char*>(uniform(sg.head)) + id * c_page +
             (at & in_page) * c_token;
      } else {
        kp = s->k_tree + (first + x) * s->n_t + h * s->n_h;
      }
      const elem* kx = reinterpret_cast<const elem*>(kp);
      const elem* qx =
          reinterpret_cast<const elem*>(s->q + (first + node) * s->q_t + hq * s->q_h);
      const uint16_t* vx = reinterpret_cast<const uint16_t*>(kp + (CHUNK ? v_cache : s->v_tree));
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
  };
  // A share's results: the item's rows, or its part of them for the join.
  auto write_out = [&](const Seg& sg) __attribute__((always_inline)) {
    const Args s = again(args);
    const int t0 = uniform(sg.t0), h = uniform(sg.h);
    const int64_t first = uniform(sg.first);
    const bool whole = t0 == 0 && uniform(sg.t1) == uniform(sg.tiles);
    constexpr int COLS = DC ? DC / 32 : ND;
    if (row_ok && sv_ok(first + node < s->T && hq < s->Hq)) {
      if (whole) {
        const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
        char* op = s->out + (first + node) * s->o_t + hq * s->o_h + 8 * half;
#pragma unroll
        for (int i = 0; i < COLS; ++i) {
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
        for (int i = 0; i < COLS; ++i) {
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
      s->split[w] = CHUNK ? Split{sg.start, first + sg.token0, sg.tiles, h, sg.heads, sg.rows}
                          : Split{sg.start, first, sg.tiles, h, sg.rt * M, n * s->G};
  };
  prepare();
  meet();
  if (more) load_rows(0);
  rows_here();
  asm volatile("s_waitcnt vmcnt(0)" : : : "memory");  // the first page ids
  int fetched = 0, done = 0;
  if constexpr (DC > 0) {
    // Many rows: two halves of the workgroup, one wavefront of each to a SIMD, take
    // turns. While one half has the matrix cores (O += V P of the tile before, S = K Q
    // of this one) the other takes the softmax of its scores on the vector units, and
    // a barrier changes them over: with all 8 wavefronts in step each unit waits for
    // the other.
    //   phase 2 i:      first half products of tile i, second half softmax of i - 1
    //   phase 2 i + 1:  first half softmax of i, second half products of i
    // Tiles are asked for during the products, a load now and then between them (all at
    // once they hold up the wavefront for longer than a third of a phase): in those of
    // tile i the keys of i + 3, whose stage was read last in phase 2 i - 1, and the
    // values of i + 2, alike. They are read from phase 2 i + 5 on (values that are not
    // finite; products from 2 i + 6 on), so each wavefront sees to it that its part is
    // here at the end of 2 i + 4, when the first half has asked for two more such batches
    // and the second for one. Behind the last tile there are loads, too, of zeros that
    // nobody reads, so the count of a batch is always the same.
    static_assert(CHUNK && KW == 1 && NB == 2 && S == 4 && SAME, "whole rows, 64 keys a tile");
    constexpr int KS = DC / 16, COLS = DC / 32, NV = 4 * COLS, NK = 2 * KS;
    constexpr int R = 8;  // fragments read ahead
    static_assert(R <= NV, "the first ones are of values");
    const bool second = wv >= RW / 2;
    auto change = [&]() __attribute__((always_inline)) {
      __builtin_amdgcn_sched_barrier(0);
      meet();
      __builtin_amdgcn_sched_barrier(0);
    };
    // this wavefront's loads but its newest `batches` are here
    auto landed = [&](auto batches) __attribute__((always_inline)) {
      asm volatile("s_waitcnt vmcnt(%0)" : : "n"(decltype(batches)::value * LOADS) : "memory");
    };
    const std::integral_constant<int, 1> one_batch;
    const std::integral_constant<int, 2> two_batches;

    // This lane's pieces of the tile that was found last: its keys, its values, and the
    // values of the one before.
    const char *kp[UNITS], *vp[UNITS], *old_vp[UNITS];
    const char* nothing = zero;  // (held, or it is found anew at every use)
    asm volatile("" : "+s"(nothing));
    const int piece = (lane % CPR) ^ swizzle<CPR>(wv * WROWS + lane_row);
    const int64_t lane_off = lane_row * c_token + piece * 16;
    const bool lane_ok = piece * 8 < a.D;
    int64_t to_values = v_cache;  // (scalar registers are short)
    asm volatile("" : "+v"(to_values));
    // Where the rows of this wavefront's loads begin, in BATCH tiles from f_batch on, one
    // a lane, and in which of them the page is none of the cache's.
    uint64_t bases = 0, bad = 0;
    int f_safe = 0;  // up to this tile all is as usual: whole tiles of good pages
    auto take_bases = [&](int box) __attribute__((always_inline)) {
      take_ids(box);
      const int row = (f_batch + lane / UNITS) * KT + lane % UNITS * (NT / CPR) + wv * WROWS;
      bad = __ballot(uint32_t(ids) >= num_pages);
      bases = reinterpret_cast<uint64_t>(f_head) + uint32_t(ids) * uint64_t(c_page) +
              uint32_t(row & in_page) * uint64_t(c_token);
      if (f_batch + BATCH < f_t1) load_lds4(id_place(f_table, f_batch + BATCH, f_len), id_at);
    };
    auto next_tile = [&]() __attribute__((always_inline)) {
#pragma unroll
      for (int u = 0; u < UNITS; ++u) old_vp[u] = vp[u];
      auto found = [&](int id0) __attribute__((always_inline)) {
#pragma unroll
        for (int u = 0; u < UNITS; ++u) {
          const uint32_t lo = uint32_t(__builtin_amdgcn_readlane(int(bases), id0 + u));
          const uint32_t hi = uint32_t(__builtin_amdgcn_readlane(int(bases >> 32), id0 + u));
          kp[u] = reinterpret_cast<const char*>((uint64_t(hi) << 32 | lo) + lane_off);
          vp[u] = kp[u] + to_values;
          if (!full) {  // narrower heads: zeros behind them
            kp[u] = lane_ok ? kp[u] : nothing;
            vp[u] = lane_ok ? vp[u] : nothing;
          }
        }
      };
      // One test for what is usual (one by one they waited in the way of the products).
      if (__builtin_expect(f_t < f_safe, 1)) {
        found((f_t - f_batch) * UNITS);
        ++f_t;
        ++fetched;
        return;
      }
      const bool fresh = f_t == f_t1;
      if (fresh) {
        if (!more) {
#pragma unroll
          for (int u = 0; u < UNITS; ++u) kp[u] = vp[u] = nothing;
          return;
        }
        const Seg& sg = segs[f_seg % SEGS];
        ++f_seg;
        f_t = uniform(sg.t0);
        f_t1 = uniform(sg.t1);
        f_len = uniform(sg.len) + uniform(sg.n);
        f_head = reinterpret_cast<const char*>(uniform(sg.head));
        f_table = reinterpret_cast<const int32_t*>(uniform(sg.table));
        f_batch = f_t;
        if (one_page) {
          // its ids are older than the tiles of the share before but the first
          if (f_tiles < S) asm volatile("s_waitcnt vmcnt(0)" : : : "memory");
          take_bases(1);
        }
        f_tiles = f_t1 - f_t;
      }
      const int t = f_t++;
      if (t - f_batch == BATCH) {
        f_batch = t;
        if (one_page) take_bases(0);
      }
      f_safe = one_page && bad == 0 ? min(min(f_t1, f_batch + BATCH), f_len / KT) : 0;
      const int id0 = (t - f_batch) * UNITS;
      const bool some = sv_ok(t * KT < f_len && f_seg <= prepared);
      if (one_page) {
        found(id0);
        // the end of the keys, pages outside the cache
        const bool wrong = bad >> id0 & ((1u << UNITS) - 1);
        if (wrong || !some || t * KT + KT > f_len) {
#pragma unroll
          for (int u = 0; u < UNITS; ++u) {
            const bool here = t * KT + u * (NT / CPR) + wv * WROWS + lane_row < f_len;
            const bool good = !(bad >> (id0 + u) & 1);
            const bool take = some && here && good;
            kp[u] = take ? kp[u] : nothing;
            vp[u] = take ? vp[u] : nothing;
            if (wrong && here && !good) set_error(again(args)->err, SV_ERR_PAGE);
          }
        }
      } else {  // pages of fewer rows than a wavefront loads
#pragma unroll
        for (int u = 0; u < UNITS; ++u) {
          const int key = t * KT + u * (NT / CPR) + wv * WROWS + lane_row;
          const bool here = key < f_len;
          const int32_t page = f_table[(here ? key : f_len - 1) >> page_shift];
          const bool good = uint32_t(page) < num_pages;
          if (here && !good) set_error(again(args)->err, SV_ERR_PAGE);
          const bool take = some && here && good && lane_ok;
          kp[u] = take ? f_head + uint32_t(page) * uint64_t(c_page) +
                             uint32_t(key & in_page) * uint64_t(c_token) + piece * 16
                       : nothing;
          vp[u] = take ? kp[u] + to_values : nothing;
        }
      }
      ++fetched;
      if (fresh) prepare();
    };
    auto ask = [&](int which, uint32_t k_stage, uint32_t v_stage) __attribute__((always_inline)) {
      if (which < UNITS) load_lds16(old_vp[which], v_stage + wv * 1024 + which * NT * 16 + KT * DP * 2);
      else load_lds16(kp[which - UNITS], k_stage + wv * 1024 + (which - UNITS) * NT * 16);
    };
    auto stage_of = [&](int x) __attribute__((always_inline)) {
      return tile_at + uint32_t(x % S) * STAGE;
    };

    typename E::vec pf[4];
    s16x8 b[R];
    // The f-th fragment of the products: values of the tile before, stage `before`, then
    // keys of this one.
    auto fragment = [&](int f, uint32_t before, uint32_t now) __attribute__((always_inline)) {
      if (f < NV) {
        const uint32_t at = (before + v_off) ^ ((f % COLS) * 64);
        const uint32_t rows = f / COLS * 16 * (DP * 2);
        const s16x4 x0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (__attribute__((address_space(3))) s16x4*)(at + rows));
        const s16x4 x1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (__attribute__((address_space(3))) s16x4*)((at ^ 32) + rows + 8 * (DP * 2)));
        return __builtin_shufflevector(x0, x1, 0, 1, 2, 3, 4, 5, 6, 7);
      }
      const int g = f - NV;
      return *reinterpret_cast<__attribute__((address_space(3))) const s16x8*>(
          ((now + k_off) ^ (g / 2 * 32)) + g % 2 * 32 * (DP * 2));
    };
    auto first_fragments = [&](uint32_t before) __attribute__((always_inline)) {
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int f = 0; f < R; ++f) b[f] = fragment(f, before, 0);
      __builtin_amdgcn_sched_barrier(0);
    };
    // Those up to `end`, with a batch of loads among them.
    auto products = [&](f32x16 (&s)[2], uint32_t before, uint32_t now, auto end, int i)
                        __attribute__((always_inline)) {
      constexpr int F1 = decltype(end)::value, EACH = (NV + NK) / LOADS;
      constexpr bool ASK = F1 > NV;
      const uint32_t k_stage = stage_of(i + 3), v_stage = stage_of(i + 2);
      if constexpr (ASK) {
        s[0] = f32x16{0};
        s[1] = f32x16{0};
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int f = 0; f < F1; ++f) {
        const s16x8 x = b[f % R];
        if (f < NV) acc[f % COLS] = E::mfma(x, pf[f / COLS], acc[f % COLS]);
        else s[(f - NV) % 2] = E::mfma(x, __builtin_bit_cast(typename E::vec, qf[(f - NV) / 2]), s[(f - NV) % 2]);
        if (f + R < F1) b[f % R] = fragment(f + R, before, now);
        if constexpr (ASK)
          if (f % EACH == EACH / 2 && f / EACH < LOADS) ask(f / EACH, k_stage, v_stage);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    auto finish = [&](int which) __attribute__((always_inline)) {
      const Seg& sg = segs[which % SEGS];
      l += __shfl_xor(l, 32);
      if (wild_of[which % SEGS] == which) add_wild(sg);
      write_out(sg);
    };

    // K 0, then V 0 and K 1, V 1 and K 2
#pragma unroll
    for (int u = 0; u < UNITS; ++u) vp[u] = nothing;
#pragma unroll 1
    for (int i = 0; i < 3; ++i) {
      next_tile();
      if (i > 0)
#pragma unroll
        for (int u = 0; u < UNITS; ++u) ask(u, 0, stage_of(i - 1));
#pragma unroll
      for (int u = 0; u < UNITS; ++u) ask(UNITS + u, stage_of(i), 0);
      meet();
    }
    if (fetched == 0) {  // its places are none of tiles
      asm volatile("s_waitcnt vmcnt(0)" : : : "memory");
      return;
    }
    landed(two_batches);
    meet();
    if (second) {
      landed(one_batch);
      change();
    }
#pragma unroll
    for (int hb = 0; hb < 4; ++hb) pf[hb] = typename E::vec{};
#pragma unroll
    for (int i = 0; i < ND; ++i) acc[i] = f32x16{0};
    bool act = false;  // whether this wavefront has rows that see the tile
    int wave_last = 0;
#pragma unroll 1
    for (; done < fetched; ++done) {
      __builtin_amdgcn_s_setprio(1);
      const bool fresh = t == t1;
      if (__builtin_expect(fresh, 0)) {
        const Seg& sg = segs[seg % SEGS];
        t = uniform(sg.t0);
        t1 = uniform(sg.t1);
        ++seg;
        const int rows = uniform(sg.rows);
        wave_ok = rw * 32 < rows;
        wave_last = uniform(sg.len) + uniform(sg.token0) +
                    (min(rows, rw * 32 + 32) - 1) / uniform(sg.heads);
      }
      f32x16 s[2];
      act = wave_ok && t * KT <= wave_last;
      // (on their way while the next tile is found)
      first_fragments(stage_of(done + S - 1));
      next_tile();
      // (All wavefronts go this way, also those without rows here: one way is fewer
      // registers than several. Where a wavefront saw nothing of the tile before its
      // weights are zeros, and the values that are not finite are so, too; in front of
      // the first tile there is anything, but no sum yet.)
      products(s, stage_of(done + S - 1), stage_of(done), std::integral_constant<int, NV + NK>{},
               done);
      __builtin_amdgcn_s_setprio(0);
      if (!second) landed(two_batches);
      change();

      if (__builtin_expect(fresh, 0)) {
        if (done > 0) finish(seg - 2);
        const Seg& sg = segs[(seg - 1) % SEGS];
        len = uniform(sg.len);
        n = uniform(sg.n);
        const int rows = uniform(sg.rows), heads = uniform(sg.heads), r = rw * 32 + col;
        row_ok = r < rows;
        const int token = (row_ok ? r : 0) / heads;
        node = uniform(sg.token0) + token;
        hq = uniform(sg.h) + (row_ok ? r - token * heads : 0);
        all_see = len + uniform(sg.token0) + 1;
        last = len + node;
#pragma unroll
        for (int i = 0; i < COLS; ++i) acc[i] = f32x16{0};
        m = -INFINITY;
        l = 0.0f;
      }
      if (__builtin_expect(!second && t * KT + KT > all_see, 0))  // read by nobody before the next phase
        if (tame_some(tile + done % S * STAGE + KT * DP * 2, t, tid,
                      std::integral_constant<int, NT / 2>{}, all_see, len + n))
          wild_of[(seg - 1) % SEGS] = seg - 1;
      if (act) {
        if (__builtin_expect(t * KT + KT > all_see, 0)) {
          const int ahead = last - (t * KT + 4 * half);
#pragma unroll
          for (int nb = 0; nb < 2; ++nb)
#pragma unroll
            for (int i = 0; i < 16; ++i)
              s[nb][i] = nb * 32 + 8 * (i / 4) + i % 4 <= ahead ? s[nb][i] : -INFINITY;
        }
        float top = -INFINITY;
#pragma unroll
        for (int nb = 0; nb < 2; ++nb)
#pragma unroll
          for (int i = 0; i < 16; ++i) top = fmaxf(top, s[nb][i]);
        top *= a.scale_log2;
        const auto halves = __builtin_amdgcn_permlane32_swap(__float_as_uint(top), __float_as_uint(top), false, false);
        top = fmaxf(__uint_as_float(halves[0]), __uint_as_float(halves[1]));
        // The reference may lag behind the maximum: weights up to 2^8 are as exact as
        // those up to 1, and sums of 2^31 of them far from float32's end.
        if (__builtin_expect(__any(top > m + 8.0f), 0)) {
          const float to = fmaxf(m, top);
          const float f = to == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m - to);
          l *= f;
#pragma unroll
          for (int i = 0; i < COLS; ++i) acc[i] *= f;
          m = to;
        }
        const float ref = m == -INFINITY ? 0.0f : m;
#pragma unroll
        for (int nb = 0; nb < 2; ++nb)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            s[nb][i] = __builtin_amdgcn_exp2f(fmaf(s[nb][i], a.scale_log2, -ref));
            l += s[nb][i];
          }
        // (rounded as below)
#pragma unroll
        for (int hb = 0; hb < 4; ++hb)
#pragma unroll
          for (int j = 0; j < 8; ++j) pf[hb][j] = elem(s[hb / 2][8 * (hb % 2) + j]);
      } else {
#pragma unroll
        for (int hb = 0; hb < 4; ++hb) pf[hb] = typename E::vec{};
      }
      if (__builtin_expect(t + 1 == t1 && fetched > done + 1, 0)) {
        load_rows(seg);
        rows_here();
      }
      if (second) landed(one_batch);
      change();
      ++t;
    }
    if (act) {
      f32x16 none[2];
      first_fragments(stage_of(done + S - 1));
      products(none, stage_of(done + S - 1), 0, std::integral_constant<int, NV>{}, 0);
    }
    finish(seg - 1);
    if (!second) change();
    asm volatile("s_waitcnt vmcnt(0)" : : : "memory");  // no load outlives the workgroup
    return;
  }
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
      const Seg& sg = segs[seg % SEGS];
      t = uniform(sg.t0);
      t1 = uniform(sg.t1);
      len = uniform(sg.len);
      n = uniform(sg.n);
      const int h = uniform(sg.h), rt = uniform(sg.rt);
      keys = len + n;
      ++seg;
      if constexpr (CHUNK) {
        const int rows = uniform(sg.rows), heads = uniform(sg.heads), r = rw * 32 + col;
        row_ok = r < rows;
        const int token = (row_ok ? r : 0) / heads;
        node = uniform(sg.token0) + token;
        hq = h + (row_ok ? r - token * heads : 0);
        wave_ok = rw * 32 < rows;
        all_see = len + uniform(sg.token0) + 1;
        last = len + node;
      } else {
        const int r = rt * M + rw * 32 + col;
        row_ok = r < n * s->G;
        node = row_ok ? r / s->G : 0;
        hq = h * s->G + (row_ok ? r - node * s->G : 0);
        wave_ok = rt * M + rw * 32 < n * s->G;
      }
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
    // (A chunk's keys that the item's first token sees are seen by all its rows.)
    const int some_see = CHUNK ? all_see : len;  // keys from here on are not seen by all
    if (t * KT + KT > some_see) {
      if (tame(tv, tid, some_see, keys)) wild_seg = seg;
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
      if (CHUNK && t * KT + KT > all_see) {
        const int ahead = last - key0;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int i = 0; i < 16; ++i)
            s[nb][i] = nb * 32 + 8 * (i / 4) + i % 4 <= ahead ? s[nb][i] : -INFINITY;
      }
      if (!CHUNK && t * KT + KT > len) {
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
      const Seg& sg = segs[(seg - 1) % SEGS];
      const int t0 = uniform(sg.t0), h = uniform(sg.h);
      const int64_t first = uniform(sg.first);
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
        add_wild(sg);
      }

      rows_here();
      write_out(sg);
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
template <int DT, int DP, bool CHUNK>
__device__ __forceinline__ void join_items(const AttnArgs& a, int block, int blocks) {
  using elem = typename Elem<DT>::type;
  constexpr int LANES = DP / 4, ROWS = kWorkers / LANES, AHEAD = 4;
  __shared__ Split item;
  __shared__ int item_second, item_unit, wave_units[kWorkers / kWave];
  const int tid = int(threadIdx.x), lane = tid % kWave;
  const Split own = a.split[tid];
  const int64_t total = a.split[kWorkers].start;
  const bool stands = own.tiles > 0 && share_start(total, kWorkers, tid - 1) <= own.start;
  const int rows = CHUNK ? own.rows : min(own.rows - own.row0, a.tile_rows);
  const int units = stands ? (rows + ROWS - 1) / ROWS : 0;
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
  for (int u = block; u < all; u += blocks) {
    if (u >= upto - units && u < upto) {
      item = own;
      item_second = tid;
      item_unit = u - (upto - units);
    }
    __syncthreads();
    const Split sp = item;
    const int second = item_second;
    const int in_tile = item_unit * ROWS + tid / LANES, r = CHUNK ? in_tile : sp.row0 + in_tile;
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
    const int heads = CHUNK ? sp.row0 : a.G;
    const int node = r / heads;
    const int hq = (CHUNK ? sp.h : sp.h * a.G) + r - node * heads;
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

template <int DT, int DP, bool CHUNK>
__global__ __launch_bounds__(kWorkers) void join_kernel(AttnArgs a) {
  join_items<DT, DP, CHUNK>(a, int(blockIdx.x), int(gridDim.x));
}

// Of two launches, half of the workgroups each.
template <int DT, int DP, bool CHUNK>
__global__ __launch_bounds__(kWorkers) void join_both_kernel(AttnArgs a, AttnArgs b) {
  const int half = int(gridDim.x / 2), block = int(blockIdx.x);
  if (block < half) {
    if (!a.whole) join_items<DT, DP, CHUNK>(a, block, half);
  } else if (!b.whole) {
    join_items<DT, DP, CHUNK>(b, block - half, half);
  }
}

}  // namespace
