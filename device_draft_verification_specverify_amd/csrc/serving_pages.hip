// serving_pages.hip -- pages of a cache taken, given back and shared (gfx950).
//
// Integer work between the model's forward passes: what it costs is launches and
// trips to memory that wait for each other. What is given back needs a decision
// over all requests (a page comes free when as many give it back as hold it) and an
// order that does not depend on which of them comes first, so it is counted by page
// and listed by page id.

#include "specverify_serving.h"
#include "tree_common.h"

namespace {

using namespace svtree;

constexpr int kBlock = 256;
constexpr int kWaves = kBlock / kWave;
constexpr int kPagesEach = 4;                     // pages of a thread
constexpr int kPagesBlock = kBlock * kPagesEach;  // 1024

__device__ __forceinline__ int64_t sum_block(int64_t x, int64_t* box) {
  const int tid = int(threadIdx.x);
  for (int d = kWave / 2; d >= 1; d /= 2) x += __shfl_xor(x, d);
  __syncthreads();
  if (tid % kWave == 0) box[tid / kWave] = x;
  __syncthreads();
  x = 0;
  for (int w = 0; w < kWaves; ++w) x += box[w];
  return x;
}

struct ResizeArgs {
  const int32_t* prefix_len;
  const int32_t* chunk_start;
  const int32_t* pages_in;
  int32_t* table;
  int32_t* free_pages;
  const int32_t* head_in;
  const int32_t* shares_in;
  int64_t B, T, table_stride, num_pages, num_free, max_pages, blocks;
  int page_shift;
  int32_t* pages_out;
  int32_t* head_out;
  int32_t* shares_out;
  int32_t* position;
  int64_t* slots;
  int32_t* err;
  // workspace
  uint32_t* given;  // [num_pages] how many give the page back
  int32_t* counts;  // [blocks] pages that come free, then whether a chunk is wrong
};

// What request b holds and is to hold.
struct Hold {
  int64_t first;
  int32_t len, n, owned, need;
  int bits;  // errors: it keeps what it owns
};
__device__ __forceinline__ Hold hold_of(const ResizeArgs& a, int64_t b) {
  Hold r;
  r.len = a.prefix_len[b];
  r.owned = a.pages_in[b];
  r.first = 0;
  r.n = 0;
  r.bits = 0;
  if (a.chunk_start) {
    const Nodes nd = nodes_of(a.chunk_start, b, a.T, INT_MAX);
    r.first = nd.first;
    r.n = nd.n < 0 ? 0 : nd.n;
    if (nd.n < 0) r.bits |= SV_ERR_TREE;
  }
  const int64_t page = int64_t(1) << a.page_shift;
  const int64_t want = (int64_t(r.len) + r.n + page - 1) >> a.page_shift;
  if (r.len < 0 || r.owned < 0 || r.owned > a.max_pages ||
      (int64_t(r.owned) << a.page_shift) < r.len || want > a.max_pages)
    r.bits |= SV_ERR_LENGTH;
  r.need = r.bits ? r.owned : int32_t(want);
  return r;
}

// Whether a request behind b has the row, too (only where a chunk_start falls: the
// row is the last one's then).
__device__ bool later_has(const ResizeArgs& a, int64_t b, int64_t row) {
  for (int64_t o = b + 1; o < a.B; ++o) {
    const Hold h = hold_of(a, o);
    if (!h.bits && row >= h.first && row < h.first + h.n) return true;
  }
  return false;
}

__device__ __forceinline__ int64_t head_of(const ResizeArgs& a) {
  const int64_t head = *a.head_in;
  return head >= 0 && head <= a.num_free ? head : a.num_free;  // wrong: nothing is free
}

// ---- one workgroup does it all: few requests, a small cache

constexpr int kOne = 1024;
constexpr int kOneWaves = kOne / kWave;
constexpr int kOnePages = 16384;
constexpr int kOneEach = kOnePages / kOne;
constexpr int64_t kOneRows = 16384;

// The sum of x over the threads before this one, and over all.
__device__ __forceinline__ int32_t scan_one(int32_t x, int32_t* box, int32_t* all) {
  const int tid = int(threadIdx.x), lane = tid % kWave;
  int32_t upto = x;
  for (int d = 1; d < kWave; d *= 2) {
    const int32_t y = __shfl_up(upto, d);
    if (lane >= d) upto += y;
  }
  __syncthreads();
  if (lane == kWave - 1) box[tid / kWave] = upto;
  __syncthreads();
  int32_t before = upto - x;
  *all = 0;
  for (int w = 0; w < kOneWaves; ++w) {
    before += w < tid / kWave ? box[w] : 0;
    *all += box[w];
  }
  return before;
}

// The request that holds the k-th of what `front` counts in front of each.
__device__ __forceinline__ int find_one(const int32_t* front, int B, int32_t k) {
  int lo = 0, hi = B;  // front[lo] <= k < front[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (front[mid] <= k) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Each thread is a request, then what all requests give back, take and write is
// shared out over the threads entry by entry. Bound by the trips to memory one
// after another (lengths, entries, the pages' shares, the list): one request of 2048
// new tokens 8 us, a call 14.5 us; the four kernels below together are 23 us for 512
// requests, and their launches alone keep the host longer than this one runs.
__global__ __launch_bounds__(kOne) void resize_one_kernel(ResizeArgs a) {
  __shared__ uint32_t given[kOnePages];
  __shared__ uint16_t freed[kOnePages];  // the pages that come free, in order
  __shared__ int32_t gives[kOne], takes[kOne], rows[kOne];  // in front of each request
  __shared__ int32_t len[kOne], owned[kOne], need[kOne];
  __shared__ int32_t first[kOne];
  __shared__ uint8_t fit[kOne];
  __shared__ int32_t box[kOneWaves];
  __shared__ int32_t unfit;
  const int tid = int(threadIdx.x), B = int(a.B);
  const int64_t wrong_head = *a.head_in, head = head_of(a);
  int bits = wrong_head != head ? SV_ERR_PAGE : 0;
  Hold me{};
  if (tid < B) {
    me = hold_of(a, tid);
    len[tid] = me.len;
    owned[tid] = me.owned;
    need[tid] = me.need;
    first[tid] = int32_t(me.first);
  }
  bits |= me.bits;
  const int32_t give = me.owned > me.need ? me.owned - me.need : 0;
  const int32_t want = me.need > me.owned ? me.need - me.owned : 0;
  int32_t all_gives, all_takes, all_rows, all_freed;
  const int32_t gives_before = scan_one(give, box, &all_gives);
  const int32_t takes_before = scan_one(want, box, &all_takes);
  const int32_t rows_before = scan_one(me.bits ? 0 : me.n, box, &all_rows);
  gives[tid] = gives_before;
  takes[tid] = takes_before;
  rows[tid] = rows_before;
  for (int64_t p = tid; p < a.num_pages; p += kOne) given[p] = 0;
  for (int64_t i = tid; i < a.T; i += kOne) {
    a.position[i] = -1;
    a.slots[i] = -1;
  }
  if (tid == 0) unfit = B;
  const bool tangled = __syncthreads_or(me.bits & SV_ERR_TREE);
  for (int32_t k = tid; k < all_gives; k += kOne) {
    const int b = find_one(gives, B, k);
    const int64_t j = need[b] + k - gives[b];
    if (!sv_ok(j >= 0 && j < a.max_pages)) continue;
    const int32_t id = a.table[b * a.table_stride + j];
    if (id >= 0 && id < a.num_pages) atomicAdd(given + id, 1u);
    else bits |= SV_ERR_PAGE;
  }
  __syncthreads();
  uint32_t free = 0;
#pragma unroll
  for (int i = 0; i < kOneEach; ++i) {
    const int p = tid * kOneEach + i;
    if (p >= a.num_pages) break;
    const int64_t n = given[p], shares = a.shares_in ? a.shares_in[p] : 0;
    if (a.shares_out) a.shares_out[p] = int32_t(n > shares ? 0 : shares - n);
    if (n > 0 && n > shares) free |= 1u << i;
  }
  int32_t rank = scan_one(__popc(free), box, &all_freed);
  // (a list without room for what comes free holds pages twice: the rest is dropped)
  const int32_t room = int32_t(all_freed < head ? all_freed : head);
  if (room < all_freed) bits |= SV_ERR_PAGE;
  for (uint32_t f = free; f; f &= f - 1) {
    const int p = tid * kOneEach + __builtin_ctz(f);
    freed[rank] = uint16_t(p);
    if (rank < room && sv_ok(head - room + rank < a.num_free)) a.free_pages[head - room + rank] = p;
    ++rank;
  }
  const int64_t new_head = head - room, avail = a.num_free - new_head;
  // Sums of the pages only grow, so the requests within reach are a leading run.
  const bool reach = takes_before + int64_t(want) <= avail;
  if (tid < B) {
    fit[tid] = reach || want == 0;
    if (!fit[tid]) bits |= SV_ERR_PAGE;
    a.pages_out[tid] = want > 0 && !reach ? me.owned : me.need;
    if (!reach) atomicMin(&unfit, tid);
  }
  __syncthreads();
  const int32_t taken = unfit < B ? takes[unfit] : all_takes;
  if (tid == 0) *a.head_out = int32_t(new_head + taken);
  const auto page_of = [&](int64_t at) {  // place `at` of the list from its new head on
    if (at < room) return int32_t(freed[at]);
    return sv_ok(new_head + at < a.num_free) ? a.free_pages[new_head + at] : -1;
  };
  for (int32_t k = tid; k < taken; k += kOne) {
    const int b = find_one(takes, B, k);
    const int64_t j = int64_t(owned[b]) + k - takes[b];
    if (!sv_ok(j >= 0 && j < a.max_pages)) continue;
    const int32_t id = page_of(k);
    const bool good = id >= 0 && id < a.num_pages;
    a.table[b * a.table_stride + j] = good ? id : -1;
    if (!good) bits |= SV_ERR_PAGE;
  }
  for (int32_t k = tid; k < all_rows; k += kOne) {
    const int b = find_one(rows, B, k);
    const int32_t i = k - rows[b];
    const int64_t at = int64_t(len[b]) + i, pg = at >> a.page_shift;
    if (!sv_ok(first[b] + i < a.T && pg < a.max_pages)) continue;
    if (tangled && later_has(a, b, first[b] + i)) continue;
    int64_t slot = -1;
    if (fit[b]) {
      const int32_t id = pg < owned[b] ? a.table[b * a.table_stride + pg]
                                       : page_of(takes[b] + pg - owned[b]);
      if (id >= 0 && id < a.num_pages)
        slot = (int64_t(id) << a.page_shift) | (at & ((int64_t(1) << a.page_shift) - 1));
      else
        bits |= SV_ERR_PAGE;
    }
    a.position[first[b] + i] = int32_t(at);
    a.slots[first[b] + i] = slot;
  }
  // bits differ between threads: one atomic for each thread that saw an error
  if (bits) set_error(a.err, bits);
}

// ---- more of either: four launches

// Nothing given back yet, no row in a chunk yet.
__global__ __launch_bounds__(kBlock) void resize_clear_kernel(ResizeArgs a) {
  const int64_t step = int64_t(gridDim.x) * kBlock;
  for (int64_t i = int64_t(blockIdx.x) * kBlock + threadIdx.x; i < a.num_pages || i < a.T;
       i += step) {
    if (i < a.num_pages) a.given[i] = 0;
    if (i == 0) a.counts[a.blocks] = 0;
    if (i < a.T) {
      a.position[i] = -1;
      a.slots[i] = -1;
    }
  }
}

// A workgroup for each request.
__global__ __launch_bounds__(kBlock) void resize_count_kernel(ResizeArgs a) {
  const int64_t b = blockIdx.x;
  if (!sv_ok(b < a.B)) return;
  const Hold me = hold_of(a, b);
  const int32_t* row = a.table + b * a.table_stride;
  bool wrong = false;
  if ((me.bits & SV_ERR_TREE) && threadIdx.x == 0) atomicOr(a.counts + a.blocks, 1);
  for (int32_t j = me.need + int(threadIdx.x); j < me.owned; j += kBlock) {
    if (!sv_ok(j < a.max_pages)) continue;
    const int32_t id = row[j];
    if (id >= 0 && id < a.num_pages) atomicAdd(a.given + id, 1u);
    else wrong = true;
  }
  if (wrong) set_error(a.err, SV_ERR_PAGE);
}

// Whether page p comes free, and how many hold it beside the first afterwards.
__device__ __forceinline__ bool comes_free(const ResizeArgs& a, int64_t p, int32_t* left) {
  const int64_t given = a.given[p];
  const int64_t shares = a.shares_in ? a.shares_in[p] : 0;
  if (a.shares_in) *left = int32_t(given > shares ? 0 : shares - given);
  return given > 0 && given > shares;
}

// Pages of each block that come free. (Counted where they are given back, by the give
// that finds as many before it as hold the page, they would need no launch of their
// own, but the counters are so few that 40000 such additions took 56 us.)
__global__ __launch_bounds__(kBlock) void resize_sum_kernel(ResizeArgs a) {
  __shared__ int64_t box[kWaves];
  int32_t left;
  int mine = 0;
#pragma unroll
  for (int i = 0; i < kPagesEach; ++i) {
    const int64_t p = int64_t(blockIdx.x) * kPagesBlock + i * kBlock + threadIdx.x;
    if (p < a.num_pages) mine += comes_free(a, p, &left);
  }
  const int64_t sum = sum_block(mine, box);
  if (threadIdx.x == 0 && sv_ok(blockIdx.x < a.blocks)) a.counts[blockIdx.x] = int32_t(sum);
}

// Pages that come free, all of them, and the block that holds the rank-th with the
// number in front of it (counts are read twice rather than kept: there are few).
struct Freed {
  int64_t all, before;
};
__device__ __forceinline__ Freed freed_of(const ResizeArgs& a, int64_t block, int64_t* box) {
  int64_t all = 0, before = 0;
  for (int64_t i = threadIdx.x; i < a.blocks; i += kBlock) {
    const int32_t n = a.counts[i];
    all += n;
    before += i < block ? n : 0;
  }
  Freed r;
  r.all = sum_block(all, box);
  r.before = sum_block(before, box);
  return r;
}

// Calls f(page, rank) for the pages of a block that come free, `rank` of which are in
// front of it; `each` is called for every page of it with what is left of its shares.
template <typename F, typename G>
__device__ __forceinline__ int64_t list_block(const ResizeArgs& a, int64_t block, int64_t rank,
                                              int32_t* waves, F f, G each) {
  const int tid = int(threadIdx.x), lane = tid % kWave;
  uint64_t ballot[kPagesEach];
#pragma unroll
  for (int i = 0; i < kPagesEach; ++i) {
    const int64_t p = block * kPagesBlock + i * kBlock + tid;
    int32_t left = 0;
    const bool free = p < a.num_pages && comes_free(a, p, &left);
    if (p < a.num_pages) each(p, left);
    ballot[i] = __ballot(free);
  }
  __syncthreads();
  if (lane == 0)
#pragma unroll
    for (int i = 0; i < kPagesEach; ++i) waves[i * kWaves + tid / kWave] = __popcll(ballot[i]);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kPagesEach; ++i) {
    int64_t at = rank + __popcll(ballot[i] & ((uint64_t(1) << lane) - 1));
    for (int w = 0; w < kWaves; ++w) {
      at += w < tid / kWave ? waves[i * kWaves + w] : 0;
      rank += waves[i * kWaves + w];
    }
    if (ballot[i] >> lane & 1) f(block * kPagesBlock + i * kBlock + tid, at);
  }
  return rank;
}

// The first workgroups list what comes free, a block of pages each; the others are
// requests, `spread` workgroups each that share out the rows. A request that takes
// pages which come free in this call finds them by going through their blocks itself:
// the list is not there yet.
__global__ __launch_bounds__(kBlock) void resize_move_kernel(ResizeArgs a, int spread) {
  __shared__ int64_t box[kWaves];
  __shared__ int32_t waves[kPagesEach * kWaves];
  const int tid = int(threadIdx.x);
  const int64_t old_head = head_of(a);
  if (blockIdx.x < a.blocks) {
    const Freed freed = freed_of(a, blockIdx.x, box);
    // (a list without room for what comes free holds pages twice: the rest is dropped)
    const int64_t room = freed.all < old_head ? freed.all : old_head;
    if (blockIdx.x == 0 && tid == 0 && (room < freed.all || *a.head_in != old_head))
      set_error(a.err, SV_ERR_PAGE);
    list_block(a, blockIdx.x, freed.before, waves,
               [&](int64_t p, int64_t at) {
                 if (at < room && sv_ok(old_head - room + at < a.num_free))
                   a.free_pages[old_head - room + at] = int32_t(p);
               },
               [&](int64_t p, int32_t left) {
                 if (a.shares_out) a.shares_out[p] = left;
               });
    return;
  }
  const int64_t unit = int64_t(blockIdx.x) - a.blocks, b = unit / spread;
  const int part = int(unit % spread);
  if (!sv_ok(b < a.B)) return;
  const Hold me = hold_of(a, b);
  const Freed freed = freed_of(a, 0, box);
  const int64_t room = freed.all < old_head ? freed.all : old_head;
  const int64_t head = old_head - room, avail = a.num_free - head;

  int64_t sum = 0;
  for (int64_t o = tid; o < b; o += kBlock) {
    const Hold h = hold_of(a, o);
    sum += h.need > h.owned ? h.need - h.owned : 0;
  }
  const int64_t before = sum_block(sum, box);
  const int64_t want = me.need > me.owned ? me.need - me.owned : 0;
  // Sums of the pages only grow, so the requests within reach are a leading run.
  const bool reach = before + want <= avail;
  const bool fits = reach || want == 0;
  const int64_t more = reach ? want : 0;
  int bits = me.bits;
  if (!fits) bits |= SV_ERR_PAGE;
  if (tid == 0 && part == 0) {
    a.pages_out[b] = want > 0 ? int32_t(me.owned + more) : me.need;
    bool last = reach && b + 1 == a.B;
    if (reach && !last) {
      const Hold next = hold_of(a, b + 1);
      last = before + want + (next.need > next.owned ? next.need - next.owned : 0) > avail;
    }
    if (last) *a.head_out = int32_t(head + before + want);
    else if (b == 0 && !reach) *a.head_out = int32_t(head);
  }
  // Its pages (each of its workgroups writes them all, the same): those that come free now ...
  int32_t* row = a.table + b * a.table_stride;
  if (more > 0 && before < room) {
    int64_t rank = 0;
    for (int64_t i = 0; i < a.blocks && rank < before + more && rank < room; ++i) {
      const int32_t n = a.counts[i];
      if (rank + n > before)
        list_block(a, i, rank, waves,
                   [&](int64_t p, int64_t at) {
                     if (at >= before && at < before + more && at < room &&
                         sv_ok(me.owned + at - before < a.max_pages))
                       row[me.owned + at - before] = int32_t(p);
                   },
                   [](int64_t, int32_t) {});
      rank += n;
    }
  }
  // ... and those that were in the list
  for (int64_t j = (room > before ? room - before : 0) + tid; j < more; j += kBlock) {
    if (!sv_ok(me.owned + j < a.max_pages && head + before + j < a.num_free)) continue;
    const int32_t id = a.free_pages[head + before + j];
    const bool good = id >= 0 && id < a.num_pages;
    row[me.owned + j] = good ? id : -1;
    if (!good) bits |= SV_ERR_PAGE;
  }
  __syncthreads();
  const bool tangled = a.counts[a.blocks] != 0;
  if (!me.bits)
    for (int64_t i = part * kBlock + tid; i < me.n; i += int64_t(spread) * kBlock) {
      const int64_t at = int64_t(me.len) + i, pg = at >> a.page_shift;
      if (!sv_ok(me.first + i < a.T && pg < a.max_pages)) continue;
      if (tangled && later_has(a, b, me.first + i)) continue;
      int64_t slot = -1;
      if (fits) {
        const int32_t id = row[pg];
        if (id >= 0 && id < a.num_pages)
          slot = (int64_t(id) << a.page_shift) | (at & ((int64_t(1) << a.page_shift) - 1));
        else
          bits |= SV_ERR_PAGE;
      }
      a.position[me.first + i] = int32_t(at);
      a.slots[me.first + i] = slot;
    }
  // bits differ between threads: one atomic for each thread that saw an error
  if (bits && (tid == 0 || (bits & SV_ERR_PAGE))) set_error(a.err, bits);
}

struct ForkArgs {
  const int32_t* source;
  const int32_t* target;
  const int32_t* len_in;
  const int32_t* pages_in;
  int32_t* table;
  const int32_t* free_pages;
  const int32_t* head_in;
  const int32_t* shares_in;
  char* k_cache;
  char* v_cache;
  int64_t c_l, c_page, c_token, c_h;  // bytes
  int64_t forks, B, layers, num_pages, num_free, max_pages, table_stride;
  int H, chunks, page_shift;  // chunks: 16-byte pieces of a head
  int32_t* len_out;
  int32_t* pages_out;
  int32_t* head_out;
  int32_t* shares_out;
  int32_t* err;
  // workspace
  int32_t* named;  // [B] the first fork whose target the request is
  int32_t* plans;  // [forks][4]: tokens (< 0: passed by), page to copy from, page to copy to,
                   // place in the table of the page taken (< 0: none)
};

constexpr int kNamed = 8192;  // requests of which `named` is held in LDS

// What fork j is about: its errors, and the tokens that it shares.
struct Fork {
  int32_t s, t, len;
  bool part;  // its last page is not full: it takes one
  int bits;
};
__device__ __forceinline__ Fork fork_of(const ForkArgs& a, const int32_t* named, int64_t j) {
  Fork f;
  f.s = a.source[j];
  f.t = a.target[j];
  f.len = 0;
  f.part = false;
  f.bits = SV_ERR_REQUEST;
  if (f.s < 0 || f.s >= a.B || f.t < 0 || f.t >= a.B || f.s == f.t) return f;
  if (a.pages_in[f.t] != 0 || a.len_in[f.t] != 0 ||
      __hip_atomic_load(named + f.t, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) != j)
    return f;
  f.bits = SV_ERR_LENGTH;
  const int32_t len = a.len_in[f.s];
  const int64_t owned = a.pages_in[f.s];
  if (len < 0 || owned < 0 || owned > a.max_pages || (owned << a.page_shift) < len) return f;
  f.bits = 0;
  f.len = len;
  f.part = (len & ((1 << a.page_shift) - 1)) != 0;
  return f;
}

// The first workgroup settles what every fork does, a thread each, in order; the
// others copy the arrays that the next launch changes in places. (With a launch of
// its own for each of these, and one for the tables, a call for four replies to one
// prompt took 22.5 us rather than 19.6.)
__global__ __launch_bounds__(kOne) void fork_plan_kernel(ForkArgs a) {
  const int tid = int(threadIdx.x);
  if (blockIdx.x > 0) {
    const int64_t step = int64_t(gridDim.x - 1) * kOne;
    for (int64_t i = int64_t(blockIdx.x - 1) * kOne + tid; i < a.num_pages || i < a.B; i += step) {
      if (i < a.num_pages) a.shares_out[i] = a.shares_in[i];
      if (i < a.B) {
        a.len_out[i] = a.len_in[i];
        a.pages_out[i] = a.pages_in[i];
      }
    }
    return;
  }
  __shared__ int32_t held[kNamed];
  __shared__ int32_t box[kOneWaves];
  int32_t* const named = a.B <= kNamed ? held : a.named;
  for (int64_t i = tid; i < a.B; i += kOne)
    __hip_atomic_store(named + i, INT_MAX, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __syncthreads();
  for (int64_t j = tid; j < a.forks; j += kOne) {
    const int32_t t = a.target[j];
    if (t >= 0 && t < a.B) atomicMin(named + t, int32_t(j));
  }
  __threadfence_block();
  __syncthreads();
  const int64_t head = *a.head_in;
  const bool good_head = head >= 0 && head <= a.num_free;
  const int64_t avail = good_head ? a.num_free - head : 0;
  int bits = a.forks > 0 && !good_head ? SV_ERR_PAGE : 0;
  int64_t before = 0;  // pages that the forks of the rounds before want
  for (int64_t j0 = 0; j0 < a.forks; j0 += kOne) {
    const int64_t j = j0 + tid;
    Fork f{};
    if (j < a.forks) f = fork_of(a, named, j);
    bits |= f.bits;
    const int32_t want = f.part ? 1 : 0;
    int32_t all;
    const int64_t at = before + scan_one(want, box, &all);
    // Sums of the pages only grow, so the forks within reach are a leading run.
    if (j < a.forks) {
      const bool done = f.bits == 0 && (want == 0 || at + want <= avail);
      if (f.bits == 0 && !done) bits |= SV_ERR_PAGE;
      int32_t from = -1, to = -1, place = -1;
      if (done && want) {
        place = f.len >> a.page_shift;
        if (sv_ok(place < a.max_pages && head + at < a.num_free)) {
          from = a.table[f.s * a.table_stride + place];
          to = a.free_pages[head + at];
        }
        if (from < 0 || from >= a.num_pages) from = -1;
        if (to < 0 || to >= a.num_pages) to = -1;
        if (from < 0 || to < 0) bits |= SV_ERR_PAGE;
      }
      int32_t* plan = a.plans + 4 * j;
      plan[0] = done ? f.len : -1;
      plan[1] = from;
      plan[2] = to;
      plan[3] = place;
    }
    before += all;
  }
  if (tid == 0) *a.head_out = int32_t(head + (before < avail ? before : avail));
  if (bits) set_error(a.err, bits);
}

// One workgroup per (fork, layer): the tokens of the last page, keys and values; that
// of the first layer writes the target's table too. 64 forks of some 16 tokens in 32
// layers (245 MB, many of one source): 35 us, and a call 60 us.
__global__ __launch_bounds__(kBlock) void fork_copy_kernel(ForkArgs a) {
  const int64_t block = int64_t(blockIdx.y) * gridDim.x + blockIdx.x;
  const int64_t j = block % a.forks, layer = block / a.forks;
  if (layer >= a.layers) return;
  const int32_t* plan = a.plans + 4 * j;
  const int32_t len = plan[0], old_page = plan[1], new_page = plan[2], place = plan[3];
  if (len < 0) return;
  if (layer == 0) {
    const int32_t s = a.source[j], t = a.target[j], full = len >> a.page_shift;
    if (!sv_ok(s >= 0 && s < a.B && t >= 0 && t < a.B && full <= a.max_pages)) return;
    bool wrong = false;
    for (int32_t i = int(threadIdx.x); i < full; i += kBlock) {
      const int32_t id = a.table[s * a.table_stride + i];
      const bool good = id >= 0 && id < a.num_pages;
      a.table[t * a.table_stride + i] = good ? id : -1;
      if (good) atomicAdd(a.shares_out + id, 1);  // whole numbers: any order
      else wrong = true;
    }
    if (wrong) set_error(a.err, SV_ERR_PAGE);
    if (threadIdx.x == 0) {
      a.len_out[t] = len;
      a.pages_out[t] = full + (place >= 0 ? 1 : 0);
      if (place >= 0) a.table[t * a.table_stride + place] = new_page;
    }
  }
  if (old_page < 0 || new_page < 0) return;
  const int64_t from = layer * a.c_l + old_page * a.c_page, to = layer * a.c_l + new_page * a.c_page;
  const int per_token = a.H * a.chunks, all = (len & ((1 << a.page_shift) - 1)) * per_token;
  constexpr int AHEAD = 4;
  for (int i0 = int(threadIdx.x); i0 < all; i0 += kBlock * AHEAD) {
    u32x4 k[AHEAD], v[AHEAD];
    int64_t at[AHEAD];
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      const int i = i0 + u * kBlock < all ? i0 + u * kBlock : i0;
      const int token = i / per_token, in = i - token * per_token;
      const int h = in / a.chunks, piece = in - h * a.chunks;
      at[u] = token * a.c_token + h * a.c_h + piece * 16;
      k[u] = *reinterpret_cast<const u32x4*>(a.k_cache + from + at[u]);
      v[u] = *reinterpret_cast<const u32x4*>(a.v_cache + from + at[u]);
    }
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      if (i0 + u * kBlock >= all) break;
      *reinterpret_cast<u32x4*>(a.k_cache + to + at[u]) = k[u];
      *reinterpret_cast<u32x4*>(a.v_cache + to + at[u]) = v[u];
    }
  }
}

bool pages_ok(int64_t B, int64_t page_size, int64_t max_pages, int64_t table_stride,
              int64_t num_pages, int64_t num_free) {
  const int64_t k31 = int64_t(1) << 31;
  return B >= 1 && B <= SV_MAX_PAGE_BATCH && pow2(page_size) && page_size < k31 && max_pages >= 1 &&
         max_pages < k31 && max_pages * page_size < k31 && num_pages >= 1 &&
         num_pages <= SV_MAX_CACHE_PAGES && num_free >= 0 && num_free < k31 &&
         table_stride >= max_pages && stride_ok(table_stride);
}

unsigned blocks_for(int64_t n) {
  const int64_t most = 1024;  // four to a CU: small arrays, and clearing is no more than that
  const int64_t b = (n + kBlock - 1) / kBlock;
  return unsigned(b < 1 ? 1 : b > most ? most : b);
}

}  // namespace

#ifdef SV_DEVICE_CHECKS
bool sv_add_serving_pages_checks(uint32_t* count, int reset) { return sv_add_checks(count, reset); }
#endif

extern "C" {

size_t specverify_pages_resize_workspace_size(int64_t B, int64_t num_pages) {
  if (B < 1 || B > SV_MAX_PAGE_BATCH || num_pages < 1 || num_pages > SV_MAX_CACHE_PAGES) return 0;
  const int64_t blocks = (num_pages + kPagesBlock - 1) / kPagesBlock;
  return align256(size_t(num_pages) * 4) + align256(size_t(blocks + 1) * 4);
}

int specverify_pages_resize(const int32_t* prefix_len, const int32_t* chunk_start,
                            const int32_t* pages_in, int32_t* block_table, int32_t* free_pages,
                            const int32_t* free_head_in, const int32_t* shares_in, int64_t B,
                            int64_t T, int64_t page_size, int64_t max_pages, int64_t table_stride,
                            int64_t num_pages, int64_t num_free, int32_t* pages_out,
                            int32_t* free_head_out, int32_t* shares_out, int32_t* position,
                            int64_t* slots, int32_t* device_error, void* workspace,
                            size_t workspace_bytes, void* stream) {
  if (!prefix_len || !pages_in || !block_table || !free_pages || !free_head_in || !pages_out ||
      !free_head_out)
    return SV_EINVAL;
  if (T < 0 || T >= (int64_t(1) << 31) || (T > 0 && (!chunk_start || !position || !slots)))
    return SV_EINVAL;
  if (!pages_ok(B, page_size, max_pages, table_stride, num_pages, num_free) ||
      num_free < num_pages || B * max_pages >= (int64_t(1) << 40))
    return SV_EINVAL;
  if ((shares_in == nullptr) != (shares_out == nullptr) || pages_out == pages_in ||
      free_head_out == free_head_in || (shares_in && shares_out == shares_in))
    return SV_EINVAL;
  int status = SV_OK;
  if (!workspace_ok(workspace, workspace_bytes, specverify_pages_resize_workspace_size(B, num_pages),
                    &status))
    return status;
  ResizeArgs a{};
  a.prefix_len = prefix_len;
  a.chunk_start = chunk_start;
  a.pages_in = pages_in;
  a.table = block_table;
  a.free_pages = free_pages;
  a.head_in = free_head_in;
  a.shares_in = shares_in;
  a.B = B;
  a.T = T;
  a.table_stride = table_stride;
  a.num_pages = num_pages;
  a.num_free = num_free;
  a.max_pages = max_pages;
  a.blocks = (num_pages + kPagesBlock - 1) / kPagesBlock;
  a.page_shift = log2_of(page_size);
  a.pages_out = pages_out;
  a.head_out = free_head_out;
  a.shares_out = shares_out;
  a.position = position;
  a.slots = slots;
  a.err = device_error;
  a.given = static_cast<uint32_t*>(workspace);
  a.counts = reinterpret_cast<int32_t*>(static_cast<char*>(workspace) +
                                        align256(size_t(num_pages) * 4));
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  if (B <= kOne && num_pages <= kOnePages && T <= kOneRows &&
      B * max_pages < (int64_t(1) << 31)) {
    hipLaunchKernelGGL(resize_one_kernel, dim3(1), dim3(kOne), 0, st, a);
    return launch_status();
  }
  // workgroups of a request: one for some 512 rows of it
  const int64_t rows = T / (B * kBlock * 2) + 1;
  const int spread = int(rows < 64 ? rows : 64);
  hipLaunchKernelGGL(resize_clear_kernel, dim3(blocks_for(num_pages > T ? num_pages : T)),
                     dim3(kBlock), 0, st, a);
  hipLaunchKernelGGL(resize_count_kernel, dim3(unsigned(B)), dim3(kBlock), 0, st, a);
  hipLaunchKernelGGL(resize_sum_kernel, dim3(unsigned(a.blocks)), dim3(kBlock), 0, st, a);
  hipLaunchKernelGGL(resize_move_kernel, dim3(unsigned(a.blocks + B * spread)), dim3(kBlock), 0, st,
                     a, spread);
  return launch_status();
}

size_t specverify_pages_fork_workspace_size(int64_t B, int64_t forks) {
  if (B < 1 || B > SV_MAX_PAGE_BATCH || forks < 0 || forks > SV_MAX_PAGE_BATCH) return 0;
  return align256(size_t(B) * 4) + align256(size_t(forks) * 16);
}

int specverify_pages_fork(const int32_t* source, const int32_t* target,
                          const int32_t* prefix_len_in, const int32_t* pages_in,
                          int32_t* block_table, const int32_t* free_pages,
                          const int32_t* free_head_in, const int32_t* shares_in, void* k_cache,
                          void* v_cache, int dtype, int64_t forks, int64_t B, int64_t layers,
                          int64_t H, int64_t D, int64_t c_stride_l, int64_t c_stride_page,
                          int64_t c_stride_token, int64_t c_stride_h, int64_t page_size,
                          int64_t max_pages, int64_t table_stride, int64_t num_pages,
                          int64_t num_free, int32_t* prefix_len_out, int32_t* pages_out,
                          int32_t* free_head_out, int32_t* shares_out, int32_t* device_error,
                          void* workspace, size_t workspace_bytes, void* stream) {
  if (!prefix_len_in || !pages_in || !block_table || !free_pages || !free_head_in || !shares_in ||
      !k_cache || !v_cache || !prefix_len_out || !pages_out || !free_head_out || !shares_out)
    return SV_EINVAL;
  if (forks < 0 || forks > SV_MAX_PAGE_BATCH || (forks > 0 && (!source || !target)))
    return SV_EINVAL;
  const int64_t k31 = int64_t(1) << 31;
  if (!pages_ok(B, page_size, max_pages, table_stride, num_pages, num_free) || layers < 1 ||
      layers >= k31 || layers * forks >= k31 || H < 1 || H >= (1 << 16) || D < 8 ||
      D > SV_MAX_HEAD_DIM || D % 8 != 0)
    return SV_EINVAL;
  if (prefix_len_out == prefix_len_in || pages_out == pages_in || free_head_out == free_head_in ||
      shares_out == shares_in)
    return SV_EINVAL;
  const int64_t strides[] = {c_stride_l, c_stride_page, c_stride_token, c_stride_h};
  for (int64_t s : strides)
    if (!stride_ok(s)) return SV_EINVAL;
  if (dtype != SV_F32 && dtype != SV_BF16 && dtype != SV_F16) return SV_EDTYPE;
  const int size = dtype == SV_F32 ? 4 : 2;
  for (int64_t s : strides)
    if (s * size % 16 != 0) return SV_EALIGN;
  if (!aligned16(k_cache) || !aligned16(v_cache)) return SV_EALIGN;
  const int64_t sizes[] = {layers, num_pages, page_size, H};
  if (!apart(4, sizes, strides, D)) return SV_EINVAL;
  // (pieces of a page are counted in 32 bits)
  if (page_size * H * (D * size / 16) >= k31) return SV_EINVAL;
  int status = SV_OK;
  if (!workspace_ok(workspace, workspace_bytes, specverify_pages_fork_workspace_size(B, forks),
                    &status))
    return status;
  ForkArgs a{};
  a.source = source;
  a.target = target;
  a.len_in = prefix_len_in;
  a.pages_in = pages_in;
  a.table = block_table;
  a.free_pages = free_pages;
  a.head_in = free_head_in;
  a.shares_in = shares_in;
  a.k_cache = static_cast<char*>(k_cache);
  a.v_cache = static_cast<char*>(v_cache);
  a.c_l = c_stride_l * size;
  a.c_page = c_stride_page * size;
  a.c_token = c_stride_token * size;
  a.c_h = c_stride_h * size;
  a.forks = forks;
  a.B = B;
  a.layers = layers;
  a.num_pages = num_pages;
  a.num_free = num_free;
  a.max_pages = max_pages;
  a.table_stride = table_stride;
  a.H = int(H);
  a.chunks = int(D * size / 16);
  a.page_shift = log2_of(page_size);
  a.len_out = prefix_len_out;
  a.pages_out = pages_out;
  a.head_out = free_head_out;
  a.shares_out = shares_out;
  a.err = device_error;
  a.named = static_cast<int32_t*>(workspace);
  a.plans = reinterpret_cast<int32_t*>(static_cast<char*>(workspace) + align256(size_t(B) * 4));
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  const int64_t copied = num_pages > B ? num_pages : B;
  const int64_t copiers = (copied + kOne * 4 - 1) / (kOne * 4);
  hipLaunchKernelGGL(fork_plan_kernel, dim3(unsigned(1 + (copiers < 512 ? copiers : 512))),
                     dim3(kOne), 0, st, a);
  if (forks > 0) {
    // (threads along x are counted in 32 bits)
    const int64_t pieces = forks * layers, most = 1 << 22, x = pieces < most ? pieces : most;
    hipLaunchKernelGGL(fork_copy_kernel, dim3(unsigned(x), unsigned((pieces + x - 1) / x)),
                       dim3(kBlock), 0, st, a);
  }
  return launch_status();
}

}  // extern "C"
