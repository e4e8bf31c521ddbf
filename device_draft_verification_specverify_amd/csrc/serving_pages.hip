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
constexpr int kPagesEach = 16;                   // consecutive pages of a thread
constexpr int kPagesBlock = kBlock * kPagesEach;  // 4096

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
  int32_t* counts;  // [blocks] pages that come free
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

__device__ __forceinline__ int64_t head_of(const ResizeArgs& a) {
  const int64_t head = *a.head_in;
  return head >= 0 && head <= a.num_free ? head : a.num_free;  // wrong: nothing is free
}

// Nothing given back yet, no row in a chunk yet.
__global__ __launch_bounds__(kBlock) void resize_clear_kernel(ResizeArgs a) {
  const int64_t step = int64_t(gridDim.x) * kBlock;
  for (int64_t i = int64_t(blockIdx.x) * kBlock + threadIdx.x; i < a.num_pages || i < a.T;
       i += step) {
    if (i < a.num_pages) a.given[i] = 0;
    if (i < a.T) {
      a.position[i] = -1;
      a.slots[i] = -1;
    }
  }
}

__global__ __launch_bounds__(kBlock) void resize_count_kernel(ResizeArgs a) {
  const int64_t b = blockIdx.x;
  if (!sv_ok(b < a.B)) return;
  const Hold me = hold_of(a, b);
  const int32_t* row = a.table + b * a.table_stride;
  bool wrong = false;
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

__global__ __launch_bounds__(kBlock) void resize_sum_kernel(ResizeArgs a) {
  __shared__ int64_t box[kWaves];
  const int64_t p0 = int64_t(blockIdx.x) * kPagesBlock;
  int32_t left;
  int mine = 0;
  for (int i = 0; i < kPagesEach; ++i) {
    const int64_t p = p0 + i * kBlock + threadIdx.x;
    if (p < a.num_pages) mine += comes_free(a, p, &left);
  }
  const int64_t sum = sum_block(mine, box);
  if (threadIdx.x == 0 && sv_ok(blockIdx.x < a.blocks)) a.counts[blockIdx.x] = int32_t(sum);
}

// Pages that come free, all of them and those of the blocks before `block`.
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

__global__ __launch_bounds__(kBlock) void resize_free_kernel(ResizeArgs a) {
  __shared__ int64_t box[kWaves];
  __shared__ int32_t waves[kWaves];
  const int tid = int(threadIdx.x), lane = tid % kWave;
  const Freed freed = freed_of(a, blockIdx.x, box);
  const int64_t head = head_of(a);
  // (a list without room for what comes free holds pages twice: the rest is dropped)
  const int64_t room = freed.all < head ? freed.all : head;
  if (room < freed.all && blockIdx.x == 0 && tid == 0) set_error(a.err, SV_ERR_PAGE);
  int64_t rank = freed.before;
  for (int i = 0; i < kPagesEach; ++i) {
    const int64_t p = int64_t(blockIdx.x) * kPagesBlock + i * kBlock + tid;
    int32_t left = 0;
    const bool free = p < a.num_pages && comes_free(a, p, &left);
    if (p < a.num_pages && a.shares_out) a.shares_out[p] = left;
    const uint64_t ballot = __ballot(free);
    __syncthreads();
    if (lane == 0) waves[tid / kWave] = __popcll(ballot);
    __syncthreads();
    int64_t at = rank + __popcll(ballot & ((uint64_t(1) << lane) - 1));
    for (int w = 0; w < kWaves; ++w) {
      at += w < tid / kWave ? waves[w] : 0;
      rank += waves[w];
    }
    if (free && at < room && sv_ok(head - room + at < a.num_free))
      a.free_pages[head - room + at] = int32_t(p);
  }
}

// A request's share of the takes; blockIdx.y shares its pages and rows out.
__global__ __launch_bounds__(kBlock) void resize_take_kernel(ResizeArgs a) {
  __shared__ int64_t box[kWaves];
  const int64_t b = blockIdx.x;
  const int tid = int(threadIdx.x);
  if (!sv_ok(b < a.B)) return;
  const Hold me = hold_of(a, b);
  const Freed freed = freed_of(a, 0, box);
  const int64_t old_head = head_of(a);
  const int64_t head = old_head - (freed.all < old_head ? freed.all : old_head);
  const int64_t avail = a.num_free - head;

  int64_t part = 0;
  for (int64_t o = tid; o < b; o += kBlock) {
    const Hold h = hold_of(a, o);
    part += h.need > h.owned ? h.need - h.owned : 0;
  }
  const int64_t before = sum_block(part, box);
  const int64_t want = me.need > me.owned ? me.need - me.owned : 0;
  // Sums of the pages only grow, so the requests within reach are a leading run.
  const bool reach = before + want <= avail;
  const bool fits = reach || want == 0;
  const int64_t more = reach ? want : 0;
  int bits = me.bits;
  if (!fits || (b == 0 && *a.head_in != old_head)) bits |= SV_ERR_PAGE;
  if (tid == 0 && blockIdx.y == 0) {
    a.pages_out[b] = want > 0 ? int32_t(me.owned + more) : me.need;
    bool last = reach && b + 1 == a.B;
    if (reach && !last) {
      const Hold next = hold_of(a, b + 1);
      last = before + want + (next.need > next.owned ? next.need - next.owned : 0) > avail;
    }
    if (last) *a.head_out = int32_t(head + before + want);
    else if (b == 0 && !reach) *a.head_out = int32_t(head);
  }
  int32_t* row = a.table + b * a.table_stride;
  const int from = int(blockIdx.y) * kBlock + tid, step = int(gridDim.y) * kBlock;
  for (int64_t j = from; j < more; j += step) {
    if (!sv_ok(me.owned + j < a.max_pages && head + before + j < a.num_free)) continue;
    const int32_t id = a.free_pages[head + before + j];
    const bool good = id >= 0 && id < a.num_pages;
    row[me.owned + j] = good ? id : -1;
    if (!good) bits |= SV_ERR_PAGE;
  }
  if (!me.bits)
    for (int64_t i = from; i < me.n; i += step) {
      const int64_t at = int64_t(me.len) + i, pg = at >> a.page_shift;
      if (!sv_ok(me.first + i < a.T && pg < a.max_pages)) continue;
      int64_t slot = -1;
      if (fits && sv_ok(pg < me.owned || head + before + pg - me.owned < a.num_free)) {
        const int32_t id = pg < me.owned ? row[pg] : a.free_pages[head + before + pg - me.owned];
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
  int32_t* copies; // [forks][3]: page to copy from, page to copy to, tokens
};

__global__ __launch_bounds__(kBlock) void fork_start_kernel(ForkArgs a) {
  const int64_t step = int64_t(gridDim.x) * kBlock;
  const int64_t at = int64_t(blockIdx.x) * kBlock + threadIdx.x;
  if (at == 0) *a.head_out = *a.head_in;
  for (int64_t i = at; i < a.num_pages; i += step) a.shares_out[i] = a.shares_in[i];
  for (int64_t i = at; i < a.B; i += step) {
    a.len_out[i] = a.len_in[i];
    a.pages_out[i] = a.pages_in[i];
    int32_t first = INT_MAX;
    for (int64_t j = a.forks - 1; j >= 0; --j) first = a.target[j] == i ? int32_t(j) : first;
    a.named[i] = first;
  }
}

// What fork j is about: its errors, and the tokens that it shares.
struct Fork {
  int32_t s, t, len, full, part;
  int bits;
};
__device__ __forceinline__ Fork fork_of(const ForkArgs& a, int64_t j) {
  Fork f;
  f.s = a.source[j];
  f.t = a.target[j];
  f.len = f.full = f.part = 0;
  f.bits = 0;
  if (f.s < 0 || f.s >= a.B || f.t < 0 || f.t >= a.B || f.s == f.t || a.pages_in[f.t] != 0 ||
      a.len_in[f.t] != 0 || a.named[f.t] != j) {
    f.bits = SV_ERR_REQUEST;
    return f;
  }
  f.len = a.len_in[f.s];
  const int64_t owned = a.pages_in[f.s];
  if (f.len < 0 || owned < 0 || owned > a.max_pages || (owned << a.page_shift) < f.len) {
    f.bits = SV_ERR_LENGTH;
    f.len = 0;
    return f;
  }
  f.full = f.len >> a.page_shift;
  f.part = f.len & ((1 << a.page_shift) - 1);
  return f;
}

// One workgroup per fork; the pages that forks before it take are summed by each.
__global__ __launch_bounds__(kBlock) void fork_kernel(ForkArgs a) {
  __shared__ int64_t box[kWaves];
  const int64_t j = blockIdx.x;
  const int tid = int(threadIdx.x);
  if (!sv_ok(j < a.forks)) return;
  const Fork me = fork_of(a, j);
  int64_t part = 0;
  for (int64_t o = tid; o < j; o += kBlock) part += fork_of(a, o).part > 0;
  const int64_t before = sum_block(part, box);
  const int64_t head = *a.head_in;
  const int64_t avail = head >= 0 && head <= a.num_free ? a.num_free - head : 0;
  const int want = me.part > 0;
  const bool reach = before + want <= avail;
  const bool done = me.bits == 0 && (reach || want == 0);
  int bits = me.bits;
  if (me.bits == 0 && !done) bits |= SV_ERR_PAGE;
  if (j == 0 && (head < 0 || head > a.num_free)) bits |= SV_ERR_PAGE;
  int32_t old_page = -1, new_page = -1;
  if (done && want) {
    if (sv_ok(me.full < a.max_pages && head + before < a.num_free)) {
      old_page = a.table[me.s * a.table_stride + me.full];
      new_page = a.free_pages[head + before];
    }
    if (new_page < 0 || new_page >= a.num_pages) new_page = -1;
    if (old_page < 0 || old_page >= a.num_pages) old_page = -1;
    if (new_page < 0 || old_page < 0) bits |= SV_ERR_PAGE;
  }
  if (tid == 0) {
    int32_t* c = a.copies + 3 * j;
    c[0] = old_page;
    c[1] = new_page;
    c[2] = old_page >= 0 && new_page >= 0 ? me.part : 0;
    if (done) {
      a.len_out[me.t] = me.len;
      a.pages_out[me.t] = me.full + want;
      if (want) a.table[me.t * a.table_stride + me.full] = new_page;
    }
    // the last fork within reach moves the head
    if (reach && (j + 1 == a.forks || before + want + (fork_of(a, j + 1).part > 0) > avail) &&
        before + want > 0)
      *a.head_out = int32_t(head + before + want);
  }
  if (done)
    for (int32_t i = tid; i < me.full; i += kBlock) {
      if (!sv_ok(i < a.max_pages)) continue;
      const int32_t id = a.table[me.s * a.table_stride + i];
      const bool good = id >= 0 && id < a.num_pages;
      a.table[me.t * a.table_stride + i] = good ? id : -1;
      if (good) atomicAdd(a.shares_out + id, 1);  // whole numbers: any order
      else bits |= SV_ERR_PAGE;
    }
  if (bits && (tid == 0 || (bits & SV_ERR_PAGE))) set_error(a.err, bits);
}

// One workgroup per (fork, layer): the tokens of the last page, keys and values.
__global__ __launch_bounds__(kBlock) void fork_copy_kernel(ForkArgs a) {
  const int64_t j = int64_t(blockIdx.x) % a.forks, layer = int64_t(blockIdx.x) / a.forks;
  if (!sv_ok(layer < a.layers)) return;
  const int32_t* c = a.copies + 3 * j;
  const int64_t from = layer * a.c_l + c[0] * a.c_page, to = layer * a.c_l + c[1] * a.c_page;
  const int per_token = a.H * a.chunks, all = c[2] * per_token;
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
  return align256(size_t(num_pages) * 4) + align256(size_t(blocks) * 4);
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
  const int64_t rows = T / (B * kBlock * 2) + 1;
  const dim3 takes(unsigned(B), unsigned(rows < 64 ? rows : 64));
  hipLaunchKernelGGL(resize_clear_kernel, dim3(blocks_for(num_pages > T ? num_pages : T)),
                     dim3(kBlock), 0, st, a);
  hipLaunchKernelGGL(resize_count_kernel, dim3(unsigned(B)), dim3(kBlock), 0, st, a);
  hipLaunchKernelGGL(resize_sum_kernel, dim3(unsigned(a.blocks)), dim3(kBlock), 0, st, a);
  hipLaunchKernelGGL(resize_free_kernel, dim3(unsigned(a.blocks)), dim3(kBlock), 0, st, a);
  hipLaunchKernelGGL(resize_take_kernel, takes, dim3(kBlock), 0, st, a);
  return launch_status();
}

size_t specverify_pages_fork_workspace_size(int64_t B, int64_t forks) {
  if (B < 1 || B > SV_MAX_PAGE_BATCH || forks < 0 || forks > SV_MAX_PAGE_BATCH) return 0;
  return align256(size_t(B) * 4) + align256(size_t(forks) * 12);
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
  a.copies = reinterpret_cast<int32_t*>(static_cast<char*>(workspace) + align256(size_t(B) * 4));
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  hipLaunchKernelGGL(fork_start_kernel, dim3(blocks_for(num_pages > B ? num_pages : B)),
                     dim3(kBlock), 0, st, a);
  if (forks > 0) {
    hipLaunchKernelGGL(fork_kernel, dim3(unsigned(forks)), dim3(kBlock), 0, st, a);
    hipLaunchKernelGGL(fork_copy_kernel, dim3(unsigned(forks * layers)), dim3(kBlock), 0, st, a);
  }
  return launch_status();
}

}  // extern "C"
