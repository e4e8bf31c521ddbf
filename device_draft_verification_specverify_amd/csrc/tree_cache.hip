// tree_cache.hip -- the plan and the commit of a drafted-tree step (gfx950).
//
// Both are small integer or copy work between the model's forward passes: what
// they cost is launches and latency, so each is one launch.

#include "tree_common.h"

namespace {

using namespace svtree;

constexpr int kPlanBlock = 256;
constexpr int kPlanWaves = kPlanBlock / kWave;

struct PlanArgs {
  const int32_t* parents;
  const int32_t* node_start;
  const int32_t* prefix_len;
  const int32_t* pages_in;
  int32_t* table;
  const int32_t* free_pages;
  const int32_t* head_in;
  int64_t B, T, table_stride, num_pages, num_free, max_pages;
  int max_nodes, max_path, page_shift, words;
  uint64_t* ancestors;
  int32_t* depth;
  int32_t* position;
  int64_t* slots;
  int32_t* pages_out;
  int32_t* head_out;
  int32_t* err;
};

// Pages that request b takes if the free list reaches (0 for wrong lengths).
struct Need {
  int32_t len, tokens, owned, more;
  bool ok;  // lengths
};
__device__ __forceinline__ Need need_of(const PlanArgs& a, int64_t b) {
  const Nodes nd = nodes_of(a.node_start, b, a.T, a.max_nodes);
  Need r;
  r.len = a.prefix_len[b];
  r.owned = a.pages_in[b];
  r.tokens = nd.n < 0 ? 0 : min(nd.n, a.max_path);
  r.more = 0;
  const int64_t page = int64_t(1) << a.page_shift;
  const int64_t want = (int64_t(r.len) + r.tokens + page - 1) >> a.page_shift;
  r.ok = r.len >= 0 && r.owned >= 0 && r.owned <= a.max_pages &&
         (int64_t(r.owned) << a.page_shift) >= r.len && want <= a.max_pages;
  if (r.ok && want > r.owned) r.more = int32_t(want - r.owned);
  return r;
}

// One workgroup per request. The pages in front of it are a sum over the
// requests before it, taken by every workgroup for itself (12 bytes a request
// out of the L2: at B = 512 a few loads a thread) rather than in a scan launch
// of its own. Ancestor masks come by pointer doubling: in round r a node holds
// the bits of its 2^r nearest ancestors and a pointer 2^r up, so 7 rounds do
// for 128 nodes whatever their shape. 512 requests of 33 nodes: 6.7 us, latency
// throughout (0.34 MB move).
__global__ __launch_bounds__(kPlanBlock) void plan_kernel(PlanArgs a) {
  const int64_t b = blockIdx.x;
  const int tid = int(threadIdx.x);
  if (!sv_ok(b < a.B)) return;
  const Nodes nd = nodes_of(a.node_start, b, a.T, a.max_nodes);
  const Need me = need_of(a, b);
  const int64_t head = *a.head_in;
  const int64_t avail = head >= 0 && head <= a.num_free ? a.num_free - head : 0;

  int64_t part = 0;
  for (int64_t o = tid; o < b; o += kPlanBlock) part += need_of(a, o).more;
  for (int d = kWave / 2; d >= 1; d /= 2) part += __shfl_xor(part, d);
  __shared__ int64_t wave_sum[kPlanWaves];
  if (tid % kWave == 0) wave_sum[tid / kWave] = part;
  __syncthreads();
  int64_t before = 0;
  for (int w = 0; w < kPlanWaves; ++w) before += wave_sum[w];

  // Sums of the pages only grow, so the requests within reach are a leading run.
  const bool reach = before + me.more <= avail;
  const bool fits = reach || me.more == 0;
  const int32_t more = reach ? me.more : 0;
  int bits = 0;
  if (!me.ok) bits |= SV_ERR_LENGTH;
  if (!fits || (b == 0 && (head < 0 || head > a.num_free))) bits |= SV_ERR_PAGE;
  if (nd.n < 0) bits |= SV_ERR_TREE;

  if (tid == 0) {
    a.pages_out[b] = me.owned + more;
    // the last request of that run moves the head
    if (reach && (b + 1 == a.B || before + me.more + need_of(a, b + 1).more > avail))
      *a.head_out = int32_t(head + before + me.more);
    else if (b == 0 && !reach)
      *a.head_out = int32_t(head);
  }

  int32_t* row = a.table + b * a.table_stride;
  for (int32_t j = tid; j < more; j += kPlanBlock) {
    if (!sv_ok(me.owned + j < a.max_pages && head + before + j < a.num_free)) continue;
    const int32_t id = a.free_pages[head + before + j];
    const bool good = id >= 0 && id < a.num_pages;
    row[me.owned + j] = good ? id : -1;
    if (!good) bits |= SV_ERR_PAGE;
  }

  // Topology: threads 0 .. n-1 hold a node each.
  __shared__ uint64_t mask[SV_MAX_TREE_NODES][2];
  __shared__ int32_t jump[SV_MAX_TREE_NODES];
  const int n = nd.n < 0 ? 0 : nd.n;
  const bool mine = tid < n;
  int32_t up = -1;
  bool wrong = false;
  uint64_t m0 = 0, m1 = 0;
  if (mine) {
    up = sv_ok(nd.first + tid < a.T) ? a.parents[nd.first + tid] : -1;
    wrong = tid == 0 ? up != -1 : (up < 0 || up >= tid);
    if (wrong) up = -1;
    (tid < 64 ? m0 : m1) = uint64_t(1) << (tid & 63);
  }
  bool bad_tree = __syncthreads_or(wrong) || nd.n < 0;
  while (true) {
    if (mine) {
      mask[tid][0] = m0;
      mask[tid][1] = m1;
      jump[tid] = up;
    }
    if (!__syncthreads_or(mine && up >= 0)) break;
    if (mine && up >= 0) {
      m0 |= mask[up][0];
      m1 |= mask[up][1];
      up = jump[up];
    }
    __syncthreads();
  }
  const int32_t deep = __popcll(m0) + __popcll(m1) - 1;
  bad_tree = __syncthreads_or(mine && deep >= a.max_path) || bad_tree;
  if (bad_tree) bits |= SV_ERR_TREE;
  if (mine && sv_ok(nd.first + tid < a.T)) {
    const int64_t i = nd.first + tid;
    a.ancestors[i * a.words] = bad_tree ? 0 : m0;
    if (a.words > 1) a.ancestors[i * a.words + 1] = bad_tree ? 0 : m1;
    a.depth[i] = bad_tree ? -1 : deep;
    a.position[i] = bad_tree || !me.ok ? -1 : me.len + deep;
  }

  for (int i = tid; i < a.max_path; i += kPlanBlock) {
    int64_t slot = -1;
    if (i < me.tokens && me.ok && fits && !bad_tree) {
      const int64_t at = int64_t(me.len) + i;
      const int64_t pg = at >> a.page_shift;
      if (!sv_ok(pg < a.max_pages && (pg < me.owned || head + before + pg - me.owned < a.num_free)))
        continue;
      const int32_t id = pg < me.owned ? row[pg] : a.free_pages[head + before + (pg - me.owned)];
      if (id >= 0 && id < a.num_pages)
        slot = (int64_t(id) << a.page_shift) | (at & ((int64_t(1) << a.page_shift) - 1));
      else
        bits |= SV_ERR_PAGE;
    }
    a.slots[b * a.max_path + i] = slot;
  }
  // bits differ between threads: one atomic for each thread that saw an error
  if (bits && (tid == 0 || (bits & SV_ERR_PAGE))) set_error(a.err, bits);
}

constexpr int kCommitBlock = 256;

struct CommitArgs {
  const char* k_tree;
  const char* v_tree;
  char* k_cache;
  char* v_cache;
  int64_t n_l, n_t, n_h, c_l, c_page, c_token, c_h;  // bytes
  int64_t B, T, slots_total;
  int H, chunks, max_nodes, max_path, page_shift;  // chunks: 16-byte pieces of a head
  const int32_t* node_start;
  const int32_t* path;
  const int32_t* accept_len;
  const int64_t* slots;
  const int32_t* len_in;
  int32_t* len_out;
  int32_t* err;
  int64_t layers;
};

// One workgroup per (request, layer): its threads take the 16-byte pieces of a
// token's keys and values, and each copies its piece of every accepted node,
// four loads in flight. 64 requests with 5 nodes in 32 layers (75 MB): 14.8 us, 5.1
// TB/s; one request in 4 layers: 3.4 us.
__global__ __launch_bounds__(kCommitBlock) void commit_kernel(CommitArgs a) {
  const int64_t b = int64_t(blockIdx.x) % a.B, layer = int64_t(blockIdx.x) / a.B;
  const int tid = int(threadIdx.x);
  if (!sv_ok(layer < a.layers)) return;
  __shared__ int64_t src[SV_MAX_TREE_NODES], dst[SV_MAX_TREE_NODES];
  const Nodes nd = nodes_of(a.node_start, b, a.T, a.max_nodes);
  const int32_t taken = a.accept_len[b];
  int bits = 0;
  if (taken >= 0) {
    if (nd.n < 1 || taken >= a.max_path) {
      bits = SV_ERR_TREE;
    } else if (tid <= taken) {
      const int32_t node = a.path[b * a.max_path + tid];
      const int64_t slot = a.slots[b * a.max_path + tid];
      if (node < 0 || node >= nd.n) bits |= SV_ERR_TREE;
      if (slot < 0 || slot >= a.slots_total) bits |= SV_ERR_PAGE;
      src[tid] = layer * a.n_l + (nd.first + node) * a.n_t;
      dst[tid] = layer * a.c_l + (slot >> a.page_shift) * a.c_page +
                 (slot & ((int64_t(1) << a.page_shift) - 1)) * a.c_token;
    }
  }
  if (layer == 0 && bits) set_error(a.err, bits);
  const bool skip = __syncthreads_or(bits != 0) || taken < 0;
  if (layer == 0 && tid == 0) a.len_out[b] = a.len_in[b] + (skip ? 0 : taken + 1);
  if (skip) return;
  const int per = a.H * a.chunks;
  for (int e = tid; e < 2 * per; e += kCommitBlock) {
    const bool val = e >= per;
    const int r = val ? e - per : e;
    const int h = r / a.chunks, c = r - h * a.chunks;
    if (!sv_ok(h < a.H && c >= 0 && nd.first + nd.n <= a.T)) continue;
    const char* from = (val ? a.v_tree : a.k_tree) + h * a.n_h + c * 16;
    char* to = (val ? a.v_cache : a.k_cache) + h * a.c_h + c * 16;
    for (int i = 0; i <= taken; i += 4) {
      u32x4 x[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (i + j <= taken) x[j] = *reinterpret_cast<const u32x4*>(from + src[i + j]);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (i + j <= taken) *reinterpret_cast<u32x4*>(to + dst[i + j]) = x[j];
    }
  }
}

bool under31(int64_t x) { return x < (int64_t(1) << 31); }

}  // namespace

#ifdef SV_DEVICE_CHECKS
bool sv_add_tree_cache_checks(uint32_t* count, int reset) { return sv_add_checks(count, reset); }
#endif

extern "C" {

int specverify_tree_plan(const int32_t* parents, const int32_t* node_start,
                         const int32_t* prefix_len, const int32_t* pages_in, int32_t* block_table,
                         const int32_t* free_pages, const int32_t* free_head_in, int64_t B,
                         int64_t T, int64_t max_nodes, int64_t max_path, int64_t page_size,
                         int64_t max_pages, int64_t table_stride, int64_t num_pages,
                         int64_t num_free, uint64_t* ancestors, int32_t* depth, int32_t* position,
                         int64_t* slots, int32_t* pages_out, int32_t* free_head_out,
                         int32_t* device_error, void* stream) {
  if (!node_start || !prefix_len || !pages_in || !block_table || !free_head_in || !slots ||
      !pages_out || !free_head_out || (num_free > 0 && !free_pages))
    return SV_EINVAL;
  if (T > 0 && (!parents || !ancestors || !depth || !position)) return SV_EINVAL;
  if (B < 1 || !under31(B) || T < 0 || !under31(T) || max_nodes < 1 ||
      max_nodes > SV_MAX_TREE_NODES || max_path < 1 || max_path > max_nodes)
    return SV_EINVAL;
  if (!pow2(page_size) || !under31(page_size) || max_pages < 1 || !under31(max_pages) ||
      num_pages < 1 || !under31(num_pages) || num_free < 0 || !under31(num_free) ||
      !under31(B * max_pages) || !under31(max_pages * page_size + max_nodes) ||
      table_stride < max_pages || !stride_ok(table_stride))
    return SV_EINVAL;
  if (pages_out == pages_in || free_head_out == free_head_in) return SV_EINVAL;
  PlanArgs a{parents,   node_start,   prefix_len, pages_in, block_table, free_pages, free_head_in,
             B,         T,            table_stride, num_pages, num_free, max_pages,
             int(max_nodes), int(max_path), log2_of(page_size), int((max_nodes + 63) / 64),
             ancestors, depth, position, slots, pages_out, free_head_out, device_error};
  hipLaunchKernelGGL(plan_kernel, dim3(unsigned(B)), dim3(kPlanBlock), 0,
                     reinterpret_cast<hipStream_t>(stream), a);
  return launch_status();
}

int specverify_tree_commit(const void* k_tree, const void* v_tree, void* k_cache, void* v_cache,
                           int dtype, int64_t layers, int64_t B, int64_t T, int64_t H, int64_t D,
                           int64_t max_nodes, int64_t max_path, int64_t n_stride_l,
                           int64_t n_stride_t, int64_t n_stride_h, int64_t c_stride_l,
                           int64_t c_stride_page, int64_t c_stride_token, int64_t c_stride_h,
                           int64_t num_pages, int64_t page_size, const int32_t* node_start,
                           const int32_t* path, const int32_t* accept_len, const int64_t* slots,
                           const int32_t* prefix_len_in, int32_t* prefix_len_out,
                           int32_t* device_error, void* stream) {
  if (!k_cache || !v_cache || !node_start || !path || !accept_len || !slots || !prefix_len_in ||
      !prefix_len_out || (T > 0 && (!k_tree || !v_tree)))
    return SV_EINVAL;
  if (layers < 1 || !under31(layers) || B < 1 || !under31(B) || !under31(layers * B) || H < 1 ||
      H >= (1 << 16) || T < 0 || !under31(T) || D < 8 || D > SV_MAX_HEAD_DIM || D % 8 != 0 ||
      max_nodes < 1 || max_nodes > SV_MAX_TREE_NODES || max_path < 1 || max_path > max_nodes)
    return SV_EINVAL;
  if (num_pages < 1 || !under31(num_pages) || !pow2(page_size) || !under31(page_size) ||
      num_pages * page_size >= (int64_t(1) << 40))
    return SV_EINVAL;
  const int64_t strides[] = {n_stride_l, n_stride_t, n_stride_h,    c_stride_l,
                             c_stride_page, c_stride_token, c_stride_h};
  for (int64_t s : strides)
    if (!stride_ok(s)) return SV_EINVAL;
  if (dtype != SV_F32 && dtype != SV_BF16 && dtype != SV_F16) return SV_EDTYPE;
  const int64_t esz = dtype == SV_F32 ? 4 : 2;
  for (int64_t s : strides)
    if (s * esz % 16 != 0) return SV_EALIGN;
  if (!aligned16(k_tree) || !aligned16(v_tree) || !aligned16(k_cache) || !aligned16(v_cache))
    return SV_EALIGN;
  const int64_t c_sizes[] = {layers, num_pages, page_size, H};
  if (!apart(4, c_sizes, strides + 3, D)) return SV_EINVAL;
  CommitArgs a{static_cast<const char*>(k_tree), static_cast<const char*>(v_tree),
               static_cast<char*>(k_cache), static_cast<char*>(v_cache),
               n_stride_l * esz, n_stride_t * esz, n_stride_h * esz, c_stride_l * esz,
               c_stride_page * esz, c_stride_token * esz, c_stride_h * esz,
               B, T, num_pages * page_size, int(H), int(D * esz / 16), int(max_nodes),
               int(max_path), log2_of(page_size), node_start, path, accept_len, slots,
               prefix_len_in, prefix_len_out, device_error, layers};
  hipLaunchKernelGGL(commit_kernel, dim3(unsigned(layers * B)), dim3(kCommitBlock), 0,
                     reinterpret_cast<hipStream_t>(stream), a);
  return launch_status();
}

}  // extern "C"
