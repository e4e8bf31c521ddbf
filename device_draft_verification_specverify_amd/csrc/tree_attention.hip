// tree_attention.hip -- attention of drafted tree nodes over a paged prefix and
// their ancestors (gfx950, matrix cores): which kernel of attention_kernel.h takes
// a call, and the C ABI's host side.

#include "attention_kernel.h"

namespace {

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
  hipLaunchKernelGGL((attention_kernel<DT, DP, RW, KW, KB, S, false>), dim3(unsigned(kWorkers)),
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
  hipLaunchKernelGGL((join_kernel<DT, DP, false>), dim3(kJoiners), dim3(kWorkers), 0, st, a);
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
