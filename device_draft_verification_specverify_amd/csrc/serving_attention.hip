// serving_attention.hip -- attention of chunks of new tokens over a paged cache
// (gfx950, matrix cores): which kernel of attention_kernel.h takes a call, and the C
// ABI's host side.

#include "attention_kernel.h"
#include "specverify_serving.h"

namespace {

// Which kernel: by the rows that a request has of a key head, tokens times query
// heads. Few of them (a single token, a short chunk) leave wavefronts of a workgroup
// for the keys of a tile, as for drafted trees; many take all of them, and each other's
// turns on the matrix cores. A batch may hold both: then either kernel passes the
// other's requests by, in a launch of its own.
constexpr int kFewRows = 64;

// What an item costs the kernel whose wavefronts take turns besides its tiles (its
// rows loaded and written, the masked tiles at its end), in tiles: 8192 tokens from
// nothing 624 us with 3, 561 us with 6, 547 us with 8; on another card 568 us with 7,
// 570 with 8, 574 with 10.
constexpr int kTurnPlaces = 8;

struct Variant {
  int rw, kw, kb, width;
  int rows() const { return 32 * rw; }
  int keys() const { return kw * kb; }
};
int width_of(int64_t D) { return D <= 64 ? 64 : D <= 128 ? 128 : 256; }
Variant variant_of(int64_t rows, int64_t D) {
  Variant v;
  v.width = width_of(D);
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

template <int DT, int DP, int RW, int KW, int KB, int S, int DC = 0>
void launch_one(const AttnArgs& a, hipStream_t st) {
  hipLaunchKernelGGL((attention_kernel<DT, DP, RW, KW, KB, S, true, DC>), dim3(unsigned(kWorkers)),
                     dim3(64 * RW * KW), 0, st, a);
}

template <int DT, int DP>
void launch(const Variant& v, const AttnArgs& a, hipStream_t st) {
  if constexpr (DP == 256) {
    if (v.rw == 2) launch_one<DT, DP, 2, 2, 32, 2>(a, st);
    else launch_one<DT, DP, 4, 1, 32, 4>(a, st);
  } else {
    constexpr int X = 128 / DP;  // stages of half the size, twice as many
    if (v.rw == 2) launch_one<DT, DP, 2, 4, 32, 2 * X>(a, st);
    else if (v.rw == 4) launch_one<DT, DP, 4, 2, 64, 2 * X>(a, st);
    else if (a.D > 96 || DP == 64) launch_one<DT, DP, 8, 1, 64, 4, DP>(a, st);
    else if constexpr (DP == 128) launch_one<DT, DP, 8, 1, 64, 4, 96>(a, st);
  }
}

// few: null where one kernel takes all requests.
template <int DT, int DP>
void launch_both(const Variant& v, const AttnArgs& a, const AttnArgs* few, hipStream_t st) {
  launch<DT, DP>(v, a, st);
  if (few) {
    launch<DT, DP>(variant_of(kFewRows, few->D), *few, st);
    if (!a.whole || !few->whole)
      hipLaunchKernelGGL((join_both_kernel<DT, DP, true>), dim3(2 * kJoiners), dim3(kWorkers), 0, st,
                         a, *few);
  } else if (!a.whole) {
    hipLaunchKernelGGL((join_kernel<DT, DP, true>), dim3(kJoiners), dim3(kWorkers), 0, st, a);
  }
}

template <int DT>
void launch_width(const Variant& v, const AttnArgs& a, const AttnArgs* few, hipStream_t st) {
  if (v.width == 64) launch_both<DT, 64>(v, a, few, st);
  else if (v.width == 128) launch_both<DT, 128>(v, a, few, st);
  else launch_both<DT, 256>(v, a, few, st);
}

bool sizes_ok(int64_t B, int64_t T, int64_t Hq, int64_t Hkv, int64_t D, int64_t max_chunk) {
  const int64_t k31 = int64_t(1) << 31;
  return B >= 1 && B < k31 && T >= 0 && T < k31 && Hq >= 1 && Hkv >= 1 && Hq < k31 && Hkv < k31 &&
         Hq % Hkv == 0 && Hq / Hkv <= (1 << 16) && D >= 8 && D <= SV_MAX_HEAD_DIM && D % 8 == 0 &&
         max_chunk >= 1 && max_chunk < k31 && B * Hkv <= (1 << 24) && T * Hq < k31;
}

// Rows of the largest chunk: no request has more than all of them.
int64_t most_rows(int64_t T, int64_t G, int64_t max_chunk) {
  return (max_chunk < T ? max_chunk : T) * G;
}

size_t workspace_of(const Variant& v) {
  return align256(size_t(kWorkers + 1) * sizeof(Split)) +
         align256(size_t(kWorkers) * 2 * v.rows() * (v.width + 4) * sizeof(float));
}

// How a kernel takes the requests whose rows are from `from` to `to`.
void take(AttnArgs& a, const Variant& v, int from, int to, int64_t most, char* workspace) {
  a.split = reinterpret_cast<Split*>(workspace);
  a.part = reinterpret_cast<float*>(workspace + align256(size_t(kWorkers + 1) * sizeof(Split)));
  a.tile_keys = v.keys();
  a.tile_rows = v.rows();
  a.GS = a.G < a.tile_rows ? a.G : a.tile_rows;
  a.parts = (a.G + a.GS - 1) / a.GS;
  a.tokens = a.tile_rows / a.GS;
  a.item_places = v.kw == 1 && v.width < 256 ? kTurnPlaces : kItemPlaces;
  a.rows_from = from;
  a.rows_to = to;
  const int64_t items = a.B * a.Hkv * a.parts * ((most + a.tokens - 1) / a.tokens);
  a.whole = a.max_keys <= kWholeTiles * int64_t(a.tile_keys) && items <= kWorkers;
}

}  // namespace

#ifdef SV_DEVICE_CHECKS
bool sv_add_serving_attention_checks(uint32_t* count, int reset) {
  return sv_add_checks(count, reset);
}
#endif

extern "C" {

size_t specverify_chunk_attention_workspace_size(int64_t B, int64_t T, int64_t Hq, int64_t Hkv,
                                                 int64_t D, int64_t max_chunk) {
  if (!sizes_ok(B, T, Hq, Hkv, D, max_chunk)) return 0;
  const Variant v = variant_of(most_rows(T, Hq / Hkv, max_chunk), D);
  return workspace_of(v) + (v.rows() > kFewRows ? workspace_of(variant_of(kFewRows, D)) : 0);
}

int specverify_chunk_attention(const void* q, const void* k_cache, const void* v_cache, int dtype,
                               int64_t B, int64_t T, int64_t Hq, int64_t Hkv, int64_t D,
                               int64_t max_chunk, int64_t q_stride_t, int64_t q_stride_h,
                               int64_t c_stride_page, int64_t c_stride_token, int64_t c_stride_h,
                               int64_t num_pages, int64_t page_size, const int32_t* block_table,
                               int64_t max_pages, int64_t table_stride, const int32_t* prefix_len,
                               const int32_t* chunk_start, float scale, void* out,
                               int64_t o_stride_t, int64_t o_stride_h, float* lse,
                               int32_t* device_error, void* workspace, size_t workspace_bytes,
                               void* stream) {
  if (!k_cache || !v_cache || !block_table || !prefix_len || !chunk_start) return SV_EINVAL;
  if (T > 0 && (!q || !out)) return SV_EINVAL;
  if (!sizes_ok(B, T, Hq, Hkv, D, max_chunk)) return SV_EINVAL;
  const int64_t k31 = int64_t(1) << 31;
  if (!pow2(page_size) || page_size >= k31 || max_pages < 1 || max_pages >= k31 ||
      max_pages * page_size > k31 - (1 << 14) || num_pages < 1 || num_pages >= k31 ||
      table_stride < max_pages || !stride_ok(table_stride))
    return SV_EINVAL;
  const int64_t strides[] = {q_stride_t,     q_stride_h, c_stride_page, c_stride_token,
                             c_stride_h,     o_stride_t, o_stride_h};
  for (int64_t s : strides)
    if (!stride_ok(s)) return SV_EINVAL;
  if (!(scale > 0.0f) || !std::isfinite(scale * kLog2e)) return SV_EINVAL;
  if (dtype != SV_BF16 && dtype != SV_F16) return SV_EDTYPE;
  for (int64_t s : strides)
    if (s % 8 != 0) return SV_EALIGN;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out))
    return SV_EALIGN;
  const int64_t out_sizes[] = {T, Hq}, out_strides[] = {o_stride_t, o_stride_h};
  if (!apart(2, out_sizes, out_strides, D)) return SV_EINVAL;
  int status = SV_OK;
  if (!workspace_ok(workspace, workspace_bytes,
                    specverify_chunk_attention_workspace_size(B, T, Hq, Hkv, D, max_chunk),
                    &status))
    return status;
  if (T == 0) return SV_OK;
  const int64_t rows = most_rows(T, Hq / Hkv, max_chunk);
  const Variant v = variant_of(rows, D);
  AttnArgs a{};
  a.q = static_cast<const char*>(q);
  a.k_cache = static_cast<const char*>(k_cache);
  a.v_cache = static_cast<const char*>(v_cache) - a.k_cache;
  a.q_t = q_stride_t * 2;
  a.q_h = q_stride_h * 2;
  a.c_page = c_stride_page * 2;
  a.c_token = c_stride_token * 2;
  a.c_h = c_stride_h * 2;
  a.o_t = o_stride_t * 2;
  a.o_h = o_stride_h * 2;
  a.table = block_table;
  a.prefix_len = prefix_len;
  a.node_start = chunk_start;
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
  a.max_nodes = int(max_chunk);
  a.page_shift = log2_of(page_size);
  a.scale_log2 = scale * kLog2e;
  const int64_t most = max_chunk < T ? max_chunk : T;
  char* const ws = static_cast<char*>(workspace);
  // Chunks of fewer rows beside the largest: not where one request is all there is, or
  // all have as many tokens as the longest may have.
  const bool mixed = v.rows() > 128 && B > 1 && T < B * most;
  take(a, v, mixed ? kFewRows + 1 : 0, INT_MAX, most, ws);
  AttnArgs few = a;
  if (mixed) take(few, variant_of(kFewRows, D), 0, kFewRows, most, ws + workspace_of(v));
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  if (dtype == SV_BF16) launch_width<SV_BF16>(v, a, mixed ? &few : nullptr, st);
  else launch_width<SV_F16>(v, a, mixed ? &few : nullptr, st);
  return launch_status();
}

}  // extern "C"
