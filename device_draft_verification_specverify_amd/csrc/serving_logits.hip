// serving_logits.hip -- penalties for repeated tokens, biases and grammar masks on
// the logits of drafted nodes (gfx950).
//
// A workgroup takes kChunk ids of a request: what the request's history says of them
// is counted into LDS once, for all its rows, and each row adds the tokens of its
// own path to it while it passes. So the history is read once for each chunk (out of
// the L2) and the logits once.
//
// Bytes bound it: 64 x 9 rows of 128256 ids in bf16 with masks and histories of 300 to
// 8000 tokens (273 MB) 64 us, 4.2 TB/s, of which some 8 us are the first workgroups'
// histories, before any of the card's rows can be written. Logits pass by once, so
// loads and stores go past the caches (75 us without).

#include "specverify_serving.h"
#include "tree_common.h"

namespace {

using namespace svtree;

constexpr int kBlock = 512;
constexpr int kVec = 8;
constexpr int kChunk = kBlock * kVec;  // 4096 ids
constexpr int64_t kMaxGrid = 1 << 22;  // workgroups along x: threads there are counted in 32 bits

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

struct PenalizeArgs {
  const char* logits;
  char* out;
  const int32_t* tokens;
  const int32_t* node_start;
  const uint64_t* anc;
  const int32_t* history;
  const int32_t* prefix_len;
  const int32_t* prompt_len;
  const float* repetition;
  const float* presence;
  const float* frequency;
  const int32_t* bias_start;
  const int32_t* bias_token;
  const float* bias;
  const uint8_t* mask;
  int64_t B, T, V, max_history, num_bias, history_stride;
  int64_t row, out_row, mask_row;  // bytes
  int max_nodes, words, chunks;
  int32_t* err;
};

// 8 logits as they are stored, the mask's bits of them, and their row's ancestors.
template <int DT>
struct Eight {
  u32x4 w[DT == SV_BF16 ? 1 : 2];
  uint32_t keep;
  uint32_t on[4];
};
__device__ __forceinline__ uint64_t uniform64(uint32_t low, uint32_t high) {
  return uint32_t(__builtin_amdgcn_readfirstlane(int(low))) |
         uint64_t(uint32_t(__builtin_amdgcn_readfirstlane(int(high)))) << 32;
}

template <int DT, bool VEC>
__device__ __forceinline__ Eight<DT> load8(const char* row, int64_t v, int64_t V) {
  constexpr int N = DT == SV_BF16 ? 1 : 2;
  Eight<DT> r;
  if (VEC && v + kVec <= V) {
#pragma unroll
    for (int j = 0; j < N; ++j)
      r.w[j] = __builtin_nontemporal_load(
          reinterpret_cast<const u32x4*>(row + v * (2 * N) + 16 * j));
  } else {
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      if constexpr (DT == SV_BF16) {
        const uint32_t x = v + i < V ? reinterpret_cast<const uint16_t*>(row)[v + i] : 0;
        if (i % 2 == 0) r.w[0][i / 2] = x;
        else r.w[0][i / 2] |= x << 16;
      } else {
        r.w[i / 4][i % 4] = v + i < V ? reinterpret_cast<const uint32_t*>(row)[v + i] : 0;
      }
    }
  }
  return r;
}

template <int DT>
__device__ __forceinline__ void widen(const Eight<DT>& r, float (&x)[kVec]) {
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    if constexpr (DT == SV_BF16)
      x[i] = __uint_as_float(i % 2 ? r.w[0][i / 2] & 0xFFFF0000u : r.w[0][i / 2] << 16);
    else
      x[i] = __uint_as_float(r.w[i / 4][i % 4]);
  }
}

template <int DT, bool VEC>
__device__ __forceinline__ void store8(char* row, int64_t v, int64_t V, const float (&x)[kVec]) {
  if constexpr (DT == SV_BF16) {
    typedef __bf16 b8 __attribute__((ext_vector_type(8)));
    b8 y;
#pragma unroll
    for (int i = 0; i < kVec; ++i) y[i] = __bf16(x[i]);
    if (VEC && v + kVec <= V) {
      __builtin_nontemporal_store(__builtin_bit_cast(u32x4, y), reinterpret_cast<u32x4*>(row + v * 2));
    } else {
#pragma unroll
      for (int i = 0; i < kVec; ++i)
        if (v + i < V) reinterpret_cast<__bf16*>(row)[v + i] = y[i];
    }
  } else if (VEC && v + kVec <= V) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      u32x4 w;
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = __float_as_uint(x[4 * j + i]);
      __builtin_nontemporal_store(w, reinterpret_cast<u32x4*>(row + v * 4 + 16 * j));
    }
  } else {
#pragma unroll
    for (int i = 0; i < kVec; ++i)
      if (v + i < V) reinterpret_cast<float*>(row)[v + i] = x[i];
  }
}

template <int DT, int OT, bool VEC>
// (8 wavefronts to a SIMD: with the scalar registers it would take, 7 fit, and 3
// workgroups to a CU instead of 4.)
__global__ __launch_bounds__(kBlock, 8) void penalize_kernel(PenalizeArgs a) {
  // of each id: twice the times it was emitted, and 1 if it is in the prompt
  __shared__ __align__(16) uint32_t seen[kChunk];
  __shared__ __align__(16) float biases[kChunk];
  __shared__ int32_t tok[SV_MAX_TREE_NODES];
  __shared__ uint64_t near[2];  // nodes whose token is among the chunk's ids
  __shared__ uint32_t biased[kChunk / 32], again[kChunk / 32];  // ids with a bias, with several
  __shared__ int several;  // whether there are any of the latter
  __shared__ __align__(16) int32_t list[kBlock];  // biases' ids and values
  __shared__ __align__(16) float adds[kBlock];
  const int64_t block = int64_t(blockIdx.z) * gridDim.x + blockIdx.x;
  const int64_t b = block / a.chunks;
  const int chunk = int(block % a.chunks);
  const int tid = int(threadIdx.x);
  if (b >= a.B) return;
  const bool speaks = chunk == 0 && blockIdx.y == 0;  // reports the request's errors
  const Nodes nd = nodes_of(a.node_start, b, a.T, a.max_nodes);
  if (nd.n <= 0 || int(blockIdx.y) >= nd.n) {
    if (nd.n < 0 && speaks && tid == 0) set_error(a.err, SV_ERR_TREE);
    return;
  }
  const int64_t v0 = int64_t(chunk) * kChunk, mine = v0 + tid * kVec;
  const float rep = a.repetition[b], pres = a.presence[b], freq = a.frequency[b];
  int bits = 0;
  bool wrong = false;
  if (!(rep > 0.0f)) {
    bits |= SV_ERR_PENALTY;
    wrong = true;
  }
  int64_t lo = 0, hi = 0;
  if (a.bias_start) {
    lo = a.bias_start[b];
    hi = a.bias_start[b + 1];
    if (lo < 0 || hi < lo || hi > a.num_bias) {
      bits |= SV_ERR_LENGTH;
      wrong = true;
    }
  }
  if (wrong) {  // no logits: NaN
    float x[kVec];
#pragma unroll
    for (int i = 0; i < kVec; ++i) x[i] = NAN;
    for (int i = int(blockIdx.y); i < nd.n; i += int(gridDim.y))
      if (mine < a.V) store8<OT, VEC>(a.out + (nd.first + i) * a.out_row, mine, a.V, x);
    if (speaks && tid == 0) set_error(a.err, bits);
    return;
  }
  const auto clamped = [&](int64_t x, int64_t most) {
    if (x < 0 || x > most) bits |= SV_ERR_LENGTH;
    return int32_t(x < 0 ? 0 : x > most ? most : x);
  };
  const int32_t len = clamped(a.prefix_len[b], a.max_history);
  const int32_t prompt = clamped(a.prompt_len[b], a.max_history);

  // The first row is on its way while the history is counted, then always the next
  // one (at 64 x 9 rows two ahead 2 us more, three 6 us).
  const int step = int(gridDim.y);
  const auto fetch = [&](int i) {
    Eight<DT> r{};
    if (i >= nd.n || !sv_ok(nd.first + i < a.T)) return r;
    if (a.anc) {
      const uint32_t* on = reinterpret_cast<const uint32_t*>(a.anc + (nd.first + i) * a.words);
      for (int j = 0; j < 4; ++j) r.on[j] = j < 2 * a.words ? on[j] : 0;
    }
    if (mine < a.V) {
      const Eight<DT> x = load8<DT, VEC>(a.logits + (nd.first + i) * a.row, mine, a.V);
#pragma unroll
      for (int j = 0; j < int(sizeof(r.w) / sizeof(r.w[0])); ++j) r.w[j] = x.w[j];
      r.keep = a.mask ? a.mask[(nd.first + i) * a.mask_row + mine / 8] : 0xFFu;
    }
    return r;
  };
  Eight<DT> next = fetch(int(blockIdx.y));
  for (int i = tid; i < kChunk; i += kBlock) seen[i] = 0;
  if (hi > lo) {
    for (int i = tid; i < kChunk; i += kBlock) biases[i] = 0.0f;
    if (tid < kChunk / 32) biased[tid] = again[tid] = 0;
    if (tid == 0) several = 0;
  }
  if (tid < 128) {
    const int32_t x = tid < nd.n && sv_ok(nd.first + tid < a.T) ? a.tokens[nd.first + tid] : 0;
    tok[tid] = x;
    if (tid < nd.n && (x < 0 || x >= a.V)) bits |= SV_ERR_TOKEN;
    const uint64_t in = __ballot(tid < nd.n && x >= v0 && x < v0 + kChunk && x < a.V);
    if (tid % kWave == 0) near[tid / kWave] = in;
  }
  __syncthreads();
  const int32_t* history = a.history + b * a.history_stride;
  constexpr int AHEAD = 4;
  for (int32_t j0 = tid; j0 < len; j0 += kBlock * AHEAD) {
    int32_t x[AHEAD];
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      const int64_t j = int64_t(j0) + u * kBlock;
      x[u] = j < len ? history[j] : -1;
      if (j < len && (x[u] < 0 || x[u] >= a.V)) bits |= SV_ERR_TOKEN;
    }
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      const int64_t d = x[u] - v0;
      if (d < 0 || d >= kChunk || x[u] >= a.V) continue;
      if (j0 + u * kBlock < prompt) atomicOr(seen + d, 1u);
      else atomicAdd(seen + d, 2u);
    }
  }
  if (hi > lo) {
    for (int64_t j = lo + tid; j < hi; j += kBlock) {
      const int32_t x = a.bias_token[j];
      const int64_t d = x - v0;
      if (x < 0 || x >= a.V) bits |= SV_ERR_TOKEN;
      if (d < 0 || d >= kChunk || x >= a.V) continue;
      const uint32_t bit = 1u << (d & 31);
      if (atomicOr(biased + d / 32, bit) & bit) {
        atomicOr(again + d / 32, bit);
        several = 1;
      } else {
        biases[d] = a.bias[j];
      }
    }
    __syncthreads();
    if (several) {
      for (int i = tid; i < kChunk; i += kBlock)
        if (again[i / 32] >> (i & 31) & 1) biases[i] = 0.0f;
    }
    // Several biases of an id are added up in their order, kBlock of the list at a time: by the
    // first one's thread, which finds the others in LDS (300 biases of some 100 ids: 19 us; out of
    // memory 41 us).
    for (int64_t j0 = several ? lo : hi; j0 < hi; j0 += kBlock) {
      const int64_t j = j0 + tid;
      const int32_t x = j < hi ? a.bias_token[j] : -1;
      const float add = j < hi ? a.bias[j] : 0.0f;
      __syncthreads();
      list[tid] = x;
      adds[tid] = add;
      __syncthreads();
      const int64_t d = x - v0;
      if (d < 0 || d >= kChunk || x >= a.V) continue;
      if (again[d / 32] >> (d & 31) & 1) {
        // (in front of the wavefront's own part of the list, in it, and behind it)
        const int own = tid & ~(kWave - 1), n = int(hi - j0 < kBlock ? hi - j0 : kBlock);
        bool first = true;
#pragma unroll 4
        for (int i = 0; i < own; i += 4) {
          const i32x4 y = *reinterpret_cast<const i32x4*>(list + i);
          first = first && y[0] != x && y[1] != x && y[2] != x && y[3] != x;
        }
        for (int i = own; i < tid; ++i) first = first && list[i] != x;
        if (!first) continue;
        float sum = biases[d];
#pragma unroll 4
        for (int i = own; i < n; i += 4) {
          const i32x4 y = *reinterpret_cast<const i32x4*>(list + i);
          const f32x4 z = *reinterpret_cast<const f32x4*>(adds + i);
#pragma unroll
          for (int e = 0; e < 4; ++e) sum += y[e] == x ? z[e] : 0.0f;
        }
        biases[d] = sum;
      }
    }
  }
  __syncthreads();

  const float inv = 1.0f / rep;
  uint64_t had[2] = {0, 0};  // the nodes that `seen` counts now
  for (int i = int(blockIdx.y); i < nd.n; i += step) {
    const int64_t r = nd.first + i;
    if (!sv_ok(r < a.T)) break;
    Eight<DT> now = next;
    // (here before the next one is asked for: a wait further down would be for both)
#pragma unroll
    for (int j = 0; j < int(sizeof(now.w) / sizeof(now.w[0])); ++j) asm volatile("" : "+v"(now.w[j]));
    asm volatile("" : "+v"(now.keep), "+v"(now.on[0]), "+v"(now.on[1]), "+v"(now.on[2]), "+v"(now.on[3]));
    next = fetch(i + step);
    // the nodes of this row's path whose tokens are here
    uint64_t on[2];
    if (a.anc) {
      on[0] = uniform64(now.on[0], now.on[1]);
      on[1] = uniform64(now.on[2], now.on[3]);
      on[0] &= nd.n >= 64 ? ~uint64_t(0) : (uint64_t(1) << nd.n) - 1;
    } else {
      on[0] = i >= 63 ? ~uint64_t(0) : (uint64_t(2) << i) - 1;
      on[1] = i < 64 ? 0 : i >= 127 ? ~uint64_t(0) : (uint64_t(2) << (i - 64)) - 1;
    }
    on[0] &= near[0];
    on[1] &= near[1];
    if (on[0] != had[0] || on[1] != had[1]) {  // (the same for the whole workgroup)
      __syncthreads();
      if (tid < 128) {
        const int change = int(on[tid / 64 & 1] >> (tid & 63) & 1) - int(had[tid / 64 & 1] >> (tid & 63) & 1);
        if (change) atomicAdd(seen + (tok[tid] - v0), uint32_t(2 * change));
      }
      __syncthreads();
      had[0] = on[0];
      had[1] = on[1];
    }
    if (mine < a.V) {
      float x[kVec];
      widen<DT>(now, x);
      const u32x4 c0 = *reinterpret_cast<const u32x4*>(seen + tid * kVec);
      const u32x4 c1 = *reinterpret_cast<const u32x4*>(seen + tid * kVec + 4);
      const u32x4 any = c0 | c1;
      if (any[0] | any[1] | any[2] | any[3]) {
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
          const uint32_t c = e < 4 ? c0[e] : c1[e - 4];
          const float turned = x[e] > 0.0f ? x[e] * inv : x[e] * rep;
          x[e] = c ? turned : x[e];
          const float less = x[e] - fmaf(freq, float(c >> 1), pres);
          x[e] = c > 1 ? less : x[e];
        }
      }
      if (hi > lo) {
#pragma unroll
        for (int e = 0; e < kVec; ++e) x[e] += biases[tid * kVec + e];
      }
#pragma unroll
      for (int e = 0; e < kVec; ++e) x[e] = now.keep >> e & 1 ? x[e] : -INFINITY;
      store8<OT, VEC>(a.out + r * a.out_row, mine, a.V, x);
    }
  }
  if (bits && speaks) set_error(a.err, bits);
}

template <int DT, int OT>
void launch(const PenalizeArgs& a, bool vec, dim3 grid, hipStream_t st) {
  if (vec) hipLaunchKernelGGL((penalize_kernel<DT, OT, true>), grid, dim3(kBlock), 0, st, a);
  else hipLaunchKernelGGL((penalize_kernel<DT, OT, false>), grid, dim3(kBlock), 0, st, a);
}

}  // namespace

#ifdef SV_DEVICE_CHECKS
bool sv_add_serving_logits_checks(uint32_t* count, int reset) { return sv_add_checks(count, reset); }
#endif

extern "C" {

int specverify_penalize(const void* logits, int dtype, const int32_t* tokens,
                        const int32_t* node_start, const uint64_t* ancestors,
                        const int32_t* history, const int32_t* prefix_len,
                        const int32_t* prompt_len, const float* repetition, const float* presence,
                        const float* frequency, const int32_t* bias_start,
                        const int32_t* bias_token, const float* bias, const int32_t* mask,
                        int64_t B, int64_t T, int64_t V, int64_t max_nodes, int64_t max_history,
                        int64_t num_bias, int64_t stride, int64_t out_stride,
                        int64_t history_stride, int64_t mask_stride, void* out, int out_dtype,
                        int32_t* device_error, void* stream) {
  const int64_t k31 = int64_t(1) << 31;
  if (!node_start || !history || !prefix_len || !prompt_len || !repetition || !presence || !frequency)
    return SV_EINVAL;
  if (T > 0 && (!logits || !tokens || !out)) return SV_EINVAL;
  const bool has_bias = bias_start != nullptr;
  if (has_bias != (bias_token != nullptr) || has_bias != (bias != nullptr)) return SV_EINVAL;
  if (B < 1 || B > (1 << 20) || T < 0 || T >= k31 || V < 1 || V > SV_MAX_TREE_VOCAB ||
      max_nodes < 1 || max_nodes > SV_MAX_TREE_NODES || max_history < 1 || max_history >= k31 ||
      num_bias < 0 || num_bias >= k31)
    return SV_EINVAL;
  if (!stride_ok(stride) || !stride_ok(out_stride) || !stride_ok(history_stride) ||
      out_stride < V || history_stride < max_history)
    return SV_EINVAL;
  if (mask && (!stride_ok(mask_stride) || mask_stride < (V + 31) / 32)) return SV_EINVAL;
  if ((dtype != SV_F32 && dtype != SV_BF16) || (out_dtype != SV_F32 && out_dtype != SV_BF16))
    return SV_EDTYPE;
  if (T > 0 && out == logits && (dtype != out_dtype || stride != out_stride)) return SV_EINVAL;
  if (T == 0) return SV_OK;
  PenalizeArgs a{};
  const int size = dtype == SV_F32 ? 4 : 2, out_size = out_dtype == SV_F32 ? 4 : 2;
  a.logits = static_cast<const char*>(logits);
  a.out = static_cast<char*>(out);
  a.tokens = tokens;
  a.node_start = node_start;
  a.anc = ancestors;
  a.history = history;
  a.prefix_len = prefix_len;
  a.prompt_len = prompt_len;
  a.repetition = repetition;
  a.presence = presence;
  a.frequency = frequency;
  a.bias_start = bias_start;
  a.bias_token = bias_token;
  a.bias = bias;
  a.mask = reinterpret_cast<const uint8_t*>(mask);
  a.B = B;
  a.T = T;
  a.V = V;
  a.max_history = max_history;
  a.num_bias = num_bias;
  a.history_stride = history_stride;
  a.row = stride * size;
  a.out_row = out_stride * out_size;
  a.mask_row = mask_stride * 4;
  a.max_nodes = int(max_nodes);
  a.words = int((max_nodes + 63) / 64);
  a.chunks = int((V + kChunk - 1) / kChunk);
  a.err = device_error;
  // Rows that begin at multiples of 16 bytes take 128-bit accesses.
  const bool vec = aligned16(logits) && aligned16(out) && a.row % 16 == 0 && a.out_row % 16 == 0;
  // A request's rows are shared out where its chunks alone leave the card idle.
  const int64_t work = B * a.chunks;
  int64_t split = 1024 / work;
  if (split > max_nodes) split = max_nodes;
  if (split < 1) split = 1;
  const int64_t x = work < kMaxGrid ? work : kMaxGrid;
  const dim3 grid{unsigned(x), unsigned(split), unsigned((work + x - 1) / x)};
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  if (dtype == SV_F32 && out_dtype == SV_F32) launch<SV_F32, SV_F32>(a, vec, grid, st);
  else if (dtype == SV_F32) launch<SV_F32, SV_BF16>(a, vec, grid, st);
  else if (out_dtype == SV_F32) launch<SV_BF16, SV_F32>(a, vec, grid, st);
  else launch<SV_BF16, SV_BF16>(a, vec, grid, st);
  return launch_status();
}

}  // extern "C"
