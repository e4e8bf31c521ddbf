// serving_rotate.hip -- norms and position rotation of queries and keys, with keys
// and values into their slots of a paged cache (gfx950).
//
// Bytes are all there is to it: every element is read once and written once. A
// workgroup, or a wavefront where the heads are few, takes a token: the angles of its
// position are the same for all heads, so they are taken once (in float64: at position
// 100000 a float32 product would leave 0.004 of a turn) and held in LDS. A head is 8, 16
// or 32 lanes of 8 elements each, which sum its squares by lane exchanges and hand each
// other the second element of a pair.
// 8192 tokens of 32 + 8 heads of 128 and values into the cache (201 MB) 44 to 49 us by
// card, 4.1 to 4.5 TB/s: 51 to 53 us with loads and stores through the caches, which
// nothing here comes back to, and one set of heads at a time.

#include "specverify_serving.h"
#include "tree_common.h"

namespace {

using namespace svtree;

constexpr int kBlock = 256;

struct RotateArgs {
  const char* q;
  const char* k;
  const char* v;
  const void* q_weight;
  const void* k_weight;
  char* q_out;
  char* k_out;
  char* k_cache;
  char* v_cache;
  int64_t q_t, q_h, k_t, k_h, qo_t, qo_h, ko_t, ko_h, c_page, c_token, c_h;  // bytes
  const int32_t* position;
  const float* inv_freq;
  const int64_t* slots;
  int32_t* err;
  int64_t T, all_slots;
  int Hq, Hkv, D, R, page_shift, weight_f32;
  float eps;
};

template <int DT>
struct Type {
  typedef float type;
};
template <>
struct Type<SV_BF16> {
  typedef __bf16 type;
};
template <>
struct Type<SV_F16> {
  typedef _Float16 type;
};

// 8 elements as they are stored.
template <int DT>
struct Eight {
  typename Type<DT>::type x[8];
};
template <int DT>
__device__ __forceinline__ Eight<DT> load8(const void* p) {
  constexpr int N = sizeof(Eight<DT>) / 16;
  struct Raw {
    u32x4 w[N];
  } raw;
#pragma unroll
  for (int i = 0; i < N; ++i)
    raw.w[i] = __builtin_nontemporal_load(static_cast<const u32x4*>(p) + i);
  return __builtin_bit_cast(Eight<DT>, raw);
}
template <int DT>
__device__ __forceinline__ void store8(void* p, const Eight<DT>& x) {
  constexpr int N = sizeof(Eight<DT>) / 16;
  struct Raw {
    u32x4 w[N];
  };
  const Raw raw = __builtin_bit_cast(Raw, x);
#pragma unroll
  for (int i = 0; i < N; ++i) __builtin_nontemporal_store(raw.w[i], static_cast<u32x4*>(p) + i);
}

constexpr int64_t kMaxGrid = 1 << 22;  // workgroups along x: threads there are counted in 32 bits

enum { kHalves, kHalvesOdd, kPairs };  // the second element of a pair: R / 2 further on
                                       // (in whole pieces of 8 or not), or the next

// What a wavefront has written to LDS is there for its own lanes.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// G threads take a token: all of the workgroup, or a wavefront.
template <int DT, int LANES, int MODE, int G>
__global__ __launch_bounds__(kBlock) void rotate_kernel(RotateArgs a) {
  using elem = typename Type<DT>::type;
  constexpr int HEADS = G / LANES;  // at once
  constexpr int AHEAD = 2;
  constexpr int PAD = 9;  // floats of a lane: 8, and one that moves the next lane's banks on
  __shared__ float all_cosines[kBlock / G][SV_MAX_HEAD_DIM / 2], all_sines[kBlock / G][SV_MAX_HEAD_DIM / 2];
  __shared__ float box[MODE == kHalvesOdd ? kBlock * PAD : 1];
  // (the same for a wavefront, and so scalar)
  const int group = G == kBlock ? 0 : __builtin_amdgcn_readfirstlane(int(threadIdx.x) / G);
  const int tid = int(threadIdx.x) - group * G;
  const int64_t t = (int64_t(blockIdx.y) * gridDim.x + blockIdx.x) * (kBlock / G) + group;
  if (t >= a.T) return;
  float* const cosines = all_cosines[group];
  float* const sines = all_sines[group];
  const int32_t position = a.position[t];
  if (position < 0) return;
  const int in = tid % LANES, d0 = in * 8, half = a.R / 2;
  const bool here = d0 < a.D;
  int64_t at = -1;  // the slot's byte offset in the cache
  if (a.slots) {
    const int64_t slot = a.slots[t];
    if (slot >= 0 && slot < a.all_slots)
      at = (slot >> a.page_shift) * a.c_page +
           (slot & ((int64_t(1) << a.page_shift) - 1)) * a.c_token;
    else if (slot != -1 && tid == 0)
      set_error(a.err, SV_ERR_PAGE);
  }
  const int heads = a.Hq + a.Hkv + (at >= 0 ? a.Hkv : 0);
  // The first heads are on their way while the angles are taken, then always the next.
  const auto fetch = [&](int h) {
    Eight<DT> x{};
    if (!here || h >= heads) return x;
    const char* from = h < a.Hq             ? a.q + t * a.q_t + h * a.q_h
                       : h < a.Hq + a.Hkv ? a.k + t * a.k_t + (h - a.Hq) * a.k_h
                                          : a.v + t * a.k_t + (h - a.Hq - a.Hkv) * a.k_h;
    return load8<DT>(from + d0 * sizeof(elem));
  };
  Eight<DT> ahead[AHEAD];
#pragma unroll
  for (int u = 0; u < AHEAD; ++u) ahead[u] = fetch(u * HEADS + tid / LANES);
  for (int j = tid; j < a.R / 2; j += G) {
    // the angle in turns, what is left of it beside whole ones
    const double turns = double(position) * double(a.inv_freq[j]) * 0.15915494309189533577;
    float s, c;
    sincospif(float(2.0 * (turns - rint(turns))), &s, &c);
    cosines[j] = c;
    sines[j] = s;
  }
  if constexpr (G == kWave) wave_sync();
  else __syncthreads();
  for (int h0 = 0; h0 < heads; h0 += HEADS) {
    const int h = h0 + tid / LANES;
    const Eight<DT> raw = ahead[0];
#pragma unroll
    for (int u = 0; u + 1 < AHEAD; ++u) ahead[u] = ahead[u + 1];
    ahead[AHEAD - 1] = fetch(h + AHEAD * HEADS);
    const bool is_q = h < a.Hq, is_k = !is_q && h < a.Hq + a.Hkv, some = here && h < heads;
    if (!is_q && !is_k) {  // a value
      if (some) {
        const int kv = h - a.Hq - a.Hkv;
        store8<DT>(a.v_cache + at + kv * a.c_h + d0 * sizeof(elem), raw);
      }
      continue;
    }
    const int kv = h - a.Hq;
    float x[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    const bool work = some && (is_q || is_k);
    if (work) {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = float(raw.x[i]);
    }
    const void* weight = is_q ? a.q_weight : a.k_weight;
    if (weight) {
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) sum = fmaf(x[i], x[i], sum);
#pragma unroll
      for (int d = 1; d < LANES; d *= 2) sum += __shfl_xor(sum, d);
      const float f = 1.0f / sqrtf(sum / float(a.D) + a.eps);
      if (work) {
        if (a.weight_f32) {
          const float* w = static_cast<const float*>(weight) + d0;
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = x[i] * f * w[i];
        } else {
          const elem* w = static_cast<const elem*>(weight) + d0;
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = x[i] * f * float(w[i]);
        }
      }
    }
    Eight<DT> y;
    if constexpr (MODE == kPairs) {
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const bool turn = d0 + i < a.R;
        const int j = turn ? (d0 + i) / 2 : 0;
        const float c = turn ? cosines[j] : 1.0f, s = turn ? sines[j] : 0.0f;
        y.x[i] = elem(turn ? x[i] * c - x[i + 1] * s : x[i]);
        y.x[i + 1] = elem(turn ? x[i + 1] * c + x[i] * s : x[i + 1]);
      }
    } else if constexpr (MODE == kHalves) {
      const bool first = d0 < half, second = !first && d0 < a.R;
      const int lane = tid % kWave;
      const int other = first ? lane + half / 8 : second ? lane - half / 8 : lane;
      const int j = first ? d0 : second ? d0 - half : 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float z = __shfl(x[i], other);
        const float c = cosines[j + i], s = first ? -sines[j + i] : sines[j + i];
        y.x[i] = elem(first || second ? x[i] * c + z * s : x[i]);
      }
    } else {
      float* mine = box + (int(threadIdx.x) - in) * PAD;  // the head's, of one wavefront
      wave_sync();
#pragma unroll
      for (int i = 0; i < 8; ++i) mine[in * PAD + i] = x[i];
      wave_sync();
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int d = d0 + i;
        const bool first = d < half, second = !first && d < a.R;
        const int j = first ? d : second ? d - half : 0;
        const int o = first ? d + half : second ? d - half : d;
        const float z = mine[o + o / 8];
        const float c = cosines[j], s = first ? -sines[j] : sines[j];
        y.x[i] = elem(first || second ? x[i] * c + z * s : x[i]);
      }
    }
    if (!work) continue;
    if (is_q) {
      store8<DT>(a.q_out + t * a.qo_t + h * a.qo_h + d0 * sizeof(elem), y);
    } else {
      if (a.k_out) store8<DT>(a.k_out + t * a.ko_t + kv * a.ko_h + d0 * sizeof(elem), y);
      if (at >= 0) store8<DT>(a.k_cache + at + kv * a.c_h + d0 * sizeof(elem), y);
    }
  }
}

template <int DT, int LANES, int MODE>
void launch_threads(const RotateArgs& a, hipStream_t st) {
  // A wavefront to a token where a workgroup would not be full of its heads: 8000 tokens
  // of 8 + 1 heads of 128 15 us, 18 us by workgroups; of 32 + 8 heads 56 us, 51 us by
  // workgroups.
  const bool wave = int64_t(a.Hq + 2 * int64_t(a.Hkv)) * LANES <= kBlock;
  const int64_t groups = wave ? (a.T + kBlock / kWave - 1) / (kBlock / kWave) : a.T;
  const int64_t x = groups < kMaxGrid ? groups : kMaxGrid;
  const dim3 grid{unsigned(x), unsigned((groups + x - 1) / x), 1u};
  if (wave) hipLaunchKernelGGL((rotate_kernel<DT, LANES, MODE, kWave>), grid, dim3(kBlock), 0, st, a);
  else hipLaunchKernelGGL((rotate_kernel<DT, LANES, MODE, kBlock>), grid, dim3(kBlock), 0, st, a);
}

template <int DT, int LANES>
void launch_mode(const RotateArgs& a, int mode, hipStream_t st) {
  if (mode == kPairs) launch_threads<DT, LANES, kPairs>(a, st);
  else if (mode == kHalves) launch_threads<DT, LANES, kHalves>(a, st);
  else launch_threads<DT, LANES, kHalvesOdd>(a, st);
}

template <int DT>
void launch_lanes(const RotateArgs& a, int mode, hipStream_t st) {
  if (a.D <= 64) launch_mode<DT, 8>(a, mode, st);
  else if (a.D <= 128) launch_mode<DT, 16>(a, mode, st);
  else launch_mode<DT, 32>(a, mode, st);
}

}  // namespace

#ifdef SV_DEVICE_CHECKS
bool sv_add_serving_rotate_checks(uint32_t* count, int reset) { return sv_add_checks(count, reset); }
#endif

extern "C" {

int specverify_rotate(const void* q, const void* k, const void* v, int dtype, int64_t T, int64_t Hq,
                      int64_t Hkv, int64_t D, int64_t R, int interleaved, int64_t q_stride_t,
                      int64_t q_stride_h, int64_t k_stride_t, int64_t k_stride_h,
                      const void* q_weight, const void* k_weight, int weight_dtype, float eps,
                      const int32_t* position, const float* inv_freq, void* q_out,
                      int64_t qo_stride_t, int64_t qo_stride_h, void* k_out, int64_t ko_stride_t,
                      int64_t ko_stride_h, const int64_t* slots, void* k_cache, void* v_cache,
                      int64_t c_stride_page, int64_t c_stride_token, int64_t c_stride_h,
                      int64_t num_pages, int64_t page_size, int32_t* device_error, void* stream) {
  const int64_t k31 = int64_t(1) << 31;
  const bool cached = k_cache != nullptr;
  if (cached != (v_cache != nullptr) || !inv_freq) return SV_EINVAL;
  if (T < 0 || T >= k31 || Hq < 1 || Hkv < 1 || Hq >= k31 || Hkv >= k31 || T * (Hq + Hkv) >= k31 ||
      Hq + 2 * Hkv >= k31 || D < 8 || D > SV_MAX_HEAD_DIM || D % 8 != 0 || R < 2 || R > D ||
      R % 2 != 0 || !(eps >= 0.0f) || !std::isfinite(eps))
    return SV_EINVAL;
  if (T > 0 && (!q || !k || !position || !q_out || (cached && (!v || !slots)) ||
                (!cached && (!k_out || slots))))
    return SV_EINVAL;
  if (cached && (num_pages < 1 || num_pages >= k31 || !pow2(page_size) || page_size >= k31 ||
                 num_pages * page_size >= (int64_t(1) << 40)))
    return SV_EINVAL;
  if (!cached) {  // not looked at
    c_stride_page = c_stride_token = c_stride_h = 0;
    page_size = num_pages = 1;
  }
  if (!k_out) ko_stride_t = ko_stride_h = 0;
  const int64_t strides[] = {q_stride_t,  q_stride_h,  k_stride_t,    k_stride_h,     qo_stride_t,
                             qo_stride_h, ko_stride_t, ko_stride_h,   c_stride_page, c_stride_token,
                             c_stride_h};
  for (int64_t s : strides)
    if (!stride_ok(s)) return SV_EINVAL;
  if (dtype != SV_F32 && dtype != SV_BF16 && dtype != SV_F16) return SV_EDTYPE;
  if ((q_weight || k_weight) && weight_dtype != dtype && weight_dtype != SV_F32) return SV_EDTYPE;
  const int size = dtype == SV_F32 ? 4 : 2;
  for (int64_t s : strides)
    if (s * size % 16 != 0) return SV_EALIGN;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q_out) || !aligned16(k_out) ||
      !aligned16(k_cache) || !aligned16(v_cache))
    return SV_EALIGN;
  const int64_t qs[] = {T, Hq}, qo[] = {qo_stride_t, qo_stride_h};
  const int64_t ks[] = {T, Hkv}, ko[] = {ko_stride_t, ko_stride_h};
  const int64_t cs[] = {num_pages, page_size, Hkv}, co[] = {c_stride_page, c_stride_token, c_stride_h};
  if (!apart(2, qs, qo, D) || (k_out && !apart(2, ks, ko, D)) || (cached && !apart(3, cs, co, D)))
    return SV_EINVAL;
  if (T == 0) return SV_OK;
  RotateArgs a{};
  a.q = static_cast<const char*>(q);
  a.k = static_cast<const char*>(k);
  a.v = static_cast<const char*>(v);
  a.q_weight = q_weight;
  a.k_weight = k_weight;
  a.q_out = static_cast<char*>(q_out);
  a.k_out = static_cast<char*>(k_out);
  a.k_cache = static_cast<char*>(k_cache);
  a.v_cache = static_cast<char*>(v_cache);
  a.q_t = q_stride_t * size;
  a.q_h = q_stride_h * size;
  a.k_t = k_stride_t * size;
  a.k_h = k_stride_h * size;
  a.qo_t = qo_stride_t * size;
  a.qo_h = qo_stride_h * size;
  a.ko_t = ko_stride_t * size;
  a.ko_h = ko_stride_h * size;
  a.c_page = c_stride_page * size;
  a.c_token = c_stride_token * size;
  a.c_h = c_stride_h * size;
  a.position = position;
  a.inv_freq = inv_freq;
  a.slots = cached ? slots : nullptr;
  a.err = device_error;
  a.T = T;
  a.all_slots = num_pages * page_size;
  a.Hq = int(Hq);
  a.Hkv = int(Hkv);
  a.D = int(D);
  a.R = int(R);
  a.page_shift = log2_of(page_size);
  a.weight_f32 = weight_dtype == SV_F32;
  a.eps = eps;
  const int mode = interleaved ? kPairs : R / 2 % 8 == 0 ? kHalves : kHalvesOdd;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  if (dtype == SV_F32) launch_lanes<SV_F32>(a, mode, st);
  else if (dtype == SV_BF16) launch_lanes<SV_BF16>(a, mode, st);
  else launch_lanes<SV_F16>(a, mode, st);
  return launch_status();
}

}  // extern "C"
