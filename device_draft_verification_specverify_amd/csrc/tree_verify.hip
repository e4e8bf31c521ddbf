// tree_verify.hip -- verification of drafted trees from probabilities and given
// uniforms (gfx950).
//
// The walk. At a node with target row p and draft row q, rejecting children one
// after another means w_0 = p, w_{k+1} = max(w_k / S_k - q / Q_k, 0) (S_k, Q_k the
// masses of w_k and of q without the children rejected before). Up to a factor
// that is w_k = max(p - a_k q, 0) with a_{k+1} = a_k + S_k / Q_k, so a node's
// whole state is one number, and S_{k+1} = sum_v max(p - a q, 0) is one pass over
// the row pair that keeps nothing. For draws without replacement the formula
// holds at the rejected tokens too: x_k was rejected because
// w_k(x) <= u S_k q(x) / Q_k < (S_k / Q_k) q(x), so its w is zero from then on.
// Accept tests read two scalars of each row, so only rejections and the last
// node cost a pass.

#include "tree_common.h"

namespace {

using namespace svtree;

constexpr int kBlock = 1024;
constexpr int kWaves = kBlock / kWave;
constexpr int kVec = 8;                   // probabilities of a thread in a chunk
constexpr int kChunk = kBlock * kVec;     // 8192
constexpr int kMaxChunks = SV_MAX_TREE_VOCAB / kChunk;

struct VerifyArgs {
  const void* p;
  const void* q;
  int64_t ps, qs;  // row strides in elements
  const int32_t* tokens;
  const int32_t* parents;
  const int32_t* node_start;
  const double* u;
  const double* r;
  int64_t T, V;
  int max_nodes, max_path, mode;
  int32_t* accept_len;
  int32_t* path;
  int32_t* emitted;
  int32_t* out_token;
  int32_t* err;
};

template <int DT>
__device__ __forceinline__ double load_one(const void* row, int64_t e) {
  if constexpr (DT == SV_BF16)
    return double(__uint_as_float(uint32_t(reinterpret_cast<const uint16_t*>(row)[e]) << 16));
  else
    return double(reinterpret_cast<const float*>(row)[e]);
}

template <int DT>
__device__ __forceinline__ const void* row_at(const void* base, int64_t stride, int64_t row) {
  return static_cast<const char*>(base) + row * stride * (DT == SV_BF16 ? 2 : 4);
}

// 8 probabilities from v0 on as float32 (exact); 0 behind the row's end.
template <int DT, bool VEC>
__device__ __forceinline__ void load8(const void* row, int64_t v0, int64_t V, float (&x)[kVec]) {
  if (VEC && v0 + kVec <= V) {
    if constexpr (DT == SV_BF16) {
      const u32x4 w = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(row) + v0);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      }
    } else {
      const u32x4* s = reinterpret_cast<const u32x4*>(static_cast<const float*>(row) + v0);
      const u32x4 a = s[0], b = s[1];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[i] = __uint_as_float(a[i]);
        x[4 + i] = __uint_as_float(b[i]);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < kVec; ++i)
      x[i] = v0 + i < V ? float(load_one<DT>(row, v0 + i)) : 0.0f;
  }
}

// What weighs the ids at one node: w(v) = max(p(v) - a q(v), 0), or p without
// the ids of the rejected children (bits of `gone`, ids in LDS).
struct Weights {
  const void* p;
  const void* q;  // null: a is 0
  double a;
  uint64_t gone0, gone1;
};

__device__ __forceinline__ bool proper(float x) { return x >= 0.0f && x < INFINITY; }

// The weights of ids v0 .. v0 + 7; false if a probability among them is none.
template <int DT, bool VEC>
__device__ __forceinline__ bool weigh(const Weights& w, const int32_t* tok, int64_t v0, int64_t V,
                                      double (&x)[kVec]) {
  float p[kVec];
  load8<DT, VEC>(w.p, v0, V, p);
  bool ok = true;
  if (w.q) {
    float q[kVec];
    load8<DT, VEC>(w.q, v0, V, q);
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      ok = ok && proper(p[i]) && proper(q[i]);
      const double d = fma(-w.a, double(q[i]), double(p[i]));
      x[i] = d > 0.0 ? d : 0.0;
    }
  } else {
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      ok = ok && proper(p[i]);
      x[i] = double(p[i]);
    }
    for (uint64_t g = w.gone0; g; g &= g - 1) {
      const int64_t at = int64_t(tok[__builtin_ctzll(g)]) - v0;
#pragma unroll
      for (int i = 0; i < kVec; ++i)
        if (at == i) x[i] = 0.0;
    }
    for (uint64_t g = w.gone1; g; g &= g - 1) {
      const int64_t at = int64_t(tok[64 + __builtin_ctzll(g)]) - v0;
#pragma unroll
      for (int i = 0; i < kVec; ++i)
        if (at == i) x[i] = 0.0;
    }
  }
  return ok;
}

__device__ __forceinline__ double scan_wave(double x) {
  const int lane = int(threadIdx.x) % kWave;
#pragma unroll
  for (int d = 1; d < kWave; d *= 2) {
    const double y = __shfl_up(x, d);
    if (lane >= d) x += y;
  }
  return x;
}

struct Shared {
  double chunk[kMaxChunks];   // mass of each chunk
  double wave[2][kWaves];
  double px[SV_MAX_TREE_NODES], qx[SV_MAX_TREE_NODES], u[SV_MAX_TREE_NODES];
  int32_t tok[SV_MAX_TREE_NODES], up[SV_MAX_TREE_NODES];
  double total;
  int found;
};

// Mass of the weights: chunk sums to sm.chunk, their sum returned to every
// thread. A thread adds its 8 ids in order, a wavefront and the workgroup scan
// in a fixed order, chunks are added in order.
template <int DT, bool VEC>
__device__ double mass_of(const Weights& w, int64_t V, Shared& sm, bool* ok) {
  const int tid = int(threadIdx.x), lane = tid % kWave, wv = tid / kWave;
  const int chunks = int((V + kChunk - 1) / kChunk);
  bool good = true;
  for (int c = 0; c < chunks; ++c) {
    double x[kVec];
    good = weigh<DT, VEC>(w, sm.tok, int64_t(c) * kChunk + tid * kVec, V, x) && good;
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < kVec; ++i) s += x[i];
    s = scan_wave(s);
    if (lane == kWave - 1) sm.wave[c & 1][wv] = s;
    __syncthreads();
    if (tid == 0) {
      double t = 0.0;
      for (int k = 0; k < kWaves; ++k) t += sm.wave[c & 1][k];
      sm.chunk[c] = t;
    }
  }
  *ok = !__syncthreads_or(!good);
  if (tid == 0) {
    double t = 0.0;
    for (int c = 0; c < chunks; ++c) t += sm.chunk[c];
    sm.total = t;
  }
  __syncthreads();
  const double t = sm.total;
  __syncthreads();
  return t;
}

// The least id whose running sum exceeds x, after mass_of of the same weights;
// the last one with a weight when rounding leaves none.
template <int DT, bool VEC>
__device__ int32_t pick(const Weights& w, double x, int64_t V, Shared& sm) {
  const int tid = int(threadIdx.x), lane = tid % kWave, wv = tid / kWave;
  const int chunks = int((V + kChunk - 1) / kChunk);
  // the chunk, and the mass in front of it (every thread for itself)
  double front = 0.0, last_front = 0.0;
  int c = 0, last = -1;
  for (; c < chunks; ++c) {
    const double s = sm.chunk[c];
    if (front + s > x) break;
    if (s > 0.0) {
      last = c;
      last_front = front;
    }
    front += s;
  }
  const bool over = c == chunks;  // x is not below the whole mass
  if (over) {
    c = last;
    front = last_front;
  }
  double v[kVec];
  const int64_t v0 = int64_t(c) * kChunk + tid * kVec;
  weigh<DT, VEC>(w, sm.tok, v0, V, v);
  double s = 0.0;
#pragma unroll
  for (int i = 0; i < kVec; ++i) s += v[i];
  const double incl = scan_wave(s);
  if (lane == kWave - 1) sm.wave[0][wv] = incl;
  if (tid == 0) sm.found = over ? -1 : INT_MAX;
  __syncthreads();
  double at = front;
  for (int k = 0; k < wv; ++k) at += sm.wave[0][k];
  const double before = __shfl_up(incl, 1);
  at += lane ? before : 0.0;
  // Ids are compared by where their own running sum stands; a thread's sums
  // start from the scan of the threads before it.
  double run = 0.0;
  int32_t hit = INT_MAX, positive = -1;
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    run += v[i];
    if (v[i] > 0.0) {
      positive = int32_t(v0 + i);
      if (hit == INT_MAX && at + run > x) hit = int32_t(v0 + i);
    }
  }
  if (over) {
    if (positive >= 0) atomicMax(&sm.found, positive);
  } else if (hit != INT_MAX) {
    atomicMin(&sm.found, hit);
  }
  __syncthreads();
  int32_t got = sm.found;
  __syncthreads();
  if (!over && got == INT_MAX) {
    // the chunk's sum passed x, its ids' running sums just did not: the last one
    if (tid == 0) sm.found = -1;
    __syncthreads();
    if (positive >= 0) atomicMax(&sm.found, positive);
    __syncthreads();
    got = sm.found;
    __syncthreads();
  }
  return got;
}

// One workgroup per request: the walk is uniform over the workgroup (every
// thread runs it on the same values from LDS), the passes use all of it.
template <int DT, bool VEC>
__global__ __launch_bounds__(kBlock) void verify_kernel(VerifyArgs a) {
  __shared__ Shared sm;
  const int64_t b = blockIdx.x;
  const int tid = int(threadIdx.x);
  const Nodes nd = nodes_of(a.node_start, b, a.T, a.max_nodes);
  const int n = nd.n < 0 ? 0 : nd.n;
  int bits = nd.n < 0 ? SV_ERR_TREE : 0;

  // What the walk needs of every node: its parent, token, uniform, and its
  // token's probabilities in the parent's rows.
  bool wrong = false;
  if (tid < n) {
    const int64_t i = nd.first + tid;
    const int32_t up = a.parents[i];
    wrong = tid == 0 ? up != -1 : (up < 0 || up >= tid);
    sm.up[tid] = wrong ? -1 : up;
    const int32_t x = a.tokens[i];
    sm.tok[tid] = x;
    sm.u[tid] = a.u[i];
    const bool fits = tid > 0 && !wrong && x >= 0 && x < a.V;
    sm.px[tid] = fits ? load_one<DT>(row_at<DT>(a.p, a.ps, nd.first + up), x) : 0.0;
    sm.qx[tid] = fits && a.q ? load_one<DT>(row_at<DT>(a.q, a.qs, nd.first + up), x) : 1.0;
  }
  if (__syncthreads_or(wrong)) bits |= SV_ERR_TREE;

  int32_t* path = a.path + b * a.max_path;
  int32_t* emitted = a.emitted ? a.emitted + b * a.max_path : nullptr;
  int taken = 0;
  int32_t y = -1;
  const double r = a.r[b];
  if (n > 0 && bits == 0 && !(r >= 0.0 && r < 1.0)) bits |= SV_ERR_UNIFORM;
  if (n > 0 && bits == 0) {
    int cur = 0;
    double mass = 1.0, left = 1.0;
    Weights w{row_at<DT>(a.p, a.ps, nd.first), nullptr, 0.0, 0, 0};
    bool summed = false;  // sm.chunk holds the sums of w
    for (int i = 1; i < n && bits == 0; ++i) {
      if (sm.up[i] != cur) continue;
      const int32_t x = sm.tok[i];
      const double u = sm.u[i], px = sm.px[i], qx = sm.qx[i];
      if (x < 0 || x >= a.V) bits |= SV_ERR_TOKEN;
      if (!(u >= 0.0 && u < 1.0)) bits |= SV_ERR_UNIFORM;
      if (!(px >= 0.0 && px < INFINITY && qx >= 0.0 && qx < INFINITY)) bits |= SV_ERR_ROW;
      if (bits) break;
      double wx, qk;
      if (a.mode == SV_DRAFT_FIXED) {
        wx = px;
        for (int o = cur + 1; o < i; ++o)
          if (sm.up[o] == cur && sm.tok[o] == x) wx = 0.0;  // rejected before
        qk = 1.0;
      } else {
        const double d = fma(-w.a, qx, px);
        wx = d > 0.0 ? d : 0.0;
        qk = left > 0.0 ? qx / left : 0.0;
      }
      if (u * qk * mass < wx) {
        if (taken + 1 >= a.max_path) {
          bits |= SV_ERR_TREE;
          break;
        }
        ++taken;
        if (tid == 0) {
          path[taken] = i;
          if (emitted) emitted[taken - 1] = x;
        }
        cur = i;
        mass = left = 1.0;
        w = Weights{row_at<DT>(a.p, a.ps, nd.first + cur), nullptr, 0.0, 0, 0};
        summed = false;
      } else if (a.mode == SV_DRAFT_FIXED) {
        mass -= wx;
        if (i < 64) w.gone0 |= uint64_t(1) << i;
        else w.gone1 |= uint64_t(1) << (i - 64);
      } else if (mass > 0.0 || !summed) {
        w.q = row_at<DT>(a.q, a.qs, nd.first + cur);
        w.a += left > 0.0 ? mass / left : 0.0;
        bool ok;
        mass = mass_of<DT, VEC>(w, a.V, sm, &ok);
        summed = true;
        if (!ok) bits |= SV_ERR_ROW;
        if (a.mode == SV_DRAFT_DISTINCT) left -= qx;
      }
    }
    if (bits == 0) {
      bool ok = true;
      double total = mass;
      if (!summed) total = mass_of<DT, VEC>(w, a.V, sm, &ok);
      if (ok && !(total > 0.0) && (w.q || w.gone0 || w.gone1)) {
        // nothing left by rounding: from the target's row itself
        w = Weights{w.p, nullptr, 0.0, 0, 0};
        total = mass_of<DT, VEC>(w, a.V, sm, &ok);
      }
      if (!ok || !(total > 0.0)) bits |= SV_ERR_ROW;
      else y = pick<DT, VEC>(w, r * total, a.V, sm);
    }
  }
  const bool none = n == 0 || bits != 0;
  __syncthreads();
  for (int i = tid; i < a.max_path; i += kBlock) {
    if (none || i > taken) path[i] = -1;
    if (emitted && (none || i > taken)) emitted[i] = -1;
  }
  if (tid == 0) {
    if (!none) {
      path[0] = 0;
      if (emitted) emitted[taken] = y;
    }
    a.accept_len[b] = none ? -1 : taken;
    a.out_token[b] = none ? -1 : y;
    if (bits) set_error(a.err, bits);
  }
}

bool sizes_ok(int64_t B, int64_t V, int64_t max_nodes) {
  return B >= 1 && B < (int64_t(1) << 31) && V >= 1 && V <= SV_MAX_TREE_VOCAB && max_nodes >= 1 &&
         max_nodes <= SV_MAX_TREE_NODES;
}

}  // namespace

extern "C" {

size_t specverify_tree_verify_workspace_size(int64_t B, int64_t V, int64_t max_nodes) {
  return sizes_ok(B, V, max_nodes) ? 256 : 0;
}

int specverify_tree_verify(const void* target_probs, const void* draft_probs, int dtype, int mode,
                           const int32_t* tokens, const int32_t* parents,
                           const int32_t* node_start, int64_t B, int64_t T, int64_t V,
                           int64_t max_nodes, int64_t max_path, int64_t t_stride, int64_t d_stride,
                           const double* u, const double* r, int32_t* accept_len, int32_t* path,
                           int32_t* emitted, int32_t* out_token, int32_t* device_error,
                           void* workspace, size_t workspace_bytes, void* stream) {
  if (!node_start || !r || !accept_len || !path || !out_token) return SV_EINVAL;
  if (T > 0 && (!target_probs || !tokens || !parents || !u)) return SV_EINVAL;
  if (mode != SV_DRAFT_FIXED && mode != SV_DRAFT_IID && mode != SV_DRAFT_DISTINCT)
    return SV_EINVAL;
  if (mode == SV_DRAFT_FIXED ? draft_probs != nullptr : (T > 0 && !draft_probs)) return SV_EINVAL;
  if (!sizes_ok(B, V, max_nodes) || T < 0 || T >= (int64_t(1) << 31) || max_path < 1 ||
      max_path > max_nodes || t_stride < 0 || d_stride < 0)
    return SV_EINVAL;
  if (dtype != SV_F32 && dtype != SV_BF16) return SV_EDTYPE;
  int st = SV_OK;
  if (!workspace_ok(workspace, workspace_bytes,
                    specverify_tree_verify_workspace_size(B, V, max_nodes), &st))
    return st;
  const int esz = dtype == SV_BF16 ? 2 : 4;
  const bool vec = aligned16(target_probs) && aligned16(draft_probs) &&
                   t_stride * esz % 16 == 0 && d_stride * esz % 16 == 0;
  VerifyArgs a{target_probs, draft_probs, t_stride, d_stride, tokens, parents, node_start, u, r, T,
               V, int(max_nodes), int(max_path), mode, accept_len, path, emitted, out_token,
               device_error};
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const dim3 grid{unsigned(B)}, block{kBlock};
  if (dtype == SV_BF16) {
    if (vec) hipLaunchKernelGGL((verify_kernel<SV_BF16, true>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((verify_kernel<SV_BF16, false>), grid, block, 0, s, a);
  } else {
    if (vec) hipLaunchKernelGGL((verify_kernel<SV_F32, true>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((verify_kernel<SV_F32, false>), grid, block, 0, s, a);
  }
  return launch_status();
}

}  // extern "C"
