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
//
// What bounds it is the chain of those passes: one is 1 MB of two float32 rows at
// V = 128256, about 4 us with its sums gathered from 8 workgroups, and none can
// begin before the one before has decided: 24 trees of 33 nodes 36 us. A chain
// takes one pass, for the rejected child or at its end (a second one only if
// rounding leaves no weight). 64 chains of 9 nodes take 15.5 us at V = 32768, 16 us
// at 65536 and 24 us at 128256, where 66 MB of rows would take 14 us; one chain at
// V = 32000 13.5 us. So a walk of one pass costs some 13 us whatever the rows: trips to
// memory that wait for each other (the request, its tokens, their probabilities, the
// rows, the other workgroups' sums, the drawn chunk again).

#include "tree_common.h"

namespace {

using namespace svtree;

constexpr int kBlock = 512;
constexpr int kWaves = kBlock / kWave;
constexpr int kVec = 8;                   // probabilities of a thread in a chunk
constexpr int kChunk = kBlock * kVec;     // 4096
constexpr int kMaxChunks = SV_MAX_TREE_VOCAB / kChunk;
// Workgroups that a call is spread over at most: two to a CU, all resident when
// the card is free.
constexpr int kWorkers = 512;
// What a workgroup waits for the others' sums, in ticks of the 100 MHz clock,
// before it takes them itself.
constexpr uint64_t kPatience = 2000;
constexpr uint64_t kEmpty = ~uint64_t(0);           // a sum not yet there
constexpr uint64_t kWrong = 0xFFF8000000000001ull;  // the chunk holds what is no probability

// In the build with index checks every second workgroup of a request finds runs
// of the others' sums missing, in some groups taken at once all, in some a few:
// what a workgroup does that has waited in vain runs wherever several share a row.
__device__ __forceinline__ bool in_vain(int share, int chunk) {
#ifdef SV_DEVICE_CHECKS
  return share % 2 == 1 && chunk / 6 % 2 == 0;
#else
  return false;
#endif
}

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
  int spread, chunks;  // workgroups of a request, chunks of a row
  uint64_t* sums;      // [B][max_nodes + 1][chunks], kEmpty at the start (spread > 1)
  int32_t* accept_len;
  int32_t* path;
  int32_t* emitted;
  int32_t* out_token;
  int32_t* err;
  int64_t B;
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

// 8 probabilities from v0 on as float32 (exact); 0 behind the row's end. VEC: rows
// begin at multiples of 16 bytes.
template <int DT, bool VEC>
__device__ __forceinline__ void load8(const void* row, int64_t v0, int64_t V, float (&x)[kVec]) {
  if (v0 + kVec <= V) {
    if constexpr (DT == SV_BF16) {
      const uint16_t* s = static_cast<const uint16_t*>(row) + v0;
      u32x4 w;
      if constexpr (VEC) {
        w = *reinterpret_cast<const u32x4*>(s);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = uint32_t(s[2 * i]) | uint32_t(s[2 * i + 1]) << 16;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      }
    } else {
      const float* s = static_cast<const float*>(row) + v0;
      if constexpr (VEC) {
        const u32x4 a = reinterpret_cast<const u32x4*>(s)[0];
        const u32x4 b = reinterpret_cast<const u32x4*>(s)[1];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[i] = __uint_as_float(a[i]);
          x[4 + i] = __uint_as_float(b[i]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < kVec; ++i) x[i] = s[i];
      }
    }
  } else {
#pragma unroll 1
    for (int i = 0; i < kVec; ++i) {
      const float y = v0 + i < V ? float(load_one<DT>(row, v0 + i)) : 0.0f;
#pragma unroll
      for (int j = 0; j < kVec; ++j)
        if (i == j) x[j] = y;
    }
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

// Target and draft probabilities of ids v0 .. v0 + 7.
struct Probs {
  float p[kVec], q[kVec];
};

template <int DT, bool VEC>
__device__ __forceinline__ void read_probs(const void* p, const void* q, int64_t v0, int64_t V,
                                           Probs& r) {
  load8<DT, VEC>(p, v0, V, r.p);
  if (q) load8<DT, VEC>(q, v0, V, r.q);
}

// The weights of these ids; false if a probability among them is none.
__device__ __forceinline__ bool weigh(const Weights& w, const int32_t* tok, int64_t v0,
                                      const Probs& r, double (&x)[kVec]) {
  bool ok = true;
  if (w.q) {
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      ok = ok && proper(r.p[i]) && proper(r.q[i]);
      const double d = fma(-w.a, double(r.q[i]), double(r.p[i]));
      x[i] = d > 0.0 ? d : 0.0;
    }
  } else {
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      ok = ok && proper(r.p[i]);
      x[i] = double(r.p[i]);
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
  double front[kMaxChunks];   // mass of the chunks up to and with each
  uint64_t some[kMaxChunks / kWave];  // a bit for each chunk that has mass itself
  double wave[4][kWaves];
  double px[SV_MAX_TREE_NODES], qx[SV_MAX_TREE_NODES], u[SV_MAX_TREE_NODES];
  int32_t tok[SV_MAX_TREE_NODES], up[SV_MAX_TREE_NODES];
  int found, found_chunk;
};

// Masses of the chunks c .. c + kAtOnce - 1 below c1, as their bits or kWrong: of
// chunk c + u to thread u. A thread adds its 8 ids in order, a wavefront and the
// workgroup in a fixed order, so whichever workgroup takes a chunk gets the same
// bits. Several at once, because one chunk's loads are not enough in flight.
template <bool VEC>
constexpr int kAtOnce = VEC ? 4 : 1;
template <bool VEC>
struct Held {
  Probs x[kAtOnce<VEC>];
};
// (behind the range: its last chunk again, not used)
template <int DT, bool VEC>
__device__ __forceinline__ void hold(Held<VEC>& h, const void* p, const void* q, int64_t V, int c,
                                     int c1) {
#pragma unroll
  for (int u = 0; u < kAtOnce<VEC>; ++u)
    read_probs<DT, VEC>(p, q, int64_t(c + u < c1 ? c + u : c1 - 1) * kChunk + threadIdx.x * kVec, V,
                        h.x[u]);
}
template <bool VEC, typename Get>  // get(u): the probabilities of chunk c + u
__device__ __forceinline__ uint64_t chunk_masses(const Weights& w, Get get, Shared& sm, int c,
                                                 int c1) {
  const int tid = int(threadIdx.x), lane = tid % kWave, wv = tid / kWave;
  double s[kAtOnce<VEC>];
  bool good[kAtOnce<VEC>];
#pragma unroll
  for (int u = 0; u < kAtOnce<VEC>; ++u) {
    double x[kVec];
    const int64_t at = c + u < c1 ? c + u : c1 - 1;
    good[u] = weigh(w, sm.tok, at * kChunk + tid * kVec, get(u), x);
    s[u] = 0.0;
#pragma unroll
    for (int i = 0; i < kVec; ++i) s[u] += x[i];
  }
#pragma unroll
  for (int u = 0; u < kAtOnce<VEC>; ++u) {
    s[u] = scan_wave(s[u]);
    if (__any(!good[u])) s[u] = __longlong_as_double((long long)kWrong);  // stays in every sum
  }
  __syncthreads();  // the sums before are read
  if (lane == kWave - 1)
#pragma unroll
    for (int u = 0; u < kAtOnce<VEC>; ++u) sm.wave[u][wv] = s[u];
  __syncthreads();
  if (tid >= kAtOnce<VEC>) return kEmpty;
  double t = 0.0;
#pragma unroll
  for (int k = 0; k < kWaves; ++k) t += sm.wave[tid][k];
  return t != t ? kWrong : (uint64_t)__double_as_longlong(t);
}

// Mass of the weights: running sums of the chunks to sm.front, which of them have
// any to sm.some, the whole returned to every thread (NaN for a wrong row).
//
// The workgroups of a request run the same walk side by side; each takes its
// share of a pass's chunks and publishes their sums, which are value and flag in
// one 64-bit word. Nothing depends on all of them being resident at once: one
// that has waited long enough takes what is missing itself (the same bits).
//
// KEEP: a workgroup has no more chunks than it takes at once, so a node's rows stay
// in registers for its further rejections (24 trees of 33 nodes at V = 128256: 37
// us so, 42 us read again; reading the next child's rows ahead on top of it cost
// 8 us, because the other workgroups' sums queue behind those loads).
template <int DT, bool VEC, bool KEEP>
__device__ __forceinline__ double mass_of(const VerifyArgs& a, const Weights& w, uint64_t* sums,
                                          int share, Shared& sm, Held<VEC>& held,
                                          bool& here) {
  const int tid = int(threadIdx.x), lane = tid % kWave;
  const int chunks = a.chunks;
  int c0 = int(int64_t(chunks) * share / a.spread);
  int c1 = int(int64_t(chunks) * (share + 1) / a.spread);
  if (!sv_ok(0 <= c0 && c0 < c1 && c1 <= chunks)) return NAN;
  for (bool own = true;; own = false) {
    for (int c = c0; c < c1; c += kAtOnce<VEC>) {
      if (!own) {  // only where one is missing
        bool there = true;
        for (int u = c; u < c + kAtOnce<VEC> && u < c1; ++u)
          there = there && (uint64_t)__double_as_longlong(sm.front[u]) != kEmpty;
        if (there) continue;
      }
      uint64_t s;
      if constexpr (KEEP) {
        if (!here || !own) hold<DT, VEC>(held, w.p, w.q, a.V, c, c1);
        here = own;
        s = chunk_masses<VEC>(w, [&](int u) -> const Probs& { return held.x[u]; }, sm, c, c1);
      } else {
        s = chunk_masses<VEC>(
            w,
            [&](int u) {
              Probs r;
              read_probs<DT, VEC>(w.p, w.q, int64_t(c + u < c1 ? c + u : c1 - 1) * kChunk + tid * kVec,
                                  a.V, r);
              return r;
            },
            sm, c, c1);
      }
      if (tid < kAtOnce<VEC> && c + tid < c1) {
        sm.front[c + tid] = __longlong_as_double((long long)s);
        if (own && a.spread > 1)
          __hip_atomic_store(sums + c + tid, s, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
    }
    if (!own || a.spread == 1) break;
    bool missing = false;
    const uint64_t began = wall_clock64();
    for (int c = tid; c < chunks; c += kBlock) {
      if (c >= c0 && c < c1) continue;
      uint64_t s = __hip_atomic_load(sums + c, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      while (s == kEmpty && wall_clock64() - began < kPatience) {
        __builtin_amdgcn_s_sleep(1);
        s = __hip_atomic_load(sums + c, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
      if (in_vain(share, c)) s = kEmpty;
      missing = missing || s == kEmpty;
      sm.front[c] = __longlong_as_double((long long)s);
    }
    if (!__syncthreads_or(missing)) break;
    c0 = 0;
    c1 = chunks;
  }
  __syncthreads();
  if (tid < kWave) {
    double before = 0.0;
    for (int c = lane; c - lane < chunks; c += kWave) {
      const double own = c < chunks ? sm.front[c] : 0.0;
      const uint64_t some = __ballot(own > 0.0);
      if (lane == 0) sm.some[c / kWave] = some;
      const double s = before + scan_wave(own);
      if (c < chunks) sm.front[c] = s;
      before = __shfl(s, kWave - 1);
    }
  }
  __syncthreads();
  return sm.front[chunks - 1];
}

// The least id whose running sum exceeds x, after mass_of of the same weights;
// the last one with a weight when rounding leaves none. -1 from a workgroup that
// does not own the id's chunk.
//
// The scan adds the chunks before two neighbours in different orders, so their
// running sums may differ in the last bit with no mass between them: a chunk
// without mass is never taken, whatever its running sum.
template <int DT, bool VEC>
__device__ __forceinline__ int32_t pick(const VerifyArgs& a, const Weights& w, double x, int share, Shared& sm,
                        bool* mine) {
  const int tid = int(threadIdx.x), lane = tid % kWave, wv = tid / kWave;
  const int chunks = a.chunks;
  const double whole = sm.front[chunks - 1];
  const bool over = !(x < whole);
  int word = (chunks - 1) / kWave;
  while (word > 0 && !sm.some[word]) --word;
  if (tid == 0) sm.found_chunk = word * kWave + kWave - 1 - __builtin_clzll(sm.some[word] | 1);
  __syncthreads();
  // the first chunk with mass whose running sum passes x, or the last with mass
  for (int c = tid; c < chunks && !over; c += kBlock)
    if ((sm.some[c / kWave] >> (c % kWave) & 1) && sm.front[c] > x) {
      atomicMin(&sm.found_chunk, c);
      break;
    }
  __syncthreads();
  const int c = sm.found_chunk;
  *mine = c >= int(int64_t(chunks) * share / a.spread) &&
          c < int(int64_t(chunks) * (share + 1) / a.spread);
  if (!*mine || !sv_ok(c >= 0)) return -1;
  double v[kVec];
  const int64_t v0 = int64_t(c) * kChunk + tid * kVec;
  Probs probs;
  read_probs<DT, VEC>(w.p, w.q, v0, a.V, probs);
  weigh(w, sm.tok, v0, probs, v);
  double s = 0.0;
#pragma unroll
  for (int i = 0; i < kVec; ++i) s += v[i];
  const double incl = scan_wave(s);
  if (lane == kWave - 1) sm.wave[0][wv] = incl;
  if (tid == 0) sm.found = over ? -1 : INT_MAX;
  __syncthreads();
  double at = c > 0 ? sm.front[c - 1] : 0.0;
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

// a.spread workgroups per request. The walk is uniform over a workgroup, and the
// same in all of a request's: every thread runs it on the same values.
template <int DT, bool VEC, bool KEEP>
__global__ __launch_bounds__(kBlock) void verify_kernel(VerifyArgs a) {
  __shared__ Shared sm;
  const int64_t b = int64_t(blockIdx.x) / a.spread;
  const int share = int(int64_t(blockIdx.x) - b * a.spread);
  const int tid = int(threadIdx.x), lane = tid % kWave;
  const Nodes nd = nodes_of(a.node_start, b, a.T, a.max_nodes);
  const int n = nd.n < 0 ? 0 : nd.n;
  if (!sv_ok(b < a.B && nd.first + n <= a.T)) return;
  int bits = nd.n < 0 ? SV_ERR_TREE : 0;

  // What the walk needs of every node: its parent, token, uniform, and its
  // token's probabilities in the parent's rows.
  bool wrong = false;
  if (tid < n) {
    const int64_t i = nd.first + tid;
    const int32_t up = a.parents[i];
    const int32_t x = a.tokens[i];
    sm.u[tid] = a.u[i];
    wrong = tid == 0 ? up != -1 : (up < 0 || up >= tid);
    sm.up[tid] = wrong ? -1 : up;
    sm.tok[tid] = x;
    const bool fits = tid > 0 && !wrong && x >= 0 && x < a.V;
    sm.px[tid] = fits ? load_one<DT>(row_at<DT>(a.p, a.ps, nd.first + up), x) : 0.0;
    sm.qx[tid] = fits && a.q ? load_one<DT>(row_at<DT>(a.q, a.qs, nd.first + up), x) : 1.0;
  }
  const double r = a.r[b];
  if (__syncthreads_or(wrong)) bits |= SV_ERR_TREE;

  // The accepted path is kept by the lanes of wavefront 0: lane l has nodes l and
  // l + 64 of it.
  int32_t step0 = 0, step1 = 0;
  int taken = 0;
  int32_t y = -1;
  bool mine = share == 0;  // who writes: the owner of the drawn id's chunk, or the first
  if (n > 0 && bits == 0 && !(r >= 0.0 && r < 1.0)) bits |= SV_ERR_UNIFORM;
  if (n > 0 && bits == 0) {
    const int up0 = lane < n ? sm.up[lane] : -2, up1 = 64 + lane < n ? sm.up[64 + lane] : -2;
    const int tok0 = lane < n ? sm.tok[lane] : -1, tok1 = 64 + lane < n ? sm.tok[64 + lane] : -1;
    uint64_t* sums = a.sums + b * (a.max_nodes + 1) * int64_t(a.chunks);
    int cur = 0;
    uint64_t kids0 = __ballot(up0 == 0), kids1 = __ballot(up1 == 0);
    double mass = 1.0, left = 1.0;
    Weights w{row_at<DT>(a.p, a.ps, nd.first), nullptr, 0.0, 0, 0};
    bool summed = false;  // sm.front holds the sums of w
    Held<VEC> held;
    int held_node = -1;  // whose rows they are
    // Walk to the next rejection or the end, take the sums that it needs, go on.
    while (true) {
      bool rejected = false;
      while ((kids0 | kids1) && !rejected) {
        const int i = kids0 ? __builtin_ctzll(kids0) : 64 + __builtin_ctzll(kids1);
        if (kids0) kids0 &= kids0 - 1;
        else kids1 &= kids1 - 1;
        const int32_t x = sm.tok[i];
        const double u = sm.u[i], px = sm.px[i], qx = sm.qx[i];
        if (x < 0 || x >= a.V) bits |= SV_ERR_TOKEN;
        if (!(u >= 0.0 && u < 1.0)) bits |= SV_ERR_UNIFORM;
        if (!(px >= 0.0 && px < INFINITY && qx >= 0.0 && qx < INFINITY)) bits |= SV_ERR_ROW;
        if (bits) break;
        double wx, qk;
        if (a.mode == SV_DRAFT_FIXED) {
          // zero if it was rejected before
          wx = (__ballot(tok0 == x) & w.gone0) | (__ballot(tok1 == x) & w.gone1) ? 0.0 : px;
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
          if (lane == (taken & 63)) (taken < 64 ? step0 : step1) = i;
          cur = i;
          kids0 = __ballot(up0 == cur);
          kids1 = __ballot(up1 == cur);
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
          if (a.mode == SV_DRAFT_DISTINCT) left -= qx;
          rejected = true;
        }
      }
      if (bits) break;
      if (!rejected && summed) {
        if (mass > 0.0) break;
        if (!w.q && !w.gone0 && !w.gone1) {
          bits |= SV_ERR_ROW;
          break;
        }
        // nothing left by rounding: from the target's row itself
        w = Weights{w.p, nullptr, 0.0, 0, 0};
      }
      if (!sv_ok(cur < n && (a.spread == 1 ||
                             sums + a.chunks <= a.sums + (b + 1) * (a.max_nodes + 1) * a.chunks))) {
        bits |= SV_ERR_ROW;
        break;
      }
      bool here = held_node == cur;
      mass = mass_of<DT, VEC, KEEP>(a, w, sums, share, sm, held, here);
      held_node = here ? cur : -1;
      sums += a.chunks;
      summed = true;
      if (mass != mass) {
        bits |= SV_ERR_ROW;
        break;
      }
    }
    if (bits == 0) y = pick<DT, VEC>(a, w, r * mass, share, sm, &mine);
  }
  const bool none = n == 0 || bits != 0;
  if (!mine || tid >= kWave) return;
  if (!sv_ok(taken < a.max_path)) return;
  int32_t* path = a.path + b * a.max_path;
  int32_t* emitted = a.emitted ? a.emitted + b * a.max_path : nullptr;
  for (int i = lane; i < a.max_path; i += kWave) {
    const bool on = !none && i <= taken;
    path[i] = on ? (i < 64 ? step0 : step1) : -1;
    if (emitted && !(on && i < taken)) emitted[i] = on ? y : -1;
    if (emitted && on && i > 0) emitted[i - 1] = sm.tok[i < 64 ? step0 : step1];
  }
  if (lane == 0) {
    a.accept_len[b] = none ? -1 : taken;
    a.out_token[b] = none ? -1 : y;
    if (bits) set_error(a.err, bits);
  }
}

__global__ __launch_bounds__(256) void clear_kernel(uint64_t* x, int64_t n) {
  for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < n; i += int64_t(gridDim.x) * 256)
    x[i] = kEmpty;
}

// Workgroups of a request: enough to fill the card, each with the chunks that it
// takes at once; with fewer, the sums travel longer than they take (rows read in
// every pass, 24 trees of 33 nodes at V = 128256: 42 us so, 65 us with a chunk
// each, 57 us with 8; one chain at V = 32000: 13 us so, 19 us with a chunk each).
int spread_of(int64_t B, int64_t chunks) {
  const int64_t shares = chunks / kAtOnce<true>, most = kWorkers / B;
  return int(most < 1 || shares < 1 ? 1 : most < shares ? most : shares);
}

bool sizes_ok(int64_t B, int64_t V, int64_t max_nodes) {
  return B >= 1 && B < (int64_t(1) << 31) && V >= 1 && V <= SV_MAX_TREE_VOCAB && max_nodes >= 1 &&
         max_nodes <= SV_MAX_TREE_NODES;
}

}  // namespace

#ifdef SV_DEVICE_CHECKS
bool sv_add_tree_verify_checks(uint32_t* count, int reset) { return sv_add_checks(count, reset); }
#endif

extern "C" {

size_t specverify_tree_verify_workspace_size(int64_t B, int64_t V, int64_t max_nodes) {
  if (!sizes_ok(B, V, max_nodes)) return 0;
  const int64_t chunks = (V + kChunk - 1) / kChunk;
  if (spread_of(B, chunks) == 1) return 256;
  return align256(size_t(B) * size_t(max_nodes + 1) * size_t(chunks) * 8);
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
      max_path > max_nodes || !stride_ok(t_stride) || !stride_ok(d_stride))
    return SV_EINVAL;
  if (dtype != SV_F32 && dtype != SV_BF16) return SV_EDTYPE;
  int st = SV_OK;
  if (!workspace_ok(workspace, workspace_bytes,
                    specverify_tree_verify_workspace_size(B, V, max_nodes), &st))
    return st;
  const int esz = dtype == SV_BF16 ? 2 : 4;
  const bool vec = aligned16(target_probs) && aligned16(draft_probs) &&
                   t_stride * esz % 16 == 0 && d_stride * esz % 16 == 0;
  const int64_t chunks = (V + kChunk - 1) / kChunk;
  const int spread = spread_of(B, chunks);
  if (B * spread >= (int64_t(1) << 31)) return SV_EINVAL;
  uint64_t* sums = static_cast<uint64_t*>(workspace);
  VerifyArgs a{target_probs, draft_probs, t_stride, d_stride, tokens, parents, node_start, u, r, T,
               V, int(max_nodes), int(max_path), mode, spread, int(chunks), sums, accept_len, path,
               emitted, out_token, device_error, B};
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (spread > 1) {
    const int64_t words = B * (max_nodes + 1) * chunks, blocks = (words + 1023) / 1024;
    hipLaunchKernelGGL(clear_kernel, dim3(unsigned(blocks < 2048 ? blocks : 2048)), dim3(256), 0, s,
                       sums, words);
  }
  const dim3 grid{unsigned(B * spread)}, block{kBlock};
  // Held rows take the registers of a second workgroup on the CU: not where the
  // grid needs it, nor for chains and given drafts, whose walks take one pass.
  const bool keep = vec && mode != SV_DRAFT_FIXED && spread > 1 && B * spread <= kWorkers / 2 &&
                    (chunks + spread - 1) / spread <= kAtOnce<true>;
  if (dtype == SV_BF16) {
    if (keep) hipLaunchKernelGGL((verify_kernel<SV_BF16, true, true>), grid, block, 0, s, a);
    else if (vec) hipLaunchKernelGGL((verify_kernel<SV_BF16, true, false>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((verify_kernel<SV_BF16, false, false>), grid, block, 0, s, a);
  } else {
    if (keep) hipLaunchKernelGGL((verify_kernel<SV_F32, true, true>), grid, block, 0, s, a);
    else if (vec) hipLaunchKernelGGL((verify_kernel<SV_F32, true, false>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((verify_kernel<SV_F32, false, false>), grid, block, 0, s, a);
  }
  return launch_status();
}

}  // extern "C"
