// Host-code driver of the operators around a verification step for a build of the
// library's host side under AddressSanitizer and UndefinedBehaviorSanitizer
// (tests/test_sanitized_serving_host.py compiles and runs it; no GPU is used). The
// entry points are called only with arguments that their host checks reject, each
// size and stride at its ends among them, so no HIP call is made; the workspace
// sizes run for real. Prints one line per check; exits with the number of failed
// checks.
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <initializer_list>
#include <limits>

#include "specverify_serving.h"

static int failed = 0;

static void expect(const char* what, long long at, long long got, long long want) {
  const bool ok = got == want;
  if (!ok) std::printf("FAIL %s %lld got %lld want %lld\n", what, at, got, want);
  else std::printf("ok %s %lld\n", what, at);
  if (!ok) ++failed;
}

static const int64_t kMost = std::numeric_limits<int64_t>::max();
static const int64_t kLeast = std::numeric_limits<int64_t>::min();

// Fake device pointers: never dereferenced.
alignas(256) static char fake[1024];
static int32_t* ip = reinterpret_cast<int32_t*>(fake);
static int32_t* jp = reinterpret_cast<int32_t*>(fake + 256);
static int64_t* lp = reinterpret_cast<int64_t*>(fake);
static float* fp = reinterpret_cast<float*>(fake);

struct Resize {
  int64_t s[7] = {2, 5, 16, 8, 8, 20, 20};  // B, T, page_size, max_pages, stride, num_pages, num_free
  size_t bytes = 0;
  int operator()() const {
    return specverify_pages_resize(ip, ip, ip, ip, ip, ip, ip, s[0], s[1], s[2], s[3], s[4], s[5],
                                   s[6], jp, jp, jp, ip, lp, nullptr, fake, bytes, nullptr);
  }
};

struct Fork {
  int dtype = SV_BF16;
  // forks, B, layers, H, D, strides of the cache, page_size, max_pages, stride, num_pages, num_free
  int64_t s[14] = {3, 4, 2, 2, 64, 40960, 2048, 128, 64, 16, 8, 8, 20, 4};
  size_t bytes = 0;
  int operator()() const {
    return specverify_pages_fork(ip, ip, ip, ip, ip, ip, ip, ip, fake, fake, dtype, s[0], s[1], s[2],
                                 s[3], s[4], s[5], s[6], s[7], s[8], s[9], s[10], s[11], s[12], s[13],
                                 jp, jp, jp, jp, nullptr, fake, bytes, nullptr);
  }
};

struct Rotate {
  int dtype = SV_BF16, weight = SV_BF16;
  int64_t s[5] = {5, 4, 2, 64, 64};  // T, Hq, Hkv, D, R
  int64_t strides[11] = {512, 64, 512, 64, 256, 64, 128, 64, 2048, 128, 64};
  int64_t num_pages = 9, page_size = 16;
  float eps = 1e-6f;
  int operator()() const {
    return specverify_rotate(fake, fake, fake, dtype, s[0], s[1], s[2], s[3], s[4], 0, strides[0],
                             strides[1], strides[2], strides[3], fake, fake, weight, eps, ip, fp, fake,
                             strides[4], strides[5], fake, strides[6], strides[7], lp, fake, fake,
                             strides[8], strides[9], strides[10], num_pages, page_size, nullptr,
                             nullptr);
  }
};

struct Attention {
  int64_t s[6] = {2, 5, 4, 2, 64, 4};  // B, T, Hq, Hkv, D, max_chunk
  int64_t strides[7] = {256, 64, 2048, 128, 64, 256, 64};
  int64_t num_pages = 9, page_size = 16, max_pages = 8, table_stride = 8;
  float scale = 0.125f;
  size_t bytes = 0;
  int operator()() const {
    return specverify_chunk_attention(fake, fake, fake, SV_BF16, s[0], s[1], s[2], s[3], s[4], s[5],
                                      strides[0], strides[1], strides[2], strides[3], strides[4],
                                      num_pages, page_size, ip, max_pages, table_stride, ip, ip, scale,
                                      fake, strides[5], strides[6], nullptr, nullptr, fake, bytes,
                                      nullptr);
  }
};

struct Penalize {
  int dtype = SV_F32;
  // B, T, V, max_nodes, max_history, num_bias, strides of logits, out, history, mask
  int64_t s[10] = {2, 5, 100, 4, 30, 6, 100, 100, 30, 4};
  int operator()() const {
    return specverify_penalize(fake, dtype, ip, ip, nullptr, ip, ip, ip, fp, fp, fp, ip, ip, fp, ip,
                               s[0], s[1], s[2], s[3], s[4], s[5], s[6], s[7], s[8], s[9], fake + 256,
                               dtype, nullptr, nullptr);
  }
};

int main() {
  const int64_t ends[] = {kMost, kMost - 7, kMost / 2 + 1, kMost / 4 + 1, kLeast, -1};
  for (int64_t x : ends) {
    for (int i = 0; i < 7; ++i) {
      Resize r;
      r.s[i] = x;
      expect("resize size", i, r(), SV_EINVAL);
    }
    for (int i = 0; i < 14; ++i)
      for (int dtype : {SV_F32, SV_BF16, SV_F16}) {
        Fork f;
        f.s[i] = x;
        f.dtype = dtype;
        expect("fork size", i, f(), SV_EINVAL);
      }
    for (int i = 0; i < 5; ++i) {
      Rotate r;
      r.s[i] = x;
      expect("rotate size", i, r(), SV_EINVAL);
    }
    for (int i = 0; i < 11; ++i)
      for (int dtype : {SV_F32, SV_BF16, SV_F16}) {
        Rotate r;
        r.dtype = r.weight = dtype;
        r.strides[i] = x;
        expect("rotate stride", i, r(), SV_EINVAL);
      }
    for (int i = 0; i < 2; ++i) {
      Rotate r;
      (i == 0 ? r.num_pages : r.page_size) = x;
      expect("rotate cache", i, r(), SV_EINVAL);
    }
    for (int i = 0; i < 6; ++i) {
      Attention a;
      a.s[i] = x;
      expect("attention size", i, a(), SV_EINVAL);
      expect("attention workspace", i,
             (long long)specverify_chunk_attention_workspace_size(a.s[0], a.s[1], a.s[2], a.s[3],
                                                                  a.s[4], a.s[5]),
             0);
    }
    for (int i = 0; i < 7; ++i) {
      Attention a;
      a.strides[i] = x;
      expect("attention stride", i, a(), SV_EINVAL);
    }
    for (int i = 0; i < 4; ++i) {
      Attention a;
      (i == 0 ? a.num_pages : i == 1 ? a.page_size : i == 2 ? a.max_pages : a.table_stride) = x;
      expect("attention cache", i, a(), SV_EINVAL);
    }
    for (int i = 0; i < 10; ++i)
      for (int dtype : {SV_F32, SV_BF16}) {
        Penalize p;
        p.s[i] = x;
        p.dtype = dtype;
        expect("penalize size", i, p(), SV_EINVAL);
      }
    expect("resize workspace", 0, (long long)specverify_pages_resize_workspace_size(x, 5), 0);
    expect("resize workspace", 1, (long long)specverify_pages_resize_workspace_size(5, x), 0);
    expect("fork workspace", 0, (long long)specverify_pages_fork_workspace_size(x, 5), 0);
    expect("fork workspace", 1, (long long)specverify_pages_fork_workspace_size(5, x), 0);
  }
  for (float x : {-1.0f, INFINITY, NAN}) {
    Rotate r;
    r.eps = x;
    expect("rotate eps", 0, r(), SV_EINVAL);
  }
  for (float x : {0.0f, -1.0f, INFINITY, NAN, 3e38f}) {
    Attention a;
    a.scale = x;
    expect("attention scale", 0, a(), SV_EINVAL);
  }
  // what is allowed reaches the workspace's check
  expect("attention workspace of nothing", 0, Attention()(), SV_EWORKSPACE);
  expect("resize workspace of nothing", 0, Resize()(), SV_EWORKSPACE);
  expect("fork workspace of nothing", 0, Fork()(), SV_EWORKSPACE);
  // the largest sizes of the library
  const int64_t k31 = int64_t(1) << 31;
  expect("attention largest", 0, specverify_chunk_attention_workspace_size(1 << 24, k31 - 1, 1, 1, 256, k31 - 1) > 0, 1);
  expect("attention largest", 1, specverify_chunk_attention_workspace_size(1, 1, 1 << 24, 1 << 24, 8, k31 - 1) > 0, 1);
  expect("resize largest", 0, specverify_pages_resize_workspace_size(SV_MAX_PAGE_BATCH, SV_MAX_CACHE_PAGES) > 0, 1);
  expect("fork largest", 0, specverify_pages_fork_workspace_size(SV_MAX_PAGE_BATCH, SV_MAX_PAGE_BATCH) > 0, 1);
  std::printf("failed %d\n", failed);
  return failed > 100 ? 100 : failed;
}
