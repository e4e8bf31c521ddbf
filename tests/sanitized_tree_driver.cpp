// Host-code driver of the operators on drafted trees for a build of the library's
// host side under AddressSanitizer and UndefinedBehaviorSanitizer
// (tests/test_sanitized_tree_host.py compiles and runs it; no GPU is used). The
// entry points are called only with arguments that their host checks reject, each
// size and stride at its ends among them, so no HIP call is made; the workspace
// sizes run for real. Prints one line per check; exits with the number of failed
// checks.
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <initializer_list>
#include <limits>

#include "specverify_tree.h"

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
static int64_t* lp = reinterpret_cast<int64_t*>(fake);
static uint64_t* up = reinterpret_cast<uint64_t*>(fake);
static float* fp = reinterpret_cast<float*>(fake);
static double* dp = reinterpret_cast<double*>(fake);

struct Plan {
  int64_t s[9] = {2, 5, 4, 3, 16, 8, 8, 20, 4};  // B, T, max_nodes .. num_free
  int operator()() const {
    return specverify_tree_plan(ip, ip, ip, ip, ip, ip, ip, s[0], s[1], s[2], s[3], s[4], s[5],
                                s[6], s[7], s[8], up, ip, ip, lp, ip + 4, ip + 4, nullptr, nullptr);
  }
};

struct Attention {
  int64_t s[6] = {2, 5, 4, 2, 64, 4};                        // B, T, Hq, Hkv, D, max_nodes
  int64_t strides[9] = {256, 64, 128, 64, 2048, 128, 64, 256, 64};  // q, nodes, cache, out
  int64_t num_pages = 9, page_size = 16, max_pages = 8, table_stride = 8;
  float scale = 0.125f;
  size_t bytes = size_t(1) << 40;
  int operator()() const {
    return specverify_tree_attention(
        fake, fake, fake, fake, fake, SV_BF16, s[0], s[1], s[2], s[3], s[4], s[5], strides[0],
        strides[1], strides[2], strides[3], strides[4], strides[5], strides[6], num_pages,
        page_size, ip, max_pages, table_stride, ip, ip, nullptr, scale, fake, strides[7],
        strides[8], nullptr, nullptr, fake, bytes, nullptr);
  }
};

struct Verify {
  int dtype = SV_F32, mode = SV_DRAFT_IID;
  int64_t s[7] = {2, 5, 100, 4, 3, 100, 100};  // B, T, V, max_nodes, max_path, strides
  size_t bytes = size_t(1) << 40;
  int operator()() const {
    return specverify_tree_verify(fake, fake, dtype, mode, ip, ip, ip, s[0], s[1], s[2], s[3], s[4],
                                  s[5], s[6], dp, dp, ip, ip, nullptr, ip, nullptr, fake, bytes,
                                  nullptr);
  }
};

struct Commit {
  int dtype = SV_BF16;
  int64_t s[7] = {2, 2, 5, 2, 64, 4, 3};  // layers, B, T, H, D, max_nodes, max_path
  int64_t strides[7] = {640, 128, 64, 18432, 2048, 128, 64};  // nodes, cache
  int64_t num_pages = 9, page_size = 16;
  int operator()() const {
    return specverify_tree_commit(fake, fake, fake, fake, dtype, s[0], s[1], s[2], s[3], s[4], s[5],
                                  s[6], strides[0], strides[1], strides[2], strides[3], strides[4],
                                  strides[5], strides[6], num_pages, page_size, ip, ip, ip, lp, ip,
                                  ip, nullptr, nullptr);
  }
};

int main() {
  const int64_t ends[] = {kMost, kMost - 7, kMost / 2 + 1, kMost / 4 + 1, kLeast, -1};
  for (int64_t x : ends) {
    for (int i = 0; i < 9; ++i) {
      Plan p;
      p.s[i] = x;
      expect("plan size", i, p(), SV_EINVAL);
    }
    for (int i = 0; i < 6; ++i) {
      Attention a;
      a.s[i] = x;
      expect("attention size", i, a(), SV_EINVAL);
      expect("attention workspace", i,
             (long long)specverify_tree_attention_workspace_size(a.s[0], a.s[1], a.s[2], a.s[3],
                                                                 a.s[4], a.s[5]),
             0);
    }
    // strides, where all else is right: refused whatever their low bits
    for (int i = 0; i < 9; ++i) {
      Attention a;
      a.strides[i] = x;
      expect("attention stride", i, a(), SV_EINVAL);
    }
    for (int i = 0; i < 4; ++i) {
      Attention a;
      (i == 0 ? a.num_pages : i == 1 ? a.page_size : i == 2 ? a.max_pages : a.table_stride) = x;
      expect("attention cache", i, a(), SV_EINVAL);
    }
    for (int i = 0; i < 7; ++i)
      for (int dtype : {SV_F32, SV_BF16}) {
        Verify v;
        v.s[i] = x;
        v.dtype = dtype;
        expect(i < 5 ? "verify size" : "verify stride", i, v(), SV_EINVAL);
      }
    for (int i = 0; i < 7; ++i) {
      Commit c;
      c.s[i] = x;
      expect("commit size", i, c(), SV_EINVAL);
    }
    for (int i = 0; i < 7; ++i)
      for (int dtype : {SV_F32, SV_BF16, SV_F16}) {
        Commit c;
        c.dtype = dtype;
        c.strides[i] = x;
        expect("commit stride", i, c(), SV_EINVAL);
      }
    for (int i = 0; i < 2; ++i) {
      Commit c;
      (i == 0 ? c.num_pages : c.page_size) = x;
      expect("commit cache", i, c(), SV_EINVAL);
    }
    expect("verify workspace", 0, (long long)specverify_tree_verify_workspace_size(x, 100, 4), 0);
    expect("verify workspace", 1, (long long)specverify_tree_verify_workspace_size(2, x, 4), 0);
    expect("verify workspace", 2, (long long)specverify_tree_verify_workspace_size(2, 100, x), 0);
  }
  for (float scale : {0.0f, -1.0f, INFINITY, NAN, 3e38f}) {
    Attention a;
    a.scale = scale;
    expect("attention scale", 0, a(), SV_EINVAL);
  }
  // what is allowed reaches the workspace's check
  Attention a;
  a.bytes = 0;
  expect("attention workspace of nothing", 0, a(), SV_EWORKSPACE);
  Verify v;
  v.bytes = 0;
  expect("verify workspace of nothing", 0, v(), SV_EWORKSPACE);
  // the largest sizes of the library
  const int64_t k31 = int64_t(1) << 31;
  expect("attention largest", 0, specverify_tree_attention_workspace_size(1 << 24, k31 - 1, 1, 1, 256, 128) > 0, 1);
  expect("attention largest", 1, specverify_tree_attention_workspace_size(1, 1, 1 << 24, 1 << 24, 8, 128) > 0, 1);
  for (int64_t B : {int64_t(1), int64_t(256), int64_t(257), k31 - 1})
    expect("verify largest", B, specverify_tree_verify_workspace_size(B, SV_MAX_TREE_VOCAB, 128) > 0, 1);
  (void)fp;
  std::printf("failed %d\n", failed);
  return failed > 100 ? 100 : failed;
}
