// Host-only driver of rotary positions, the page operations and awq_kv_attention_ex for
// sanitizer builds: arguments that validation rejects or that leave nothing to do (so no HIP
// call is made), limits of every integer type among them, and the workspace sizes and
// frequencies over sweeps (their arithmetic).  Built with AddressSanitizer and
// UndefinedBehaviorSanitizer on the host side by tests/test_host_sanitizers_kv_more.py; prints
// "host cache extensions ABI check ok" at the end.
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <limits>

#include "awq355.h"

static int failures = 0;
#define EXPECT(cond)                                                     \
  do {                                                                   \
    if (!(cond)) {                                                       \
      std::printf("FAILED %s:%d: %s\n", __FILE__, __LINE__, #cond);     \
      ++failures;                                                        \
    }                                                                    \
  } while (0)

template <class T>
static T *at(uintptr_t a) { return reinterpret_cast<T *>(a); }   // never dereferenced

int main() {
  const awq_config c64{4, 64, 1}, sym{4, 64, 0};
  const int32_t top = std::numeric_limits<int32_t>::max(), low = std::numeric_limits<int32_t>::min();
  const int64_t top64 = std::numeric_limits<int64_t>::max(), low64 = std::numeric_limits<int64_t>::min();
  const awq_kv_cache good{at<uint32_t>(0x10000), at<uint16_t>(0x200000), at<uint8_t>(0x300000), 8, 16, 2, 64};
  void *A = at<void>(0x1000000), *B = at<void>(0x2000000), *O = at<void>(0x3000000), *P = at<void>(0x3800000);
  int32_t *i[10];
  for (int k = 0; k < 10; ++k) i[k] = at<int32_t>(0x4000000 + 0x100000 * k);
  void *W = at<void>(0x8000000);

  // ---- rotary positions
  const awq_rope_args fine{i[0], at<double>(0x6000000), 1.0, 64, 0, 0};
  auto rope = [&](const awq_rope_args *r, int32_t heads, int64_t qs, int64_t qo, int32_t kv, int64_t ks, int64_t n, int32_t D) {
    return awq_rope(A, B, heads, qs, qo, O, P, kv, ks, ks, 0, n, D, r, nullptr);
  };
  auto append = [&](const awq_rope_args *r, int32_t heads, int64_t qs, int64_t ks, int64_t n, const awq_kv_cache *c, awq_config cfg) {
    return awq_kv_append_rope(A, B, heads, qs, qs, O, P, 0, n, ks, ks, c, cfg, i[1], r, nullptr, nullptr);
  };
  for (int64_t n : {low64, (int64_t)-1, ((int64_t)1 << 27) + 1, top64}) {
    EXPECT(rope(&fine, 2, 128, 128, 2, 128, n, 64) != AWQ_OK);
    EXPECT(append(&fine, 2, 128, 128, n, &good, c64) != AWQ_OK);
  }
  for (int64_t s : {low64, (int64_t)-8, (int64_t)0, (int64_t)120, (int64_t)132, top64, top64 & ~(int64_t)7, (int64_t)1 << 59}) {
    EXPECT(rope(&fine, 2, s, 128, 2, 128, 5, 64) != AWQ_OK);
    EXPECT(rope(&fine, 2, 128, s, 2, 128, 5, 64) != AWQ_OK);
    EXPECT(rope(&fine, 2, 128, 128, 2, s, 5, 64) != AWQ_OK);
    EXPECT(append(&fine, 2, s, 128, 5, &good, c64) != AWQ_OK);
    EXPECT(append(&fine, 2, 128, s, 5, &good, c64) != AWQ_OK);
  }
  for (int32_t v : {low, -1, 1025, top}) {
    EXPECT(rope(&fine, v, (int64_t)1 << 40, (int64_t)1 << 40, 2, 128, 5, 64) != AWQ_OK);
    EXPECT(append(&fine, v, (int64_t)1 << 40, 128, 5, &good, c64) != AWQ_OK);
  }
  for (int32_t v : {low, -16, 0, 8, 24, 72, 528, top}) EXPECT(rope(&fine, 2, 2048, 2048, 2, 2048, 5, v) != AWQ_OK);
  for (int32_t v : {low, -16, 0, 8, 24, 80, top}) {
    awq_rope_args r = fine;
    r.rotary_dim = v;
    EXPECT(rope(&r, 2, 128, 128, 2, 128, 5, 64) != AWQ_OK);
    EXPECT(append(&r, 2, 128, 128, 5, &good, c64) != AWQ_OK);
  }
  EXPECT(rope(&fine, 0, low64, top64, 0, low64, 5, 64) == AWQ_OK);
  EXPECT(rope(&fine, 2, 128, 128, 2, 128, 0, 64) == AWQ_OK);
  EXPECT(append(&fine, 2, 128, 128, 0, &good, c64) == AWQ_OK);
  EXPECT(append(&fine, 2, 128, 128, 5, nullptr, c64) != AWQ_OK);

  double inv[AWQ_ROPE_MAX_DIM / 2], factor;
  for (int32_t R : {low, -16, 0, 8, 20, 528, top}) EXPECT(awq_rope_frequencies(R, 1e4, nullptr, inv, &factor) != AWQ_OK);
  for (int32_t R = 16; R <= AWQ_ROPE_MAX_DIM; R += 16)
    for (int32_t kind = low; kind < 7; kind = kind == low ? -1 : kind + 1)
      for (double s : {-1.0, 0.0, 1e-300, 0.5, 1.0, 32.0, 1e300, (double)INFINITY, (double)NAN})
        for (double L : {0.0, 1.0, 4096.0, 1e300}) {
          const awq_rope_scaling sc{kind, s, L, 0, 0};
          if (awq_rope_frequencies(R, 10000.0, &sc, inv, &factor) != AWQ_OK) continue;
          EXPECT(kind >= 0 && kind <= 4);
          for (int j = 0; j < R / 2; ++j) EXPECT(inv[j] >= 0.0);
          EXPECT(factor >= 1.0);
        }

  // ---- pages
  for (int64_t n : {low64, (int64_t)-1, ((int64_t)1 << 27) + 1, top64})
    EXPECT(awq_kv_copy_pages(&good, c64, i[0], i[1], n, nullptr) == AWQ_ERR_INVALID_ARG);
  EXPECT(awq_kv_copy_pages(&good, c64, i[0], i[1], 0, nullptr) == AWQ_OK);
  for (int32_t v : {low, -1, top}) {
    EXPECT(awq_kv_fork(&good, c64, i[0], i[1], i[2], v, i[3], 4, 4, i[4], i[5], 3, nullptr, i[6], nullptr) != AWQ_OK);
    EXPECT(awq_kv_fork(&good, c64, i[0], i[1], i[2], 2, i[3], v, 4, i[4], i[5], 3, nullptr, i[6], nullptr) != AWQ_OK);
    EXPECT(awq_kv_fork(&good, c64, i[0], i[1], i[2], 2, i[3], 4, v, i[4], i[5], 3, nullptr, i[6], nullptr) != AWQ_OK);
    EXPECT(awq_kv_release(i[0], v, 4, 16, i[1], nullptr, nullptr, i[2], 8, i[3], 3, nullptr, i[4], 8, i[5], nullptr, 0, nullptr) != AWQ_OK);
    EXPECT(awq_kv_release(i[0], 4, v, 16, i[1], nullptr, nullptr, i[2], 8, i[3], 3, nullptr, i[4], 8, i[5], nullptr, 0, nullptr) != AWQ_OK);
    EXPECT(awq_kv_release(i[0], 4, 4, v, i[1], nullptr, nullptr, i[2], 8, i[3], 3, nullptr, i[4], 8, i[5], nullptr, 0, nullptr) != AWQ_OK);
    EXPECT(awq_kv_compact(&good, c64, i[0], v, 4, i[1], i[2], i[3], i[4], W, 1 << 20, nullptr) != AWQ_OK);
    EXPECT(awq_kv_compact(&good, c64, i[0], 4, v, i[1], i[2], i[3], i[4], W, 1 << 20, nullptr) != AWQ_OK);
  }
  EXPECT(awq_kv_fork(&good, c64, i[0], i[1], i[2], 2, i[3], 4, 4, i[4], i[5], low, nullptr, i[6], nullptr) != AWQ_OK);
  EXPECT(awq_kv_release(i[0], 4, 4, 16, i[1], nullptr, nullptr, i[2], 8, i[3], top, nullptr, i[4], 8, i[5], nullptr, 0, nullptr) == AWQ_ERR_WORKSPACE);
  EXPECT(awq_kv_release(i[0], 4, 4, 16, i[1], nullptr, nullptr, i[2], 8, i[3], 3, nullptr, i[4], top, i[5], nullptr, 0, nullptr) == AWQ_ERR_INVALID_ARG);
  for (int64_t n : {low64, (int64_t)-1, (int64_t)0, ((int64_t)1 << 27) + 1, top64}) {
    EXPECT(awq_kv_release(i[0], 4, 4, 16, i[1], nullptr, nullptr, i[2], n, i[3], 3, nullptr, i[4], 8, i[5], nullptr, 0, nullptr) != AWQ_OK);
    EXPECT(awq_kv_release_workspace_size(n, 5) == 0 && awq_kv_compact_workspace_size(n, 16) == 0);
  }
  for (int64_t n = 1; n <= (int64_t)1 << 27; n *= 3) {
    EXPECT(awq_kv_release_workspace_size(n, top) > 0 && awq_kv_release_workspace_size(n, low) == 0);
    EXPECT(awq_kv_compact_workspace_size(n, 16) >= (size_t)n * 13);
  }

  // ---- attention over some keys
  auto size = [&](int64_t T, int32_t seqs, int32_t heads, int32_t mq, int64_t mk, awq_kv_attention_options o) {
    return awq_kv_attention_ex_workspace_size(T, seqs, heads, &good, c64, mq, mk, &o);
  };
  auto attend = [&](int64_t T, int32_t seqs, int32_t mq, int64_t mk, awq_kv_attention_options o, size_t ws) {
    return awq_kv_attention_ex(A, 0, T, 256, 4, &good, c64, i[0], 4, i[1], i[2], seqs, mq, mk, 0.1f, &o, O, nullptr, W, ws, nullptr);
  };
  for (int32_t v : {low, -1, ((int32_t)1 << 30) + 1, top}) {
    EXPECT(attend(3, 3, 1, 64, {1, 4, v, 0, nullptr, 0}, 1 << 20) != AWQ_OK);
    EXPECT(attend(3, 3, 1, 64, {1, 0, 0, v, i[3], 8}, 1 << 20) != AWQ_OK);
    EXPECT(attend(3, 3, 1, 64, {1, 0, 0, v, i[3], top}, 1 << 20) != AWQ_OK);
  }
  for (int32_t v : {low, -1, 0, 1}) EXPECT(attend(3, 3, 1, 64, {1, 0, 0, 20, i[3], v}, 1 << 20) != AWQ_OK);
  EXPECT(attend(3, 3, 1, 64, {1, low, 0, 0, nullptr, 0}, 1 << 20) != AWQ_OK);
  EXPECT(attend(3, 3, 1, 64, {1, top, 1, 20, i[3], 8}, 1 << 20) != AWQ_OK);
  EXPECT(attend(3, 3, 1, 64, {1, 0, 0, 20, i[3], 8}, 0) == AWQ_ERR_WORKSPACE);
  EXPECT(attend(0, 0, 1, 64, {1, 0, 0, 20, i[3], 8}, 0) == AWQ_OK);
  for (int64_t T : {(int64_t)1, (int64_t)7, (int64_t)100, (int64_t)70000, (int64_t)1 << 29, top64})
    for (int32_t seqs : {1, 3, 65535, 65536, top})
      for (int32_t mq : {0, 1, 9, 4000, top})
        for (int64_t mk : {(int64_t)0, (int64_t)1, (int64_t)5000, (int64_t)1 << 31, top64})
          for (int32_t prefix : {0, 1, 16, 17, 5000, (int32_t)1 << 30})
            for (int32_t window : {0, 1, 1000, top}) {
              const size_t n = size(T, seqs, 4, mq, mk, {1, window, prefix ? 0 : 1 << 30, prefix, i[3], (int32_t)1 << 26});
              EXPECT(n % 4 == 0);
              if (prefix && !window && T <= 70000 && seqs <= 65535 && mq == 1 && mq * 2 <= 1 << 30) EXPECT(n > 0);
              if (prefix && window) EXPECT(n == 0);
            }
  EXPECT(awq_kv_attention_ex_workspace_size(3, 3, 4, &good, sym, 1, 64, nullptr) == 0);
  std::printf(failures ? "FAILED\n" : "host cache extensions ABI check ok\n");
  return failures ? 1 : 0;
}
