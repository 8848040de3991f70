// Host-only driver of the key/value cache's and the epilogue's entry points for
// sanitizer builds: arguments that validation rejects or that leave nothing to do
// (so no HIP call is made), limits of every integer type among them, and the
// attention's workspace sizes over a sweep (its plan's arithmetic).  Built with
// AddressSanitizer and UndefinedBehaviorSanitizer on the host side by
// tests/test_host_sanitizers_kv.py; prints "host cache ABI check ok" at the end.
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
  const awq_config c64{4, 64, 1}, c128{4, 128, 1}, sym{4, 64, 0};
  const int32_t top = std::numeric_limits<int32_t>::max(), low = std::numeric_limits<int32_t>::min();
  const int64_t top64 = std::numeric_limits<int64_t>::max(), low64 = std::numeric_limits<int64_t>::min();
  const awq_kv_cache good{at<uint32_t>(0x10000), at<uint16_t>(0x200000), at<uint8_t>(0x300000), 8, 16, 2, 64};
  void *A = at<void>(0x1000000), *B = at<void>(0x2000000), *O = at<void>(0x3000000);
  int32_t *i = at<int32_t>(0x4000000), *j = at<int32_t>(0x5000000);

  // caches that no entry point takes
  awq_kv_cache c = good;
  auto all_refuse = [&](const awq_kv_cache *p, awq_config cfg) {
    EXPECT(awq_kv_append(A, B, 0, 3, 128, 128, p, cfg, i, nullptr, nullptr) != AWQ_OK);
    EXPECT(awq_kv_gather(p, cfg, i, 3, A, B, 0, nullptr) != AWQ_OK);
    EXPECT(awq_kv_attention(A, 0, 3, 256, 4, p, cfg, i, 4, j, nullptr, 3, 1, 64, 0.1f, 1, 0, O, nullptr, nullptr, 0,
                            nullptr) != AWQ_OK);
    EXPECT(awq_kv_attention_workspace_size(3, 3, 4, p, cfg, 1, 64, 0) == 0);
  };
  all_refuse(nullptr, c64);
  all_refuse(&good, c128);
  all_refuse(&good, awq_config{8, 64, 1});
  all_refuse(&good, awq_config{4, 64, 7});
  for (int32_t v : {low, -1, 0, 15, 48, 2048, top}) { c = good; c.page_size = v; all_refuse(&c, c64); }
  for (int32_t v : {low, -1, 0, 1025, top}) { c = good; c.num_kv_heads = v; all_refuse(&c, c64); }
  for (int32_t v : {low, -64, 0, 96, 256, top}) { c = good; c.head_dim = v; all_refuse(&c, c64); }
  for (int64_t v : {low64, (int64_t)-1, (int64_t)0, (int64_t)1 << 32, top64}) { c = good; c.num_pages = v; all_refuse(&c, c64); }

  // append and gather
  for (int64_t n : {low64, (int64_t)-1, ((int64_t)1 << 27) + 1, top64}) {
    EXPECT(awq_kv_append(A, B, 0, n, 128, 128, &good, c64, i, nullptr, nullptr) == AWQ_ERR_INVALID_ARG);
    EXPECT(awq_kv_gather(&good, c64, i, n, A, B, 0, nullptr) == AWQ_ERR_INVALID_ARG);
  }
  for (int64_t s : {low64, (int64_t)-8, (int64_t)0, (int64_t)127, (int64_t)132, top64})
    EXPECT(awq_kv_append(A, B, 0, 3, s, 128, &good, c64, i, nullptr, nullptr) == AWQ_ERR_INVALID_ARG);
  EXPECT(awq_kv_append(A, B, 2, 3, 128, 128, &good, c64, i, nullptr, nullptr) == AWQ_ERR_INVALID_ARG);
  EXPECT(awq_kv_append(A, good.codes, 0, 3, 128, 128, &good, c64, i, nullptr, nullptr) == AWQ_ERR_INVALID_ARG);
  EXPECT(awq_kv_append(A, B, 0, 1 << 27, top64 & ~(int64_t)7, 128, &good, c64, i, nullptr, nullptr) == AWQ_ERR_INVALID_ARG);
  EXPECT(awq_kv_append(nullptr, nullptr, 0, 0, 128, 128, &good, sym, nullptr, nullptr, nullptr) == AWQ_OK);
  EXPECT(awq_kv_gather(&good, c64, i, 3, A, A, 0, nullptr) == AWQ_ERR_INVALID_ARG);
  EXPECT(awq_kv_gather(&good, c64, i, 3, A, B, 3, nullptr) == AWQ_ERR_INVALID_ARG);
  EXPECT(awq_kv_gather(&good, c64, nullptr, 0, nullptr, nullptr, 0, nullptr) == AWQ_OK);

  // assign
  auto assign = [&](int32_t n, int32_t page, int32_t blocks, int32_t free, int64_t slots, int32_t *out) {
    return awq_kv_assign(i, at<int32_t>(0x4100000), n, page, at<int32_t>(0x4200000), blocks, at<int32_t>(0x4300000), free,
                         at<int32_t>(0x4400000), at<int32_t>(0x4500000), at<int32_t>(0x4600000), slots, out, nullptr);
  };
  for (int32_t v : {low, -1, 0, 3, 2048, top}) EXPECT(assign(3, v, 4, 5, 7, j) == AWQ_ERR_UNSUPPORTED);
  for (int32_t v : {low, -1}) {
    EXPECT(assign(v, 16, 4, 5, 7, j) == AWQ_ERR_INVALID_ARG);
    EXPECT(assign(3, 16, v, 5, 7, j) == AWQ_ERR_INVALID_ARG);
    EXPECT(assign(3, 16, 4, v, 7, j) == AWQ_ERR_INVALID_ARG);
    EXPECT(assign(3, 16, 4, 5, v, j) == AWQ_ERR_INVALID_ARG);
  }
  EXPECT(assign(3, 16, top, 5, 7, j) == AWQ_ERR_UNSUPPORTED);
  EXPECT(assign(3, 16, 4, 5, top64, j) == AWQ_ERR_INVALID_ARG);
  EXPECT(assign(3, 16, 4, 5, 7, i) == AWQ_ERR_INVALID_ARG);
  EXPECT(assign(top, 16, (1 << 27) - 1, top, top, j) == AWQ_ERR_INVALID_ARG);    // (spans of 2^58 bytes overlap)
  EXPECT(assign(3, 16, 4, 5, 7, nullptr) == AWQ_ERR_INVALID_ARG);

  // attention
  auto attend = [&](int64_t T, int32_t heads, int64_t stride, int32_t blocks, int32_t n, int32_t most, int64_t longest,
                    float scale, int32_t causal, int32_t window, void *ws, size_t bytes, const int32_t *start = nullptr) {
    return awq_kv_attention(A, 1, T, stride, heads, &good, c64, i, blocks, j, start, n, most, longest, scale, causal,
                            window, O, nullptr, ws, bytes, nullptr);
  };
  for (int64_t v : {low64, (int64_t)-1, (int64_t)1 << 31, top64})
    EXPECT(attend(v, 4, 256, 4, 3, 1, 64, 0.1f, 1, 0, nullptr, 0) == AWQ_ERR_INVALID_ARG);
  for (int32_t v : {low, -2, 0, 3, 1026, top}) EXPECT(attend(3, v, top64 & ~(int64_t)7, 4, 3, 1, 64, 0.1f, 1, 0, nullptr, 0) == AWQ_ERR_INVALID_ARG);
  for (int64_t v : {low64, (int64_t)-8, (int64_t)255, (int64_t)260}) EXPECT(attend(3, 4, v, 4, 3, 1, 64, 0.1f, 1, 0, nullptr, 0) == AWQ_ERR_INVALID_ARG);
  for (int32_t v : {low, -1, 1 << 27, top}) EXPECT(attend(3, 4, 256, v, 3, 1, 64, 0.1f, 1, 0, nullptr, 0) == AWQ_ERR_INVALID_ARG);
  for (int32_t v : {low, -1, 65536, top}) EXPECT(attend(3, 4, 256, 4, v, 1, 64, 0.1f, 1, 0, nullptr, 0) != AWQ_OK);
  for (int32_t v : {low, -1, 2, 1 << 30, top}) EXPECT(attend(3, 4, 256, 4, 3, v, 64, 0.1f, 1, 0, nullptr, 0) != AWQ_OK);
  for (int64_t v : {low64, (int64_t)-1}) EXPECT(attend(3, 4, 256, 4, 3, 1, v, 0.1f, 1, 0, nullptr, 0) == AWQ_ERR_INVALID_ARG);
  for (float v : {std::numeric_limits<float>::infinity(), -std::numeric_limits<float>::infinity(), std::numeric_limits<float>::quiet_NaN()})
    EXPECT(attend(3, 4, 256, 4, 3, 1, 64, v, 1, 0, nullptr, 0) == AWQ_ERR_INVALID_ARG);
  EXPECT(attend(3, 4, 256, 4, 3, 1, 64, 0.1f, 2, 0, nullptr, 0) == AWQ_ERR_INVALID_ARG);
  EXPECT(attend(3, 4, 256, 4, 3, 1, 64, 0.1f, 0, 5, nullptr, 0) == AWQ_ERR_INVALID_ARG);
  EXPECT(attend(3, 4, 256, 4, 3, 1, 64, 0.1f, 1, low, nullptr, 0) == AWQ_ERR_INVALID_ARG);
  EXPECT(attend(1, 4, 256, 4, 1, 1, top64, 0.1f, 1, 0, nullptr, 0) == AWQ_ERR_WORKSPACE);
  EXPECT(attend(1, 4, 256, 4, 1, 1, top64, 0.1f, 1, 0, A, 1) == AWQ_ERR_WORKSPACE);
  EXPECT(attend(1, 4, 256, 4, 1, 1, top64, 0.1f, 1, 0, A, 1 << 30) == AWQ_ERR_INVALID_ARG);
  EXPECT(attend(0, 4, 256, 4, 0, 1, 64, 0.1f, 1, 0, nullptr, 0) == AWQ_OK);

  // the plan: sizes within what the layout holds, whole and monotone in nothing but its own terms
  size_t total = 0;
  for (int64_t T : {(int64_t)1, (int64_t)3, (int64_t)48, (int64_t)517, (int64_t)65535, (int64_t)top})
    for (int32_t n : {1, 3, 48, 65535})
      for (int32_t heads : {2, 4, 16, 1024})
        for (int32_t most : {1, 4, 33, 515, 1 << 20})
          for (int64_t longest : {(int64_t)0, (int64_t)1, (int64_t)700, (int64_t)5000, (int64_t)1 << 30, top64})
            for (int32_t window : {0, 1, 1000, top}) {
              if ((int64_t)most * (heads / 2) > 1 << 30) continue;
              const size_t b = awq_kv_attention_workspace_size(T, n, heads, &good, c64, most, longest, window);
              EXPECT(b % ((size_t)T * heads * (64 * 4 + 8 + 4)) == 0);
              EXPECT(b <= (size_t)64 * T * heads * (64 * 4 + 8 + 4));
              total += b;
            }
  std::printf("sizes checksum %zu\n", total);

  // the layer's epilogue
  const uint32_t *qw = at<uint32_t>(0x6000000);
  const uint16_t *sc = at<uint16_t>(0x7000000);
  const uint8_t *zr = at<uint8_t>(0x8000000);
  auto linear = [&](const awq_epilogue *e, int64_t M, int64_t N, int64_t K) {
    return awq_linear_epilogue(A, 0, qw, sc, zr, M, N, K, c128, e, O, 0, 0, nullptr, 0, nullptr);
  };
  const awq_epilogue none{nullptr, nullptr, 0};
  EXPECT(linear(nullptr, 3, 64, 256) == AWQ_ERR_INVALID_ARG);
  for (int32_t a : {low, -1, 5, top}) {
    const awq_epilogue e{nullptr, nullptr, a};
    EXPECT(linear(&e, 3, 64, 256) == AWQ_ERR_INVALID_ARG);
  }
  const awq_epilogue over{at<void>(0x3000000 + 2), nullptr, 0}, across{nullptr, at<void>(0x3000000 - 2), 0},
      odd{at<void>(0x9000001), nullptr, 0}, far{at<void>(0x9000000), at<void>(0x9100000), 3};
  EXPECT(linear(&over, 3, 64, 256) == AWQ_ERR_INVALID_ARG);
  EXPECT(linear(&across, 3, 64, 256) == AWQ_ERR_INVALID_ARG);
  EXPECT(linear(&odd, 3, 64, 256) == AWQ_ERR_INVALID_ARG);
  for (int64_t v : {low64, (int64_t)-1, top64}) {
    EXPECT(linear(&far, v, 64, 256) != AWQ_OK);
    EXPECT(linear(&far, 3, v, 256) != AWQ_OK);
    EXPECT(linear(&far, 3, 64, v) != AWQ_OK);
  }
  EXPECT(linear(&none, 0, 64, 256) == AWQ_OK);
  if (failures) return 1;
  std::printf("host cache ABI check ok\n");
  return 0;
}
