// Argument checks that the entry points around the 4-bit key/value cache share
// (api_kv.cpp, api_kv_pages.cpp, api_rope.cpp).
#pragma once

#include "api_common.h"
#include "awq_internal.h"

namespace awq {

constexpr int64_t kMaxGrid = 65535;          // HIP's limit on grid y and z
// Tokens of an append or gather: 16 or more to a workgroup of 256, and a grid
// holds less than 2^32 threads.
constexpr int64_t kMaxTokens = (int64_t)1 << 27;
// Tokens of a request that attention reads: key numbers stay within 32 bits, a
// tile or two past the last key included.
constexpr int64_t kMaxContext = (int64_t)1 << 30;
// Elements from the first to the last token of a strided array, so that its bytes
// count in 64 bits.
constexpr int64_t kMaxExtent = (int64_t)1 << 60;
inline bool too_far(int64_t tokens, int64_t stride) { return tokens > 0 && stride > kMaxExtent / tokens; }

inline bool power_of_two(int64_t x) { return x > 0 && (x & (x - 1)) == 0; }

inline awq_status check_page(const char *who, int32_t page_size) {
  if (!power_of_two(page_size) || page_size < AWQ_KV_MIN_PAGE || page_size > AWQ_KV_MAX_PAGE)
    return fail(AWQ_ERR_UNSUPPORTED, "%s: page_size=%d: must be a power of two in [%d, %d]", who,
                page_size, AWQ_KV_MIN_PAGE, AWQ_KV_MAX_PAGE);
  return AWQ_OK;
}

inline awq_status check_cache(const char *who, const awq_kv_cache *c, awq_config cfg, bool need_ptrs) {
  if (!c) return fail(AWQ_ERR_INVALID_ARG, "%s: cache is NULL", who);
  if (cfg.w_bit != 4) return fail(AWQ_ERR_UNSUPPORTED, "%s: w_bit=%d: only 4 is supported", who, cfg.w_bit);
  if (cfg.zero_point != 0 && cfg.zero_point != 1)
    return fail(AWQ_ERR_INVALID_ARG, "%s: zero_point=%d: must be 1 (asymmetric) or 0 (symmetric)", who,
                cfg.zero_point);
  if (c->head_dim != 64 && c->head_dim != 128)
    return fail(AWQ_ERR_UNSUPPORTED, "%s: head_dim=%d: supported values are 64 and 128", who, c->head_dim);
  if (cfg.group_size != c->head_dim)
    return fail(AWQ_ERR_UNSUPPORTED, "%s: group_size=%d: a token's head is one group, so it must be head_dim=%d",
                who, cfg.group_size, c->head_dim);
  const awq_status st = check_page(who, c->page_size);
  if (st != AWQ_OK) return st;
  if (c->num_kv_heads < 1 || c->num_kv_heads > AWQ_KV_MAX_HEADS)
    return fail(AWQ_ERR_INVALID_ARG, "%s: num_kv_heads=%d: must be in [1, %d]", who, c->num_kv_heads,
                AWQ_KV_MAX_HEADS);
  if (c->num_pages < 1) return fail(AWQ_ERR_INVALID_ARG, "%s: num_pages=%lld: must be positive", who, (long long)c->num_pages);
  if (c->num_pages > ((int64_t)1 << 31) / c->page_size)
    return fail(AWQ_ERR_UNSUPPORTED, "%s: %lld pages of %d tokens exceed 2^31 slots", who,
                (long long)c->num_pages, c->page_size);
  if (!need_ptrs) return AWQ_OK;
  if (!c->codes || !c->scales || (cfg.zero_point && !c->zeros))
    return fail(AWQ_ERR_INVALID_ARG, "%s: a cache array is NULL", who);
  if (!aligned(c->codes, 16) || !aligned(c->scales, 16) || (cfg.zero_point && !aligned(c->zeros, 16)))
    return fail(AWQ_ERR_INVALID_ARG, "%s: the cache arrays must be 16-byte aligned", who);
  return AWQ_OK;
}

inline KvCache kv_cache(const awq_kv_cache *c, awq_config cfg) {
  return KvCache{c->codes, c->scales, cfg.zero_point ? c->zeros : nullptr, c->num_pages,
                 c->page_size, c->num_kv_heads, c->head_dim};
}

// Bytes that a call reads or writes.
struct Span {
  const void *p;
  size_t n;
};
template <size_t A, size_t B>
bool all_apart(const Span (&a)[A], const Span (&b)[B]) {
  for (const Span &x : a)
    for (const Span &y : b)
      if (!apart(x.p, x.n, y.p, y.n)) return false;
  return true;
}
// `tokens` rows of `width` elements of `size` bytes, `stride` elements apart.
inline size_t strided_bytes(int64_t tokens, int64_t stride, int64_t width, size_t size) {
  return ((size_t)(tokens - 1) * (size_t)stride + (size_t)width) * size;
}
// Rows of two strided arrays share no element: their extents do not, or they are
// slices of the same rows (one stride) that lie beside each other in it.
inline bool rows_apart(const Span &a, int64_t a_stride, int64_t a_width, const Span &b, int64_t b_stride,
                       int64_t b_width, size_t size) {
  if (apart(a.p, a.n, b.p, b.n)) return true;
  if (a_stride != b_stride) return false;
  const int64_t row = a_stride * (int64_t)size;
  const int64_t from = (int64_t)(reinterpret_cast<uintptr_t>(b.p) - reinterpret_cast<uintptr_t>(a.p)) % row;
  const int64_t at = from < 0 ? from + row : from;
  return at >= a_width * (int64_t)size && at + b_width * (int64_t)size <= row;
}
struct CacheSpans {
  Span codes, scales, zeros;
};
inline CacheSpans cache_spans(const KvCache &c) {
  const size_t n = (size_t)c.pages * c.page_size * c.heads;      // (less than 2^41)
  return CacheSpans{{c.codes, n * c.head_dim}, {c.scales, n * 4}, {c.zeros, c.zeros ? n * 2 : 0}};
}

// A call that writes the cache reads and writes nothing else of it: its arrays lie apart.
inline bool arrays_apart(const CacheSpans &c) {
  return apart(c.codes.p, c.codes.n, c.scales.p, c.scales.n) && apart(c.codes.p, c.codes.n, c.zeros.p, c.zeros.n) &&
         apart(c.scales.p, c.scales.n, c.zeros.p, c.zeros.n);
}

// The arguments of a call that quantizes keys and values into the cache.
inline awq_status check_append(const char *who, const void *K, const void *V, int32_t x_dtype, int64_t num_tokens,
                               int64_t k_stride, int64_t v_stride, const awq_kv_cache *cache, awq_config cfg,
                               const int32_t *slots, const int32_t *nonfinite_count) {
  const awq_status st = check_cache(who, cache, cfg, num_tokens > 0);
  if (st != AWQ_OK) return st;
  if (x_dtype != AWQ_F16 && x_dtype != AWQ_BF16)
    return fail(AWQ_ERR_INVALID_ARG, "%s: x_dtype=%d: must be AWQ_F16 or AWQ_BF16", who, x_dtype);
  if (num_tokens < 0) return fail(AWQ_ERR_INVALID_ARG, "%s: num_tokens=%lld is negative", who, (long long)num_tokens);
  if (num_tokens > kMaxTokens) return fail(AWQ_ERR_INVALID_ARG, "%s: more than 2^27 tokens", who);
  const int64_t width = (int64_t)cache->num_kv_heads * cache->head_dim;
  if (k_stride < width || v_stride < width || k_stride % 8 != 0 || v_stride % 8 != 0)
    return fail(AWQ_ERR_INVALID_ARG,
                "%s: token strides %lld and %lld must be multiples of 8 of at least num_kv_heads * head_dim", who,
                (long long)k_stride, (long long)v_stride);
  if (too_far(num_tokens, k_stride) || too_far(num_tokens, v_stride))
    return fail(AWQ_ERR_INVALID_ARG, "%s: token strides reach beyond 2^60 elements", who);
  if (num_tokens == 0) return AWQ_OK;
  if (!K || !V || !slots) return fail(AWQ_ERR_INVALID_ARG, "%s: a required pointer is NULL", who);
  if (!aligned(K, 16) || !aligned(V, 16))
    return fail(AWQ_ERR_INVALID_ARG, "%s: K and V must be 16-byte aligned", who);
  if (!aligned(slots, 4) || (nonfinite_count && !aligned(nonfinite_count, 4)))
    return fail(AWQ_ERR_INVALID_ARG, "%s: slots and nonfinite_count must be 4-byte aligned", who);
  const KvCache kc = kv_cache(cache, cfg);
  const CacheSpans cs = cache_spans(kc);
  const Span in[] = {{K, strided_bytes(num_tokens, k_stride, width, 2)}, {V, strided_bytes(num_tokens, v_stride, width, 2)},
                     {slots, (size_t)num_tokens * 4}},
             arrays[] = {cs.codes, cs.scales, cs.zeros}, count[] = {{nonfinite_count, nonfinite_count ? 4u : 0u}};
  if (!all_apart(in, arrays) || !all_apart(in, count) || !all_apart(count, arrays))
    return fail(AWQ_ERR_INVALID_ARG, "%s: K, V, slots, nonfinite_count and the cache may not overlap", who);
  if (!arrays_apart(cs))
    return fail(AWQ_ERR_INVALID_ARG, "%s: the cache arrays overlap each other", who);
  return AWQ_OK;
}

}  // namespace awq
