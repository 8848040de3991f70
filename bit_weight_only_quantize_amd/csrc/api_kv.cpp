// C ABI of the 4-bit paged key/value cache (awq_kv_*): argument validation and
// dispatch.  Every check runs before any HIP call.

#include <hip/hip_runtime.h>

#include <cmath>

#include "api_common.h"
#include "awq_internal.h"

using namespace awq;

namespace {

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
bool too_far(int64_t tokens, int64_t stride) { return tokens > 0 && stride > kMaxExtent / tokens; }

bool power_of_two(int64_t x) { return x > 0 && (x & (x - 1)) == 0; }

awq_status check_page(const char *who, int32_t page_size) {
  if (!power_of_two(page_size) || page_size < AWQ_KV_MIN_PAGE || page_size > AWQ_KV_MAX_PAGE)
    return fail(AWQ_ERR_UNSUPPORTED, "%s: page_size=%d: must be a power of two in [%d, %d]", who,
                page_size, AWQ_KV_MIN_PAGE, AWQ_KV_MAX_PAGE);
  return AWQ_OK;
}

awq_status check_cache(const char *who, const awq_kv_cache *c, awq_config cfg, bool need_ptrs) {
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

KvCache kv_cache(const awq_kv_cache *c, awq_config cfg) {
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
size_t strided_bytes(int64_t tokens, int64_t stride, int64_t width, size_t size) {
  return ((size_t)(tokens - 1) * (size_t)stride + (size_t)width) * size;
}
struct CacheSpans {
  Span codes, scales, zeros;
};
CacheSpans cache_spans(const KvCache &c) {
  const size_t n = (size_t)c.pages * c.page_size * c.heads;      // (less than 2^41)
  return CacheSpans{{c.codes, n * c.head_dim}, {c.scales, n * 4}, {c.zeros, c.zeros ? n * 2 : 0}};
}

// Sizes of an attention call that its workspace depends on.
awq_status check_attention_sizes(const char *who, int64_t num_tokens, int32_t num_seqs,
                                 int32_t num_heads, const awq_kv_cache *cache, awq_config cfg,
                                 int32_t max_query_len, int64_t max_seq_len, int32_t window,
                                 bool need_ptrs) {
  const awq_status st = check_cache(who, cache, cfg, need_ptrs);
  if (st != AWQ_OK) return st;
  if (num_tokens < 0 || num_seqs < 0)
    return fail(AWQ_ERR_INVALID_ARG, "%s: negative num_tokens or num_seqs", who);
  if (num_tokens > ((int64_t)1 << 31) - 1) return fail(AWQ_ERR_INVALID_ARG, "%s: too many tokens", who);
  if (num_seqs > kMaxGrid)
    return fail(AWQ_ERR_UNSUPPORTED, "%s: num_seqs=%d exceeds %lld", who, num_seqs, (long long)kMaxGrid);
  if (num_heads < 1 || num_heads % cache->num_kv_heads != 0)
    return fail(AWQ_ERR_INVALID_ARG, "%s: num_heads=%d is not a positive multiple of num_kv_heads=%d", who,
                num_heads, cache->num_kv_heads);
  if (num_heads > AWQ_KV_MAX_HEADS)
    return fail(AWQ_ERR_INVALID_ARG, "%s: num_heads=%d exceeds %d", who, num_heads, AWQ_KV_MAX_HEADS);
  if (max_query_len < 0 || max_seq_len < 0)
    return fail(AWQ_ERR_INVALID_ARG, "%s: negative max_query_len or max_seq_len", who);
  // rows of one key/value head and request are counted in 32 bits
  if ((int64_t)max_query_len * (num_heads / cache->num_kv_heads) > ((int64_t)1 << 30))
    return fail(AWQ_ERR_UNSUPPORTED, "%s: max_query_len=%d times the query heads per key/value head exceeds 2^30",
                who, max_query_len);
  if (window < 0) return fail(AWQ_ERR_INVALID_ARG, "%s: window=%d is negative", who, window);
  return AWQ_OK;
}

}  // namespace

extern "C" {

awq_status awq_kv_assign(const int32_t *old_lens, const int32_t *new_lens, int32_t num_seqs,
                         int32_t page_size, int32_t *block_table, int32_t max_blocks,
                         const int32_t *free_pages, int32_t num_free, int32_t *seq_lens,
                         int32_t *query_start, int32_t *slots, int64_t num_slots,
                         int32_t *pages_used, awq_stream_t stream) {
  const char *who = "awq_kv_assign";
  const awq_status st = check_page(who, page_size);
  if (st != AWQ_OK) return st;
  if (num_seqs < 0 || max_blocks < 0 || num_free < 0 || num_slots < 0)
    return fail(AWQ_ERR_INVALID_ARG, "%s: negative num_seqs, max_blocks, num_free or num_slots", who);
  if (num_slots > ((int64_t)1 << 31) - 1) return fail(AWQ_ERR_INVALID_ARG, "%s: too many slots", who);
  if ((int64_t)max_blocks * page_size > ((int64_t)1 << 31) - 1)
    return fail(AWQ_ERR_UNSUPPORTED, "%s: max_blocks=%d pages of %d tokens exceed 2^31 - 1", who, max_blocks,
                page_size);
  if (!query_start || !pages_used) return fail(AWQ_ERR_INVALID_ARG, "%s: a required pointer is NULL", who);
  if (num_seqs > 0 && (!old_lens || !new_lens || !seq_lens || (max_blocks > 0 && !block_table)))
    return fail(AWQ_ERR_INVALID_ARG, "%s: a required pointer is NULL", who);
  if ((num_free > 0 && !free_pages) || (num_slots > 0 && !slots))
    return fail(AWQ_ERR_INVALID_ARG, "%s: a required pointer is NULL", who);
  const size_t seqs = (size_t)num_seqs * 4;
  const struct { const void *p; size_t n; } in[] = {{old_lens, seqs}, {new_lens, seqs}, {free_pages, (size_t)num_free * 4}},
      out[] = {{block_table, seqs * (size_t)max_blocks}, {seq_lens, seqs}, {query_start, seqs + 4},
               {slots, (size_t)num_slots * 4}, {pages_used, 4}};
  for (const auto &x : in)
    if (x.n && !aligned(x.p, 4)) return fail(AWQ_ERR_INVALID_ARG, "%s: arrays must be 4-byte aligned", who);
  for (const auto &y : out) {
    if (y.n && !aligned(y.p, 4)) return fail(AWQ_ERR_INVALID_ARG, "%s: arrays must be 4-byte aligned", who);
    for (const auto &x : in)
      if (!apart(x.p, x.n, y.p, y.n))
        return fail(AWQ_ERR_INVALID_ARG, "%s: an output overlaps an input", who);
    for (const auto &z : out)
      if (&z != &y && !apart(z.p, z.n, y.p, y.n))
        return fail(AWQ_ERR_INVALID_ARG, "%s: two outputs overlap", who);
  }
  return hip_status(launch_kv_assign(old_lens, new_lens, num_seqs, page_size, block_table, max_blocks,
                                     free_pages, num_free, seq_lens, query_start, slots, num_slots,
                                     pages_used, as_stream(stream)),
                    who);
}

awq_status awq_kv_append(const void *K, const void *V, int32_t x_dtype, int64_t num_tokens,
                         int64_t k_stride, int64_t v_stride, const awq_kv_cache *cache,
                         awq_config cfg, const int32_t *slots, int32_t *nonfinite_count,
                         awq_stream_t stream) {
  const char *who = "awq_kv_append";
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
  if (num_tokens == 0) return ok();
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
  if (!apart(cs.codes.p, cs.codes.n, cs.scales.p, cs.scales.n) || !apart(cs.codes.p, cs.codes.n, cs.zeros.p, cs.zeros.n) ||
      !apart(cs.scales.p, cs.scales.n, cs.zeros.p, cs.zeros.n))
    return fail(AWQ_ERR_INVALID_ARG, "%s: the cache arrays overlap each other", who);
  return hip_status(launch_kv_append(reinterpret_cast<const uint16_t *>(K), reinterpret_cast<const uint16_t *>(V),
                                     x_dtype == AWQ_BF16 ? XType::BF16 : XType::F16, num_tokens, k_stride,
                                     v_stride, slots, kc, nonfinite_count,
                                     as_stream(stream)),
                    who);
}

awq_status awq_kv_gather(const awq_kv_cache *cache, awq_config cfg, const int32_t *slots,
                         int64_t num_tokens, void *K, void *V, int32_t out_dtype,
                         awq_stream_t stream) {
  const char *who = "awq_kv_gather";
  const awq_status st = check_cache(who, cache, cfg, num_tokens > 0);
  if (st != AWQ_OK) return st;
  if (out_dtype != AWQ_F16 && out_dtype != AWQ_BF16 && out_dtype != AWQ_F32)
    return fail(AWQ_ERR_INVALID_ARG, "%s: out_dtype=%d: must be AWQ_F16, AWQ_BF16 or AWQ_F32", who, out_dtype);
  if (num_tokens < 0) return fail(AWQ_ERR_INVALID_ARG, "%s: num_tokens=%lld is negative", who, (long long)num_tokens);
  if (num_tokens > kMaxTokens) return fail(AWQ_ERR_INVALID_ARG, "%s: more than 2^27 tokens", who);
  if (num_tokens == 0) return ok();
  if (!K || !V || !slots) return fail(AWQ_ERR_INVALID_ARG, "%s: a required pointer is NULL", who);
  if (!aligned(K, 16) || !aligned(V, 16) || !aligned(slots, 4))
    return fail(AWQ_ERR_INVALID_ARG, "%s: K and V must be 16-byte aligned, slots 4", who);
  const size_t bytes = (size_t)num_tokens * cache->num_kv_heads * cache->head_dim * (out_dtype == AWQ_F32 ? 4 : 2);
  if (!apart(K, bytes, V, bytes)) return fail(AWQ_ERR_INVALID_ARG, "%s: K and V overlap", who);
  const KvCache kc = kv_cache(cache, cfg);
  const CacheSpans cs = cache_spans(kc);
  const Span out[] = {{K, bytes}, {V, bytes}},
             in[] = {cs.codes, cs.scales, cs.zeros, {slots, (size_t)num_tokens * 4}};
  if (!all_apart(out, in)) return fail(AWQ_ERR_INVALID_ARG, "%s: K or V overlaps the cache or the slots", who);
  const YType ot = out_dtype == AWQ_F16 ? YType::F16 : out_dtype == AWQ_BF16 ? YType::BF16 : YType::F32;
  return hip_status(launch_kv_gather(kc, slots, num_tokens, K, V, ot, as_stream(stream)), who);
}

size_t awq_kv_attention_workspace_size(int64_t num_tokens, int32_t num_seqs, int32_t num_heads,
                                       const awq_kv_cache *cache, awq_config cfg,
                                       int32_t max_query_len, int64_t max_seq_len, int32_t window) {
  if (check_attention_sizes("awq_kv_attention_workspace_size", num_tokens, num_seqs, num_heads, cache, cfg,
                            max_query_len, max_seq_len, window, false) != AWQ_OK)
    return 0;
  if (num_tokens == 0 || num_seqs == 0 || max_query_len == 0) return 0;
  if (max_query_len > num_tokens) max_query_len = (int32_t)num_tokens;
  return kv_attention_plan(num_tokens, num_seqs, cache->num_kv_heads, num_heads / cache->num_kv_heads,
                           cache->head_dim, max_query_len, max_seq_len, window)
      .workspace_bytes;
}

awq_status awq_kv_attention(const void *Q, int32_t q_dtype, int64_t num_tokens, int64_t q_stride,
                            int32_t num_heads, const awq_kv_cache *cache, awq_config cfg,
                            const int32_t *block_table, int32_t max_blocks, const int32_t *seq_lens,
                            const int32_t *query_start, int32_t num_seqs, int32_t max_query_len,
                            int64_t max_seq_len, float scale, int32_t causal, int32_t window, void *O,
                            float *lse, void *workspace, size_t workspace_bytes, awq_stream_t stream) {
  const char *who = "awq_kv_attention";
  const bool work = num_tokens > 0 && num_seqs > 0 && max_query_len > 0;
  awq_status st = check_attention_sizes(who, num_tokens, num_seqs, num_heads, cache, cfg, max_query_len,
                                        max_seq_len, window, work);
  if (st != AWQ_OK) return st;
  if (q_dtype != AWQ_F16 && q_dtype != AWQ_BF16)
    return fail(AWQ_ERR_INVALID_ARG, "%s: q_dtype=%d: must be AWQ_F16 or AWQ_BF16", who, q_dtype);
  if (q_stride < (int64_t)num_heads * cache->head_dim || q_stride % 8 != 0)
    return fail(AWQ_ERR_INVALID_ARG, "%s: q_stride=%lld must be a multiple of 8 of at least num_heads * head_dim",
                who, (long long)q_stride);
  if (too_far(num_tokens, q_stride)) return fail(AWQ_ERR_INVALID_ARG, "%s: q_stride reaches beyond 2^60 elements", who);
  if (causal != 0 && causal != 1) return fail(AWQ_ERR_INVALID_ARG, "%s: causal=%d: must be 0 or 1", who, causal);
  if (window > 0 && !causal) return fail(AWQ_ERR_INVALID_ARG, "%s: a window needs causal = 1", who);
  if (!std::isfinite(scale)) return fail(AWQ_ERR_INVALID_ARG, "%s: scale is not finite", who);
  if (max_blocks < 0 || (int64_t)max_blocks * cache->page_size > kMaxContext)
    return fail(AWQ_ERR_INVALID_ARG, "%s: max_blocks=%d: negative, or beyond 2^30 tokens", who, max_blocks);
  if (!query_start && (num_tokens != num_seqs || max_query_len > 1))
    return fail(AWQ_ERR_INVALID_ARG, "%s: without query_start every request has one query token", who);
  if (workspace && !aligned(workspace, kAlign))
    return fail(AWQ_ERR_INVALID_ARG, "%s: workspace is not 256-byte aligned", who);
  if (!work) return ok();
  if (!Q || !O || !seq_lens || (max_blocks > 0 && !block_table))
    return fail(AWQ_ERR_INVALID_ARG, "%s: a required pointer is NULL", who);
  if (!aligned(Q, 16) || !aligned(O, 16)) return fail(AWQ_ERR_INVALID_ARG, "%s: Q and O must be 16-byte aligned", who);
  if (!aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(query_start, 4) || !aligned(lse, 4))
    return fail(AWQ_ERR_INVALID_ARG, "%s: block_table, seq_lens, query_start and lse must be 4-byte aligned", who);
  const size_t o_bytes = (size_t)num_tokens * num_heads * cache->head_dim * 2;
  const size_t lse_bytes = lse ? (size_t)num_tokens * num_heads * 4 : 0;
  // (no request has more query tokens than there are; the same in ..._workspace_size)
  if (max_query_len > num_tokens) max_query_len = (int32_t)num_tokens;
  const int group = num_heads / cache->num_kv_heads;
  const KvAttnPlan plan = kv_attention_plan(num_tokens, num_seqs, cache->num_kv_heads, group, cache->head_dim,
                                            max_query_len, max_seq_len, window);
  if (plan.workspace_bytes > 0 && (!workspace || workspace_bytes < plan.workspace_bytes))
    return fail(AWQ_ERR_WORKSPACE, "%s: workspace of %zu bytes, %zu needed (awq_kv_attention_workspace_size)", who,
                workspace ? workspace_bytes : 0, plan.workspace_bytes);
  const CacheSpans cs = cache_spans(kv_cache(cache, cfg));
  const Span out[] = {{O, o_bytes}, {lse, lse_bytes}, {workspace, plan.workspace_bytes}},
             in[] = {{Q, strided_bytes(num_tokens, q_stride, (int64_t)num_heads * cache->head_dim, 2)},
                     cs.codes, cs.scales, cs.zeros, {block_table, (size_t)num_seqs * max_blocks * 4},
                     {seq_lens, (size_t)num_seqs * 4}, {query_start, query_start ? ((size_t)num_seqs + 1) * 4 : 0}};
  if (!all_apart(out, in))
    return fail(AWQ_ERR_INVALID_ARG, "%s: O, lse or the workspace overlaps Q, the cache or the request arrays", who);
  if (!apart(lse, lse_bytes, O, o_bytes) || !apart(workspace, plan.workspace_bytes, O, o_bytes) ||
      !apart(workspace, plan.workspace_bytes, lse, lse_bytes))
    return fail(AWQ_ERR_INVALID_ARG, "%s: O, lse and the workspace may not overlap each other", who);
  KvAttn p{};
  p.Q = reinterpret_cast<const uint16_t *>(Q);
  p.q_stride = q_stride;
  p.O = O;
  p.lse = lse;
  p.codes = cache->codes;
  p.scales = cache->scales;
  p.zeros = cfg.zero_point ? cache->zeros : nullptr;
  p.pages = cache->num_pages;
  p.T = num_tokens;
  p.pshift = __builtin_ctz((unsigned)cache->page_size);
  p.heads = cache->num_kv_heads;
  p.group = group;
  p.by_heads = make_divisor(cache->num_kv_heads);
  p.by_group = make_divisor(group);
  p.table = block_table;
  p.max_blocks = max_blocks;
  p.seq_lens = seq_lens;
  p.query_start = query_start;
  p.max_q = max_query_len;
  p.causal = causal;
  p.window = window;
  p.scale_log2 = scale * 1.4426950408889634f;
  return hip_status(launch_kv_attention(p, num_seqs, cache->head_dim,
                                        q_dtype == AWQ_BF16 ? XType::BF16 : XType::F16, plan, workspace,
                                        as_stream(stream)),
                    who);
}

}  // extern "C"
