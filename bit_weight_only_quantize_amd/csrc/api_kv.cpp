// C ABI of the 4-bit paged key/value cache (awq_kv_*): argument validation and
// dispatch.  Every check runs before any HIP call.

#include <hip/hip_runtime.h>

#include <cmath>

#include "api_kv.h"

using namespace awq;

namespace {

// Sizes of an attention call that its workspace depends on.
awq_status check_attention_sizes(const char *who, int64_t num_tokens, int32_t num_seqs,
                                 int32_t num_heads, const awq_kv_cache *cache, awq_config cfg,
                                 int32_t max_query_len, int64_t max_seq_len,
                                 const awq_kv_attention_options *opts, bool need_ptrs) {
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
  if (!opts) return fail(AWQ_ERR_INVALID_ARG, "%s: opts is NULL", who);
  if (opts->window < 0) return fail(AWQ_ERR_INVALID_ARG, "%s: window=%d is negative", who, opts->window);
  if (opts->sinks < 0 || opts->sinks > kMaxContext)
    return fail(AWQ_ERR_INVALID_ARG, "%s: sinks=%d: must be in [0, 2^30]", who, opts->sinks);
  if (opts->prefix_len < 0 || opts->prefix_blocks < 0)
    return fail(AWQ_ERR_INVALID_ARG, "%s: negative prefix_len or prefix_blocks", who);
  if (opts->prefix_len > 0) {
    if (opts->window > 0) return fail(AWQ_ERR_UNSUPPORTED, "%s: a shared prefix takes no window", who);
    if (opts->prefix_table && opts->prefix_len > (int64_t)opts->prefix_blocks * cache->page_size)
      return fail(AWQ_ERR_INVALID_ARG, "%s: prefix_len=%d is beyond the prefix_blocks=%d pages of %d tokens", who,
                  opts->prefix_len, opts->prefix_blocks, cache->page_size);
    if (opts->prefix_len > kMaxContext) return fail(AWQ_ERR_UNSUPPORTED, "%s: prefix_len=%d exceeds 2^30", who, opts->prefix_len);
    // (the rows of all requests are counted as one's, and a grid of waves joins a row each)
    if (num_tokens * (num_heads / cache->num_kv_heads) > ((int64_t)1 << 25))
      return fail(AWQ_ERR_UNSUPPORTED, "%s: a shared prefix takes at most 2^25 query tokens times the query heads per key/value head", who);
  }
  return AWQ_OK;
}

// The plan of a call: of one over all keys, or of one over a shared prefix and the rest.
struct AttentionPlan {
  bool prefix;
  KvAttnPlan whole;
  KvPrefixPlan split;
  size_t bytes() const { return prefix ? split.workspace_bytes : whole.workspace_bytes; }
};
AttentionPlan plan_of(int64_t num_tokens, int32_t num_seqs, int heads, int group, int D, int32_t max_query_len,
                      int64_t max_seq_len, const awq_kv_attention_options &o) {
  AttentionPlan p{};
  if (o.prefix_len > 0) {
    p.split = kv_prefix_plan(num_tokens, num_seqs, heads, group, D, max_query_len, max_seq_len, o.prefix_len);
    p.prefix = o.prefix_table || kv_prefix_pays(p.split, num_tokens, num_seqs, heads, group, D, max_query_len, o.prefix_len);
  }
  if (!p.prefix) p.whole = kv_attention_plan(num_tokens, num_seqs, heads, group, D, max_query_len, max_seq_len, o.window, o.sinks);
  return p;
}

size_t attention_workspace(const char *who, int64_t num_tokens, int32_t num_seqs, int32_t num_heads,
                           const awq_kv_cache *cache, awq_config cfg, int32_t max_query_len, int64_t max_seq_len,
                           const awq_kv_attention_options *opts) {
  if (check_attention_sizes(who, num_tokens, num_seqs, num_heads, cache, cfg, max_query_len, max_seq_len, opts, false) !=
      AWQ_OK)
    return 0;
  if (num_tokens == 0 || num_seqs == 0 || max_query_len == 0) return 0;
  if (max_query_len > num_tokens) max_query_len = (int32_t)num_tokens;
  return plan_of(num_tokens, num_seqs, cache->num_kv_heads, num_heads / cache->num_kv_heads, cache->head_dim,
                 max_query_len, max_seq_len, *opts)
      .bytes();
}

awq_status attend(const char *who, const void *Q, int32_t q_dtype, int64_t num_tokens, int64_t q_stride,
                  int32_t num_heads, const awq_kv_cache *cache, awq_config cfg, const int32_t *block_table,
                  int32_t max_blocks, const int32_t *seq_lens, const int32_t *query_start, int32_t num_seqs,
                  int32_t max_query_len, int64_t max_seq_len, float scale, const awq_kv_attention_options *opts,
                  void *O, float *lse, void *workspace, size_t workspace_bytes, awq_stream_t stream) {
  const bool work = num_tokens > 0 && num_seqs > 0 && max_query_len > 0;
  awq_status st = check_attention_sizes(who, num_tokens, num_seqs, num_heads, cache, cfg, max_query_len,
                                        max_seq_len, opts, work);
  if (st != AWQ_OK) return st;
  const awq_kv_attention_options &o = *opts;
  if (q_dtype != AWQ_F16 && q_dtype != AWQ_BF16)
    return fail(AWQ_ERR_INVALID_ARG, "%s: q_dtype=%d: must be AWQ_F16 or AWQ_BF16", who, q_dtype);
  if (q_stride < (int64_t)num_heads * cache->head_dim || q_stride % 8 != 0)
    return fail(AWQ_ERR_INVALID_ARG, "%s: q_stride=%lld must be a multiple of 8 of at least num_heads * head_dim",
                who, (long long)q_stride);
  if (too_far(num_tokens, q_stride)) return fail(AWQ_ERR_INVALID_ARG, "%s: q_stride reaches beyond 2^60 elements", who);
  if (o.causal != 0 && o.causal != 1) return fail(AWQ_ERR_INVALID_ARG, "%s: causal=%d: must be 0 or 1", who, o.causal);
  if (o.window > 0 && !o.causal) return fail(AWQ_ERR_INVALID_ARG, "%s: a window needs causal = 1", who);
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
  if (o.prefix_len > 0 && !o.prefix_table && o.prefix_len > (int64_t)max_blocks * cache->page_size)
    return fail(AWQ_ERR_INVALID_ARG, "%s: prefix_len=%d is beyond the max_blocks=%d pages of %d tokens", who,
                o.prefix_len, max_blocks, cache->page_size);
  if (!aligned(Q, 16) || !aligned(O, 16)) return fail(AWQ_ERR_INVALID_ARG, "%s: Q and O must be 16-byte aligned", who);
  if (!aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(query_start, 4) || !aligned(lse, 4) ||
      !aligned(o.prefix_table, 4))
    return fail(AWQ_ERR_INVALID_ARG, "%s: block_table, seq_lens, query_start, prefix_table and lse must be 4-byte aligned", who);
  const size_t o_bytes = (size_t)num_tokens * num_heads * cache->head_dim * 2;
  const size_t lse_bytes = lse ? (size_t)num_tokens * num_heads * 4 : 0;
  // (no request has more query tokens than there are; the same in ..._workspace_size)
  if (max_query_len > num_tokens) max_query_len = (int32_t)num_tokens;
  const int group = num_heads / cache->num_kv_heads;
  const AttentionPlan plan = plan_of(num_tokens, num_seqs, cache->num_kv_heads, group, cache->head_dim, max_query_len,
                                     max_seq_len, o);
  const size_t need = plan.bytes();
  if (need > 0 && (!workspace || workspace_bytes < need))
    return fail(AWQ_ERR_WORKSPACE, "%s: workspace of %zu bytes, %zu needed (%s_workspace_size)", who,
                workspace ? workspace_bytes : 0, need, who);
  const CacheSpans cs = cache_spans(kv_cache(cache, cfg));
  const Span out[] = {{O, o_bytes}, {lse, lse_bytes}, {workspace, need}},
             in[] = {{Q, strided_bytes(num_tokens, q_stride, (int64_t)num_heads * cache->head_dim, 2)},
                     cs.codes, cs.scales, cs.zeros, {block_table, (size_t)num_seqs * max_blocks * 4},
                     {seq_lens, (size_t)num_seqs * 4}, {query_start, query_start ? ((size_t)num_seqs + 1) * 4 : 0},
                     {o.prefix_table, o.prefix_table && o.prefix_len > 0 ? (size_t)o.prefix_blocks * 4 : 0}};
  if (!all_apart(out, in))
    return fail(AWQ_ERR_INVALID_ARG, "%s: O, lse or the workspace overlaps Q, the cache or the request arrays", who);
  if (!apart(lse, lse_bytes, O, o_bytes) || !apart(workspace, need, O, o_bytes) ||
      !apart(workspace, need, lse, lse_bytes))
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
  p.causal = o.causal;
  p.window = o.window;
  p.num_seqs = num_seqs;
  p.sinks = o.window > 0 ? o.sinks : 0;
  p.after = plan.prefix ? o.prefix_len : 0;
  p.prefix_table = o.prefix_table;                   // (null: the kernel finds a row that holds it)
  p.prefix_blocks = o.prefix_table ? o.prefix_blocks : max_blocks;
  p.scale_log2 = scale * 1.4426950408889634f;
  const XType xt = q_dtype == AWQ_BF16 ? XType::BF16 : XType::F16;
  return hip_status(plan.prefix
                        ? launch_kv_attention_prefix(p, num_seqs, cache->head_dim, xt, plan.split, workspace, as_stream(stream))
                        : launch_kv_attention(p, num_seqs, cache->head_dim, xt, plan.whole, workspace, as_stream(stream)),
                    who);
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
  const awq_status st = check_append(who, K, V, x_dtype, num_tokens, k_stride, v_stride, cache, cfg, slots, nonfinite_count);
  if (st != AWQ_OK) return st;
  if (num_tokens == 0) return ok();
  return hip_status(launch_kv_append(reinterpret_cast<const uint16_t *>(K), reinterpret_cast<const uint16_t *>(V),
                                     x_dtype == AWQ_BF16 ? XType::BF16 : XType::F16, num_tokens, k_stride,
                                     v_stride, slots, kv_cache(cache, cfg), nonfinite_count,
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
  const awq_kv_attention_options o{1, window, 0, 0, nullptr, 0};
  return attention_workspace("awq_kv_attention_workspace_size", num_tokens, num_seqs, num_heads, cache, cfg,
                             max_query_len, max_seq_len, &o);
}

awq_status awq_kv_attention(const void *Q, int32_t q_dtype, int64_t num_tokens, int64_t q_stride,
                            int32_t num_heads, const awq_kv_cache *cache, awq_config cfg,
                            const int32_t *block_table, int32_t max_blocks, const int32_t *seq_lens,
                            const int32_t *query_start, int32_t num_seqs, int32_t max_query_len,
                            int64_t max_seq_len, float scale, int32_t causal, int32_t window, void *O,
                            float *lse, void *workspace, size_t workspace_bytes, awq_stream_t stream) {
  const awq_kv_attention_options o{causal, window, 0, 0, nullptr, 0};
  return attend("awq_kv_attention", Q, q_dtype, num_tokens, q_stride, num_heads, cache, cfg, block_table, max_blocks,
                seq_lens, query_start, num_seqs, max_query_len, max_seq_len, scale, &o, O, lse, workspace,
                workspace_bytes, stream);
}

size_t awq_kv_attention_ex_workspace_size(int64_t num_tokens, int32_t num_seqs, int32_t num_heads,
                                          const awq_kv_cache *cache, awq_config cfg, int32_t max_query_len,
                                          int64_t max_seq_len, const awq_kv_attention_options *opts) {
  return attention_workspace("awq_kv_attention_ex_workspace_size", num_tokens, num_seqs, num_heads, cache, cfg,
                             max_query_len, max_seq_len, opts);
}

awq_status awq_kv_attention_ex(const void *Q, int32_t q_dtype, int64_t num_tokens, int64_t q_stride, int32_t num_heads,
                               const awq_kv_cache *cache, awq_config cfg, const int32_t *block_table,
                               int32_t max_blocks, const int32_t *seq_lens, const int32_t *query_start,
                               int32_t num_seqs, int32_t max_query_len, int64_t max_seq_len, float scale,
                               const awq_kv_attention_options *opts, void *O, float *lse, void *workspace,
                               size_t workspace_bytes, awq_stream_t stream) {
  return attend("awq_kv_attention_ex", Q, q_dtype, num_tokens, q_stride, num_heads, cache, cfg, block_table, max_blocks,
                seq_lens, query_start, num_seqs, max_query_len, max_seq_len, scale, opts, O, lse, workspace,
                workspace_bytes, stream);
}

}  // extern "C"
