// C ABI of the cache's page operations (awq_kv_copy_pages, awq_kv_fork, awq_kv_release,
// awq_kv_compact): argument validation and dispatch.  Every check runs before any HIP
// call.

#include <hip/hip_runtime.h>

#include "api_kv.h"

using namespace awq;

namespace {

constexpr int64_t kMaxRows = (int64_t)1 << 20;
constexpr int32_t kMaxForks = 65535;

awq_status check_table(const char *who, const int32_t *table, int32_t num_seqs, int32_t max_blocks, int32_t page_size) {
  if (num_seqs < 0 || max_blocks < 0)
    return fail(AWQ_ERR_INVALID_ARG, "%s: negative num_seqs or max_blocks", who);
  if (num_seqs > kMaxRows) return fail(AWQ_ERR_UNSUPPORTED, "%s: num_seqs=%d exceeds 2^20", who, num_seqs);
  if ((int64_t)max_blocks * page_size > ((int64_t)1 << 31) - 1)
    return fail(AWQ_ERR_UNSUPPORTED, "%s: max_blocks=%d pages of %d tokens exceed 2^31 - 1", who, max_blocks, page_size);
  if (num_seqs > 0 && max_blocks > 0 && !table) return fail(AWQ_ERR_INVALID_ARG, "%s: a required pointer is NULL", who);
  return AWQ_OK;
}

Span ints(const int32_t *p, int64_t n) { return Span{p, p ? (size_t)n * 4 : 0}; }

template <size_t N>
bool all_aligned(const Span (&a)[N]) {
  for (const Span &x : a)
    if (x.n && !aligned(x.p, 4)) return false;
  return true;
}
// What is written lies apart from what is read and from each other.
template <size_t N, size_t M>
awq_status check_spans(const char *who, const Span (&out)[N], const Span (&in)[M]) {
  if (!all_aligned(out) || !all_aligned(in)) return fail(AWQ_ERR_INVALID_ARG, "%s: arrays must be 4-byte aligned", who);
  if (!all_apart(out, in)) return fail(AWQ_ERR_INVALID_ARG, "%s: an output overlaps an input", who);
  for (size_t i = 0; i < N; ++i)
    for (size_t j = 0; j < i; ++j)
      if (!apart(out[i].p, out[i].n, out[j].p, out[j].n))
        return fail(AWQ_ERR_INVALID_ARG, "%s: two arrays that are written overlap", who);
  return AWQ_OK;
}
awq_status check_workspace(const char *who, const void *workspace, size_t bytes, size_t need) {
  if (workspace && !aligned(workspace, kAlign))
    return fail(AWQ_ERR_INVALID_ARG, "%s: workspace is not 256-byte aligned", who);
  if (need > 0 && (!workspace || bytes < need))
    return fail(AWQ_ERR_WORKSPACE, "%s: workspace of %zu bytes, %zu needed", who, workspace ? bytes : 0, need);
  return AWQ_OK;
}
int shift_of(int32_t page_size) { return __builtin_ctz((unsigned)page_size); }
bool pages_fit(int64_t num_pages, int32_t page_size) {
  return num_pages >= 1 && num_pages <= ((int64_t)1 << 31) / page_size;
}

}  // namespace

extern "C" {

awq_status awq_kv_copy_pages(const awq_kv_cache *cache, awq_config cfg, const int32_t *src, const int32_t *dst,
                             int64_t num_copies, awq_stream_t stream) {
  const char *who = "awq_kv_copy_pages";
  const awq_status st = check_cache(who, cache, cfg, num_copies > 0);
  if (st != AWQ_OK) return st;
  if (num_copies < 0 || num_copies > ((int64_t)1 << 27))
    return fail(AWQ_ERR_INVALID_ARG, "%s: num_copies=%lld: must be in [0, 2^27]", who, (long long)num_copies);
  if (num_copies == 0) return ok();
  if (!src || !dst) return fail(AWQ_ERR_INVALID_ARG, "%s: a required pointer is NULL", who);
  const KvCache kc = kv_cache(cache, cfg);
  const CacheSpans cs = cache_spans(kc);
  const Span out[] = {cs.codes, cs.scales, cs.zeros}, in[] = {ints(src, num_copies), ints(dst, num_copies)};
  const awq_status sp = check_spans(who, out, in);
  if (sp != AWQ_OK) return sp;
  return hip_status(launch_kv_copy_pages(kc, src, dst, num_copies, as_stream(stream)), who);
}

awq_status awq_kv_fork(const awq_kv_cache *cache, awq_config cfg, const int32_t *parents, const int32_t *children,
                       const int32_t *lens, int32_t num_forks, int32_t *block_table, int32_t num_seqs,
                       int32_t max_blocks, int32_t *shared, const int32_t *free_pages, int32_t num_free,
                       const int32_t *taken, int32_t *pages_used, awq_stream_t stream) {
  const char *who = "awq_kv_fork";
  awq_status st = check_cache(who, cache, cfg, num_forks > 0);
  if (st != AWQ_OK) return st;
  st = check_table(who, block_table, num_seqs, max_blocks, cache->page_size);
  if (st != AWQ_OK) return st;
  if (num_forks < 0 || num_free < 0) return fail(AWQ_ERR_INVALID_ARG, "%s: negative num_forks or num_free", who);
  if (num_forks > kMaxForks) return fail(AWQ_ERR_UNSUPPORTED, "%s: num_forks=%d exceeds %d", who, num_forks, kMaxForks);
  if (!pages_used || (num_forks > 0 && (!parents || !children || !lens || !shared)) || (num_free > 0 && !free_pages))
    return fail(AWQ_ERR_INVALID_ARG, "%s: a required pointer is NULL", who);
  const KvCache kc = kv_cache(cache, cfg);
  CacheSpans cs = cache_spans(kc);
  if (num_forks == 0) cs.codes.n = cs.scales.n = cs.zeros.n = 0;
  const Span out[] = {cs.codes, cs.scales, cs.zeros, ints(block_table, (int64_t)num_seqs * max_blocks),
                      ints(shared, num_forks > 0 ? cache->num_pages : 0), ints(pages_used, 1)},
             in[] = {ints(parents, num_forks), ints(children, num_forks), ints(lens, num_forks),
                     ints(free_pages, num_free), ints(taken, 1)};
  st = check_spans(who, out, in);
  if (st != AWQ_OK) return st;
  const ForkArgs a{parents, children, lens, num_forks, num_seqs, max_blocks, shift_of(cache->page_size), block_table,
                   shared, cache->num_pages, free_pages, num_free, taken, pages_used};
  return hip_status(launch_kv_fork(a, kc, as_stream(stream)), who);
}

size_t awq_kv_release_workspace_size(int64_t num_pages, int32_t num_free) {
  if (!pages_fit(num_pages, AWQ_KV_MIN_PAGE) || num_free < 0) {
    (void)fail(AWQ_ERR_INVALID_ARG, "awq_kv_release_workspace_size: num_pages=%lld, num_free=%d",
               (long long)num_pages, num_free);
    return 0;
  }
  return kv_release_workspace(num_pages, num_free);
}

awq_status awq_kv_release(int32_t *block_table, int32_t num_seqs, int32_t max_blocks, int32_t page_size,
                          const int32_t *seq_lens, const int32_t *start, const int32_t *end, int32_t *shared,
                          int64_t num_pages, const int32_t *free_pages, int32_t num_free, const int32_t *taken,
                          int32_t *free_out, int32_t num_out, int32_t *num_free_out, void *workspace,
                          size_t workspace_bytes, awq_stream_t stream) {
  const char *who = "awq_kv_release";
  awq_status st = check_page(who, page_size);
  if (st != AWQ_OK) return st;
  st = check_table(who, block_table, num_seqs, max_blocks, page_size);
  if (st != AWQ_OK) return st;
  if (!pages_fit(num_pages, page_size))
    return fail(AWQ_ERR_INVALID_ARG, "%s: num_pages=%lld: must be positive, and at most 2^31 slots", who, (long long)num_pages);
  if (num_free < 0 || num_out < 0) return fail(AWQ_ERR_INVALID_ARG, "%s: negative num_free or num_out", who);
  if (!shared || !num_free_out || (num_seqs > 0 && !seq_lens) || (num_free > 0 && !free_pages) || (num_out > 0 && !free_out))
    return fail(AWQ_ERR_INVALID_ARG, "%s: a required pointer is NULL", who);
  const size_t need = kv_release_workspace(num_pages, num_free);
  st = check_workspace(who, workspace, workspace_bytes, need);
  if (st != AWQ_OK) return st;
  const Span out[] = {ints(block_table, (int64_t)num_seqs * max_blocks), ints(shared, num_pages), ints(free_out, num_out),
                      ints(num_free_out, 1), {workspace, need}},
             in[] = {ints(seq_lens, num_seqs), ints(start, num_seqs), ints(end, num_seqs), ints(free_pages, num_free),
                     ints(taken, 1)};
  st = check_spans(who, out, in);
  if (st != AWQ_OK) return st;
  const ReleaseArgs a{block_table, num_seqs, max_blocks, shift_of(page_size), seq_lens, start, end, shared, num_pages,
                      free_pages, num_free, taken, free_out, num_out, num_free_out};
  return hip_status(launch_kv_release(a, workspace, as_stream(stream)), who);
}

size_t awq_kv_compact_workspace_size(int64_t num_pages, int32_t page_size) {
  if (check_page("awq_kv_compact_workspace_size", page_size) != AWQ_OK) return 0;
  if (!pages_fit(num_pages, page_size)) {
    (void)fail(AWQ_ERR_INVALID_ARG, "awq_kv_compact_workspace_size: num_pages=%lld", (long long)num_pages);
    return 0;
  }
  return kv_compact_workspace(num_pages);
}

awq_status awq_kv_compact(const awq_kv_cache *cache, awq_config cfg, int32_t *block_table, int32_t num_seqs,
                          int32_t max_blocks, const int32_t *seq_lens, int32_t *shared, int32_t *free_out,
                          int32_t *num_used, void *workspace, size_t workspace_bytes, awq_stream_t stream) {
  const char *who = "awq_kv_compact";
  awq_status st = check_cache(who, cache, cfg, true);
  if (st != AWQ_OK) return st;
  st = check_table(who, block_table, num_seqs, max_blocks, cache->page_size);
  if (st != AWQ_OK) return st;
  if (!shared || !free_out || !num_used || (num_seqs > 0 && !seq_lens))
    return fail(AWQ_ERR_INVALID_ARG, "%s: a required pointer is NULL", who);
  const size_t need = kv_compact_workspace(cache->num_pages);
  st = check_workspace(who, workspace, workspace_bytes, need);
  if (st != AWQ_OK) return st;
  const KvCache kc = kv_cache(cache, cfg);
  const CacheSpans cs = cache_spans(kc);
  const Span out[] = {cs.codes, cs.scales, cs.zeros, ints(block_table, (int64_t)num_seqs * max_blocks),
                      ints(shared, cache->num_pages), ints(free_out, cache->num_pages), ints(num_used, 1), {workspace, need}},
             in[] = {ints(seq_lens, num_seqs)};
  st = check_spans(who, out, in);
  if (st != AWQ_OK) return st;
  const CompactArgs a{block_table, num_seqs, max_blocks, shift_of(cache->page_size), seq_lens, shared, free_out, num_used,
                      nullptr, nullptr, nullptr, nullptr};
  return hip_status(launch_kv_compact(a, kc, workspace, as_stream(stream)), who);
}

}  // extern "C"
