// C ABI of rotary positions (awq_rope*, awq_kv_append_rope): argument validation and
// dispatch, before any HIP call; the frequencies' host arithmetic.

#include <hip/hip_runtime.h>

#include <cmath>

#include "api_kv.h"

using namespace awq;

namespace {

constexpr double kTwoPi = 6.283185307179586;
// Four tokens to a workgroup of 256, and a grid holds less than 2^32 threads.
constexpr int64_t kMaxRopeTokens = (int64_t)1 << 25;

awq_status check_rope(const char *who, const awq_rope_args *r, int32_t head_dim) {
  if (!r) return fail(AWQ_ERR_INVALID_ARG, "%s: rope is NULL", who);
  if (r->rotary_dim < 16 || r->rotary_dim % 16 != 0 || r->rotary_dim > head_dim)
    return fail(AWQ_ERR_UNSUPPORTED, "%s: rotary_dim=%d: must be a multiple of 16 in [16, head_dim=%d]", who,
                r->rotary_dim, head_dim);
  if ((r->interleaved != 0 && r->interleaved != 1) || (r->inverse != 0 && r->inverse != 1))
    return fail(AWQ_ERR_INVALID_ARG, "%s: interleaved=%d and inverse=%d must be 0 or 1", who, r->interleaved,
                r->inverse);
  if (!std::isfinite(r->attention_factor))
    return fail(AWQ_ERR_INVALID_ARG, "%s: attention_factor is not finite", who);
  return AWQ_OK;
}
awq_status check_rope_arrays(const char *who, const awq_rope_args *r) {
  if (!r->positions || !r->inv_freq) return fail(AWQ_ERR_INVALID_ARG, "%s: a required pointer is NULL", who);
  if (!aligned(r->positions, 4) || !aligned(r->inv_freq, 8))
    return fail(AWQ_ERR_INVALID_ARG, "%s: positions must be 4-byte aligned, inv_freq 8", who);
  return AWQ_OK;
}
RopeArgs rope_args(const awq_rope_args *r) {
  return RopeArgs{r->positions, r->inv_freq, r->attention_factor, r->rotary_dim, r->interleaved == 1, r->inverse == 1};
}

awq_status check_heads(const char *who, const char *name, int32_t heads, int64_t width, int64_t tokens, int64_t in,
                       int64_t out) {
  if (heads < 0 || heads > AWQ_KV_MAX_HEADS)
    return fail(AWQ_ERR_INVALID_ARG, "%s: %d heads of %s: must be in [0, %d]", who, heads, name, AWQ_KV_MAX_HEADS);
  if (heads == 0) return AWQ_OK;
  if (in < width || out < width || in % 8 != 0 || out % 8 != 0)
    return fail(AWQ_ERR_INVALID_ARG, "%s: %s: token strides %lld and %lld must be multiples of 8 of at least %lld", who,
                name, (long long)in, (long long)out, (long long)width);
  if (too_far(tokens, in) || too_far(tokens, out))
    return fail(AWQ_ERR_INVALID_ARG, "%s: %s: token strides reach beyond 2^60 elements", who, name);
  return AWQ_OK;
}
awq_status check_pointers(const char *who, const char *name, int32_t heads, const void *x, const void *y) {
  if (heads == 0) return AWQ_OK;
  if (!x || !y) return fail(AWQ_ERR_INVALID_ARG, "%s: a required pointer is NULL", who);
  if (!aligned(x, 16) || !aligned(y, 16))
    return fail(AWQ_ERR_INVALID_ARG, "%s: %s and its output must be 16-byte aligned", who, name);
  return AWQ_OK;
}
Span rows(const void *p, int32_t heads, int64_t tokens, int64_t stride, int32_t D) {
  return Span{p, heads == 0 ? 0 : strided_bytes(tokens, stride, (int64_t)heads * D, 2)};
}
// One tensor of a call: what is read, and what is written.
struct RopeRows {
  Span in, out;
  int64_t in_stride, out_stride, width;
};
RopeRows rope_rows(const void *x, const void *y, int32_t heads, int64_t tokens, int64_t xs, int64_t ys, int32_t D) {
  return RopeRows{rows(x, heads, tokens, xs, D), rows(y, heads, tokens, ys, D), xs, ys, (int64_t)heads * D};
}
bool in_place_or_apart(const RopeRows &r) {
  return (r.in.p == r.out.p && r.in_stride == r.out_stride) ||
         rows_apart(r.in, r.in_stride, r.width, r.out, r.out_stride, r.width, 2);
}
bool written_apart(const RopeRows &r, const Span &other, int64_t stride, int64_t width) {
  return rows_apart(r.out, r.out_stride, r.width, other, stride, width, 2);
}
RopeArray rope_array(const void *x, void *y, int64_t xs, int64_t ys, int32_t heads) {
  return RopeArray{reinterpret_cast<const uint16_t *>(x), reinterpret_cast<uint16_t *>(y), xs, ys, heads};
}

}  // namespace

extern "C" {

awq_status awq_rope_frequencies(int32_t rotary_dim, double base, const awq_rope_scaling *scaling, double *inv_freq,
                                double *attention_factor) {
  const char *who = "awq_rope_frequencies";
  if (rotary_dim < 16 || rotary_dim % 16 != 0 || rotary_dim > AWQ_ROPE_MAX_DIM)
    return fail(AWQ_ERR_UNSUPPORTED, "%s: rotary_dim=%d: must be a multiple of 16 in [16, %d]", who, rotary_dim,
                AWQ_ROPE_MAX_DIM);
  if (!std::isfinite(base) || base <= 1.0) return fail(AWQ_ERR_INVALID_ARG, "%s: base must be above 1", who);
  if (!inv_freq || !attention_factor) return fail(AWQ_ERR_INVALID_ARG, "%s: a required pointer is NULL", who);
  const awq_rope_scaling none{};
  const awq_rope_scaling &sc = scaling ? *scaling : none;
  const double R = rotary_dim, s = sc.factor, L = sc.original_len;
  if (sc.kind < AWQ_ROPE_NONE || sc.kind > AWQ_ROPE_BANDS)
    return fail(AWQ_ERR_INVALID_ARG, "%s: scaling kind %d is unknown", who, sc.kind);
  if (sc.kind != AWQ_ROPE_NONE && !(std::isfinite(s) && s > 0.0))
    return fail(AWQ_ERR_INVALID_ARG, "%s: the scaling's factor must be positive", who);
  const bool ranged = sc.kind == AWQ_ROPE_YARN || sc.kind == AWQ_ROPE_BANDS;
  const double low = sc.low == 0.0 ? 1.0 : sc.low, high = sc.high == 0.0 ? (sc.kind == AWQ_ROPE_YARN ? 32.0 : 4.0) : sc.high;
  if (ranged && !(std::isfinite(L) && L > 0.0))
    return fail(AWQ_ERR_INVALID_ARG, "%s: the scaling's original_len must be positive", who);
  if (ranged && !(std::isfinite(low) && std::isfinite(high) && low > 0.0 && high > low))
    return fail(AWQ_ERR_INVALID_ARG, "%s: the scaling's low and high must satisfy 0 < low < high", who);
  const double b = sc.kind == AWQ_ROPE_NTK ? base * std::pow(s, R / (R - 2.0)) : base;
  if (!std::isfinite(b) || b <= 1.0) return fail(AWQ_ERR_INVALID_ARG, "%s: the scaled base must be above 1", who);
  // number of the pair that turns n times within L positions, as a real number
  auto pair_of = [&](double n) { return R * std::log(L / (n * kTwoPi)) / (2.0 * std::log(base)); };
  const double first = sc.kind == AWQ_ROPE_YARN ? std::fmax(std::floor(pair_of(high)), 0.0) : 0.0;
  const double last = sc.kind == AWQ_ROPE_YARN ? std::fmin(std::ceil(pair_of(low)), R - 1.0) : 0.0;
  for (int32_t j = 0; j < rotary_dim / 2; ++j) {
    const double f = std::pow(b, -2.0 * j / R);
    double v = f;
    if (sc.kind == AWQ_ROPE_LINEAR) {
      v = f / s;
    } else if (sc.kind == AWQ_ROPE_YARN) {
      const double m = std::fmin(std::fmax((j - first) / std::fmax(last - first, 0.001), 0.0), 1.0);
      v = f / s * m + f * (1.0 - m);
    } else if (sc.kind == AWQ_ROPE_BANDS) {
      const double turns = L * f / kTwoPi;
      const double m = std::fmin(std::fmax((turns - low) / (high - low), 0.0), 1.0);
      v = f / s * (1.0 - m) + f * m;
    }
    inv_freq[j] = v;
  }
  *attention_factor = sc.kind == AWQ_ROPE_YARN && s > 1.0 ? 0.1 * std::log(s) + 1.0 : 1.0;
  return ok();
}

awq_status awq_rope(const void *Q, void *Q_out, int32_t num_heads, int64_t q_stride, int64_t qo_stride, const void *K,
                    void *K_out, int32_t num_kv_heads, int64_t k_stride, int64_t ko_stride, int32_t x_dtype,
                    int64_t num_tokens, int32_t head_dim, const awq_rope_args *rope, awq_stream_t stream) {
  const char *who = "awq_rope";
  if (x_dtype != AWQ_F16 && x_dtype != AWQ_BF16)
    return fail(AWQ_ERR_INVALID_ARG, "%s: x_dtype=%d: must be AWQ_F16 or AWQ_BF16", who, x_dtype);
  if (head_dim < 16 || head_dim % 16 != 0 || head_dim > AWQ_ROPE_MAX_DIM)
    return fail(AWQ_ERR_UNSUPPORTED, "%s: head_dim=%d: must be a multiple of 16 in [16, %d]", who, head_dim,
                AWQ_ROPE_MAX_DIM);
  if (num_tokens < 0 || num_tokens > kMaxRopeTokens)
    return fail(AWQ_ERR_INVALID_ARG, "%s: num_tokens=%lld: must be in [0, 2^25]", who, (long long)num_tokens);
  awq_status st = check_rope(who, rope, head_dim);
  if (st == AWQ_OK) st = check_heads(who, "Q", num_heads, (int64_t)num_heads * head_dim, num_tokens, q_stride, qo_stride);
  if (st == AWQ_OK) st = check_heads(who, "K", num_kv_heads, (int64_t)num_kv_heads * head_dim, num_tokens, k_stride, ko_stride);
  if (st != AWQ_OK) return st;
  if (num_tokens == 0 || (num_heads == 0 && num_kv_heads == 0)) return ok();
  st = check_rope_arrays(who, rope);
  if (st == AWQ_OK) st = check_pointers(who, "Q", num_heads, Q, Q_out);
  if (st == AWQ_OK) st = check_pointers(who, "K", num_kv_heads, K, K_out);
  if (st != AWQ_OK) return st;
  const RopeRows q = rope_rows(Q, Q_out, num_heads, num_tokens, q_stride, qo_stride, head_dim),
                 k = rope_rows(K, K_out, num_kv_heads, num_tokens, k_stride, ko_stride, head_dim);
  const Span out[] = {q.out, k.out},
             in[] = {{rope->positions, (size_t)num_tokens * 4}, {rope->inv_freq, (size_t)rope->rotary_dim * 4}};
  if (!all_apart(out, in)) return fail(AWQ_ERR_INVALID_ARG, "%s: an output overlaps positions or inv_freq", who);
  if (!in_place_or_apart(q) || !in_place_or_apart(k))
    return fail(AWQ_ERR_INVALID_ARG, "%s: an output overlaps its input without being it", who);
  if (!written_apart(q, k.in, k_stride, k.width) || !written_apart(k, q.in, q_stride, q.width) ||
      !written_apart(q, k.out, ko_stride, k.width))
    return fail(AWQ_ERR_INVALID_ARG, "%s: an output overlaps the other's input or output", who);
  return hip_status(launch_rope(rope_args(rope), rope_array(Q, Q_out, q_stride, qo_stride, num_heads),
                                rope_array(K, K_out, k_stride, ko_stride, num_kv_heads),
                                x_dtype == AWQ_BF16 ? XType::BF16 : XType::F16, num_tokens, head_dim, as_stream(stream)),
                    who);
}

awq_status awq_kv_append_rope(const void *Q, void *Q_out, int32_t num_heads, int64_t q_stride, int64_t qo_stride,
                              const void *K, const void *V, int32_t x_dtype, int64_t num_tokens, int64_t k_stride,
                              int64_t v_stride, const awq_kv_cache *cache, awq_config cfg, const int32_t *slots,
                              const awq_rope_args *rope, int32_t *nonfinite_count, awq_stream_t stream) {
  const char *who = "awq_kv_append_rope";
  awq_status st = check_append(who, K, V, x_dtype, num_tokens, k_stride, v_stride, cache, cfg, slots, nonfinite_count);
  if (st != AWQ_OK) return st;
  if (num_tokens > kMaxRopeTokens) return fail(AWQ_ERR_INVALID_ARG, "%s: more than 2^25 tokens", who);
  const int32_t D = cache->head_dim;
  st = check_rope(who, rope, D);
  if (st == AWQ_OK) st = check_heads(who, "Q", num_heads, (int64_t)num_heads * D, num_tokens, q_stride, qo_stride);
  if (st != AWQ_OK) return st;
  if (num_tokens == 0) return ok();
  st = check_rope_arrays(who, rope);
  if (st == AWQ_OK) st = check_pointers(who, "Q", num_heads, Q, Q_out);
  if (st != AWQ_OK) return st;
  const KvCache kc = kv_cache(cache, cfg);
  const CacheSpans cs = cache_spans(kc);
  const RopeRows q = rope_rows(Q, Q_out, num_heads, num_tokens, q_stride, qo_stride, D);
  const int64_t width = (int64_t)cache->num_kv_heads * D;
  const Span pos = {rope->positions, (size_t)num_tokens * 4}, freq = {rope->inv_freq, (size_t)rope->rotary_dim * 4},
             count = {nonfinite_count, nonfinite_count ? 4u : 0u};
  const Span read[] = {pos, freq, q.in}, written[] = {cs.codes, cs.scales, cs.zeros, count},
             q_out[] = {q.out}, others[] = {pos, freq, {slots, (size_t)num_tokens * 4}, cs.codes, cs.scales, cs.zeros, count};
  if (!all_apart(read, written))
    return fail(AWQ_ERR_INVALID_ARG, "%s: Q, positions, inv_freq, nonfinite_count and the cache may not overlap", who);
  if (!in_place_or_apart(q)) return fail(AWQ_ERR_INVALID_ARG, "%s: Q_out overlaps Q without being it", who);
  if (!all_apart(q_out, others) ||
      !written_apart(q, {K, strided_bytes(num_tokens, k_stride, width, 2)}, k_stride, width) ||
      !written_apart(q, {V, strided_bytes(num_tokens, v_stride, width, 2)}, v_stride, width))
    return fail(AWQ_ERR_INVALID_ARG, "%s: Q_out overlaps K, V, the cache or the arrays that are read", who);
  return hip_status(launch_kv_append_rope(rope_args(rope), rope_array(Q, Q_out, q_stride, qo_stride, num_heads),
                                          reinterpret_cast<const uint16_t *>(K), reinterpret_cast<const uint16_t *>(V),
                                          x_dtype == AWQ_BF16 ? XType::BF16 : XType::F16, num_tokens, k_stride,
                                          v_stride, slots, kc, nonfinite_count, as_stream(stream)),
                    who);
}

}  // extern "C"
