// Attention over the 4-bit paged key/value cache on gfx950.
//
// For a query row q (one head of one token) over the keys t that it sees:
//   S_t = sum_d q_d (kc_td - kz_t)          exact integers kc - kz, fp32 sums
//   u_t = S_t * ks_t * scale * log2(e)
//   O   = sum_t 2^(u_t) vs_t (vc_t - vz_t) / sum_t 2^(u_t)
// with codes c, zero points z and steps s of the key and value of token t.
// Codes reach the matrix cores as exact small integers in fp16 (or as exact
// subnormals, below) and queries as fp16, after a power-of-two factor per row
// where needed, so the only operand that is rounded is the weight
// P'_t = 2^(u_t - M) vs_t, once, to fp16 (2^-11 relative); sums, the running
// maximum and the normalizer are fp32.  M follows the row's largest u_t + log2 vs_t,
// the largest weight times its step (not the largest of each, which a large step
// of no weight would drive apart), and is kept so that the largest P' lies between
// 2^(kRaise - kSpread) and 2^kLimit: nothing overflows, and weights are rounded to
// less than 11 bits (fp16's subnormals, steps of 2^-24) only below 2^-16 of the
// largest, an error of 2^-27 of it at most.  M moves only when a tile might pass
// 2^kLimit, which makes the rescaling of O (and the exchange between lanes that it
// needs) rare: a wave tests one ballot, of the tile's largest u against `slack`,
// which allows for the largest step that the tile may have, and of its steps
// against that.
//
// Rows of one key/value head are packed: row r of a request is query token
// r / group, head r % group of the `group` query heads that share the
// key/value head, so that shared heads cost one pass over the cache.
//
// Products are taken transposed, S^T = K Q^T and O^T = V^T P^T: the result of
// the first then holds, in each lane, several keys of one query row, which is
// the operand layout of the second, with no exchange between lanes.  The
// contraction over keys may run in any order, so the key order inside an MFMA
// is the one that falls out of the first product; the cache interleaves four
// tokens of a value word to match.

#include <type_traits>

#include "awq_internal.h"
#include "device_common.h"

namespace awq {

typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr float kRaise = 7.0f;         // log2 of the largest P' where M is set, at most
constexpr float kLimit = 15.0f;        // ... and before it is set again
constexpr int kSpread = 5;             // log2 by which M may be above that for more slack
constexpr float kLeastStep = 0x1p-14f; // of what awq_kv_append writes; smaller ones count as this
constexpr float kNone = -__FLT_MAX__;  // "no key yet": finite, so kNone - kNone is 0

__device__ __forceinline__ f32x16 mfma32x16(u32x4 a, u32x4 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a),
                                                __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

__device__ __forceinline__ float lo_half(uint32_t w) { return half_bits_to_float((uint16_t)(w & 0xFFFFu)); }
__device__ __forceinline__ float hi_half(uint32_t w) { return half_bits_to_float((uint16_t)(w >> 16)); }

__device__ __forceinline__ uint32_t pack_half2(float a, float b) {
  const f16x2 h = {(_Float16)a, (_Float16)b};
  return __builtin_bit_cast(uint32_t, h);
}

// Two bfloat16 values, rounded to nearest even by one instruction.
__device__ __forceinline__ uint32_t pack_bf16x2(float a, float b) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  const bf16x2 h = {(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, h);
}

// a * (half h of w) with the half widened by the instruction (v_fma_mix_f32).
__device__ __forceinline__ float mul_lo_half(float a, uint32_t w) { return __builtin_fmaf(a, lo_half(w), 0.0f); }
__device__ __forceinline__ float mul_hi_half(float a, uint32_t w) { return __builtin_fmaf(a, hi_half(w), 0.0f); }

__device__ __forceinline__ uint32_t max_half2(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(f16x2, a),
                                                                __builtin_bit_cast(f16x2, b)));
}

// Bytes b of x and y as the low bytes of the two halves of a word.
template <int B>
__device__ __forceinline__ uint32_t byte_pair(uint32_t x, uint32_t y) {
  return __builtin_amdgcn_perm(y, x, 0x0C000C00u | ((4u + B) << 16) | (uint32_t)B);
}
// byte_pair with the byte pair's selector in a register.
__device__ __forceinline__ uint32_t byte_pair(uint32_t x, uint32_t y, uint32_t sel) {
  return __builtin_amdgcn_perm(y, x, sel);
}

__device__ __forceinline__ uint32_t add_half2(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, a) + __builtin_bit_cast(f16x2, b));
}

// Power of two that brings a row's largest finite magnitude (fp32 bits of a
// non-negative value) into [2^14, 2^15): bfloat16 queries times it are fp16
// numbers, exactly, unless they are below 2^-31 of the largest.  At most 2^100,
// so that its inverse is normal.
__device__ __forceinline__ float half_range_factor(uint32_t max_bits) {
  const int e = (int)(max_bits >> 23);
  if (e == 0) return 1.0f;
  const int k = 268 - e;                             // biased exponent of 2^(14 - (e - 127))
  return __builtin_bit_cast(float, (uint32_t)(k > 227 ? 227 : k) << 23);
}
__device__ __forceinline__ uint32_t finite_magnitude(float x) {
  const uint32_t b = __builtin_bit_cast(uint32_t, x) & 0x7FFFFFFFu;
  return b < 0x7F800000u ? b : 0u;
}

// Largest finite magnitude of eight fp16 values, as fp32 bits.
__device__ __forceinline__ uint32_t half_magnitude8(u32x4 raw) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t r = raw[i];
    const uint32_t a = finite_magnitude(lo_half(r)), b = finite_magnitude(hi_half(r));
    m = m > a ? m : a;
    m = m > b ? m : b;
  }
  return m;
}

// Eight bfloat16 values as fp16 after multiplication by f.
__device__ __forceinline__ u32x4 bf16_to_half8(u32x4 raw, float f) {
  u32x4 out;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t r = raw[i];
    out[i] = pack_half2(__builtin_bit_cast(float, r << 16) * f,
                        __builtin_bit_cast(float, r & 0xFFFF0000u) * f);
  }
  return out;
}
__device__ __forceinline__ uint32_t bf16_magnitude8(u32x4 raw) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t r = raw[i];
    const uint32_t a = finite_magnitude(__builtin_bit_cast(float, r << 16));
    const uint32_t b = finite_magnitude(__builtin_bit_cast(float, r & 0xFFFF0000u));
    m = m > a ? m : a;
    m = m > b ? m : b;
  }
  return m;
}

// The logits' scale times log2(e) as the kernels use it: positive (a scale of 0
// as one too small to matter), so that -inf times it stays -inf.
__device__ __forceinline__ float positive_scale(float cs) { return cs > 0x1p-120f ? cs : 0x1p-120f; }

__device__ __forceinline__ float power_of_two(int e) { return __builtin_bit_cast(float, (uint32_t)(e + 127) << 23); }

// Logits so large that fp32 hardly holds their fractions (top: the row's largest,
// cs its factor).  Exponents of steps cannot then be added to them: weights are
// taken relative to the largest logit itself, and no logit may exceed it.
__device__ __forceinline__ bool past_fractions(float top, float cs) {
  return top != kNone && __builtin_fabsf(top * cs) >= 0x1p22f;
}
// (no row is past_fractions while this is false of its M, which is within 2^6 of
// top * cs until then)
__device__ __forceinline__ bool nearly_past(float M) { return M != kNone && __builtin_fabsf(M) >= 0x1p21f; }
// What a row's weights are relative to, 2^(hi + lo), exactly: rescaling and the
// joins of waves and parts shift sums by just the difference of their references,
// whatever the logits' size.  lo is 0 but for rows past_fractions of the decode
// kernel, whose top * cs is rounded.
struct Reference {
  float hi, lo;
};
__device__ __forceinline__ Reference reference(float top, float cs, float M) {
  return Reference{M, past_fractions(top, cs) ? __builtin_fmaf(top, cs, -M) : 0.0f};
}
// (lo is 0 below this)
__device__ __forceinline__ bool may_have_low_part(float hi) {
  return __builtin_fabsf(hi) >= 0x1p22f && hi != kNone;
}
__device__ __forceinline__ float exp2_difference(Reference a, Reference b) {
  return __builtin_amdgcn_exp2f((a.hi - b.hi) + (a.lo - b.lo));
}

// ln (2^reference * sum)
__device__ __forceinline__ float natural_log(float reference, float sum) {
  return (reference + __builtin_amdgcn_logf(sum)) * 0.69314718055994531f;
}

// What a workgroup knows about its request.
struct Request {
  int64_t token0;        // first query token
  int qn, ql;            // query tokens in all, and those served (at most max_q)
  int kv;                // tokens in the cache
};
__device__ __forceinline__ Request request_of(const KvAttn &p, int b) {
  Request r;
  if (p.query_start) {
    int64_t a = p.query_start[b], z = p.query_start[b + 1];
    a = a < 0 ? 0 : a > p.T ? p.T : a;
    z = z < a ? a : z > p.T ? p.T : z;
    r.token0 = a;
    r.qn = (int)(z - a);
  } else {
    r.token0 = b;
    r.qn = 1;
  }
  r.ql = r.qn < p.max_q ? r.qn : p.max_q;
  const int64_t cap = (int64_t)p.max_blocks << p.pshift;
  const int64_t n = p.seq_lens[b];
  r.kv = (int)(n < 0 ? 0 : n > cap ? cap : n);
  return r;
}
__device__ __forceinline__ int divide(int x, Divisor d) {
  return (int)(((uint64_t)(uint32_t)x * d.m) >> d.shift);
}
// Query token of row r.
__device__ __forceinline__ int token_of(const KvAttn &p, int r) { return divide(r, p.by_group); }

// Last key that query token qi sees, and the first (the window's start).
__device__ __forceinline__ int last_key(const KvAttn &p, const Request &r, int qi) {
  return p.causal ? r.kv - r.qn + qi : r.kv - 1;
}
__device__ __forceinline__ int first_key(const KvAttn &p, int last) {
  return p.window && last >= p.window ? last - p.window + 1 : 0;
}

// The keys of a tile of rows row0 .. row1, from `lo` (a multiple of `align`) to
// `end`, and how they are cut: into equal parts of `each` (a multiple of 64), as
// many as keep p.chunk keys each but at most p.splits.  Short requests of a
// batch thus take fewer parts, and a row with one part needs no join.
struct Keys {
  int lo, end, parts, each;
};
__device__ __forceinline__ Keys keys_of(const KvAttn &p, const Request &r, int row0, int row1, int align) {
  Keys k;
  k.lo = first_key(p, last_key(p, r, token_of(p, row0))) & -align;
  k.end = last_key(p, r, token_of(p, row1)) + 1;
  const int n = k.end > k.lo ? k.end - k.lo : 1;
  if (p.splits == 1) {                               // (no divisions on the way to the first load)
    k.each = (n + 63) & -64;
    k.parts = 1;
    return k;
  }
  const int most = (n - 1) / p.chunk + 1;
  const int want = most < p.splits ? most : p.splits;
  k.each = ((n - 1) / want + 64) & -64;
  k.parts = (n - 1) / k.each + 1;
  return k;
}

// ---- few query rows: the decode kernel ------------------------------------------------------
// Bound by reading the cache, D/2 bytes of key and of value codes and 4 to 6
// bytes of steps and zero points per token and key/value head, and close behind
// by the VALU that turns codes into operands.  A workgroup serves 16 query rows
// of one key/value head; each of its waves streams its own run of tokens, 32 at a
// time, straight from memory into MFMA operands (no LDS but for the queries, no
// barrier until the end), the next 32 in flight meanwhile.  The waves' results
// meet in LDS; with few requests the tokens are split over several workgroups as
// well, whose results a second kernel joins.
//
// The operands are the code nibbles as they lie in the cache, masked to subnormal
// fp16 numbers (code * 2^-24 or 2^-20), which the MFMA multiplies exactly: two
// operations per pair of codes fewer than exact integers code - zero.  The zero
// points come off the sums: sum q (code - z) = sum q code - z sum q, and for the
// values sum P' code - sum P' z, with the weights as they were rounded.
//
// Lane (c = l & 15, kq = l >> 4).  Per 16 tokens: one 16-byte load of key
// codes (D = 128: words 4kq.. of token c; 1 KiB per wave, one run), one of
// value codes (word c of tokens 4kq..4kq+3), one of their steps, and 8 bytes
// of zero points.  S^T comes out as keys 4kq + e of row c.
//
// Registers hold one tile: key codes are refilled with the next tile's as soon
// as they are used, steps and zero points after the softmax, value codes after
// their products, so a load has most of a tile's work to arrive in while four
// waves share a SIMD.  (48 requests of up to 4096 tokens, 32 heads of 128: two
// register sets, two waves per SIMD, measured 128 us where one set and three
// waves took 113; later three waves took 94 and four 90.)
//
// Measured there (429.6 MB): 88 us from an idle card, 4.9 TB/s of the 5.1 that a
// copy reaches, and 98 - 110 repeated back to back; the VALU is active 75% of the
// time, the MFMA 15%, and memory delivers 1.01 times the bytes.  Four requests of up
// to 65536 tokens, 64 heads over 8 (158.3 MB, symmetric): 28 us repeated, when the
// last-level cache holds part of it, about 35 from memory, and 4 for the join.  One
// request of 777 tokens, 32 heads over 8: 9.4 us in a graph, which is latency:
// lengths, table, codes, and the waves' join, one after the other.
template <int D>
struct DecodeTile {
  static constexpr int kWords = D / 32;              // key words per lane and token
  uint32_t k[2][kWords];
  u32x4 v[2];
  u32x4 sc[2];
  u32x2 z[2];
};
// Where a tile's halves lie, in bytes of codes and of zero points (steps take
// twice that); bit i of bad: half i has no page (it reads page 0's).
struct DecodeAt {
  int64_t code[2], meta[2];
  uint32_t bad;
};

template <int D, bool SYM, bool BF16, int NW>
__global__ __launch_bounds__(64 * NW) __attribute__((amdgpu_waves_per_eu(4, 4)))
void kv_decode_kernel(KvAttn p) {
  constexpr int kWords = D / 32, kTiles = D / 16;
  constexpr int kRow = D + 4;                        // floats per row in LDS
  __shared__ __attribute__((aligned(16))) float red[NW][16][kRow];
  __shared__ float red_m[NW][16], red_lo[NW][16], red_l[NW][16];
  __shared__ u32x4 sq[kWords][64];                   // the queries as MFMA operands, per lane
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c = lane & 15, kq = lane >> 4;
  const int row_tile = divide(blockIdx.x, p.by_heads);
  const int h = (int)blockIdx.x - row_tile * p.heads, row0 = row_tile * 16;
  const int split = blockIdx.y, b = blockIdx.z;
  const Request rq = request_of(p, b);
  const int rows = rq.ql * p.group;
  if (row0 >= rows) return;
  const int row_last = row0 + 15 < rows ? row0 + 15 : rows - 1;
  const int row = row0 + c < rows ? row0 + c : rows - 1;
  const int qi = token_of(p, row);
  const int32_t *table = p.table + (int64_t)b * p.max_blocks;
  int page_base = 0;
  int32_t page_ids = -1;                             // lane i: page page_base + i of the request
  auto load_pages = [&](int first) {
    page_base = first;
    const int at = first + lane;
    page_ids = at < p.max_blocks ? table[at] : -1;
  };
  // (the first pages and the queries do not wait for the request's length, which
  // the rest depends on)
  load_pages(0);
  // queries: lane (c, kq) holds channels 32kq.. (D = 128) or 16kq.. (D = 64)
  // of row c, the channels of the key words that it will load
  const uint16_t *qp = p.Q + (rq.token0 + qi) * p.q_stride +
                       (int64_t)(h * p.group + row - qi * p.group) * D + kq * (8 * kWords);
  u32x4 q[kWords];
#pragma unroll
  for (int j = 0; j < kWords; ++j) q[j] = *reinterpret_cast<const u32x4 *>(qp + 8 * j);
  const int my_last = last_key(p, rq, qi), my_first = first_key(p, my_last);
  // keys that all rows see
  const int all_last = last_key(p, rq, token_of(p, row0));
  const int all_first = first_key(p, last_key(p, rq, token_of(p, row_last)));
  const Keys keys = keys_of(p, rq, row0, row_last, 32);
  if (split >= keys.parts) return;
  const int t_lo = keys.lo + split * keys.each;
  const int t_hi = split + 1 < keys.parts ? t_lo + keys.each : keys.end;
  const int nt = t_hi > t_lo ? (t_hi - t_lo + 31) / 32 : 0;
  const int i0 = nt * wave / NW, i1 = nt * (wave + 1) / NW;

  // The key operand is the nibble pair as it lies in the word, a subnormal fp16:
  // code * 2^-24 for channels 0, 1, 4, 5 of a word, 16 times that for the others
  // (the MFMA takes subnormals exactly).  The queries make up for it: each row's
  // scaled by a power of two into [2^14, 2^15) at most, those of the other channels
  // by a sixteenth of it.  (Values below 2^-24 of the row's largest lose bits.)
  uint32_t qmax = 0;
#pragma unroll
  for (int j = 0; j < kWords; ++j) {
    const uint32_t x = BF16 ? bf16_magnitude8(q[j]) : half_magnitude8(q[j]);
    qmax = qmax > x ? qmax : x;
  }
#pragma unroll
  for (int d = 32; d > 8; d >>= 1) {                 // (the row's lanes)
    const uint32_t x = (uint32_t)__shfl_xor((int)qmax, d, 64);
    qmax = qmax > x ? qmax : x;
  }
  const float f = half_range_factor(qmax);
  // (negated for a negative scale, so that larger sums are larger logits)
  const float fs = p.scale_log2 < 0.0f ? -f : f;
  const float abs_scale = __builtin_fabsf(p.scale_log2);
  // (bfloat16 queries near the end of their range, where this factor or its inverse
  // would pass fp32's: the sums then take 2^60 of it, in all rows alike)
  const bool wide = __any(abs_scale * (1.0f / f) * 0x1p24f > 0x1p100f);
  const float cs = positive_scale(wide ? abs_scale * 0x1p-36f * (1.0f / f) : abs_scale * (1.0f / f) * 0x1p24f);
  // sum of the row's queries, for the zero points: sum q (code - z) = sum q code - z sum q
  float qsum = 0.0f;
#pragma unroll
  for (int j = 0; j < kWords; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w = q[j][i];
      const float g = i & 1 ? fs * 0x1p-4f : fs;
      const uint32_t x = BF16 ? pack_half2(__builtin_bit_cast(float, w << 16) * g,
                                           __builtin_bit_cast(float, w & 0xFFFF0000u) * g)
                              : pack_half2(lo_half(w) * g, hi_half(w) * g);
      q[j][i] = x;
      qsum += (lo_half(x) + hi_half(x)) * (i & 1 ? 0x1p-20f : 0x1p-24f);
    }
  qsum += __shfl_xor(qsum, 16, 64);
  qsum += __shfl_xor(qsum, 32, 64);
  // (every wave has the same 16 rows; in registers they would cost the loop 16
  // of them, and with those a wave per SIMD)
  if (wave == 0) {
#pragma unroll
    for (int j = 0; j < kWords; ++j) sq[j][lane] = q[j];
  }

  const int pmask = (1 << p.pshift) - 1;
  // A load's address is a uniform base (the tile's place) plus the lane's byte
  // offset within 16 tokens' key words, value words, and steps (zero points:
  // half of that).
  const uint32_t k_lane = D == 128 ? c * 64 + kq * 16 : c * 32 + kq * 8;
  const uint32_t v_lane = kq * (2 * D) + (c & (D / 8 - 1)) * 16, s_lane = kq * 16;
  const int64_t P = (int64_t)pmask + 1;
  const int64_t code_stride = (int64_t)p.heads * P * D, meta_stride = (int64_t)p.heads * P * 2;
  const int64_t v_offset = code_stride / 2;
  const char *codes = reinterpret_cast<const char *>(p.codes) + h * P * (D / 2);
  const char *scales = reinterpret_cast<const char *>(p.scales) + h * P * 4;
  const char *zeros = reinterpret_cast<const char *>(p.zeros) + h * P * 2;
  const int pages = p.pages < 0x7FFFFFFF ? (int)p.pages : 0x7FFFFFFF;
  auto place = [&](int t) {
    DecodeAt at;
    at.bad = 0;
    // the pages of both halves lie within 64 of page_base, or are fetched
    if (((t + 31) >> p.pshift) - page_base > 63) load_pages(t >> p.pshift);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int tt = t + 16 * i;
      int id = __builtin_amdgcn_readlane(page_ids, (tt >> p.pshift) - page_base);
      if ((uint32_t)id >= (uint32_t)pages) {
        at.bad |= 1u << i;
        id = 0;
      }
      at.code[i] = id * code_stride + (tt & pmask) * (D / 2);
      at.meta[i] = id * meta_stride + (tt & pmask) * 2;
    }
    return at;
  };
  DecodeTile<D> T;
  auto load_keys = [&](const DecodeAt &at) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const char *src = codes + at.code[i];
      if constexpr (D == 128) {
        const u32x4 w = *reinterpret_cast<const u32x4 *>(src + k_lane);
#pragma unroll
        for (int j = 0; j < 4; ++j) T.k[i][j] = w[j];
      } else {
        const u32x2 w = *reinterpret_cast<const u32x2 *>(src + k_lane);
#pragma unroll
        for (int j = 0; j < 2; ++j) T.k[i][j] = w[j];
      }
    }
  };
  auto load_meta = [&](const DecodeAt &at) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const char *src = scales + 2 * at.meta[i];
      T.sc[i] = *reinterpret_cast<const u32x4 *>(src + s_lane);
      if constexpr (!SYM) {
        const char *zsrc = zeros + at.meta[i];
        T.z[i] = *reinterpret_cast<const u32x2 *>(zsrc + s_lane / 2);
      }
    }
  };
  auto load_values = [&](const DecodeAt &at) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const char *src = codes + (at.code[i] + v_offset);
      T.v[i] = *reinterpret_cast<const u32x4 *>(src + v_lane);
    }
  };

  f32x4 o[kTiles];
#pragma unroll
  for (int n = 0; n < kTiles; ++n) o[n] = f32x4{0.f, 0.f, 0.f, 0.f};
  // top: the largest sum so far (times the key's step), the row's for a row
  // past_fractions, whose M is top * cs; vlim: above the steps that slack allows for
  float M = kNone, top = kNone, slack = kNone, vlim = 0.0f, l = 0.0f, pz = 0.0f;
  const float inv_cs = 1.0f / cs;
  bool any_past = false;                             // a row of the wave is past_fractions (uniform)
  // The nibble pairs of word w (of shifted words, the next two): subnormal fp16
  constexpr uint32_t kLoNibbles = 0x000F000Fu, kHiNibbles = 0x00F000F0u;
  // D = 64 has 8 words per token but an MFMA operand 16 rows: lanes c and
  // c + 8 take the same word, the first its even channels (bytes 0, 1), the
  // second its odd ones (bytes 2, 3)
  const uint32_t sel0 = D == 128 ? 0u : (c < 8 ? 0x0C040C00u : 0x0C060C02u);
  const uint32_t sel1 = D == 128 ? 0u : (c < 8 ? 0x0C050C01u : 0x0C070C03u);

  // One tile of 32 tokens at t (in T, placed at `at`); `next`: the tile to refill T with.
  auto tile = [&](int t, const DecodeAt &at, const DecodeAt &next, auto more_tag) {
    constexpr bool kMore = decltype(more_tag)::value;
    f32x4 s[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float s0 = SYM ? -8.0f * qsum : 0.0f;    // without zeros every zero is 8
      s[i] = f32x4{s0, s0, s0, s0};
#pragma unroll
      for (int j = 0; j < kWords; ++j) {
        const uint32_t w = T.k[i][j], w8 = w >> 8;
        s[i] = mfma32<TagF16>(u32x4{w & kLoNibbles, w & kHiNibbles, w8 & kLoNibbles, w8 & kHiNibbles},
                              sq[j][lane], s[i]);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    if constexpr (kMore) {
      __builtin_amdgcn_sched_barrier(0);
      load_keys(next);
      __builtin_amdgcn_sched_barrier(0);
    }
    float u[8];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t w = T.sc[i][e];
        float x = s[i][e];
        if constexpr (!SYM) {
          const uint32_t zz = T.z[i][e >> 1];
          x = __builtin_fmaf(-(float)((zz >> (16 * (e & 1))) & 0xFFu), qsum, x);
        }
        u[4 * i + e] = mul_lo_half(x, w);
      }
    if (wide) {
#pragma unroll
      for (int i = 0; i < 8; ++i) u[i] *= 0x1p60f;
    }
    if (at.bad || t < all_first || t + 31 > all_last) {
      // key first <= e <= last, as one unsigned comparison of (e - first).  (The three
      // conditions joined by && became branches per lane for one element, and with
      // them the compiler has lost that element's -inf.)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const bool any = (my_first <= my_last) & (((at.bad >> i) & 1u) == 0u);
        const uint32_t first = any ? my_first - t - 16 * i - 4 * kq : 0x40000000, span = any ? my_last - my_first : 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const bool seen = e - first <= span;
          u[4 * i + e] = seen ? u[4 * i + e] : -__builtin_inff();
          T.sc[i][e] = seen ? T.sc[i][e] : 0u;
        }
      }
    }
    float umax = u[0];
    uint32_t smax = T.sc[0][0];
#pragma unroll
    for (int i = 1; i < 8; ++i) {
      const uint32_t w = T.sc[i >> 2][i & 3];
      umax = fmaxf(umax, u[i]);
      smax = max_half2(smax, w);
    }
    if (__any(umax > slack || hi_half(smax) > vlim)) {
      // the row's largest weight times step, steps by their exponent field alone
      // (hidden keys have u = -inf), and no less than it: the largest of each
      float best = kNone, most = __builtin_fmaf(umax, cs, (float)((smax >> 26) & 31u));
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t w = T.sc[i >> 2][i & 3];
        best = fmaxf(best, __builtin_fmaf(u[i], cs, (float)((w >> 26) & 31u)));
      }
#pragma unroll
      for (int d = 16; d <= 32; d <<= 1) {
        best = fmaxf(best, __shfl_xor(best, d, 64));
        most = fmaxf(most, __shfl_xor(most, d, 64));
      }
      // twice the largest step of this lane's keys, about that of the others too
      const float m_before = M, vexp = (float)((smax >> 26) & 31u) - 13.0f;
      M = fmaxf(M, fminf(most, best + (kSpread - 1)) - (14.0f + kRaise));
      vlim = power_of_two((int)vexp);
      float a = __builtin_amdgcn_exp2f(m_before - M);
      slack = M == kNone ? kNone : (M + (kLimit - vexp)) * inv_cs;
      float top_before = top;
      top = fmaxf(top, umax);                        // (of this lane's keys, until it matters)
      if (__builtin_expect(any_past | (bool)__any(nearly_past(M)), 0)) {
#pragma unroll
        for (int d = 16; d <= 32; d <<= 1) {
          top_before = fmaxf(top_before, __shfl_xor(top_before, d, 64));
          top = fmaxf(top, __shfl_xor(top, d, 64));
        }
        const bool past = past_fractions(top, cs);
        M = past ? top * cs : M;
        slack = past ? top : slack;
        a = exp2_difference(reference(top_before, cs, m_before), reference(top, cs, M));
        any_past = __any(past);
      }
      l *= a;
      pz *= a;
#pragma unroll
      for (int n = 0; n < kTiles; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[n][e] *= a;
    }
    float ref = M;
    if (any_past) {
      const bool past = past_fractions(top, cs);
#pragma unroll
      for (int i = 0; i < 8; ++i) u[i] -= past ? top : 0.0f;
      ref = past ? 0.0f : M;
    }
    u32x4 pb;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float pr[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float x = __builtin_amdgcn_exp2f(__builtin_fmaf(u[4 * i + e], cs, -ref));
        l += x;
        const uint32_t w = T.sc[i][e];
        pr[e] = mul_hi_half(x, w);
      }
      pb[2 * i] = pack_half2(pr[0], pr[1]);
      pb[2 * i + 1] = pack_half2(pr[2], pr[3]);
      // the zero points' share, sum P' z, with the weights as they are rounded:
      // sum P' code - sum P' z then has the rounding of sum P' (code - z)
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const uint32_t w = pb[2 * i + g];
        if constexpr (SYM) {
          pz = __builtin_amdgcn_fdot2(__builtin_bit_cast(f16x2, w), f16x2{(_Float16)8.0f, (_Float16)8.0f}, pz, false);
        } else {
          const uint32_t zz = T.z[i][g];
          pz = __builtin_fmaf(lo_half(w), (float)((zz >> 8) & 0xFFu), pz);
          pz = __builtin_fmaf(hi_half(w), (float)(zz >> 24), pz);
        }
      }
    }
    if constexpr (kMore) {
      __builtin_amdgcn_sched_barrier(0);
      load_meta(next);
      __builtin_amdgcn_sched_barrier(0);
    }
    // value operands: byte b of the words of tokens (2j, 2j+1) in the halves
    // of a word, then each nibble, again as subnormals
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) w[4 * i + e] = T.v[i][e];
    auto product = [&](auto byte_of, int n) {
      u32x4 lo, hi;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t x = byte_of(w[2 * j], w[2 * j + 1]);
        lo[j] = x & kLoNibbles;
        hi[j] = x & kHiNibbles;
      }
      o[n] = mfma32<TagF16>(lo, pb, o[n]);
      o[n + 1] = mfma32<TagF16>(hi, pb, o[n + 1]);
      __builtin_amdgcn_sched_barrier(0);             // (bounds the registers in use)
    };
    if constexpr (D == 128) {
      product([](uint32_t x, uint32_t y) { return byte_pair<0>(x, y); }, 0);
      product([](uint32_t x, uint32_t y) { return byte_pair<1>(x, y); }, 2);
      product([](uint32_t x, uint32_t y) { return byte_pair<2>(x, y); }, 4);
      product([](uint32_t x, uint32_t y) { return byte_pair<3>(x, y); }, 6);
    } else {
      product([&](uint32_t x, uint32_t y) { return byte_pair(x, y, sel0); }, 0);
      product([&](uint32_t x, uint32_t y) { return byte_pair(x, y, sel1); }, 2);
    }
    if constexpr (kMore) {
      __builtin_amdgcn_sched_barrier(0);
      load_values(next);
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  __syncthreads();
  if (i0 < i1) {
    int t = t_lo + 32 * i0;
    DecodeAt at = place(t);
    load_keys(at);
    load_meta(at);
    load_values(at);
    for (int i = i0; i + 1 < i1; ++i, t += 32) {
      const DecodeAt next = place(t + 32);
      tile(t, at, next, std::true_type{});
      at = next;
    }
    tile(t, at, at, std::false_type{});
  }

  // ---- join the waves --------------------------------------------------------------
  l += __shfl_xor(l, 16, 64);
  l += __shfl_xor(l, 32, 64);
  pz += __shfl_xor(pz, 16, 64);
  pz += __shfl_xor(pz, 32, 64);
  // channel of MFMA tile n, result row 4kq + e (see the operand layouts above)
  constexpr int kOrder[8] = {0, 2, 4, 6, 1, 3, 5, 7};
#pragma unroll
  for (int n = 0; n < kTiles; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int r = 4 * kq + e;
      const int d = D == 128 ? 8 * r + kOrder[n] : 8 * (r & 7) + 2 * n + (r >> 3);
      red[wave][c][d] = o[n][e] * (n & 1 ? 0x1p20f : 0x1p24f) - pz;
    }
  if (kq == 0) {
    red_m[wave][c] = M;
    red_lo[wave][c] = any_past ? reference(top, cs, M).lo : 0.0f;
    red_l[wave][c] = l;
  }
  __syncthreads();
  constexpr int kPer = D / (4 * NW);                 // channels per thread
  const int r = tid / (4 * NW), d0 = (tid % (4 * NW)) * kPer;
  if (row0 + r >= rows) return;
  Reference m = {red_m[0][r], 0.0f};
#pragma unroll
  for (int w = 1; w < NW; ++w) m.hi = fmaxf(m.hi, red_m[w][r]);
  const bool large = may_have_low_part(m.hi);
  if (__builtin_expect(large, 0)) {
    m.lo = kNone;
    for (int w = 0; w < NW; ++w) m.lo = red_m[w][r] == m.hi ? fmaxf(m.lo, red_lo[w][r]) : m.lo;
  }
  float sum = 0.0f, acc[kPer] = {};
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    float e = red_m[w][r] - m.hi;
    if (__builtin_expect(large, 0)) e += red_lo[w][r] - m.lo;
    const float a = __builtin_amdgcn_exp2f(e);
    sum = __builtin_fmaf(red_l[w][r], a, sum);
#pragma unroll
    for (int i = 0; i < kPer; ++i) acc[i] = __builtin_fmaf(red[w][r][d0 + i], a, acc[i]);
  }
  const bool none = sum == 0.0f;                     // the row sees no key
  const float inv = none ? 0.0f : 1.0f / sum;
  const int rr = row0 + r;
  const int rqi = token_of(p, rr);
  const int64_t head_row = (rq.token0 + rqi) * ((int64_t)p.heads * p.group) + h * p.group + rr - rqi * p.group;
  if (keys.parts > 1) {
    const int64_t at = split * p.T * p.heads * p.group + head_row;
    float *po = p.part_o + at * D + d0;
    if (!none) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) po[i] = acc[i] * inv;
    }
    if (d0 == 0) {
      p.part_sum[at] = float2{m.hi, sum};
      if (__builtin_expect(large, 0)) p.part_lo[at] = m.lo;
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const float v = none ? 0.0f : acc[i] * inv;
    if constexpr (BF16) reinterpret_cast<uint16_t *>(p.O)[head_row * D + d0 + i] = float_to_bf16_bits(v);
    else reinterpret_cast<uint16_t *>(p.O)[head_row * D + d0 + i] = float_to_half_bits(v);
  }
  if (p.lse && d0 == 0) p.lse[head_row] = none ? -__builtin_inff() : natural_log(m.hi, sum);
}

// ---- many query rows: the prompt kernel --------------------------------------------------------
// Bound by the VALU next to the matrix products: per row and key the softmax
// takes seven operations (one an exp2 at a quarter of the rate) and turning codes
// into operands three more.  A workgroup serves 128 rows (four waves of 32) of one
// key/value head and walks its keys 64 at a time.  Turning codes into fp16
// integers costs as much VALU work per wave as the softmax of 32 rows, so it
// is done once per workgroup: each thread turns 16 bytes of key and of value
// codes into LDS, one tile ahead of the products, which read them as MFMA
// operands.  32x32x16 MFMA, transposed as described above: lane (q = l & 31,
// hh = l >> 5) holds keys 8g + 4hh + e of row q.
//
// A workgroup's waves stage 16 tokens each, so a page lookup is one per wave.
//
// Measured: a prompt of 8192 tokens, 32 heads over 8, D = 128, bfloat16 (550
// Gflop causal): 705 - 735 us, 750 - 780 Tflop/s, at 1.92 - 1.95 GHz.  The VALU is
// active 58% of the time, the MFMA 38% and the LDS 49% (a fifth of that conflicts):
// 96% of VALU and MFMA together, so on a SIMD the two take turns nearly all the
// time although the units can run side by side (an MFMA with seven independent VALU
// operations after it takes 20.4 ns where the two alone take 16.0 and 7.9).  With
// D = 64 three waves fit a SIMD: 507 and 530 us (two waves 531 and 572).
//
// With NG = 2 a workgroup has two groups of four waves that walk alternate tiles
// of the same rows, each with buffers of its own, and the second group's sums join
// the first's through LDS: half the steps for a request, at one workgroup per CU.
// Six ragged requests of up to 515 new tokens after up to 3000, window 1000, 16
// heads over 4, D = 64: 31.5 us, where one group took 37 (a set of shorter lengths:
// 25.8 and 39.8).
//
// Slower on the long prompt: eight waves and 256 rows (993 us when this took 834),
// a pipeline of half tiles (1376), the running maximum from a bound in LDS (1115),
// 64 rows per wave at one wave per SIMD (the accumulators travel between register
// files at every branch; D = 64: 1102 us for 616), the staging between the MFMAs
// instead of after them (760 for 721).
constexpr int kPtKeys = 64, kPtRows = 128, kPtThreads = 256;

// LDS rows end in 16 spare bytes, which puts the 16 rows of an operand read on
// distinct banks with the operand's place in the row as the instruction's
// offset (an XOR swizzle needs a register per place).
template <int D>
struct PromptSmem {
  static constexpr int kKeyRow = 2 * D + 16, kValueRow = 2 * kPtKeys + 16;   // bytes
  char k[2][kPtKeys * kKeyRow];
  char v[2][D * kValueRow];      // row ch * D/8 + word: channel 8 word + ch
  float ks[2][kPtKeys];          // key step * step_scale
  float vs[2][kPtKeys];          // value step; 0 past the last token, -0 where a page is missing
};

template <int D, bool SYM, bool BF16, int NG>
__global__ __launch_bounds__(kPtThreads *NG, D == 64 && NG == 1 ? 3 : 2) void kv_prompt_kernel(KvAttn p) {
  constexpr int kRows = kPtRows;
  using Smem = PromptSmem<D>;
  constexpr int kSteps = D / 16, kTiles = D / 32;
  __shared__ __attribute__((aligned(16))) Smem sms[NG];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane((tid >> 6) & 3);
  const int grp = NG == 1 ? 0 : __builtin_amdgcn_readfirstlane(tid >> 8);
  Smem &sm = sms[grp];
  const int qc = lane & 31, hh = lane >> 5;
  const int tile = (int)gridDim.x - 1 - (int)blockIdx.x;     // longest rows first
  const int split = divide(blockIdx.y, p.by_heads), h = (int)blockIdx.y - split * p.heads, b = blockIdx.z;
  const Request rq = request_of(p, b);
  const int rows = rq.ql * p.group, row0 = tile * kRows;
  if (row0 >= rows) return;
  auto clamp_row = [&](int r) { return r < rows ? r : rows - 1; };
  const int wrow0 = clamp_row(row0 + wave * 32), wrow1 = clamp_row(row0 + wave * 32 + 31);
  const int row = clamp_row(row0 + wave * 32 + qc);
  const bool wave_live = row0 + wave * 32 < rows;
  const int qi = token_of(p, row);
  const int my_last = last_key(p, rq, qi), my_first = first_key(p, my_last);
  const int w_any_last = last_key(p, rq, token_of(p, wrow1));
  const int w_all_last = last_key(p, rq, token_of(p, wrow0));
  const int w_any_first = first_key(p, w_all_last), w_all_first = first_key(p, w_any_last);
  const Keys keys = keys_of(p, rq, row0, clamp_row(row0 + kRows - 1), kPtKeys);
  if (split >= keys.parts) return;
  const int t_lo = keys.lo + split * keys.each;
  const int t_hi = split + 1 < keys.parts ? t_lo + keys.each : keys.end;
  const int nt = t_hi > t_lo ? (t_hi - t_lo + kPtKeys - 1) / kPtKeys : 0;

  // ---- staging: codes of one tile to registers, then as integers to LDS.  The
  // pieces are dealt out by groups of 16 tokens, which lie in one page, one group
  // to a wave: a lane takes a quarter of a key's words, and one value word of four
  // tokens (D = 128) or of two (D = 64).
  constexpr int kKw = D / 32, kVt = D / 32;                  // key words; tokens of the value word
  const int kkey = 16 * wave + (lane >> 2), kquad = lane & 3;
  const int vblk = 4 * wave + (lane >> 4), vword = D == 128 ? lane & 15 : (lane & 15) >> 1;
  const int vpair = D == 128 ? 0 : lane & 1;
  const int pmask = (1 << p.pshift) - 1;
  const int64_t P = (int64_t)pmask + 1;
  const int64_t code_stride = (int64_t)p.heads * P * D, meta_stride = (int64_t)p.heads * P * 2;
  const char *codes = reinterpret_cast<const char *>(p.codes) + h * P * (D / 2);
  const char *scales = reinterpret_cast<const char *>(p.scales) + h * P * 4;
  const char *zeros = reinterpret_cast<const char *>(p.zeros) + h * P * 2;
  const int pages = p.pages < 0x7FFFFFFF ? (int)p.pages : 0x7FFFFFFF;
  const int32_t *table = p.table + (int64_t)b * p.max_blocks;
  int page_id = -1;                                          // of the tile to load next (uniform)
  int page_left = 0;                                         // its tokens of this wave's group
  uint32_t kc[kKw], vc[kVt];
  uint32_t ksc = 0, kzz = 0x0808u, vzz[kVt / 2];
  int left = 0;                                              // tokens of the loaded group
  bool hole = false;                                         // ... which should be there, but have no page
  // (past the last key there is no page: page 0 is read and counts for nothing)
  auto load_page = [&](int t0) {
    const int t = t0 + 16 * wave;
    page_id = t < rq.kv ? table[t >> p.pshift] : -1;
    page_left = rq.kv - t;
  };
  auto load_codes = [&](int t0) {
    int id = __builtin_amdgcn_readfirstlane(page_id);
    const bool none = (uint32_t)id >= (uint32_t)pages;
    left = none ? 0 : page_left;
    hole = none && page_left > 0;
    if (none) id = 0;
    const int off = (t0 + 16 * wave) & pmask;
    const char *kp = codes + (id * code_stride + off * (D / 2));
    const char *vp = kp + code_stride / 2;
    const char *sp = scales + (id * meta_stride + off * 2) * 2;
    const char *zp = zeros + (id * meta_stride + off * 2);
    using Piece = std::conditional_t<D == 128, u32x4, u32x2>;
    const Piece kw = *reinterpret_cast<const Piece *>(kp + lane * (4 * kKw));
    const Piece vw = *reinterpret_cast<const Piece *>(vp + lane * (4 * kVt));
#pragma unroll
    for (int j = 0; j < kKw; ++j) kc[j] = kw[j];
#pragma unroll
    for (int j = 0; j < kVt; ++j) vc[j] = vw[j];
    ksc = *reinterpret_cast<const uint32_t *>(sp + (lane >> 2) * 4);
    if constexpr (!SYM) {
      kzz = *reinterpret_cast<const uint16_t *>(zp + (lane >> 2) * 2);
#pragma unroll
      for (int j = 0; j < kVt / 2; ++j)
        vzz[j] = *reinterpret_cast<const uint32_t *>(zp + (lane >> 4) * 8 + vpair * 4 + 4 * j);
    } else {
#pragma unroll
      for (int j = 0; j < kVt / 2; ++j) vzz[j] = 0x08080808u;
    }
  };
  const DeqRegs dq;
  // scale * log2(e) = step_scale * row_scale: the mantissa goes into the key steps
  // in LDS, the power of two (and the inverse of the row's factor) into the exponent;
  // of a scale above 1, up to 2^60 into the steps too, so that the rest times the
  // inverse factor (at most 2^113) is a number
  const uint32_t scale_bits = __builtin_bit_cast(uint32_t, __builtin_fabsf(p.scale_log2));
  const int above = (int)(scale_bits >> 23) - 127;
  const uint32_t kept = (uint32_t)(above < 0 ? 0 : above > 60 ? 60 : above) << 23;
  const float step_scale = __builtin_bit_cast(float, (scale_bits & 0x007FFFFFu) | (0x3F800000u + kept));
  const float row_scale = __builtin_bit_cast(float, (scale_bits & 0x7F800000u) - kept);
  auto stage_keys = [&](int buf) {
    const DeqF16 deq(kzz & 0xFFu);
#pragma unroll
    for (int j = 0; j < kKw; ++j)
      *reinterpret_cast<u32x4 *>(sm.k[buf] + kkey * Smem::kKeyRow + (kquad * kKw + j) * 16) = deq(kc[j], dq);
    // (the key's four lanes store the same)
    const bool held = (lane >> 2) < left;
    const float vstep = hi_half(ksc);
    sm.ks[buf][kkey] = held ? lo_half(ksc) * step_scale : 0.0f;
    // (an infinite or NaN step as a finite one too large for fp16, so that the
    // zero weight of a row that does not see the key stays zero; steps of written
    // slots are positive)
    sm.vs[buf][kkey] = held ? fmaxf(fminf(vstep, 0x1p127f), 0.0f) : hole ? -0.0f : 0.0f;
  };
  auto stage_values = [&](int buf) {
    // word vword of kVt tokens: channel d's codes side by side
    uint32_t a[kVt / 2], b[kVt / 2];
#pragma unroll
    for (int j = 0; j < kVt / 2; ++j) {
      const uint32_t z = (vzz[j] >> 8) & 0x00FF00FFu;        // value zero points of two tokens
      a[j] = z | 0xE400E400u;
      b[j] = (z << 4) | 0xD400D400u;
    }
    // tokens 16s + 8x + 4y + e sit at position 16s + 8y + 4x + e of the row
    const int chunk = (vblk >> 2) * 2 + (vblk & 1), half = (vblk >> 1) & 1;
    char *row = sm.v[buf] + vword * Smem::kValueRow + chunk * 16 + 8 * half + 4 * vpair;
    auto bytes = [&](auto tag, int lo_ch, int hi_ch) {
      constexpr int kB = decltype(tag)::value;
      uint32_t lo[kVt / 2], hi[kVt / 2];
#pragma unroll
      for (int j = 0; j < kVt / 2; ++j) {
        const uint32_t x = byte_pair<kB>(vc[2 * j], vc[2 * j + 1]);
        lo[j] = add_half2((x & dq.lo) | dq.e1024, a[j]);
        hi[j] = add_half2((x & dq.hi) | dq.e64, b[j]);
      }
      char *lp = row + lo_ch * (D / 8) * Smem::kValueRow, *hp = row + hi_ch * (D / 8) * Smem::kValueRow;
      if constexpr (D == 128) {
        *reinterpret_cast<u32x2 *>(lp) = u32x2{lo[0], lo[1]};
        *reinterpret_cast<u32x2 *>(hp) = u32x2{hi[0], hi[1]};
      } else {
        *reinterpret_cast<uint32_t *>(lp) = lo[0];
        *reinterpret_cast<uint32_t *>(hp) = hi[0];
      }
    };
    bytes(std::integral_constant<int, 0>{}, 0, 2);
    bytes(std::integral_constant<int, 1>{}, 4, 6);
    bytes(std::integral_constant<int, 2>{}, 1, 3);
    bytes(std::integral_constant<int, 3>{}, 5, 7);
  };

  // ---- queries, and the power of two of their logits in the exponent
  float cs = row_scale;
  const uint16_t *qp = p.Q + (rq.token0 + qi) * p.q_stride +
                       (int64_t)(h * p.group + row - qi * p.group) * D + 8 * hh;
  u32x4 q[kSteps];
#pragma unroll
  for (int s = 0; s < kSteps; ++s) q[s] = *reinterpret_cast<const u32x4 *>(qp + 16 * s);
  if constexpr (BF16) {
    uint32_t m = 0;                                          // the row's largest
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const uint32_t x = bf16_magnitude8(q[s]);
      m = m > x ? m : x;
    }
    const uint32_t x = (uint32_t)__shfl_xor((int)m, 32, 64);
    m = m > x ? m : x;
    const float f = half_range_factor(m);
#pragma unroll
    for (int s = 0; s < kSteps; ++s) q[s] = bf16_to_half8(q[s], f);
    cs *= 1.0f / f;
  }
  cs = positive_scale(cs);
  if (p.scale_log2 < 0.0f) {
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
#pragma unroll
      for (int i = 0; i < 4; ++i) q[s][i] ^= 0x80008000u;
  }

  f32x16 o[kTiles];
#pragma unroll
  for (int n = 0; n < kTiles; ++n)
#pragma unroll
    for (int e = 0; e < 16; ++e) o[n][e] = 0.0f;
  float M = kNone, top = kNone, slack = kNone, l = 0.0f;
  float vlim = 0.0f;                                         // above the steps that slack allows for (uniform)

  // The order of a tile's instructions is spelled out for the scheduler: left
  // to itself it keeps one operand register and waits out the LDS latency
  // before every MFMA (measured 915 us where this order took 834, on 8192 tokens of 32 heads over 8,
  // D = 128).
  constexpr int kMfma = 0x008, kValu = 0x002, kLdsRead = 0x100;
  auto compute = [&](int buf, int t0) {
    const char *kl = sm.k[buf] + qc * Smem::kKeyRow + 16 * hh;
    const char *vl = sm.v[buf] + qc * Smem::kValueRow + 16 * hh;
    // the four keys 32i + 8g + 4hh + e of result group g
    auto per_key = [&](const float *x, int i, int g) {
      return *reinterpret_cast<const f32x4 *>(x + 32 * i + 8 * g + 4 * hh);
    };
    auto key_frag = [&](int i, int st) {
      return *reinterpret_cast<const u32x4 *>(kl + 32 * i * Smem::kKeyRow + 32 * st);
    };
    auto value_frag = [&](int s, int n) {
      return *reinterpret_cast<const u32x4 *>(vl + 32 * n * Smem::kValueRow + 32 * s);
    };
    const float vstep = sm.vs[buf][lane];                    // (of the tile's key `lane`)
    f32x16 s[2];
    u32x4 kf[kSteps];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int e = 0; e < 16; ++e) s[i][e] = 0.0f;
#pragma unroll
    for (int st = 0; st < kSteps; ++st) kf[st] = key_frag(0, st);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int st = 0; st < kSteps; ++st) {
      s[0] = mfma32x16(kf[st], q[st], s[0]);
      kf[st] = key_frag(1, st);
    }
#pragma unroll
    for (int st = 0; st < kSteps; ++st) {
      __builtin_amdgcn_sched_group_barrier(kMfma, 1, 0);
      __builtin_amdgcn_sched_group_barrier(kLdsRead, 1, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
    float u[32];
    auto scaled = [&](int i) {
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const f32x4 a = per_key(sm.ks[buf], i, g);
#pragma unroll
        for (int e = 0; e < 4; ++e) u[16 * i + 4 * g + e] = s[i][4 * g + e] * a[e];
      }
    };
#pragma unroll
    for (int st = 0; st < kSteps; ++st) s[1] = mfma32x16(kf[st], q[st], s[1]);
    scaled(0);
    __builtin_amdgcn_sched_group_barrier(kLdsRead, 4, 0);
#pragma unroll
    for (int st = 0; st < kSteps; ++st) {
      __builtin_amdgcn_sched_group_barrier(kMfma, 1, 0);
      __builtin_amdgcn_sched_group_barrier(kValu, 16 / kSteps, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
    u32x4 vf[2][kTiles];
#pragma unroll
    for (int n = 0; n < kTiles; ++n) vf[0][n] = value_frag(0, n);
    scaled(1);
    const bool holes = __any(__builtin_bit_cast(uint32_t, vstep) == 0x80000000u);
    const bool partial = t0 < w_all_first || t0 + kPtKeys - 1 > w_all_last || holes;
    if (partial) {
      // key first <= at <= last, as one unsigned comparison of (at - first)
      const bool any = my_first <= my_last;
      const uint32_t first = any ? my_first - t0 - 4 * hh : 0x40000000, span = any ? my_last - my_first : 0;
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          u[4 * j + e] = 8 * j + e - first <= span ? u[4 * j + e] : -__builtin_inff();
      if (holes) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const f32x4 v = per_key(sm.vs[buf], j >> 2, j & 3);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float ve = v[e];
            u[4 * j + e] = __builtin_bit_cast(uint32_t, ve) == 0x80000000u ? -__builtin_inff() : u[4 * j + e];
          }
        }
      }
    }
    float umax = u[0];
#pragma unroll
    for (int j = 1; j < 32; ++j) umax = fmaxf(umax, u[j]);
    if (__any(umax > slack || vstep > vlim)) {
      // the least power of two (from kLeastStep on) that no step of the tile exceeds
      int ve = -14;
#pragma unroll
      for (int bit = 16; bit > 0; bit >>= 1) ve += __any(vstep > power_of_two(ve + bit - 1)) ? bit : 0;
      vlim = power_of_two(ve);
      // each row's largest weight times step is at most the largest of each, and by
      // less than 2^kSpread so unless steps (hidden ones among them) differ by more
      float most = __builtin_fmaf(umax, cs, (float)ve);
      if (__any(vstep > 0.0f && vstep < power_of_two(ve - kSpread))) {
        float best = kNone;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const f32x4 v = per_key(sm.vs[buf], j >> 2, j & 3);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            best = fmaxf(best, __builtin_fmaf(u[4 * j + e], cs, (float)__builtin_amdgcn_frexp_expf(fminf(fmaxf(v[e], kLeastStep), 65504.0f))));
          __builtin_amdgcn_sched_barrier(0);                 // (bounds the registers in use)
        }
        best = fmaxf(best, __shfl_xor(best, 32, 64));
        most = fminf(fmaxf(most, __shfl_xor(most, 32, 64)), best + (kSpread - 1));
      }
      most = fmaxf(most, __shfl_xor(most, 32, 64));
      const float m_before = M;
      M = fmaxf(M, most - kRaise);
      slack = M == kNone ? kNone : __builtin_ldexpf(M + (kLimit - ve), 1 - __builtin_amdgcn_frexp_expf(cs));
      top = fmaxf(top, umax);                                // (of this lane's keys, until it matters)
      if (__builtin_expect(__any(nearly_past(M)), 0)) {
        // (top * cs is exact, and so is every weight's exponent u cs - M)
        top = fmaxf(top, __shfl_xor(top, 32, 64));
        const bool past = past_fractions(top, cs);
        M = past ? top * cs : M;
        slack = past ? top : slack;
      }
      const float a = __builtin_amdgcn_exp2f(m_before - M);
      l *= a;
#pragma unroll
      for (int n = 0; n < kTiles; ++n)
#pragma unroll
        for (int e = 0; e < 16; ++e) o[n][e] *= a;
    }
    // weights of 16 keys, then their products, with the next 16's weights and
    // operands under way between the MFMAs
    auto weights = [&](int st) {
      u32x4 pb;
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const f32x4 v = per_key(sm.vs[buf], st >> 1, 2 * (st & 1) + g);
        float pr[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float x = __builtin_amdgcn_exp2f(__builtin_fmaf(u[8 * st + 4 * g + e], cs, -M));
          l += x;
          pr[e] = x * v[e];
        }
        pb[2 * g] = pack_half2(pr[0], pr[1]);
        pb[2 * g + 1] = pack_half2(pr[2], pr[3]);
      }
      return pb;
    };
    u32x4 pb = weights(0);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int st = 0; st < 4; ++st) {
      u32x4 next = pb;
      if (st < 3) {
#pragma unroll
        for (int n = 0; n < kTiles; ++n) vf[(st + 1) & 1][n] = value_frag(st + 1, n);
        next = weights(st + 1);
      }
#pragma unroll
      for (int n = 0; n < kTiles; ++n) o[n] = mfma32x16(vf[st & 1][n], pb, o[n]);
      if (st < 3) {
        __builtin_amdgcn_sched_group_barrier(kLdsRead, kTiles + 2, 0);
#pragma unroll
        for (int n = 0; n < kTiles; ++n) {
          __builtin_amdgcn_sched_group_barrier(kMfma, 1, 0);
          __builtin_amdgcn_sched_group_barrier(kValu, (36 + kTiles - 1) / kTiles, 0);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
      pb = next;
    }
  };

  // group g of four waves walks the tiles g, g + NG, ...
  constexpr int kStride = kPtKeys * NG;
  if (nt > 0) {
    const int t_first = t_lo + kPtKeys * grp;
    if (grp < nt) {
      load_page(t_first);
      load_codes(t_first);
      load_page(t_first + kStride);
      stage_keys(0);
      stage_values(0);
    }
    __syncthreads();
    for (int s = 0; s * NG < nt; ++s) {
      const int i = s * NG + grp, t0 = t_lo + kPtKeys * i, buf = s & 1;
      const bool more = i + NG < nt;
      if (more) {
        load_codes(t0 + kStride);
        load_page(t0 + 2 * kStride);
      }
      if (wave_live && i < nt && t0 <= w_any_last && t0 + kPtKeys > w_any_first) compute(buf, t0);
      if (more) {
        stage_keys(buf ^ 1);
        stage_values(buf ^ 1);
      }
      __syncthreads();
    }
  }
  if constexpr (NG == 2) {                                   // the second group's sums through LDS to the first's waves
    float *po = reinterpret_cast<float *>(sms) + wave * (16 * kTiles + 2) * 64 + lane;
    if (grp == 1) {
#pragma unroll
      for (int n = 0; n < kTiles; ++n)
#pragma unroll
        for (int e = 0; e < 16; ++e) po[(16 * n + e) * 64] = o[n][e];
      po[16 * kTiles * 64] = M;
      po[(16 * kTiles + 1) * 64] = l;
    }
    __syncthreads();
    if (grp == 1) return;
    const float M1 = po[16 * kTiles * 64], m2 = fmaxf(M, M1);
    const float a0 = __builtin_amdgcn_exp2f(M - m2), a1 = __builtin_amdgcn_exp2f(M1 - m2);
    M = m2;
    l = l * a0 + po[(16 * kTiles + 1) * 64] * a1;
#pragma unroll
    for (int n = 0; n < kTiles; ++n)
#pragma unroll
      for (int e = 0; e < 16; ++e) o[n][e] = o[n][e] * a0 + po[(16 * n + e) * 64] * a1;
  }

  // ---- store: lane (q, hh) holds LDS rows 32n + 8g + 4hh + e of row q, all
  // eight channels of D/16 of its words
  l += __shfl_xor(l, 32, 64);
  if (row0 + wave * 32 + qc >= rows) return;
  const bool none = l == 0.0f;
  const float inv = none ? 0.0f : 1.0f / l;
  const int64_t head_row = (rq.token0 + qi) * ((int64_t)p.heads * p.group) + h * p.group + row - qi * p.group;
  const int64_t at = keys.parts > 1 ? split * p.T * p.heads * p.group + head_row : head_row;
  if (keys.parts > 1) {
    if (hh == 0) {
      p.part_sum[at] = float2{M, l};
      if (__builtin_expect(may_have_low_part(M), 0)) p.part_lo[at] = 0.0f;
    }
    if (none) return;
  } else if (p.lse && hh == 0) {
    p.lse[at] = none ? -__builtin_inff() : natural_log(M, l);
  }
#pragma unroll
  for (int x = 0; x < D / 16; ++x) {
    const int word = D == 128 ? 8 * (x >> 2) + 4 * hh + (x & 3) : 4 * hh + x;
    float v[8];
#pragma unroll
    for (int ch = 0; ch < 8; ++ch) {
      const int n = D == 128 ? ch >> 1 : ch >> 2;
      const int g = D == 128 ? 2 * (ch & 1) + (x >> 2) : ch & 3;
      v[ch] = none ? 0.0f : o[n][4 * g + (x & 3)] * inv;
    }
    const int64_t d = at * D + 8 * word;
    if (keys.parts > 1) {
      float4 *po = reinterpret_cast<float4 *>(p.part_o + d);
      po[0] = float4{v[0], v[1], v[2], v[3]};
      po[1] = float4{v[4], v[5], v[6], v[7]};
    } else {
      u32x4 w;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[i] = BF16 ? pack_bf16x2(v[2 * i], v[2 * i + 1]) : pack_half2(v[2 * i], v[2 * i + 1]);
      *reinterpret_cast<u32x4 *>(reinterpret_cast<uint16_t *>(p.O) + d) = w;
    }
  }
}

// ---- join the splits ---------------------------------------------------------------------------
// Row (token, head): weights 2^(reference_s - the largest) sum_s over at most
// kMaxSplits splits (kept apart: in one logarithm a large reference would swallow
// the sum), WPR waves of a workgroup of four per row: lane s reads split s's
// reference and sum, wave w of the row sums the splits s = w mod WPR, their rows
// loaded eight at a time, and the waves' sums meet in LDS.  (Many splits of few
// rows, a decode step's, want the waves on one row: 32 splits of 256 rows took one
// wave per row 24 us, four 4.  Few splits of many rows, a prompt's, want a wave
// each: 2 splits of 12360 rows of 64 took four waves per row 38 us.)  A split in
// which the row saw no key has written a sum of 0 and no O.  Rows that no request
// serves were not written and are not read.
constexpr int kMaxSplits = 64;

template <int D, bool BF16, int WPR>
__global__ __launch_bounds__(256) void kv_join_kernel(KvAttn p) {
  constexpr int kPer = D / 64, kChunk = 8;
  __shared__ float part[4][D], part_sum[4];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int b = blockIdx.z, h = blockIdx.y;
  const int w0 = WPR == 4 ? wave : 0, r = WPR == 4 ? (int)blockIdx.x : (int)blockIdx.x * 4 + wave;
  const Request rq = request_of(p, b);
  const int rows = rq.ql * p.group;
  if (r >= rows) return;
  const int row0 = r - r % p.tile_rows, row1 = row0 + p.tile_rows <= rows ? row0 + p.tile_rows - 1 : rows - 1;
  const int parts = keys_of(p, rq, row0, row1, p.tile_rows == 16 ? 32 : kPtKeys).parts;
  if (parts == 1) return;                            // stored by its one workgroup
  const int64_t n = p.T * p.heads * p.group;
  const int qi = token_of(p, r);
  const int64_t at = (rq.token0 + qi) * ((int64_t)p.heads * p.group) + h * p.group + r - qi * p.group;
  const float2 mine = lane < parts ? p.part_sum[lane * n + at] : float2{kNone, 0.0f};
  const float l = mine.y;
  Reference x = {l != 0.0f ? mine.x : kNone, 0.0f}, m = x;
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) m.hi = fmaxf(m.hi, __shfl_xor(m.hi, d, 64));
  if (__builtin_expect(__any(may_have_low_part(x.hi)), 0)) {
    x.lo = may_have_low_part(x.hi) ? p.part_lo[lane * n + at] : 0.0f;
    m.lo = x.hi == m.hi ? x.lo : kNone;
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) m.lo = fmaxf(m.lo, __shfl_xor(m.lo, d, 64));
  }
  const float w = l != 0.0f ? exp2_difference(x, m) * l : 0.0f;
  float sum = 0.0f, acc[kPer] = {};
  for (int s0 = w0; s0 < parts; s0 += WPR * kChunk) {
    float v[kChunk][kPer], ws[kChunk];
#pragma unroll
    for (int u = 0; u < kChunk; ++u) {
      const int s = s0 + WPR * u < parts ? s0 + WPR * u : s0;
      ws[u] = s0 + WPR * u < parts ? __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, w), s)) : 0.0f;
      const float *src = p.part_o + (s * n + at) * D + lane * kPer;
#pragma unroll
      for (int i = 0; i < kPer; ++i) v[u][i] = src[i];
    }
#pragma unroll
    for (int u = 0; u < kChunk; ++u) {
      sum += ws[u];
#pragma unroll
      for (int i = 0; i < kPer; ++i) acc[i] = ws[u] != 0.0f ? __builtin_fmaf(v[u][i], ws[u], acc[i]) : acc[i];
    }
  }
  if constexpr (WPR == 4) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) part[wave][lane * kPer + i] = acc[i];
    if (lane == 0) part_sum[wave] = sum;
    __syncthreads();
    if (wave != 0) return;
    sum = (part_sum[0] + part_sum[1]) + (part_sum[2] + part_sum[3]);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int d = lane * kPer + i;
      acc[i] = (part[0][d] + part[1][d]) + (part[2][d] + part[3][d]);
    }
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const float v = sum == 0.0f ? 0.0f : acc[i] / sum;
    reinterpret_cast<uint16_t *>(p.O)[at * D + lane * kPer + i] = BF16 ? float_to_bf16_bits(v) : float_to_half_bits(v);
  }
  if (p.lse && lane == 0 && w0 == 0)
    p.lse[at] = sum == 0.0f ? -__builtin_inff() : natural_log(m.hi, sum);
}

// ---- plan and launch ------------------------------------------------------------------------------
KvAttnPlan kv_attention_plan(int64_t T, int B, int heads, int group, int D, int max_q, int64_t max_kv,
                             int window) {
  KvAttnPlan pl{};
  const int64_t rows = (int64_t)max_q * group;
  // keys that a tile of rows can see at most
  int64_t span = max_kv;
  if (window > 0 && (int64_t)window + max_q < span) span = (int64_t)window + max_q;
  span = span < 1 ? 1 : span > 0x7FFFFF00 ? 0x7FFFFF00 : span;
  pl.prompt = rows > 32;
  pl.tile_rows = pl.prompt ? kPtRows : 16;
  const int64_t wgs = (int64_t)B * heads * ((rows + pl.tile_rows - 1) / pl.tile_rows);
  pl.waves = 4;
  int64_t splits;
  if (pl.prompt) {
    // Fewer workgroups than two per CU: eight waves each, two groups over
    // alternate tiles, which halves the time of the longest request (six ragged
    // requests, 408 workgroups of D = 64: 25.8 us against 39.8; seven, 476 of D =
    // 128: 67 against 107; three of one length, 384, are slower, 87 against 78).
    // From 512 on four waves serve better (2048 tokens, 32 heads over 8: 84 us
    // against 93).  Every request is counted with max_q tokens, so these are more
    // than the workgroups that have rows where lengths differ; counted by the tokens
    // in all, some batches gain and some lose (a chunk of 200 among 11 single tokens
    // after 20000: 361 -> 105 us; one of 512 among 15 after 4000: 422 -> 600).  Keys are split while there is less than a workgroup per CU, into
    // parts of 512 keys, or 256 for few rows: the parts' fp32 results are written
    // and read again (512 tokens of 32 heads: 19.9 us in one part, 29.3 in two; 64
    // tokens after 936: 19.8 us in four parts, 23.9 in two).
    pl.chunk = wgs < 64 ? 256 : 512;
    if (wgs < 512) pl.waves = 8;
    splits = wgs > 0 && wgs < 256 ? 256 / wgs : 1;
  } else if (span <= 1536 && wgs < 512) {
    // Short contexts of few requests: eight waves and no join, which costs a launch
    // (1500 tokens, 32 heads over 8: one request 16.2 -> 13.0 us a call, in a graph
    // 11.6 -> 12.5; sixteen 16.8 -> 13.7 and 14.8 -> 13.3).  Later the waves' own
    // steps cost more (2048 tokens, one request: 11.4 us in a graph, 15.0 with eight).
    pl.waves = 8;
    pl.chunk = 1536;
    splits = 1;
  } else {
    // four workgroups to a CU; with as many rows as that anyway, two parts for
    // the long requests of a batch, which would otherwise finish last
    pl.chunk = wgs < 1024 ? 512 : 1024;
    splits = wgs > 0 && wgs < 1024 ? 1024 / wgs : 2;
  }
  const int64_t most = (span + pl.chunk - 1) / pl.chunk;
  splits = splits < most ? splits : most;
  splits = splits < kMaxSplits ? splits : kMaxSplits;
  pl.splits = splits < 1 ? 1 : (int)splits;
  if (pl.splits > 1) {
    const int64_t n = T * heads * group;
    pl.sum_offset = (size_t)pl.splits * n * D * 4;
    pl.lo_offset = pl.sum_offset + (size_t)pl.splits * n * 8;
    pl.workspace_bytes = pl.lo_offset + (size_t)pl.splits * n * 4;
  }
  return pl;
}

namespace {
template <int D, bool SYM, bool BF16>
hipError_t attn_go(const KvAttn &p, int B, const KvAttnPlan &pl, hipStream_t st) {
  const int64_t rows = (int64_t)p.max_q * p.group;
  if (pl.prompt) {
    const dim3 grid((unsigned)((rows + kPtRows - 1) / kPtRows), (unsigned)(p.heads * p.splits), (unsigned)B);
    if (pl.waves == 8) kv_prompt_kernel<D, SYM, BF16, 2><<<grid, 2 * kPtThreads, 0, st>>>(p);
    else kv_prompt_kernel<D, SYM, BF16, 1><<<grid, kPtThreads, 0, st>>>(p);
  } else {
    const dim3 grid((unsigned)((rows + 15) / 16 * p.heads), (unsigned)p.splits, (unsigned)B);
    if (pl.waves == 8) kv_decode_kernel<D, SYM, BF16, 8><<<grid, 512, 0, st>>>(p);
    else kv_decode_kernel<D, SYM, BF16, 4><<<grid, 256, 0, st>>>(p);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.splits == 1) return e;
  if (p.splits > 8)
    kv_join_kernel<D, BF16, 4><<<dim3((unsigned)rows, (unsigned)p.heads, (unsigned)B), 256, 0, st>>>(p);
  else
    kv_join_kernel<D, BF16, 1><<<dim3((unsigned)((rows + 3) / 4), (unsigned)p.heads, (unsigned)B), 256, 0, st>>>(p);
  return hipGetLastError();
}
}  // namespace

hipError_t launch_kv_attention(KvAttn p, int B, int D, XType xt, const KvAttnPlan &pl,
                               void *workspace, hipStream_t st) {
  p.splits = pl.splits;
  p.chunk = pl.chunk;
  p.tile_rows = pl.tile_rows;
  if (pl.splits > 1) {
    p.part_o = reinterpret_cast<float *>(workspace);
    p.part_sum = reinterpret_cast<float2 *>(reinterpret_cast<char *>(workspace) + pl.sum_offset);
    p.part_lo = reinterpret_cast<float *>(reinterpret_cast<char *>(workspace) + pl.lo_offset);
  }
  const bool sym = p.zeros == nullptr, bf16 = xt == XType::BF16;
  if (D == 128) {
    if (sym) return bf16 ? attn_go<128, true, true>(p, B, pl, st) : attn_go<128, true, false>(p, B, pl, st);
    return bf16 ? attn_go<128, false, true>(p, B, pl, st) : attn_go<128, false, false>(p, B, pl, st);
  }
  if (sym) return bf16 ? attn_go<64, true, true>(p, B, pl, st) : attn_go<64, true, false>(p, B, pl, st);
  return bf16 ? attn_go<64, false, true>(p, B, pl, st) : attn_go<64, false, false>(p, B, pl, st);
}

}  // namespace awq
