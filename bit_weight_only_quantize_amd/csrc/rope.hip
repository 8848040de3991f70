// Rotary positions on gfx950: queries and keys turned by angles that grow with
// their positions (awq_rope), alone or on the way into the 4-bit key/value cache
// (awq_kv_append_rope).
//
// Of each head's first R channels, pair j < R/2 is (a, b) = channels (j, j + R/2),
// or (2j, 2j + 1) where neighbours are paired:
//   a' = a c - b s,   b' = b c + a s,   c, s = factor * cos, sin(position * inv_freq_j).
// The angle is an fp64 product and so are its cosine and sine, to about 2^-50,
// rounded once to fp32: at position 2^20 an fp32 angle would be off by 2^-4.  The
// products and the sum are fp32, each rounded once and not fused, so what they give
// does not depend on the kernel, and the codes that a cache gets neither.
//
// A workgroup takes a run of tokens, computes their cosines and sines once, a
// thread for each (LDS, 8 KiB at most), and keeps a lane's in registers while it
// walks heads: a lane holds eight channels of a token.  Paired halves are R/16 lanes
// apart and exchanged between lanes, so every channel is read once.
//
// Bound by memory; few tokens by a launch's latency and the chain of fp64 operations
// (about 30 per angle).

#include "awq_internal.h"
#include "device_common.h"
#include "kv_place.h"
#include "quant_group.h"

namespace awq {

constexpr int kRopeThreads = 256, kRopePairs = 1024;   // pairs of a workgroup's tokens, at most
constexpr int kRopeAhead = 4;                          // heads whose loads are in flight together

// cos and sin of x, each times factor, rounded to fp32.  x = n pi/2 + r, |r| <= pi/4
// (a little more for |x| past 2^31), then the Taylor series of r: the first terms left out
// are r^15/15! and r^16/16!, below 2^-45 of the results.
__device__ __forceinline__ float2 cos_sin(double x, double factor) {
  const double n = __builtin_rint(x * 0x1.45f306dc9c883p-1);          // 2/pi
  double r = __builtin_fma(-n, 0x1.921fb54442d18p0, x);                // pi/2 in two parts
  r = __builtin_fma(-n, 0x1.1a62633145c07p-54, r);
  const double r2 = r * r;
  double s = __builtin_fma(r2, 1.0 / 6227020800.0, -1.0 / 39916800.0);
  s = __builtin_fma(r2, s, 1.0 / 362880.0);
  s = __builtin_fma(r2, s, -1.0 / 5040.0);
  s = __builtin_fma(r2, s, 1.0 / 120.0);
  s = __builtin_fma(r2, s, -1.0 / 6.0);
  s = __builtin_fma(r * r2, s, r);
  double c = __builtin_fma(r2, -1.0 / 87178291200.0, 1.0 / 479001600.0);
  c = __builtin_fma(r2, c, -1.0 / 3628800.0);
  c = __builtin_fma(r2, c, 1.0 / 40320.0);
  c = __builtin_fma(r2, c, -1.0 / 720.0);
  c = __builtin_fma(r2, c, 1.0 / 24.0);
  c = __builtin_fma(r2, c, -0.5);
  c = __builtin_fma(r2, c, 1.0);
  const int quarter = (int)(int64_t)n & 3;
  const double a = quarter & 1 ? s : c, b = quarter & 1 ? c : s;
  return float2{(float)((quarter == 1 || quarter == 2 ? -a : a) * factor), (float)((quarter & 2 ? -b : b) * factor)};
}

// What a lane does with its eight channels: out = own * c + partner * s.
struct Turn {
  float c[8], s[8];
  int from;              // the partner's lane (paired halves)
  bool on;               // the channels are among the first R
};

// Cosines and sines of `tokens` tokens from t0 on into `table` [token][R/2].
__device__ __forceinline__ void fill_turns(const RopeArgs &p, int64_t t0, int tokens, int64_t T, float2 *table) {
  const int half = p.rotary_dim / 2;
  for (int i = threadIdx.x; i < tokens * half; i += kRopeThreads) {
    const int t = i / half, j = i - t * half;
    const int64_t at = t0 + t < T ? t0 + t : T - 1;
    float2 cs = cos_sin((double)p.positions[at] * p.inv_freq[j], p.factor);
    if (p.inverse) cs.y = -cs.y;
    table[i] = cs;
  }
}

// The lane's turn, of the token at place `token` of the workgroup's, channels 8w on.
template <bool PAIRS>
__device__ __forceinline__ Turn turn_of(const RopeArgs &p, const float2 *table, int token, int w, int lane) {
  Turn t;
  const int half = p.rotary_dim / 2, apart = half / 8;
  t.on = w < 2 * apart;
  const bool low = w < apart;
  t.from = lane + (t.on ? (low ? apart : -apart) : 0);
  const float2 *row = table + token * half;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int j = !t.on ? 0 : PAIRS ? 4 * w + i / 2 : 8 * (low ? w : w - apart) + i;
    const float2 cs = row[j];
    t.c[i] = cs.x;
    t.s[i] = (PAIRS ? (i & 1) == 0 : low) ? -cs.y : cs.y;
  }
  return t;
}

// Eight channels, turned.  All lanes of a wave call it.
template <bool BF16, bool PAIRS>
__device__ __forceinline__ void turn8(const Turn &t, u32x4 raw, float (&v)[8]) {
  widen8<BF16>(raw, v);
  float other[8];
  if constexpr (PAIRS) {
#pragma unroll
    for (int i = 0; i < 8; ++i) other[i] = v[i ^ 1];
  } else {
    u32x4 theirs;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t r = raw[i];
      theirs[i] = (uint32_t)__shfl((int)r, t.from, 64);
    }
    widen8<BF16>(theirs, other);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float y = v[i] * t.c[i] + other[i] * t.s[i];
    v[i] = t.on ? y : v[i];
  }
}

template <bool BF16>
__device__ __forceinline__ u32x4 narrow8(const float (&v)[8]) {
  u32x4 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = BF16 ? float_to_bf16_bits(v[2 * i]) : float_to_half_bits(v[2 * i]);
    const uint32_t hi = BF16 ? float_to_bf16_bits(v[2 * i + 1]) : float_to_half_bits(v[2 * i + 1]);
    r[i] = lo | (hi << 16);
  }
  return r;
}

// Heads begin .. end of the lane's token: from x (its channels of head 0) to y, D
// channels a head.  x and y may be the same place: a wave has read a head's
// channels before any of its lanes writes one.
template <bool BF16, bool PAIRS>
__device__ __forceinline__ void turn_heads(const Turn &t, const uint16_t *x, uint16_t *y, int D, int begin, int end,
                                           bool active) {
  for (int h = begin; h < end; h += kRopeAhead) {
    u32x4 raw[kRopeAhead];
#pragma unroll
    for (int i = 0; i < kRopeAhead; ++i) {
      raw[i] = u32x4{0u, 0u, 0u, 0u};
      if (active && h + i < end) raw[i] = *reinterpret_cast<const u32x4 *>(x + (int64_t)(h + i) * D);
    }
#pragma unroll
    for (int i = 0; i < kRopeAhead; ++i) {
      float v[8];
      turn8<BF16, PAIRS>(t, raw[i], v);
      if (active && h + i < end) *reinterpret_cast<u32x4 *>(y + (int64_t)(h + i) * D) = narrow8<BF16>(v);
    }
  }
}

// Heads of part `part` of `parts`.
__device__ __forceinline__ int part_begin(int heads, int part, int parts) { return (int)((int64_t)heads * part / parts); }

template <bool BF16, bool PAIRS>
__global__ __launch_bounds__(kRopeThreads) void rope_kernel(RopeArgs p, RopeArray q, RopeArray k, int64_t T, int D) {
  __shared__ float2 table[kRopePairs];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  // a wave takes as many whole tokens as fit its lanes (D need not divide 512)
  const int lanes = D / 8, per_wave = 64 / lanes;
  const int mine = lane / lanes < per_wave ? lane / lanes : per_wave - 1;
  const int token = wave * per_wave + mine, w = lane < per_wave * lanes ? lane - mine * lanes : 0;
  const int64_t t0 = (int64_t)blockIdx.x * (4 * per_wave), t = t0 + token;
  fill_turns(p, t0, 4 * per_wave, T, table);
  __syncthreads();
  const Turn turn = turn_of<PAIRS>(p, table, token, w, lane);
  const bool active = t < T && lane < per_wave * lanes;
  const int part = blockIdx.y, parts = gridDim.y;
  turn_heads<BF16, PAIRS>(turn, q.x + t * q.x_stride + w * 8, q.y + t * q.y_stride + w * 8, D,
                          part_begin(q.heads, part, parts), part_begin(q.heads, part + 1, parts), active);
  turn_heads<BF16, PAIRS>(turn, k.x + t * k.x_stride + w * 8, k.y + t * k.y_stride + w * 8, D,
                          part_begin(k.heads, part, parts), part_begin(k.heads, part + 1, parts), active);
}

template <int D, bool SYM, bool BF16, bool PAIRS>
__global__ __launch_bounds__(kRopeThreads) void kv_append_rope_kernel(
    RopeArgs p, RopeArray q, const uint16_t *__restrict__ K, const uint16_t *__restrict__ V, int64_t T, int heads,
    int64_t k_stride, int64_t v_stride, const int32_t *__restrict__ slots, int64_t num_slots, int pshift,
    uint32_t *__restrict__ codes, uint16_t *__restrict__ scales, uint8_t *__restrict__ zeros,
    int32_t *__restrict__ nonfinite) {
  constexpr int kLanes = D / 8, kTokens = kRopeThreads / kLanes;
  __shared__ float2 table[kRopePairs];
  const int lane = threadIdx.x & 63;
  const int token = threadIdx.x / kLanes, w = threadIdx.x % kLanes;
  const int64_t t0 = (int64_t)blockIdx.x * kTokens, t = t0 + token;
  const int32_t slot = t < T ? slots[t] : -1;
  fill_turns(p, t0, kTokens, T, table);
  __syncthreads();
  const Turn turn = turn_of<PAIRS>(p, table, token, w, lane);
  const int part = blockIdx.y, parts = gridDim.y;
  if (q.heads > 0)
    turn_heads<BF16, PAIRS>(turn, q.x + t * q.x_stride + w * 8, q.y + t * q.y_stride + w * 8, D,
                            part_begin(q.heads, part, parts), part_begin(q.heads, part + 1, parts), t < T);
  // lanes of a group share their token, so a group is active as a whole
  const bool active = slot >= 0 && slot < num_slots;
  int bad = 0;
  const int end = part_begin(heads, part + 1, parts);
  for (int h = part_begin(heads, part, parts); h < end; ++h) {
    u32x4 kr = {0u, 0u, 0u, 0u}, vr = kr;
    if (active) {
      kr = *reinterpret_cast<const u32x4 *>(K + t * k_stride + (int64_t)h * D + w * 8);
      vr = *reinterpret_cast<const u32x4 *>(V + t * v_stride + (int64_t)h * D + w * 8);
    }
    float k[8], v[8];
    turn8<BF16, PAIRS>(turn, kr, k);
    widen8<BF16>(vr, v);
    const QuantWord qk = quantize_word<kLanes, SYM>(k, bad), qv = quantize_word<kLanes, SYM>(v, bad);
    if (!active) continue;
    if (nonfinite != nullptr && w == 0) bad += (int)qk.overflow + (int)qv.overflow;
    const KvPlace at = kv_place<D>(slot, pshift, h, heads, w);
    codes[at.k_word] = qk.word;
    codes[at.v_word] = qv.word;
    if (w == 0) {
      *reinterpret_cast<uint32_t *>(scales + at.meta) =
          (uint32_t)__builtin_bit_cast(uint16_t, qk.step) | ((uint32_t)__builtin_bit_cast(uint16_t, qv.step) << 16);
      if constexpr (!SYM)
        *reinterpret_cast<uint16_t *>(zeros + at.meta) = (uint16_t)((uint32_t)qk.zero | ((uint32_t)qv.zero << 8));
    }
  }
  if (nonfinite != nullptr) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) bad += __shfl_xor(bad, off, 64);
    if (lane == 0 && bad) atomicAdd(nonfinite, bad);
  }
}

namespace {
// Workgroups along the tokens and along the heads: parts of the heads while there are
// fewer than eight workgroups per CU, a head each at least.
dim3 rope_grid(int64_t T, int tokens, int heads) {
  const int64_t along = (T + tokens - 1) / tokens;
  int64_t parts = (2048 + along - 1) / along;
  parts = parts < heads ? parts : heads;
  return dim3((unsigned)along, (unsigned)(parts < 1 ? 1 : parts));
}

template <int D, bool SYM, bool BF16>
hipError_t append_rope_go(const RopeArgs &p, const RopeArray &q, const uint16_t *K, const uint16_t *V, int64_t T,
                          int64_t ks, int64_t vs, const int32_t *slots, const KvCache &c, int32_t *nonfinite,
                          hipStream_t st) {
  const dim3 grid = rope_grid(T, kRopeThreads / (D / 8), q.heads > c.heads ? q.heads : c.heads);
  const int sh = __builtin_ctz((unsigned)c.page_size);
  const int64_t ns = c.pages * c.page_size;
  if (p.pairs) kv_append_rope_kernel<D, SYM, BF16, true><<<grid, kRopeThreads, 0, st>>>(p, q, K, V, T, c.heads, ks, vs, slots, ns, sh, c.codes, c.scales, c.zeros, nonfinite);
  else kv_append_rope_kernel<D, SYM, BF16, false><<<grid, kRopeThreads, 0, st>>>(p, q, K, V, T, c.heads, ks, vs, slots, ns, sh, c.codes, c.scales, c.zeros, nonfinite);
  return hipGetLastError();
}
}  // namespace

hipError_t launch_rope(const RopeArgs &p, const RopeArray &q, const RopeArray &k, XType xt, int64_t T, int D,
                       hipStream_t st) {
  const dim3 grid = rope_grid(T, 4 * (64 / (D / 8)), q.heads > k.heads ? q.heads : k.heads);
  const bool bf16 = xt == XType::BF16;
  if (bf16 && p.pairs) rope_kernel<true, true><<<grid, kRopeThreads, 0, st>>>(p, q, k, T, D);
  else if (bf16) rope_kernel<true, false><<<grid, kRopeThreads, 0, st>>>(p, q, k, T, D);
  else if (p.pairs) rope_kernel<false, true><<<grid, kRopeThreads, 0, st>>>(p, q, k, T, D);
  else rope_kernel<false, false><<<grid, kRopeThreads, 0, st>>>(p, q, k, T, D);
  return hipGetLastError();
}

hipError_t launch_kv_append_rope(const RopeArgs &p, const RopeArray &q, const uint16_t *K, const uint16_t *V, XType xt,
                                 int64_t T, int64_t ks, int64_t vs, const int32_t *slots, const KvCache &c,
                                 int32_t *nonfinite, hipStream_t st) {
  const bool bf16 = xt == XType::BF16, sym = c.zeros == nullptr;
  if (c.head_dim == 128) {
    if (sym) return bf16 ? append_rope_go<128, true, true>(p, q, K, V, T, ks, vs, slots, c, nonfinite, st)
                         : append_rope_go<128, true, false>(p, q, K, V, T, ks, vs, slots, c, nonfinite, st);
    return bf16 ? append_rope_go<128, false, true>(p, q, K, V, T, ks, vs, slots, c, nonfinite, st)
                : append_rope_go<128, false, false>(p, q, K, V, T, ks, vs, slots, c, nonfinite, st);
  }
  if (sym) return bf16 ? append_rope_go<64, true, true>(p, q, K, V, T, ks, vs, slots, c, nonfinite, st)
                       : append_rope_go<64, true, false>(p, q, K, V, T, ks, vs, slots, c, nonfinite, st);
  return bf16 ? append_rope_go<64, false, true>(p, q, K, V, T, ks, vs, slots, c, nonfinite, st)
              : append_rope_go<64, false, false>(p, q, K, V, T, ks, vs, slots, c, nonfinite, st);
}

}  // namespace awq
