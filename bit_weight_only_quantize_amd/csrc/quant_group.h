// One group's quantization on gfx950, shared by the weight quantizer
// (quantize_pack.hip) and the key/value cache writer (kv_cache.hip): both
// produce the codes, step and zero point that awq_quantize_pack documents.
#pragma once

#include <type_traits>

#include "device_common.h"

namespace awq {

// Largest value over the g/8 lanes of a group (aligned runs of 8 or 16 lanes)
// with DPP lane exchanges: swap neighbours, swap pairs, mirror within 8, then
// (g = 128) mirror within 16.  Each step pairs every lane with one of the other
// half of its current run, so after log2(g/8) steps every lane of a group
// holds the group's maximum.  Applied to the bit patterns of floats of one
// sign it is an exact float reduction: non-negative floats order like their
// patterns, and non-positive ones in reverse (so the largest pattern is the
// minimum).  Integer maxima need no NaN quieting before each exchange, which
// a float min or max does (two more instructions per step).
template <int LANES>
__device__ __forceinline__ uint32_t group_umax(uint32_t v) {
  auto step = [](uint32_t x, auto ctrl_tag) {
    constexpr int kCtrl = decltype(ctrl_tag)::value;
    const uint32_t y = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, kCtrl, 0xF, 0xF, true);
    return x > y ? x : y;
  };
  v = step(v, std::integral_constant<int, 0xB1>{});    // quad_perm [1,0,3,2]
  v = step(v, std::integral_constant<int, 0x4E>{});    // quad_perm [2,3,0,1]
  v = step(v, std::integral_constant<int, 0x141>{});   // row_half_mirror
  if constexpr (LANES == 16) v = step(v, std::integral_constant<int, 0x140>{});   // row_mirror
  return v;
}
// Minimum of non-positive floats and maximum of non-negative floats over the
// group (lo <= 0 <= hi by construction).
template <int LANES>
__device__ __forceinline__ float group_min_nonpos(float v) {
  return __builtin_bit_cast(float, group_umax<LANES>(__builtin_bit_cast(uint32_t, v)));
}
template <int LANES>
__device__ __forceinline__ float group_max_nonneg(float v) {
  return __builtin_bit_cast(float, group_umax<LANES>(__builtin_bit_cast(uint32_t, v)));
}

// What a lane stores of its group: its word of eight codes, the step as fp16
// and the zero point (0..15; 8 for the symmetric grid).  `overflow`: the group holds
// no infinity, but its step does not fit fp16.
struct QuantWord {
  uint32_t word;
  _Float16 step;
  float zero;
  bool overflow;
};

// Quantizes a group held by LANES consecutive lanes, eight values (v, in
// channel order) per lane.  `bad` grows by the number of non-finite values.
template <int LANES, bool SYM>
__device__ __forceinline__ QuantWord quantize_word(const float (&v)[8], int &bad) {
  float lo = 0.0f, hi = 0.0f, step, most;              // most: the group's largest magnitude
  if constexpr (SYM) {
    // the largest magnitude of the group on level +-7: one IEEE division
    // per lane and group
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = fmaxf(amax, __builtin_fabsf(v[i]));
    amax = group_max_nonneg<LANES>(amax);
    step = amax / 7.0f;
    most = amax;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      lo = fminf(lo, v[i]);
      hi = fmaxf(hi, v[i]);
    }
    lo = group_min_nonpos<LANES>(lo);
    hi = group_max_nonneg<LANES>(hi);

    // (hi - lo) / 15, correctly rounded, from the product with RN(1/15)
    // and one exact-remainder correction (Markstein): checked against IEEE
    // division for every non-negative finite fp32 dividend; an infinite
    // dividend (the only other value hi - lo takes) passes through as the
    // division would give it.
    const float d = hi - lo;
    const float q0 = d * 0x1.111112p-4f;
    const float q1 = __builtin_fmaf(__builtin_fmaf(-15.0f, q0, d), 0x1.111112p-4f, q0);
    step = d == __builtin_inff() ? d : q1;
    most = fmaxf(hi, -lo);
  }
  const _Float16 sh = (_Float16)fmaxf(step, 0x1p-14f);
  const float sf = (float)sh;

  // rint(v / sf) with the correctly rounded quotient q, without eight
  // divisions: |v / sf| < 16 (|v| <= hi - lo <= 15 sf (1 + 2^-10), or
  // symmetric |v| <= max |v| <= 7 sf (1 + 2^-10)), so q
  // lies within 2^-20 of the exact v / sf, and y = fl(v * rcp(sf)), with
  // the hardware reciprocal (specified to 1 ulp; up to 7 ulp would do),
  // within 2^-16 - 2^-20.  Unless y is within 2^-16 of a half-integer, both
  // round to the same integer (ties included: a q exactly at k + 1/2 puts
  // y that close to it); the rare lanes that are that close divide.  The
  // zero point's -lo / sf (also below 16) takes the same path.  The test is
  // written so that a NaN y also fails it: every non-finite v makes its own
  // lane's y NaN (v * rcp(sf) is NaN or +-inf, and inf - rint(inf) is NaN;
  // an inf in the group makes sf inf and rcp(sf) 0), so those lanes take
  // the slow path too, where they are counted.
  const float rs = __builtin_amdgcn_rcpf(sf);
  const float zy = -lo * rs;          // symmetric: lo = 0, so zq = 0
  float zq = __builtin_rintf(zy);
  bool near_half = !(__builtin_fabsf(zy - zq) <= 0.5f - 0x1p-16f);
  float qv[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float y = v[i] * rs;
    qv[i] = __builtin_rintf(y);
    // y - rint(y) is exact
    near_half |= !(__builtin_fabsf(y - qv[i]) <= 0.5f - 0x1p-16f);
  }
  if (near_half) {
    if constexpr (!SYM) zq = __builtin_rintf(-lo / sf);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      qv[i] = __builtin_rintf(v[i] / sf);
      bad += !__builtin_isfinite(v[i]);
    }
  }
  // asymmetric: codes rint(v/s) + z clamped to [0, 15]; symmetric:
  // rint(v/s) clamped to [-8, 7], plus 8
  const float zf = SYM ? 8.0f : fminf(fmaxf(zq, 0.0f), 15.0f);
  const float qlo = SYM ? -8.0f : 0.0f, qhi = SYM ? 7.0f : 15.0f;
  uint32_t word = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float qf = SYM ? fminf(fmaxf(qv[i], qlo), qhi) + zf
                         : fminf(fmaxf(qv[i] + zf, qlo), qhi);
    word |= ((uint32_t)qf) << (4 * nibble_of_channel(i));
  }
  return QuantWord{word, sh, zf, sf == __builtin_inff() && most < __builtin_inff()};
}

}  // namespace awq
