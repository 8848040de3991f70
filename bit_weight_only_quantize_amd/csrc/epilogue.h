// The linear layer's epilogue on gfx950 (awq_linear_epilogue): per output
// element, act(sum + bias[n]) + residual[m][n] in fp32 before the one rounding
// to the output type.  The kernels take it as a compile-time variant, so the
// layer without one keeps its code.
#pragma once

#include <type_traits>

#include "awq_internal.h"
#include "device_common.h"

namespace awq {

// The kernels' epilogue argument: nothing where there is none (24 bytes more of
// arguments cost the single-token kernel 0.1 us).
struct NoEpilogue {
  __host__ __device__ NoEpilogue(const Epilogue &) {}
};
template <bool EPI>
using EpilogueArg = std::conditional_t<EPI, Epilogue, NoEpilogue>;

// Element i of an array of output type YT (bias and residual have Y's type).
template <int YT>
__device__ __forceinline__ float load_as(const void *p, int64_t i) {
  if constexpr (YT == (int)YType::F16)
    return half_bits_to_float(reinterpret_cast<const uint16_t *>(p)[i]);
  else if constexpr (YT == (int)YType::BF16)
    return __builtin_bit_cast(float, (uint32_t)reinterpret_cast<const uint16_t *>(p)[i] << 16);
  else
    return reinterpret_cast<const float *>(p)[i];
}
__device__ __forceinline__ float load_as(const void *p, int64_t i, int yt) {
  return yt == (int)YType::F16    ? load_as<(int)YType::F16>(p, i)
         : yt == (int)YType::BF16 ? load_as<(int)YType::BF16>(p, i)
                                  : load_as<(int)YType::F32>(p, i);
}

template <int YT>
__device__ __forceinline__ void store_as(void *p, int64_t i, float v) {
  if constexpr (YT == (int)YType::F16)
    reinterpret_cast<uint16_t *>(p)[i] = float_to_half_bits(v);
  else if constexpr (YT == (int)YType::BF16)
    reinterpret_cast<uint16_t *>(p)[i] = float_to_bf16_bits(v);
  else
    reinterpret_cast<float *>(p)[i] = v;
}
// Two 16-bit outputs as one word.
template <int YT>
__device__ __forceinline__ uint32_t pack_as(float a, float b) {
  if constexpr (YT == (int)YType::F16)
    return (uint32_t)float_to_half_bits(a) | ((uint32_t)float_to_half_bits(b) << 16);
  else
    return (uint32_t)float_to_bf16_bits(a) | ((uint32_t)float_to_bf16_bits(b) << 16);
}

// erfc(z) for z >= 0: e^(-z^2) t P(t), t = 1 / (1 + z/2).  P is a least-squares
// Chebyshev fit of erfc(z) e^(z^2) / t over t in (0, 1], good to 1.8e-7.  In fp32
// the exponent's roundings add up to z^2 2^-23, tail included, which 1 - erf(z)
// would lose: 4.6e-7 relative up to z = 1, 1.4e-6 up to 4, 7.9e-6 up to 9.3, the
// end of fp32's normal numbers.
__device__ __forceinline__ float erfc_nonneg(float z) {
  const float t = 1.0f / __builtin_fmaf(0.5f, z, 1.0f);
  constexpr float c[10] = {0.2820947468280792f, 0.28210368752479553f, 0.2465251237154007f,
                           0.18029476702213287f, 0.0588173009455204f, 0.07803553342819214f,
                           -0.19639277458190918f, 0.028879432007670403f, 0.06533099710941315f,
                           -0.02568896673619747f};
  float p = c[9];
#pragma unroll
  for (int i = 8; i >= 0; --i) p = __builtin_fmaf(p, t, c[i]);
  return p * t * __expf(-z * z);
}

// x / (1 + e^-z) is the sigmoid form of both SiLU (z = x) and the tanh form of
// GELU, 0.5 x (1 + tanh(y)) = x / (1 + e^-2y); e^-z overflows to infinity for
// very negative z, and the quotient is then the limit, 0.  GELU's 0.5 x (1 +
// erf(x / sqrt 2)) goes by erfc, so that small results keep their precision.
struct ActNone { __device__ __forceinline__ float operator()(float x) const { return x; } };
struct ActRelu { __device__ __forceinline__ float operator()(float x) const { return x < 0.0f ? 0.0f : x; } };
struct ActSilu { __device__ __forceinline__ float operator()(float x) const { return x / (1.0f + __expf(-x)); } };
struct ActGelu {
  __device__ __forceinline__ float operator()(float x) const {
    const float half = 0.5f * x * erfc_nonneg(__builtin_fabsf(x) * 0.70710678118654752f);
    return x < 0.0f ? half : x - __builtin_fminf(half, 1.0f);   // (half <= 0.17; inf * 0 at infinity)
  }
};
struct ActGeluTanh {
  __device__ __forceinline__ float operator()(float x) const {
    return x / (1.0f + __expf(-1.5957691216057308f * __builtin_fmaf(0.044715f * x * x, x, x)));
  }
};

// Calls f with the activation's function: the uniform choice is made once, not
// per element of a tile.
template <class F>
__device__ __forceinline__ void with_activation(Act act, F f) {
  switch (act) {
    case Act::Relu: return f(ActRelu{});
    case Act::Silu: return f(ActSilu{});
    case Act::Gelu: return f(ActGelu{});
    case Act::GeluTanh: return f(ActGeluTanh{});
    default: return f(ActNone{});
  }
}
__device__ __forceinline__ float activate(float x, Act act) {
  with_activation(act, [&](auto fn) { x = fn(x); });
  return x;
}

}  // namespace awq
