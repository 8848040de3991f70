// Where the 4-bit key/value cache keeps a token's words, steps and zero points, and
// how its writers load 16-bit activations (kv_cache.hip, rope.hip).
#pragma once

#include "device_common.h"

namespace awq {

__device__ __forceinline__ float bf16_bits_to_float(uint32_t b) {
  return __builtin_bit_cast(float, b << 16);
}

template <bool BF16>
__device__ __forceinline__ void widen8(u32x4 raw, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t r = raw[i];
    v[2 * i] = BF16 ? bf16_bits_to_float(r & 0xFFFFu) : half_bits_to_float((uint16_t)(r & 0xFFFFu));
    v[2 * i + 1] = BF16 ? bf16_bits_to_float(r >> 16) : half_bits_to_float((uint16_t)(r >> 16));
  }
}
template <bool BF16>
__device__ __forceinline__ void load8(const uint16_t *p, float (&v)[8]) {
  widen8<BF16>(*reinterpret_cast<const u32x4 *>(p), v);
}

// Where slot s of head h keeps its words, and its step and zero point.
struct KvPlace {
  int64_t k_word, v_word, meta;
};
template <int D>
__device__ __forceinline__ KvPlace kv_place(int32_t slot, int pshift, int h, int heads, int word) {
  const int64_t page = slot >> pshift;
  const int64_t P = (int64_t)1 << pshift, off = slot & (P - 1);
  KvPlace p;
  const int64_t base = (page * 2 * heads + h) * P * (D / 8);
  p.k_word = base + off * (D / 8) + word;
  p.v_word = base + heads * P * (D / 8) + (off >> 2) * (D / 2) + word * 4 + (off & 3);
  p.meta = ((page * heads + h) * P + off) * 2;
  return p;
}

}  // namespace awq
