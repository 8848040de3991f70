// Rotary positions on gfx950: queries and keys turned by angles that grow with
// their positions (awq_rope), alone or on the way into the 4-bit key/value cache
// (awq_kv_append_rope).
//
// Of each head's first R channels, pair j < R/2 is (a, b) = channels (j, j + R/2),
// or (2j, 2j + 1) where neighbours are paired:
//   a' = a c - b s,   b' = b c + a s,   c, s = factor * cos, sin(position * inv_freq_j).
// The angle is an fp64 product and so are its cosine and sine, to 2^-51 (cos_sin.h),
// rounded once to fp32: at position 2^20 an fp32 angle would be off by 2^-4.  The
// products and the sum are fp32, each rounded once and not fused, so what they give
// does not depend on the kernel, and the codes that a cache gets neither.
//
// A workgroup takes four tokens, computes their cosines and sines, one or two to a thread
// (LDS, 8 KiB at most), and walks heads.  A lane holds eight channels; paired halves are
// R/16 lanes apart and exchanged between lanes, so every channel is read once.  Queries: a wave
// per token, neighbouring heads side by side in its lanes, which is one run of memory.  Keys and
// values on their way into the cache: the four tokens of a head side by side, because their
// value words interleave.  Loads of the next heads are under way while some are turned,
// and the first before the angles are.
//
// Bound by memory: 4097 tokens, 32 and 8 heads of 128 of which 64 channels turn, 84 MB: 15.6 us, 5.4
// TB/s, a copy's rate (16 tokens to a workgroup, a wave on four tokens of one head: 20.0).  Into the
// cache 8192 tokens, 32 heads of 128 each, 304 MB: 78 us, 3.9 TB/s, its VALU 72% busy; 32 of 430
// VALU instructions per step fewer in the quantizer gave 1%, and neither twice the workgroups nor
// loads two heads ahead gave any.  Few tokens by a launch's latency and the chain of fp64 operations, about 32 per angle (32
// tokens: 5.8 us).

#include "awq_internal.h"
#include "cos_sin.h"
#include "device_common.h"
#include "kv_place.h"
#include "quant_group.h"

namespace awq {

constexpr int kRopeThreads = 256, kRopeTokens = 4;
constexpr int kRopePairs = kRopeTokens * kRopeMaxDim / 2;
constexpr int kRopeAhead = 4;                          // loads of a lane that are in flight together

// cos and sin of x, each times factor, rounded to fp32.
__device__ __forceinline__ float2 turn_by(double x, double factor) {
  double c, s;
  cos_sin(x, c, s);
  return float2{(float)(c * factor), (float)(s * factor)};
}

// What a lane does with its eight channels: out = own * c + partner * s.
struct Turn {
  float c[8], s[8];
  int from;              // the partner's lane (paired halves)
  uint32_t on;           // all bits where the channels are among the first R, else none
};

// Cosines and sines of the workgroup's tokens, from t0 on, into `table` [token][R/2].
__device__ __forceinline__ void fill_turns(const RopeArgs &p, int64_t t0, int64_t T, float2 *table) {
  const int half = p.rotary_dim / 2;
  for (int i = threadIdx.x; i < kRopeTokens * half; i += kRopeThreads) {
    const int t = i / half, j = i - t * half;
    const int64_t at = t0 + t < T ? t0 + t : T - 1;
    float2 cs = turn_by((double)p.positions[at] * p.inv_freq[j], p.factor);
    if (p.inverse) cs.y = -cs.y;
    table[i] = cs;
  }
}

// The lane's turn, of the token at place `token` of the workgroup's, channels 8w on.
template <bool PAIRS>
__device__ __forceinline__ Turn turn_of(const RopeArgs &p, const float2 *table, int token, int w, int lane) {
  Turn t;
  const int half = p.rotary_dim / 2, apart = half / 8;
  const bool on = w < 2 * apart, low = w < apart;
  t.on = on ? ~0u : 0u;
  t.from = lane + (on ? (low ? apart : -apart) : 0);
  const float2 *row = table + token * half;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int j = !on ? 0 : PAIRS ? 4 * w + i / 2 : 8 * (low ? w : w - apart) + i;
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
  // (chosen by bits: the compiler makes branches of a choice between a product and a value)
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t y = __builtin_bit_cast(uint32_t, v[i] * t.c[i] + other[i] * t.s[i]);
    v[i] = __builtin_bit_cast(float, (y & t.on) | (__builtin_bit_cast(uint32_t, v[i]) & ~t.on));
  }
}

// Rounded to nearest even; bfloat16 pairs by one instruction.
template <bool BF16>
__device__ __forceinline__ u32x4 narrow8(const float (&v)[8]) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  u32x4 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (BF16) r[i] = __builtin_bit_cast(uint32_t, bf16x2{(__bf16)v[2 * i], (__bf16)v[2 * i + 1]});
    else r[i] = __builtin_bit_cast(uint32_t, f16x2{(_Float16)v[2 * i], (_Float16)v[2 * i + 1]});
  }
  return r;
}

// Which heads a lane turns of a token: first, first + step, ... before `end`.
struct Heads {
  int first, step, end;
};
// Heads of part blockIdx.y of gridDim.y, `side` of them side by side, the lane's the `mine`-th.
__device__ __forceinline__ Heads heads_of(int heads, int side, int mine) {
  const int part = blockIdx.y, parts = gridDim.y;
  return Heads{(int)((int64_t)heads * part / parts) + mine, side, (int)((int64_t)heads * (part + 1) / parts)};
}

// A lane's channels of kRopeAhead of its heads, from x (its channels of head 0), D to a head.
struct Loaded {
  u32x4 raw[kRopeAhead];
  __device__ __forceinline__ void load(const uint16_t *x, int D, const Heads &hs, int h, bool active) {
#pragma unroll
    for (int i = 0; i < kRopeAhead; ++i) {
      raw[i] = u32x4{0u, 0u, 0u, 0u};
      const int at = h + i * hs.step;
      if (active && at < hs.end) raw[i] = *reinterpret_cast<const u32x4 *>(x + (int64_t)at * D);
    }
  }
};
// Heads from x to y; `l` holds the first ones.  x and y may be the same place: a lane reads a
// head's channels, its own and by exchange its partner's, before it writes them.
// The wave's lanes run as many steps as any of them needs (hs.first - mine is the same in all).
template <bool BF16, bool PAIRS>
__device__ __forceinline__ void turn_heads(const Turn &t, const uint16_t *x, uint16_t *y, int D, const Heads &hs, int mine,
                                           bool active, Loaded &l) {
  for (int h = hs.first; h - mine < hs.end;) {
    const int next = h + kRopeAhead * hs.step;
    Loaded more;
    more.load(x, D, hs, next, active);
#pragma unroll
    for (int i = 0; i < kRopeAhead; ++i) {
      float v[8];
      turn8<BF16, PAIRS>(t, l.raw[i], v);
      const int at = h + i * hs.step;
      if (active && at < hs.end) *reinterpret_cast<u32x4 *>(y + (int64_t)at * D) = narrow8<BF16>(v);
    }
    l = more;
    h = next;
  }
}

// How a wave's lanes lie over the heads of a token, D / 8 lanes each (D need not divide 512).
struct HeadLanes {
  int side, mine, w;     // heads side by side; the lane's; its channels are 8w on
  bool used;
  __device__ __forceinline__ HeadLanes(int D, int lane) {
    const int lanes = D / 8;
    side = 64 / lanes;
    used = lane < side * lanes;
    mine = used ? lane / lanes : 0;
    w = used ? lane - mine * lanes : 0;
  }
};

template <bool BF16, bool PAIRS>
__global__ __launch_bounds__(kRopeThreads) void rope_kernel(RopeArgs p, RopeArray q, RopeArray k, int64_t T, int D) {
  __shared__ float2 table[kRopePairs];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const HeadLanes at(D, lane);
  const int64_t t0 = (int64_t)blockIdx.x * kRopeTokens, t = t0 + wave;
  const bool active = at.used && t < T;
  const Heads qh = heads_of(q.heads, at.side, at.mine), kh = heads_of(k.heads, at.side, at.mine);
  const uint16_t *qx = q.x + t * q.x_stride + at.w * 8, *kx = k.x + t * k.x_stride + at.w * 8;
  Loaded lq, lk;
  lq.load(qx, D, qh, qh.first, active);
  fill_turns(p, t0, T, table);
  __syncthreads();
  const Turn turn = turn_of<PAIRS>(p, table, wave, at.w, lane);
  turn_heads<BF16, PAIRS>(turn, qx, q.y + t * q.y_stride + at.w * 8, D, qh, at.mine, active, lq);
  if (k.heads == 0) return;
  lk.load(kx, D, kh, kh.first, active);
  turn_heads<BF16, PAIRS>(turn, kx, k.y + t * k.y_stride + at.w * 8, D, kh, at.mine, active, lk);
}

template <int D, bool SYM, bool BF16, bool PAIRS>
__global__ __launch_bounds__(kRopeThreads) void kv_append_rope_kernel(
    RopeArgs p, RopeArray q, const uint16_t *__restrict__ K, const uint16_t *__restrict__ V, int64_t T, int heads,
    int64_t k_stride, int64_t v_stride, const int32_t *__restrict__ slots, int64_t num_slots, int pshift,
    uint32_t *__restrict__ codes, uint16_t *__restrict__ scales, uint8_t *__restrict__ zeros,
    int32_t *__restrict__ nonfinite) {
  constexpr int kLanes = D / 8, kSide = 64 / kLanes;
  __shared__ float2 table[kRopeTokens * D / 2];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, w = lane % kLanes;
  const int64_t t0 = (int64_t)blockIdx.x * kRopeTokens;
  // queries: wave's token, kSide heads; keys and values: four tokens of 256 / (4 kLanes) heads
  constexpr int kKvSide = kRopeThreads / (kRopeTokens * kLanes);
  const int64_t tq = t0 + wave;
  const int kv_token = (threadIdx.x / kLanes) % kRopeTokens, kv_mine = threadIdx.x / (kLanes * kRopeTokens);
  const int64_t t = t0 + kv_token;
  const int32_t slot = t < T ? slots[t] : -1;
  const Heads qh = heads_of(q.heads, kSide, lane / kLanes), kh = heads_of(heads, kKvSide, kv_mine);
  const uint16_t *qx = q.x + tq * q.x_stride + w * 8;
  Loaded l;
  l.load(qx, D, qh, qh.first, tq < T);
  // lanes of a group share their token, so a group is active as a whole
  const bool active = slot >= 0 && slot < num_slots;
  const uint16_t *kx = K + t * k_stride + w * 8, *vx = V + t * v_stride + w * 8;
  auto load_pair = [&](u32x4 &k, u32x4 &v, int h) {
    k = v = u32x4{0u, 0u, 0u, 0u};
    if (active && h < kh.end) {
      k = *reinterpret_cast<const u32x4 *>(kx + (int64_t)h * D);
      v = *reinterpret_cast<const u32x4 *>(vx + (int64_t)h * D);
    }
  };
  u32x4 kr, vr;
  load_pair(kr, vr, kh.first);
  fill_turns(p, t0, T, table);
  __syncthreads();
  if (q.heads > 0) {
    const Turn turn = turn_of<PAIRS>(p, table, wave, w, lane);
    turn_heads<BF16, PAIRS>(turn, qx, q.y + tq * q.y_stride + w * 8, D, qh, lane / kLanes, tq < T, l);
  }
  const Turn turn = turn_of<PAIRS>(p, table, kv_token, w, lane);
  int bad = 0;
  // (places of the lane's first head; the next ones' lie as far apart)
  KvPlace at = kv_place<D>(active ? slot : 0, pshift, kh.first, heads, w);
  const int64_t apart = (int64_t)kKvSide << pshift;
  for (int h = kh.first; h - kv_mine < kh.end; h += kKvSide) {
    u32x4 kn, vn;
    load_pair(kn, vn, h + kKvSide);
    float k[8], v[8];
    turn8<BF16, PAIRS>(turn, kr, k);
    widen8<BF16>(vr, v);
    kr = kn;
    vr = vn;
    const QuantWord qk = quantize_word<kLanes, SYM>(k, bad), qv = quantize_word<kLanes, SYM>(v, bad);
    const KvPlace here = at;
    at.k_word += apart * kLanes;
    at.v_word += apart * kLanes;
    at.meta += apart * 2;
    if (!active || h >= kh.end) continue;
    if (nonfinite != nullptr && w == 0) bad += (int)qk.overflow + (int)qv.overflow;
    codes[here.k_word] = qk.word;
    codes[here.v_word] = qv.word;
    if (w == 0) {
      *reinterpret_cast<uint32_t *>(scales + here.meta) =
          (uint32_t)__builtin_bit_cast(uint16_t, qk.step) | ((uint32_t)__builtin_bit_cast(uint16_t, qv.step) << 16);
      if constexpr (!SYM)
        *reinterpret_cast<uint16_t *>(zeros + here.meta) = (uint16_t)((uint32_t)qk.zero | ((uint32_t)qv.zero << 8));
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
// fewer than eight workgroups per CU, `side` heads each at least.
dim3 rope_grid(int64_t T, int heads, int side) {
  const int64_t along = (T + kRopeTokens - 1) / kRopeTokens, most = (heads + side - 1) / side;
  int64_t parts = (2048 + along - 1) / along;
  parts = parts < most ? parts : most;
  return dim3((unsigned)along, (unsigned)(parts < 1 ? 1 : parts));
}

template <int D, bool SYM, bool BF16>
hipError_t append_rope_go(const RopeArgs &p, const RopeArray &q, const uint16_t *K, const uint16_t *V, int64_t T,
                          int64_t ks, int64_t vs, const int32_t *slots, const KvCache &c, int32_t *nonfinite,
                          hipStream_t st) {
  const dim3 grid = rope_grid(T, q.heads > c.heads ? q.heads : c.heads, 64 / (D / 8));
  const int sh = __builtin_ctz((unsigned)c.page_size);
  const int64_t ns = c.pages * c.page_size;
  if (p.pairs) kv_append_rope_kernel<D, SYM, BF16, true><<<grid, kRopeThreads, 0, st>>>(p, q, K, V, T, c.heads, ks, vs, slots, ns, sh, c.codes, c.scales, c.zeros, nonfinite);
  else kv_append_rope_kernel<D, SYM, BF16, false><<<grid, kRopeThreads, 0, st>>>(p, q, K, V, T, c.heads, ks, vs, slots, ns, sh, c.codes, c.scales, c.zeros, nonfinite);
  return hipGetLastError();
}
}  // namespace

hipError_t launch_rope(const RopeArgs &p, const RopeArray &q, const RopeArray &k, XType xt, int64_t T, int D,
                       hipStream_t st) {
  const dim3 grid = rope_grid(T, q.heads > k.heads ? q.heads : k.heads, 64 / (D / 8));
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
