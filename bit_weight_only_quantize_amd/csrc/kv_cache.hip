// The 4-bit paged key/value cache on gfx950: pages and slots for the tokens
// of a step (awq_kv_assign), quantizing new keys and values into their slots
// (awq_kv_append) and reading slots back (awq_kv_gather).
//
// Format (include/awq355.h has it in full): a token's key, and its value, of
// one head is one quantization group of D = 64 or 128 channels, quantized as
// awq_quantize_pack quantizes a weight group.  Keys keep a token's words
// together, [P][D/8]; values interleave four tokens, [P/4][D/8][4], so that
// one 16-byte load gives a lane the same eight channels of four tokens: the
// attention kernels need eight tokens of a channel side by side in a lane,
// and get them from two such loads with byte permutes instead of an exchange
// between lanes.  No word is shared by two tokens, so tokens are written
// without atomics.

#include "awq_internal.h"
#include "device_common.h"
#include "quant_group.h"

namespace awq {

// ---- pages and slots ---------------------------------------------------------------
// Request b holds old_b tokens in have_b = ceil(old_b / P) pages and gets new_b
// more: fresh pages have_b .. want_b - 1, want_b = ceil((old_b + new_b) / P),
// taken from the free list at first_b = sum over c < b of (want_c - have_c).
//
// One launch with no exchange between workgroups (which would cost more than
// the work): each workgroup scans the requests' lengths itself, in chunks of
// 1024 (both running sums in 64 bits), finds the tokens of its range by
// binary search in the chunk's starts in LDS, and stops when its range is
// done.  The lengths are a few KiB that stay in L2.  The token that opens a
// fresh page writes the page into the table; entries of pages that a request
// had before are only read, so no workgroup reads what another writes.
//
// Bound by latency: a launch, the lengths, two barriers, the table, the slots.
// Measured 4.0 us for 24 requests of one token each, 5.3 us for 500 requests and
// 16640 slots; there 256 slots to a workgroup took 5.1 us, 1024 took 8.0.
constexpr int kAssignThreads = 256;
constexpr int kAssignPer = 4;                               // requests per thread and chunk
constexpr int kAssignChunk = kAssignThreads * kAssignPer;
constexpr int kAssignTokens = 256;                          // slots per workgroup

__device__ __forceinline__ int32_t saturate32(int64_t v) {
  return v > 0x7FFFFFFF ? 0x7FFFFFFF : (int32_t)v;
}

__global__ __launch_bounds__(kAssignThreads) void kv_assign_kernel(
    const int32_t *__restrict__ old_lens, const int32_t *__restrict__ new_lens, int B, int pshift,
    int32_t *table, int max_blocks, const int32_t *__restrict__ free_pages, int num_free,
    int32_t *__restrict__ seq_lens, int32_t *__restrict__ query_start, int32_t *__restrict__ slots,
    int64_t num_slots, int32_t *__restrict__ pages_used) {
  __shared__ int64_t s_start[kAssignChunk + 1];             // first token of each request
  __shared__ int64_t s_first[kAssignChunk];                 // first fresh page in the free list
  __shared__ int32_t s_old[kAssignChunk];
  __shared__ int64_t s_wave[2][kAssignThreads / 64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t t_begin = (int64_t)blockIdx.x * kAssignTokens;
  const int64_t t_end = t_begin + kAssignTokens < num_slots ? t_begin + kAssignTokens : num_slots;
  const int64_t round = ((int64_t)1 << pshift) - 1;
  int64_t tok_base = 0, page_base = 0;
  const int chunks = B > 0 ? (B + kAssignChunk - 1) / kAssignChunk : 1;
  // the lengths and starts of chunk c are workgroup c mod gridDim.x's to write
  const int wgs = (int)gridDim.x, me = (int)blockIdx.x;
  const int last_own = me < chunks ? me + (chunks - 1 - me) / wgs * wgs : -1;
  for (int ch = 0; ch < chunks; ++ch) {
    const bool writer = ch % wgs == me;
    const int b0 = ch * kAssignChunk + tid * kAssignPer;
    int64_t o[kAssignPer], n[kAssignPer], tok = 0, pg = 0, tok_at[kAssignPer], pg_at[kAssignPer];
#pragma unroll
    for (int i = 0; i < kAssignPer; ++i) {
      o[i] = b0 + i < B ? old_lens[b0 + i] : 0;
      n[i] = b0 + i < B ? new_lens[b0 + i] : 0;
    }
#pragma unroll
    for (int i = 0; i < kAssignPer; ++i) {
      o[i] = o[i] > 0 ? o[i] : 0;
      n[i] = n[i] > 0 ? n[i] : 0;
      tok_at[i] = tok;
      pg_at[i] = pg;
      tok += n[i];
      pg += ((o[i] + n[i] + round) >> pshift) - ((o[i] + round) >> pshift);
    }
    int64_t ts = tok, ps = pg;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int64_t a = __shfl_up(ts, d, 64), b = __shfl_up(ps, d, 64);
      if (lane >= d) {
        ts += a;
        ps += b;
      }
    }
    if (lane == 63) {
      s_wave[0][wave] = ts;
      s_wave[1][wave] = ps;
    }
    __syncthreads();
    int64_t tb = tok_base + ts - tok, pb = page_base + ps - pg, tok_all = 0, page_all = 0;
#pragma unroll
    for (int w = 0; w < kAssignThreads / 64; ++w) {
      if (w < wave) {
        tb += s_wave[0][w];
        pb += s_wave[1][w];
      }
      tok_all += s_wave[0][w];
      page_all += s_wave[1][w];
    }
#pragma unroll
    for (int i = 0; i < kAssignPer; ++i) {
      const int j = tid * kAssignPer + i;
      s_start[j] = tb + tok_at[i];
      s_first[j] = pb + pg_at[i];
      s_old[j] = (int32_t)o[i];
      if (writer && b0 + i < B) {
        seq_lens[b0 + i] = saturate32(o[i] + n[i]);
        query_start[b0 + i] = saturate32(tb + tok_at[i]);
      }
    }
    tok_base += tok_all;
    page_base += page_all;
    if (tid == 0) s_start[kAssignChunk] = tok_base;
    if (writer && ch == chunks - 1 && tid == 0) {
      query_start[B] = saturate32(tok_base);
      *pages_used = saturate32(page_base);
    }
    __syncthreads();
    // the tokens of this workgroup's range that belong to the chunk's requests
    const int64_t lo = s_start[0] > t_begin ? s_start[0] : t_begin;
    const int64_t hi = tok_base < t_end ? tok_base : t_end;
    for (int64_t t = lo + tid; t < hi; t += kAssignThreads) {
      int a = 0, z = kAssignChunk;                          // start[a] <= t < start[z]
      while (z - a > 1) {
        const int m = (a + z) >> 1;
        if (s_start[m] <= t) a = m; else z = m;
      }
      const int64_t old = s_old[a], pos = old + (t - s_start[a]);
      const int64_t block = pos >> pshift, have = (old + round) >> pshift;
      int64_t page = -1;
      if (block < max_blocks) {
        int32_t *entry = table + (int64_t)(ch * kAssignChunk + a) * max_blocks + block;
        if (block < have) {
          page = *entry;
        } else {
          const int64_t at = s_first[a] + block - have;
          if (at < num_free) page = free_pages[at];
          if ((pos & round) == 0) *entry = (int32_t)page;
        }
      }
      const int64_t slot = (page << pshift) + (pos & round);
      slots[t] = page >= 0 && slot <= 0x7FFFFFFF ? (int32_t)slot : -1;
    }
    __syncthreads();                                        // before the next chunk overwrites LDS
    // done: the range's tokens are written, and no later chunk is this workgroup's to report
    if (tok_base >= t_end && ch >= last_own) break;
  }
  // slots behind the last request's tokens
  const int64_t pad = tok_base > t_begin ? tok_base : t_begin;
  for (int64_t t = pad + tid; t < t_end; t += kAssignThreads) slots[t] = -1;
}

hipError_t launch_kv_assign(const int32_t *old_lens, const int32_t *new_lens, int B, int page_size,
                            int32_t *table, int max_blocks, const int32_t *free_pages, int num_free,
                            int32_t *seq_lens, int32_t *query_start, int32_t *slots,
                            int64_t num_slots, int32_t *pages_used, hipStream_t st) {
  int64_t wgs = (num_slots + kAssignTokens - 1) / kAssignTokens;
  if (wgs < 1) wgs = 1;                                     // lengths and starts are written anyway
  kv_assign_kernel<<<(unsigned)wgs, kAssignThreads, 0, st>>>(
      old_lens, new_lens, B, __builtin_ctz((unsigned)page_size), table, max_blocks, free_pages,
      num_free, seq_lens, query_start, slots, num_slots, pages_used);
  return hipGetLastError();
}

// ---- append and gather -----------------------------------------------------------------
// One lane per word of eight channels, for the key and the value alike; D/8
// lanes make a token's group, so a wave holds 4 (D = 128) or 8 (D = 64)
// consecutive tokens of one head.  Where those tokens sit in consecutive
// slots, as a prompt's do, the wave's key words are one run of 256 bytes, and
// so are its value words (four tokens to each 16 bytes).
//
// Bound by memory.  8192 tokens of 32 heads of 128, fp16: the append (reads
// 134 MB, writes 36) takes 42 - 49 us, 3.5 - 4.0 TB/s; the gather into fp16, the
// other way round, 29 - 35 us, 4.9 - 5.9 TB/s.  32 tokens of 8 heads: 3.8 and
// 3.2 us, a launch's latency.
__device__ __forceinline__ float bf16_bits_to_float(uint32_t b) {
  return __builtin_bit_cast(float, b << 16);
}

template <bool BF16>
__device__ __forceinline__ void load8(const uint16_t *p, float (&v)[8]) {
  const u32x4 raw = *reinterpret_cast<const u32x4 *>(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t r = raw[i];
    v[2 * i] = BF16 ? bf16_bits_to_float(r & 0xFFFFu) : half_bits_to_float((uint16_t)(r & 0xFFFFu));
    v[2 * i + 1] = BF16 ? bf16_bits_to_float(r >> 16) : half_bits_to_float((uint16_t)(r >> 16));
  }
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

template <int D, bool SYM, bool BF16>
__global__ __launch_bounds__(256) void kv_append_kernel(
    const uint16_t *__restrict__ K, const uint16_t *__restrict__ V, int64_t T, int heads,
    int64_t k_stride, int64_t v_stride, const int32_t *__restrict__ slots, int64_t num_slots,
    int pshift, uint32_t *__restrict__ codes, uint16_t *__restrict__ scales,
    uint8_t *__restrict__ zeros, int32_t *__restrict__ nonfinite) {
  constexpr int kLanes = D / 8, kTokens = 256 / kLanes;     // tokens per workgroup
  const int word = threadIdx.x % kLanes;
  const int64_t t = (int64_t)blockIdx.x * kTokens + threadIdx.x / kLanes;
  const int32_t slot = t < T ? slots[t] : -1;
  // lanes of a group share their token, so a group is active as a whole
  const bool active = slot >= 0 && slot < num_slots;
  int bad = 0;
  for (int h = blockIdx.y; h < heads; h += gridDim.y) {
    float k[8] = {}, v[8] = {};
    if (active) {
      load8<BF16>(K + t * k_stride + (int64_t)h * D + word * 8, k);
      load8<BF16>(V + t * v_stride + (int64_t)h * D + word * 8, v);
    }
    const QuantWord qk = quantize_word<kLanes, SYM>(k, bad), qv = quantize_word<kLanes, SYM>(v, bad);
    if (!active) continue;
    if (nonfinite != nullptr && word == 0) bad += (int)qk.overflow + (int)qv.overflow;
    const KvPlace p = kv_place<D>(slot, pshift, h, heads, word);
    codes[p.k_word] = qk.word;
    codes[p.v_word] = qv.word;
    if (word == 0) {
      *reinterpret_cast<uint32_t *>(scales + p.meta) =
          (uint32_t)__builtin_bit_cast(uint16_t, qk.step) |
          ((uint32_t)__builtin_bit_cast(uint16_t, qv.step) << 16);
      if constexpr (!SYM)
        *reinterpret_cast<uint16_t *>(zeros + p.meta) =
            (uint16_t)((uint32_t)qk.zero | ((uint32_t)qv.zero << 8));
    }
  }
  if (nonfinite != nullptr) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) bad += __shfl_xor(bad, off, 64);
    if ((threadIdx.x & 63) == 0 && bad) atomicAdd(nonfinite, bad);
  }
}

template <int D, int OT>
__global__ __launch_bounds__(256) void kv_gather_kernel(
    const uint32_t *__restrict__ codes, const uint16_t *__restrict__ scales,
    const uint8_t *__restrict__ zeros, int pshift, const int32_t *__restrict__ slots,
    int64_t num_slots, int64_t T, int heads, void *__restrict__ K, void *__restrict__ V) {
  constexpr int kLanes = D / 8, kTokens = 256 / kLanes;
  const int word = threadIdx.x % kLanes;
  const int64_t t = (int64_t)blockIdx.x * kTokens + threadIdx.x / kLanes;
  if (t >= T) return;
  const int32_t slot = slots[t];
  const bool held = slot >= 0 && slot < num_slots;
  for (int h = blockIdx.y; h < heads; h += gridDim.y) {
    uint32_t w[2] = {0u, 0u}, sc = 0u, z = 0u;
    if (held) {
      const KvPlace p = kv_place<D>(slot, pshift, h, heads, word);
      w[0] = codes[p.k_word];
      w[1] = codes[p.v_word];
      sc = *reinterpret_cast<const uint32_t *>(scales + p.meta);
      z = zeros ? *reinterpret_cast<const uint16_t *>(zeros + p.meta) : 0x0808u;
    }
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      const float s = half_bits_to_float((uint16_t)(sc >> (16 * kv)));
      const float zf = (float)((z >> (8 * kv)) & 0xFFu);
      const uint32_t cw = w[kv];
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        v[i] = held ? ((float)((cw >> (4 * nibble_of_channel(i))) & 0xFu) - zf) * s : 0.0f;
      const int64_t o = (t * heads + h) * D + word * 8;
      void *out = kv ? V : K;
      if constexpr (OT == (int)YType::F32) {
        float4 *q = reinterpret_cast<float4 *>(reinterpret_cast<float *>(out) + o);
        q[0] = float4{v[0], v[1], v[2], v[3]};
        q[1] = float4{v[4], v[5], v[6], v[7]};
      } else {
        u32x4 r;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t lo = OT == (int)YType::F16 ? float_to_half_bits(v[2 * i]) : float_to_bf16_bits(v[2 * i]);
          const uint32_t hi = OT == (int)YType::F16 ? float_to_half_bits(v[2 * i + 1]) : float_to_bf16_bits(v[2 * i + 1]);
          r[i] = lo | (hi << 16);
        }
        *reinterpret_cast<u32x4 *>(reinterpret_cast<uint16_t *>(out) + o) = r;
      }
    }
  }
}

namespace {
template <int D>
dim3 kv_grid(int64_t T, int heads) {
  return dim3((unsigned)((T + 256 / (D / 8) - 1) / (256 / (D / 8))), (unsigned)heads);
}

template <int D>
hipError_t append_go(const uint16_t *K, const uint16_t *V, bool bf16, int64_t T, int64_t ks,
                     int64_t vs, const int32_t *slots, const KvCache &c, int32_t *nonfinite,
                     hipStream_t st) {
  const dim3 grid = kv_grid<D>(T, c.heads);
  const int sh = __builtin_ctz((unsigned)c.page_size);
  const int64_t ns = c.pages * c.page_size;
  if (c.zeros) {
    if (bf16) kv_append_kernel<D, false, true><<<grid, 256, 0, st>>>(K, V, T, c.heads, ks, vs, slots, ns, sh, c.codes, c.scales, c.zeros, nonfinite);
    else kv_append_kernel<D, false, false><<<grid, 256, 0, st>>>(K, V, T, c.heads, ks, vs, slots, ns, sh, c.codes, c.scales, c.zeros, nonfinite);
  } else {
    if (bf16) kv_append_kernel<D, true, true><<<grid, 256, 0, st>>>(K, V, T, c.heads, ks, vs, slots, ns, sh, c.codes, c.scales, c.zeros, nonfinite);
    else kv_append_kernel<D, true, false><<<grid, 256, 0, st>>>(K, V, T, c.heads, ks, vs, slots, ns, sh, c.codes, c.scales, c.zeros, nonfinite);
  }
  return hipGetLastError();
}

template <int D>
hipError_t gather_go(const KvCache &c, const int32_t *slots, int64_t T, void *K, void *V, YType ot,
                     hipStream_t st) {
  const dim3 grid = kv_grid<D>(T, c.heads);
  const int sh = __builtin_ctz((unsigned)c.page_size);
  const int64_t ns = c.pages * c.page_size;
  if (ot == YType::F32) kv_gather_kernel<D, (int)YType::F32><<<grid, 256, 0, st>>>(c.codes, c.scales, c.zeros, sh, slots, ns, T, c.heads, K, V);
  else if (ot == YType::BF16) kv_gather_kernel<D, (int)YType::BF16><<<grid, 256, 0, st>>>(c.codes, c.scales, c.zeros, sh, slots, ns, T, c.heads, K, V);
  else kv_gather_kernel<D, (int)YType::F16><<<grid, 256, 0, st>>>(c.codes, c.scales, c.zeros, sh, slots, ns, T, c.heads, K, V);
  return hipGetLastError();
}
}  // namespace

hipError_t launch_kv_append(const uint16_t *K, const uint16_t *V, XType xt, int64_t T,
                            int64_t k_stride, int64_t v_stride, const int32_t *slots,
                            const KvCache &c, int32_t *nonfinite, hipStream_t st) {
  const bool bf16 = xt == XType::BF16;
  if (c.head_dim == 128) return append_go<128>(K, V, bf16, T, k_stride, v_stride, slots, c, nonfinite, st);
  return append_go<64>(K, V, bf16, T, k_stride, v_stride, slots, c, nonfinite, st);
}

hipError_t launch_kv_gather(const KvCache &c, const int32_t *slots, int64_t T, void *K, void *V,
                            YType ot, hipStream_t st) {
  if (c.head_dim == 128) return gather_go<128>(c, slots, T, K, V, ot, st);
  return gather_go<64>(c, slots, T, K, V, ot, st);
}

}  // namespace awq
