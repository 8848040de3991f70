// The GEMM's plan and launcher, its bf16 row prescan and the search's loss GEMM
// (gemm_f16.h holds the kernel).

#include "gemm_f16.h"

namespace awq {

// Per-row activation factor for bf16 input: the power of two that brings the
// row's largest magnitude into [2^14, 2^15), so every value of the row is
// within fp16's range.  Scaled values of at least 2^-17 (every value at least
// 2^-31 times the row's largest) are fp16 numbers and keep their full 8-bit
// precision; smaller ones fall on fp16's subnormal grid (spacing 2^-24) and
// are truncated, with an absolute error below 2^-38 times the row's largest
// magnitude (exponent capped to stay a normal fp32); 1 for rows that are all
// zero or hold inf or NaN.  One workgroup per row.  With Xh, the row is also
// written there multiplied by its factor and converted to fp16 (round toward
// zero, as the GEMM's own staging does), for the 256-row tile.
__global__ __launch_bounds__(256) void bf16_row_factor_kernel(const uint16_t *__restrict__ X,
                                                              int K, float *__restrict__ rowf,
                                                              uint16_t *__restrict__ Xh) {
  __shared__ float red[4];
  __shared__ float fsh;
  const int64_t row = blockIdx.x;
  const rsrc_t rX = make_rsrc(X + row * K, (uint32_t)K * 2u);
  float mx = 0.0f;
  for (int c = threadIdx.x; c * 8 < K; c += 256) {
    const u32x4 v = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rX, (uint32_t)c * 16u, 0, 0));
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const uint32_t u = v[x];
      mx = __builtin_fmaxf(mx, __builtin_fabsf(__builtin_bit_cast(float, u << 16)));
      mx = __builtin_fmaxf(mx, __builtin_fabsf(__builtin_bit_cast(float, u & 0xFFFF0000u)));
    }
  }
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) mx = __builtin_fmaxf(mx, __shfl_xor(mx, off, 64));
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = mx;
  __syncthreads();
  if (threadIdx.x == 0) {
    const float m = __builtin_fmaxf(__builtin_fmaxf(red[0], red[1]), __builtin_fmaxf(red[2], red[3]));
    float f = 1.0f;
    if (m > 0.0f && __builtin_isfinite(m)) {
      // floor(log2 m) from the fp32 bits (bf16 subnormals widen to fp32
      // subnormals: biased exponent 0, read here as -127, so they scale up by
      // at most the cap)
      const int ex = (int)((__builtin_bit_cast(uint32_t, m) >> 23) & 0xFF) - 127;
      int e = 14 - ex;                                  // m * 2^e in [2^14, 2^15)
      e = e > 126 ? 126 : e;
      f = __builtin_bit_cast(float, (uint32_t)(127 + e) << 23);
    }
    rowf[row] = f;
    fsh = f;
  }
  if (!Xh) return;
  __syncthreads();
  const float f = fsh;
  const rsrc_t rH = make_rsrc(Xh + row * K, (uint32_t)K * 2u);
  for (int c = threadIdx.x; c * 8 < K; c += 256) {
    u32x4 v = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rX, (uint32_t)c * 16u, 0, 0));
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const uint32_t u = v[x];
      const float lo = __builtin_bit_cast(float, u << 16) * f;
      const float hi = __builtin_bit_cast(float, u & 0xFFFF0000u) * f;
      v[x] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pkrtz(lo, hi));
    }
    __builtin_amdgcn_raw_buffer_store_b128(v, rH, (uint32_t)c * 16u, 0, 0);
  }
}

// Row tile and K split.  M <= 32 and M <= 64 take 32- and 64-row tiles (the
// weight stream dominates there), larger M the 128-row tile, and shapes whose
// 256-row tiles fill every CU without a K split the 256-row tile (not for
// bf16 input under Scratch::Bounded, which has no room for its converted
// copy of X).  When the tiles cannot give every CU a workgroup, K is split
// (unless Scratch::None) into as many parts as still fit in one round (up to
// 8 with at least two K blocks each, up to 16 with at least four), with the
// fp32 partial tiles in the workspace.  bf16 input adds one fp32 activation
// factor per row, and with the 256-row tile its fp16 copy scaled by them.
GemmPlan gemm_f16_plan(int64_t M, int64_t N, int64_t K, bool bf16, Scratch sc) {
  GemmPlan p{};
  p.mt = M <= 32 ? 2 : M <= 64 ? 4 : 8;
  // 256-row tiles that alone fill every CU: the 256-row tile (each
  // dequantized weight then feeds 16 MFMAs instead of 8)
  if (K % kBK == 0 && ((M + 255) / 256) * ((N + kBN - 1) / kBN) >= kSlots &&
      !(bf16 && sc == Scratch::Bounded))
    p.mt = 16;
  const int64_t bm = 16 * p.mt;
  p.tiles = ((M + bm - 1) / bm) * ((N + kBN - 1) / kBN);
  const int64_t nkb = (K + kBK - 1) / kBK;
  p.splits = 1;
  if (p.tiles < kSlots && sc != Scratch::None) {
    int64_t sp = kSlots / p.tiles;
    // at least 2 K blocks per split up to 8 splits, at least 4 beyond (up to
    // 16): a split of few blocks is mostly pipeline fill and drain
    const int64_t c2 = nkb / 2 < 8 ? nkb / 2 : 8;
    const int64_t c4 = nkb / 4 < kMaxSplits ? nkb / 4 : kMaxSplits;
    const int64_t cap = c2 > c4 ? c2 : c4;
    sp = sp < cap ? sp : cap;
    p.splits = sp > 1 ? (int)sp : 1;
  }
  size_t bytes = 0;
  if (p.splits > 1) bytes = (size_t)p.tiles * p.splits * bm * kBN * 4;   // partials
  if (bf16) {
    p.rowf_offset = (bytes + 255) / 256 * 256;
    bytes = p.rowf_offset + (size_t)M * 4;
    if (p.mt == 16) {
      p.xh_offset = (bytes + 255) / 256 * 256;
      bytes = p.xh_offset + (size_t)M * (size_t)K * 2;
    }
  }
  p.workspace_bytes = bytes;
  return p;
}

hipError_t launch_gemm_f16(const uint16_t *X, bool bf16, const uint32_t *qweight,
                           const uint16_t *scales, const uint8_t *zeros, int64_t M, int64_t N,
                           int64_t K, int gs, void *Y, YType yt, const GemmPlan &p,
                           void *workspace, hipStream_t st, const Epilogue &epi) {
  if (M == 0 || N == 0) return hipSuccess;
  if (p.workspace_bytes > 0 && !workspace) return hipErrorInvalidValue;
  SplitK sk{1, nullptr};
  if (p.splits > 1) {
    sk.splits = p.splits;
    sk.partials = reinterpret_cast<float *>(workspace);
  }
  float *rowf = nullptr;
  if (bf16) {
    rowf = reinterpret_cast<float *>(reinterpret_cast<char *>(workspace) + p.rowf_offset);
    uint16_t *xh = p.xh_offset ? reinterpret_cast<uint16_t *>(reinterpret_cast<char *>(workspace) + p.xh_offset)
                               : nullptr;
    bf16_row_factor_kernel<<<dim3((unsigned)M), 256, 0, st>>>(X, (int)K, rowf, xh);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (xh) X = xh;
  }
  if (epi.any())
    return launch_gemm_f16_epilogue(X, qweight, scales, zeros, M, N, K, gs, Y, yt, p.mt, sk, rowf,
                                    epi, st);
  return f16_types<false>(X, qweight, scales, zeros, M, N, K, gs, Y, yt, p.mt, sk, rowf, epi, st);
}

// ---- the search's loss GEMM ------------------------------------------------------
int64_t gemm_tile_count(int64_t M, int64_t N) {
  return ((M + 127) / 128) * ((N + kBN - 1) / kBN);
}

template <int GS, bool KTAIL>
static hipError_t loss_go(const uint16_t *A, const uint32_t *qw, const uint16_t *sc,
                          const uint8_t *zr, int64_t M, int64_t N, int64_t K, const float *Yref,
                          double *partials, hipStream_t st) {
  constexpr int64_t bm = 128;
  const int64_t rows = f16_rows_per_launch(N, K, bm);
  if (rows <= 0) return hipErrorInvalidValue;
  int64_t tile_base = 0;
  for (int64_t m0 = 0; m0 < M; m0 += rows) {
    const int64_t mm = M - m0 < rows ? M - m0 : rows;
    const int64_t tiles = ((mm + bm - 1) / bm) * ((N + kBN - 1) / kBN);
    gemm_f16_kernel<GS, (int)YType::F32, 8, KTAIL, false, 1, 4><<<dim3((unsigned)tiles), 256, 0, st>>>(
        A + m0 * K, qw, sc, zr, (int)mm, (int)N, (int)K, nullptr, SplitK{1, nullptr},
        nullptr, Yref + m0 * N, partials + tile_base, Epilogue{});
    tile_base += tiles;
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_gemm_loss(const uint16_t *A, const uint32_t *qweight, const uint16_t *scales,
                            const uint8_t *zeros, int64_t M, int64_t N, int64_t K, int gs,
                            const float *Yref, double *partials, hipStream_t st) {
  if (M == 0 || N == 0) return hipSuccess;
  if (gs == 128) return loss_go<128, false>(A, qweight, scales, zeros, M, N, K, Yref, partials, st);
  if (K % kBK != 0) return loss_go<64, true>(A, qweight, scales, zeros, M, N, K, Yref, partials, st);
  return loss_go<64, false>(A, qweight, scales, zeros, M, N, K, Yref, partials, st);
}

}  // namespace awq
