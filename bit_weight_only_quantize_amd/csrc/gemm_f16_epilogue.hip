// The GEMM (gemm_f16.h) with the epilogue of awq_linear_epilogue.

#include "gemm_f16.h"

namespace awq {

hipError_t launch_gemm_f16_epilogue(const uint16_t *X, const uint32_t *qweight,
                                    const uint16_t *scales, const uint8_t *zeros, int64_t M,
                                    int64_t N, int64_t K, int gs, void *Y, YType yt, int mt,
                                    SplitK sk, const float *rowf, const Epilogue &epi,
                                    hipStream_t st) {
  return f16_types<true>(X, qweight, scales, zeros, M, N, K, gs, Y, yt, mt, sk, rowf, epi, st);
}

}  // namespace awq
