// The tile GEMM of a linear layer: bias, activation and residual in the
// epilogue (kernels: gemm_kernel.h, gemm_fused_rb.h with EPI = kLinear).

#include "gemm_kernel.h"

namespace mq {

hipError_t launch_gemm_linear(int fmt, const uint16_t *X, int ldx, const void *W, int64_t ldw,
                              void *Y, int ldy, int M, int N, int K, const GemmPlan &plan,
                              float *ws, const EpiSpec &epi, hipStream_t stream) {
    return launch_gemm_epi<kLinear>(fmt, X, ldx, W, ldw, Y, ldy, M, N, K, plan, ws, epi, stream);
}

}  // namespace mq
