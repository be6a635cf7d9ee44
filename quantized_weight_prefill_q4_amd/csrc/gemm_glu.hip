// The tile GEMM of a gated layer: gate and up rows in one tile, combined in the
// epilogue (kernels: gemm_kernel.h, gemm_fused_rb.h with EPI = kGlu).

#include "gemm_kernel.h"

namespace mq {

hipError_t launch_gemm_glu(int fmt, const uint16_t *X, int ldx, const void *W, int64_t ldw,
                           void *Y, int ldy, int M, int N, int K, const GemmPlan &plan, float *ws,
                           const EpiSpec &epi, hipStream_t stream) {
    return launch_gemm_epi<kGlu>(fmt, X, ldx, W, ldw, Y, ldy, M, N, K, plan, ws, epi, stream);
}

}  // namespace mq
