// Product of two 4-bit matrices.

#include "mx4_simt.h"

namespace tgemm {

cudaError_t mx4_gemm(int M, int N, int K, const Mx4Operand& A, const Mx4Operand& B, int fmt,
                     const Mx4Out& out, int num_sms, cudaStream_t s) {
    return fmt == TGEMM_MXFP4 ? mx4_simt::launch<TGEMM_MXFP4, true>(M, N, K, A, nullptr, 0, B, out, s)
                              : mx4_simt::launch<TGEMM_NVFP4, true>(M, N, K, A, nullptr, 0, B, out, s);
}

}  // namespace tgemm
