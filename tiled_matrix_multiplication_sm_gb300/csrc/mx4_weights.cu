// Product of BF16 rows with a kept 4-bit matrix.

#include "mx4_simt.h"

namespace tgemm {

cudaError_t mx4_weights(int M, int N, int K, const void* A, long lda, const Mx4Operand& B, int fmt,
                        const Mx4Out& out, int num_sms, cudaStream_t s) {
    if (K == 0) return mx4_empty_sum(M, N, out, s);
    if (M <= MX4_FEW_ROWS) return mx4_weights_rows(M, N, K, A, lda, B, fmt, out, num_sms, s);
    const Mx4Operand none{};
    return fmt == TGEMM_MXFP4 ? mx4_simt::launch<TGEMM_MXFP4, false>(M, N, K, none, A, lda, B, out, s)
                              : mx4_simt::launch<TGEMM_NVFP4, false>(M, N, K, none, A, lda, B, out, s);
}

}  // namespace tgemm
