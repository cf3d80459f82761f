// Block-scaled 8-bit operators and the mixture-of-experts layer: entry points
// behind include/tlrgemm.h (block.hip, moe.hip).
#ifndef TLR_OPS_H
#define TLR_OPS_H

#include "tlr_plan.h"

namespace tlr {

tlr_status block_quantize(tlr_dtype dt, tlr_dtype fmt, int32_t block, int64_t rows, int64_t k, const void *X,
                          int64_t ldx, void *codes, int64_t ldq, float *scales, int64_t lds, void *codes_t,
                          int64_t ldq_t, float *scales_t, int64_t lds_t, void *stream);
tlr_status block_gemm_workspace(int64_t m, int64_t n, int64_t k, size_t *bytes);
tlr_status block_gemm_plan(int64_t m, int64_t n, int64_t k, uint32_t flags, tlr_block_gemm_choice *out);
tlr_status block_gemm(tlr_dtype dt, int64_t m, int64_t n, int64_t k, double alpha, const tlr_block_matrix *A,
                      const tlr_block_matrix *B, double beta, void *C, int64_t ldc, uint32_t flags, void *ws,
                      size_t ws_bytes, void *stream);
tlr_status moe_workspace(const tlr_moe_layer *layer, int32_t max_tokens, size_t *bytes);
tlr_status moe_init(const tlr_moe_layer *layer, void *ws, size_t ws_bytes, void *stream);
tlr_status moe(const tlr_moe_layer *layer, int32_t tokens, const void *X, int64_t ldx, void *Y, int64_t ldy,
               int32_t *ids, float *weights, void *ws, size_t ws_bytes, void *stream);

}  // namespace tlr

#endif  // TLR_OPS_H
