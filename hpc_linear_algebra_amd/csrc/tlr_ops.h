// Operators of language models: entry points behind include/tlrgemm.h (block.hip,
// moe.hip, int8.hip, experts.hip, gated.hip).
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
tlr_status row_quantize(tlr_dtype dt, int64_t rows, int64_t k, const void *X, int64_t x_rows, int64_t ldx, const int32_t *index,
                        void *codes, int64_t ldq, float *scales, void *stream);
tlr_status row_gemm_plan(int64_t m, int64_t n, int64_t k, int32_t groups, tlr_block_gemm_choice *out);
tlr_status row_gemm(tlr_dtype dt, int64_t m, int64_t n, int64_t k, const tlr_row_matrix *A, const tlr_row_matrix *B,
                    const tlr_row_groups *groups, void *C, int64_t ldc, void *ws, size_t ws_bytes, void *stream);
tlr_status row_linear_workspace(int64_t m, int64_t n, int64_t k, size_t *bytes);
tlr_status row_linear(tlr_dtype dt, int64_t m, int64_t n, int64_t k, const tlr_row_matrix *A, const void *X, int64_t ldx, void *C,
                      int64_t ldc, void *ws, size_t ws_bytes, void *stream);
tlr_status expert_sort_workspace(int64_t tokens, int32_t topk, int32_t experts, size_t *bytes);
tlr_status expert_sort(int32_t id_bytes, int64_t tokens, int32_t topk, int32_t experts, const void *ids, int32_t *offsets,
                       int32_t *place, int32_t *rows, void *ws, size_t ws_bytes, void *stream);
tlr_status expert_gather(tlr_dtype dt, int64_t tokens, int32_t topk, int64_t hidden, const void *X, int64_t ldx,
                         const int32_t *place, const int32_t *end, void *Y, int64_t ldy, void *stream);
tlr_status expert_combine(tlr_dtype dt, int64_t tokens, int32_t topk, int64_t hidden, const void *Y, int64_t ldy,
                          const int32_t *place, const int32_t *end, const float *weights, void *out, int64_t ldo, void *stream);
tlr_status expert_combine_grad(tlr_dtype dt, int64_t tokens, int32_t topk, int64_t hidden, const void *dout, int64_t ldd,
                               const void *Y, int64_t ldy, const int32_t *place, const int32_t *end, const float *weights,
                               void *dY, int64_t lddy, float *dweights, void *stream);
tlr_status gated(tlr_dtype dt, int64_t rows, int64_t inter, const void *X, int64_t ldx, void *Y, int64_t ldy, void *codes,
                 int64_t ldq, float *scales, int64_t lds, void *stream);
tlr_status gated_grad(tlr_dtype dt, int64_t rows, int64_t inter, const void *dY, int64_t lddy, const void *codes, int64_t ldq,
                      const float *scales, int64_t lds, void *dX, int64_t lddx, void *stream);

}  // namespace tlr

#endif  // TLR_OPS_H
