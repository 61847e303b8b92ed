// Launchers of the operators beside the staged layer: the layer for a few tokens
// and the dense products.
#pragma once

#include "common.hpp"

namespace moe {

// Dense products with a fused epilogue (dense.hip)
size_t dense_packed_bytes(const moe_dense_shape& s);
int launch_pack_dense(const moe_dense_shape& s, const void* w, const void* w_up, int dtype, uint16_t* packed,
                      hipStream_t st);
int launch_dense_gemm(const moe_dense_shape& s, const uint16_t* a, int a_dtype, int64_t lda, const uint16_t* packed,
                      int epilogue, const float* bias, const void* r, int r_dtype, int64_t ldr, void* c, int c_dtype,
                      int64_t ldc, hipStream_t st);

// The layer for a few tokens (few.hip)
struct FewWs {
    double* part;      // partial logits
    int32_t* idx;
    float* w;
    uint16_t* x;       // parts of float32 rows
    int* x_exp;        // exponents of those rows' scales
    uint16_t* h;       // parts of the weighted SwiGLU rows, at each level
    float* sums;       // partial sums of the down step
    int* arrived;      // their counters
    uint32_t* levels;  // levels of those rows' units, four to a word, and a word for all
};
// Whether the shape is within the few-token layer's limits.
bool few_tokens_fits(const moe_shape& s);
// Bytes of its workspace; with w, carves it from base.
size_t few_tokens_workspace(const moe_shape& s, void* base, FewWs* w);
int launch_few_tokens(const moe_shape& s, const void* x, int x_dtype, const void* w_router, const float* bias,
                      const void* packed, bool mx, float* out, int32_t* idx, float* tw, void* ws, hipStream_t st);

}  // namespace moe
