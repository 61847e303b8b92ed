// Dense products of 16-bit operands: packing and entry (the kernels and the choice among them are in dense.hpp).
#include "dense.hpp"

namespace moe {
namespace {

// ---- packing --------------------------------------------------------------------------
// One thread: 8 consecutive k of one packed column (a lane slot of a fragment block).
template <typename ST, bool F16>
__global__ __launch_bounds__(256) void pack_dense_kernel(const ST* __restrict__ w, const ST* __restrict__ w_up, int N,
                                                         int K, int Kp, int gated, int cols, uint16_t* __restrict__ dst) {
    const int pc = blockIdx.x * 256 + threadIdx.x;
    const int k8 = blockIdx.y;
    if (pc >= cols) return;
    const int col = gated ? (pc >> 6) * 32 + (pc & 31) : pc;
    const ST* src = gated && (pc & 32) ? w_up : w;
    uint32_t v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int k = k8 * 8 + j;
        v[j] = 0;
        if (col < N && k < K) {
            const ST x = src[static_cast<int64_t>(k) * N + col];
            if constexpr (sizeof(ST) == 2) v[j] = x;
            else v[j] = f32_to_f16_or_nan(x);
        }
    }
    uint16_t* d = dst + ((static_cast<int64_t>(pc >> 6) * (Kp >> 4) + (k8 >> 1)) * 2 + ((pc >> 5) & 1)) * 512 +
                  ((pc & 31) + 32 * (k8 & 1)) * 8;
    *reinterpret_cast<u32x4*>(d) = u32x4{v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16};
}

}  // namespace

size_t dense_packed_bytes(const moe_dense_shape& s) {
    return static_cast<size_t>(pairs_of(s)) * k_padded<kBF16>(s) * 128;
}

int launch_pack_dense(const moe_dense_shape& s, const void* w, const void* w_up, int dtype, uint16_t* packed,
                      hipStream_t st) {
    const int cols = static_cast<int>(pairs_of(s) * 64), Kp = k_padded<kBF16>(s);
    const dim3 g((cols + 255) / 256, Kp / 8);
    if (dtype == MOE_F32)
        hipLaunchKernelGGL((pack_dense_kernel<float, true>), g, dim3(256), 0, st, static_cast<const float*>(w),
                           static_cast<const float*>(w_up), s.N, s.K, Kp, s.gated, cols, packed);
    else
        hipLaunchKernelGGL((pack_dense_kernel<uint16_t, false>), g, dim3(256), 0, st, static_cast<const uint16_t*>(w),
                           static_cast<const uint16_t*>(w_up), s.N, s.K, Kp, s.gated, cols, packed);
    MOE_CHECK_LAUNCH();
    return MOE_OK;
}

int launch_dense_gemm(const moe_dense_shape& s, const uint16_t* a, int a_dtype, int64_t lda, const uint16_t* packed,
                      int epilogue, const float* bias, const void* r, int r_dtype, int64_t ldr, void* c, int c_dtype,
                      int64_t ldc, hipStream_t st) {
    DenseArgs p = dense_args(s, epilogue, bias, r, r_dtype, ldr, c, c_dtype, ldc);
    p.a = a;
    p.b = packed;
    p.lda = lda * 2;
    p.Kh = s.K;
    p.Kp = k_padded<kBF16>(s);
    return a_dtype == MOE_F16 ? launch_dense<kF16>(p, pairs_of(s), st) : launch_dense<kBF16>(p, pairs_of(s), st);
}

}  // namespace moe
