// Dense products of int8 codes with a scale per row of A and per column of W:
//   C = act((sum_k a w) sa sw + bias) + R,   or, gated, with a gate and an up weight.
// The sums are int32 and exact (K is at most 131071, |a w| at most 2^14), so no order of them matters; the kernels
// are the 16-bit products' (dense.hpp), whose operands hold sixteen codes in the bytes of eight values.
//
// Packed weights: the 16-bit layout with a code in each byte, blocks of 32 columns x 32 k, K padded to a multiple of
// 128; then the columns' scales, padded to the packed columns (gated: the gate's, then the up's).
#include "dense.hpp"
#include "int8.hpp"

namespace moe {
namespace {

// Scales of 64 columns (int8 rule over K); 16 waves share the k out.
template <typename ST>
__device__ __forceinline__ float weight_at(const ST* w, int64_t i, int dtype) {
    if constexpr (sizeof(ST) == 4) return w[i];
    else return dtype == MOE_BF16 ? bf16_to_f32(w[i]) : f16_to_f32(w[i]);
}

template <typename ST>
__global__ __launch_bounds__(1024) void column_scales_kernel(const ST* __restrict__ w, int dtype, int N, int K,
                                                             float* __restrict__ scales) {
    __shared__ uint32_t s_most[16][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int col = blockIdx.x * 64 + lane;
    uint32_t most = 0;
    if (col < N)
        for (int k = wave; k < K; k += 16)
            most = max(most, abs_bits(weight_at(w, static_cast<int64_t>(k) * N + col, dtype)));
    s_most[wave][lane] = most;
    __syncthreads();
    if (wave != 0 || col >= N) return;
    for (int q = 1; q < 16; ++q) most = max(most, s_most[q][lane]);
    scales[col] = int8_scale(most);
}

// Scales beyond the columns are zero; given ones are copied.
__global__ __launch_bounds__(256) void copy_scales_kernel(const float* __restrict__ src, int N, int padded,
                                                          float* __restrict__ dst) {
    const int col = blockIdx.x * 256 + threadIdx.x;
    if (col >= padded) return;
    if (col >= N) dst[col] = 0.0f;
    else if (src != nullptr) dst[col] = src[col];
}

// One thread: 16 consecutive k of one packed column (a lane slot of a fragment block).
template <typename ST>
__global__ __launch_bounds__(256) void pack_dense_int8_kernel(const ST* __restrict__ w, const ST* __restrict__ w_up,
                                                              int dtype, const float* __restrict__ scales, int sb_up,
                                                              int N, int K, int Kp, int gated, int cols,
                                                              uint8_t* __restrict__ dst) {
    const int pc = blockIdx.x * 256 + threadIdx.x;
    const int k16 = blockIdx.y;
    if (pc >= cols) return;
    const bool up = gated && (pc & 32);
    const int col = gated ? (pc >> 6) * 32 + (pc & 31) : pc;
    const ST* src = up ? w_up : w;
    u32x4 v = {0u, 0u, 0u, 0u};
    float scale = 0.0f, inv = 0.0f;
    if (sizeof(ST) != 1 && col < N) {
        scale = scales[(up ? sb_up : 0) + col];
        inv = 1.0f / scale;
    }
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        const int k = k16 * 16 + j;
        if (col >= N || k >= K) continue;
        const int64_t i = static_cast<int64_t>(k) * N + col;
        uint32_t code;
        if constexpr (sizeof(ST) == 1) code = src[i];
        else code = scale == scale ? static_cast<uint32_t>(int8_code(weight_at(src, i, dtype), scale, inv)) & 0xFFu : 0u;
        v[j >> 2] |= code << (8 * (j & 3));
    }
    uint8_t* d = dst + ((static_cast<int64_t>(pc >> 6) * (Kp >> 4) + (k16 >> 1)) * 2 + ((pc >> 5) & 1)) * 1024 +
                 ((pc & 31) + 32 * (k16 & 1)) * 16;
    *reinterpret_cast<u32x4*>(d) = v;
}

inline size_t code_bytes(const moe_dense_shape& s) {
    return static_cast<size_t>(pairs_of(s)) * k_padded<kI8>(s) * 128;
}
inline int scales_per_weight(const moe_dense_shape& s) { return static_cast<int>(pairs_of(s) * (s.gated ? 32 : 64)); }

template <typename ST>
int pack(const moe_dense_shape& s, const void* w, const void* w_up, int dtype, const float* given,
         const float* up_given, uint8_t* packed, hipStream_t st) {
    const int cols = static_cast<int>(pairs_of(s) * 64), Kp = k_padded<kI8>(s), per = scales_per_weight(s);
    float* scales = reinterpret_cast<float*>(packed + code_bytes(s));
    for (int part = 0; part <= s.gated; ++part) {
        float* to = scales + part * per;
        hipLaunchKernelGGL(copy_scales_kernel, dim3((per + 255) / 256), dim3(256), 0, st, part ? up_given : given, s.N,
                           per, to);
        if constexpr (sizeof(ST) != 1)
            hipLaunchKernelGGL(column_scales_kernel<ST>, dim3((s.N + 63) / 64), dim3(1024), 0, st,
                               static_cast<const ST*>(part ? w_up : w), dtype, s.N, s.K, to);
    }
    hipLaunchKernelGGL(pack_dense_int8_kernel<ST>, dim3((cols + 255) / 256, Kp / 8), dim3(256), 0, st,
                       static_cast<const ST*>(w), static_cast<const ST*>(w_up), dtype, scales, per, s.N, s.K, Kp,
                       s.gated, cols, packed);
    MOE_CHECK_LAUNCH();
    return MOE_OK;
}

}  // namespace

size_t dense_int8_packed_bytes(const moe_dense_shape& s) {
    return code_bytes(s) + static_cast<size_t>(scales_per_weight(s)) * (s.gated ? 2 : 1) * sizeof(float);
}

int launch_pack_dense_int8(const moe_dense_shape& s, const void* w, const void* w_up, int dtype, const float* scales,
                           const float* up_scales, uint8_t* packed, hipStream_t st) {
    if (dtype == MOE_I8) return pack<uint8_t>(s, w, w_up, dtype, scales, up_scales, packed, st);
    if (dtype == MOE_F32) return pack<float>(s, w, w_up, dtype, nullptr, nullptr, packed, st);
    return pack<uint16_t>(s, w, w_up, dtype, nullptr, nullptr, packed, st);
}

int launch_dense_gemm_int8(const moe_dense_shape& s, const int8_t* a, int64_t lda, const float* a_scales,
                           const uint8_t* packed, int epilogue, const float* bias, const void* r, int r_dtype,
                           int64_t ldr, void* c, int c_dtype, int64_t ldc, hipStream_t st) {
    DenseArgs p = dense_args(s, epilogue, bias, r, r_dtype, ldr, c, c_dtype, ldc);
    p.a = reinterpret_cast<const uint16_t*>(a);
    p.b = reinterpret_cast<const uint16_t*>(packed);
    p.sa = a_scales;
    p.sb = reinterpret_cast<const float*>(packed + code_bytes(s));
    p.sb_up = scales_per_weight(s);
    p.lda = lda;
    p.Kh = s.K / 2;
    p.Kp = k_padded<kI8>(s);
    return launch_dense<kI8>(p, pairs_of(s), st);
}

}  // namespace moe
