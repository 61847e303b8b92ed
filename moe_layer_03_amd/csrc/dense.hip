// Dense products with a fused epilogue, for the projections around the experts:
//   C = act(A W + bias) + R,   or, gated,   C = silu(A Wg + bg) * (A Wu + bu) + R,
// A [M, K] 16-bit, W [K, N] packed once, sums in float32, one rounding to C's type.
//
// Packed weights are the grouped GEMMs' fragment blocks of 32 columns x 16 k, K
// padded to a multiple of 64 and the columns to whole 64-column pairs (gated:
// 32 gate columns and the same 32 up columns to a pair, so a lane holds g and u
// of one output element); the padding is zero, so only A's reads need masks.
#include "stream.hpp"

namespace moe {
namespace {

struct DenseArgs {
    const uint16_t* a;
    const uint16_t* b;         // packed
    const float* bias;         // [N], gated [2][N], or NULL
    const void* r;             // residual, or NULL
    void* c;
    int64_t lda, ldr, ldc;
    int M, N, K, Kp;
    int gated, act, r_dtype, c_dtype;
};

// ---- epilogue ------------------------------------------------------------------

__device__ __forceinline__ float activate(float v, int act) {
    switch (act) {                                     // uniform
        case MOE_EPI_SILU: return v / (1.0f + expf(-v));
        case MOE_EPI_GELU: return 0.5f * v * erfcf(v * -0.70710678118654752f);
        // (1 + tanh z) / 2 = 1 / (1 + exp(-2 z)): no cancellation for negative z
        case MOE_EPI_GELU_TANH:
            return v / (1.0f + expf(-1.5957691216057308f * (v + 0.044715f * v * v * v)));
        case MOE_EPI_RELU: return fmaxf(v, 0.0f);
        default: return v;
    }
}

__device__ __forceinline__ float load_as(const void* p, int64_t i, int dtype) {
    if (dtype == MOE_F32) return static_cast<const float*>(p)[i];
    const uint16_t v = static_cast<const uint16_t*>(p)[i];
    return dtype == MOE_BF16 ? bf16_to_f32(v) : f16_to_f32(v);
}

__device__ __forceinline__ void store_as(void* p, int64_t i, int dtype, float v) {
    if (dtype == MOE_F32) static_cast<float*>(p)[i] = v;
    else static_cast<uint16_t*>(p)[i] = dtype == MOE_BF16 ? f32_to_bf16(v) : f32_to_f16_sat(v);
}

// The element (row, col): v is its sum (gated: the gate's, u the up's).  The
// residual is read by the thread that writes the element, so it may be C itself.
__device__ __forceinline__ void finish(const DenseArgs& p, int row, int col, float v, float u) {
    if (row >= p.M || col >= p.N) return;
    if (p.bias != nullptr) v += p.bias[col];
    if (p.gated) {
        if (p.bias != nullptr) u += p.bias[p.N + col];
        v = v / (1.0f + expf(-v)) * u;
    } else {
        v = activate(v, p.act);
    }
    if (p.r != nullptr) v += load_as(p.r, row * p.ldr + col, p.r_dtype);
    store_as(p.c, row * p.ldc + col, p.c_dtype, v);
}

// ---- any alignment -----------------------------------------------------------------
// 64 rows x one 64-column pair per workgroup of 4 waves; a wave owns 32 rows x
// 16 columns of each half.  A goes through LDS element by element, so rows may
// start at any address.
constexpr int kAnyLd = 40;                             // LDS row of 32 k, padded against bank conflicts

template <bool F16>
__global__ __launch_bounds__(256) void dense_any_kernel(DenseArgs p) {
    __shared__ __attribute__((aligned(16))) uint16_t s_a[64 * kAnyLd];
    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int pair = blockIdx.x, c0 = (wave & 1) * 16, r0 = (wave >> 1) * 32;
    const int row0 = blockIdx.y * 64;
    const uint8_t* b = reinterpret_cast<const uint8_t*>(p.b) + static_cast<int64_t>(pair) * (p.Kp / 32) * kStepBytes;
    const int o0 = step_lane_offset<false>(0, c0), o1 = step_lane_offset<false>(1, c0);
    floatx4 acc[2][2];
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i >> 1][i & 1] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
    const int lr = tid >> 2, lk = (tid & 3) * 8;       // this thread's 8 elements of a step
    for (int k0 = 0; k0 < p.K; k0 += 32) {
        uint16_t v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int row = row0 + lr, k = k0 + lk + j;
            v[j] = row < p.M && k < p.K ? p.a[row * p.lda + k] : uint16_t(0);
        }
        __syncthreads();                               // the last step's reads are done
#pragma unroll
        for (int j = 0; j < 8; ++j) s_a[lr * kAnyLd + lk + j] = v[j];
        __syncthreads();
        const uint8_t* bs = b + static_cast<int64_t>(k0 / 32) * kStepBytes;
        const u32x4 b0 = *reinterpret_cast<const u32x4*>(bs + o0), b1 = *reinterpret_cast<const u32x4*>(bs + o1);
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            const u32x4 a =
                *reinterpret_cast<const u32x4*>(&s_a[(r0 + m * 16 + (lane & 15)) * kAnyLd + (lane >> 4) * 8]);
            acc[m][0] = mfma16(F16, a, b0, acc[m][0]);
            acc[m][1] = mfma16(F16, a, b1, acc[m][1]);
        }
    }
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = row0 + r0 + m * 16 + (lane >> 4) * 4 + i, cc = c0 + (lane & 15);
            if (p.gated) {
                finish(p, row, pair * 32 + cc, acc[m][0][i], acc[m][1][i]);
            } else {
                finish(p, row, pair * 64 + cc, acc[m][0][i], 0.0f);
                finish(p, row, pair * 64 + 32 + cc, acc[m][1][i], 0.0f);
            }
        }
}

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
            else v[j] = f32_to_f16_sat(x);
        }
    }
    uint16_t* d = dst + ((static_cast<int64_t>(pc >> 6) * (Kp >> 4) + (k8 >> 1)) * 2 + ((pc >> 5) & 1)) * 512 +
                  ((pc & 31) + 32 * (k8 & 1)) * 8;
    *reinterpret_cast<u32x4*>(d) = u32x4{v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16};
}

inline int k_padded(const moe_dense_shape& s) { return static_cast<int>((static_cast<int64_t>(s.K) + 63) / 64 * 64); }
inline int64_t pairs_of(const moe_dense_shape& s) {
    const int w = s.gated ? 32 : 64;
    return (static_cast<int64_t>(s.N) + w - 1) / w;
}

}  // namespace

size_t dense_packed_bytes(const moe_dense_shape& s) {
    return static_cast<size_t>(pairs_of(s)) * k_padded(s) * 128;
}

int launch_pack_dense(const moe_dense_shape& s, const void* w, const void* w_up, int dtype, uint16_t* packed,
                      hipStream_t st) {
    const int cols = static_cast<int>(pairs_of(s) * 64), Kp = k_padded(s);
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
    DenseArgs p{};
    p.a = a;
    p.b = packed;
    p.bias = bias;
    p.r = r;
    p.c = c;
    p.lda = lda;
    p.ldr = ldr;
    p.ldc = ldc;
    p.M = s.M;
    p.N = s.N;
    p.K = s.K;
    p.Kp = k_padded(s);
    p.gated = s.gated;
    p.act = epilogue;
    p.r_dtype = r_dtype;
    p.c_dtype = c_dtype;
    const dim3 g(static_cast<unsigned>(pairs_of(s)), (s.M + 63) / 64);
    if (a_dtype == MOE_F16) hipLaunchKernelGGL((dense_any_kernel<true>), g, dim3(256), 0, st, p);
    else hipLaunchKernelGGL((dense_any_kernel<false>), g, dim3(256), 0, st, p);
    MOE_CHECK_LAUNCH();
    return MOE_OK;
}

}  // namespace moe
