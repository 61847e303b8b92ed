// Rows on their way into a product: the norm with the residual's sum,
//   h = x + residual (rounded to the residual's type),   s = 1 / sqrt(mean(h^2) + eps),   v = (h s) w,
// and the codes of v, or of rows given, in 8 bits: int8 with a scale per row, MXFP8 with one per 32.
//
// The mean and s are computed in double and s is rounded to float32; v takes two float32 products.  A double sum
// differs by 2^-50 or so from one order of summation to another, which moves the rounded s once in millions of
// rows; so v, and the codes, which turn on which side of a half a quotient lies, do not depend on the order, nor on
// the kernel's shape.  The conversion and the double fma of an element cost what two float32 operations do.
#include "block.hpp"
#include "int8.hpp"
#include "stream.hpp"

namespace moe {
namespace {

struct RowArgs {
    const void *x, *r, *w;     // w, r or NULL
    void *sum, *y;             // or NULL
    uint8_t* codes;            // or NULL
    void* scales;
    int64_t ldx, ldr, lds, ldy, ldq;
    double eps;
    int H;
    int x_dtype, r_dtype, w_dtype, y_dtype, q_dtype;
};

// Eight elements at an element's alignment (the hardware takes unaligned addresses).
typedef u32x4 u32x4_at2 __attribute__((aligned(2)));
typedef floatx4 floatx4_at4 __attribute__((aligned(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef u32x2 u32x2_at1 __attribute__((aligned(1)));

// Elements k .. k + 7 of a row at p, n of which exist (at least one); the rest are zero.
template <int B>
__device__ __forceinline__ void load8(const void* p, int k, int n, bool bf16, float (&v)[8]) {
    if constexpr (B == 4) {
        const float* f = static_cast<const float*>(p) + k;
        if (n >= 8) {
            const floatx4 a = *reinterpret_cast<const floatx4_at4*>(f), b = *reinterpret_cast<const floatx4_at4*>(f + 4);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[j] = a[j];
                v[4 + j] = b[j];
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = j < n ? f[j] : 0.0f;
        }
    } else {
        const uint16_t* h = static_cast<const uint16_t*>(p) + k;
        uint32_t u[4];
        if (n >= 8) {
            const u32x4 a = *reinterpret_cast<const u32x4_at2*>(h);
#pragma unroll
            for (int j = 0; j < 4; ++j) u[j] = a[j];
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                u[j] = (2 * j < n ? h[2 * j] : 0u) | (2 * j + 1 < n ? static_cast<uint32_t>(h[2 * j + 1]) << 16 : 0u);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[2 * j] = bf16 ? __uint_as_float(u[j] << 16) : f16_to_f32(static_cast<uint16_t>(u[j]));
            v[2 * j + 1] = bf16 ? __uint_as_float(u[j] & 0xFFFF0000u) : f16_to_f32(static_cast<uint16_t>(u[j] >> 16));
        }
    }
}

__device__ __forceinline__ void load8_as(const void* p, int k, int n, int dtype, float (&v)[8]) {
    if (dtype == MOE_F32) load8<4>(p, k, n, false, v);
    else load8<2>(p, k, n, dtype == MOE_BF16, v);
}

__device__ __forceinline__ void store8_as(void* p, int k, int n, int dtype, const float (&v)[8]) {
    if (dtype == MOE_F32) {
        float* f = static_cast<float*>(p) + k;
        if (n >= 8) {
            *reinterpret_cast<floatx4_at4*>(f) = floatx4{v[0], v[1], v[2], v[3]};
            *reinterpret_cast<floatx4_at4*>(f + 4) = floatx4{v[4], v[5], v[6], v[7]};
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j < n) f[j] = v[j];
        }
        return;
    }
    uint16_t* h = static_cast<uint16_t*>(p) + k;
    u32x4 u;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        u[j] = dtype == MOE_BF16 ? pack_bf16x2_or_nan(v[2 * j], v[2 * j + 1])
                                 : f32_to_f16_or_nan(v[2 * j]) | static_cast<uint32_t>(f32_to_f16_or_nan(v[2 * j + 1])) << 16;
    if (n >= 8) {
        *reinterpret_cast<u32x4_at2*>(h) = u;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < n) h[j] = static_cast<uint16_t>(u[j >> 1] >> (16 * (j & 1)));
    }
}

__device__ __forceinline__ void store8_codes(uint8_t* p, int k, int n, u32x2 u) {
    if (n >= 8) {
        *reinterpret_cast<u32x2_at1*>(p + k) = u;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < n) p[k + j] = static_cast<uint8_t>(u[j >> 2] >> (8 * (j & 3)));
    }
}

__device__ __forceinline__ float round_as(float v, int dtype) {
    if (dtype == MOE_F32) return v;
    return dtype == MOE_BF16 ? bf16_to_f32(f32_to_bf16_or_nan(v)) : f16_to_f32(f32_to_f16_or_nan(v));
}

__device__ __forceinline__ uint32_t most_of(const float (&v)[8]) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, abs_bits(v[j]));
    return m;
}

// ---- int8 ----------------------------------------------------------------------
__device__ __forceinline__ u32x2 int8_codes(const float (&v)[8], float scale, float inv) {
    u32x2 u = {0u, 0u};
    if (scale != scale) return u;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        u[j >> 2] |= (static_cast<uint32_t>(int8_code(v[j], scale, inv)) & 0xFFu) << (8 * (j & 3));
    }
    return u;
}

// ---- MXFP8 ---------------------------------------------------------------------
// Shared exponent floor(log2 amax) - 8 in [-127, 127]; codes v / 2^shared to the nearest E4M3 value, ties to even,
// saturating: the conversion instruction's rounding, after a clamp (the division is exact but where it is far below
// the least code).  A block with an infinity or NaN has the scale byte 255 and NaN codes.
__device__ __forceinline__ int mx_scale_byte(uint32_t most) {
    return most >= kInfBits ? 255 : max(static_cast<int>(most >> 23) - 8, 0);
}

__device__ __forceinline__ u32x2 mx_codes(const float (&v)[8], int byte) {
    if (byte == 255) return u32x2{0x7F7F7F7Fu, 0x7F7F7F7Fu};
    const float inv = __uint_as_float(static_cast<uint32_t>(254 - byte) << 23);   // byte <= 246: normal
    u32x2 u;
#pragma unroll
    for (int g = 0; g < 2; ++g) {
        float c[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) c[j] = fminf(fmaxf(v[4 * g + j] * inv, -448.0f), 448.0f);
        int w = __builtin_amdgcn_cvt_pk_fp8_f32(c[0], c[1], 0, false);
        w = __builtin_amdgcn_cvt_pk_fp8_f32(c[2], c[3], w, true);
        u[g] = static_cast<uint32_t>(w);
    }
    return u;
}

// ---- a row over a workgroup ------------------------------------------------------
template <typename V, int T, typename Op>
__device__ __forceinline__ V over_row(V v, V* s, Op&& op) {
#pragma unroll
    for (int off = 1; off < kWave; off <<= 1) v = op(v, __shfl_xor(v, off, kWave));
    if constexpr (T > kWave) {
        const int wave = threadIdx.x >> 6;
        if ((threadIdx.x & (kWave - 1)) == 0) s[wave] = v;
        __syncthreads();
        v = s[0];
#pragma unroll
        for (int q = 1; q < T / kWave; ++q) v = op(v, s[q]);
    }
    return v;
}

// One row per workgroup of T threads, eight elements a thread at a time; the row is read again for each pass: once
// for the sum of squares, once for the largest |v| (int8), once for the codes.  Passes after the first read h from
// `sum` where it is written (each thread what it wrote itself), since that may lie over x or the residual.
template <bool NORM, int T>
__global__ __launch_bounds__(T) void rows_kernel(RowArgs p) {
    __shared__ double s_sum[T / kWave];
    __shared__ uint32_t s_max[T / kWave];
    const int64_t row = blockIdx.x;
    const int tid = threadIdx.x;
    auto at = [&](const void* base, int64_t ld, int dtype) {
        return static_cast<const uint8_t*>(base) + row * ld * (dtype == MOE_F32 ? 4 : 2);
    };
    const void* x = at(p.x, p.ldx, p.x_dtype);
    const void* r = at(p.r, p.ldr, p.r_dtype);
    void* sum = const_cast<uint8_t*>(at(p.sum, p.lds, p.r_dtype));
    void* y = const_cast<uint8_t*>(at(p.y, p.ldy, p.y_dtype));
    uint8_t* codes = p.codes + row * p.ldq;
    auto load_h = [&](int k, float (&h)[8], bool again) {
        const int n = p.H - k;
        if (again && p.sum != nullptr) {
            load8_as(sum, k, n, p.r_dtype, h);
            return;
        }
        load8_as(x, k, n, p.x_dtype, h);
        if (NORM && p.r != nullptr) {
            float a[8];
            load8_as(r, k, n, p.r_dtype, a);
#pragma unroll
            for (int j = 0; j < 8; ++j) h[j] = round_as(h[j] + a[j], p.r_dtype);
        }
    };
    float s = 1.0f;
    if constexpr (NORM) {
        double sq = 0.0;
        for (int k = tid * 8; k < p.H; k += T * 8) {
            float h[8];
            load_h(k, h, false);
            if (p.sum != nullptr) store8_as(sum, k, p.H - k, p.r_dtype, h);
#pragma unroll
            for (int j = 0; j < 8; ++j) sq = fma(static_cast<double>(h[j]), static_cast<double>(h[j]), sq);
        }
        sq = over_row<double, T>(sq, s_sum, [](double a, double b) { return a + b; });
        s = static_cast<float>(1.0 / sqrt(sq / p.H + p.eps));
    }
    auto load_v = [&](int k, float (&v)[8]) {
        load_h(k, v, true);
        if constexpr (NORM) {
            float w[8];
            if (p.w != nullptr) load8_as(p.w, k, p.H - k, p.w_dtype, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[j] *= s;
                if (p.w != nullptr) v[j] *= w[j];
            }
        }
    };
    float scale = 0.0f, inv = 0.0f;
    if (p.codes != nullptr && p.q_dtype == MOE_I8) {
        uint32_t most = 0;
        for (int k = tid * 8; k < p.H; k += T * 8) {
            float v[8];
            load_v(k, v);
            most = max(most, most_of(v));
        }
        most = over_row<uint32_t, T>(most, s_max, [](uint32_t a, uint32_t b) { return max(a, b); });
        scale = int8_scale(most);
        inv = 1.0f / scale;
        if (tid == 0) static_cast<float*>(p.scales)[row] = scale;
    }
    for (int k = tid * 8; k < p.H; k += T * 8) {
        float v[8];
        load_v(k, v);
        if (p.y != nullptr) store8_as(y, k, p.H - k, p.y_dtype, v);
        if (p.codes == nullptr) continue;
        if (p.q_dtype == MOE_I8) {
            store8_codes(codes, k, p.H - k, int8_codes(v, scale, inv));
        } else {                                       // H is a multiple of 32: four neighbours share a block
            uint32_t most = most_of(v);
            most = max(most, static_cast<uint32_t>(__shfl_xor(most, 1, 4)));
            most = max(most, static_cast<uint32_t>(__shfl_xor(most, 2, 4)));
            const int byte = mx_scale_byte(most);
            store8_codes(codes, k, 8, mx_codes(v, byte));
            if ((k & 31) == 0) static_cast<uint8_t*>(p.scales)[row * (p.H / 32) + k / 32] = static_cast<uint8_t>(byte);
        }
    }
}

template <bool NORM>
int launch_rows(const RowArgs& p, int64_t rows, hipStream_t st) {
    hipLaunchKernelGGL((rows_kernel<NORM, 256>), dim3(static_cast<unsigned>(rows)), dim3(256), 0, st, p);
    MOE_CHECK_LAUNCH();
    return MOE_OK;
}

}  // namespace

int launch_add_rmsnorm(int64_t rows, int H, const void* x, int x_dtype, int64_t ldx, const void* r, int r_dtype,
                       int64_t ldr, void* sum, int64_t lds, const void* w, int w_dtype, double eps, void* y, int y_dtype,
                       int64_t ldy, uint8_t* codes, int q_dtype, int64_t ldq, void* scales, hipStream_t st) {
    RowArgs p{};
    p.x = x;
    p.r = r;
    p.w = w;
    p.sum = sum;
    p.y = y;
    p.codes = codes;
    p.scales = scales;
    p.ldx = ldx;
    p.ldr = ldr;
    p.lds = lds;
    p.ldy = ldy;
    p.ldq = ldq;
    p.eps = eps;
    p.H = H;
    p.x_dtype = x_dtype;
    p.r_dtype = r_dtype;
    p.w_dtype = w_dtype;
    p.y_dtype = y_dtype;
    p.q_dtype = q_dtype;
    return launch_rows<true>(p, rows, st);
}

int launch_quantize_int8(int64_t rows, int K, const void* x, int x_dtype, int64_t ldx, uint8_t* codes, int64_t ldq,
                         float* scales, hipStream_t st) {
    RowArgs p{};
    p.x = x;
    p.codes = codes;
    p.scales = scales;
    p.ldx = ldx;
    p.ldq = ldq;
    p.H = K;
    p.x_dtype = x_dtype;
    p.q_dtype = MOE_I8;
    return launch_rows<false>(p, rows, st);
}

}  // namespace moe
