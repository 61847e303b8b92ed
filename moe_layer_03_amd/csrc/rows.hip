// Rows on their way into a product: the norm with the residual's sum,
//   h = x + residual (rounded to the residual's type),   s = 1 / sqrt(mean(h^2) + eps),   v = (h s) w,
// and the codes of v, or of rows given, in 8 bits: int8 with a scale per row, MXFP8 with one per 32.
//
// The mean and s are computed in double and s is rounded to float32; v takes two float32 products.  A thread adds up n
// squares, at most 16 for H to 2^14 and 8 ceil(H / 8192) beyond, before ten steps join the threads, so an order of
// summation is off by (n + 10) 2^-53 of the sum at most and by half of that in s, whose double steps add 2^-52.  That moves
// the rounded s to its neighbour where s lies that close to the middle of two: in fewer than one row of ten million, of a
// million for the longest.  In all others v, and the codes, which turn on which side of a half a quotient lies, depend
// neither on the order nor on the kernel's shape.  The conversion and the double fma of an element cost what two float32
// operations do.
//
// Bound by memory: 6000 x 4096, bf16 in, sum and out with int8 codes, moves 221 MB in 42.8 us, 5.2 TB/s, a large copy's
// rate; 16384 x 1536 quantised 75 MB in 17.4 us (4.3 TB/s, two rounds of rows and a launch).  Few rows are bound by the
// chain of loads and two reductions: 1 x 4096 4.3 us, of which a launch is 2.3.
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
    int64_t rows;
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

// Outputs that are more than the L2 caches hold go past them: 6000 x 4096 with everything written 42.6 us, 49.5 through
// the caches; less than that stays, for the kernel that reads it next (512 rows through two products 63.7 us, 66.6
// past the caches).  A constant of the kernel: the compiler makes one ordinary store of the two sides of a branch.
struct At16 { typedef u32x4 __attribute__((aligned(1))) type; };
struct At8 { typedef u32x2 __attribute__((aligned(1))) type; };
template <typename At, bool PAST, typename V>
__device__ __forceinline__ void put(void* p, V v) {
    auto* to = static_cast<typename At::type*>(p);
    if constexpr (PAST) __builtin_nontemporal_store(v, to);
    else *to = v;
}
template <bool PAST>
__device__ __forceinline__ void store8_as(void* p, int k, int n, int dtype, const float (&v)[8]) {
    if (dtype == MOE_F32) {
        float* f = static_cast<float*>(p) + k;
        if (n >= 8) {
            put<At16, PAST>(f, __builtin_bit_cast(u32x4, floatx4{v[0], v[1], v[2], v[3]}));
            put<At16, PAST>(f + 4, __builtin_bit_cast(u32x4, floatx4{v[4], v[5], v[6], v[7]}));
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
        put<At16, PAST>(h, u);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < n) h[j] = static_cast<uint16_t>(u[j >> 1] >> (16 * (j & 1)));
    }
}

template <bool PAST>
__device__ __forceinline__ void store8_codes(uint8_t* p, int k, int n, u32x2 u) {
    if (n >= 8) {
        put<At8, PAST>(p + k, u);
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
// Eight codes, without the remainder (6000 x 4096 49.9 us, 52.0 with it, before the stores went past the caches).
// v * inv + 1.5 * 2^23 rounds to the integer next to the product and leaves its two's complement in the low bits;
// only where some product is next to a half, which one group of 64 x 8 in ten has, the remainder is looked at
// (int8_code).  |v| <= 127.00001 scale, so no code passes 127.
__device__ __forceinline__ u32x2 int8_codes(const float (&v)[8], float scale, float inv) {
    if (scale != scale) return u32x2{0u, 0u};
    constexpr float kMagic = 12582912.0f;
    uint32_t t[8];
    float most = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float m = fmaf(v[j], inv, kMagic);
        most = fmaxf(most, fabsf(fmaf(v[j], inv, kMagic - m)));   // the product less its code, exact to 2^-24
        t[j] = __float_as_uint(m);
    }
    if (most > 0.4999f) {
#pragma unroll
        for (int j = 0; j < 8; ++j) t[j] = static_cast<uint32_t>(int8_code(v[j], scale, inv));
    }
    u32x2 u;
#pragma unroll
    for (int g = 0; g < 2; ++g) {
        const uint32_t lo = __builtin_amdgcn_perm(t[4 * g + 1], t[4 * g], 0x0c0c0400u);
        const uint32_t hi = __builtin_amdgcn_perm(t[4 * g + 3], t[4 * g + 2], 0x0c0c0400u);
        u[g] = lo | hi << 16;
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

// ---- a row over its lanes and waves ----------------------------------------------
// v of another lane of 16: lane ^ 1, lane ^ 2, then the mirror images in 8 and in 16 lanes, whose values stand for the
// lanes' across by then.  A DPP move takes a few cycles where a shuffle through LDS takes a hundred (128 x 4096
// with MXFP8 codes 4.3 us, 4.5 with shuffles).
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
    return static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), CTRL, 0xF, 0xF, true));
}
template <int CTRL>
__device__ __forceinline__ double dpp(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    return __builtin_bit_cast(double, static_cast<uint64_t>(dpp<CTRL>(static_cast<uint32_t>(u >> 32))) << 32 |
                                          dpp<CTRL>(static_cast<uint32_t>(u)));
}
constexpr int kWholeGroup = 1024;                      // a row to a workgroup, whose size is the launch's
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kMirror8 = 0x141, kMirror16 = 0x140;

template <typename V, typename Op>
__device__ __forceinline__ V over_16(V v, Op&& op) {
    v = op(v, dpp<kXor1>(v));
    v = op(v, dpp<kXor2>(v));
    v = op(v, dpp<kMirror8>(v));
    return op(v, dpp<kMirror16>(v));
}

// op over a row's threads, in an order that does not depend on timing; every thread has the result.
template <typename V, int T, typename Op>
__device__ __forceinline__ V over_row(V v, V* s, Op&& op) {
    static_assert(T == kWholeGroup || T == 16 || T == 32 || T == kWave, "threads of a row");
    v = over_16(v, op);
    if constexpr (T > 16) v = op(v, __shfl_xor(v, 16, kWave));
    if constexpr (T > 32) v = op(v, __shfl_xor(v, 32, kWave));
    if constexpr (T == kWholeGroup) {
        const int lane = threadIdx.x & (kWave - 1), waves = blockDim.x >> 6;
        if (lane == 0) s[threadIdx.x >> 6] = v;
        __syncthreads();
        v = over_16((lane & 15) < waves ? s[lane & 15] : V{0}, op);   // 0 changes neither a sum nor a largest value
    }
    return v;
}

// A row over T threads (16, 32, a wave: 256 / T rows to a workgroup; kWholeGroup: all of one), eight elements a thread
// at a time.
// C > 0: the row stays in registers, C groups of eight a thread, and is read once.  All of a row's loads, the weight's
//   too, are on their way before the first reduction.
// C = 0: rows of any length; the row is read again for each pass: once for the sum of squares, once for the largest |v|
//   (int8), once for the codes.  Passes after the first read h from `sum` where it is written (each thread what it
//   wrote itself), since that may lie over x or the residual.
// XB and RB: bytes of x's and the residual's elements (RB 0: no residual).
template <bool NORM, int XB, int RB, bool PAST, int T, int C>
__global__ __launch_bounds__(T <= kWave ? 256 : T) void rows_kernel(RowArgs p) {
    constexpr int kRows = T <= kWave ? 256 / T : 1;    // of a workgroup
    constexpr int kGroups = C > 0 ? C : 1;
    __shared__ double s_sum[kWholeGroup / kWave];
    __shared__ uint32_t s_max[kWholeGroup / kWave];
    const int stride = (kRows == 1 ? static_cast<int>(blockDim.x) : T) * 8;   // elements that a row's threads hold at once
    const int64_t row = kRows == 1 ? blockIdx.x : static_cast<int64_t>(blockIdx.x) * kRows + (threadIdx.x / T);
    if (kRows > 1 && row >= p.rows) return;            // all of the row's lanes
    const int tid = kRows == 1 ? threadIdx.x : threadIdx.x % T;
    const bool x_bf16 = p.x_dtype == MOE_BF16, r_bf16 = p.r_dtype == MOE_BF16;
    const int sum_dtype = RB == 4 ? MOE_F32 : p.r_dtype;
    auto at = [&](const void* base, int64_t ld, int bytes) { return static_cast<const uint8_t*>(base) + row * ld * bytes; };
    const void* x = at(p.x, p.ldx, XB);
    const void* r = at(p.r, p.ldr, RB);
    void* sum = const_cast<uint8_t*>(at(p.sum, p.lds, RB));
    void* y = const_cast<uint8_t*>(at(p.y, p.ldy, p.y_dtype == MOE_F32 ? 4 : 2));
    uint8_t* codes = p.codes + row * p.ldq;
    auto add_residual = [&](float (&h)[8], const float (&a)[8]) {
#pragma unroll
        for (int j = 0; j < 8; ++j) h[j] = round_as(h[j] + a[j], sum_dtype);
    };
    auto factor = [&](double sq) {
        sq = over_row<double, T>(sq, s_sum, [](double a, double b) { return a + b; });
        return static_cast<float>(1.0 / sqrt(sq / p.H + p.eps));
    };
    auto scale_of = [&](uint32_t most) {
        most = over_row<uint32_t, T>(most, s_max, [](uint32_t a, uint32_t b) { return max(a, b); });
        const float scale = int8_scale(most);
        if (tid == 0) static_cast<float*>(p.scales)[row] = scale;
        return scale;
    };
    auto square = [](double sq, const float (&h)[8]) {
#pragma unroll
        for (int j = 0; j < 8; ++j) sq = fma(static_cast<double>(h[j]), static_cast<double>(h[j]), sq);
        return sq;
    };
    // a group's codes; most: its largest |v|
    auto write_mx = [&](int k, const float (&v)[8]) {  // H is a multiple of 32: four neighbours share a block
        uint32_t most = most_of(v);
        most = max(most, dpp<kXor1>(most));
        most = max(most, dpp<kXor2>(most));
        const int byte = mx_scale_byte(most);
        store8_codes<PAST>(codes, k, 8, mx_codes(v, byte));
        if ((k & 31) == 0) static_cast<uint8_t*>(p.scales)[row * (p.H / 32) + k / 32] = static_cast<uint8_t>(byte);
    };
    const bool int8 = p.codes != nullptr && p.q_dtype == MOE_I8;
    const int k0 = tid * 8;
    if constexpr (C > 0) {
        float v[kGroups][8];
        float w[NORM ? kGroups : 1][8];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int k = k0 + c * stride;
            if (k < p.H) load8<XB>(x, k, p.H - k, x_bf16, v[c]);
            else
#pragma unroll
                for (int j = 0; j < 8; ++j) v[c][j] = 0.0f;
        }
        if constexpr (RB != 0) {
            float a[kGroups][8];
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int k = k0 + c * stride;
                if (k < p.H) load8<RB>(r, k, p.H - k, r_bf16, a[c]);
            }
#pragma unroll
            for (int c = 0; c < C; ++c)
                if (k0 + c * stride < p.H) add_residual(v[c], a[c]);
        }
        if constexpr (NORM) {
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int k = k0 + c * stride;
                if (p.w != nullptr && k < p.H) load8_as(p.w, k, p.H - k, p.w_dtype, w[c]);
            }
            double sq = 0.0;
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int k = k0 + c * stride;
                if (RB != 0 && p.sum != nullptr && k < p.H) store8_as<PAST>(sum, k, p.H - k, sum_dtype, v[c]);
                sq = square(sq, v[c]);
            }
            const float s = factor(sq);
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    v[c][j] *= s;
                    if (p.w != nullptr && k0 + c * stride < p.H) v[c][j] *= w[c][j];
                }
        }
        if (p.y != nullptr) {
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int k = k0 + c * stride;
                if (k < p.H) store8_as<PAST>(y, k, p.H - k, p.y_dtype, v[c]);
            }
        }
        if (p.codes == nullptr) return;
        if (!int8) {
#pragma unroll
            for (int c = 0; c < C; ++c)
                if (k0 + c * stride < p.H) write_mx(k0 + c * stride, v[c]);
            return;
        }
        uint32_t most = 0;
#pragma unroll
        for (int c = 0; c < C; ++c)
            if (k0 + c * stride < p.H) most = max(most, most_of(v[c]));
        const float scale = scale_of(most), inv = 1.0f / scale;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int k = k0 + c * stride;
            if (k < p.H) store8_codes<PAST>(codes, k, p.H - k, int8_codes(v[c], scale, inv));
        }
        return;
    }
    auto load_h = [&](int k, float (&h)[8], bool again) {
        if (RB != 0 && again && p.sum != nullptr) {
            load8<RB>(sum, k, p.H - k, r_bf16, h);
            return;
        }
        load8<XB>(x, k, p.H - k, x_bf16, h);
        if constexpr (RB != 0) {
            float a[8];
            load8<RB>(r, k, p.H - k, r_bf16, a);
            add_residual(h, a);
        }
    };
    float s = 1.0f;
    if constexpr (NORM) {
        double sq = 0.0;
        for (int k = k0; k < p.H; k += stride) {
            float h[8];
            load_h(k, h, false);
            if (RB != 0 && p.sum != nullptr) store8_as<PAST>(sum, k, p.H - k, sum_dtype, h);
            sq = square(sq, h);
        }
        s = factor(sq);
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
    if (int8) {
        uint32_t most = 0;
        for (int k = k0; k < p.H; k += stride) {
            float v[8];
            load_v(k, v);
            most = max(most, most_of(v));
        }
        scale = scale_of(most);
        inv = 1.0f / scale;
    }
    for (int k = k0; k < p.H; k += stride) {
        float v[8];
        load_v(k, v);
        if (p.y != nullptr) store8_as<PAST>(y, k, p.H - k, p.y_dtype, v);
        if (int8) store8_codes<PAST>(codes, k, p.H - k, int8_codes(v, scale, inv));
        else if (p.codes != nullptr) write_mx(k, v);
    }
}

template <bool NORM, int XB, int RB, bool PAST, int T, int C>
int launch_shape(const RowArgs& p, int threads, hipStream_t st) {
    constexpr int kRows = T <= kWave ? 256 / T : 1;
    hipLaunchKernelGGL((rows_kernel<NORM, XB, RB, PAST, T, C>), dim3(static_cast<unsigned>((p.rows + kRows - 1) / kRows)),
                       dim3(T <= kWave ? 256 : threads), 0, st, p);
    MOE_CHECK_LAUNCH();
    return MOE_OK;
}

// One group of eight a thread while the rows' waves fit the chip at once (24 to a CU), for the shorter chain: 512 x 4096
// 7.9 us, 9.3 with two; from there on two, for the loads in flight: 1000 x 4096 10.3 us, 10.9 with one, 6000 x 4096 42.8
// and 47.8.  The quantiser takes two only where they leave no more lanes idle: 16384 x 1536 17.4 us, 17.8 with two.
constexpr int64_t kFewWaves = 256 * 24;
constexpr int64_t kL2Bytes = 32 << 20;                 // of all eight L2 caches

template <bool NORM, int XB, int RB, bool PAST>
int launch_shapes(const RowArgs& p, hipStream_t st) {
    const int groups = (p.H + 7) / 8;
    if (groups <= 16) return launch_shape<NORM, XB, RB, PAST, 16, 1>(p, 0, st);
    if (groups <= 32) return launch_shape<NORM, XB, RB, PAST, 32, 1>(p, 0, st);
    if (groups <= 64) return launch_shape<NORM, XB, RB, PAST, 64, 1>(p, 0, st);
    auto whole = [](int n) { return (n + kWave - 1) / kWave * kWave; };
    const int one = whole(groups), two = whole((groups + 1) / 2);
    // nine bytes of output an element at most: a norm's few waves write less than the caches hold
    static_assert(kFewWaves * kWave * 8 * 9 <= kL2Bytes, "");
    if constexpr (!NORM || !PAST)
        if (groups <= kWholeGroup && (p.rows * (one / kWave) <= kFewWaves || (!NORM && one < 2 * two)))
            return launch_shape<NORM, XB, RB, PAST, kWholeGroup, 1>(p, one, st);
    if (groups <= 128) return launch_shape<NORM, XB, RB, PAST, 64, 2>(p, 0, st);
    if (groups <= 2 * kWholeGroup) return launch_shape<NORM, XB, RB, PAST, kWholeGroup, 2>(p, two, st);
    return launch_shape<NORM, XB, RB, PAST, kWholeGroup, 0>(p, kWholeGroup, st);
}

template <bool NORM, int XB, int RB>
int launch_types(const RowArgs& p, hipStream_t st) {
    auto size = [](const void* q, int dtype) { return q == nullptr ? 0 : dtype == MOE_F32 ? 4 : 2; };
    const int64_t bytes = p.rows * p.H * (size(p.sum, p.r_dtype) + size(p.y, p.y_dtype) + (p.codes != nullptr));
    return bytes > kL2Bytes ? launch_shapes<NORM, XB, RB, true>(p, st) : launch_shapes<NORM, XB, RB, false>(p, st);
}

template <bool NORM>
int launch_rows(const RowArgs& p, hipStream_t st) {
    const bool wide = p.x_dtype == MOE_F32;
    if constexpr (NORM) {
        if (p.r != nullptr && p.r_dtype == MOE_F32)
            return wide ? launch_types<true, 4, 4>(p, st) : launch_types<true, 2, 4>(p, st);
        if (p.r != nullptr) return wide ? launch_types<true, 4, 2>(p, st) : launch_types<true, 2, 2>(p, st);
    }
    return wide ? launch_types<NORM, 4, 0>(p, st) : launch_types<NORM, 2, 0>(p, st);
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
    p.rows = rows;
    p.H = H;
    p.x_dtype = x_dtype;
    p.r_dtype = r_dtype;
    p.w_dtype = w_dtype;
    p.y_dtype = y_dtype;
    p.q_dtype = q_dtype;
    return launch_rows<true>(p, st);
}

int launch_quantize_int8(int64_t rows, int K, const void* x, int x_dtype, int64_t ldx, uint8_t* codes, int64_t ldq,
                         float* scales, hipStream_t st) {
    RowArgs p{};
    p.x = x;
    p.codes = codes;
    p.scales = scales;
    p.ldx = ldx;
    p.ldq = ldq;
    p.rows = rows;
    p.H = K;
    p.x_dtype = x_dtype;
    p.q_dtype = MOE_I8;
    return launch_rows<false>(p, st);
}

}  // namespace moe
