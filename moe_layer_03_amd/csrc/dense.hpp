// Dense products with a fused epilogue, for the projections around the experts:
//   C = act(A W + bias) + R,   or, gated,   C = silu(A Wg + bg) * (A Wu + bu) + R,
// A [M, K] 16-bit, W [K, N] packed once, sums in float32, one rounding to C's type; or
// A and W in int8 codes, sums in int32, with a scale per row and per column.  The
// kernels of the 16-bit products and the choice among them, and what dense_int8.hip
// shares: the epilogues, weight streaming for a few rows, the kernel for rows far apart.
//
// Packed weights are the grouped GEMMs' fragment blocks of 32 columns x 16 k, K
// padded to a multiple of 64 and the columns to whole 64-column pairs (gated:
// 32 gate columns and the same 32 up columns to a pair, so a lane holds g and u
// of one output element); the padding is zero, so only A's reads need masks.
#pragma once

#include <algorithm>

#include "block.hpp"
#include "stream.hpp"

namespace moe {
namespace {

// What A and W hold.  int8 codes come sixteen to an operand where 16-bit values come eight, in the same bytes and
// lanes, and multiply into int32: every length below is in 16-bit units, of which a code is half a one, but for K.
enum Kind { kBF16 = 0, kF16 = 1, kI8 = 2 };
template <int KIND> constexpr int codes_per_unit() { return KIND == kI8 ? 2 : 1; }   // elements of a 16-bit unit

typedef int intx4 __attribute__((ext_vector_type(4)));
typedef int intx16 __attribute__((ext_vector_type(16)));
template <int KIND> struct Sums {
    typedef float one;
    typedef floatx4 four;
    typedef floatx16 sixteen;
};
template <> struct Sums<kI8> {
    typedef int one;
    typedef intx4 four;
    typedef intx16 sixteen;
};

struct DenseArgs {
    const uint16_t* a;
    const uint16_t* b;         // packed
    const float *sa, *sb;      // int8: the scales of A's rows and of the columns (gated: gate, then up at sb_up)
    int sb_up;
    const float* bias;         // [N], gated [2][N], or NULL
    const void* r;             // residual, or NULL
    void* c;
    int64_t lda, ldr, ldc;     // lda in bytes
    int M, N, K;
    int Kh, Kp;                // K in whole 16-bit units, and padded as the weights are
    int gated, act, r_dtype, c_dtype;
    int vec;                   // rows of R and C start on four elements, of which N is a multiple
};

// ---- epilogue ------------------------------------------------------------------

// v / (1 + exp(-y)).  16-bit outputs take the hardware's exp2 and reciprocal (6000 x
// 4096 x 4096 with bias and SiLU to bf16 186 us, against 199 for the float32 form
// below and output): an ulp each, which is 2 u (u = 2^-24), one rounding in 1 + e and one in the
// product are 6 u, and the exponent's own roundings, 1.3 |y| u, make (1.3 |y| + 6) u
// of the result, against half a step of 2^16 u (bf16) or 2^13 u (fp16).  The
// reciprocal underflows below y = -87, where the result is under 1e-36: zero.
__device__ __forceinline__ float over_one_plus_exp_fast(float v, float y) {
    return v * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.4426950408889634f * y));
}

// The same for float32 outputs.  exp(-y) = 2^(-y / ln 2), whose product's rounding
// and the constant's own are put back to first order (3 u with the last rounding),
// the sum, a Newton step of the reciprocal and the product round once each: 6 u.
// Far below zero it is v exp(y), in two factors (6 u), down to float32's last digit.
__device__ __forceinline__ float over_one_plus_exp(float v, float y) {
    if (y < -80.0f) {
        const float e = expf(0.5f * y);
        return v * e * e;
    }
    constexpr float kLog2e = 1.4426950408889634f, kRest = static_cast<float>(1.4426950408889634 - kLog2e);
    const float z = -fminf(y, 128.0f), x = z * kLog2e;      // 1 + exp(-128) is 1, and y may be infinite
    const float lost = fmaf(z, kLog2e, -x) + z * kRest;
    float e = __builtin_amdgcn_exp2f(x);
    e = fmaf(e, lost * 0.69314718055994531f, e);
    const float s = 1.0f + e, r = __builtin_amdgcn_rcpf(s);
    return v * fmaf(r, fmaf(-s, r, 1.0f), r);
}

// N values at once.  tanh-GELU is v / (1 + exp(-2 z)), without (1 + tanh z)'s
// cancellation for negative z; y = 2 z has seven roundings, 7 |y| u of the result.
template <int ACT, bool FAST, int N>
__device__ __forceinline__ void activate_as(float (&v)[N]) {
    auto tanh_y = [](float x) { return 1.5957691216057308f * (x + 0.044715f * x * x * x); };
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float x = v[i];
        if constexpr (ACT == MOE_EPI_SWIGLU || ACT == MOE_EPI_SILU)   // SwiGLU: the gate's
            v[i] = FAST ? over_one_plus_exp_fast(x, x) : over_one_plus_exp(x, x);
        else if constexpr (ACT == MOE_EPI_GELU)
            v[i] = 0.5f * x * erfcf(x * -0.70710678118654752f);
        else if constexpr (ACT == MOE_EPI_GELU_TANH)
            v[i] = FAST ? over_one_plus_exp_fast(x, tanh_y(x)) : over_one_plus_exp(x, tanh_y(x));
        else if constexpr (ACT == MOE_EPI_RELU)
            v[i] = x < 0.0f ? 0.0f : x;                // NaN stays
    }
}
template <bool FAST, int N>
__device__ __forceinline__ void activate(float (&v)[N], int act) {
    switch (act) {                                     // uniform
        case MOE_EPI_SWIGLU:
        case MOE_EPI_SILU: activate_as<MOE_EPI_SILU, FAST>(v); break;
        case MOE_EPI_GELU: activate_as<MOE_EPI_GELU, FAST>(v); break;
        case MOE_EPI_GELU_TANH: activate_as<MOE_EPI_GELU_TANH, FAST>(v); break;
        case MOE_EPI_RELU: activate_as<MOE_EPI_RELU, FAST>(v); break;
        default: break;
    }
}

__device__ __forceinline__ float load_as(const void* p, int64_t i, int dtype) {
    if (dtype == MOE_F32) return static_cast<const float*>(p)[i];
    const uint16_t v = static_cast<const uint16_t*>(p)[i];
    return dtype == MOE_BF16 ? bf16_to_f32(v) : f16_to_f32(v);
}

__device__ __forceinline__ void store_as(void* p, int64_t i, int dtype, float v) {
    if (dtype == MOE_F32) static_cast<float*>(p)[i] = v;
    else static_cast<uint16_t*>(p)[i] = dtype == MOE_BF16 ? f32_to_bf16_or_nan(v) : f32_to_f16_or_nan(v);
}

// A sum with its scales, of either sign.  The int32 sum and two products round once each.  The row's scale comes first
// where it is at most one in magnitude, the column's else, so that no product overflows where the result does not: up to
// one, |sum * sa| lies between |sa| and 2^31; above, sum * sw overflows only if the result does.  Nor is a digit lost
// below the normal numbers: an integer times a subnormal one is a multiple of its last digit.
__device__ __forceinline__ float scaled(int v, float sa, float sw) {
    const float f = static_cast<float>(v);
    return fabsf(sa) > 1.0f ? f * sw * sa : f * sa * sw;
}

// The element (row, col): v is its sum (gated: the gate's, u the up's).  The
// residual is read by the thread that writes the element, so it may be C itself.
template <int KIND>
__device__ __forceinline__ void finish(const DenseArgs& p, int row, int col, typename Sums<KIND>::one v0,
                                       typename Sums<KIND>::one u0) {
    if (row >= p.M || col >= p.N) return;
    float v, u;
    if constexpr (KIND == kI8) {
        const float sa = p.sa[row];
        v = scaled(v0, sa, p.sb[col]);
        u = p.gated ? scaled(u0, sa, p.sb[p.sb_up + col]) : 0.0f;
    } else {
        v = v0;
        u = u0;
    }
    if (p.bias != nullptr) v += p.bias[col];
    float g[1] = {v};
    if (p.c_dtype == MOE_F32) activate<false>(g, p.act);
    else activate<true>(g, p.act);
    v = g[0];
    if (p.gated) {
        if (p.bias != nullptr) u += p.bias[p.N + col];
        v *= u;
    }
    if (p.r != nullptr) v += load_as(p.r, row * p.ldr + col, p.r_dtype);
    store_as(p.c, row * p.ldc + col, p.c_dtype, v);
}

// ---- four columns at once -----------------------------------------------------------
// A lane finishes columns col .. col + 3 of one row after another, in a loop made for the activation: 24 rows of four
// a lane for a 192 x 256 tile, where a branch or a conversion more in each step shows.  Nothing in a step branches on a
// lane: rows past M and columns past N have offsets that load zeros and store nothing.  So the compiler knows what is
// in flight, and a step that needs a part of the residual waits for that and not for the stores behind it.
// VEC: rows of R and C start on four elements and N is a multiple of four, so that four columns move at once.
struct Columns {
    floatx4 b0, b1, s0, s1;    // bias and scales of the gate's or only weight, and of the up's
};

template <int KIND>
__device__ __forceinline__ Columns load_columns(const DenseArgs& p, int col) {
    Columns c;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int at = min(col + i, p.N - 1);          // past N: never stored
        c.b0[i] = p.bias != nullptr ? p.bias[at] : 0.0f;
        c.b1[i] = p.bias != nullptr && p.gated ? p.bias[p.N + at] : 0.0f;
        c.s0[i] = KIND == kI8 ? p.sb[at] : 0.0f;
        c.s1[i] = KIND == kI8 && p.gated ? p.sb[p.sb_up + at] : 0.0f;
    }
    return c;
}

typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

// Four sums with their scales, in the order of scaled().
__device__ __forceinline__ floatx4 scaled4(const intx4& v, float sa, const floatx4& sw) {
    floatx4 f = __builtin_convertvector(v, floatx4);
    const bool big = fabsf(sa) > 1.0f;
    if (__builtin_amdgcn_ballot_w64(big) == 0) return f * sa * sw;
    const floatx4 all = {sa, sa, sa, sa};
    return f * (big ? sw : all) * (big ? all : sw);
}

// C and R from row `first` on, as buffers; the launcher keeps the offsets of the rows reached from there below the range.
// A tile's epilogue goes on 16 rows at a time, which costs a few scalar instructions: so rows may lie some 128 MiB apart
// (1024 x 4096 x 4096 into rows 8 MiB apart 38 us; with one base for all of a tile's rows such C fell to
// dense_any_kernel, an element at a time, 72 us).  A lane's row is u, uniform, and its own beyond that: the offset of a
// part of C or R is a register, a scalar and a constant.
template <int KIND, bool VEC>
struct Finisher {
    const DenseArgs& p;
    const uint8_t *c_at, *r_at;
    int c_rows, r_rows;        // rows from there on that exist
    int c_row, r_row;          // bytes of a row
    bool c_wide, r_wide;
    int own, col;              // the lane's row beyond u, and its first column
    uint32_t c_off, r_off;

    __device__ __forceinline__ Finisher(const DenseArgs& args, int first, int lane_row, int lane_col)
        : p(args), own(lane_row), col(lane_col) {
        c_wide = p.c_dtype == MOE_F32;
        r_wide = p.r_dtype == MOE_F32;
        c_row = static_cast<int>(p.ldc) * (c_wide ? 4 : 2);
        r_row = static_cast<int>(p.ldr) * (r_wide ? 4 : 2);
        c_at = static_cast<const uint8_t*>(p.c) + static_cast<int64_t>(first) * c_row;
        r_at = static_cast<const uint8_t*>(p.r) + static_cast<int64_t>(first) * r_row;
        c_rows = r_rows = p.M - first;
        c_off = own * c_row + col * (c_wide ? 4 : 2);
        r_off = own * r_row + col * (r_wide ? 4 : 2);
    }
    // The residual is loaded ahead of C: each goes on by itself.
    __device__ __forceinline__ void next_c(int n) {
        c_at += static_cast<int64_t>(c_row) * n;
        c_rows -= n;
    }
    __device__ __forceinline__ void next_r(int n) {
        r_at += static_cast<int64_t>(r_row) * n;
        r_rows -= n;
    }
    __device__ __forceinline__ static __amdgpu_buffer_rsrc_t buffer(const uint8_t* at) {
        return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(at), 0, kBufferRange, kBufferFlags);
    }
    // Offsets of the elements col .. col + 3, but for a constant each, `off` or out of range.  Opaque: the constants belong
    // into the instructions, and one set of registers is then all that the branches on a type need; where they took some
    // of their own, which loads of the other branch might be writing, they waited for all that is in flight (6000 x 4095 x
    // 1024 onto a float32 residual 101 us, 105).
    __device__ __forceinline__ void each(bool row, uint32_t off, uint32_t (&o)[4]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            o[i] = row && col + i < p.N ? off : kOutOfRange;
            asm("" : "+v"(o[i]));
        }
    }
    // The residual's four elements of the row: a word each, or (16-bit, VEC) two to a word.
    __device__ __forceinline__ u32x4 load(int u) const {
        u32x4 q = {0u, 0u, 0u, 0u};
        if (p.r == nullptr) return q;                  // uniform, as the types are
        const __amdgpu_buffer_rsrc_t r = buffer(r_at);
        const bool row = own < r_rows - u;
        const int at = u * r_row;
        uint32_t o[4];
        if constexpr (!VEC) each(row, r_off, o);
        if (r_wide) {
            if constexpr (VEC) {
                q = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                                  r, row && col < p.N ? r_off : kOutOfRange, at, 0));
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    q[i] = __builtin_amdgcn_raw_buffer_load_b32(r, o[i] + 4 * i, at, 0);
            }
        } else {
            if constexpr (VEC) {
                const u32x2_t v = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_raw_buffer_load_b64(
                                                                  r, row && col < p.N ? r_off : kOutOfRange, at, 0));
                q[0] = v[0];
                q[1] = v[1];
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    q[i] = __builtin_amdgcn_raw_buffer_load_b16(r, o[i] + 2 * i, at, 0);
            }
        }
        return q;
    }
    template <int ACT>
    __device__ __forceinline__ void finish(int u_row, const typename Sums<KIND>::four& v0,
                                           const typename Sums<KIND>::four& u0, const Columns& k, float sa,
                                           const u32x4& q) const {
        floatx4 v, u;
        if constexpr (KIND == kI8) v = scaled4(v0, sa, k.s0);
        else v = v0;
        v += k.b0;
        if constexpr (ACT != MOE_EPI_NONE) {
            float g[4] = {v[0], v[1], v[2], v[3]};
            if (c_wide) activate_as<ACT, false>(g);
            else activate_as<ACT, true>(g);
            v = floatx4{g[0], g[1], g[2], g[3]};
        }
        if constexpr (ACT == MOE_EPI_SWIGLU) {
            if constexpr (KIND == kI8) u = scaled4(u0, sa, k.s1);
            else u = u0;
            v *= u + k.b1;
        }
        if (p.r != nullptr) {
            if (r_wide) {
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] += __uint_as_float(q[i]);
            } else {
                uint32_t e[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) e[i] = VEC ? q[i >> 1] >> (16 * (i & 1)) : q[i];
                if (p.r_dtype == MOE_BF16) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[i] += __uint_as_float(e[i] << 16);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[i] += f16_to_f32(static_cast<uint16_t>(e[i]));
                }
            }
        }
        const __amdgpu_buffer_rsrc_t c = buffer(c_at);
        const bool row = own < c_rows - u_row;
        const int at = u_row * c_row;
        uint32_t o[4];
        if constexpr (!VEC) each(row, c_off, o);
        if (c_wide) {
            if constexpr (VEC) {
                __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), c,
                                                       row && col < p.N ? c_off : kOutOfRange, at, 0);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v[i]), c, o[i] + 4 * i, at, 0);
            }
            return;
        }
        u32x2_t h;
        if (p.c_dtype == MOE_BF16)
            h = u32x2_t{pack_bf16x2_or_nan(v[0], v[1]), pack_bf16x2_or_nan(v[2], v[3])};
        else
            h = u32x2_t{f32_to_f16_or_nan(v[0]) | static_cast<uint32_t>(f32_to_f16_or_nan(v[1])) << 16,
                        f32_to_f16_or_nan(v[2]) | static_cast<uint32_t>(f32_to_f16_or_nan(v[3])) << 16};
        if constexpr (VEC) {
            __builtin_amdgcn_raw_buffer_store_b64(h, c, row && col < p.N ? c_off : kOutOfRange, at, 0);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                __builtin_amdgcn_raw_buffer_store_b16(static_cast<uint16_t>(h[i >> 1] >> (16 * (i & 1))), c,
                                                      o[i] + 2 * i, at, 0);
        }
    }
};

// f(activation), a constant for it (uniform).
template <typename F>
__device__ __forceinline__ void with_activation(int act, F&& f) {
    switch (act) {
        case MOE_EPI_SWIGLU: f(IntC<MOE_EPI_SWIGLU>{}); break;
        case MOE_EPI_SILU: f(IntC<MOE_EPI_SILU>{}); break;
        case MOE_EPI_GELU: f(IntC<MOE_EPI_GELU>{}); break;
        case MOE_EPI_GELU_TANH: f(IntC<MOE_EPI_GELU_TANH>{}); break;
        case MOE_EPI_RELU: f(IntC<MOE_EPI_RELU>{}); break;
        default: f(IntC<MOE_EPI_NONE>{}); break;
    }
}

// Rows that may start at any address: 16 bytes at an element's alignment (one
// load, the hardware takes unaligned addresses).
template <int KIND> struct AnyRow { typedef u32x4 __attribute__((aligned(2))) type; };
template <> struct AnyRow<kI8> { typedef u32x4 __attribute__((aligned(1))) type; };
template <int KIND>
__device__ __forceinline__ u32x4 load_any(const uint8_t* p) {
    return *reinterpret_cast<const typename AnyRow<KIND>::type*>(p);
}

// The 8 units k .. k + 7 of a row, zeros from K (elements) on.
template <int KIND>
__device__ __forceinline__ u32x4 load_tail(const uint8_t* row, int k, int K) {
    uint32_t v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int i = k + j;
        if constexpr (KIND == kI8)
            v[j] = (2 * i < K ? row[2 * i] : 0u) | (2 * i + 1 < K ? static_cast<uint32_t>(row[2 * i + 1]) << 8 : 0u);
        else
            v[j] = i < K ? reinterpret_cast<const uint16_t*>(row)[i] : 0u;
    }
    return u32x4{v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16};
}

typedef int i8x16_t __attribute__((ext_vector_type(4)));   // an operand of the int8 MFMAs

template <int KIND>
__device__ __forceinline__ typename Sums<KIND>::four mfma16k(const u32x4& a, const u32x4& b,
                                                             typename Sums<KIND>::four c) {
    if constexpr (KIND == kI8)
        return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i8x16_t, a), __builtin_bit_cast(i8x16_t, b), c,
                                                     0, 0, 0);
    else
        return mfma16(KIND == kF16, a, b, c);
}

// ---- many rows, any alignment --------------------------------------------------------
// 64 rows x one 64-column pair per workgroup of 4 waves; a wave owns 32 rows x
// 16 columns of each half.  Direct copies to LDS need aligned rows, so A goes
// through registers, and a stage is 128 k long to have as few waits as possible:
// the next stage's rows and weights are on their way while one is multiplied.
// Bound by the latency of a stage, 1.65 us: 283 x 1516 x 1396 18.4 us (streaming,
// which the rule takes there, 18.8; 500 x 515 x 2011 28.5 and 26.1).
constexpr int kAnyK = 128;
constexpr int kAnyLd = kAnyK + 8;                      // LDS row, 16 of them in distinct banks
constexpr int kAnyOut = 64 + 4;                        // row of sums on the way out
// Rows of R and C: four elements at once, one at a time, or so far apart that 16 of them pass a buffer's range.
enum OutRows { kByFour = 0, kByOne = 1, kFarRows = 2 };

template <int KIND, int OUT>
__global__ __launch_bounds__(256) void dense_any_kernel(DenseArgs p) {
    static_assert(KIND != kI8 || OUT == kFarRows, "int8 rows within reach have kernels of their own");
    __shared__ __attribute__((aligned(16))) uint16_t s_a[2][64 * kAnyLd];
    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int pair = blockIdx.x, c0 = (wave & 1) * 16, r0 = (wave >> 1) * 32;
    const int row0 = blockIdx.y * 64;
    const int nk32 = p.Kp / 32;
    // k group lane / 16 of 8 in a 32-k step: block lane / 32, half (lane / 16) % 2
    const uint8_t* b = reinterpret_cast<const uint8_t*>(p.b) + static_cast<int64_t>(pair) * nk32 * kStepBytes +
                       (lane >> 5) * 2048 + (((lane >> 4) & 1) * 32 + c0 + (lane & 15)) * 16;
    typename Sums<KIND>::four acc[2][2];
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i >> 1][i & 1] = typename Sums<KIND>::four{0, 0, 0, 0};
    const int Kc = (p.K + codes_per_unit<KIND>() - 1) / codes_per_unit<KIND>();
    const int lr = tid >> 2, lk = (tid & 3) * 32;      // this thread's 32 units of a stage
    const uint8_t* row = reinterpret_cast<const uint8_t*>(p.a) +
                         static_cast<int64_t>(min(row0 + lr, p.M - 1)) * p.lda;   // rows past M: dropped below
    u32x4 ra[4], rb[4][2], nb[4][2];
    auto load_a = [&](int k0) {
        if (k0 + kAnyK <= p.Kh) {                      // uniform
#pragma unroll
            for (int j = 0; j < 4; ++j) ra[j] = load_any<KIND>(row + (k0 + lk + j * 8) * 2);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) ra[j] = load_tail<KIND>(row, k0 + lk + j * 8, p.K);
        }
    };
    auto load_b = [&](u32x4 (&r)[4][2], int k0) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int h = 0; h < 2; ++h)                // zeros past the end, as A's (an infinity times A's would be NaN)
                r[q][h] = k0 / 32 + q < nk32           // uniform
                              ? *reinterpret_cast<const u32x4*>(
                                    b + static_cast<int64_t>(k0 / 32 + q) * kStepBytes + h * 1024)
                              : u32x4{0u, 0u, 0u, 0u};
    };
    load_a(0);
    load_b(rb, 0);
    int buf = 0;
    for (int k0 = 0; k0 < Kc; k0 += kAnyK, buf ^= 1) {
#pragma unroll
        for (int j = 0; j < 4; ++j) *reinterpret_cast<u32x4*>(&s_a[buf][lr * kAnyLd + lk + j * 8]) = ra[j];
        lds_barrier();                                 // the other buffer is no longer read either
        if (k0 + kAnyK < Kc) {
            load_a(k0 + kAnyK);
            load_b(nb, k0 + kAnyK);
        }
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const u32x4 a = *reinterpret_cast<const u32x4*>(
                    &s_a[buf][(r0 + m * 16 + (lane & 15)) * kAnyLd + q * 32 + (lane >> 4) * 8]);
                acc[m][0] = mfma16k<KIND>(a, rb[q][0], acc[m][0]);
                acc[m][1] = mfma16k<KIND>(a, rb[q][1], acc[m][1]);
            }
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int h = 0; h < 2; ++h) rb[q][h] = nb[q][h];
    }
    // through LDS, so that a thread has four columns of a row; one copy of the code for all of them (48 KB, which a cold
    // launch has to fetch, were it once per register)
    typedef typename Sums<KIND>::one Sum;
    static_assert(sizeof(s_a) >= 64 * kAnyOut * sizeof(Sum), "");
    Sum* s_c = reinterpret_cast<Sum*>(&s_a[0][0]);
    __syncthreads();                                   // the last stage has been read
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                s_c[(r0 + m * 16 + (lane >> 4) * 4 + i) * kAnyOut + h * 32 + c0 + (lane & 15)] = acc[m][h][i];
    const int lc = p.gated ? (tid & 7) * 4 : (tid & 15) * 4, dr = p.gated ? 32 : 16;
    const int col = pair * (p.gated ? 32 : 64) + lc;
    const int wr = wave * (p.gated ? 8 : 4), in_wave = p.gated ? lane >> 3 : lane >> 4;   // row wr + in_wave, then each dr-th
    if constexpr (OUT == kFarRows) {
        __syncthreads();
#pragma unroll 1
        for (int r = wr + in_wave; r < 64; r += dr)
#pragma unroll 1
            for (int i = 0; i < 4; ++i) {
                const Sum* e = s_c + r * kAnyOut + lc + i;
                finish<KIND>(p, row0 + r, col + i, *e, p.gated ? e[32] : 0);
            }
    } else {
        const Columns columns = load_columns<KIND>(p, col);
        __syncthreads();
        with_activation(p.act, [&](auto act) __attribute__((always_inline)) {
            constexpr int ACT = decltype(act)::value;
            Finisher<KIND, OUT == kByFour> f(p, row0 + wr, in_wave, col);
            u32x4 part = f.load(0);
#pragma unroll 1
            for (int i = wr; i < 64; i += dr) {        // uniform
                const u32x4 now = part;
                f.next_r(dr);
                part = f.load(0);
                const Sum* e = s_c + (i + in_wave) * kAnyOut + lc;
                floatx4 u = {0.0f, 0.0f, 0.0f, 0.0f};
                if constexpr (ACT == MOE_EPI_SWIGLU) u = *reinterpret_cast<const floatx4*>(e + 32);
                f.template finish<ACT>(0, *reinterpret_cast<const floatx4*>(e), u, columns, 0.0f, now);
                f.next_c(dr);
            }
        });
    }
}

// ---- few rows: weight streaming ------------------------------------------------------
// Bound by what a CU reads (its unit's rows and columns), 37 bytes/ns from the
// caches: 128 rows of 4096 x 4096 take 23.3 us, 786 KB on each CU, against 5.6 us
// for one pass over memory; a unit that reads less needs the reduction split over
// workgroups, and partial sums in memory.  One row is bound by the launch and
// one round of latency: 1536 columns, gated, 25 MB in 7.0 us (3.6 TB/s); 12288
// columns, gated, 201 MB in 31.2 us (6.45 TB/s).
// A workgroup owns MT * 16 rows x 16 columns of CT column halves (CT = 1, gated:
// 8 gate and 8 up columns) and its kNW waves take every kNW-th step of the
// reduction, so the weights go straight from memory to registers, each element
// once per MT * 16 rows.  The partial tiles are added through LDS in wave order.
constexpr int kNW = 8;

// ROWS16: rows on 16 bytes and K a multiple of 8; rows past M and k past K then
// load zeros through an out-of-range buffer offset.  Otherwise rows past M load
// the last row (their results are dropped), and the step that K ends in is done
// apart, element by element.  int8: rows on 16 bytes, at most 16 of them (others go through LDS, in dense_int8.hip).
template <int KIND, bool ROWS16, int MT, int CT>
struct DenseCursor {
    static_assert(KIND != kI8 || (ROWS16 && MT == 1), "");
    const uint8_t* b;          // this lane's bytes of the step, first column half of the tile
    __amdgpu_buffer_rsrc_t rows;
    const uint8_t* base;       // the tile's first row
    uint32_t off[MT];          // byte offset of this lane's k group in its row, or out of range
    int k, K;                  // first k of the lane's group in this step, and K, in units

    __device__ __forceinline__ void load_b(StepRegs<1, false, MT, CT>& s) {
#pragma unroll
        for (int c = 0; c < CT; ++c) {
            if constexpr (KIND == kI8) {
                s.b[c][0] = *reinterpret_cast<const u32x4*>(b + c * 1024);
                s.b[c][1] = *reinterpret_cast<const u32x4*>(b + c * 1024 + 512);
            } else {
                load_weights<false>(b + c * 1024, s.b[c]);
            }
        }
    }
    __device__ __forceinline__ void load(StepRegs<1, false, MT, CT>& s) {
        load_b(s);
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int l = 0; l < 2; ++l) {
                if constexpr (ROWS16)
                    s.a[m][0][l] = __builtin_bit_cast(
                        u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                   rows, k + l * 8 < K ? off[m] + l * 16 : kOutOfRange, 0, 0));
                else
                    s.a[m][0][l] = load_any<kBF16>(base + off[m] + l * 16);
            }
        b += kNW * step_bytes<false>();
        k += kNW * 64;
#pragma unroll
        for (int m = 0; m < MT; ++m) off[m] += kNW * 128;
    }
};

// The sums of a wave: float32's, or int32's.
template <int KIND, int MT, int CT> struct DenseAcc : Acc<1, KIND == kF16, false, MT, CT> {};
template <int MT, int CT>
struct DenseAcc<kI8, MT, CT> {
    intx4 v[MT][CT];

    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int c = 0; c < CT; ++c) v[m][c] = intx4{0, 0, 0, 0};
    }
    __device__ __forceinline__ void add(const StepRegs<1, false, MT, CT>& s) {
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int c = 0; c < CT; ++c)
#pragma unroll
                for (int m = 0; m < MT; ++m) v[m][c] = mfma16k<kI8>(s.a[m][0][q], s.b[c][q], v[m][c]);
    }
    __device__ __forceinline__ int value(int m, int c, int i) const { return v[m][c][i]; }
};

template <int KIND, bool ROWS16, int MT, int CT>
__global__ __launch_bounds__(kNW * 64, MT == 4 ? 1 : 2) void dense_stream_kernel(DenseArgs p) {
    typedef typename Sums<KIND>::one Sum;
    __shared__ __attribute__((aligned(16))) Sum s_red[kNW][MT][CT][4][kWave];
    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int unit = blockIdx.x, row0 = blockIdx.y * MT * kRowTile;
    // CT = 2: both halves of a pair; CT = 1: one half, or 8 columns of each
    const int pair = CT == 2 ? unit >> 1 : unit >> 2;
    const bool eights = CT == 1 && p.gated;            // uniform
    const int half = CT == 2 ? 0 : (eights ? (lane >> 3) & 1 : (unit >> 1) & 1);
    const int c0 = eights ? (unit & 3) * 8 - half * 8 : (unit & 1) * 16;   // column of the lane: c0 + lane % 16
    const int nk = ROWS16 ? (p.Kh + 63) / 64 : p.Kh / 64;
    DenseCursor<KIND, ROWS16, MT, CT> cur;
    cur.b = reinterpret_cast<const uint8_t*>(p.b) +
            (static_cast<int64_t>(pair) * (p.Kp / 64) + wave) * step_bytes<false>() + step_lane_offset<false>(half, c0);
    const uint8_t* first = reinterpret_cast<const uint8_t*>(p.a) + row0 * p.lda;
    cur.base = first;
    cur.rows = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(first), 0, kBufferRange, kBufferFlags);
    cur.k = wave * 64 + (lane >> 4) * 16;
    cur.K = p.Kh;
    const int steps = nk > wave ? (nk - wave + kNW - 1) / kNW : 0;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const int r = m * kRowTile + (lane & 15);
        const int row = ROWS16 ? r : min(r, p.M - 1 - row0);
        cur.off[m] = ROWS16 && row0 + r >= p.M
                         ? kOutOfRange
                         : static_cast<uint32_t>(row * static_cast<int>(p.lda) + cur.k * 2);
    }
    DenseAcc<KIND, MT, CT> acc;
    acc.clear();
    StepRegs<1, false, MT, CT> ring[MT == 1 ? 4 : 2];
    start_steps(steps, cur, ring);
    run_steps(steps, cur, ring, acc);
    if (!ROWS16 && p.K % 64 != 0 && wave == nk % kNW) {   // the cursor stands at the last, short step
        StepRegs<1, false, MT, CT> last;
        cur.load_b(last);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const int row = min(m * kRowTile + (lane & 15), p.M - 1 - row0);
#pragma unroll
            for (int l = 0; l < 2; ++l)
                last.a[m][0][l] = load_tail<kBF16>(first + static_cast<int64_t>(row) * p.lda, cur.k + l * 8, p.K);
        }
        acc.add(last);
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int c = 0; c < CT; ++c)
#pragma unroll
            for (int v = 0; v < 4; ++v) s_red[wave][m][c][v][lane] = acc.value(m, c, v);
    __syncthreads();
    for (int i = tid; i < MT * 256; i += kNW * 64) {
        const int m = i >> 8, v = (i >> 6) & 3;
        const int row = row0 + m * kRowTile + (lane >> 4) * 4 + v, cc = c0 + (lane & 15);
        if (CT == 1 && eights) {
            if (half != 0) continue;
            Sum g = 0, u = 0;
#pragma unroll
            for (int q = 0; q < kNW; ++q) {
                g += s_red[q][m][0][v][lane];
                u += s_red[q][m][0][v][lane + 8];
            }
            finish<KIND>(p, row, pair * 32 + cc, g, u);
            continue;
        }
        Sum s[CT];
#pragma unroll
        for (int c = 0; c < CT; ++c) {
            s[c] = 0;
#pragma unroll
            for (int q = 0; q < kNW; ++q) s[c] += s_red[q][m][c][v][lane];
        }
        if constexpr (CT == 1) {
            finish<KIND>(p, row, pair * 64 + half * 32 + cc, s[0], 0);
        } else if (p.gated) {
            finish<KIND>(p, row, pair * 32 + cc, s[0], s[1]);
        } else {
            finish<KIND>(p, row, pair * 64 + cc, s[0], 0);
            finish<KIND>(p, row, pair * 64 + 32 + cc, s[1], 0);
        }
    }
}

// ---- many rows: LDS tiles --------------------------------------------------------------
// A workgroup of 8 waves owns MW * NA * 32 rows x NW 64-column pairs.  Its waves
// are KG groups of MW x NW; a wave owns NA * 32 rows x one pair, NA x 2 tiles of
// v_mfma_f32_32x32x16, and the groups share out the k of a stage (small tiles:
// a stage has to be long, since its barriers cost the same whatever it holds).
// Both operands reach LDS by direct copies into a ring of kTileNB stages of SL
// slices of 32 k; the ring runs on from a tile into the workgroup's next one.
//
// The two waves of a SIMD (w and w + 4) alternate: while one runs a stage's MFMAs
// from registers, the other reads its next fragments from LDS and issues copies;
// a barrier ends each phase and the roles swap.  So the matrix unit always has a
// wave whose operands are ready, and one register set of fragments suffices (128
// accumulators + 48 fragment registers at NA = 4).
//   phase 2s:     waves 0-3 read stage s, waves 4-7 multiply stage s - 1
//   phase 2s + 1: waves 0-3 multiply stage s, waves 4-7 read stage s
// Stage s is read in phases 2s and 2s + 1 (the reads are complete at the phase's
// end), so from phase 2s + 2 on its buffer may be refilled: a wave reading stage
// s copies stage s + NB - 1 into the buffer of stage s - 1.  At the end of phase
// 2s + 1 every wave has issued copies up to stage s + NB - 1 and waits until its
// copies of stage s + 1 have landed.
//
// A's rows go through a buffer resource based at the tile's first row: rows past
// M and k past K copy zeros.
//
// Bound by the matrix unit at the clock the power limit leaves it (random inputs
// hold 1.7 GHz; zeros run a fifth faster): 8192^3 833 us, 1320 TFLOP/s (a library
// product 792); 6000 x 4096 x 4096 182 us, 1106 TFLOP/s (164), with bias and SiLU
// 186 (164 and two passes over C: 207), 192 x 256 tiles, of which 512 fill the chip
// exactly twice.  Besides the clock LDS bounds it: a stage of the 256 x 256 tile
// reads 96 KB and copies 32 KB while the MFMAs take 1024
// cycles (without the MFMAs 685 us, without the copies 775, then 899 in all).
// Tried at 8192^3, then 851 us: 4 waves of 128 x 128 each 897 us, weights straight
// to registers 893, copies issued in the multiplying phase 929.
constexpr int kTileNB = 4;
constexpr int kTileBK = 32;

__device__ __forceinline__ int tile_swz(int row, int kg) {
    // 16-byte granule kg of a 64-byte row, XORed so that a fragment read's 16
    // consecutive rows fall into different banks
    return row * kTileBK + ((kg ^ ((row >> 2) & 3)) << 3);
}

template <int KIND>
__device__ __forceinline__ typename Sums<KIND>::sixteen mfma32d(const u32x4& a, const u32x4& b,
                                                                typename Sums<KIND>::sixteen c) {
    if constexpr (KIND == kI8)
        return __builtin_amdgcn_mfma_i32_32x32x32_i8(__builtin_bit_cast(i8x16_t, a), __builtin_bit_cast(i8x16_t, b), c,
                                                     0, 0, 0);
    else if constexpr (KIND == kF16)
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(halfx8_t, a),
                                                      __builtin_bit_cast(halfx8_t, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b),
                                                       c, 0, 0, 0);
}

// One 16-byte-per-lane buffer -> LDS copy: lane l's bytes, at its offset plus the
// uniform one, land at the wave's base + 16 l.
__device__ __forceinline__ void copy_to_lds(__amdgpu_buffer_rsrc_t rsrc, void* lds_wave_base, int lane_offset,
                                            int offset) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        rsrc, reinterpret_cast<__attribute__((address_space(3))) void*>(reinterpret_cast<uintptr_t>(lds_wave_base)),
        16, lane_offset, offset, 0, 0);
}

// End of a phase: nothing moves across it.
__device__ __forceinline__ void phase_end() {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

// The same where LDS written before it is read after it.
__device__ __forceinline__ void phase_end_lds() {
    wait_lgkmcnt0();
    phase_end();
}

// The end of a wave's NA * 32 rows x 64 columns: a register holds column lane % 32, row 8 (v / 4) + 4 (lane / 32) + v % 4
// of a 32 x 32 tile; 16 rows at a time go through LDS (columns XORed by 32 in every other group of four rows, against
// bank conflicts), so that a lane ends up with four columns of a row.  KG waves hold sums of the same rows, added in
// LDS in their order: `mine` is the wave's place, `parts` the first's, the others' STRIDE places apart.  One copy of the
// code for all of the registers: rows are loaded and finished in a loop, and only the way to LDS is written out.
// `first` is the wave's first row.
template <int KIND, int NA, int KG, int STRIDE, bool VEC>
__device__ __forceinline__ void finish_tile(const DenseArgs& p, const typename Sums<KIND>::sixteen (&acc)[NA][2],
                                            typename Sums<KIND>::one (*mine)[64], const typename Sums<KIND>::one (*parts)[64],
                                            int kg, int first, int col, const Columns& columns,
                                            const float (&sa)[(NA + 1) / 2]) {
    typedef typename Sums<KIND>::one Sum;
    typedef typename Sums<KIND>::four Sum4;
    typedef Finisher<KIND, VEC> Finish;
    const int lane = threadIdx.x & (kWave - 1);
    const int lc = p.gated ? (lane & 7) * 4 : (lane & 15) * 4;
    const int lr = p.gated ? lane >> 3 : lane >> 4;    // of the rows that a wave takes at once
    auto put = [&](auto i, auto hf) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int v = 0; v < 8; ++v) {
                const int r = 8 * (v >> 2) + 4 * (lane >> 5) + (v & 3);
                mine[r][((lane & 31) + 32 * j) ^ ((lane >> 5) * 32)] = acc[decltype(i)::value][j][decltype(hf)::value * 8 + v];
            }
        // keeps the compiler from making one block of two cases, whose registers would have to lie in memory
        asm volatile("; rows %0" ::"n"(decltype(i)::value * 2 + decltype(hf)::value));
    };
    with_activation(p.act, [&](auto act) __attribute__((always_inline)) {
        constexpr int ACT = decltype(act)::value;
        constexpr int dr = ACT == MOE_EPI_SWIGLU ? 8 : 4;      // rows a wave takes at once
        constexpr int R = KG * dr < 16 ? 16 / (KG * dr) : 1;   // times that for its share of 16
        const int mine0 = kg * dr;                             // the first of it; 16 and more: none
        u32x4 part[R];
        Finish f(p, first, lr, col);
        auto load = [&]() __attribute__((always_inline)) {
#pragma unroll
            for (int i = 0; i < R; ++i) part[i] = f.load(mine0 + i * KG * dr);
            f.next_r(16);
        };
        constexpr bool kAhead = KIND == kI8 || NA < 4;         // 128 float32 sums and 48 of fragments leave no room for it
        if (kAhead && mine0 < 16) load();
#pragma unroll 1
        for (int g = 0; g < NA * 2; ++g) {
            switch (g) {                               // uniform
                case 0: put(IntC<0>{}, IntC<0>{}); break;
                case 1: put(IntC<0>{}, IntC<1>{}); break;
                case 2: if constexpr (NA > 1) put(IntC<1>{}, IntC<0>{}); break;
                case 3: if constexpr (NA > 1) put(IntC<1>{}, IntC<1>{}); break;
                case 4: if constexpr (NA > 2) put(IntC<2>{}, IntC<0>{}); break;
                case 5: if constexpr (NA > 2) put(IntC<2>{}, IntC<1>{}); break;
                case 6: if constexpr (NA > 3) put(IntC<3>{}, IntC<0>{}); break;
                default: if constexpr (NA > 3) put(IntC<3>{}, IntC<1>{}); break;
            }
            if constexpr (KG > 1) phase_end_lds();
            if (mine0 < 16) {
                u32x4 now[R];
                if constexpr (!kAhead) load();
#pragma unroll
                for (int i = 0; i < R; ++i) now[i] = part[i];
                if (kAhead && g + 1 < NA * 2) load();
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    const int r = mine0 + i * KG * dr + lr, x = (r & 4) * 8;
                    Sum4 v = {0, 0, 0, 0}, u = v, ev[KG], eu[KG];
#pragma unroll
                    for (int q = 0; q < KG; ++q) {
                        const Sum* e = &parts[q * STRIDE * 16 + r][0];
                        ev[q] = *reinterpret_cast<const Sum4*>(e + (lc ^ x));
                        if constexpr (ACT == MOE_EPI_SWIGLU) eu[q] = *reinterpret_cast<const Sum4*>(e + ((lc + 32) ^ x));
                    }
                    if constexpr (KG > 1) __builtin_amdgcn_sched_barrier(0);   // all on their way before the first is added
#pragma unroll
                    for (int q = 0; q < KG; ++q) {
                        v += ev[q];
                        if constexpr (ACT == MOE_EPI_SWIGLU) u += eu[q];
                    }
                    float scale = 0.0f;
                    if constexpr (KIND == kI8) {
                        scale = __shfl(sa[0], g * 16 + r, kWave);
                        if constexpr (NA > 2) scale = g < 4 ? scale : __shfl(sa[1], g * 16 + r, kWave);
                    }
                    f.template finish<ACT>(mine0 + i * KG * dr, v, u, columns, scale, now[i]);
                }
                f.next_c(16);
            }
            if constexpr (KG > 1) phase_end_lds();
        }
    });
}

template <int KIND, bool VEC, int MW, int NW, int NA, int SL>
__global__ __launch_bounds__(512, 1) void dense_tile_kernel(DenseArgs p, int mtiles, int ntiles, int pairs) {
    static_assert(KIND != kI8, "int8 tiles are dense_int8.hip's");
    constexpr int KG = 8 / (MW * NW);                  // wave groups along k
    constexpr int WS = SL * 2 / KG;                    // k-steps of 16 of a wave per stage
    constexpr int UM = MW * NA * 32;                   // rows of the tile
    constexpr int AB = UM / 16;                        // 16-row copy blocks of a slice
    constexpr int AC = (SL * AB + 7) / 8;              // copy blocks per wave and stage
    constexpr int BD = SL * NW * 4 / 8;                // 1 KiB weight blocks per wave and stage
    constexpr int LOADS = AC + BD;
    static_assert(KG * WS == SL * 2 && (SL * NW * 4) % 8 == 0, "a stage splits evenly");
    static_assert(BD <= 4 && 4 % BD == 0, "a wave's weight blocks lie in one pair and slice");
    __shared__ __attribute__((aligned(16))) uint16_t s_a[kTileNB][AC * 8 * 16 * kTileBK];   // [slice][row][32]
    __shared__ __attribute__((aligned(16))) uint16_t s_b[kTileNB][SL * NW * 4][512];        // [slice][pair][4]
    __shared__ __attribute__((aligned(16))) float s_e[8][16][64];     // epilogue: 16 rows of each wave
    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const bool late = wave >= 4;                       // reads in odd phases
    const int kg = wave / (MW * NW), mh = (wave / NW) % MW, nq = wave % NW;
    // stages, in whole turns of the ring (a stage past K multiplies zeros), so that ring places are constants
    const int nk32 = p.Kp / kTileBK, nk = (nk32 + SL * kTileNB - 1) / (SL * kTileNB) * kTileNB;
    const int total = mtiles * ntiles;
    const int G = gridDim.x, b = blockIdx.x;
    // A workgroup's only tile may leave the zero stages out.  The longest stages do (1000 x 1024 x 1096: 13.4 -> 12.5
    // us); with shorter ones the test costs more than the at most three stages (1024 x 4096 x 4096: 49 -> 51 us).
    const int run = SL > 2 && total <= G ? (nk32 + SL - 1) / SL : nk;
    // one contiguous range of tiles per XCD and round, 8 row tiles x 4 column tiles of it at a time
    const int lid = (G % 8 == 0) ? (b % 8) * (G / 8) + (b / 8) : b;
    constexpr int kGroup = 8;
    auto place = [&](int tile, int& m_tile, int& n_tile) {
        const int group = tile / (kGroup * ntiles), in = tile - group * kGroup * ntiles;
        const int gm = min(kGroup, mtiles - group * kGroup);
        n_tile = in / gm;
        m_tile = group * kGroup + in - n_tile * gm;
    };
    // what this wave copies of a tile: A blocks i * 8 + wave (slice, then row block; lane: row lane / 4,
    // granule position lane % 4) and weight blocks wave * BD + d (slice, pair, block)
    struct Source {
        __amdgpu_buffer_rsrc_t a, b;
        uint32_t a_off[AC];
    };
    int a_k[AC];
#pragma unroll
    for (int i = 0; i < AC; ++i) {
        const int row = (i * 8 + wave) % AB * 16 + (lane >> 2);
        a_k[i] = ((lane & 3) ^ ((row >> 2) & 3)) * 8;
    }
    const int b_slice = wave * BD / (NW * 4), b_pair = wave * BD / 4 % NW, b_first = wave * BD % 4;
    auto source = [&](int tile) {
        Source s;
        int m_tile, n_tile;
        place(tile, m_tile, n_tile);
        const int row0 = m_tile * UM;
        s.a = __builtin_amdgcn_make_buffer_rsrc(
            reinterpret_cast<uint8_t*>(const_cast<uint16_t*>(p.a)) + static_cast<int64_t>(row0) * p.lda, 0,
            kBufferRange, kBufferFlags);
#pragma unroll
        for (int i = 0; i < AC; ++i) {
            const int blk = i * 8 + wave, row = blk % AB * 16 + (lane >> 2);
            s.a_off[i] = blk < SL * AB && row0 + row < p.M
                             ? static_cast<uint32_t>(row * static_cast<int>(p.lda) + a_k[i] * 2)
                             : kOutOfRange;
        }
        const int pair = min(n_tile * NW + b_pair, pairs - 1);
        s.b = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<uint16_t*>(p.b) + static_cast<int64_t>(pair) * nk32 * (kStepBytes / 2), 0, kBufferRange,
            kBufferFlags);
        return s;
    };
    // Copies of stage kt of a tile into ring place st.  The place along k is the
    // uniform offset of a copy; only a slice that K ends in, or past K, looks at
    // each lane's k.  Past the packed end both sides are zero: a weight read again
    // there would turn an infinity of the last slice into NaN.
    auto issue = [&](const Source& s, int kt, int st) {
#pragma unroll
        for (int i = 0; i < AC; ++i) {
            const int k0 = (kt * SL + (i * 8 + wave) / AB) * kTileBK;
            uint32_t off = s.a_off[i];
            if (k0 + kTileBK > p.Kh) off = k0 + a_k[i] < p.Kh ? off : kOutOfRange;   // uniform condition
            copy_to_lds(s.a, &s_a[st][(i * 8 + wave) * 16 * kTileBK], static_cast<int>(off), k0 * 2);
        }
        const int ks = kt * SL + b_slice, kc = min(ks, nk32 - 1);
        const int off_b = ks < nk32 ? lane * 16 : static_cast<int>(kOutOfRange);
#pragma unroll
        for (int d = 0; d < BD; ++d)
            copy_to_lds(s.b, &s_b[st][wave * BD + d][0], off_b, kc * kStepBytes + (b_first + d) * 1024);
    };

    int tile = lid;                                    // the grid has no more workgroups than tiles
    Source cur = source(tile);
#pragma unroll
    for (int q = 0; q + 1 < kTileNB; ++q) issue(cur, q, q);
    wait_vmcnt<LOADS * (kTileNB - 2)>();
    phase_end();
    for (;;) {
        const bool more = tile + G < total;            // uniform
        const Source next = source(more ? tile + G : tile);
        // what the epilogue needs of this tile's columns, loaded ahead where registers are left for it
        int m_tile, n_tile;
        place(tile, m_tile, n_tile);
        const int lc = p.gated ? (lane & 7) * 4 : (lane & 15) * 4;
        const int first = mh * NA * 32, col = (n_tile * NW + nq) * (p.gated ? 32 : 64) + lc;   // of the wave's part
        Columns columns;
        if constexpr (NA < 4) columns = load_columns<KIND>(p, col);
        floatx16 acc[NA][2];
#pragma unroll
        for (int i = 0; i < NA; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int v = 0; v < 16; ++v) acc[i][j][v] = 0;

        u32x4 fa[WS][NA], fb[WS][2];
        auto read_stage = [&](int st) {
#pragma unroll
            for (int w = 0; w < WS; ++w) {
                const int ks = kg * WS + w, slice = ks >> 1, kq = (ks & 1) * 2 + (lane >> 5);
#pragma unroll
                for (int i = 0; i < NA; ++i)
                    fa[w][i] = *reinterpret_cast<const u32x4*>(
                        &s_a[st][slice * (UM * kTileBK) + tile_swz((mh * NA + i) * 32 + (lane & 31), kq)]);
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    fb[w][j] =
                        *reinterpret_cast<const u32x4*>(&s_b[st][(slice * NW + nq) * 4 + 2 * (ks & 1) + j][lane * 8]);
            }
        };
        auto multiply = [&]() {
            __builtin_amdgcn_s_setprio(1);
#pragma unroll
            for (int w = 0; w < WS; ++w)
#pragma unroll
                for (int i = 0; i < NA; ++i) {
                    acc[i][0] = mfma32d<KIND>(fa[w][i], fb[w][0], acc[i][0]);
                    acc[i][1] = mfma32d<KIND>(fa[w][i], fb[w][1], acc[i][1]);
                }
            __builtin_amdgcn_s_setprio(0);
        };
        if (late) phase_end();                         // the first phase belongs to waves 0-3
        for (int s0 = 0; s0 < nk; s0 += kTileNB) {
            const bool last = s0 + kTileNB == nk;      // uniform
#pragma unroll
            for (int q = 0; q < kTileNB; ++q) {
                if constexpr (SL > 2)
                    if (s0 + q >= run) break;          // uniform
                // phase 2s (late: 2s + 1): read stage s = s0 + q, refill the buffer of stage s - 1
                read_stage(q);
                if (q == 0 || !last) issue(cur, s0 + q + kTileNB - 1, (q + kTileNB - 1) % kTileNB);
                else issue(next, q - 1, q - 1);
                if (late) wait_vmcnt<LOADS * (kTileNB - 2)>();
                wait_lgkmcnt0();
                phase_end();
                // phase 2s + 1 (late: 2s + 2): multiply
                multiply();
                if (!late) wait_vmcnt<LOADS * (kTileNB - 2)>();
                phase_end();
            }
        }
        if (!late) phase_end();                        // the late waves' last multiply

        if constexpr (NA >= 4) columns = load_columns<KIND>(p, col);
        constexpr float no_scales[(NA + 1) / 2] = {};
        finish_tile<KIND, NA, KG, MW * NW, VEC>(p, acc, s_e[wave], s_e[mh * NW + nq], kg, m_tile * UM + first, col, columns, no_scales);
        if (!more) break;
        tile += G;
        cur = next;
    }
    wait_vmcnt<0>();                                   // no copy is in flight when the workgroup's LDS is given back
}

// ---- which kernel and shape ---------------------------------------------------------------
// The reduction in 16-bit units, padded to whole steps of 64.
template <int KIND>
inline int k_padded(const moe_dense_shape& s) {
    constexpr int step = 64 * codes_per_unit<KIND>();
    return static_cast<int>((static_cast<int64_t>(s.K) + step - 1) / step * 64);
}
inline int64_t pairs_of(const moe_dense_shape& s) {
    const int w = s.gated ? 32 : 64;
    return (static_cast<int64_t>(s.N) + w - 1) / w;
}

constexpr int kCUs = 256;
constexpr int kStreamRows = 512;                       // most rows the weight-streaming kernel is considered for

// A kernel's shape and the time expected of it, in ns.
struct Choice {
    int shape;
    double ns;
};

template <int KIND, bool ROWS16, int MT, int CT>
int launch_stream_tiles(const DenseArgs& p, int64_t pairs, hipStream_t st) {
    const dim3 g(static_cast<unsigned>(pairs * (4 / CT)), (p.M + MT * kRowTile - 1) / (MT * kRowTile));
    hipLaunchKernelGGL((dense_stream_kernel<KIND, ROWS16, MT, CT>), g, dim3(kNW * 64), 0, st, p);
    MOE_CHECK_LAUNCH();
    return MOE_OK;
}

// Unit shape: what the busiest CU reads, at the 37 bytes/ns it gets from the
// caches (half that with unaligned rows), decides; few rows are bound there and
// not by memory.  64 x 1024 x 4096: 16 x 16 8.1 us, 64 x 16 19.7; 64 x 4096 x
// 4096: 32 x 32 16.1 us, 64 x 16 20.8; 16 x 8192 x 4096: 16 x 32 12.8 us, 16 x 16
// 16.0.  Expected times were within 20 % of measured ones from 4 to 65 us.
struct UnitShape {
    int mt, ct;
};
constexpr UnitShape kUnitShapes[] = {{4, 2}, {2, 2}, {2, 1}, {1, 2}, {1, 1}};   // 4, 1 reads more than 2, 2 always
constexpr int kUnitShape11 = 4;

Choice stream_choice(const DenseArgs& p, int64_t pairs, bool rows16) {
    Choice best{0, 0.0};
    for (int i = 0; i < 5; ++i) {
        const int ct = kUnitShapes[i].ct, rows = kUnitShapes[i].mt * kRowTile;
        if (rows > kRowTile && p.M <= rows / 2) continue;   // half of its rows would be past M
        const int64_t groups = pairs * (4 / ct) * ((p.M + rows - 1) / rows);
        const int64_t read = (groups + kCUs - 1) / kCUs * (std::min(rows, p.M) + ct * kRowTile) * p.Kp * 2;
        const double ns = read / (rows16 ? 37.0 : 18.5) + 2000.0;
        if (best.ns == 0.0 || ns < best.ns) best = Choice{i, ns};
    }
    return best;
}

template <int KIND, bool ROWS16>
int launch_stream(const DenseArgs& p, int64_t pairs, int shape, hipStream_t st) {
    switch (shape) {
        case 0: return launch_stream_tiles<KIND, ROWS16, 4, 2>(p, pairs, st);
        case 1: return launch_stream_tiles<KIND, ROWS16, 2, 2>(p, pairs, st);
        case 2: return launch_stream_tiles<KIND, ROWS16, 2, 1>(p, pairs, st);
        case 3: return launch_stream_tiles<KIND, ROWS16, 1, 2>(p, pairs, st);
        default: return launch_stream_tiles<KIND, ROWS16, 1, 1>(p, pairs, st);
    }
}

template <int KIND, bool VEC, int MW, int NW, int NA, int SL>
int launch_tile(const DenseArgs& p, int64_t pairs, hipStream_t st) {
    constexpr int UM = MW * NA * 32;
    const int ntiles = static_cast<int>((pairs + NW - 1) / NW), mtiles = (p.M + UM - 1) / UM;
    const int64_t tiles = static_cast<int64_t>(mtiles) * ntiles;
    const unsigned grid = static_cast<unsigned>(tiles < kCUs ? tiles : kCUs);   // persistent, one to a CU
    hipLaunchKernelGGL((dense_tile_kernel<KIND, VEC, MW, NW, NA, SL>), dim3(grid), dim3(512), 0, st, p, mtiles, ntiles,
                       static_cast<int>(pairs));
    MOE_CHECK_LAUNCH();
    return MOE_OK;
}

// Tile shape: the least time of the busiest CU.  A stage takes the longer of its
// multiplications and its copies, and a fixed part for its two barriers.
struct TileShape {
    int rows, pairs, slices;
};
constexpr TileShape kTileShapes[] = {{256, 4, 1}, {192, 4, 1}, {128, 4, 1}, {128, 2, 2}, {64, 2, 2}, {64, 1, 4}};

Choice tile_choice(const DenseArgs& p, int64_t pairs) {
    Choice best{0, 0.0};
    for (int i = 0; i < 6; ++i) {
        const TileShape& t = kTileShapes[i];
        const int64_t tiles = ((p.M + t.rows - 1) / t.rows) * ((pairs + t.pairs - 1) / t.pairs);
        const int64_t stages = (p.Kp / kTileBK + t.slices - 1) / t.slices + 8;
        const double mul = t.rows * t.pairs * t.slices / 1024.0 * 1200, copy = (t.rows + t.pairs * 64) * t.slices / 512.0 * 850;
        const double cycles = static_cast<double>((tiles + kCUs - 1) / kCUs) * stages * ((mul > copy ? mul : copy) + 250);
        const double ns = cycles * 0.52 + 2000.0;      // about 1.9 GHz, and what a launch takes
        if (best.ns == 0.0 || ns < best.ns) best = Choice{i, ns};
    }
    return best;
}

template <int KIND, bool VEC>
int launch_tiles(const DenseArgs& p, int64_t pairs, int shape, hipStream_t st) {
    switch (shape) {
        case 0: return launch_tile<KIND, VEC, 2, 4, 4, 1>(p, pairs, st);
        case 1: return launch_tile<KIND, VEC, 2, 4, 3, 1>(p, pairs, st);
        case 2: return launch_tile<KIND, VEC, 2, 4, 2, 1>(p, pairs, st);
        case 3: return launch_tile<KIND, VEC, 2, 2, 2, 2>(p, pairs, st);
        case 4: return launch_tile<KIND, VEC, 1, 2, 2, 2>(p, pairs, st);
        default: return launch_tile<KIND, VEC, 1, 1, 2, 4>(p, pairs, st);
    }
}

// Whether the rows of a tile, of A, and that many rows of R and C lie within a buffer's range.
inline bool a_near(const DenseArgs& p) { return p.lda * 256 <= kBufferRange; }
inline bool out_near(const DenseArgs& p, int rows) {
    const int64_t widest = std::max(p.ldc * (p.c_dtype == MOE_F32 ? 4 : 2), p.r == nullptr ? 0 : p.ldr * (p.r_dtype == MOE_F32 ? 4 : 2));
    return widest <= (kBufferRange - MOE_DENSE_MAX_COLS * 4) / rows;
}

template <int KIND>
int launch_any(const DenseArgs& p, int64_t pairs, hipStream_t st) {
    const dim3 g(static_cast<unsigned>(pairs), (p.M + 63) / 64);
    if (KIND == kI8 || !out_near(p, 16))               // int8 rows within reach take another kernel
        hipLaunchKernelGGL((dense_any_kernel<KIND, kFarRows>), g, dim3(256), 0, st, p);
    else if constexpr (KIND != kI8) {
        if (p.vec) hipLaunchKernelGGL((dense_any_kernel<KIND, kByFour>), g, dim3(256), 0, st, p);
        else hipLaunchKernelGGL((dense_any_kernel<KIND, kByOne>), g, dim3(256), 0, st, p);
    }
    MOE_CHECK_LAUNCH();
    return MOE_OK;
}

// 16-bit operands.
template <int KIND>
int launch_dense(const DenseArgs& p, int64_t pairs, hipStream_t st) {
    // direct copies to LDS and 16-byte buffer loads need every row to start on 16
    // bytes, and a k group to end within the row
    const bool rows16 = reinterpret_cast<uintptr_t>(p.a) % 16 == 0 && p.lda % 16 == 0 && p.K % 8 == 0;
    // byte offsets within a tile of rows stay below the buffer range (streaming finishes an element at a time, at any
    // address of C and R)
    const bool near = a_near(p);
    const Choice stream = stream_choice(p, pairs, rows16);
    const bool few = near && p.M <= kStreamRows;
    if (rows16 && near && out_near(p, 16)) {
        // 96 x 12288 x 4096: tiles 38.5 us, streaming 64.8; 256 x 1024 x 4096: 19.6 and 13.6
        const Choice tile = tile_choice(p, pairs);
        if (!few || stream.ns > tile.ns)
            return p.vec ? launch_tiles<KIND, true>(p, pairs, tile.shape, st)
                         : launch_tiles<KIND, false>(p, pairs, tile.shape, st);
        return launch_stream<KIND, true>(p, pairs, stream.shape, st);
    }
    // a stage of the any-alignment kernel takes about 1.65 us while its workgroups fit the chip twice over.
    // 128 x 1003 x 1091: streaming 8.2 us, 16.2 there; 128 x 4099 x 1091: 26.3 and 16.4
    const double rounds = std::max(1.0, static_cast<double>(pairs) * ((p.M + 63) / 64) / (2 * kCUs));
    if (few && stream.ns <= (p.Kp + kAnyK - 1) / kAnyK * 1650.0 * rounds)
        return rows16 ? launch_stream<KIND, true>(p, pairs, stream.shape, st)
                      : launch_stream<KIND, false>(p, pairs, stream.shape, st);
    return launch_any<KIND>(p, pairs, st);
}

// All of a product but its operands.
inline DenseArgs dense_args(const moe_dense_shape& s, int epilogue, const float* bias, const void* r, int r_dtype,
                            int64_t ldr, void* c, int c_dtype, int64_t ldc) {
    DenseArgs p{};
    p.bias = bias;
    p.r = r;
    p.c = c;
    p.ldr = ldr;
    p.ldc = ldc;
    p.M = s.M;
    p.N = s.N;
    p.K = s.K;
    p.gated = s.gated;
    p.act = epilogue;
    p.r_dtype = r_dtype;
    p.c_dtype = c_dtype;
    auto on_four = [](const void* q, int64_t ld, int dtype) {
        return reinterpret_cast<uintptr_t>(q) % (dtype == MOE_F32 ? 16 : 8) == 0 && ld % 4 == 0;
    };
    p.vec = s.N % 4 == 0 && on_four(c, ldc, c_dtype) && (r == nullptr || on_four(r, ldr, r_dtype));
    return p;
}

}  // namespace
}  // namespace moe
