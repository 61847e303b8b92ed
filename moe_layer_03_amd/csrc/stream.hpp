// Weight-streaming products of a few rows: the building blocks shared by the
// few-token layer and the dense product.
//
// A wave multiplies up to MT * 16 rows by CT tiles of 16 columns with
// v_mfma_f32_16x16x32: every weight element passes through the wave's
// registers exactly once, so the product runs at the rate the weights arrive.
// Weights come in the packed layouts of the grouped GEMMs, which keep a 64-column
// pair's reduction contiguous; a step here is 64 k of it:
//   16-bit:  8 KiB, [4 k blocks of 16][2 column halves][64 lanes][16 bytes],
//   MXFP8:   4 KiB, [2 column halves][2 scale blocks of 32 k][64 lanes][16 bytes],
// and in both a lane slot is (column c of 32) + 32 * (k half of the block).  Lane l
// takes column l % 16 of 16 and k group l / 16, 16 consecutive k of the step, as
// two MFMA operands of 8 (the MFMA's own order of k does not matter as long as
// both operands share it).  So a row's four lanes read 128 consecutive bytes, a
// whole cache line, in two loads (32 rows of 4096 x 4096: 15.8 us, against 18.0 us
// with 64 bytes of a line at a time).
//
// Rows are held as NP 16-bit parts whose sum is the row's value:
//   1 part: the value itself;
//   2 parts (fp16): v = p0 + 2^-11 p1, |error| <= 2^-22 |v| for 2^-14 <= |v| <=
//     65504 (p1 is scaled up so that it stays a normal fp16 number), 2^-36 below,
//     so callers scale rows by a power of two; the parts have their own
//     accumulators, joined at the end;
//   3 parts (bf16): v = p0 + p1 + p2, exact for |v| >= 2^-102; one accumulator.
// The MFMAs of the extra parts are free here: the weights' arrival bounds the
// product, and a row held to 22 bits or more keeps the float32 output's digits.
#pragma once

#include "gemm_common.hpp"

namespace moe {
namespace {

constexpr float kLoScale = 2048.0f;                    // 2^11, the second fp16 part's scale
constexpr int kStepBytes = 4096;                       // 16-bit packed weights of a 64-column pair per 32 k
template <bool MX> constexpr int step_bytes() { return MX ? 4096 : 8192; }   // of a step
constexpr int kRowTile = 16;                           // rows (and columns) of an MFMA tile

// Barrier for LDS data; loads to registers stay in flight across it.
__device__ __forceinline__ void lds_barrier() {
    wait_lgkmcnt0();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

__device__ __forceinline__ floatx4 mfma16(bool f16, const u32x4& a, const u32x4& b, floatx4 c) {
    if (f16)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(halfx8_t, a),
                                                      __builtin_bit_cast(halfx8_t, b), c, 0, 0, 0);
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c,
                                                   0, 0, 0);
}

// Eight E4M3 codes (two words) times 2^(scale byte - 127), as bf16: exact, a code has 4 significant bits.
__device__ __forceinline__ u32x4 mx_to_bf16(uint32_t w0, uint32_t w1, uint32_t scale_byte) {
    const float s = __uint_as_float(scale_byte << 23);
    u32x4 r;
    r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, s, false));
    r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, s, true));
    r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, s, false));
    r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, s, true));
    return r;
}

// fp16, saturating at 65504; NaN stays NaN.
__device__ __forceinline__ uint16_t f32_to_f16_or_nan(float v) { return v == v ? f32_to_f16_sat(v) : uint16_t{0x7E00}; }

// bf16, to nearest even; NaN of any payload stays NaN (f32_to_bf16 takes finite
// values only: it carries a full payload into the sign).  One instruction.
__device__ __forceinline__ uint16_t f32_to_bf16_or_nan(float v) {
    return __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
}
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef float floatx2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t pack_bf16x2_or_nan(float lo, float hi) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((floatx2{lo, hi}), bf16x2_t));
}

// Parts of v (see above); fp16 saturates at 65504, NaN stays in the first part.
// bf16 parts are cut off, not rounded: three times the top 8 of the 24 bits left,
// exact, and the first part of no number becomes infinite.  A NaN whose payload
// is cut off leaves an infinity in the first part and NaN in the second.
template <int NP, bool F16>
__device__ __forceinline__ void split_parts(float v, uint16_t (&p)[NP]) {
    if constexpr (F16) {
        p[0] = f32_to_f16_or_nan(v);
        if constexpr (NP == 2) {
            const float c = fminf(fmaxf(v, -65504.0f), 65504.0f);
            p[1] = f32_to_f16_sat((c - f16_to_f32(p[0])) * kLoScale);
        }
    } else {
        float rest = v;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            p[i] = static_cast<uint16_t>(__float_as_uint(rest) >> 16);
            rest -= bf16_to_f32(p[i]);                 // exact
        }
    }
}

// One step's operands of a wave: CT column tiles, MT row tiles of NP parts.
template <int NP, bool MX, int MT, int CT>
struct StepRegs {
    u32x4 b[CT][MX ? 1 : 2];
    uint32_t sc[MX ? CT : 1];
    u32x4 a[MT][NP][2];
};

template <int NP, bool F16, bool MX, int MT, int CT>
struct Acc {
    static constexpr int NA = (F16 && NP == 2) ? 2 : 1;
    floatx4 v[NA][MT][CT];

    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int n = 0; n < NA; ++n)
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int c = 0; c < CT; ++c) v[n][m][c] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    __device__ __forceinline__ void add(const StepRegs<NP, MX, MT, CT>& s) {
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int c = 0; c < CT; ++c) {
                u32x4 b;
                if constexpr (MX) b = mx_to_bf16(s.b[c][0][2 * q], s.b[c][0][2 * q + 1], s.sc[c]);
                else b = s.b[c][q];
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int p = 0; p < NP; ++p) {
                        const int n = NA == 2 ? p : 0;
                        v[n][m][c] = mfma16(F16, s.a[m][p][q], b, v[n][m][c]);
                    }
            }
    }
    __device__ __forceinline__ float value(int m, int c, int i) const {
        if constexpr (NA == 2) return v[0][m][c][i] + v[1][m][c][i] * (1.0f / kLoScale);
        else return v[0][m][c][i];
    }
};

// Byte offset of this lane's weights within a step: column half `half`, columns
// c0 .. c0 + 15 of it (c0 0 or 16).  16-bit: its first 8 k; the next 8 are 512
// bytes further.
template <bool MX>
__device__ __forceinline__ int step_lane_offset(int half, int c0) {
    const int lane = threadIdx.x & (kWave - 1);
    const int col = lane & 15, kq = lane >> 4;
    return MX ? half * 2048 + (kq >> 1) * 1024 + ((kq & 1) * 32 + c0 + col) * 16
              : kq * 2048 + half * 1024 + (c0 + col) * 16;
}

template <bool MX>
__device__ __forceinline__ void load_weights(const uint8_t* p, u32x4 (&b)[MX ? 1 : 2]) {
    b[0] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));   // read once
    if constexpr (!MX) b[1] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p + 512));
}

// A row's 16 k of a step at a byte offset into a buffer.
__device__ __forceinline__ void load_row(__amdgpu_buffer_rsrc_t rows, uint32_t off, u32x4 (&a)[2]) {
    a[0] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rows, off, 0, 0));
    a[1] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rows, off + 16, 0, 0));
}

// A product of n steps whose first D loads are already on their way: start_steps
// issues them (cur.load(regs) issues the loads of cur's next step), run_steps adds
// all n steps, loading D ahead (after() follows each).  Whole turns of the ring have no branch inside, so
// the wait before a step leaves the younger D - 1 steps' loads in flight; only
// the last turns test whether a step is there.
template <int D, int NP, bool MX, int MT, int CT, typename Cursor>
__device__ __forceinline__ void start_steps(int n, Cursor& cur, StepRegs<NP, MX, MT, CT> (&ring)[D]) {
#pragma unroll
    for (int j = 0; j < D; ++j)
        if (j < n) cur.load(ring[j]);                  // uniform
}

template <int D, int NP, bool F16, bool MX, int MT, int CT, typename Cursor, typename After>
__device__ __forceinline__ void run_steps(int n, Cursor& cur, StepRegs<NP, MX, MT, CT> (&ring)[D],
                                          Acc<NP, F16, MX, MT, CT>& acc, After&& after) {
    int i = 0;
    for (; i + 2 * D <= n; i += D) {
#pragma unroll
        for (int j = 0; j < D; ++j) {
            acc.add(ring[j]);
            cur.load(ring[j]);
            after();
        }
    }
#pragma unroll
    for (int j = 0; j < 2 * D - 1; ++j)
        if (i + j < n) {                               // uniform
            acc.add(ring[j % D]);
            if (j < D && i + j + D < n) cur.load(ring[j % D]);
            after();
        }
}

template <int D, int NP, bool F16, bool MX, int MT, int CT, typename Cursor>
__device__ __forceinline__ void run_steps(int n, Cursor& cur, StepRegs<NP, MX, MT, CT> (&ring)[D],
                                          Acc<NP, F16, MX, MT, CT>& acc) {
    run_steps(n, cur, ring, acc, [] {});
}

}  // namespace
}  // namespace moe
