// Dense products of int8 codes with a scale per row of A and per column of W:
//   C = act((sum_k a w) sa sw + bias) + R,   or, gated, with a gate and an up weight.
// The sums are int32 and exact (K is at most 131071, |a w| at most 2^14), so no order of them matters; the kernels
// are of the 16-bit products' kind (dense.hpp), with sixteen codes in the bytes of eight values.
//
// Packed weights: the 16-bit layout with a code in each byte, blocks of 32 columns x 32 k, K padded to a multiple of
// 128; then the columns' scales, padded to the packed columns (gated: the gate's, then the up's).
#include "dense.hpp"
#include "int8.hpp"

namespace moe {
namespace {

template <typename ST>
__device__ __forceinline__ float weight_at(const ST* w, int64_t i, int dtype) {
    if constexpr (sizeof(ST) == 4) return w[i];
    else return dtype == MOE_BF16 ? bf16_to_f32(w[i]) : f16_to_f32(w[i]);
}

// Scales of 64 columns (int8 rule over K); 16 waves share the k out.  Few workgroups, and the weights are read again for
// the codes: packing 4096 x 4096 takes 110 us from bf16, 16 from codes, once for a model's weights.
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

// ---- some rows: weight streaming with the rows through LDS ----------------------------------
// As dense_stream_kernel: a workgroup owns MT * 16 rows x 16 columns of CT column halves (CT = 4: all of a 64-column
// pair), its eight waves take every eighth step of 128 k, and the weights go straight to registers.  There A's rows do
// too, and a quarter of a wave, 16 lanes, reads 16 bytes of 16 rows: 64 accesses to the L1 for a KiB, which bound it
// (128 x 4096 x 4096: 19 thousand accesses on each CU in 14.1 us).  Here each wave copies its rows' 128 bytes of a step
// to LDS, eight lanes to a row, 8 accesses for a KiB, into a ring of its own: no barrier until the sums are joined.
// A granule of 16 bytes lies at its place XOR row / 2 % 8, so that the 16 rows of a fragment read fall into all banks.
// Two steps are in flight (three and four: no faster, and fewer workgroups fit a CU); weights are loaded as others are
// (past the caches 9.7 us at 128 x 4096 x 4096, 7.8 on the same card).
// Bound by what a CU reads, some 106 bytes/ns once it has several workgroups and 80 with one: 64 x 4096 x 4096 6.8 us,
// 128 rows 8.7, 256 rows 11.3, of which a launch is 2.3.
// ROWS16: rows on 16 bytes, copied directly.  PART: K ends inside a granule.  The codes behind it up to the next 16 bytes
// come along, from between the rows, and meet zero weights; behind the last row there may be nothing, so that one's
// end is put there code by code (1000 x 1003 x 1100 on rows 1104 apart 8.6 us, 11.0 through registers; in the other
// kernels this would cost 3 %).  Rows off 16 bytes go through registers.
constexpr int kDepth = 2;

// Bytes n .. 15 of v moved down to 0 .., zeros behind them; n uniform, 0 to 15.
__device__ __forceinline__ u32x4 shift_down(u32x4 v, int n) {
    if (n & 8) v = u32x4{v[2], v[3], 0u, 0u};
    if (n & 4) v = u32x4{v[1], v[2], v[3], 0u};
    const uint32_t b = n & 3;
    return u32x4{__builtin_amdgcn_alignbyte(v[1], v[0], b), __builtin_amdgcn_alignbyte(v[2], v[1], b),
                 __builtin_amdgcn_alignbyte(v[3], v[2], b), __builtin_amdgcn_alignbyte(0u, v[3], b)};
}

template <bool VEC, bool ROWS16, bool PART, int MT, int CT>
__global__ __launch_bounds__(kNW * 64, MT < 4 ? 4 : 2) void int8_rows_kernel(DenseArgs p) {
    constexpr int kStep = MT * 16 * 128;               // bytes of the rows' part of a step
    constexpr int D = kDepth, kRing = kNW * D * kStep, kRed = kNW * MT * CT * 1024;
    __shared__ __attribute__((aligned(16))) uint8_t s_all[kRing > kRed ? kRing : kRed];
    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int unit = blockIdx.x, row0 = blockIdx.y * MT * kRowTile;
    const int pair = CT == 4 ? unit : unit >> 1, c0 = CT == 4 ? 0 : (unit & 1) * 16;
    const int nk = (p.K + 127) / 128, steps = nk > wave ? (nk - wave + kNW - 1) / kNW : 0;
    // rows through registers: the step that K ends in is its wave's first, so that what it costs more is in no loop (the
    // order of the steps does not matter to exact sums)
    const bool ends_here = !ROWS16 && p.K % 128 != 0 && (nk - 1) % kNW == wave;
    // weights: this lane's bytes of the step; tile c: half c % 2, columns c0 + c / 2 * 16
    const uint8_t* b = reinterpret_cast<const uint8_t*>(p.b) +
                       (static_cast<int64_t>(pair) * (p.Kp / 64) + wave) * step_bytes<false>() + (lane >> 5) * 2048 +
                       (((lane >> 4) & 1) * 32 + c0 + (lane & 15)) * 16;
    // rows: copy i brings rows 8 i .. 8 i + 7, lane: row lane / 8, place lane % 8
    uint8_t* const first = reinterpret_cast<uint8_t*>(const_cast<uint16_t*>(p.a)) + row0 * p.lda;
    const __amdgpu_buffer_rsrc_t rows = __builtin_amdgcn_make_buffer_rsrc(first, 0, kBufferRange, kBufferFlags);
    const int granule0 = (lane & 7) ^ (lane >> 4);
    auto granule = [&](int i) { return granule0 ^ ((i & 1) * 4); };   // row / 2 % 8 is lane / 16, and 4 more for odd i
    uint32_t off[MT * 2];
#pragma unroll
    for (int i = 0; i < MT * 2; ++i) {
        const int row = i * 8 + (lane >> 3);
        const uint32_t at = static_cast<uint32_t>(min(row, p.M - 1 - row0) * static_cast<int>(p.lda) + granule(i) * 16);
        off[i] = ROWS16 && row0 + row >= p.M ? kOutOfRange : at;   // rows past M: zeros, or the last row's; not stored
    }
    uint8_t* ring = s_all + wave * (D * kStep);
    u32x4 wb[D][CT][2], ra[ROWS16 ? 1 : D][MT * 2];
    int next = wave;                                   // the step that is loaded next
    auto load_weights_of = [&](int slot) __attribute__((always_inline)) {
#pragma unroll
        for (int c = 0; c < CT; ++c)
#pragma unroll
            for (int l = 0; l < 2; ++l)
                wb[slot][c][l] = *reinterpret_cast<const u32x4*>(b + (c & 1) * 1024 + (c >> 1) * 256 + l * 4096);
    };
    auto load = [&](int slot) __attribute__((always_inline)) {
        const bool last = ROWS16 && (next + 1) * 128 > p.K;   // uniform: K ends in the step
#pragma unroll
        for (int i = 0; i < MT * 2; ++i) {
            if constexpr (ROWS16) {
                uint32_t o = off[i];
                if (last && !PART) {
                    o = next * 128 + granule(i) * 16 < p.K ? o : kOutOfRange;
                } else if (last) {
                    const int end = p.K - next * 128 - granule(i) * 16;      // codes of the granule that exist
                    const bool last_row = row0 + i * 8 + (lane >> 3) == p.M - 1;
                    o = end >= 16 || (end > 0 && !last_row) ? o : kOutOfRange;
                }
                copy_to_lds(rows, ring + slot * kStep + i * 1024, static_cast<int>(o), next * 128);
            } else {
                ra[slot][i] = load_any<kI8>(first + next * 128 + off[i]);
            }
        }
        load_weights_of(slot);
        b += kNW * step_bytes<false>();
        next += kNW;
    };
    intx4 acc[MT][CT];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int c = 0; c < CT; ++c) acc[m][c] = intx4{0, 0, 0, 0};
    constexpr int LOADS = MT * 2 + CT * 2;
    // operand l of row tile m: row m * 16 + lane % 16, granule l * 4 + lane / 16
    const int fr = (lane & 15) * 128 + ((lane >> 4) ^ ((lane & 15) >> 1)) * 16;
    auto multiply = [&](int slot) __attribute__((always_inline)) {
        if constexpr (!ROWS16) {
#pragma unroll
            for (int i = 0; i < MT * 2; ++i) *reinterpret_cast<u32x4*>(ring + slot * kStep + i * 1024 + lane * 16) = ra[slot][i];
        }
        u32x4 a[MT][2];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int l = 0; l < 2; ++l)
                a[m][l] = *reinterpret_cast<const u32x4*>(ring + slot * kStep + m * 2048 + (fr ^ (l * 64)));
#pragma unroll
        for (int l = 0; l < 2; ++l)
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int c = 0; c < CT; ++c) acc[m][c] = mfma16k<kI8>(a[m][l], wb[slot][c][l], acc[m][c]);
    };
    // the oldest step has landed, n younger ones may be on their way (what goes to registers the compiler waits for)
    auto landed = [&](auto n) __attribute__((always_inline)) {
        if constexpr (ROWS16) wait_vmcnt<LOADS * decltype(n)::value>();
        asm volatile("" ::: "memory");
    };
    // the fragments are read: their place may be filled again
    auto read = [&]() __attribute__((always_inline)) {
        if constexpr (ROWS16) wait_lgkmcnt0();
        asm volatile("" ::: "memory");
    };
    // the granule that K ends in, of the last row, and its place in a step
    u32x4 row_end = {0u, 0u, 0u, 0u};
    const int end_row = p.M - 1 - row0, end_granule = p.K / 16 % 8;
    const int end_place = (end_row >> 3) * 1024 + (end_row & 7) * 128 + ((end_granule ^ (end_row >> 1)) & 7) * 16;
    const bool put_end = PART && end_row < MT * 16 && (nk - 1) % kNW == wave;   // uniform
    if (put_end && lane == 0)
        row_end = load_tail<kI8>(first + static_cast<int64_t>(end_row) * p.lda, (nk - 1) * 64 + end_granule * 8, p.K);
    if constexpr (!ROWS16) {
        if (ends_here) {                               // whole granules, and the row's last 16 bytes for the one K ends in
            const uint8_t* start = b;
            b += static_cast<int64_t>(nk - 1 - wave) * step_bytes<false>();
            load_weights_of(0);
            b = start;
#pragma unroll
            for (int i = 0; i < MT * 2; ++i) {
                const int k = (nk - 1) * 128 + granule(i) * 16;
                const uint8_t* row = first + off[i] - granule(i) * 16;
                if (p.K < 16) {                        // uniform
                    ra[0][i] = load_tail<kI8>(row, granule(i) * 8, p.K);
                } else {
                    const u32x4 v = load_any<kI8>(row + min(k, p.K - 16)), end = shift_down(v, (16 - p.K % 16) & 15);
                    ra[0][i] = k + 16 <= p.K ? v : k < p.K ? end : u32x4{0u, 0u, 0u, 0u};
                }
            }
        }
    }
#pragma unroll
    for (int j = 0; j < D; ++j)
        if (j < steps && !(j == 0 && ends_here)) load(j);   // uniform
    int i = 0;
    for (; i + 2 * D <= steps; i += D) {
#pragma unroll
        for (int j = 0; j < D; ++j) {
            landed(IntC<D - 1>{});
            multiply(j);
            read();
            load(j);
        }
    }
#pragma unroll
    for (int j = 0; j < 2 * D - 1; ++j)
        if (i + j < steps) {                           // uniform
            if (i + j + D <= steps) landed(IntC<D - 1>{});
            else landed(IntC<0>{});
            if (put_end && i + j == steps - 1 && lane == 0)
                *reinterpret_cast<u32x4*>(ring + j % D * kStep + end_place) = row_end;
            multiply(j % D);
            if (j < D && i + j + D < steps) {
                read();
                load(j % D);
            }
        }
    // the waves' sums are joined in LDS: [wave][m][c][v][lane], where lane is column lane % 16, row (lane / 16) * 4 + v
    __syncthreads();
    int* red = reinterpret_cast<int*>(s_all);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int c = 0; c < CT; ++c)
#pragma unroll
            for (int v = 0; v < 4; ++v) red[((wave * MT + m) * CT + c) * 256 + v * 64 + lane] = acc[m][c][v];
    __syncthreads();
    // four lanes are four columns of a row; gated: the up's are the tile after the gate's
    with_activation(p.act, [&](auto act) __attribute__((always_inline)) {
        constexpr int ACT = decltype(act)::value;
        constexpr bool kGated = ACT == MOE_EPI_SWIGLU;
        for (int i = tid; i < MT * CT * (kGated ? 32 : 64); i += kNW * 64) {
            const int q = i & 15, v = (i >> 4) & 3, t = i >> 6;        // lanes 4 q .. 4 q + 3
            const int m = kGated ? t / (CT / 2) : t / CT, c = kGated ? t % (CT / 2) * 2 : t % CT;
            const int row = m * 16 + (q >> 2) * 4 + v, in = c0 + (c >> 1) * 16 + (q & 3) * 4;
            const int col = kGated ? pair * 32 + in : pair * 64 + (c & 1) * 32 + in;
            const float sa = p.sa[min(row0 + row, p.M - 1)];
            const Columns columns = load_columns<kI8>(p, col);
            const Finisher<kI8, VEC> f(p, row0, row, col);
            const u32x4 part = f.load(0);
            intx4 s = {0, 0, 0, 0}, u = s;
#pragma unroll
            for (int w = 0; w < kNW; ++w) {
                const int* e = red + ((w * MT + m) * CT + c) * 256 + v * 64 + q * 4;
                s += *reinterpret_cast<const intx4*>(e);
                if constexpr (kGated) u += *reinterpret_cast<const intx4*>(e + 256);
            }
            f.template finish<ACT>(0, s, u, columns, sa, part);
        }
    });
}

// ---- many rows: two workgroups to a CU -------------------------------------------------------
// (three of them with tiles of 64 rows and less).
// A workgroup of 4 waves owns NA * 32 rows x four 64-column pairs, a pair to a wave: NA x 2 tiles of
// v_mfma_i32_32x32x32.  A stage is 128 k.  The rows reach LDS by direct copies into a ring of four stages (granules XORed
// by row / 2 % 8, as above: no bank conflicts), one barrier a stage; each weight belongs to one wave and goes straight to
// its registers, two stages of it.  Two workgroups share a CU, and while one is at its barrier, its loads or its
// epilogue, which at 6000 x 4096 x 4096 is a seventh of its time, the other multiplies.
// Where K ends inside a granule the last stage's copies bring what lies behind it, but the last row's end comes code by
// code, as above (2000 x 4096 x 4090, rows 4096 apart, 42.2 us, 71.3 by int8_rows_kernel; K 4096 42.2).
// The loop has no branch around a load and the fragments of a step are asked for before the step before is multiplied:
// 6000 x 4096 x 4096 97 us (2080 TOP/s; a library product 101.7), with bias and SiLU 99.7, 107 with such branches;
// gated, 1536 columns, 77; the 16-bit products' kernel, one workgroup of 8 waves to a CU: 109, 110 and 97 on the same
// card.  Bound by the matrix unit at the clock that the power limit leaves (1.75 GHz: half of the cycles multiply) and the
// latency of the weights.
template <bool VEC, int NA>
__global__ __launch_bounds__(256, NA <= 2 ? 3 : 2) void int8_tile_kernel(DenseArgs p, int mtiles, int ntiles, int pairs) {
    constexpr int UM = NA * 32, kStage = UM * 128, kStages = 4;
    __shared__ __attribute__((aligned(16))) uint8_t s_a[kStages * kStage > 16384 ? kStages * kStage : 16384];
    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int G = gridDim.x, blk = blockIdx.x;
    // one contiguous range of tiles per XCD, 8 row tiles x 4 column tiles of it at a time
    const int lid = (G % 8 == 0) ? (blk % 8) * (G / 8) + (blk / 8) : blk;
    constexpr int kGroup = 8;
    const int group = lid / (kGroup * ntiles), in = lid - group * kGroup * ntiles;
    const int gm = min(kGroup, mtiles - group * kGroup);
    const int n_tile = in / gm, m_tile = group * kGroup + in - n_tile * gm;
    const int row0 = m_tile * UM, pair = n_tile * 4 + wave;
    const __amdgpu_buffer_rsrc_t rows = __builtin_amdgcn_make_buffer_rsrc(
        reinterpret_cast<uint8_t*>(const_cast<uint16_t*>(p.a)) + static_cast<int64_t>(row0) * p.lda, 0, kBufferRange, kBufferFlags);
    uint32_t off[NA];
    int granule[NA];
#pragma unroll
    for (int i = 0; i < NA; ++i) {
        const int row = (wave * NA + i) * 8 + (lane >> 3);
        granule[i] = (lane & 7) ^ ((row >> 1) & 7);
        off[i] = row0 + row < p.M ? static_cast<uint32_t>(row * static_cast<int>(p.lda) + granule[i] * 16) : kOutOfRange;
    }
    const uint8_t* b = reinterpret_cast<const uint8_t*>(p.b) +
                       static_cast<int64_t>(min(pair, pairs - 1)) * (p.Kp / 64) * step_bytes<false>() + lane * 16;
    const int nk = p.Kp / 64;
    const int end_row = p.M - 1 - row0;                // as in int8_rows_kernel: its end comes code by code
    u32x4 wb[2][4][2];                                 // [stage % 2][32 k][column half]
    auto load_a = [&](int s, auto inside) __attribute__((always_inline)) {
        const bool last = !decltype(inside)::value && s * 64 + 64 > p.Kh;   // uniform: K ends in the stage
#pragma unroll
        for (int i = 0; i < NA; ++i) {
            uint32_t o = off[i];
            if (last) {
                const int end = p.K - s * 128 - granule[i] * 16;             // codes of the granule that exist
                const bool last_row = (wave * NA + i) * 8 + (lane >> 3) == end_row;
                o = end >= 16 || (end > 0 && !last_row) ? o : kOutOfRange;
            }
            copy_to_lds(rows, s_a + (s & 3) * kStage + (wave * NA + i) * 1024, static_cast<int>(o), s * 128);
        }
    };
    auto load_bk = [&](int s, auto buf, int k) __attribute__((always_inline)) {
        const uint8_t* at = b + static_cast<int64_t>(s) * step_bytes<false>();
#pragma unroll
        for (int h = 0; h < 2; ++h)
            wb[decltype(buf)::value][k][h] = *reinterpret_cast<const u32x4*>(at + k * 2048 + h * 1024);
    };
    auto load_b = [&](int s, auto buf) __attribute__((always_inline)) {
#pragma unroll
        for (int k = 0; k < 4; ++k) load_bk(s, buf, k);
    };
    intx16 acc[NA][2];
#pragma unroll
    for (int i = 0; i < NA; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[i][j][v] = 0;
    const int fr = (lane & 31) * 128;
    // Stage s, its weights in buffer s % 2.  Loads are issued in the order A(s + 1), B(s), A(s + 2), B(s + 1), ..., so when all
    // but A(s + 2) and B(s + 1) have landed, stage s is here; behind the barrier every wave's part of it is, and the place of
    // stage s - 1, A(s + 3)'s, is no longer read.
    auto stage = [&](int s, auto buf, auto inside) __attribute__((always_inline)) {
        constexpr int B = decltype(buf)::value;
        constexpr bool kInside = decltype(inside)::value;
        if (kInside || s + 2 < nk) wait_vmcnt<NA + 8>();
        else if (s + 1 < nk) wait_vmcnt<8>();
        else wait_vmcnt<0>();
        if constexpr (!kInside) {
            if (s + 1 == nk && p.K % 16 != 0 && (end_row >> 3) / NA == wave) {     // uniform
                const int g = p.K / 16 % 8;
                const uint8_t* row = reinterpret_cast<const uint8_t*>(p.a) + static_cast<int64_t>(p.M - 1) * p.lda;
                if (lane == 0)
                    *reinterpret_cast<u32x4*>(s_a + (s & 3) * kStage + (end_row >> 3) * 1024 + (end_row & 7) * 128 +
                                              ((g ^ (end_row >> 1)) & 7) * 16) = load_tail<kI8>(row, s * 64 + g * 8, p.K);
                wait_lgkmcnt0();
            }
        }
        phase_end();
        if (kInside || s + 3 < nk) load_a(s + 3, inside);
        const uint8_t* at = s_a + (s & 3) * kStage + fr;
        u32x4 a[2][NA];
        auto read = [&](int k) __attribute__((always_inline)) {
#pragma unroll
            for (int i = 0; i < NA; ++i)
                a[k & 1][i] = *reinterpret_cast<const u32x4*>(at + i * 4096 + (((k * 2 + (lane >> 5)) ^ ((lane >> 1) & 7)) * 16));
        };
        read(0);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (k < 3) read(k + 1);
            if constexpr (NA > 2) __builtin_amdgcn_sched_barrier(0);   // the next fragments are asked for before these are multiplied
#pragma unroll
            for (int i = 0; i < NA; ++i) {
                acc[i][0] = mfma32d<kI8>(a[k & 1][i], wb[B][k][0], acc[i][0]);
                acc[i][1] = mfma32d<kI8>(a[k & 1][i], wb[B][k][1], acc[i][1]);
            }
            if (kInside || s + 2 < nk) load_bk(s + 2, buf, k);
        }
    };
    int s = 0;
    if (nk > 5) {                                      // no branch around a load, here and in the loop: the compiler counts
        load_a(0, IntC<1>{});
        load_a(1, IntC<1>{});
        load_b(0, IntC<0>{});
        load_a(2, IntC<1>{});
        load_b(1, IntC<1>{});
        do {
            stage(s, IntC<0>{}, IntC<1>{});
            stage(s + 1, IntC<1>{}, IntC<1>{});
            s += 2;
        } while (s + 5 < nk);
    } else {
        load_a(0, IntC<0>{});
        if (nk > 1) load_a(1, IntC<0>{});
        load_b(0, IntC<0>{});
        if (nk > 2) load_a(2, IntC<0>{});
        if (nk > 1) load_b(1, IntC<1>{});
    }
    for (; s < nk; s += 2) {
        stage(s, IntC<0>{}, IntC<0>{});
        if (s + 1 < nk) stage(s + 1, IntC<1>{}, IntC<0>{});
    }
    phase_end_lds();
    const int col = pair * (p.gated ? 32 : 64) + (p.gated ? lane & 7 : lane & 15) * 4;
    const Columns columns = load_columns<kI8>(p, col);
    float sa[(NA + 1) / 2];                            // of the rows lane, lane + 64
#pragma unroll
    for (int i = 0; i < (NA + 1) / 2; ++i) sa[i] = p.sa[min(row0 + i * 64 + lane, p.M - 1)];
    int(*mine)[64] = reinterpret_cast<int(*)[64]>(s_a + wave * 4096);
    finish_tile<kI8, NA, 1, 1, VEC>(p, acc, mine, mine, 0, row0, col, columns, sa);
}

// Rows of a tile: the least time expected.  Tiles take a launch, and the busiest CU's tiles one after another, each a fixed
// part and a part by the reduction (ns, of 4096 k); a CU's only tile waits for its loads a little longer.  Measured with N
// a multiple of four and K of sixteen: there within 13 % in nine of ten, 17 % at most, from 16 to 97 us.
struct TileCost {
    double ends, whole;
};
constexpr TileCost kTileCosts[] = {{1100, 12500}, {2100, 17900}, {5300, 23300}, {8500, 30000}};   // 32, 64, 96, 128 rows

Choice int8_tile_choice(const DenseArgs& p, int64_t pairs) {
    Choice best{0, 0.0};
    for (int i = 0; i < 4; ++i) {
        const int rows = (i + 1) * 32;
        const int64_t tiles = (p.M + rows - 1) / rows * ((pairs + 3) / 4), each = (tiles + kCUs - 1) / kCUs;
        if (tiles >= 1 << 24) continue;                // a grid's limit is 2^32 threads
        const double one = kTileCosts[i].ends + (kTileCosts[i].whole - kTileCosts[i].ends) * p.Kp / 2048;
        const double ns = 5000.0 + each * one * (each == 1 ? 1.15 : 1.0);
        if (best.ns == 0.0 || ns < best.ns) best = Choice{i, ns};
    }
    return best;
}

template <bool VEC, int NA>
int launch_int8_tile(const DenseArgs& p, int64_t pairs, hipStream_t st) {
    const int ntiles = static_cast<int>((pairs + 3) / 4), mtiles = (p.M + NA * 32 - 1) / (NA * 32);
    hipLaunchKernelGGL((int8_tile_kernel<VEC, NA>), dim3(static_cast<unsigned>(mtiles * ntiles)), dim3(256), 0, st, p, mtiles,
                       ntiles, static_cast<int>(pairs));
    MOE_CHECK_LAUNCH();
    return MOE_OK;
}

template <bool VEC>
int launch_int8_tiles(const DenseArgs& p, int64_t pairs, int shape, hipStream_t st) {
    switch (shape) {
        case 0: return launch_int8_tile<VEC, 1>(p, pairs, st);
        case 1: return launch_int8_tile<VEC, 2>(p, pairs, st);
        case 2: return launch_int8_tile<VEC, 3>(p, pairs, st);
        default: return launch_int8_tile<VEC, 4>(p, pairs, st);
    }
}

// Unit shapes of int8_rows_kernel, and the time expected of each: a launch, what the shape takes at the ends (ns), and
// what the busiest CU reads (bytes/ns), its first unit and then the others at the rate they reach together, but no less
// than a unit takes anyhow; rows off 16 bytes pass through registers, more slowly (32 rows x 64 columns then leave room
// for one workgroup on a CU: not taken).  Measured with N a multiple of four: within 16 % from 3.5 to 25 us (19 % at 512 x
// 512, 3000 rows and more), and the kernel and shape chosen within 4 % of the best but for three sizes of 72 (15 to 31 %).
// Stores of an element each, where N is none, and K's end are in no figure: 2000 x 2050 x 1000 is expected to take 13.7
// us here and takes 23.4, 17.3 in tiles.
struct RowsShape {
    int mt, ct;
    double ends, rate, rate_any, least;
};
constexpr RowsShape kRowsShapes[] = {{1, 2, 800, 106, 60, 500}, {2, 2, 800, 106, 58, 950}, {1, 4, 1000, 106, 75, 900},
                                     {2, 4, 950, 95, 0, 1150}, {4, 4, 2000, 62, 45, 3600}};

Choice rows_choice(const DenseArgs& p, int64_t pairs, bool rows16) {
    Choice best{0, 0.0};
    for (int i = 0; i < 5; ++i) {
        const RowsShape& u = kRowsShapes[i];
        if (!rows16 && u.rate_any == 0) continue;
        const int rows = u.mt * kRowTile;
        if ((p.M + rows - 1) / rows > 65535) continue; // the grid's limit; the tallest shape stays within it
        const int64_t groups = pairs * (4 / u.ct) * ((p.M + rows - 1) / rows), each = (groups + kCUs - 1) / kCUs;
        const double bytes = (std::min(rows, p.M) + u.ct * kRowTile) * 2.0 * p.Kp;
        const double ns = 2300.0 + u.ends + bytes / (rows16 ? 80 : 65) +
                          (each - 1) * std::max(bytes / (rows16 ? u.rate : u.rate_any) + u.ends / 8, u.least);
        if (best.ns == 0.0 || ns < best.ns) best = Choice{i, ns};
    }
    return best;
}

template <bool VEC, bool ROWS16, bool PART>
int launch_rows(const DenseArgs& p, int64_t pairs, int shape, hipStream_t st) {
    const RowsShape& u = kRowsShapes[shape];
    const dim3 g(static_cast<unsigned>(pairs * (4 / u.ct)), (p.M + u.mt * kRowTile - 1) / (u.mt * kRowTile));
    switch (shape) {
        case 0: hipLaunchKernelGGL((int8_rows_kernel<VEC, ROWS16, PART, 1, 2>), g, dim3(kNW * 64), 0, st, p); break;
        case 1: hipLaunchKernelGGL((int8_rows_kernel<VEC, ROWS16, PART, 2, 2>), g, dim3(kNW * 64), 0, st, p); break;
        case 2: hipLaunchKernelGGL((int8_rows_kernel<VEC, ROWS16, PART, 1, 4>), g, dim3(kNW * 64), 0, st, p); break;
        case 3:
            if constexpr (ROWS16) hipLaunchKernelGGL((int8_rows_kernel<VEC, ROWS16, PART, 2, 4>), g, dim3(kNW * 64), 0, st, p);
            break;
        default: hipLaunchKernelGGL((int8_rows_kernel<VEC, ROWS16, PART, 4, 4>), g, dim3(kNW * 64), 0, st, p); break;
    }
    MOE_CHECK_LAUNCH();
    return MOE_OK;
}

constexpr int kVeryFewRows = 8;

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
    const int64_t pairs = pairs_of(s);
    if (!a_near(p) || !out_near(p, 64)) return launch_any<kI8>(p, pairs, st);   // 64 rows of a unit of int8_rows_kernel
    const bool rows16 = reinterpret_cast<uintptr_t>(a) % 16 == 0 && lda % 16 == 0;
    const Choice rows = rows_choice(p, pairs, rows16);
    if (!rows16)
        return p.vec ? launch_rows<true, false, false>(p, pairs, rows.shape, st) : launch_rows<false, false, false>(p, pairs, rows.shape, st);
    // a few rows need no detour through LDS, and units of 16 columns: 1 x 4096 x 1536 3.1 us, 3.5 through LDS
    if (s.M <= kVeryFewRows && s.K % 16 == 0) {
        if (stream_choice(p, pairs, true).shape == kUnitShape11) return launch_stream_tiles<kI8, true, 1, 1>(p, pairs, st);
        return launch_stream_tiles<kI8, true, 1, 2>(p, pairs, st);
    }
    // 1024 x 4096 x 4096: tiles 27 us, 34 by rows; 512 x 1536 x 4096: 18 and 10.9
    const Choice tile = int8_tile_choice(p, pairs);
    if (tile.ns > 0.0 && tile.ns < rows.ns)
        return p.vec ? launch_int8_tiles<true>(p, pairs, tile.shape, st) : launch_int8_tiles<false>(p, pairs, tile.shape, st);
    if (s.K % 16 != 0)
        return p.vec ? launch_rows<true, true, true>(p, pairs, rows.shape, st) : launch_rows<false, true, true>(p, pairs, rows.shape, st);
    return p.vec ? launch_rows<true, true, false>(p, pairs, rows.shape, st) : launch_rows<false, true, false>(p, pairs, rows.shape, st);
}

}  // namespace moe
