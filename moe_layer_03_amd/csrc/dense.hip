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

// ---- few rows: weight streaming ------------------------------------------------------
// A workgroup owns MT * 16 rows x 16 columns of CT column halves (gated: gate
// and up, CT = 2) and its kNW waves take every kNW-th step of the reduction, so
// the weights go straight from memory to registers, each element once per
// MT * 16 rows.  The partial tiles are added through LDS in wave order.  Rows
// past M and k past K (a multiple of 8) load zeros through an out-of-range
// buffer offset.
constexpr int kNW = 8;

template <int MT, int CT>
struct DenseCursor {
    const uint8_t* b;          // this lane's bytes of the step, first column half of the tile
    int half;                  // bytes to the second
    __amdgpu_buffer_rsrc_t rows;
    uint32_t off[MT];          // byte offset of this lane's k group, or out of range
    int k, K;                  // first k of the lane's group in this step
    int left;

    __device__ __forceinline__ void load(StepRegs<1, false, MT, CT>& s) {
#pragma unroll
        for (int c = 0; c < CT; ++c)
            s.b[c] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(b + c * half));
#pragma unroll
        for (int m = 0; m < MT; ++m)
            s.a[m][0][0] = __builtin_bit_cast(
                u32x4, __builtin_amdgcn_raw_buffer_load_b128(rows, k < K ? off[m] : kOutOfRange, 0, 0));
        const int go = left > 0 ? 1 : 0;               // uniform
        left -= go;
        b += go * (kNW * kStepBytes);
        k += go * (kNW * 32);
#pragma unroll
        for (int m = 0; m < MT; ++m) off[m] += go * (kNW * 64);
    }
};

template <bool F16, int MT, int CT>
__global__ __launch_bounds__(kNW * 64, MT == 4 ? 1 : 2) void dense_stream_kernel(DenseArgs p) {
    __shared__ __attribute__((aligned(16))) float s_red[kNW][MT][CT][4][kWave];
    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int unit = blockIdx.x, row0 = blockIdx.y * MT * kRowTile;
    // CT = 2: both halves of a pair; CT = 1: one half
    const int pair = CT == 2 ? unit >> 1 : unit >> 2, half = CT == 2 ? 0 : (unit >> 1) & 1, c0 = (unit & 1) * 16;
    const int nk = (p.K + 31) / 32;
    DenseCursor<MT, CT> cur;
    cur.b = reinterpret_cast<const uint8_t*>(p.b) + (static_cast<int64_t>(pair) * (p.Kp / 32) + wave) * kStepBytes +
            step_lane_offset<false>(half, c0);
    cur.half = 1024;
    cur.rows = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(p.a) + row0 * p.lda, 0, kBufferRange,
                                                 kBufferFlags);
    cur.k = wave * 32 + (lane >> 4) * 8;
    cur.K = p.K;
    const int steps = nk > wave ? (nk - wave + kNW - 1) / kNW : 0;
    cur.left = steps - 1;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const int r = m * kRowTile + (lane & 15);
        cur.off[m] = row0 + r < p.M ? static_cast<uint32_t>(r * static_cast<int>(p.lda) + cur.k) * 2 : kOutOfRange;
    }
    Acc<1, F16, false, MT, CT> acc;
    acc.clear();
    stream_steps<4>(steps, cur, acc);
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
        float s[CT];
#pragma unroll
        for (int c = 0; c < CT; ++c) {
            s[c] = 0.0f;
#pragma unroll
            for (int q = 0; q < kNW; ++q) s[c] += s_red[q][m][c][v][lane];
        }
        if constexpr (CT == 1) {
            finish(p, row, pair * 64 + half * 32 + cc, s[0], 0.0f);
        } else if (p.gated) {
            finish(p, row, pair * 32 + cc, s[0], s[1]);
        } else {
            finish(p, row, pair * 64 + cc, s[0], 0.0f);
            finish(p, row, pair * 64 + 32 + cc, s[1], 0.0f);
        }
    }
}

// ---- many rows: LDS tiles --------------------------------------------------------------
// A workgroup of 8 waves owns um <= 256 rows x 256 packed columns; a wave owns one
// of two row halves (up to 128 rows) x one 64-column pair: up to 4 x 2 tiles of
// v_mfma_f32_32x32x16.  Both operands reach LDS by direct copies into a ring of
// NB = 4 stages of 32 k, read one k-step of 16 ahead of the MFMAs; waits are
// explicit and the once-per-stage barrier sits between a stage's two k-steps.
// A's rows go through a buffer resource based at the tile's first row: rows past
// M and k past K copy zeros.
constexpr int kTileNB = 4;
constexpr int kTileBK = 32;

__device__ __forceinline__ int tile_swz(int row, int kg) {
    // 16-byte granule kg of a 64-byte row, XORed so that a fragment read's 16
    // consecutive rows fall into different banks
    return row * kTileBK + ((kg ^ ((row >> 2) & 3)) << 3);
}

__device__ __forceinline__ floatx16 mfma32d(bool f16, const u32x4& a, const u32x4& b, floatx16 c) {
    if (f16)
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(halfx8_t, a),
                                                      __builtin_bit_cast(halfx8_t, b), c, 0, 0, 0);
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c,
                                                   0, 0, 0);
}

template <bool F16>
__global__ __launch_bounds__(512, 1) void dense_tile_kernel(DenseArgs p, int um, int mtiles, int ntiles, int pairs) {
    __shared__ __attribute__((aligned(16))) uint16_t s_a[kTileNB][256 * kTileBK];
    __shared__ __attribute__((aligned(16))) uint16_t s_b[kTileNB][4][4][512];
    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int mh = wave >> 2, nq = wave & 3;
    const int hm = (um / 2 + 31) & ~31;                // rows of the first half
    const int nk = p.Kp / kTileBK;
    const int total = mtiles * ntiles;
    const int G = gridDim.x, b = blockIdx.x;
    // one contiguous range of tiles per XCD and round, 8 row tiles x 4 column tiles of it at a time
    const int lid = (G % 8 == 0) ? (b % 8) * (G / 8) + (b / 8) : b;
    constexpr int kGroup = 8;

    for (int tile = lid; tile < total; tile += G) {
        const int group = tile / (kGroup * ntiles), in = tile - group * kGroup * ntiles;
        const int gm = min(kGroup, mtiles - group * kGroup);
        const int n_tile = in / gm, m_tile = group * kGroup + in - n_tile * gm;
        const int row0 = m_tile * um;
        const int rows_valid = min(um, p.M - row0);
        const int half0 = mh * hm;                     // first row of this wave's half
        const int my_rows = min(rows_valid - half0, mh == 0 ? hm : um - hm);
        const int na = my_rows > 0 ? (my_rows + 31) >> 5 : 0;

        const __amdgpu_buffer_rsrc_t a_rsrc = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<uint16_t*>(p.a) + static_cast<int64_t>(row0) * p.lda, 0, kBufferRange, kBufferFlags);
        // copy i of column quarter nq: 16-row block i * 4 + nq of the half
        uint32_t a_off[2];
        int a_k[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int row = (i * 4 + nq) * 16 + (lane >> 2);
            const int kg = (lane & 3) ^ ((row >> 2) & 3);
            a_k[i] = kg * 8;
            a_off[i] = row < my_rows ? static_cast<uint32_t>((half0 + row) * static_cast<int>(p.lda) + kg * 8) * 2
                                     : kOutOfRange;
        }
        // weight copies: wave (mh, nq) copies blocks 2 mh, 2 mh + 1 of pair nq
        const int pair = min(n_tile * 4 + nq, pairs - 1);
        const uint16_t* b_src = p.b + static_cast<int64_t>(pair) * (p.Kp / 32) * (kStepBytes / 2) + mh * 1024 + lane * 8;
        auto issue = [&](auto ac, int kt, int st) {
            constexpr int AC = decltype(ac)::value;
            const int k0 = kt * kTileBK;
#pragma unroll
            for (int i = 0; i < AC; ++i)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(
                    a_rsrc,
                    reinterpret_cast<__attribute__((address_space(3))) void*>(
                        reinterpret_cast<uintptr_t>(&s_a[st][(mh * 128 + (i * 4 + nq) * 16) * kTileBK])),
                    16, static_cast<int>(k0 + a_k[i] < p.K ? a_off[i] + k0 * 2 : kOutOfRange), 0, 0, 0);
#pragma unroll
            for (int d = 0; d < 2; ++d)
                dma16(b_src + static_cast<int64_t>(kt) * (kStepBytes / 2) + d * 512, &s_b[st][nq][mh * 2 + d][0]);
        };
        floatx16 acc[4][2];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;

        auto kloop = [&](auto nac) {
            constexpr int NA = decltype(nac)::value;
            constexpr int AC = (2 * NA + 3) / 4;       // blocks of this thread that hold the half's row groups
            constexpr int LOADS = AC + 2;
#pragma unroll
            for (int q = 0; q + 1 < kTileNB; ++q) issue(IntC<AC>{}, min(q, nk - 1), q);
            u32x4 fa[2][4], fb[2][2];
            auto read_frags = [&](int buf, int st, int ks) {
                const int kg = ks * 2 + (lane >> 5);
#pragma unroll
                for (int i = 0; i < NA; ++i)
                    fa[buf][i] = *reinterpret_cast<const u32x4*>(&s_a[st][tile_swz(mh * 128 + i * 32 + (lane & 31), kg)]);
                fb[buf][0] = *reinterpret_cast<const u32x4*>(&s_b[st][nq][2 * ks][lane * 8]);
                fb[buf][1] = *reinterpret_cast<const u32x4*>(&s_b[st][nq][2 * ks + 1][lane * 8]);
            };
            auto mfmas = [&](int buf) {
#pragma unroll
                for (int i = 0; i < NA; ++i) {
                    acc[i][0] = mfma32d(F16, fa[buf][i], fb[buf][0], acc[i][0]);
                    acc[i][1] = mfma32d(F16, fa[buf][i], fb[buf][1], acc[i][1]);
                }
            };
            // entered with the stage's first fragments in buffer 0
            auto step = [&](int kt, int st) {
                if constexpr (NA > 0) {
                    read_frags(1, st, 1);
                    __builtin_amdgcn_sched_barrier(0);
                    asm volatile("" ::: "memory");
                    mfmas(0);
                }
                wait_vmcnt<LOADS * (kTileNB - 3)>();   // this wave's copies of the next stage have landed ...
                __builtin_amdgcn_s_barrier();          // ... and everyone's; nobody reads the stage refilled below
                issue(IntC<AC>{}, min(kt + kTileNB - 1, nk - 1), (st + kTileNB - 1) % kTileNB);
                if constexpr (NA > 0) {
                    read_frags(0, (st + 1) % kTileNB, 0);
                    __builtin_amdgcn_sched_barrier(0);
                    asm volatile("" ::: "memory");
                    mfmas(1);
                }
            };
            wait_vmcnt<LOADS * (kTileNB - 2)>();
            __builtin_amdgcn_s_barrier();
            if constexpr (NA > 0) read_frags(0, 0, 0);
            int kt0 = 0;
            for (; kt0 + kTileNB <= nk; kt0 += kTileNB) {
#pragma unroll
                for (int q = 0; q < kTileNB; ++q) step(kt0 + q, q);
            }
#pragma unroll
            for (int q = 0; q + 1 < kTileNB; ++q)
                if (kt0 + q < nk) step(kt0 + q, q);
        };
        switch (na) {
            case 4: kloop(IntC<4>{}); break;
            case 3: kloop(IntC<3>{}); break;
            case 2: kloop(IntC<2>{}); break;
            case 1: kloop(IntC<1>{}); break;
            default: kloop(IntC<0>{}); break;
        }
        // lane: column lane % 32, rows 8 (v / 4) + 4 (lane / 32) + v % 4 of each 32 x 32 tile
        const int cc = lane & 31, pc = n_tile * 4 + nq;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int v = 0; v < 16; ++v) {
                const int r = i * 32 + 8 * (v >> 2) + 4 * (lane >> 5) + (v & 3);
                if (r >= my_rows) continue;
                const int row = row0 + half0 + r;
                if (p.gated) {
                    finish(p, row, pc * 32 + cc, acc[i][0][v], acc[i][1][v]);
                } else {
                    finish(p, row, pc * 64 + cc, acc[i][0][v], 0.0f);
                    finish(p, row, pc * 64 + 32 + cc, acc[i][1][v], 0.0f);
                }
            }
        __syncthreads();                               // LDS reuse; drains this tile's copies
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

constexpr int kCUs = 256;

template <bool F16, int MT, int CT>
int launch_stream(const DenseArgs& p, int64_t pairs, hipStream_t st) {
    const dim3 g(static_cast<unsigned>(pairs * (4 / CT)), (p.M + MT * kRowTile - 1) / (MT * kRowTile));
    hipLaunchKernelGGL((dense_stream_kernel<F16, MT, CT>), g, dim3(kNW * 64), 0, st, p);
    MOE_CHECK_LAUNCH();
    return MOE_OK;
}

template <bool F16>
int launch_dense(const DenseArgs& p, int64_t pairs, hipStream_t st) {
    // 16-byte loads need every row to start on 16 bytes, and a k group to end within the row
    const bool rows16 = reinterpret_cast<uintptr_t>(p.a) % 16 == 0 && p.lda % 8 == 0 && p.K % 8 == 0;
    // byte offsets within a tile of rows stay below the buffer range
    const bool near = p.lda * 2 * 256 <= kBufferRange;
    if (!rows16 || !near) {
        const dim3 g(static_cast<unsigned>(pairs), (p.M + 63) / 64);
        hipLaunchKernelGGL((dense_any_kernel<F16>), g, dim3(256), 0, st, p);
        MOE_CHECK_LAUNCH();
        return MOE_OK;
    }
    if (p.M <= 16)
        return p.gated ? launch_stream<F16, 1, 2>(p, pairs, st) : launch_stream<F16, 1, 1>(p, pairs, st);
    if (p.M <= 32) return launch_stream<F16, 2, 2>(p, pairs, st);
    if (p.M <= 512) return launch_stream<F16, 4, 2>(p, pairs, st);
    const int ntiles = static_cast<int>((pairs + 3) / 4);
    // tile height: the fewest rows through the busiest CU, counting 64 rows' worth of time for a tile's weight copies
    int um = 256;
    int64_t best = -1;
    for (int h = 256; h >= 64; h -= 32) {
        const int64_t tiles = static_cast<int64_t>((p.M + h - 1) / h) * ntiles;
        const int64_t cost = (tiles + kCUs - 1) / kCUs * (h + 64);
        if (best < 0 || cost < best) {
            best = cost;
            um = h;
        }
    }
    const int mtiles = (p.M + um - 1) / um;
    const int64_t tiles = static_cast<int64_t>(mtiles) * ntiles;
    const unsigned grid = static_cast<unsigned>(tiles < kCUs ? tiles : kCUs);
    hipLaunchKernelGGL((dense_tile_kernel<F16>), dim3(grid), dim3(512), 0, st, p, um, mtiles, ntiles,
                       static_cast<int>(pairs));
    MOE_CHECK_LAUNCH();
    return MOE_OK;
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
    return a_dtype == MOE_F16 ? launch_dense<true>(p, pairs_of(s), st) : launch_dense<false>(p, pairs_of(s), st);
}

}  // namespace moe
