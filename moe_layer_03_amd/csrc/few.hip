// The whole layer for a few tokens (at most MOE_FEW_TOKENS_MAX).
//
// Mathematics, for token t:
//   l[t,e] = sum_h x[t,h] Wr[h,e] + b[e], summed in double precision;
//   the K largest, ties to the lower index; w_j = exp(l_j - l_0) / sum_i exp(l_i - l_0);
//   a_{t,j} = w_j silu(x_t Wg_e) (x_t Wu_e), e the expert of slot j;
//   out_t = sum over local slots of a_{t,j} Wd_e.
// With so few rows the layer is bound by reading the chosen experts' weights
// once: 6 H I bytes per expert (16-bit) against 6 H I operations per row.
//
// Three launches (hidden 4096, expert 1536, top 8 of 128, one token: 4.9, 39.6
// and 20.5 us with 16-bit weights, 4.6, 27.3 and 16.6 us with MXFP8; 63 and 47 us
// in all, where the weights alone take 46 and 24 at 6.6 TB/s):
//   route    partial logits over slices of H, double-precision MFMA;
//   gate/up  every workgroup sums the partials and selects the experts itself
//            (T rows of E values, cheaper than another launch), then takes
//            (chosen expert, 16 columns) units; its waves share the unit's H;
//   down     the weights w_j are folded into the rows a, so the down product
//            and the weighted combination over experts are ONE product with a
//            long reduction: out[T, n] = [rows of every chosen expert] x
//            [their down weights stacked], where row t of an expert's slice is
//            zero if token t did not choose it.  A workgroup owns 16 output
//            columns and a part of the reduction, so nothing is scattered, and
//            the parts are added in their order, whatever the timing.
// In gate/up an MFMA row is a token: rows of tokens that did not choose the
// expert load zeros through an out-of-range buffer offset, without memory
// traffic.  In down, an expert's rows are compacted, their parts stacked into
// one tile (RowMap).
//
// One kernel for gate/up and down, handing over by counters in memory, was
// right and slower wherever the grid fills the chip (one token, MXFP8: 72 us
// against 49.5): the workgroups' atomics and looks at shared counters cost about
// 25 us.  Kernel boundaries cost 1.6 us each.
//
// Precision: the rows a are kept to 22 bits (two fp16 parts; of small values to
// 2^-27 of the token's largest, see kLevels) or 24 (three bf16 parts, MXFP8), and
// nothing else is rounded below float32, so the float32 output is a float32
// result, not an fp16 one (stream.hpp).
#include <algorithm>

#include "block.hpp"
#include "stream.hpp"

namespace moe {
namespace {

constexpr int kNW = 8;                                 // waves per workgroup of the two products

// Steps a gate/up wave has in flight (2 KiB of weights each in MXFP8, 4 else), as
// many as the registers of four waves per SIMD hold, four at most: two workgroups
// on a CU then have 128 KiB or more in flight.  Rows of many parts (float32 rows
// with MXFP8 weights) keep two steps and half the waves.
constexpr int gate_up_step_regs(int NP, bool MX, int MT) { return (MX ? 10 : 16) + MT * NP * 8; }
constexpr int gate_up_ring(int NP, bool MX, int MT) {
    const int n = (96 - MT * 8 * (NP == 2 ? 2 : 1)) / gate_up_step_regs(NP, MX, MT);
    return n > 4 ? 4 : (n < 2 ? 2 : n);
}
constexpr int gate_up_waves(int NP, bool MX, int MT) {
    return 2 * gate_up_step_regs(NP, MX, MT) > 80 ? 2 : 4;
}
constexpr int kRouteNW = 16;
constexpr int kRouteGroups = 2;                        // 32-h groups of a wave in flight together
constexpr int kMaxSlices = 16;
constexpr int kMaxParts = 8;

// Levels of the rows a where they have two fp16 parts: those hold 22 bits of values
// from 2^-14 on but 2^-36 below, so a token whose rows are small needs them scaled
// up.  By how much is known only once all its rows are, and one sum adds up a
// token's rows across experts, so the scale is the token's: level l multiplies by
// 2^(24 l).  Gate/up writes a unit's 16 columns of a row at every level at which
// they stay below 2^15: level 0 always, and no other where one is 2^-9 or more, as
// rows commonly have.  The down step takes the highest level that all units of the
// token have.  Its largest value there is 2^-9 or more, and 2^-36 at most 2^-27 of
// it, for any largest value that float32 holds.  Small rows cost the writing and the
// reading of their levels: inputs of 1e-3 instead of 1, one token 64.6 us against
// 62.7, 32 tokens 726 against 699.
constexpr int kLevelBits = 24;
constexpr int kLevels = 6;

typedef double doublex4 __attribute__((ext_vector_type(4)));

struct FewArgs {
    const uint16_t* a;         // gate/up rows: parts [NP][T][H]
    int64_t a_part;            // elements per part
    const int* a_exp;          // [T] the parts are of the row times 2^this (two parts)
    const uint8_t* gu;         // packed gate/up weights (16-bit or MXFP8 codes)
    const uint8_t* gu_scales;
    const uint8_t* dn;
    const uint8_t* dn_scales;
    const double* part;        // [S][T][E] partial logits
    const float* bias;
    uint16_t* h;               // rows a_{t,j}: parts [NPH][T * K][I]
    int32_t* idx;              // [T][K]
    float* w;                  // [T][K]
    float* out;                // [T][H]
    float* sums;               // [H / 16][parts][T][16] partial sums of the down step
    int* arrived;              // [H / 16] workgroups that have written theirs; cleared by the route step
    uint8_t* levels;           // [T * K][I / 16] highest level written of a row's unit; cleared by the route step
    int* above;                // whether one is above 0; cleared by the route step
    int top;                   // highest level there is memory for
    int S, T, H, E, K, I, e_begin, E_loc;
};

template <int CTRL>
__device__ __forceinline__ uint32_t row_rotate(uint32_t v) {
    return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, 0xf, 0xf, false));
}

// The largest of a row of 16 lanes, in all of them.
__device__ __forceinline__ uint32_t row_max(uint32_t m) {
    m = max(m, row_rotate<0x128>(m));                  // row_ror:8, :4, :2, :1
    m = max(m, row_rotate<0x124>(m));
    m = max(m, row_rotate<0x122>(m));
    return max(m, row_rotate<0x121>(m));
}

// ---- route -------------------------------------------------------------------

template <typename XT> __device__ __forceinline__ double widen(XT v);
template <> __device__ __forceinline__ double widen<uint16_t>(uint16_t v) { return bf16_to_f32(v); }
template <> __device__ __forceinline__ double widen<float>(float v) { return v; }

// Bound by latency: one round of loads, at most 16 double-precision MFMAs per wave
// and a reduction through LDS, 4.9 us (one token of 4096 to 128 experts, 1 MB of
// router weights) to 6.1 (32), of which an empty launch takes 1.6.  float32 rows
// and weights are twice the bytes and have their parts to write: 5.4 us (one token)
// to 15.7 (16), and 21.3 (13) with the MXFP8 form's three parts.
// One workgroup: 16 experts x 16 tokens x one slice of H; its waves take 32-h
// groups in turn, at most kRouteGroups each, all loads issued before the first
// product.  v_mfma_f64_16x16x4: lane l holds row (column) l % 16 and k = l / 16;
// the four k of a group's step j are h = 8 (l / 16) + j.  The products of bf16
// (float32) inputs are exact in double, so only the additions round.
// NPX > 0: the first expert column also writes the rows' parts for the gate/up
// product.  Two fp16 parts hold 22 bits of values from 2^-14 on and 2^-36 below, so
// a row is scaled by a power of two until its largest value lies in [2^14, 2^15):
// 2^-36 is then 2^-50 of that.  The scale's exponent goes to xe.
template <typename XT, int NPX, bool F16>
__global__ __launch_bounds__(kRouteNW * 64) void few_route_kernel(const XT* __restrict__ x, const XT* __restrict__ w,
                                                                  int T, int H, int E, double* __restrict__ part,
                                                                  uint16_t* __restrict__ xp, int64_t xp_part,
                                                                  int* __restrict__ xe, int* __restrict__ arrived,
                                                                  uint32_t* __restrict__ levels, int level_words) {
    __shared__ double s_red[kRouteNW][4][kWave];
    constexpr int V = 16 / sizeof(XT);                 // elements of a 16-byte load
    typedef XT vec __attribute__((ext_vector_type(V)));
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, kq = lane >> 4;
    const int t = blockIdx.y * kRowTile + r, e = blockIdx.x * kRowTile + r;
    const int groups = H / 32, step = gridDim.z * kRouteNW;
    const int g0 = blockIdx.z * kRouteNW + wave;
    if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0)
        for (int i = threadIdx.x; i < H / kRowTile; i += kRouteNW * 64) arrived[i] = 0;
    const int block = (blockIdx.z * gridDim.y + blockIdx.y) * gridDim.x + blockIdx.x;
    const int threads = gridDim.x * gridDim.y * gridDim.z * (kRouteNW * 64);
    for (int i = block * (kRouteNW * 64) + threadIdx.x; i < level_words; i += threads) levels[i] = 0u;
    // For the rows' largest values: the waves share out the tile's rows (n of them, span waves each), a wave's first
    // load goes with those of the products.
    __shared__ uint32_t s_top[kRowTile];
    const int n = min(T - static_cast<int>(blockIdx.y) * kRowTile, kRowTile), span = kRouteNW / n;
    const bool top = F16 && blockIdx.x == 0 && wave < n * span;   // uniform over a wave
    const XT* row = x + static_cast<int64_t>(blockIdx.y * kRowTile + wave % n) * H;
    const int h_top = (wave / n * kWave + lane) * V;
    vec first = {};
    if constexpr (F16) {
        if (top && h_top < H) first = *reinterpret_cast<const vec*>(row + h_top);
        if (threadIdx.x < kRowTile) s_top[threadIdx.x] = 0u;
    }
    doublex4 acc = {0.0, 0.0, 0.0, 0.0};
    vec xv[kRouteGroups][8 / V];
    for (int gb = g0; gb < groups; gb += kRouteGroups * step) {
        XT wv[kRouteGroups][8];
#pragma unroll
        for (int q = 0; q < kRouteGroups; ++q) {
            const int g = gb + q * step;
            const bool in = g < groups;                // uniform
            const int h0 = (in ? g : g0) * 32 + kq * 8;
            const XT* wp = w + static_cast<int64_t>(h0) * E + min(e, E - 1);
#pragma unroll
            for (int j = 0; j < 8; ++j) wv[q][j] = wp[static_cast<int64_t>(j) * E];
            const vec* xs = reinterpret_cast<const vec*>(x + static_cast<int64_t>(min(t, T - 1)) * H + h0);
#pragma unroll
            for (int j = 0; j < 8 / V; ++j) xv[q][j] = xs[j];
        }
        // values of rows past T and columns past E are computed and dropped
#pragma unroll
        for (int q = 0; q < kRouteGroups; ++q) {
            if (gb + q * step >= groups) break;        // uniform
#pragma unroll
            for (int j = 0; j < 8; ++j)
                acc = __builtin_amdgcn_mfma_f64_16x16x4f64(widen<XT>(xv[q][j / V][j % V]), widen<XT>(wv[q][j]), acc, 0,
                                                           0, 0);
            if constexpr (NPX > 0 && !F16) {
                if (blockIdx.x == 0 && t < T) {
                    const int h0 = (gb + q * step) * 32 + kq * 8;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        uint16_t p[NPX];
                        split_parts<NPX, F16>(static_cast<float>(xv[q][j / V][j % V]), p);
#pragma unroll
                        for (int n = 0; n < NPX; ++n) xp[n * xp_part + static_cast<int64_t>(t) * H + h0 + j] = p[n];
                    }
                }
            }
        }
    }
#pragma unroll
    for (int v = 0; v < 4; ++v) s_red[wave][v][lane] = acc[v];
    __syncthreads();
    if constexpr (F16) {
        if (top) {
            float m = 0.0f;
            auto take = [&](const vec& v) {
#pragma unroll
                for (int i = 0; i < V; ++i) m = fmaxf(m, fabsf(v[i]));   // past NaN
            };
            take(first);
#pragma unroll 4
            for (int h = h_top + span * kWave * V; h < H; h += span * kWave * V)
                take(*reinterpret_cast<const vec*>(row + h));
            const uint32_t most = row_max(__float_as_uint(fminf(m, 65504.0f)));
            if (r == 0) atomicMax(&s_top[wave % n], most);
        }
        if (blockIdx.x == 0) __syncthreads();          // uniform over the workgroup
        if (blockIdx.x == 0 && t < T) {
            const int exp = 14 + 127 - static_cast<int>(s_top[r] >> 23);
            if (blockIdx.z == 0 && wave == 0 && kq == 0) xe[t] = exp;
            const bool held = groups <= step;          // the wave's only group is still in registers
            for (int g = g0; g < groups; g += step) {
                const int h0 = g * 32 + kq * 8;
                const int64_t at = static_cast<int64_t>(t) * H + h0;
                uint32_t part[NPX][8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float v = held ? xv[0][j / V][j % V] : x[at + j], c = fminf(fmaxf(v, -65504.0f), 65504.0f);
                    uint16_t q[NPX];
                    split_parts<NPX, true>(ldexpf(v == v ? c : v, exp), q);
#pragma unroll
                    for (int i = 0; i < NPX; ++i) part[i][j] = q[i];
                }
#pragma unroll
                for (int i = 0; i < NPX; ++i)
                    *reinterpret_cast<u32x4*>(xp + i * xp_part + at) =
                        u32x4{part[i][0] | part[i][1] << 16, part[i][2] | part[i][3] << 16,
                              part[i][4] | part[i][5] << 16, part[i][6] | part[i][7] << 16};
            }
        }
    }
    if (threadIdx.x < 256) {
        const int v = threadIdx.x >> 6;
        double s = 0.0;
#pragma unroll
        for (int q = 0; q < kRouteNW; ++q) s += s_red[q][v][lane];
        // register v of lane l: row 4 v + l / 16, column l % 16
        const int tt = blockIdx.y * kRowTile + 4 * v + kq;
        if (tt < T && e < E) part[(static_cast<int64_t>(blockIdx.z) * T + tt) * E + e] = s;
    }
}

// ---- selection ------------------------------------------------------------------

// The logit of (t, e): its slices' sums, then the bias.
__device__ __forceinline__ double logit_of(const FewArgs& p, int t, int e) {
    const double* q = p.part + static_cast<int64_t>(t) * p.E + e;
    const int64_t slice = static_cast<int64_t>(p.T) * p.E;
    double v = 0.0;
    for (int s = 0; s < p.S; ++s) v += q[s * slice];
    if (p.bias != nullptr) v += p.bias[e];
    return v + 0.0;                                    // -0 and +0 compare equal
}

// A double's bits in the order of the numbers, and back.
__device__ __forceinline__ uint64_t ordered(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    return u ^ ((u >> 63) ? ~0ull : (1ull << 63));
}
__device__ __forceinline__ double unordered(uint64_t u) {
    return __builtin_bit_cast(double, u ^ ((u >> 63) ? (1ull << 63) : ~0ull));
}

// The better of this lane's (key, index) and the one N lanes on in its row of 16.
template <int CTRL>
__device__ __forceinline__ void row_best(uint64_t& key, int& index) {
    const uint64_t k = (static_cast<uint64_t>(row_rotate<CTRL>(static_cast<uint32_t>(key >> 32))) << 32) |
                       row_rotate<CTRL>(static_cast<uint32_t>(key));
    const int i = static_cast<int>(row_rotate<CTRL>(static_cast<uint32_t>(index)));
    const bool take = k > key || (k == key && i < index);
    key = take ? k : key;
    index = take ? i : index;
}

// The highest level at which a row's 16 columns, one to each of 16 lanes, stay below 2^15.
__device__ __forceinline__ int level_of(float v, int top) {
    const uint32_t m = row_max(__float_as_uint(fabsf(v)));   // ordered as the numbers, NaN above them
    const int room = 127 + 14 - static_cast<int>(m >> 23);
    return room < kLevelBits ? 0 : min(room / kLevelBits, top);
}

// K rounds of a row whose keys its lanes hold, HELD each: winner k's index to
// idx[k], its key to mine[k] (in LDS the row's keys are no longer needed).
template <int HELD>
__device__ __forceinline__ void held_rounds(int E, int K, bool on, uint64_t* mine, int* idx) {
    const int lane = threadIdx.x & (kWave - 1), c = lane & 15;
    uint64_t held[HELD];
#pragma unroll
    for (int q = 0; q < HELD; ++q) held[q] = q * 16 + c < E ? mine[q * 16 + c] : 0;
#pragma unroll 1
    for (int k = 0; k < K; ++k) {
        uint64_t key = held[0];
        int index = c;
#pragma unroll
        for (int q = 1; q < HELD; ++q) {
            const bool take = held[q] > key;   // the lower index stays
            key = take ? held[q] : key;
            index = take ? q * 16 + c : index;
        }
        const uint32_t own = static_cast<uint32_t>(key >> 32), m = row_max(own);
        const uint32_t best = static_cast<uint32_t>(__ballot(own == m) >> (lane & 48)) & 0xFFFFu;
        bool win = own == m;
        if (__ballot((best & (best - 1u)) != 0u) != 0ull) {   // some row's upper words agree
            uint64_t top = key;
            int where = index;
            row_best<0x128>(top, where);
            row_best<0x124>(top, where);
            row_best<0x122>(top, where);
            row_best<0x121>(top, where);
            win = where == index;
        }
        if (win) {
            if (on) {
                idx[k] = index;
                mine[k] = key;
            }
#pragma unroll
            for (int q = 0; q < HELD; ++q)
                if (index == q * 16 + c) held[q] = 0;
        }
    }
}

// Every token's K best experts in order (larger logit first, equal ones by index)
// and their weights, to LDS (idx, w: [T K]).  Tokens are taken as many at a time
// as `keys` (`room` of them) holds the ordered logits of, one to a row of 16
// lanes, whose K rounds run side by side.  A lane owns every 16th expert; a round
// takes the best of its keys, then the best of the row.  Up to 256 experts the
// keys stay in registers and the row compares their upper words by DPP maxima,
// the rest only where two lanes' agree; beyond that a round scans the LDS keys.
// The rounds' loop is left rolled: a launch starts with a cold instruction
// cache, and straight code runs at the rate it is fetched (unrolled rounds of one
// token after the other took 9 us for 24 tokens, these take under 3).
__device__ __forceinline__ void select_experts(const FewArgs& p, uint64_t* keys, int room, int* idx, float* w) {
    const int tid = threadIdx.x, lane = tid & (kWave - 1), c = lane & 15;
    constexpr int kRows = kNW * 4;
    const int batch = min(kRows, room / p.E);
    for (int t0 = 0; t0 < p.T; t0 += batch) {
        const int n = min(batch, p.T - t0);
        for (int i = tid; i < n * p.E; i += kNW * kWave) {
            const int t = i / p.E;
            keys[i] = ordered(logit_of(p, t0 + t, i - t * p.E));
        }
        __syncthreads();
        const int row = tid >> 4;
        const bool on = row < n;
        uint64_t* mine = keys + (on ? row : 0) * p.E;
        const int at = (t0 + row) * p.K;               // used where on
        if (p.E <= 128) held_rounds<8>(p.E, p.K, on, mine, idx + at);       // uniform
        else if (p.E <= 256) held_rounds<16>(p.E, p.K, on, mine, idx + at);
        else {
            double top = 0.0;
#pragma unroll 1
            for (int k = 0; k < p.K; ++k) {
                uint64_t key = 0;
                int index = 0x7FFFFFFF;
#pragma unroll 2
                for (int e = c; e < p.E; e += 16) {
                    const uint64_t v = mine[e];
                    if (v > key || index == 0x7FFFFFFF) {
                        key = v;
                        index = e;
                    }
                }
                row_best<0x128>(key, index);
                row_best<0x124>(key, index);
                row_best<0x122>(key, index);
                row_best<0x121>(key, index);
                if (on && c == 0) {
                    mine[index] = 0;
                    const double v = unordered(key);
                    if (k == 0) top = v;
                    idx[at + k] = index;
                    w[at + k] = static_cast<float>(v - top);
                }
                asm volatile("" ::: "memory");         // a wave's LDS operations run in order
            }
        }
        if (on) {
            if (p.E <= 256)
                for (int k = c; k < p.K; k += 16) w[at + k] = static_cast<float>(unordered(mine[k]) - unordered(mine[0]));
            asm volatile("" ::: "memory");
            for (int k = c; k < p.K; k += 16) w[at + k] = expf(w[at + k]);
            asm volatile("" ::: "memory");
            float sum = 0.0f;
            for (int k = 0; k < p.K; ++k) sum += w[at + k];
            asm volatile("" ::: "memory");
            for (int k = c; k < p.K; k += 16) w[at + k] = w[at + k] / sum;
        }
        __syncthreads();
    }
}

// LDS tables of the routing, sized by the call (T K pairs, at most `amax` chosen
// local experts).
struct Tables {
    int* idx;          // [T K] expert of (t, j)
    float* w;          // [T K]
    int* act;          // [amax] local index of the a-th chosen expert, ascending
    int* pos;          // [E_loc] 0 or 1 + its place in act
    int8_t* slot;      // [amax][T] slot of token t that chose expert a, or -1
    int* count;        // number of chosen local experts
};

struct TableSizes {
    size_t idx, w, act, pos, slot, count, total;
};

__host__ __device__ inline TableSizes table_sizes(int T, int K, int E_loc) {
    const int pairs = T * K, amax = pairs < E_loc ? pairs : E_loc;
    TableSizes z;
    z.idx = 0;
    z.w = z.idx + 4 * static_cast<size_t>(pairs);
    z.act = z.w + 4 * static_cast<size_t>(pairs);
    z.pos = z.act + 4 * static_cast<size_t>(amax);
    z.count = z.pos + 4 * static_cast<size_t>(E_loc);
    z.slot = z.count + 4;
    z.total = (z.slot + static_cast<size_t>(amax) * T + 15) & ~size_t(15);
    return z;
}

__device__ __forceinline__ Tables carve_tables(char* base, const FewArgs& p) {
    const TableSizes z = table_sizes(p.T, p.K, p.E_loc);
    Tables s;
    s.idx = reinterpret_cast<int*>(base + z.idx);
    s.w = reinterpret_cast<float*>(base + z.w);
    s.act = reinterpret_cast<int*>(base + z.act);
    s.pos = reinterpret_cast<int*>(base + z.pos);
    s.count = reinterpret_cast<int*>(base + z.count);
    s.slot = reinterpret_cast<int8_t*>(base + z.slot);
    return s;
}

// From idx (complete, synchronised): the chosen local experts and who chose them.
// Every thread of the workgroup takes part.
__device__ __forceinline__ void build_tables(const Tables& s, const FewArgs& p) {
    const int tid = threadIdx.x, n = blockDim.x, pairs = p.T * p.K;
    const int amax = min(pairs, p.E_loc);
    for (int i = tid; i < p.E_loc; i += n) s.pos[i] = 0;
    for (int i = tid; i < amax * p.T; i += n) s.slot[i] = -1;
    __syncthreads();
    for (int i = tid; i < pairs; i += n) {
        const int e = s.idx[i] - p.e_begin;
        if (e >= 0 && e < p.E_loc) s.pos[e] = 1;
    }
    __syncthreads();
    if (tid < kWave) {
        int run = 0;
        for (int b = 0; b < p.E_loc; b += kWave) {
            const int e = b + tid;
            const bool on = e < p.E_loc && s.pos[e] != 0;
            const uint64_t m = __ballot(on);
            if (on) {
                const int a = run + __popcll(m & ((1ull << tid) - 1ull));
                s.act[a] = e;
                s.pos[e] = 1 + a;
            }
            run += __popcll(m);
        }
        if (tid == 0) *s.count = run;
    }
    __syncthreads();
    for (int i = tid; i < pairs; i += n) {
        const int e = s.idx[i] - p.e_begin;
        if (e >= 0 && e < p.E_loc) {
            const int t = i / p.K;
            s.slot[(s.pos[e] - 1) * p.T + t] = static_cast<int8_t>(i - t * p.K);
        }
    }
    __syncthreads();
}

// ---- gate and up ------------------------------------------------------------------
// Bound by the weights' arrival once the launch has started and selected (about
// 5 us): 32 tokens, who choose 111 of 128 experts, read 2.8 GB in 443 us (6.3
// TB/s); one token 201 MB in 39.6 us (5.1), with MXFP8 104 MB in 27.3 (3.8).
// An even number of units for every workgroup (384 of them, two each, for 768
// units) was slower than 512 workgroups of which half take two: 53 us against 47
// for the MXFP8 layer.

// Steps wave, wave + kNW, ... of a gate/up unit.
template <int NP, bool MX, int MT>
struct GateUpCursor {
    const uint8_t* b;          // this lane's gate bytes of the step
    const uint8_t* sc;         // its scale bytes (MXFP8): gate, and `sc_up` further the up column's
    int sc_up;
    __amdgpu_buffer_rsrc_t rows;
    uint32_t off[MT];          // byte offset of this lane's k group in part 0 of its row, or out of range
    uint32_t part_bytes;

    __device__ __forceinline__ void load(StepRegs<NP, MX, MT, 2>& s) {
        load_weights<MX>(b, s.b[0]);
        load_weights<MX>(b + (MX ? 2048 : 1024), s.b[1]);   // up columns: the other half of the pair
        if constexpr (MX) {
            s.sc[0] = sc[0];
            s.sc[1] = sc[sc_up];
        }
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int q = 0; q < NP; ++q) load_row(rows, off[m] + q * part_bytes, s.a[m][q]);
        b += kNW * step_bytes<MX>();
        if constexpr (MX) sc += kNW * 2;
#pragma unroll
        for (int m = 0; m < MT; ++m) off[m] += kNW * 128;
    }
};

static_assert(kNW * 2 * 4 * kWave * 4 / 8 >= 1024, "one token's keys fit the reduction buffer");

template <int NP, bool F16, bool MX, int MT, int NPH, bool F16H>
__global__ __launch_bounds__(kNW * 64, gate_up_waves(NP, MX, MT)) void few_gate_up_kernel(FewArgs p) {
    extern __shared__ __attribute__((aligned(16))) char smem[];
    __shared__ __attribute__((aligned(16))) float s_red[kNW][MT][2][4][kWave];
    const Tables tb = carve_tables(smem, p);
    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

    select_experts(p, reinterpret_cast<uint64_t*>(&s_red[0][0][0][0][0]), sizeof(s_red) / 8, tb.idx, tb.w);
    if (blockIdx.x == 0)
        for (int i = tid; i < p.T * p.K; i += kNW * 64) {
            p.idx[i] = tb.idx[i];
            p.w[i] = tb.w[i];
        }
    build_tables(tb, p);

    // the token that this thread finishes: a unit's thread -> (row tile, register, lane), row 4 (lane / 16) + register,
    // column lane % 16
    const int token = (tid >> 8) * kRowTile + (lane >> 4) * 4 + ((tid >> 6) & 3);
    int a_exp = 0;
    if constexpr (NP == 2)
        if (token < p.T) a_exp = p.a_exp[token];
    const int nb = p.I / kRowTile;                     // units per expert
    const int units = *tb.count * nb;
    const int nk = p.H / 64;                           // steps of a unit
    const __amdgpu_buffer_rsrc_t rows =
        __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(p.a), 0, kBufferRange, kBufferFlags);
    GateUpCursor<NP, MX, MT> cur;
    cur.rows = rows;
    cur.part_bytes = static_cast<uint32_t>(p.a_part * 2);
    cur.sc_up = p.H;                                   // 32 columns further, H / 32 bytes each
    const int steps = nk > wave ? (nk - wave + kNW - 1) / kNW : 0;
    auto enter = [&](int unit) {
        const int a = unit / nb, u = unit - a * nb;
        const int e = __builtin_amdgcn_readfirstlane(tb.act[a]);
        const int pair = u >> 1, c0 = (u & 1) * 16;
        const int8_t* slot = tb.slot + a * p.T;
        const int64_t first = (static_cast<int64_t>(e) * (p.I >> 5) + pair) * nk + wave;
        cur.b = p.gu + first * step_bytes<MX>() + step_lane_offset<MX>(0, c0);
        if constexpr (MX) {
            const int64_t col = static_cast<int64_t>(e) * 2 * p.I + pair * 64 + c0 + (lane & 15);
            cur.sc = p.gu_scales + col * (p.H / 32) + wave * 2 + (lane >> 5);
        }
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const int t = m * kRowTile + (lane & 15);
            const bool on = t < p.T && slot[t < p.T ? t : 0] >= 0;
            cur.off[m] = on ? static_cast<uint32_t>(t * p.H + (wave * 4 + (lane >> 4)) * 16) * 2 : kOutOfRange;
        }
    };
    StepRegs<NP, MX, MT, 2> ring[gate_up_ring(NP, MX, MT)];
    int unit = blockIdx.x;
    if (unit < units) {
        enter(unit);
        start_steps(steps, cur, ring);
    }
    while (unit < units) {                             // uniform over the workgroup
        Acc<NP, F16, MX, MT, 2> acc;
        acc.clear();
        run_steps(steps, cur, ring, acc);
        // the next unit's first loads are on their way while this one is finished
        const int done = unit;
        unit += gridDim.x;
        if (unit < units) {
            enter(unit);
            start_steps(steps, cur, ring);
        }
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int v = 0; v < 4; ++v) s_red[wave][m][c][v][lane] = acc.value(m, c, v);
        lds_barrier();
        if (tid < MT * 256) {
            const int a = done / nb, u = done - a * nb;
            const int m = tid >> 8, v = (tid >> 6) & 3, t = token;
            float g = 0.0f, up = 0.0f;
#pragma unroll
            for (int q = 0; q < kNW; ++q) {
                g += s_red[q][m][0][v][lane];
                up += s_red[q][m][1][v][lane];
            }
            if constexpr (NP == 2) {
                g = ldexpf(g, -a_exp);
                up = ldexpf(up, -a_exp);
            }
            const int j = t < p.T ? tb.slot[a * p.T + t] : -1;
            if (j >= 0) {
                const int row = t * p.K + j;
                const float act = g / (1.0f + expf(-g)) * up * tb.w[row];
                const int64_t pairs = static_cast<int64_t>(p.T) * p.K;
                auto write = [&](int level, float v) {
                    uint16_t part[NPH];
                    split_parts<NPH, F16H>(v, part);
#pragma unroll
                    for (int q = 0; q < NPH; ++q)
                        p.h[((level * NPH + q) * pairs + row) * p.I + u * kRowTile + (lane & 15)] = part[q];
                };
                write(0, act);
                if constexpr (F16H) {
                    const int level = level_of(act, p.top);
                    if (level > 0) {
                        float v = act;
#pragma unroll 1
                        for (int l = 1; l <= level; ++l) write(l, v *= 1 << kLevelBits);
                        if ((lane & 15) == 0) {
                            p.levels[row * nb + u] = static_cast<uint8_t>(level);
                            *p.above = 1;
                        }
                    }
                }
            }
        }
        lds_barrier();                                 // s_red is free
    }
}

// ---- down and combine -----------------------------------------------------------------

// The rows a_{t,j} grouped for the down product: pairs (t, j) with a local expert,
// ordered by expert; a segment is up to RV of one expert's pairs.
struct Segments {
    int16_t* order;    // [T K] pairs t K + j
    int16_t* start;    // [T K] first pair of a segment in order
    int16_t* expert;   // [T K] its local expert
    int8_t* rows;      // [T K] its pairs
    int* first;        // [E_loc] first place of an expert's pairs
    uint32_t* tokens;  // [E_loc] bit t: token t chose the expert
    int* count;        // segments
};

struct SegmentSizes {
    size_t order, start, expert, first, tokens, count, rows, total;
};

__host__ __device__ inline SegmentSizes segment_sizes(int T, int K, int E_loc) {
    const size_t pairs = static_cast<size_t>(T) * K, E = static_cast<size_t>(E_loc);
    SegmentSizes z;
    z.first = 0;
    z.tokens = z.first + 4 * E;
    z.count = z.tokens + 4 * E;
    z.order = z.count + 4;
    z.start = z.order + 2 * pairs;
    z.expert = z.start + 2 * pairs;
    z.rows = z.expert + 2 * pairs;
    z.total = (z.rows + pairs + 15) & ~size_t(15);
    return z;
}

__device__ __forceinline__ Segments carve_segments(char* base, const FewArgs& p) {
    const SegmentSizes z = segment_sizes(p.T, p.K, p.E_loc);
    Segments s;
    s.order = reinterpret_cast<int16_t*>(base + z.order);
    s.start = reinterpret_cast<int16_t*>(base + z.start);
    s.expert = reinterpret_cast<int16_t*>(base + z.expert);
    s.rows = reinterpret_cast<int8_t*>(base + z.rows);
    s.first = reinterpret_cast<int*>(base + z.first);
    s.tokens = reinterpret_cast<uint32_t*>(base + z.tokens);
    s.count = reinterpret_cast<int*>(base + z.count);
    return s;
}

// Every thread of the workgroup takes part.  An expert's pairs are in order of
// their tokens (at most 32, a bit each), so every workgroup builds the same list.
__device__ __forceinline__ void build_segments(const Segments& s, const FewArgs& p, int RV) {
    const int tid = threadIdx.x, n = blockDim.x, pairs = p.T * p.K;
    for (int i = tid; i < p.E_loc; i += n) s.tokens[i] = 0u;
    __syncthreads();
    for (int i = tid; i < pairs; i += n) {
        const int e = p.idx[i] - p.e_begin;
        if (e >= 0 && e < p.E_loc) atomicOr(&s.tokens[e], 1u << (i / p.K));
    }
    __syncthreads();
    if (tid < kWave) {
        int run = 0, segs = 0;                         // pairs and segments of the experts before
        for (int b = 0; b < p.E_loc; b += kWave) {
            const int e = b + tid;
            const int c = e < p.E_loc ? __popc(s.tokens[e]) : 0, g = (c + RV - 1) / RV;
            int ic = c, ig = g;
#pragma unroll
            for (int off = 1; off < kWave; off <<= 1) {
                const int oc = __shfl_up(ic, off, kWave), og = __shfl_up(ig, off, kWave);
                if (tid >= off) {
                    ic += oc;
                    ig += og;
                }
            }
            const int f = run + ic - c;
            if (e < p.E_loc) s.first[e] = f;
            for (int q = 0; q < g; ++q) {
                const int at = segs + ig - g + q;
                s.start[at] = static_cast<int16_t>(f + q * RV);
                s.expert[at] = static_cast<int16_t>(e);
                s.rows[at] = static_cast<int8_t>(min(RV, c - q * RV));
            }
            run += __shfl(ic, kWave - 1, kWave);
            segs += __shfl(ig, kWave - 1, kWave);
        }
        if (tid == 0) *s.count = segs;
    }
    __syncthreads();
    for (int i = tid; i < pairs; i += n) {
        const int e = p.idx[i] - p.e_begin;
        if (e >= 0 && e < p.E_loc)
            s.order[s.first[e] + __popc(s.tokens[e] & ((1u << (i / p.K)) - 1u))] = static_cast<int16_t>(i);
    }
    __syncthreads();
}

// The level of every token's rows: the least of its units'.  Every thread of the
// workgroup takes part; a wave takes every kNW-th pair, a lane four units at once.
__device__ __forceinline__ void token_levels(const Segments& s, const FewArgs& p, int* level) {
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int words = p.I / 64, segs = *s.count, pairs = segs > 0 ? s.start[segs - 1] + s.rows[segs - 1] : 0;
    const uint32_t* units = reinterpret_cast<const uint32_t*>(p.levels);
    if (tid < p.T) level[tid] = kLevels - 1;
    __syncthreads();
#pragma unroll 4
    for (int q = wave; q < pairs; q += kNW) {
        const int pair = s.order[q];
        for (int i = lane; i < words; i += kWave) {
            const uint32_t v = units[pair * words + i];
            const uint32_t least = min(min(v & 255u, v >> 8 & 255u), min(v >> 16 & 255u, v >> 24));
            atomicMin(&level[pair / p.K], static_cast<int>(least));
        }
    }
    __syncthreads();
}

// How a segment's rows and their parts share the RT * 16 MFMA rows: part and row
// of MFMA row r of tile m.  Stacking the parts costs one A load per tile where
// separate products would cost one per part, and loads are what a step is made of.
template <int NP, int RT> struct RowMap;
template <> struct RowMap<2, 1> {                      // 8 rows: part 0 in MFMA rows 0-7, part 1 in 8-15
    static constexpr int RV = 8;
    __device__ static int part(int, int r) { return r >> 3; }
    __device__ static int row(int, int r) { return r & 7; }
};
template <> struct RowMap<2, 2> {                      // 16 rows, a tile per part
    static constexpr int RV = 16;
    __device__ static int part(int m, int) { return m; }
    __device__ static int row(int, int r) { return r; }
};
template <> struct RowMap<3, 1> {                      // 4 rows, parts in groups of four MFMA rows
    static constexpr int RV = 4;
    __device__ static int part(int, int r) { return r >> 2; }
    __device__ static int row(int, int r) { return r & 3; }
};
template <> struct RowMap<3, 2> {                      // 8 rows: parts 0 and 1 in tile 0, part 2 in tile 1
    static constexpr int RV = 8;
    __device__ static int part(int m, int r) { return m * 2 + (r >> 3); }
    __device__ static int row(int, int r) { return r & 7; }
};

// The segment rows' sums from the accumulators: register v of this lane, valid in
// the lanes of the first RV MFMA rows (row 4 (lane / 16) + v, column lane % 16).
template <int NP, int RT, typename AccT>
__device__ __forceinline__ float joined(const AccT& acc, int v) {
    if constexpr (NP == 2 && RT == 1) {
        return acc.v[0][0][0][v] + __shfl_xor(acc.v[0][0][0][v], 32, kWave) * (1.0f / kLoScale);
    } else if constexpr (NP == 2) {
        return acc.v[0][0][0][v] + acc.v[0][1][0][v] * (1.0f / kLoScale);
    } else if constexpr (RT == 1) {
        const float x = acc.v[0][0][0][v];
        return (x + __shfl(x, (threadIdx.x + 16) & 63, kWave)) + __shfl(x, (threadIdx.x + 32) & 63, kWave);
    } else {
        return (acc.v[0][0][0][v] + __shfl_xor(acc.v[0][0][0][v], 32, kWave)) + acc.v[0][1][0][v];
    }
}

// The loads of consecutive steps: the I of a segment, then the next segment's.
template <int NP, bool MX, int RT>
struct DownCursor {
    const FewArgs* p;
    const Segments* sg;
    const int* level;          // [T] of the tokens' rows, or NULL: 0
    bool whole;                // one row per token throughout: every expert's segment has the tokens as its rows
    const uint8_t* b0;         // this lane's bytes of expert 0's step 0
    const uint8_t* sc0;        // this lane's scale byte of expert 0's step 0
    int64_t b_expert, sc_expert;   // bytes per expert
    __amdgpu_buffer_rsrc_t rows;
    uint32_t part_bytes;
    int nk, seg, ks;           // steps per segment; the next step
    const uint8_t* b;
    const uint8_t* sc;
    uint32_t off[RT];

    __device__ __forceinline__ void enter() {
        typedef RowMap<NP, RT> Map;
        const int lane = threadIdx.x & (kWave - 1);
        const int e = __builtin_amdgcn_readfirstlane(sg->expert[seg]);
        const int first = __builtin_amdgcn_readfirstlane(sg->start[seg]);
        const int n = __builtin_amdgcn_readfirstlane(sg->rows[seg]);
        b = b0 + e * b_expert + static_cast<int64_t>(ks) * step_bytes<MX>();
        if constexpr (MX) sc = sc0 + e * sc_expert + ks * 2;
#pragma unroll
        for (int m = 0; m < RT; ++m) {
            const int part = Map::part(m, lane & 15), row = Map::row(m, lane & 15);
            int pair = -1;
            if (whole) {
                for (int i = 0; i < n; ++i) {          // uniform; at most a row per token
                    const int q = sg->order[first + i];
                    if (q / p->K == row) pair = q;
                }
            } else if (row < n) {
                pair = sg->order[first + row];
            }
            off[m] = pair >= 0 && part < NP ? part * part_bytes + (static_cast<uint32_t>(pair) * p->I +
                                                                   (ks * 4 + (lane >> 4)) * 16) * 2
                                            : kOutOfRange;
            if (NP == 2 && level != nullptr && off[m] != kOutOfRange) off[m] += level[pair / p->K] * NP * part_bytes;
        }
    }
    __device__ __forceinline__ void load(StepRegs<1, MX, RT, 1>& s) {
        load_weights<MX>(b, s.b[0]);
        if constexpr (MX) s.sc[0] = sc[0];
#pragma unroll
        for (int m = 0; m < RT; ++m) load_row(rows, off[m], s.a[m][0]);
        b += step_bytes<MX>();
        if constexpr (MX) sc += 2;
#pragma unroll
        for (int m = 0; m < RT; ++m) off[m] += 128;
        if (++ks == nk) {                              // uniform
            ks = 0;
            if (++seg < *sg->count) enter();
        }
    }
};

// Bound as gate/up is, behind the segments' tables (about 3 us) and the handing
// over of partial sums (3 us): 32 tokens 1.4 GB in 220 us (6.4 TB/s), one token
// 101 MB in 20.5 us (4.9), with MXFP8 52 MB in 16.6 (3.1).
// A workgroup owns 16 output columns and part blockIdx.y of the steps, each wave a
// contiguous run of them.  A wave adds its rows' sums to its own [T][16] in LDS
// where the segment ends (or once at its end, where MFMA rows are tokens all
// along); the waves' are added in order.  With more than one part, the partial
// sums go to memory, and the workgroup that finds all others done adds them, in
// order of the parts, whatever the order of arrival.
template <int NP, bool F16, bool MX, int RT>
__global__ __launch_bounds__(kNW * 64, 4) void few_down_kernel(FewArgs p) {
    typedef RowMap<NP, RT> Map;
    // Steps in flight, 1 KiB (MXFP8) or 2 of weights each.  Not a close choice: from three on, calls of one to 32
    // tokens took the same within 1 %; fewer cost 8 MXFP8 tokens 2 % (212 us, 207), more would spill registers.
    constexpr int D = MX ? (RT == 1 ? 6 : 4) : (RT == 1 ? 4 : 3);
    extern __shared__ __attribute__((aligned(16))) char smem[];
    float* s_out = reinterpret_cast<float*>(smem);     // [kNW][T][16]
    const Segments sg = carve_segments(smem + kNW * p.T * 64, p);
    __shared__ int s_last, s_level[MOE_FEW_TOKENS_MAX];
    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int unit = blockIdx.x, parts = gridDim.y;

    const bool leveled = NP == 2 && *p.above != 0;     // uniform
    for (int i = tid; i < kNW * p.T * 16; i += kNW * 64) s_out[i] = 0.0f;
    const bool whole = p.T <= Map::RV;
    build_segments(sg, p, Map::RV);
    if (leveled) token_levels(sg, p, s_level);

    const int n64 = unit >> 2, half = (unit >> 1) & 1, c0 = (unit & 1) * 16;
    DownCursor<NP, MX, RT> cur;
    cur.p = &p;
    cur.sg = &sg;
    cur.level = leveled ? s_level : nullptr;
    cur.whole = whole;
    cur.nk = p.I / 64;
    const int segs = __builtin_amdgcn_readfirstlane(*sg.count);
    cur.b_expert = static_cast<int64_t>(p.H >> 6) * cur.nk * step_bytes<MX>();
    cur.b0 = p.dn + static_cast<int64_t>(n64) * cur.nk * step_bytes<MX>() + step_lane_offset<MX>(half, c0);
    if constexpr (MX) {
        cur.sc_expert = static_cast<int64_t>(p.H) * (p.I / 32);
        cur.sc0 = p.dn_scales + static_cast<int64_t>(unit * kRowTile + (lane & 15)) * (p.I / 32) + (lane >> 5);
    }
    cur.rows = __builtin_amdgcn_make_buffer_rsrc(p.h, 0, kBufferRange, kBufferFlags);
    cur.part_bytes = static_cast<uint32_t>(static_cast<int64_t>(p.T) * p.K * p.I * 2);
    // this wave's steps: an even share of all
    const int64_t total = static_cast<int64_t>(segs) * cur.nk, shares = static_cast<int64_t>(parts) * kNW;
    const int64_t share = blockIdx.y * kNW + wave;
    const int64_t lo = total * share / shares, hi = total * (share + 1) / shares;
    const int steps = static_cast<int>(hi - lo);
    cur.seg = static_cast<int>(lo / cur.nk);
    cur.ks = static_cast<int>(lo - static_cast<int64_t>(cur.seg) * cur.nk);
    if (steps > 0) cur.enter();
    int seg = cur.seg, ks = cur.ks;                    // the next step to be added

    Acc<1, F16, MX, RT, 1> acc;
    acc.clear();
    float* mine = s_out + wave * p.T * 16;
    auto flush = [&]() {                               // rows of segment seg
        const int n = whole ? p.T : __builtin_amdgcn_readfirstlane(sg.rows[seg]);
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const float x = joined<NP, RT>(acc, v);
            const int r = (lane >> 4) * 4 + v;
            if (r < n) {
                const int t = whole ? r : sg.order[sg.start[seg] + r] / p.K;
                mine[t * 16 + (lane & 15)] += x;
            }
        }
        acc.clear();
    };
    StepRegs<1, MX, RT, 1> ring[D];
    start_steps(steps, cur, ring);
    run_steps(steps, cur, ring, acc, [&]() {           // after every step
        if (++ks == cur.nk) {                          // uniform
            if (!whole) flush();
            ks = 0;
            ++seg;
        }
    });
    if (steps > 0 && (whole || ks != 0)) flush();
    __syncthreads();
    const int cells = p.T * 16;
    auto write = [&](int i, float s) {                 // element i of [T][16]
        if (leveled) s = ldexpf(s, -kLevelBits * s_level[i >> 4]);
        p.out[static_cast<int64_t>(i >> 4) * p.H + unit * kRowTile + (i & 15)] = s;
    };
    if (parts == 1) {
        for (int i = tid; i < cells; i += kNW * 64) {
            float s = 0.0f;
#pragma unroll
            for (int q = 0; q < kNW; ++q) s += s_out[q * cells + i];
            write(i, s);
        }
        return;
    }
    // Partial sums and the counter move by agent-scope relaxed atomics.  What orders
    // them is not the language's memory model (relaxed atomics have no order) but
    // two properties of gfx950: the vector-memory counter counts an agent-scope store
    // as outstanding until it is where every XCD sees it, and an agent-scope load
    // issued after that returns no older copy.  With the wait for the counter and
    // the barrier before the count, the workgroup that counts last reads complete
    // sums.  (A release or acquire at agent scope would write back and invalidate a
    // whole L2 per workgroup: 8 to 12 us here.)
    for (int i = tid; i < cells; i += kNW * 64) {
        float s = 0.0f;
#pragma unroll
        for (int q = 0; q < kNW; ++q) s += s_out[q * cells + i];
        __hip_atomic_store(&p.sums[(static_cast<int64_t>(unit) * parts + blockIdx.y) * cells + i], s, __ATOMIC_RELAXED,
                           __HIP_MEMORY_SCOPE_AGENT);
    }
    wait_vmcnt<0>();                                   // this thread's stores are complete
    __syncthreads();
    if (tid == 0)
        s_last = __hip_atomic_fetch_add(&p.arrived[unit], 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == parts - 1;
    __syncthreads();
    if (!s_last) return;
    for (int i = tid; i < cells; i += kNW * 64) {
        float s = 0.0f;
        for (int q = 0; q < parts; ++q)
            s += __hip_atomic_load(&p.sums[(static_cast<int64_t>(unit) * parts + q) * cells + i], __ATOMIC_RELAXED,
                                   __HIP_MEMORY_SCOPE_AGENT);
        write(i, s);
    }
}

// ---- host -----------------------------------------------------------------------------

// Slices of H in the route step: few enough that a wave has at most
// kRouteGroups groups in flight at once and that every gate/up workgroup adds
// them up quickly; up to eight tokens take twice as many, as their partials are
// short.  The layer with 8 of 128 experts of hidden 4096, more slices and fewer:
// one token 24.5 and 24.8 us, 4 tokens 32.6 and 33.0, 8 tokens 36.0 and 35.5, 9
// tokens 45.5 and 43.9, 32 tokens 75.0 and 69.0.
int route_slices(int T, int H) {
    const int groups = H / 32;
    const int most = (groups + kRouteNW - 1) / kRouteNW;           // one group a wave
    const int few = (groups + kRouteNW * kRouteGroups - 1) / (kRouteNW * kRouteGroups);
    const int S = T <= 8 ? most : few;
    return S < kMaxSlices ? S : kMaxSlices;
}

// Highest level of the rows a (two parts each): the last, or as many as offsets below the buffer range allow.
int top_level(const moe_shape& s) {
    const int64_t level = static_cast<int64_t>(s.T) * s.K * s.I * 2 * 2;
    return static_cast<int>(std::min<int64_t>(kLevels, kBufferRange / std::max<int64_t>(level, 1))) - 1;
}

// Workgroups that share the down step's reduction for 16 columns: up to two
// workgroups on every CU, as long as a wave keeps 8 KiB of weights of what T
// tokens are expected to choose (it has that much in flight); below that the
// handing over of partial sums (about 3 us) costs more than it saves.
int down_parts(const moe_shape& s, bool mx) {
    const int E_loc = s.e_end - s.e_begin;
    double none = 1.0;                                 // an expert that no token chooses
    for (int t = 0; t < s.T; ++t) none *= 1.0 - static_cast<double>(s.K) / s.E;
    const double steps = E_loc * (1.0 - none) * (s.I / 64) / kNW;
    int n = 512 / (s.H / kRowTile);
    const int least = mx ? 8 : 4;
    if (n > steps / least) n = static_cast<int>(steps / least);
    return n < 1 ? 1 : (n > kMaxParts ? kMaxParts : n);
}

size_t down_lds(const moe_shape& s) {
    return static_cast<size_t>(kNW) * s.T * 64 + segment_sizes(s.T, s.K, s.e_end - s.e_begin).total;
}

template <int NP, bool F16, bool MX>
int launch_down(const FewArgs& p, int parts, size_t lds, hipStream_t st) {
    const dim3 g(p.H / kRowTile, parts), block(kNW * 64);
    // One tile of MFMA rows while the tokens fit it, or an evenly routed expert gets at most half of its rows; with
    // more rows to an expert, two tiles save reading its weights again.  Hidden 4096, expert 1536, one tile and two: 16
    // tokens to 4 of 32 experts (2 rows each) 178 and 182 us, of 16 (4) 108.7 and 110.9, of 12 (5.3) 90.1 and 90.0, of
    // 8 (8) 68.9 and 66.3; MXFP8, half the rows to a tile, to 4 of 32 (2) 127 and 136, of 16 (4) 91.6 and 89.2.
    constexpr int RV = RowMap<NP, 1>::RV;
    const bool narrow = p.T <= RV || p.T * p.K <= p.E * RV / 2;
    if (narrow) hipLaunchKernelGGL((few_down_kernel<NP, F16, MX, 1>), g, block, lds, st, p);
    else hipLaunchKernelGGL((few_down_kernel<NP, F16, MX, 2>), g, block, lds, st, p);
    MOE_CHECK_LAUNCH();
    return MOE_OK;
}

template <int MT>
int launch_gate_up(const FewArgs& p, int x_dtype, bool mx, hipStream_t st) {
    const int64_t experts = p.T * p.K < p.E_loc ? p.T * p.K : p.E_loc;
    const int64_t most = experts * (p.I / kRowTile);
    const dim3 g(static_cast<unsigned>(most < 512 ? most : 512)), block(kNW * 64);
    const size_t lds = table_sizes(p.T, p.K, p.E_loc).total;
    if (mx && x_dtype == MOE_BF16)
        hipLaunchKernelGGL((few_gate_up_kernel<1, false, true, MT, 3, false>), g, block, lds, st, p);
    else if (mx)
        hipLaunchKernelGGL((few_gate_up_kernel<3, false, true, MT, 3, false>), g, block, lds, st, p);
    else if (x_dtype == MOE_BF16)
        hipLaunchKernelGGL((few_gate_up_kernel<1, false, false, MT, 2, true>), g, block, lds, st, p);
    else
        hipLaunchKernelGGL((few_gate_up_kernel<2, true, false, MT, 2, true>), g, block, lds, st, p);
    MOE_CHECK_LAUNCH();
    return MOE_OK;
}

inline size_t up256(size_t v) { return (v + 255) & ~size_t(255); }

}  // namespace

static_assert(MOE_FEW_TOKENS_MAX <= 32, "a bit per token");

bool few_tokens_fits(const moe_shape& s) {
    const int64_t rows = static_cast<int64_t>(s.T) * s.K * s.I * 2 * 3, x = static_cast<int64_t>(s.T) * s.H * 2 * 3;
    return s.T <= MOE_FEW_TOKENS_MAX && rows <= kBufferRange && x <= kBufferRange;
}

size_t few_tokens_workspace(const moe_shape& s, void* base, FewWs* w) {
    char* p = static_cast<char*>(base);
    size_t off = 0;
    auto take = [&](size_t bytes) -> char* {
        char* r = p ? p + off : nullptr;
        off += up256(bytes);
        return r;
    };
    const size_t pairs = static_cast<size_t>(s.T) * s.K;
    FewWs z;
    z.part = reinterpret_cast<double*>(take(static_cast<size_t>(kMaxSlices) * s.T * s.E * 8));
    z.idx = reinterpret_cast<int32_t*>(take(pairs * 4));
    z.w = reinterpret_cast<float*>(take(pairs * 4));
    z.x = reinterpret_cast<uint16_t*>(take(static_cast<size_t>(3) * s.T * s.H * 2));
    z.x_exp = reinterpret_cast<int*>(take(static_cast<size_t>(s.T) * 4));
    const size_t h_parts = std::max(3, 2 * (top_level(s) + 1));    // three (MXFP8), or two at each level
    z.h = reinterpret_cast<uint16_t*>(take(h_parts * pairs * s.I * 2));
    z.sums = reinterpret_cast<float*>(take(static_cast<size_t>(kMaxParts) * s.T * s.H * 4));
    z.arrived = reinterpret_cast<int*>(take(static_cast<size_t>(s.H) / kRowTile * 4));
    z.levels = reinterpret_cast<uint32_t*>(take(pairs * (s.I / kRowTile) + 4));
    if (w != nullptr) *w = z;
    return off;
}

int launch_few_tokens(const moe_shape& s, const void* x, int x_dtype, const void* w_router, const float* bias,
                      const void* packed, bool mx, float* out, int32_t* idx, float* tw, void* ws, hipStream_t st) {
    FewWs z;
    few_tokens_workspace(s, ws, &z);
    FewArgs p{};
    p.T = s.T;
    p.H = s.H;
    p.E = s.E;
    p.K = s.K;
    p.I = s.I;
    p.e_begin = s.e_begin;
    p.E_loc = s.e_end - s.e_begin;
    p.S = route_slices(s.T, s.H);
    p.part = z.part;
    p.bias = bias;
    p.h = z.h;
    p.idx = idx ? idx : z.idx;
    p.w = tw ? tw : z.w;
    p.out = out;
    p.sums = z.sums;
    p.arrived = z.arrived;
    const int level_words = s.T * s.K * (s.I / 64);
    p.levels = reinterpret_cast<uint8_t*>(z.levels);
    p.above = reinterpret_cast<int*>(z.levels + level_words);
    p.top = top_level(s);
    p.a = x_dtype == MOE_BF16 ? static_cast<const uint16_t*>(x) : z.x;
    p.a_part = static_cast<int64_t>(s.T) * s.H;
    p.a_exp = z.x_exp;
    const uint8_t* b = static_cast<const uint8_t*>(packed);
    p.gu = b;
    if (mx) {
        p.dn = p.gu + mx_packed_gate_up_code_bytes(s);
        p.gu_scales = p.dn + mx_packed_down_code_bytes(s);
        p.dn_scales = p.gu_scales + mx_packed_gate_up_code_bytes(s) / 32;
    } else {
        p.dn = p.gu + packed_gate_up_elems(s) * 2;
    }
    const dim3 g((s.E + kRowTile - 1) / kRowTile, (s.T + kRowTile - 1) / kRowTile, p.S), block(kRouteNW * 64);
    if (x_dtype == MOE_BF16)
        hipLaunchKernelGGL((few_route_kernel<uint16_t, 0, false>), g, block, 0, st, static_cast<const uint16_t*>(x),
                           static_cast<const uint16_t*>(w_router), s.T, s.H, s.E, z.part, z.x, p.a_part,
                           z.x_exp, z.arrived, z.levels, mx ? 0 : level_words + 1);
    else if (mx)
        hipLaunchKernelGGL((few_route_kernel<float, 3, false>), g, block, 0, st, static_cast<const float*>(x),
                           static_cast<const float*>(w_router), s.T, s.H, s.E, z.part, z.x, p.a_part,
                           z.x_exp, z.arrived, z.levels, mx ? 0 : level_words + 1);
    else
        hipLaunchKernelGGL((few_route_kernel<float, 2, true>), g, block, 0, st, static_cast<const float*>(x),
                           static_cast<const float*>(w_router), s.T, s.H, s.E, z.part, z.x, p.a_part,
                           z.x_exp, z.arrived, z.levels, mx ? 0 : level_words + 1);
    MOE_CHECK_LAUNCH();
    MOE_TRY(s.T <= kRowTile ? launch_gate_up<1>(p, x_dtype, mx, st) : launch_gate_up<2>(p, x_dtype, mx, st));
    const int parts = down_parts(s, mx);
    return mx ? launch_down<3, false, true>(p, parts, down_lds(s), st)
              : launch_down<2, true, false>(p, parts, down_lds(s), st);
}

}  // namespace moe
