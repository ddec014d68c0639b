// moe.hip -- a mixture-of-experts layer for a few tokens, and the router's choice.
//
// The choice, for a token's logits over E experts: the top_k largest (equal ones by the
// lowest index), weights = their softmax (over the chosen, or over all experts).
// The layer, with [gate; up] and down of every expert in E4M3 codes and 128 x 128 blocks:
//   h = silu(Wg_e x) * (Wu_e x),   y = sum over the token's experts of p_e Wd_e h
// A few tokens reach many experts, so the work is to read each of these experts' codes
// once, at HBM's rate.  Pairs (a token and a choice) are put in order by expert, up to NX of
// an expert make an item, and an item's workgroups read the expert's rows past the registers
// into LDS, 128 or 256 columns a step and one or two steps ahead; from there a wave takes
// them as rows of the matrix instruction, turned into BF16 (exactly: E4M3 has four bits), with
// the pairs as its columns.  Outputs of the pairs are added up per token in the order of its
// choices, so that a result does not hang on which workgroup was first.
//
// Launches: plan, up (with silu and the product as its epilogue), down, join.  With one or two
// tokens, whose pairs fit a wave, the plan is made by each wave itself and the sum belongs to
// down: two launches.
#include "e4m3.hpp"
#include "lds_load.hpp"

#include <algorithm>
#include <type_traits>

namespace pulse {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int ME_EXPERTS = 1024;  // most experts

// ---- the router's choice ----------------------------------------------------------
// A wave takes a token; a lane holds the logits lane, lane + 64, ... as keys that are
// ordered as the logits and, where these are equal, against their indices.
__device__ __forceinline__ uint32_t ordered(float v) {  // -inf ... +inf, then NaN
    const uint32_t b = __float_as_uint(v + 0.0f);  // -0 equals 0
    if ((b & 0x7FFFFFFFu) > 0x7F800000u) return 0xFFFFFFFFu;
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

constexpr uint32_t kMinusInf = 0x007FFFFFu;  // ordered(-inf)

template <int PER>
__global__ __launch_bounds__(256) void k_moe_route(const float *__restrict__ logits, int64_t ld, int32_t T, int32_t E,
                                                   int32_t top_k, int32_t over_all, float scale,
                                                   int32_t *__restrict__ ids, float *__restrict__ weights) {
    const int t = blockIdx.x * 4 + wave_id(), lane = lane_id();
    if (t >= T) return;
    float v[PER];
    uint32_t key[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = i * kWave + lane;
        v[i] = e < E ? logits[(int64_t)t * ld + e] : 0.0f;
        key[i] = e < E ? ordered(v[i]) : 0u;
    }
    float most = 0, sum = 0, chosen = 0;
    int mine = -1;  // lane j: the j-th choice; chosen: its logit
    for (int j = 0; j < top_k; ++j) {
        uint32_t best = 0;
        int at = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (key[i] > best) best = key[i], at = i;
        const uint32_t top = __builtin_amdgcn_readlane(wave_incl_max(best), 63);
        // of the lanes that hold it, the lowest index: the lowest place first, then the lowest lane
        const uint32_t mine_at = (uint32_t)(at * kWave + lane), tie = best == top ? mine_at : 0xFFFFFFFFu;
        const uint64_t ties = __ballot(best == top);
        const uint32_t e = (ties & (ties - 1)) ? ~(uint32_t)__builtin_amdgcn_readlane(wave_incl_max(~tie), 63)
                                               : (uint32_t)__builtin_amdgcn_readlane(mine_at, __builtin_ctzll(ties));
        const bool live = top > kMinusInf;  // an expert with -inf is not chosen
        if (lane == j) mine = live ? (int)e : -1;
        const uint32_t bits = top & 0x80000000u ? top ^ 0x80000000u : ~top;
        const float x = __uint_as_float(bits);
        if (j == 0) most = x;
        if (lane == j) chosen = x;
        if (live)
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (tie == e && i == at) key[i] = 0u;
    }
    if (over_all) {
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (i * kWave + lane < E) sum += expf(v[i] - most);
        sum = wave_reduce_sum(sum);
    } else {
        sum = wave_reduce_sum(mine >= 0 ? expf(chosen - most) : 0.0f);
    }
    if (lane < top_k) {
        ids[(int64_t)t * top_k + lane] = mine;
        weights[(int64_t)t * top_k + lane] = mine >= 0 ? expf(chosen - most) / sum * scale : 0.0f;
    }
}

// f with the logits of a lane as a constant: the least of these that hold E, for each choice goes over
// them all.  Microseconds of 1 and of 65536 tokens, top 8, in this one and in the next: 2 (E = 128) 3.1 and 3.4,
// 31 and 38; 4 (256) 3.6 and 4.1, 42 and 49; 6 (384) 4.4 and 4.5, 53 and 59; 8 (512) 4.8 and, in 16, 6.5, 63 and 98.
template <typename F>
inline void with_logits(int64_t E, F &&f) {
    static_assert(ME_EXPERTS <= 16 * kWave, "the largest holds them all");
    switch ((E + 2 * kWave - 1) / (2 * kWave)) {
    case 1: return f(std::integral_constant<int, 2>{});
    case 2: return f(std::integral_constant<int, 4>{});
    case 3: return f(std::integral_constant<int, 6>{});
    case 4: return f(std::integral_constant<int, 8>{});
    case 5:
    case 6: return f(std::integral_constant<int, 12>{});
    default: return f(std::integral_constant<int, 16>{});
    }
}

// ---- the plan: pairs of token and choice by expert -----------------------------------
// Items of up to NX pairs of one expert.  Where a pair stands among its expert's may
// differ from call to call; its results do not, for every pair is a column of its own.
struct MoePlan {
    int32_t *count;   // [1] items
    int32_t *expert;  // [items]
    int32_t *first;   // [items + 1] first pair of an item in `order`
    int32_t *order;   // [pairs]
};

__global__ __launch_bounds__(1024) void k_moe_plan(const int32_t *__restrict__ ids, int32_t P, int32_t E, int32_t nx,
                                                   MoePlan plan, uint32_t *__restrict__ status) {
    __shared__ int32_t s_n[ME_EXPERTS], s_item[ME_EXPERTS];
    __shared__ int32_t s_sum[2][16];
    const int tid = threadIdx.x;
    s_n[tid] = 0;
    __syncthreads();
    bool bad = false;
    for (int i = tid; i < P; i += 1024) {
        const int e = ids[i];
        if ((uint32_t)e < (uint32_t)E) atomicAdd(&s_n[e], 1);
        else bad |= e != -1;
    }
    if (bad && status) atomicOr(status, 2u);  // PULSE_DS_BADINDEX
    __syncthreads();
    // expert tid: its pairs, its items, and where both begin
    const int n = s_n[tid], items = (n + nx - 1) / nx;
    int total = 0, total_items = 0;
    const int pair0 = block_excl_sum<16>(n, s_sum[0], &total);
    const int item0 = block_excl_sum<16>(items, s_sum[1], &total_items);
    for (int i = 0; i < items; ++i) {
        plan.expert[item0 + i] = tid;
        plan.first[item0 + i] = pair0 + i * nx;
    }
    if (tid == 0) {
        plan.count[0] = total_items;
        plan.first[total_items] = total;
    }
    s_item[tid] = pair0;
    __syncthreads();
    for (int i = tid; i < P; i += 1024) {
        const int e = ids[i];
        if ((uint32_t)e < (uint32_t)E) plan.order[atomicAdd(&s_item[e], 1)] = i;
    }
}

// ---- the experts' products -------------------------------------------------------------
struct MoeArgs {
    const uint16_t *x;   // up: [T][ldx]; down: h [2][pairs][I], the nearest BF16 and that of what it leaves
    int64_t ldx;
    const uint8_t *w;    // [E][R][K] codes
    const float *sw;     // [E][blocks of R][blocks of K]
    uint16_t *h;         // up: written
    float *out;          // down: [pairs][R], written
    const int32_t *ids;  // [pairs]
    MoePlan plan;
    int32_t P, E, R, K;  // R: rows of w (up: 2 I)
    int32_t top_k;
    uint32_t *status;
};

constexpr int MR = 32;  // rows of a wave: 16 of gate and of up, or 32 of down

typedef const __attribute__((address_space(4))) float *scalar_floats;

// A lane's operand of 16 x 16 x 32: eight codes as BF16 (exactly: E4M3 has four bits)
__device__ __forceinline__ bf16x8 widen_codes(uint32_t lo, uint32_t hi) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
    const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
    return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// The n-th set bit (n < popcount)
__device__ __forceinline__ int nth_bit(uint64_t m, int n) {
    for (int i = 0; i < n; ++i) m &= m - 1;
    return __builtin_ctzll(m);
}

// An item: an expert (or -1) and its pairs: bits of `few`, or order[first ...].
struct MoeItem {
    int expert, count, first;
    uint64_t few;
};

__device__ __forceinline__ MoeItem planned_item(const MoeArgs &g, int item, int nx) {
    MoeItem t{-1, 0, 0, 0};
    if (item >= g.plan.count[0]) return t;
    const int e = g.plan.expert[item], p0 = g.plan.first[item];
    int np = g.plan.first[item + 1] - p0;
    // (whatever the plan's buffer holds, nothing outside the tensors is touched)
    if ((uint32_t)e >= (uint32_t)g.E || (uint32_t)p0 >= (uint32_t)g.P || np <= 0) return t;
    np = np < nx ? np : nx;
    return {e, np < g.P - p0 ? np : g.P - p0, p0, 0};
}

// Without a plan: up to 64 pairs, a lane's each.  Items go by the first pair of their expert.
__device__ __forceinline__ MoeItem few_item(const MoeArgs &g, int item, int nx) {
    const int lane = lane_id(), id = lane < g.P ? g.ids[lane] : -1;
    const bool live = (uint32_t)id < (uint32_t)g.E;
    if (item == 0 && blockIdx.x == 0 && !live && id != -1) atomicOr(g.status, 2u);  // PULSE_DS_BADINDEX
    uint64_t left = __ballot(live);
    while (left) {
        const int e = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
        uint64_t same = __ballot(live && id == e);
        left &= ~same;
        for (; same; --item) {  // up to nx of them make an item
            uint64_t part = same;
            for (int i = 0; i < nx && same; ++i) same &= same - 1;
            part &= ~same;
            if (item == 0) return {e, __builtin_popcountll(part), 0, part};
        }
    }
    return {-1, 0, 0, 0};
}

// A step's buffer in LDS: the rows of codes of every wave, and NX rows of x (down: twice,
// h's two parts), for all of them or, with one or two tokens (FEW), for each.  Two workgroups
// a compute unit, so that one begins while the other is under way, where LDS holds them.
// Piece p (16 bytes) of row r lies at p ^ r's low bits, where neither the loads, which fill
// whole rows, nor the reads, 8 rows at one piece, have two lanes in a bank.
template <bool UP, int NX, bool FEW>
struct MoeStage {
    static constexpr int MW = NX >= 64 ? 8 : 4;  // waves: eight share the largest x
    static constexpr int parts = UP ? 1 : 2;
    // Waves that share a tile's contraction.  One token: 1, 2 and 4 of them, 8 of 384 experts x (7168, 2048)
    // 63.7, 63.7 and 64.8 us, 4 of 60 x (2048, 1408) 20.1, 17.4, 17.2, 2 of 16 x (4096, 14336) 79, 80, 86.
    static constexpr int kw = FEW ? 2 : 1;
    static constexpr int cols = NX <= 8 || (NX == 16 && UP) ? 256 : 128;  // of a step
    static constexpr int w_bytes = MR * cols, x_bytes = parts * NX * cols * 2;
    static constexpr int bytes = MW * w_bytes + (FEW ? MW : 1) * x_bytes;
    static constexpr int wp = cols / 16, xp = cols / 8;        // pieces of a row
    static constexpr int w_rows = 64 / wp, x_rows = 64 / xp;   // rows of a load
    static constexpr int w_loads = w_bytes / 1024, x_loads = x_bytes / 1024 / (FEW ? 1 : MW);
    static constexpr int loads = w_loads + x_loads;
    static constexpr int lds = MW == 8 ? 160 * 1024 : 80 * 1024;  // of a workgroup
    static constexpr int stages = 4 * bytes <= lds ? 4 : 3 * bytes <= lds ? 3 : 2;
    static_assert(x_loads * 1024 * (FEW ? 1 : MW) == x_bytes && stages * bytes <= lds, "LDS of a compute unit");
    static_assert((stages - 2) * loads <= 63, "loads in flight");
};

template <bool UP, int NX, bool FEW>
__global__ __launch_bounds__((MoeStage<UP, NX, FEW>::MW * kWave), 2) void k_moe_rows(MoeArgs g) {
    using S = MoeStage<UP, NX, FEW>;
    constexpr int MW = S::MW, kw = S::kw;
    constexpr int CT = (NX + 15) / 16;  // tiles of tokens
    __shared__ __attribute__((aligned(1024))) uint8_t s_mem[S::stages * S::bytes];
    const MoeItem item = FEW ? few_item(g, blockIdx.y, NX) : planned_item(g, blockIdx.y, NX);
    if (item.expert < 0) return;
    const int e = __builtin_amdgcn_readfirstlane(item.expert), np = item.count;
    const auto pair_of = [&](int n) {  // n < np
        if (FEW) return nth_bit(item.few, n);
        const int p = g.plan.order[item.first + n];
        return (uint32_t)p < (uint32_t)g.P ? p : 0;
    };
    const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(wave_id()), c16 = lane & 15, q = lane >> 4;
    const int half = g.R / 2;                               // up: gate's rows
    const int tile = (int)blockIdx.x * (MW / kw) + wave / kw, share = wave % kw;
    const int tiles = UP ? half / 16 : (g.R + MR - 1) / MR;
    const bool live = tile < tiles;
    // first rows of the wave's two tiles of 16 (where there is none, rows that are there)
    const int row0 = live ? (UP ? tile * 16 : tile * MR) : 0;
    const bool two = UP || row0 + 16 < g.R;
    const int row1 = UP ? half + row0 : two ? row0 + 16 : row0;
    const int kb = (g.K + 127) / 128, steps = (g.K + S::cols - 1) / S::cols;
    const uint8_t *const w0 = load_base(g.w + ((int64_t)e * g.R + row0) * g.K);
    const uint8_t *const w1 = load_base(g.w + ((int64_t)e * g.R + row1) * g.K);
    const uint16_t *const xb = load_base(g.x);
    const scalar_floats sw = (scalar_floats)(uint64_t)g.sw + (int64_t)e * ((g.R + 127) / 128) * kb;
    const scalar_floats sw0 = sw + (int64_t)(row0 / 128) * kb, sw1 = sw + (int64_t)(row1 / 128) * kb;

    uint32_t wo[S::w_loads / 2], xo[S::x_loads];
    const auto w_row = [&](int i) { return i * S::w_rows + lane / S::wp; };
    const auto w_piece = [&](int i) { return (lane % S::wp) ^ (w_row(i) % S::wp); };
    const auto x_row = [&](int i) { return ((FEW ? 0 : wave * S::x_loads) + i) * S::x_rows + lane / S::xp; };
    const auto x_piece = [&](int i) { return (lane % S::xp) ^ (x_row(i) % NX % 16); };
#pragma unroll
    for (int i = 0; i < S::w_loads / 2; ++i) wo[i] = (uint32_t)w_row(i) * (uint32_t)g.K;
#pragma unroll
    for (int i = 0; i < S::x_loads; ++i) {
        const int r = x_row(i), c = r % NX, pair = pair_of(c < np ? c : np - 1);
        const uint32_t row = UP ? (uint32_t)(pair / g.top_k) : (uint32_t)(r / NX * g.P + pair);
        xo[i] = row * (uint32_t)g.ldx * 2;
    }
    const uint32_t mem = __builtin_amdgcn_readfirstlane(lds_at(s_mem));
    const uint32_t w_at = wave * S::w_bytes, x_at = MW * S::w_bytes + (FEW ? wave * S::x_bytes : 0);
    // a step's loads; pieces past the end of a row are taken from its beginning (x's are cleared below)
    const auto issue = [&](int s, int turn) {
        const uint32_t at = mem + (uint32_t)(turn % S::stages) * S::bytes, c = (uint32_t)s * S::cols;
        const int left = g.K - s * S::cols;
#pragma unroll
        for (int i = 0; i < S::w_loads; ++i) {
            const int p = w_piece(i % (S::w_loads / 2)) * 16;
            load_lds16_once(at + w_at + i * 1024, i < S::w_loads / 2 ? w0 : w1,
                            wo[i % (S::w_loads / 2)] + c + (p < left ? p : 0));
        }
#pragma unroll
        for (int i = 0; i < S::x_loads; ++i) {
            const int p = x_piece(i) * 8;
            load_lds16(at + x_at + ((FEW ? 0 : wave * S::x_loads) + i) * 1024, xb, xo[i] + (c + (p < left ? p : 0)) * 2);
        }
    };

    f32x4 acc[2][CT];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int c = 0; c < CT; ++c) acc[t][c] = f32x4{0, 0, 0, 0};
    int ahead = share, turns = 0, turn = 0;
    for (int i = 0; i < S::stages - 1; ++i, ahead += kw)
        if (ahead < steps) issue(ahead, turns++);
    for (int s = share; s < steps; s += kw, ++turn) {
        if (turns - turn >= S::stages - 1 && S::stages > 2) wait_loads<(S::stages - 2) * S::loads>();
        else wait_loads<0>();
        if (FEW) asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the last step's reads are done
        else lds_barrier();
        uint8_t *const buf = s_mem + (turn % S::stages) * S::bytes;
        uint8_t *const bx = buf + x_at;
        if (g.K - s * S::cols < S::cols) {  // the ragged end
            const int from = (g.K - s * S::cols) / 8, gone = S::xp - from;
            for (int i = FEW ? lane : (int)threadIdx.x; i < S::parts * NX * gone; i += FEW ? kWave : MW * kWave) {
                const int r = i / gone, p = from + i % gone;
                *reinterpret_cast<u32x4 *>(bx + r * S::cols * 2 + (p ^ (r % NX % 16)) * 16) = u32x4{0, 0, 0, 0};
            }
            if (!FEW) lds_barrier();
        }
        if (ahead < steps) issue(ahead, turns++);
        ahead += kw;
        const uint8_t *const bw = buf + w_at;
#pragma unroll
        for (int b = 0; b < S::cols / 128; ++b) {
            const int at = s * (S::cols / 128) + b < kb ? s * (S::cols / 128) + b : kb - 1;
            const float f0 = sw0[at], f1 = sw1[at];
            f32x4 p[2][CT];
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int c = 0; c < CT; ++c) p[t][c] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int piece = b * 8 + h * 4 + q;
                bf16x8 a[2][2];
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const u32x4 v =
                        *reinterpret_cast<const u32x4 *>(bw + (t * 16 + c16) * S::cols + (piece ^ (c16 % S::wp)) * 16);
                    a[t][0] = widen_codes(v[0], v[1]);
                    a[t][1] = widen_codes(v[2], v[3]);
                }
#pragma unroll
                for (int c = 0; c < CT; ++c)
#pragma unroll
                    for (int part = 0; part < S::parts; ++part) {
                        const int r = c * 16 + c16 % (NX < 16 ? NX : 16);
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const bf16x8 xv = *reinterpret_cast<const bf16x8 *>(
                                bx + (part * NX + r) * S::cols * 2 + ((2 * piece + k) ^ (r % 16)) * 16);
#pragma unroll
                            for (int t = 0; t < 2; ++t)
                                p[t][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[t][k], xv, p[t][c], 0, 0, 0);
                        }
                    }
            }
#pragma unroll
            for (int c = 0; c < CT; ++c)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    acc[0][c][i] = __builtin_fmaf(f0, p[0][c][i], acc[0][c][i]);
                    acc[1][c][i] = __builtin_fmaf(f1, p[1][c][i], acc[1][c][i]);
                }
        }
    }
    if (FEW && kw > 1) {  // the waves' shares, in their order
        __syncthreads();
        f32x4 *const sums = reinterpret_cast<f32x4 *>(s_mem);
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int c = 0; c < CT; ++c) sums[((wave * 2 + t) * CT + c) * kWave + lane] = acc[t][c];
        __syncthreads();
        if (share != 0) return;
        for (int v = 1; v < kw; ++v)
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int c = 0; c < CT; ++c) acc[t][c] += sums[(((wave + v) * 2 + t) * CT + c) * kWave + lane];
    }
    if (!live) return;
#pragma unroll
    for (int c = 0; c < CT; ++c) {
        const int place = c * 16 + c16;
        if (place >= np) continue;
        const int pair = pair_of(place);
        if constexpr (UP) {
            // two BF16 hold 16 bits of h, 2^-8 of what y's rounding leaves; one would be as coarse as y itself, and
            // a third would take down's matrix instructions and x's place in LDS half as often again
            float h[4], rest[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                h[i] = silu(acc[0][c][i]) * acc[1][c][i];
                const float near = __uint_as_float(cast_pair(0.0f, h[i]));
                rest[i] = fabsf(near) < __builtin_inff() ? h[i] - near : 0.0f;
            }
            uint16_t *const out = g.h + (int64_t)pair * half + row0 + q * 4;
            *reinterpret_cast<u32x2 *>(out) = u32x2{cast_pair(h[0], h[1]), cast_pair(h[2], h[3])};
            *reinterpret_cast<u32x2 *>(out + (int64_t)g.P * half) = u32x2{cast_pair(rest[0], rest[1]), cast_pair(rest[2], rest[3])};
        } else {
            float *const out = g.out + (int64_t)pair * g.R + row0 + q * 4;
            *reinterpret_cast<f32x4 *>(out) = acc[0][c];
            if (two) *reinterpret_cast<f32x4 *>(out + 16) = acc[1][c];
        }
    }
}

// One or two tokens: a workgroup makes 16 columns of y whole.  Its waves take the live pairs in
// turn, 16 rows of the pair's down and the two parts of its h as two columns of the matrix
// instruction, a pair's first steps on their way while the last one's end is multiplied.
constexpr int FD_STAGES = 3, FD_WAVES = 4;

__global__ __launch_bounds__(FD_WAVES *kWave) void k_moe_few_down(MoeArgs g, const float *__restrict__ weights, int32_t T,
                                                           uint16_t *__restrict__ y, int64_t ldy) {
    constexpr int MW = FD_WAVES, cols = 256, w_bytes = 16 * cols, bytes = w_bytes + 1024, loads = 5;
    __shared__ __attribute__((aligned(1024))) uint8_t s_mem[MW * FD_STAGES * bytes];
    const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(wave_id()), c16 = lane & 15, q = lane >> 4;
    const int row0 = (int)blockIdx.x * 16, kb = (g.K + 127) / 128, steps = (g.K + cols - 1) / cols;
    const int id = lane < g.P ? g.ids[lane] : -1;
    const float weight = lane < g.P ? weights[lane] : 0.0f;
    const uint64_t pairs = __ballot((uint32_t)id < (uint32_t)g.E);
    const int n = __builtin_popcountll(pairs), mine = n > wave ? (n - wave + MW - 1) / MW : 0;
    const uint8_t *const wb = load_base(g.w);
    const uint16_t *const xb = load_base(g.x);
    uint8_t *const buf = s_mem + wave * FD_STAGES * bytes;
    const uint32_t mem = __builtin_amdgcn_readfirstlane(lds_at(buf));
    uint32_t wo[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) wo[i] = (uint32_t)(i * 4 + (lane >> 4)) * (uint32_t)g.K;
    const int xr = lane >> 5;  // part of h

    // what is to be loaded next: step ls of pair lp (the wave's li-th)
    int li = 0, ls = 0, lp = mine ? nth_bit(pairs, wave) : 0;
    const auto issue = [&](int turn) {
        const uint32_t at = mem + (uint32_t)(turn % FD_STAGES) * bytes;
        const int e = __builtin_amdgcn_readlane(id, lp), left = g.K - ls * cols;
        const uint8_t *const base = load_base(wb + ((int64_t)e * g.R + row0) * g.K + ls * cols);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int p = (c16 ^ (i * 4 + (lane >> 4))) * 16;
            load_lds16_once(at + i * 1024, base, wo[i] + (p < left ? p : 0));
        }
        const int p = ((lane & 31) ^ xr) * 8;
        load_lds16(at + w_bytes, xb, ((uint32_t)(xr * g.P + lp) * (uint32_t)g.K + ls * cols + (p < left ? p : 0)) * 2);
        if (++ls == steps) {
            ls = 0;
            if (++li < mine) lp = nth_bit(pairs, wave + li * MW);
        }
    };
    const int total = mine * steps;
    int turns = 0;
    while (turns < FD_STAGES - 1 && turns < total) issue(turns), ++turns;
    f32x4 sum[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};  // of token 0 and 1
    int turn = 0;
    for (int i = 0; i < mine; ++i) {
        const int pair = nth_bit(pairs, wave + i * MW), e = __builtin_amdgcn_readlane(id, pair);
        const scalar_floats sw =
            (scalar_floats)(uint64_t)g.sw + ((int64_t)e * ((g.R + 127) / 128) + row0 / 128) * kb;
        f32x4 acc = {0, 0, 0, 0};
        for (int s = 0; s < steps; ++s, ++turn) {
            if (turns < total) {
                asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the last step's reads are done: its buffer is free
                issue(turns), ++turns;
                wait_loads<(FD_STAGES - 1) * loads>();
            } else {
                wait_loads<0>();
            }
            uint8_t *const at = buf + (turn % FD_STAGES) * bytes, *const bx = at + w_bytes;
            if (g.K - s * cols < cols) {
                const int from = (g.K - s * cols) / 8, gone = 32 - from;
                for (int k = lane; k < 2 * gone; k += kWave) {
                    const int r = k / gone, p = from + k % gone;
                    *reinterpret_cast<u32x4 *>(bx + r * 512 + (p ^ r) * 16) = u32x4{0, 0, 0, 0};
                }
            }
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                f32x4 p = {0, 0, 0, 0};
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int piece = b * 8 + h * 4 + q, r = c16 & 1;
                    const u32x4 v = *reinterpret_cast<const u32x4 *>(at + c16 * cols + (piece ^ c16) * 16);
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const bf16x8 xv = *reinterpret_cast<const bf16x8 *>(bx + r * 512 + ((2 * piece + k) ^ r) * 16);
                        p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen_codes(v[2 * k], v[2 * k + 1]), xv, p, 0, 0, 0);
                    }
                }
                const float f = sw[2 * s + b < kb ? 2 * s + b : kb - 1];
#pragma unroll
                for (int k = 0; k < 4; ++k) acc[k] = __builtin_fmaf(f, p[k], acc[k]);
            }
        }
        const float share = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(weight), pair));
        const int t = pair / g.top_k;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            // (columns 0 and 1 are the products of h's parts)
            const float both = acc[k] + __shfl_xor(acc[k], 1, kWave);
            if (t == 0) sum[0][k] = __builtin_fmaf(share, both, sum[0][k]);
            else sum[1][k] = __builtin_fmaf(share, both, sum[1][k]);
        }
    }
    __syncthreads();
    f32x4 *const sums = reinterpret_cast<f32x4 *>(s_mem);
    if (c16 == 0)
#pragma unroll
        for (int t = 0; t < 2; ++t) sums[(wave * 2 + t) * 4 + q] = sum[t];
    __syncthreads();
    if (threadIdx.x >= 8) return;
    const int t = threadIdx.x >> 2, quarter = threadIdx.x & 3;
    if (t >= T) return;
    f32x4 v = sums[t * 4 + quarter];
    for (int w = 1; w < MW; ++w) v += sums[(w * 2 + t) * 4 + quarter];
    *reinterpret_cast<u32x2 *>(y + (int64_t)t * ldy + row0 + quarter * 4) = u32x2{cast_pair(v[0], v[1]), cast_pair(v[2], v[3])};
}

// y = the sum over a token's choices, in their order: a thread takes four columns
__global__ __launch_bounds__(256) void k_moe_join(const float *__restrict__ parts, const int32_t *__restrict__ ids,
                                                  const float *__restrict__ weights, int32_t T, int32_t top_k, int32_t E,
                                                  int32_t H, uint16_t *__restrict__ y, int64_t ldy) {
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (i >= (int64_t)T * H) return;
    const int t = (int)(i / H), c = (int)(i - (int64_t)t * H);
    f32x4 v = {0, 0, 0, 0};
    for (int j = 0; j < top_k; ++j) {
        const int pair = t * top_k + j;
        if ((uint32_t)ids[pair] >= (uint32_t)E) continue;
        const f32x4 part = *reinterpret_cast<const f32x4 *>(parts + (int64_t)pair * H + c);
        const float p = weights[pair];
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = __builtin_fmaf(p, part[k], v[k]);
    }
    *reinterpret_cast<u32x2 *>(y + (int64_t)t * ldy + c) = u32x2{cast_pair(v[0], v[1]), cast_pair(v[2], v[3])};
}

// The workspace's parts, each on a boundary of 256 bytes.
struct MoeWs {
    int64_t plan, order, h, out, total;
};

inline MoeWs moe_ws(int64_t P, int64_t H, int64_t I) {
    const auto up = [](int64_t n) { return (n + 255) / 256 * 256; };
    MoeWs w;
    w.plan = 0;
    w.order = up((2 * (P + 1) + 1) * 4);  // items are at most as many as pairs
    w.h = w.order + up(P * 4);
    w.out = w.h + up(2 * P * I * 2);
    w.total = w.out + up(P * H * 4);
    return w;
}

// Pairs of an item, by an expert's average: more of them, and most experts are read once; fewer,
// and less of LDS and of the columns is empty.  Microseconds with items of 8, 16, 32 and 64:
// 1.9 an expert (30 tokens, top 4 of 64 x (4096, 2048)) 248, 249, 257, 336; 4 an expert (61, 4 of 60 x
// (2048, 1408)) 97, 94, 97, 125; 8 an expert (64, 4 of 32 x (4096, 2048)) 183, 165, 165, 201; 16 an
// expert (128 tokens) 249, 199, 171, 205; 32 an expert (128, 4 of 16) 202, 148, 126, 114; 64 an expert
// (256 tokens) 338, 228, 177, 169.
inline int moe_nx(int64_t P, int64_t E) { return P <= 2 * E ? 8 : P <= 10 * E ? 16 : P <= 20 * E ? 32 : 64; }

// One or two tokens, whose choices fit a wave, and two launches instead of four: one token, 8 of 384 experts
// x (7168, 2048) 63.7 and 76.8 us, 4 of 60 x (2048, 1408) 17.4 and 30.1; two tokens 116 and 121, 24.1 and 31.9.
inline bool moe_few(int64_t T, int64_t P) { return T <= 2 && P <= kWave; }

template <bool UP, int NX, bool FEW>
inline void launch_rows(const MoeArgs &g, unsigned items, hipStream_t stream) {
    using S = MoeStage<UP, NX, FEW>;
    constexpr int waves = S::MW, per = waves / S::kw;
    const unsigned tiles = (unsigned)(UP ? g.R / 2 / 16 : (g.R + MR - 1) / MR);
    k_moe_rows<UP, NX, FEW><<<dim3((tiles + per - 1) / per, items), dim3(waves * kWave), 0, stream>>>(g);
}

template <int NX>
inline void launch_both(const MoeArgs &u, const MoeArgs &d, unsigned items, hipStream_t stream) {
    launch_rows<true, NX, false>(u, items, stream);
    launch_rows<false, NX, false>(d, items, stream);
}

}  // namespace pulse

using namespace pulse;

extern "C" {

int64_t pulse_moe_ws_size(int64_t T, int64_t H, int64_t I, int64_t top_k) { return moe_ws(T * top_k, H, I).total; }

int pulse_launch_moe_route(const float *logits, int64_t ld, int64_t T, int64_t E, int32_t top_k, int32_t over_all,
                           float scale, int32_t *ids, float *weights, hipStream_t stream) {
    const dim3 grid((unsigned)((T + 3) / 4)), block(256);
    with_logits(E, [&](auto per) {
        k_moe_route<decltype(per)::value>
            <<<grid, block, 0, stream>>>(logits, ld, (int32_t)T, (int32_t)E, top_k, over_all, scale, ids, weights);
    });
    return hipGetLastError() == hipSuccess ? 0 : -5;
}

int pulse_launch_moe_forward(const uint16_t *x, int64_t ldx, const int32_t *ids, const float *weights,
                             const uint8_t *up, const float *up_scales, const uint8_t *down, const float *down_scales,
                             int64_t T, int64_t H, int64_t I, int64_t E, int64_t top_k, uint16_t *y, int64_t ldy,
                             uint32_t *status, void *ws, hipStream_t stream) {
    const int64_t P = T * top_k;
    const MoeWs at = moe_ws(P, H, I);
    char *const mem = static_cast<char *>(ws);
    int32_t *const words = reinterpret_cast<int32_t *>(mem);
    const MoePlan plan{words, words + 1, words + 1 + P, reinterpret_cast<int32_t *>(mem + at.order)};
    uint16_t *const h = reinterpret_cast<uint16_t *>(mem + at.h);
    float *const out = reinterpret_cast<float *>(mem + at.out);
    const MoeArgs u{x, ldx, up, up_scales, h, nullptr, ids, plan, (int32_t)P, (int32_t)E, (int32_t)(2 * I), (int32_t)H,
              (int32_t)top_k, status};
    const MoeArgs d{h, I, down, down_scales, nullptr, out, ids, plan, (int32_t)P, (int32_t)E, (int32_t)H, (int32_t)I,
              (int32_t)top_k, status};
    if (moe_few(T, P)) {
        launch_rows<true, 2, true>(u, (unsigned)P, stream);
        k_moe_few_down<<<dim3((unsigned)(H / 16)), dim3(FD_WAVES * kWave), 0, stream>>>(d, weights, (int32_t)T, y, ldy);
        return hipGetLastError() == hipSuccess ? 0 : -5;
    }
    const int nx = moe_nx(P, E);
    const unsigned items = (unsigned)std::min<int64_t>(P, E + P / nx);
    k_moe_plan<<<dim3(1), dim3(1024), 0, stream>>>(ids, (int32_t)P, (int32_t)E, nx, plan, status);
    switch (nx) {
    case 8: launch_both<8>(u, d, items, stream); break;
    case 16: launch_both<16>(u, d, items, stream); break;
    case 32: launch_both<32>(u, d, items, stream); break;
    default: launch_both<64>(u, d, items, stream); break;
    }
    k_moe_join<<<dim3((unsigned)((T * H / 4 + 255) / 256)), dim3(256), 0, stream>>>(out, ids, weights, (int32_t)T,
                                                                                    (int32_t)top_k, (int32_t)E,
                                                                                    (int32_t)H, y, ldy);
    return hipGetLastError() == hipSuccess ? 0 : -5;
}
}
