// moe.hip -- a mixture-of-experts layer for a few tokens, and the router's choice.
//
// The choice, for a token's logits over E experts: the top_k largest (equal ones by the
// lowest index), weights = their softmax (over the chosen, or over all experts).
// The layer, with [gate; up] and down of every expert in E4M3 codes and 128 x 128 blocks:
//   h = silu(Wg_e x) * (Wu_e x),   y = sum over the token's experts of p_e Wd_e h
// A few tokens reach many experts, so the work is to read each of these experts' codes
// once, at HBM's rate: 2 bytes of matrix work for a byte read.  Codes go past the
// registers into LDS, rows of 256 bytes at a time, from where a wave takes them as
// rows of the matrix instruction, turned into BF16 (exactly: E4M3 has four bits), with
// up to 16 tokens as its columns.
#include "e4m3.hpp"
#include "lds_load.hpp"

#include <algorithm>

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
    float most = 0, sum = 0;
    int mine = -1;      // lane j: the j-th choice and its logit
    float chosen = 0;
    for (int j = 0; j < top_k; ++j) {
        uint32_t best = 0;
        int at = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (key[i] > best) best = key[i], at = i;
        const uint32_t top = wave_reduce_max(best);
        // of the lanes that hold it, the lowest index: the lowest place first, then the lowest lane
        const uint32_t tie = best == top ? (uint32_t)(at * kWave + lane) : 0xFFFFFFFFu;
        const uint32_t e = ~wave_reduce_max(~tie);
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
    MoePlan plan;
    int32_t P, E, R, K;  // R: rows of w (up: 2 I)
    int32_t top_k;
    int32_t kw;          // waves that share the contraction: 1, 2 or 4
};

constexpr int MW = 4;          // waves of a workgroup
constexpr int MR = 32;         // rows of a wave: 16 of gate and of up, or 32 of down
constexpr int MS = 256;        // columns of a step

__device__ __forceinline__ bf16x8 widen_codes(uint32_t lo, uint32_t hi) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
    const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
    return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// A step's buffer in LDS: the rows of codes of every wave, and NX rows of x (down: twice,
// h's two parts) for all of them (SHARED) or for each.  Piece p (16 bytes) of row r lies at
// p ^ (r & 15), where neither the loads, which fill whole rows, nor the reads, 16 rows at
// one piece, have two lanes in a bank.
template <bool UP, int NX, bool SHARED>
struct MoeStage {
    static constexpr int parts = UP ? 1 : 2;
    static constexpr int w_bytes = MR * MS, x_bytes = parts * NX * MS * 2;
    static constexpr int x_copies = SHARED ? 1 : MW;
    static constexpr int bytes = MW * w_bytes + x_copies * x_bytes;
    static constexpr int w_loads = w_bytes / 1024, x_loads = x_bytes / 1024 / (SHARED ? MW : 1);
    static constexpr int loads = w_loads + x_loads;
    static constexpr int stages = 3 * bytes <= 160 * 1024 && SHARED ? 3 : 2;
    static_assert(x_loads * 1024 * (SHARED ? MW : 1) == x_bytes && stages * bytes <= 160 * 1024, "LDS of a compute unit");
    static_assert((stages - 2) * loads <= 63, "loads in flight");
};

template <bool UP, int NX, bool SHARED>
__global__ __launch_bounds__(MW *kWave) void k_moe_rows(MoeArgs g) {
    using S = MoeStage<UP, NX, SHARED>;
    constexpr int CT = (NX + 15) / 16;  // tiles of tokens
    __shared__ __attribute__((aligned(1024))) uint8_t s_mem[S::stages * S::bytes];
    const int item = blockIdx.y;
    if (item >= g.plan.count[0]) return;
    const int e = g.plan.expert[item], p0 = g.plan.first[item];
    int np = g.plan.first[item + 1] - p0;
    // (whatever the plan's buffer holds, nothing outside the tensors is touched)
    if ((uint32_t)e >= (uint32_t)g.E || (uint32_t)p0 >= (uint32_t)g.P || np <= 0) return;
    np = np < NX ? np : NX;
    np = np < g.P - p0 ? np : g.P - p0;
    const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(wave_id()), c16 = lane & 15, q = lane >> 4;
    const int kw = SHARED ? 1 : g.kw;
    const int half = g.R / 2;                               // up: gate's rows
    const int tile = (int)blockIdx.x * (MW / kw) + wave / kw, share = wave % kw;
    const int tiles = UP ? half / 16 : (g.R + MR - 1) / MR;
    const bool live = tile < tiles;
    // first rows of the wave's two tiles of 16 (where there is none, rows that are there)
    const int row0 = live ? (UP ? tile * 16 : tile * MR) : 0;
    const bool two = UP || row0 + 16 < g.R;
    const int row1 = UP ? half + row0 : two ? row0 + 16 : row0;
    const int kb = (g.K + 127) / 128, steps = (g.K + MS - 1) / MS;
    const uint8_t *w0 = load_base(g.w + ((int64_t)e * g.R + row0) * g.K + share * MS);
    const uint8_t *w1 = load_base(g.w + ((int64_t)e * g.R + row1) * g.K + share * MS);
    const uint16_t *xb = load_base(g.x + share * MS);
    const float *const sw = g.sw + (int64_t)e * ((g.R + 127) / 128) * kb;
    const float *const sw0 = sw + (int64_t)(row0 / 128) * kb, *const sw1 = sw + (int64_t)(row1 / 128) * kb;

    uint32_t wo[S::w_loads / 2], xo[S::x_loads];
#pragma unroll
    for (int i = 0; i < S::w_loads / 2; ++i) {
        const int r = i * 4 + (lane >> 4);
        wo[i] = (uint32_t)r * (uint32_t)g.K + (uint32_t)(c16 ^ r) * 16;
    }
    const auto x_row = [&](int i) { return ((SHARED ? wave * S::x_loads : 0) + i) * 2 + (lane >> 5); };
#pragma unroll
    for (int i = 0; i < S::x_loads; ++i) {
        const int r = x_row(i), c = r % NX;
        int pair = g.plan.order[p0 + (c < np ? c : np - 1)];
        if ((uint32_t)pair >= (uint32_t)g.P) pair = 0;
        const uint32_t row = UP ? (uint32_t)(pair / g.top_k) : (uint32_t)(r / NX * g.P + pair);
        xo[i] = row * (uint32_t)g.ldx * 2 + (uint32_t)((lane & 31) ^ (c & 15)) * 16;
    }
    const uint32_t mem = __builtin_amdgcn_readfirstlane(lds_at(s_mem));
    const uint32_t w_at = wave * S::w_bytes, x_at = MW * S::w_bytes + (SHARED ? 0 : wave * S::x_bytes);
    // a step's loads; pieces past the end of a row are taken from its beginning (x's are cleared below)
    const auto issue = [&](int s, int turn) {
        const uint32_t at = mem + (uint32_t)(turn % S::stages) * S::bytes;
        const int left = g.K - s * MS;
#pragma unroll
        for (int i = 0; i < S::w_loads; ++i) {
            uint32_t o = wo[i % (S::w_loads / 2)];
            if (left < MS) {
                const int p = c16 ^ (i % (S::w_loads / 2) * 4 + (lane >> 4));
                if (p * 16 >= left) o -= p * 16;
            }
            load_lds16_once(at + w_at + i * 1024, i < S::w_loads / 2 ? w0 : w1, o);
        }
#pragma unroll
        for (int i = 0; i < S::x_loads; ++i) {
            uint32_t o = xo[i];
            if (left < MS) {
                const int p = (lane & 31) ^ (x_row(i) % NX & 15);
                if (p * 8 >= left) o -= p * 16;
            }
            load_lds16(at + x_at + ((SHARED ? wave * S::x_loads : 0) + i) * 1024, xb, o);
        }
        w0 += kw * MS;
        w1 += kw * MS;
        xb += kw * MS;
    };

    f32x4 acc[2][CT];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int c = 0; c < CT; ++c) acc[t][c] = f32x4{0, 0, 0, 0};
    int ahead = share, turns = 0;
    for (int i = 0; i < S::stages - 1; ++i, ahead += kw)
        if (ahead < steps) issue(ahead, turns++);
    int turn = 0;
    for (int s = share; s < steps; s += kw, ++turn) {
        if (turns - turn >= S::stages - 1 && S::stages > 2) wait_loads<(S::stages - 2) * S::loads>();
        else wait_loads<0>();
        if (SHARED) lds_barrier();
        else asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the last step's reads are done
        uint8_t *const buf = s_mem + (turn % S::stages) * S::bytes;
        uint8_t *const bx = buf + x_at;
        if (g.K - s * MS < MS) {  // the ragged end
            const int from = (g.K - s * MS) / 8, gone = MS / 8 - from;
            for (int i = SHARED ? (int)threadIdx.x : lane; i < S::parts * NX * gone; i += SHARED ? MW * kWave : kWave) {
                const int r = i / gone, p = from + i % gone;
                *reinterpret_cast<u32x4 *>(bx + r * MS * 2 + (p ^ (r % NX & 15)) * 16) = u32x4{0, 0, 0, 0};
            }
            if (SHARED) lds_barrier();
        }
        if (ahead < steps) issue(ahead, turns++);
        ahead += kw;
        const uint8_t *const bw = buf + w_at;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
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
                    const u32x4 v = *reinterpret_cast<const u32x4 *>(bw + (t * 16 + c16) * MS + (piece ^ c16) * 16);
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
                                bx + (part * NX + r) * MS * 2 + ((2 * piece + k) ^ (r & 15)) * 16);
#pragma unroll
                            for (int t = 0; t < 2; ++t)
                                p[t][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[t][k], xv, p[t][c], 0, 0, 0);
                        }
                    }
            }
            const int at = 2 * s + b < kb ? 2 * s + b : kb - 1;
            const float f0 = sw0[at], f1 = sw1[at];
#pragma unroll
            for (int c = 0; c < CT; ++c)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    acc[0][c][i] = __builtin_fmaf(f0, p[0][c][i], acc[0][c][i]);
                    acc[1][c][i] = __builtin_fmaf(f1, p[1][c][i], acc[1][c][i]);
                }
        }
    }
    if (!SHARED && kw > 1) {  // the waves' shares, in their order
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
        const int pair = g.plan.order[p0 + place];
        if ((uint32_t)pair >= (uint32_t)g.P) continue;
        if constexpr (UP) {
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

// Pairs of an item
inline int moe_nx(int64_t T, int64_t P, int64_t E) {
    if (T <= 2) return 2;
    return P > 16 * E ? 32 : 16;
}

}  // namespace pulse

using namespace pulse;

extern "C" {

int64_t pulse_moe_ws_size(int64_t T, int64_t H, int64_t I, int64_t top_k) { return moe_ws(T * top_k, H, I).total; }

int pulse_launch_moe_route(const float *logits, int64_t ld, int64_t T, int64_t E, int32_t top_k, int32_t over_all,
                           float scale, int32_t *ids, float *weights, hipStream_t stream) {
    const dim3 grid((unsigned)((T + 3) / 4)), block(256);
    if (E <= 128) k_moe_route<2><<<grid, block, 0, stream>>>(logits, ld, (int32_t)T, (int32_t)E, top_k, over_all, scale, ids, weights);
    else if (E <= 384) k_moe_route<6><<<grid, block, 0, stream>>>(logits, ld, (int32_t)T, (int32_t)E, top_k, over_all, scale, ids, weights);
    else k_moe_route<16><<<grid, block, 0, stream>>>(logits, ld, (int32_t)T, (int32_t)E, top_k, over_all, scale, ids, weights);
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
    const int nx = moe_nx(T, P, E);
    const int64_t items = std::min<int64_t>(P, E + P / nx);
    k_moe_plan<<<dim3(1), dim3(1024), 0, stream>>>(ids, (int32_t)P, (int32_t)E, nx, plan, status);
    uint16_t *const h = reinterpret_cast<uint16_t *>(mem + at.h);
    float *const out = reinterpret_cast<float *>(mem + at.out);
    MoeArgs u{x, ldx, up, up_scales, h, nullptr, plan, (int32_t)P, (int32_t)E, (int32_t)(2 * I), (int32_t)H,
              (int32_t)top_k, 1};
    MoeArgs d{h, I, down, down_scales, nullptr, out, plan, (int32_t)P, (int32_t)E, (int32_t)H, (int32_t)I,
              (int32_t)top_k, 1};
    if (nx == 2) {
        u.kw = H >= 4096 ? 4 : 1;
        d.kw = I >= 4096 ? 4 : 1;
    }
    const auto grid = [&](int64_t tiles, int kw) {
        const int64_t per = MW / kw;
        return dim3((unsigned)((tiles + per - 1) / per), (unsigned)items);
    };
    const dim3 gu = grid(I / 16, u.kw), gd = grid((H + MR - 1) / MR, d.kw), block(MW * kWave);
    if (nx == 2) {
        k_moe_rows<true, 2, false><<<gu, block, 0, stream>>>(u);
        k_moe_rows<false, 2, false><<<gd, block, 0, stream>>>(d);
    } else if (nx == 16) {
        k_moe_rows<true, 16, true><<<gu, block, 0, stream>>>(u);
        k_moe_rows<false, 16, true><<<gd, block, 0, stream>>>(d);
    } else {
        k_moe_rows<true, 32, true><<<gu, block, 0, stream>>>(u);
        k_moe_rows<false, 32, true><<<gd, block, 0, stream>>>(d);
    }
    k_moe_join<<<dim3((unsigned)((T * H / 4 + 255) / 256)), dim3(256), 0, stream>>>(out, ids, weights, (int32_t)T,
                                                                                    (int32_t)top_k, (int32_t)E,
                                                                                    (int32_t)H, y, ldy);
    return hipGetLastError() == hipSuccess ? 0 : -5;
}
}
