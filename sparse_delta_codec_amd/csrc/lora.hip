// lora.hip -- low-rank adapters of many requests beside a shared projection,
// forward and backward.
//
// The mathematics, for a token with row x, output row y and adapter i of rank R
// (A_i [R, K], B_i [R, N], both stored with the long axis contiguous):
//   h  = s_i A_i x            y  += B_i^T h
//   dh = s_i B_i dy           dx += A_i^T dh
//   dA_i = sum over i's tokens of dh x^T        dB_i = sum of h dy^T
// so three kernels serve both directions, because A and B have one layout:
//   shrink  [tokens, C] by [R, C]   -> [tokens, R]   contracted over the long axis
//   expand  [tokens, R] by [R, C]   -> added to [tokens, C]
//   outer   [tokens, R] by [tokens, C] -> [R, C]     contracted over tokens
// All of them are bound by reading or writing the [tokens, C] matrices (an
// element takes 2 R multiplications for 2 to 4 bytes), so the work is to touch
// those once, with wide loads, and to keep the matrix instructions fed from
// registers: the two operands that a matrix instruction wants along the other
// axis (expand's adapter, outer's tokens) are transposed in registers, one
// v_perm_b32 per pair of values, without a trip through LDS.
//
// A plan groups a batch's tokens by adapter: tiles of 64 places, each of one
// adapter, whose places hold token numbers in ascending order (-1: empty).
// Every kernel works on tiles, so a token is found by its place and sums over
// tokens have one order whatever the launch.
#include "device.hpp"

namespace pulse {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x4 __attribute__((ext_vector_type(4)));

constexpr int LT = 64;            // places of a tile
constexpr int LP_THREADS = 512;   // the plan's workgroup, two adapters a thread
constexpr int LP_WAVES = LP_THREADS / kWave;

// The plan's parts for T tokens and S adapters (32-bit words in one buffer).
struct LoraPlan {
    int32_t *ntiles;      // [16] tiles in use, then padding
    int32_t *tile_slot;   // [max_tiles] adapter of a tile, -1: unused
    int32_t *tile_count;  // [max_tiles] tokens of a tile
    int32_t *slot_tile;   // [S + 1] first tile of an adapter
    int32_t *order;       // [max_tiles * 64] token of a place, -1: empty
};

__host__ __device__ inline int64_t lora_max_tiles(int64_t T, int64_t S) {
    const int64_t t = (T + LT - 1) / LT + S;
    return T < t ? T : t;
}

__host__ __device__ inline int64_t lora_round4(int64_t n) { return (n + 3) / 4 * 4; }

__host__ __device__ inline LoraPlan lora_plan_parts(void *plan, int64_t T, int64_t S) {
    const int64_t mt = lora_max_tiles(T, S);
    LoraPlan p;
    p.ntiles = static_cast<int32_t *>(plan);
    p.tile_slot = p.ntiles + 16;
    p.tile_count = p.tile_slot + lora_round4(mt);
    p.slot_tile = p.tile_count + lora_round4(mt);
    p.order = p.slot_tile + lora_round4(S + 1);
    return p;
}

inline int64_t lora_plan_size(int64_t T, int64_t S) {
    const int64_t mt = lora_max_tiles(T, S);
    return 4 * (16 + 2 * lora_round4(mt) + lora_round4(S + 1) + mt * LT);
}

// ---- the plan: a stable counting sort by adapter -----------------------------
// One workgroup.  Wave w owns the tokens [w T/8, (w+1) T/8) and counts them
// per adapter in its own row of an LDS table; the rows' prefix sums give each
// wave its first place for every adapter; then every wave deals its tokens out
// in order, 64 at a time, ranking equal adapters with ballots.
__global__ __launch_bounds__(LP_THREADS) void k_lora_plan(const int32_t *__restrict__ ids, int32_t T, int32_t S,
                                                          LoraPlan p, int32_t max_tiles, uint32_t *d_status) {
    extern __shared__ int32_t sh[];  // [8][S] counts, then first places
    __shared__ int32_t s_scan[LP_WAVES];
    const int tid = threadIdx.x, w = wave_id(), l = lane_id();
    for (int i = tid; i < LP_WAVES * S; i += LP_THREADS) sh[i] = 0;
    __syncthreads();
    const int per = ((T + LP_WAVES - 1) / LP_WAVES + kWave - 1) / kWave * kWave;
    const int t0 = w * per, t1 = t0 + per < T ? t0 + per : T;
    bool bad = false;
    for (int t = t0 + l; t < t1; t += kWave) {
        const int id = ids[t];
        if (id >= 0 && id < S) atomicAdd(&sh[w * S + id], 1);
        else if (id != -1) bad = true;
    }
    if (__ballot(bad) && l == 0) or_agent32(d_status, 2u /*PULSE_DS_BADINDEX*/);
    __syncthreads();
    // adapters 2 tid and 2 tid + 1: their counts, their tiles, every wave's first place
    int cnt[2] = {0, 0}, tiles[2], total;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int a = 2 * tid + k;
        if (a < S) {
#pragma unroll
            for (int i = 0; i < LP_WAVES; ++i) {
                const int c = sh[i * S + a];
                sh[i * S + a] = cnt[k];
                cnt[k] += c;
            }
        }
        tiles[k] = (cnt[k] + LT - 1) / LT;
    }
    int first = block_excl_sum<LP_WAVES>(tiles[0] + tiles[1], s_scan, &total);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int a = 2 * tid + k;
        if (a < S) {
#pragma unroll
            for (int i = 0; i < LP_WAVES; ++i) sh[i * S + a] += first * LT;
            p.slot_tile[a] = first;
            for (int i = 0; i < tiles[k]; ++i) {
                p.tile_slot[first + i] = a;
                p.tile_count[first + i] = cnt[k] - i * LT < LT ? cnt[k] - i * LT : LT;
            }
            for (int i = cnt[k]; i < tiles[k] * LT; ++i) p.order[first * LT + i] = -1;
        }
        first += tiles[k];
    }
    if (tid == 0) {
        p.slot_tile[S] = total;
        *p.ntiles = total;
    }
    for (int i = total + tid; i < max_tiles; i += LP_THREADS) p.tile_slot[i] = -1;
    __syncthreads();
    volatile int32_t *mine = sh + w * S;
    for (int tb = t0; tb < t1; tb += kWave) {
        const int t = tb + l;
        int id = t < t1 ? ids[t] : -1;
        if (id < 0 || id >= S) id = -1;
        uint64_t same = __ballot(id >= 0);
        for (int b = 1; b < S; b <<= 1) {
            const uint64_t m = __ballot(id & b);
            same &= (id & b) ? m : ~m;
        }
        if (id >= 0) {
            const uint32_t rank = lanes_below(same);
            const int place = mine[id] + (int)rank;
            p.order[place] = t;
            // the last of the equal lanes moves the adapter's next place on (all have read it:
            // a wave's LDS accesses are in order)
            if ((same >> l) == 1ull) mine[id] = place + 1;
        }
        __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
    }
}

// ---- what the kernels share -----------------------------------------------------
// h (or dh) of every place, in the three forms its readers want: BF16
// [place][Rp] for expand; for outer, whose sums over tokens go out in float32,
// the float32 value as the sum of two BF16 (16 bits of mantissa), each [Rp][place].
struct LoraHidden {
    uint16_t *rows;
    uint16_t *hi;
    uint16_t *lo;
};

inline int64_t lora_hidden_size(int64_t T, int64_t S, int64_t R, bool train) {
    const int64_t rp = (R + 15) / 16 * 16, places = lora_max_tiles(T, S) * LT;
    return places * rp * 2 * (train ? 3 : 1);
}

inline LoraHidden lora_hidden_parts(void *h, int64_t T, int64_t S, int64_t R, bool train) {
    const int64_t rp = (R + 15) / 16 * 16, places = lora_max_tiles(T, S) * LT;
    LoraHidden p;
    p.rows = static_cast<uint16_t *>(h);
    p.hi = train ? p.rows + places * rp : nullptr;
    p.lo = train ? p.hi + places * rp : nullptr;
    return p;
}

// A place's token.  Whatever a plan's buffer holds, no kernel leaves its tensors:
// tokens, adapters, counts and chunks out of range are taken as empty or cut off.
__device__ __forceinline__ int token_of(int t, int T) { return (uint32_t)t < (uint32_t)T ? t : -1; }

__device__ __forceinline__ u32x4 ld16(const uint16_t *p) { return *reinterpret_cast<const u32x4 *>(p); }

__device__ __forceinline__ bf16x8 as_bf(const u32x4 &v) { return __builtin_bit_cast(bf16x8, v); }

// h's four values of ranks r .. r+3 at one place, in its three forms
__device__ __forceinline__ void store_hidden(const LoraHidden &h, int64_t place, int64_t places, int rp, int r,
                                             const f32x4 &v) {
    const uint32_t p0 = cast_pair(v[0], v[1]), p1 = cast_pair(v[2], v[3]);
    *reinterpret_cast<u32x2 *>(h.rows + place * rp + r) = u32x2{p0, p1};
    if (h.hi) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t top = (i < 2 ? p0 : p1) >> (16 * (i & 1)) & 0xFFFFu;
            const float rest = v[i] - __uint_as_float(top << 16);
            h.hi[(r + i) * places + place] = (uint16_t)top;
            h.lo[(r + i) * places + place] = (uint16_t)cast_pair(rest, 0.0f);
        }
    }
}

// ---- shrink: h = s A x ----------------------------------------------------------
struct ShrinkArgs {
    const uint16_t *x;
    int64_t ldx;
    const uint16_t *a;
    const float *scales;
    LoraPlan plan;
    LoraHidden h;
    float *partial;     // [ksplit][places][Rp] (ksplit > 1)
    uint32_t *done;     // [tiles * 4] (ksplit > 1) workgroups finished; the last one sets it back to zero
    int64_t places;
    int32_t T, S, C, R, ksplit;
};

// A workgroup takes 16 places of a tile; its four waves, and ksplit workgroups,
// share the long axis.  Matrix instruction: rows = ranks, columns = places, 32
// elements of the long axis, so both operands are 16-byte pieces of rows.
template <int RT>
__global__ __launch_bounds__(256) void k_lora_shrink(ShrinkArgs g) {
    __shared__ f32x4 s_acc[3][RT][kWave];
    __shared__ uint32_t s_last;
    const int tile = blockIdx.x >> 2, sub = blockIdx.x & 3;
    const int slot = g.plan.tile_slot[tile];
    if ((uint32_t)slot >= (uint32_t)g.S || sub * 16 >= g.plan.tile_count[tile]) return;
    const int w = __builtin_amdgcn_readfirstlane(wave_id()), l = lane_id(), c16 = l & 15, q = l >> 4;
    const int64_t place = (int64_t)tile * LT + sub * 16 + c16;
    const int tok = token_of(g.plan.order[place], g.T);
    const uint16_t *px = g.x + (int64_t)(tok < 0 ? 0 : tok) * g.ldx + q * 8;
    const uint16_t *pa = g.a + ((int64_t)slot * g.R + c16) * g.C + q * 8;
    const int steps = (g.C + 31) / 32, parts = g.ksplit * 4;
    const int part = blockIdx.y * 4 + w;
    const int per = (steps + parts - 1) / parts;
    const int k0 = part * per * 32, k1 = (part + 1) * per * 32 < g.C ? (part + 1) * per * 32 : g.C;
    f32x4 acc[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) acc[rt] = f32x4{0, 0, 0, 0};
#pragma unroll 4
    for (int k = k0; k < k1; k += 32) {
        const bool in = k + q * 8 < g.C;
        u32x4 xv = {0, 0, 0, 0};
        if (in && tok >= 0) xv = ld16(px + k);
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            u32x4 av = {0, 0, 0, 0};
            if (in && rt * 16 + c16 < g.R) av = ld16(pa + (int64_t)rt * 16 * g.C + k);
            acc[rt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf(av), as_bf(xv), acc[rt], 0, 0, 0);
        }
    }
    if (w > 0) {
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) s_acc[w - 1][rt][l] = acc[rt];
    }
    __syncthreads();
    const int rp = RT * 16;
    const float scale = g.scales[slot];
    if (w == 0) {
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            f32x4 v = acc[rt];
#pragma unroll
            for (int i = 0; i < 3; ++i) v += s_acc[i][rt][l];
            if (g.ksplit == 1) {
                store_hidden(g.h, place, g.places, rp, rt * 16 + q * 4, v * scale);
            } else {
                float *o = g.partial + ((int64_t)blockIdx.y * g.places + place) * rp + rt * 16 + q * 4;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    __hip_atomic_store(o + i, v[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            }
        }
        if (g.ksplit > 1) {
            // the partial sums were written through to memory; they have arrived before the count goes up
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            if (l == 0) s_last = add_agent32(&g.done[blockIdx.x], 1u) == (uint32_t)g.ksplit - 1;
        }
    }
    if (g.ksplit == 1) return;
    __syncthreads();
    if (!s_last) return;
    // the last workgroup of the 16 places adds the parts in their order
    for (int i = threadIdx.x; i < 16 * RT * 4; i += 256) {
        const int64_t pl = (int64_t)tile * LT + sub * 16 + (i & 15);
        const int r = (i >> 4) * 4;
        f32x4 v = {0, 0, 0, 0};
        for (int s = 0; s < g.ksplit; ++s) {
            const float *o = g.partial + ((int64_t)s * g.places + pl) * rp + r;
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] += __hip_atomic_load(o + k, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
        store_hidden(g.h, pl, g.places, rp, r, v * scale);
    }
    if (threadIdx.x == 0) st_agent32(&g.done[blockIdx.x], 0u);
}

// ---- expand: y += W^T h ---------------------------------------------------------
struct ExpandArgs {
    const uint16_t *h;  // [place][Rp]
    const uint16_t *w;  // [S][R][C]
    uint16_t *y;
    int64_t ldy;
    LoraPlan plan;
    int32_t T, S, C, R, max_tiles;
};

// A wave takes 128 columns of one tile's 64 places.  Matrix instruction: rows =
// columns of y, columns = places, 16 ranks.  Lane c of the row axis holds the
// 8-column piece pi(c) = 4 (c mod 4) + c / 4, instruction j its column j: then
// the lane's results i = 0..3 are, for j = 0..7, eight neighbouring columns of
// piece 4 i + q, one 16-byte access to y, and the four lanes of a token touch
// 64 contiguous bytes.
template <int RT>
__global__ __launch_bounds__(256) void k_lora_expand(ExpandArgs g) {
    const int w = __builtin_amdgcn_readfirstlane(wave_id()), l = lane_id(), c16 = l & 15, q = l >> 4;
    // workgroups go round the eight XCDs: with eight column blocks or more, one XCD keeps to
    // every eighth block and goes through all tiles of it, whose adapters then stay in its L2
    const int b = blockIdx.x, blocks = (g.C + 511) / 512;
    const int cb = blocks >= 8 ? ((b >> 3) / g.max_tiles) * 8 + (b & 7) : b % blocks;
    const int tile = blocks >= 8 ? (b >> 3) % g.max_tiles : b / blocks;
    const int base = (cb * 4 + w) * 128;
    const int slot = g.plan.tile_slot[tile];
    if ((uint32_t)slot >= (uint32_t)g.S || base >= g.C) return;
    const int count = g.plan.tile_count[tile] < LT ? g.plan.tile_count[tile] : LT;
    const int col = base + ((c16 & 3) * 4 + (c16 >> 2)) * 8;
    s16x4 frag[RT][8];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        u32x4 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = rt * 16 + q * 4 + i;
            v[i] = u32x4{0, 0, 0, 0};
            if (r < g.R && col < g.C) v[i] = ld16(g.w + ((int64_t)slot * g.R + r) * g.C + col);
        }
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            const u32x2 lo = {__builtin_amdgcn_perm(v[1][d], v[0][d], 0x05040100u),
                              __builtin_amdgcn_perm(v[3][d], v[2][d], 0x05040100u)};
            const u32x2 hi = {__builtin_amdgcn_perm(v[1][d], v[0][d], 0x07060302u),
                              __builtin_amdgcn_perm(v[3][d], v[2][d], 0x07060302u)};
            frag[rt][2 * d] = __builtin_bit_cast(s16x4, lo);
            frag[rt][2 * d + 1] = __builtin_bit_cast(s16x4, hi);
        }
    }
    for (int sub = 0; sub * 16 < count; ++sub) {
        const int64_t place = (int64_t)tile * LT + sub * 16 + c16;
        const int tok = token_of(g.plan.order[place], g.T);
        uint16_t *py = g.y + (int64_t)(tok < 0 ? 0 : tok) * g.ldy + base + q * 8;
        u32x4 yv[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            yv[i] = u32x4{0, 0, 0, 0};
            if (tok >= 0 && base + (i * 4 + q) * 8 < g.C) yv[i] = ld16(py + i * 32);
        }
        f32x4 acc[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            const s16x4 hv =
                __builtin_bit_cast(s16x4, *reinterpret_cast<const u32x2 *>(g.h + place * (RT * 16) + rt * 16 + q * 4));
#pragma unroll
            for (int j = 0; j < 8; ++j)
                acc[j] = __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(frag[rt][j], hv, acc[j], 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (tok >= 0 && base + (i * 4 + q) * 8 < g.C) {
                u32x4 o;
#pragma unroll
                for (int d = 0; d < 4; ++d)
                    o[d] = cast_pair(__uint_as_float(yv[i][d] << 16) + acc[2 * d][i],
                                     __uint_as_float(yv[i][d] & 0xFFFF0000u) + acc[2 * d + 1][i]);
                *reinterpret_cast<u32x4 *>(py + i * 32) = o;
            }
        }
    }
}

// ---- outer: G_i = sum over i's tokens of u z^T ------------------------------------
struct OuterSide {
    const uint16_t *hi, *lo;  // u: [Rp][place]
    const uint16_t *z;        // [tokens][ldz]
    int64_t ldz;
    float *out;               // [S][R][C]
    float *partial;           // [chunks][2][R][C]
    int32_t C;
    int32_t waves;            // column blocks
};

struct OuterArgs {
    OuterSide side[2];
    LoraPlan plan;
    int64_t places;
    int32_t T, R, S, max_tiles;
    int32_t q, chunks, accumulate, wg0;  // q: tiles of a chunk; wg0: workgroups of side 0 per chunk
};

template <int W>
struct ZVec;
template <>
struct ZVec<8> {
    typedef u32x4 T;
};
template <>
struct ZVec<4> {
    typedef u32x2 T;
};

// A wave takes 16 W columns and one chunk of q tiles.  Matrix instruction: rows
// = ranks, columns = columns of z, 32 tokens.  Lane c of the column axis holds
// W neighbouring columns of eight tokens, transposed in registers; instruction
// j takes its column j.  A chunk may cover several adapters and an adapter
// several chunks: a run that lies in one chunk goes straight to the output, the
// others to the chunk's partial sums (0: continues an earlier chunk's run, 1:
// begins here), which k_lora_outer_sum adds in order.
template <int RT, int W>
__global__ __launch_bounds__(256) void k_lora_outer(OuterArgs g) {
    typedef typename ZVec<W>::T ZV;
    const int w = __builtin_amdgcn_readfirstlane(wave_id()), l = lane_id(), c16 = l & 15, q = l >> 4;
    const int sd = (int)blockIdx.x >= g.wg0 ? 1 : 0;
    const OuterSide &s = g.side[sd];
    const int cb = ((int)blockIdx.x - (sd ? g.wg0 : 0)) * 4 + w, chunk = blockIdx.y;
    if (cb >= s.waves) return;
    const int ntiles = *g.plan.ntiles < g.max_tiles ? *g.plan.ntiles : g.max_tiles;
    const int ta = chunk * g.q, tb = ta + g.q < ntiles ? ta + g.q : ntiles;
    const int col = cb * 16 * W + c16 * W;
    const bool colok = col < s.C;
    f32x4 acc[RT][W];
    auto flush = [&](int slot) {
        const int t0 = g.plan.slot_tile[slot], t1 = g.plan.slot_tile[slot + 1];
        const bool direct = t0 / g.q == (t1 - 1) / g.q;
        float *o = direct ? s.out + (int64_t)slot * g.R * s.C
                          : s.partial + ((int64_t)chunk * 2 + (t0 >= ta ? 1 : 0)) * g.R * s.C;
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = rt * 16 + q * 4 + i;
                if (r < g.R && colok) {
                    float *p = o + (int64_t)r * s.C + col;
#pragma unroll
                    for (int j = 0; j < W; j += 4) {
                        f32x4 v = {acc[rt][j][i], acc[rt][j + 1][i], acc[rt][j + 2][i], acc[rt][j + 3][i]};
                        if (direct && g.accumulate) v += *reinterpret_cast<const f32x4 *>(p + j);
                        *reinterpret_cast<f32x4 *>(p + j) = v;
                    }
                }
            }
    };
    int cur = -1;
    for (int t = ta; t < tb; ++t) {
        const int slot = __builtin_amdgcn_readfirstlane(g.plan.tile_slot[t]);
        const int raw = __builtin_amdgcn_readfirstlane(g.plan.tile_count[t]), count = raw < LT ? raw : LT;
        if ((uint32_t)slot >= (uint32_t)g.S) break;
        if (slot != cur) {
            if (cur >= 0) flush(cur);
            cur = slot;
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                for (int j = 0; j < W; ++j) acc[rt][j] = f32x4{0, 0, 0, 0};
        }
        for (int half = 0; half * 32 < count; ++half) {
            const int64_t place = (int64_t)t * LT + half * 32 + q * 8;
            const i32x4 o0 = *reinterpret_cast<const i32x4 *>(g.plan.order + place);
            const i32x4 o1 = *reinterpret_cast<const i32x4 *>(g.plan.order + place + 4);
            ZV z[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int tok = token_of(i < 4 ? o0[i & 3] : o1[i & 3], g.T);
                z[i] = ZV{};
                if (tok >= 0 && colok) z[i] = *reinterpret_cast<const ZV *>(s.z + (int64_t)tok * s.ldz + col);
            }
            // places past the last 16 that hold a token have no u
            const bool some = half * 32 + q * 8 < (count + 15) / 16 * 16;
            u32x4 uh[RT], ul[RT];
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                uh[rt] = u32x4{0, 0, 0, 0};
                ul[rt] = u32x4{0, 0, 0, 0};
                if (some) {
                    uh[rt] = ld16(s.hi + (int64_t)(rt * 16 + c16) * g.places + place);
                    ul[rt] = ld16(s.lo + (int64_t)(rt * 16 + c16) * g.places + place);
                }
            }
#pragma unroll
            for (int j = 0; j < W; ++j) {
                const uint32_t sel = (j & 1) ? 0x07060302u : 0x05040100u;
                u32x4 zt;
#pragma unroll
                for (int d = 0; d < 4; ++d)
                    zt[d] = __builtin_amdgcn_perm(z[2 * d + 1][j >> 1], z[2 * d][j >> 1], sel);
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) {
                    acc[rt][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf(ul[rt]), as_bf(zt), acc[rt][j], 0, 0, 0);
                    acc[rt][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf(uh[rt]), as_bf(zt), acc[rt][j], 0, 0, 0);
                }
            }
        }
    }
    if (cur >= 0) flush(cur);
}

// The gradients of adapters that lie in several chunks: their partial sums in
// the chunks' order; adapters without tokens: zero.
__global__ __launch_bounds__(256) void k_lora_outer_sum(OuterArgs g) {
    const OuterSide &s = g.side[blockIdx.z];
    const int slot = blockIdx.y;
    const int t0 = g.plan.slot_tile[slot], t1 = g.plan.slot_tile[slot + 1];
    const int64_t n = (int64_t)g.R * s.C;
    const int64_t e = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (e >= n || (t1 > t0 && t0 / g.q == (t1 - 1) / g.q) || (t1 == t0 && g.accumulate)) return;
    float *o = s.out + (int64_t)slot * n + e;
    f32x4 v = {0, 0, 0, 0};
    if (t1 > t0) {
        const int c0 = t0 / g.q, c1 = (t1 - 1) / g.q < g.chunks ? (t1 - 1) / g.q : g.chunks - 1;
        if (g.accumulate) v = *reinterpret_cast<const f32x4 *>(o);
#pragma unroll 4
        for (int c = c0 < 0 ? 0 : c0; c <= c1; ++c)
            v += *reinterpret_cast<const f32x4 *>(s.partial + ((int64_t)c * 2 + (c == c0 ? 1 : 0)) * n + e);
    }
    *reinterpret_cast<f32x4 *>(o) = v;
}

// ---- launches ---------------------------------------------------------------------
// Parts of the long axis in shrink: enough that the tiles' workgroups come to
// about 1024, each wave keeping 4 steps of 32 or more.
int lora_ksplit(int64_t T, int64_t S, int64_t C) {
    const int64_t groups = (T + 15) / 16 > lora_max_tiles(T, S) ? (T + 15) / 16 : lora_max_tiles(T, S);
    const int64_t most = C / 512 > 1 ? C / 512 : 1;
    int64_t k = 1024 / groups;
    if (k > most) k = most;
    if (k > 16) k = 16;
    return (int)(k < 1 ? 1 : k);
}

// Bytes of shrink's counters and partial sums, for this T and every smaller one.
// ksplit > 1 means at most 512 tiles, so 2048 counters, and 1024 tiles times
// parts.  The counters stay at the front whatever the sizes: they are zero
// between calls, and no call may leave anything else there.
constexpr int64_t kShrinkCounters = 2048;

int64_t lora_shrink_ws(int64_t T, int64_t S, int64_t R) {
    const int64_t rp = (R + 15) / 16 * 16, mt = lora_max_tiles(T, S), parts = mt * 16 < 1024 ? mt * 16 : 1024;
    return kShrinkCounters * 4 + parts * LT * rp * 4;
}

// Tiles of a chunk in outer: about 2048 waves over both sides, 256 tokens or more.
int64_t lora_outer_waves(int64_t K, int64_t N, int64_t R) {
    const int64_t width = R > 64 ? 64 : 128;
    return (K + width - 1) / width + (N + width - 1) / width;
}

int lora_chunk(int64_t T, int64_t S, int64_t K, int64_t N, int64_t R) {
    const int64_t q = lora_max_tiles(T, S) * lora_outer_waves(K, N, R) / 2048;
    return (int)(q < 4 ? 4 : (q > 64 ? 64 : q));
}

int64_t lora_chunks(int64_t T, int64_t S, int q) { return (lora_max_tiles(T, S) + q - 1) / q; }

// Most chunks of this T and every smaller one: a chunk has 4 tiles, or more
// than 4/5 of the tiles that make 2048 waves, or 64 tiles.
int64_t lora_most_chunks(int64_t T, int64_t S, int64_t K, int64_t N, int64_t R) {
    const int64_t mt = lora_max_tiles(T, S), a = mt / 4 + 1, b = 2560 / lora_outer_waves(K, N, R) + 2, c = mt / 64 + 1;
    const int64_t m = a < b ? a : b;
    return m > c ? m : c;
}

void launch_shrink(const ShrinkArgs &g, int64_t tiles, int rt, hipStream_t stream) {
    const dim3 grid((unsigned)(tiles * 4), (unsigned)g.ksplit), block(256);
    switch (rt) {
    case 1: k_lora_shrink<1><<<grid, block, 0, stream>>>(g); break;
    case 2: k_lora_shrink<2><<<grid, block, 0, stream>>>(g); break;
    case 3: k_lora_shrink<3><<<grid, block, 0, stream>>>(g); break;
    case 4: k_lora_shrink<4><<<grid, block, 0, stream>>>(g); break;
    case 5: k_lora_shrink<5><<<grid, block, 0, stream>>>(g); break;
    case 6: k_lora_shrink<6><<<grid, block, 0, stream>>>(g); break;
    case 7: k_lora_shrink<7><<<grid, block, 0, stream>>>(g); break;
    default: k_lora_shrink<8><<<grid, block, 0, stream>>>(g); break;
    }
}

void launch_expand(const ExpandArgs &g, int rt, hipStream_t stream) {
    const int64_t blocks = ((int64_t)g.C + 511) / 512;
    const dim3 grid((unsigned)((blocks >= 8 ? (blocks + 7) / 8 * 8 : blocks) * g.max_tiles)), block(256);
    switch (rt) {
    case 1: k_lora_expand<1><<<grid, block, 0, stream>>>(g); break;
    case 2: k_lora_expand<2><<<grid, block, 0, stream>>>(g); break;
    case 3: k_lora_expand<3><<<grid, block, 0, stream>>>(g); break;
    case 4: k_lora_expand<4><<<grid, block, 0, stream>>>(g); break;
    case 5: k_lora_expand<5><<<grid, block, 0, stream>>>(g); break;
    case 6: k_lora_expand<6><<<grid, block, 0, stream>>>(g); break;
    case 7: k_lora_expand<7><<<grid, block, 0, stream>>>(g); break;
    default: k_lora_expand<8><<<grid, block, 0, stream>>>(g); break;
    }
}

void launch_outer(const OuterArgs &g, int rt, int64_t wgs, int64_t chunks, hipStream_t stream) {
    const dim3 grid((unsigned)wgs, (unsigned)chunks), block(256);
    switch (rt) {
    case 1: k_lora_outer<1, 8><<<grid, block, 0, stream>>>(g); break;
    case 2: k_lora_outer<2, 8><<<grid, block, 0, stream>>>(g); break;
    case 3: k_lora_outer<3, 8><<<grid, block, 0, stream>>>(g); break;
    case 4: k_lora_outer<4, 8><<<grid, block, 0, stream>>>(g); break;
    case 5: k_lora_outer<5, 4><<<grid, block, 0, stream>>>(g); break;
    case 6: k_lora_outer<6, 4><<<grid, block, 0, stream>>>(g); break;
    case 7: k_lora_outer<7, 4><<<grid, block, 0, stream>>>(g); break;
    default: k_lora_outer<8, 4><<<grid, block, 0, stream>>>(g); break;
    }
}

int64_t round256(int64_t n) { return (n + 255) / 256 * 256; }

}  // namespace pulse

using namespace pulse;

extern "C" int64_t pulse_lora_plan_size(int64_t T, int64_t S) { return lora_plan_size(T, S); }

extern "C" int64_t pulse_lora_hidden_size(int64_t T, int64_t S, int64_t R) { return lora_hidden_size(T, S, R, true); }

// Workspace: the workgroup counters and partial sums of shrink, at the front and
// any T up to the one given; then h of a forward pass, or in a backward pass dh
// and the partial sums of both gradients.
extern "C" int64_t pulse_lora_ws_size(int64_t T, int64_t K, int64_t N, int64_t R, int64_t S, int32_t train) {
    int64_t n = round256(lora_shrink_ws(T, S, R)) + round256(lora_hidden_size(T, S, R, train != 0));
    if (train) n += lora_most_chunks(T, S, K, N, R) * 2 * R * (K + N) * 4;
    return n;
}

extern "C" int pulse_launch_lora_plan(const int32_t *ids, int64_t T, int32_t S, void *plan, uint32_t *d_status,
                                      hipStream_t stream) {
    k_lora_plan<<<dim3(1), dim3(LP_THREADS), (size_t)LP_WAVES * S * 4, stream>>>(
        ids, (int32_t)T, S, lora_plan_parts(plan, T, S), (int32_t)lora_max_tiles(T, S), d_status);
    return hipGetLastError() == hipSuccess ? 0 : -5;
}

namespace {

void shrink(const uint16_t *x, int64_t ldx, const uint16_t *a, const float *scales, const LoraPlan &plan,
            const LoraHidden &h, void *ws, int64_t T, int64_t C, int64_t R, int64_t S, hipStream_t stream) {
    const int64_t mt = lora_max_tiles(T, S);
    ShrinkArgs g{};
    g.x = x;
    g.ldx = ldx;
    g.a = a;
    g.scales = scales;
    g.plan = plan;
    g.h = h;
    g.done = static_cast<uint32_t *>(ws);
    g.partial = reinterpret_cast<float *>(static_cast<char *>(ws) + kShrinkCounters * 4);
    g.places = mt * LT;
    g.T = (int32_t)T;
    g.S = (int32_t)S;
    g.C = (int32_t)C;
    g.R = (int32_t)R;
    g.ksplit = lora_ksplit(T, S, C);
    launch_shrink(g, mt, (int)((R + 15) / 16), stream);
}

void expand(const uint16_t *h, const uint16_t *w, uint16_t *y, int64_t ldy, const LoraPlan &plan, int64_t T, int64_t C,
            int64_t R, int64_t S, hipStream_t stream) {
    ExpandArgs g{};
    g.h = h;
    g.w = w;
    g.y = y;
    g.ldy = ldy;
    g.plan = plan;
    g.T = (int32_t)T;
    g.S = (int32_t)S;
    g.C = (int32_t)C;
    g.R = (int32_t)R;
    g.max_tiles = (int32_t)lora_max_tiles(T, S);
    launch_expand(g, (int)((R + 15) / 16), stream);
}

}  // namespace

extern "C" int pulse_launch_lora_forward(const uint16_t *x, int64_t ldx, const uint16_t *a, const uint16_t *b,
                                         const float *scales, const void *plan, int64_t T, int64_t K, int64_t N, int64_t R,
                                         int64_t S, uint16_t *y, int64_t ldy, void *h, void *ws, hipStream_t stream) {
    const LoraPlan p = lora_plan_parts(const_cast<void *>(plan), T, S);
    const LoraHidden hp = h ? lora_hidden_parts(h, T, S, R, true)
                            : lora_hidden_parts(static_cast<char *>(ws) + round256(lora_shrink_ws(T, S, R)), T, S, R, false);
    shrink(x, ldx, a, scales, p, hp, ws, T, K, R, S, stream);
    expand(hp.rows, b, y, ldy, p, T, N, R, S, stream);
    return hipGetLastError() == hipSuccess ? 0 : -5;
}

extern "C" int pulse_launch_lora_backward(const uint16_t *x, int64_t ldx, const uint16_t *dy, int64_t lddy,
                                          const uint16_t *a, const uint16_t *b, const float *scales, const void *plan,
                                          int64_t T, int64_t K, int64_t N, int64_t R, int64_t S, const void *h,
                                          uint16_t *dx, int64_t lddx, float *da, float *db, int32_t accumulate,
                                          void *ws, hipStream_t stream) {
    const LoraPlan p = lora_plan_parts(const_cast<void *>(plan), T, S);
    char *w = static_cast<char *>(ws) + round256(lora_shrink_ws(T, S, R));
    const LoraHidden dh = lora_hidden_parts(w, T, S, R, true), hp = lora_hidden_parts(const_cast<void *>(h), T, S, R, true);
    shrink(dy, lddy, b, scales, p, dh, ws, T, N, R, S, stream);
    if (dx) expand(dh.rows, a, dx, lddx, p, T, K, R, S, stream);
    const int rt = (int)((R + 15) / 16), width = rt > 4 ? 64 : 128;
    OuterArgs g{};
    g.plan = p;
    g.places = lora_max_tiles(T, S) * LT;
    g.T = (int32_t)T;
    g.R = (int32_t)R;
    g.S = (int32_t)S;
    g.max_tiles = (int32_t)lora_max_tiles(T, S);
    g.q = lora_chunk(T, S, K, N, R);
    g.accumulate = accumulate;
    const int64_t chunks = lora_chunks(T, S, g.q);
    g.chunks = (int32_t)chunks;
    float *part = reinterpret_cast<float *>(w + round256(lora_hidden_size(T, S, R, true)));
    g.side[0] = OuterSide{dh.hi, dh.lo, x, ldx, da, part, (int32_t)K, (int32_t)((K + width - 1) / width)};
    g.side[1] = OuterSide{hp.hi, hp.lo, dy, lddy, db, part + chunks * 2 * R * K, (int32_t)N,
                          (int32_t)((N + width - 1) / width)};
    g.wg0 = (g.side[0].waves + 3) / 4;
    launch_outer(g, rt, g.wg0 + (g.side[1].waves + 3) / 4, chunks, stream);
    const int64_t most = R * (K > N ? K : N);
    k_lora_outer_sum<<<dim3((unsigned)((most / 4 + 255) / 256), (unsigned)S, 2), dim3(256), 0, stream>>>(g);
    return hipGetLastError() == hipSuccess ? 0 : -5;
}
