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
// Large batches are bound by reading or writing the [tokens, C] matrices (an
// element takes 2 R multiplications for 2 to 4 bytes), so the work is to touch
// those once, in rows of 256 contiguous bytes that are on their way while the
// last ones are multiplied: shrink turns its rows round in LDS, and the two
// operands that a matrix instruction wants along the other axis (expand's
// adapter, outer's tokens) are transposed in registers, one v_perm_b32 per pair
// of values.  Small batches are bound by launches and round trips to memory: they
// make h and y in one launch, and need no sum over chunks.
//
// A plan groups a batch's tokens by adapter: tiles of 64 places, each of one
// adapter, whose places hold token numbers in ascending order (-1: empty).
// Every kernel works on tiles, so a token is found by its place, and no atomic's
// order reaches a result: the same call gives the same bits.  Another batch may not:
// how many tiles a partial sum covers, and how many workgroups share the long axis,
// go by the batch's size.
#include "device.hpp"

namespace pulse {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x4 __attribute__((ext_vector_type(4)));

constexpr int LT = 64;            // places of a tile
constexpr int LP_ADAPTERS = 1024;  // most adapters

// The plan's parts for T tokens and S adapters (32-bit words in one buffer).
struct LoraPlan {
    int32_t *ntiles;      // [16] tiles in use, then padding
    int32_t *tile_slot;   // [max_tiles] adapter of a tile, -1: unused
    int32_t *tile_count;  // [max_tiles] tokens of a tile
    int32_t *slot_tile;   // [S + 1] first tile of an adapter
    int32_t *order;       // [max_tiles * 64] token of a place, -1: empty
    int32_t *group;       // [max_groups] tile * 4 + its 16 places, for every 16 that hold a token, -1: unused
};

__host__ __device__ inline int64_t lora_max_tiles(int64_t T, int64_t S) {
    const int64_t t = (T + LT - 1) / LT + S;
    return T < t ? T : t;
}

// the 16 places that hold a token: one for each 16 tokens, and one more for each adapter
__host__ __device__ inline int64_t lora_max_groups(int64_t T, int64_t S) {
    const int64_t t = (T + 15) / 16 + S;
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
    p.group = p.order + mt * LT;
    return p;
}

inline int64_t lora_plan_size(int64_t T, int64_t S) {
    const int64_t mt = lora_max_tiles(T, S);
    return 4 * (16 + 2 * lora_round4(mt) + lora_round4(S + 1) + lora_round4(lora_max_groups(T, S)) + mt * LT);
}

// ---- the plan: a stable counting sort by adapter -----------------------------
// One workgroup of NW waves.  Wave w owns a run of tokens and counts them per
// adapter in its own row of an LDS table; the rows' prefix sums give each wave
// its first place for every adapter; then every wave deals its tokens out in
// order, 64 at a time, ranking equal adapters with ballots.  It is bound by
// latency: the ids are read sixteen loads at a time and stay in registers up to 16384
// tokens, and one lane of each adapter
// counts for the 64 (equal lanes' LDS atomics would queue).
constexpr int LP_AHEAD = 16;

// a lane's ids of the next tokens; -1 past the end
__device__ __forceinline__ void read_ids(const int32_t *__restrict__ ids, int t, int t1, int (&id)[LP_AHEAD]) {
#pragma unroll
    for (int k = 0; k < LP_AHEAD; ++k) id[k] = t + k * kWave < t1 ? ids[t + k * kWave] : -1;
}

// the lanes whose id (-1: none) equals this lane's; bits: of the largest adapter's number
__device__ __forceinline__ uint64_t equal_lanes(int id, int bits) {
    uint64_t same = __ballot(id >= 0);
    for (int b = 0; b < bits; ++b) {
        const uint64_t m = __ballot((id >> b) & 1);
        same &= ((id >> b) & 1) ? m : ~m;
    }
    return same;
}

template <int NW>
__global__ __launch_bounds__(NW *kWave) void k_lora_plan(const int32_t *__restrict__ ids, int32_t T, int32_t S,
                                                         LoraPlan p, int32_t max_tiles, int32_t max_groups,
                                                         uint32_t *d_status) {
    constexpr int kThreads = NW * kWave, kPer = LP_ADAPTERS / kThreads > 1 ? LP_ADAPTERS / kThreads : 1;
    extern __shared__ int32_t sh[];  // [NW][S] counts, then first places; [S] counts; [S] first tiles; [S] first groups
    __shared__ int32_t s_scan[2][NW];
    int32_t *const s_cnt = sh + NW * S, *const s_tile = s_cnt + S, *const s_group = s_tile + S;
    const int tid = threadIdx.x, w = wave_id(), l = lane_id();
    const int per = ((T + NW - 1) / NW + kWave - 1) / kWave * kWave;
    const int t0 = w * per, t1 = t0 + per < T ? t0 + per : T;
    const int bits = S > 1 ? 32 - __builtin_clz(S - 1) : 0;
    int id[LP_AHEAD];
    read_ids(ids, t0 + l, t1, id);
    for (int i = tid; i < NW * S; i += kThreads) sh[i] = 0;
    __syncthreads();
    bool bad = false;
    for (int tb = t0; tb < t1; tb += LP_AHEAD * kWave) {
        if (tb != t0) read_ids(ids, tb + l, t1, id);
#pragma unroll
        for (int k = 0; k < LP_AHEAD; ++k) {
            if (tb + k * kWave >= t1) break;
            const int a = id[k] >= 0 && id[k] < S ? id[k] : -1;
            bad |= a != id[k] && id[k] != -1;
            const uint64_t same = equal_lanes(a, bits);
            if (a >= 0 && (same >> l) == 1ull) atomicAdd(&sh[w * S + a], __builtin_popcountll(same));
        }
    }
    if (__ballot(bad) && l == 0) or_agent32(d_status, 2u /*PULSE_DS_BADINDEX*/);
    __syncthreads();
    // a thread's adapters: every wave's tokens before it, tiles, and groups of 16 places
    int before[kPer][NW], cnt[kPer], tsum = 0, gsum = 0;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const int a = kPer * tid + k;
#pragma unroll
        for (int i = 0; i < NW; ++i) before[k][i] = a < S ? sh[i * S + a] : 0;
        cnt[k] = 0;
#pragma unroll
        for (int i = 0; i < NW; ++i) {
            const int c = before[k][i];
            before[k][i] = cnt[k];
            cnt[k] += c;
        }
        tsum += (cnt[k] + LT - 1) / LT;
        gsum += (cnt[k] + 15) / 16;
    }
    // the first tile and group of the thread's adapters, and the totals
    int first = wave_incl_sum(tsum), gfirst = wave_incl_sum(gsum), total = 0, gtotal = 0;
    if (l == kWave - 1) {
        s_scan[0][w] = first;
        s_scan[1][w] = gfirst;
    }
    first -= tsum;
    gfirst -= gsum;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NW; ++i) {
        const int t = s_scan[0][i], n = s_scan[1][i];
        first += i < w ? t : 0;
        gfirst += i < w ? n : 0;
        total += t;
        gtotal += n;
    }
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const int a = kPer * tid + k;
        if (a < S) {
#pragma unroll
            for (int i = 0; i < NW; ++i) sh[i * S + a] = first * LT + before[k][i];
            s_cnt[a] = cnt[k];
            s_tile[a] = first;
            s_group[a] = gfirst;
            p.slot_tile[a] = first;
        }
        first += (cnt[k] + LT - 1) / LT;
        gfirst += (cnt[k] + 15) / 16;
    }
    if (tid == 0) {
        p.slot_tile[S] = total;
        *p.ntiles = total;
    }
    __syncthreads();
    for (int tb = t0; tb < t1; tb += LP_AHEAD * kWave) {
        if (t0 + LP_AHEAD * kWave < t1) read_ids(ids, tb + l, t1, id);
#pragma unroll
        for (int k = 0; k < LP_AHEAD; ++k) {
            if (tb + k * kWave >= t1) break;
            const int a = id[k] >= 0 && id[k] < S ? id[k] : -1;
            const uint64_t same = equal_lanes(a, bits);
            if (a >= 0) {
                const int place = sh[w * S + a] + (int)lanes_below(same);
                p.order[place] = tb + k * kWave + l;
                // the last of the equal lanes moves the adapter's next place on (all have read it: a
                // wave's LDS accesses are in order; a volatile pointer would make them flat ones, which
                // wait for the stores of the tokens)
                if ((same >> l) == 1ull) sh[w * S + a] = place + 1;
            }
            asm volatile("" ::: "memory");  // the next 64 tokens read what these wrote
        }
    }
    // the places past an adapter's last token are empty
    for (int a = w; a < S; a += NW) {
        const int c = s_cnt[a];
        if (l >= c % LT && c % LT != 0) p.order[(s_tile[a] + c / LT) * LT + l] = -1;
    }
    // a group's adapter: the last one that begins at or before it (an empty one begins where the next
    // does); every fourth of an adapter begins a tile
    for (int i = tid; i < max_groups; i += kThreads) {
        int v = -1;
        if (i < gtotal) {
            int lo = 0, hi = S;
            while (hi - lo > 1) {
                const int mid = (lo + hi) / 2;
                if (s_group[mid] <= i) lo = mid;
                else hi = mid;
            }
            const int n = i - s_group[lo];
            v = s_tile[lo] * 4 + n;
            if (n % 4 == 0) {
                const int c = s_cnt[lo] - n * 16;
                p.tile_slot[v / 4] = lo;
                p.tile_count[v / 4] = c < LT ? c : LT;
            }
        }
        p.group[i] = v;
    }
    for (int i = total + tid; i < max_tiles; i += kThreads) p.tile_slot[i] = -1;
}

// ---- what the kernels share -----------------------------------------------------
// h (or dh) of every place, in the forms its readers want: for expand, whose sums go
// out with 8 bits of mantissa, two BF16 (16 bits) in the order of its matrix operand
// (put_row); for outer, whose sums over tokens go out in float32, the float32 value
// as the exact sum of three BF16 (8 bits of mantissa each), each [Rp][place].
struct LoraHidden {
    uint16_t *rows;
    uint16_t *part[3];
};

inline int64_t lora_hidden_size(int64_t T, int64_t S, int64_t R, bool train) {
    const int64_t rp = (R + 15) / 16 * 16, places = lora_max_tiles(T, S) * LT;
    return places * rp * 2 * (train ? 5 : 2);
}

inline LoraHidden lora_hidden_parts(void *h, int64_t T, int64_t S, int64_t R, bool train) {
    const int64_t rp = (R + 15) / 16 * 16, places = lora_max_tiles(T, S) * LT;
    LoraHidden p;
    p.rows = static_cast<uint16_t *>(h);
    for (int i = 0; i < 3; ++i) p.part[i] = train ? p.rows + (i + 2) * places * rp : nullptr;
    return p;
}

// A place's token.  Whatever a plan's buffer holds, no kernel leaves its tensors:
// tokens, adapters, counts and chunks out of range are taken as empty or cut off.
__device__ __forceinline__ int token_of(int t, int T) { return (uint32_t)t < (uint32_t)T ? t : -1; }

// Where the row of place i of a list that begins with a tile lies; an empty place
// stands for the first of its 16, or of its tile where those are all empty.
__device__ __forceinline__ int64_t row_of(const int32_t *order, int i, int T, int64_t ld) {
    int t = token_of(order[i], T);
    if (t < 0) t = token_of(order[i & ~15], T);
    if (t < 0) t = token_of(order[i & ~(LT - 1)], T);
    return (t < 0 ? 0 : t) * ld;
}

__device__ __forceinline__ u32x4 ld16(const uint16_t *p) { return *reinterpret_cast<const u32x4 *>(p); }

// What is read once goes past the last-level cache: there it would displace lines
// that earlier kernels left to be written back, which halves its rate (470 MB after
// a 512 MB copy: 4.3 TB/s, non-temporal 6.0).
__device__ __forceinline__ u32x4 ld16_once(const uint16_t *p) {
    return __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(p));
}

__device__ __forceinline__ bf16x8 as_bf(const u32x4 &v) { return __builtin_bit_cast(bf16x8, v); }

// Four float32 values as two BF16 each: the nearest one, at most the largest, and what
// is left with its infinities and NaN (an infinity in the first part would leave no
// number for the second).
struct Split {
    u32x2 top, rest;
    f32x4 left;  // of which rest is the nearest BF16
};

__device__ __forceinline__ Split split4(const f32x4 &v) {
    constexpr float kMost = 0x1.FEp127f;  // the largest BF16
    Split s;
    s.top = u32x2{cast_pair(__builtin_amdgcn_fmed3f(v[0], -kMost, kMost), __builtin_amdgcn_fmed3f(v[1], -kMost, kMost)),
                  cast_pair(__builtin_amdgcn_fmed3f(v[2], -kMost, kMost), __builtin_amdgcn_fmed3f(v[3], -kMost, kMost))};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        s.left[i] = v[i] - __uint_as_float((i & 1) ? (s.top[i >> 1] & 0xFFFF0000u) : (s.top[i >> 1] << 16));
    s.rest = u32x2{cast_pair(s.left[0], s.left[1]), cast_pair(s.left[2], s.left[3])};
    return s;
}

// h's four values of ranks 16 rt + 4 q .. + 3 at one place of `rows`.  Expand's matrix
// instruction takes 32 products, two rank tiles with their first parts, and once more
// with their second ones; a tile that is left over takes two instructions of 16.
// Operand i of a place's RT, for the lanes of quarter q, is the 16 bytes at
// (place * RT + i) * 4 + q; of the tile left over, both its parts.
__device__ __forceinline__ void put_row(u32x2 *rows, int64_t place, int RT, int rt, int q, const Split &s) {
    const bool alone = rt == RT - 1 && (RT & 1);
    u32x2 *const to = rows + ((place * RT + (alone ? rt : rt & ~1)) * 4 + q) * 2 + (alone ? 0 : rt & 1);
    to[0] = s.top;
    to[alone ? 1 : 8] = s.rest;
}

// the same operands in registers, from the values of all tiles
template <int RT>
__device__ __forceinline__ void row_operands(const f32x4 (&v)[RT], u32x4 (&h)[RT]) {
#pragma unroll
    for (int rt = 0; rt < RT; rt += 2) {
        const Split a = split4(v[rt]);
        if (rt + 1 < RT) {
            const Split b = split4(v[rt + 1 < RT ? rt + 1 : rt]);
            h[rt] = u32x4{a.top.x, a.top.y, b.top.x, b.top.y};
            h[rt + 1 < RT ? rt + 1 : rt] = u32x4{a.rest.x, a.rest.y, b.rest.x, b.rest.y};
        } else {
            h[rt] = u32x4{a.top.x, a.top.y, a.rest.x, a.rest.y};
        }
    }
}

// A part of h below the first may be zero or of the other sign, and would make a NaN of
// an infinity that its first part has multiplied into the sum already: there the lower
// parts are multiplied with one of its sign instead.
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t ones_for_infinities(uint32_t pair) {
    if ((pair & 0x7F80u) == 0x7F80u) pair = (pair & 0xFFFF8000u) | 0x3F80u;
    if ((pair & 0x7F800000u) == 0x7F800000u) pair = (pair & 0x8000FFFFu) | 0x3F800000u;
    return pair;
}

// the larger magnitudes of two pairs, and whether a pair of magnitudes holds one that is not finite
__device__ __forceinline__ uint32_t most_of(uint32_t m, uint32_t pair) {
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, m),
                                                                  __builtin_bit_cast(u16x2, pair & 0x7FFF7FFFu)));
}

__device__ __forceinline__ bool not_finite(uint32_t m) { return m >= 0x7F800000u || (m & 0xFFFFu) >= 0x7F80u; }

// The adapter's operands beside h's: of each column of a lane's eight, the values of ranks
// 4 q .. 4 q + 3 of two rank tiles, or of the one that is left over.
template <int RT>
struct Columns {
    u32x4 pair[RT > 1 ? RT / 2 : 1][8];
    u32x2 last[RT & 1 ? 8 : 1];
};

// rows(rt, v): the four ranks' rows, eight columns each.  Returns whether the columns are all finite.
template <int RT, typename F>
__device__ __forceinline__ bool read_columns(Columns<RT> &f, F &&rows) {
    const auto low = [](uint32_t x, uint32_t y) { return __builtin_amdgcn_perm(y, x, 0x05040100u); };
    const auto high = [](uint32_t x, uint32_t y) { return __builtin_amdgcn_perm(y, x, 0x07060302u); };
    uint32_t most = 0;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        u32x4 v[4];
        rows(rt, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int d = j / 2;
            const u32x2 c = (j & 1) ? u32x2{high(v[0][d], v[1][d]), high(v[2][d], v[3][d])}
                                    : u32x2{low(v[0][d], v[1][d]), low(v[2][d], v[3][d])};
            if (rt == RT - 1 && (RT & 1)) f.last[RT & 1 ? j : 0] = c;
            else f.pair[rt / 2][j][2 * (rt & 1)] = c.x, f.pair[rt / 2][j][2 * (rt & 1) + 1] = c.y;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int d = 0; d < 4; ++d) most = most_of(most, v[i][d]);
    }
    return __ballot(not_finite(most)) == 0;
}

// out += h times eight columns.  Where these are not all finite, they are not the
// adapter's any more afterwards.
template <int RT>
__device__ __forceinline__ void multiply_rows(const u32x4 *h, Columns<RT> &f, bool finite, f32x4 (&out)[8]) {
    const auto last = [&](int half) {
        const s16x4 a = __builtin_bit_cast(s16x4, u32x2{h[RT - 1][half * 2], h[RT - 1][half * 2 + 1]});
#pragma unroll
        for (int j = 0; j < 8; ++j)
            out[j] = __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(a, __builtin_bit_cast(s16x4, f.last[RT & 1 ? j : 0]), out[j], 0,
                                                               0, 0);
    };
#pragma unroll
    for (int i = 0; i < RT / 2; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j)
            out[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf(h[2 * i]), as_bf(f.pair[i][j]), out[j], 0, 0, 0);
    if constexpr (RT & 1) last(0);
    if (!finite) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
#pragma unroll
            for (int i = 0; i < RT / 2; ++i)
#pragma unroll
                for (int d = 0; d < 4; ++d) f.pair[i][j][d] = ones_for_infinities(f.pair[i][j][d]);
            if constexpr (RT & 1) f.last[j] = u32x2{ones_for_infinities(f.last[j].x), ones_for_infinities(f.last[j].y)};
        }
    }
#pragma unroll
    for (int i = 0; i < RT / 2; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j)
            out[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf(h[2 * i + 1]), as_bf(f.pair[i][j]), out[j], 0, 0, 0);
    if constexpr (RT & 1) last(1);
}

// h's four values of ranks r .. r+3 at one place, in its forms
__device__ __forceinline__ void store_hidden(const LoraHidden &h, int64_t place, int64_t places, int rp, int r,
                                             const f32x4 &v) {
    const Split s = split4(v);
    put_row(reinterpret_cast<u32x2 *>(h.rows), place, rp / 16, r / 16, r % 16 / 4, s);
    if (h.part[0]) {
        const Split t = split4(s.left);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t at = (r + i) * places + place;
            h.part[0][at] = (uint16_t)(s.top[i >> 1] >> (16 * (i & 1)));
            h.part[1][at] = (uint16_t)(t.top[i >> 1] >> (16 * (i & 1)));
            h.part[2][at] = (uint16_t)(t.rest[i >> 1] >> (16 * (i & 1)));
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
    float *partial;  // [gridDim.y][places][Rp] (SH_PARTS)
    int64_t places;
    int32_t T, S, C, R, max_tiles, max_groups;
    const uint16_t *w;  // [S][R][N] (SH_APPLY)
    uint16_t *y;
    int64_t ldy;
    int32_t N;
};

// SH_WHOLE: h in its forms; SH_PARTS: the workgroups' sums over their shares of the
// long axis; SH_APPLY: y += W^T h too, and h in its forms where they are asked for.
enum ShrinkMode { SH_WHOLE, SH_PARTS, SH_APPLY };

// A wave's piece of LDS: rows of P 16-byte pieces (128 columns, or 64), which it
// writes as they were loaded (four rows an instruction, 256 contiguous bytes each)
// and reads as a matrix instruction wants them (16 rows, 64 bytes each).  Piece p
// of row r lies at p ^ r, so that neither side has two lanes in a bank.
template <int P = 16>
__device__ __forceinline__ int staged(int row, int piece) {
    return row * P + (piece ^ (row & (P - 1)));
}

// Columns of a wave's step, and waves of a workgroup: two waves a SIMD or more in
// the 160 KB of LDS, so that one loads while another turns its rows round, and at
// low ranks two workgroups a compute unit, so that one begins while another adds up
// (16384 x 4096 at rank 16: 29 us, with sixteen waves and one workgroup 35).
constexpr int shrink_cols(int rt, int mt) { return rt + mt <= 4 ? 128 : 64; }
constexpr int SH_WAVES = 8;

// A workgroup takes 16 MT places of a tile; its waves, and with SH_PARTS gridDim.y
// workgroups, share the long axis in steps of 128 or 64 columns, and the waves' sums
// are added through LDS, in their order.  Matrix instruction: rows = ranks,
// columns = places, 32 elements of the long axis.  Read as the instruction wants
// them, 64 bytes of 16 rows at once, rows came in at 10 to 15 bytes a clock and
// compute unit; 256 bytes of 4 rows, turned round in LDS, are not held back.
// The rows of the next step are read while these are multiplied.  Measured:
// 8192 x 5120 at rank 64 27 us (3.1 TB/s of x), 16384 x 4096 at rank 16 30 us
// (4.5); of the reads of x alone, in any order, 16384 x 4096 took 25 to 34 us.
// SH_APPLY serves small batches, which wait for launches and round trips more
// than for bytes: gridDim.y workgroups each make the same h, keep it in LDS and go
// through their share of y's columns as k_lora_expand does; a wave's first rows and
// adapter columns are read before h is made.
template <int RT, int MT, int MODE>
__global__ __launch_bounds__(SH_WAVES * kWave) void k_lora_shrink(ShrinkArgs g) {
    constexpr int NW = SH_WAVES, COLS = shrink_cols(RT, MT), P = COLS / 8;
    constexpr int LOADS = P / 4, ROWS = 64 / P;  // loads of 16 rows, rows of a load
    constexpr bool APPLY = MODE == SH_APPLY, AHEAD = RT <= 4;
    static_assert(!APPLY || MT == 1, "16 places in SH_APPLY");
    __shared__ u32x4 s_h[APPLY ? 64 * RT : 1];  // h of 16 places as put_row lays it out
    __shared__ u32x4 s_stage[NW][(MT + RT) * 16 * P];
    __shared__ int s_tok[16 * MT];
    // 16 places: from the plan's list, which leaves out the empty ones (a workgroup that finds nothing
    // to do still takes the LDS of a whole one)
    const int at = MT == 1 ? g.plan.group[blockIdx.x] : (int)blockIdx.x * MT;
    if ((uint32_t)at >= (uint32_t)g.max_tiles * 4) return;
    const int tile = at >> 2, sub = at & 3;
    const int slot = g.plan.tile_slot[tile];
    if ((uint32_t)slot >= (uint32_t)g.S || sub * 16 >= g.plan.tile_count[tile]) return;
    const int w = __builtin_amdgcn_readfirstlane(wave_id()), l = lane_id(), c16 = l & 15, q = l >> 4;
    const int64_t place0 = (int64_t)at * 16;
    const float scale = g.scales[slot];
    const int lp = l % P, lr = l / P;  // a lane's piece and row in a load
    const uint16_t *const pa = g.a + ((int64_t)slot * g.R + lr) * g.C;
    const uint16_t *px[MT][LOADS];
    int tok[MT][LOADS];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < LOADS; ++i) tok[m][i] = token_of(g.plan.order[place0 + m * 16 + i * ROWS + lr], g.T);
    const int some = __builtin_amdgcn_readfirstlane(tok[0][0]) < 0 ? 0 : __builtin_amdgcn_readfirstlane(tok[0][0]);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            if (w == 0 && lp == 0) s_tok[m * 16 + i * ROWS + lr] = tok[m][i];
            px[m][i] = g.x + (int64_t)(tok[m][i] < 0 ? some : tok[m][i]) * g.ldx;  // an empty place's sums are dropped
        }
    // SH_APPLY: where the rows of places 4 q + i lie (an empty place stands for the first), and a block
    // of 128 columns of them and of the adapter
    const int in = APPLY ? g.plan.tile_count[tile] - sub * 16 : 0, jstride = NW * (int)gridDim.y;
    int jb = (int)blockIdx.y * NW + w;
    int64_t row[4];
    u32x4 yv[4], wv[AHEAD ? RT : 1][4];
    const auto adapter_row = [&](int r) { return g.w + ((int64_t)slot * g.R + (r < g.R ? r : 0)) * g.N; };
    const auto piece = [&](int b) {
        const int base = b * 128, col = base + c16 * 8 < g.N ? base + c16 * 8 : base;
#pragma unroll
        for (int i = 0; i < 4; ++i) yv[i] = ld16(g.y + row[i] + col);
#pragma unroll
        for (int rt = 0; rt < (AHEAD ? RT : 0); ++rt)
#pragma unroll
            for (int i = 0; i < 4; ++i) wv[rt][i] = ld16(adapter_row(rt * 16 + q * 4 + i) + col);
        return col;
    };
    int col = 0;
    if constexpr (APPLY) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = token_of(g.plan.order[place0 + (q * 4 + i < in ? q * 4 + i : 0)], g.T);
            row[i] = (int64_t)(t < 0 ? 0 : t) * g.ldy;
        }
        if (jb * 128 < g.N) col = piece(jb);
    }
    const int steps = (g.C + COLS - 1) / COLS, stride = NW * (MODE == SH_PARTS ? (int)gridDim.y : 1);
    u32x4 xr[MT][LOADS], ar[RT][LOADS];
    auto load = [&](int s) {
        const int k = s * COLS + lp * 8, kc = k < g.C ? k : 0;
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int i = 0; i < LOADS; ++i) {  // (R is a multiple of 8: a load is all ranks or none)
                ar[rt][i] = u32x4{0, 0, 0, 0};
                if (rt * 16 + i * ROWS < g.R) ar[rt][i] = ld16(pa + (int64_t)(rt * 16 + i * ROWS) * g.C + kc);
            }
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int i = 0; i < LOADS; ++i) xr[m][i] = ld16_once(px[m][i] + kc);
        if (s * COLS + COLS > g.C && k >= g.C) {
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                for (int i = 0; i < LOADS; ++i) ar[rt][i] = u32x4{0, 0, 0, 0};
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int i = 0; i < LOADS; ++i) xr[m][i] = u32x4{0, 0, 0, 0};
        }
    };
    f32x4 acc[MT][RT];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) acc[m][rt] = f32x4{0, 0, 0, 0};
    u32x4 *const st = s_stage[w];
    int s = (MODE == SH_PARTS ? (int)blockIdx.y * NW : 0) + w;
    if (s < steps) load(s);
    for (; s < steps; s += stride) {
        __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");  // the last step's reads are done
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int i = 0; i < LOADS; ++i) st[m * 16 * P + staged<P>(i * ROWS + lr, lp)] = xr[m][i];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int i = 0; i < LOADS; ++i) st[(MT + rt) * 16 * P + staged<P>(i * ROWS + lr, lp)] = ar[rt][i];
        __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");  // the lanes' pieces are visible to the wave
        if (s + stride < steps) load(s + stride);
        sched_fence();
#pragma unroll
        for (int k = 0; k < COLS / 32; ++k) {
            u32x4 xv[MT];
#pragma unroll
            for (int m = 0; m < MT; ++m) xv[m] = st[m * 16 * P + staged<P>(c16, k * 4 + q)];
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                const u32x4 av = st[(MT + rt) * 16 * P + staged<P>(c16, k * 4 + q)];
#pragma unroll
                for (int m = 0; m < MT; ++m)
                    acc[m][rt] =
                        __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf(av), as_bf(xv[m]), acc[m][rt], 0, 0, 0);
            }
        }
    }
    __syncthreads();  // the stages are free: the waves' sums go there
    f32x4 *const sums = reinterpret_cast<f32x4 *>(&s_stage[0][0]);
#pragma unroll
    for (int c = 0; c < RT * MT; ++c) sums[(w * RT * MT + c) * kWave + l] = acc[c / RT][c % RT];
    __syncthreads();
    for (int c = w; c < RT * MT; c += NW) {
        f32x4 v = sums[c * kWave + l];
#pragma unroll
        for (int p = 1; p < NW; ++p) v += sums[(p * RT * MT + c) * kWave + l];
        const int m = c / RT, r = (c % RT) * 16 + q * 4;
        const int64_t place = place0 + m * 16 + c16;
        const bool live = s_tok[m * 16 + c16] >= 0 && r < g.R;  // R is a multiple of 8: all four ranks or none
        v = live ? v * scale : f32x4{0, 0, 0, 0};
        if constexpr (MODE == SH_PARTS) {
            *reinterpret_cast<f32x4 *>(g.partial + ((int64_t)blockIdx.y * g.places + place) * (RT * 16) + r) = v;
        } else {
            if (!APPLY || (g.h.rows && blockIdx.y == 0)) store_hidden(g.h, place, g.places, RT * 16, r, v);
            if constexpr (APPLY) put_row(reinterpret_cast<u32x2 *>(s_h), c16, RT, c % RT, q, split4(v));
        }
    }
    if constexpr (APPLY) {
        lds_barrier();
        u32x4 hv[RT];
#pragma unroll
        for (int i = 0; i < RT; ++i) hv[i] = s_h[((c16 < in ? c16 : 0) * RT + i) * 4 + q];
        while (jb * 128 < g.N) {
            f32x4 out[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) out[j] = f32x4{0, 0, 0, 0};
            const auto rows_of = [&](int rt, u32x4 (&v)[4]) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if constexpr (AHEAD) v[i] = wv[rt][i];
                    else v[i] = ld16(adapter_row(rt * 16 + q * 4 + i) + col);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (rt * 16 + q * 4 + i >= g.R) v[i] = u32x4{0, 0, 0, 0};
            };
#pragma unroll
            for (int rt = 0; rt < RT; rt += 2) {  // two tiles at a time
                constexpr int kOne = RT & 1;
                if (rt + 1 < RT) {
                    Columns<2> f;
                    const bool finite = read_columns<2>(f, [&](int i, u32x4(&v)[4]) { rows_of(rt + i, v); });
                    multiply_rows<2>(hv + rt, f, finite, out);
                } else if constexpr (kOne) {
                    Columns<1> f;
                    const bool finite = read_columns<1>(f, [&](int, u32x4(&v)[4]) { rows_of(RT - 1, v); });
                    multiply_rows<1>(hv + RT - 1, f, finite, out);
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                u32x4 o;
#pragma unroll
                for (int d = 0; d < 4; ++d)
                    o[d] = cast_pair(__uint_as_float(yv[i][d] << 16) + out[2 * d][i],
                                     __uint_as_float(yv[i][d] & 0xFFFF0000u) + out[2 * d + 1][i]);
                *reinterpret_cast<u32x4 *>(g.y + row[i] + col) = o;
            }
            jb += jstride;
            if (jb * 128 < g.N) col = piece(jb);
        }
    }
}

// ---- expand: y += W^T h ---------------------------------------------------------
constexpr int EX_TILES = 4;  // most tiles of a workgroup
enum ExpandMode { EX_PLAIN, EX_PARTS, EX_ONCE };  // EX_PARTS: h in parts; EX_ONCE: y past the last-level cache

struct ExpandArgs {
    const uint16_t *h;     // rows of put_row
    const float *partial;  // or its parts [parts][place][Rp] (EX_PARTS)
    const uint16_t *w;     // [S][R][C]
    uint16_t *y;
    int64_t ldy;
    LoraPlan plan;
    int64_t places;
    int32_t T, S, C, R, max_tiles, per, groups;  // per: tiles of a workgroup; groups: workgroups of a column block
    int32_t parts;
};

// What 16 places of a tile need in expand: where a lane's rows of places 4 q + i
// lie, the rows, and h of place c.
template <int RT>
struct ExpandRows {
    int64_t at[4];
    u32x4 y[4];
    u32x4 h[RT];
};

// A wave takes 128 columns of the 64 places of each of its tiles.  Matrix
// instruction: rows = places, columns = columns of y, the ranks of two tiles (of the
// one left over, 16), once for each part of h.  Lane c of the
// column axis holds the 8-column piece c, instruction j its column j: then the
// lane's results i = 0..3 are, for j = 0..7, one 16-byte piece of the row of
// place 4 q + i, and sixteen lanes touch 256 contiguous bytes; neighbouring
// workgroups take neighbouring columns of the same rows.  The rows and h of the
// next 16 places are on their way while these are computed and written, into the
// other of two buffers.  Loads and stores count down one counter in their order,
// so the body has no branch around either: an empty place stands for the first
// of its 16 and a lane past the last column for the wave's first piece, and both
// write again what that one writes.  Bound by reading and writing y: 8192 x 27648 at
// rank 64 170 us (5.3 TB/s; with one part of h 161, with the branches 206 then), 16384 x
// 14336 at rank 16 184 us (5.1; a large copy 5.2).
template <int RT, int MODE>
__global__ __launch_bounds__(256, RT <= 2 ? 3 : (RT <= 4 ? 2 : 1)) void k_lora_expand(ExpandArgs g) {
    const int w = __builtin_amdgcn_readfirstlane(wave_id()), l = lane_id(), c16 = l & 15, q = l >> 4;
    const int blocks = (g.C + 511) / 512;
    const int base = ((int)blockIdx.x % blocks * 4 + w) * 128, col = base + c16 * 8 < g.C ? base + c16 * 8 : base;
    const int ta = (int)blockIdx.x / blocks * g.per, tb = ta + g.per < g.max_tiles ? ta + g.per : g.max_tiles;
    // the tiles' adapters and rows wait in LDS: a load behind the stores of a row would wait for those too
    __shared__ int64_t s_row[EX_TILES * LT];
    __shared__ int32_t s_slot[EX_TILES], s_count[EX_TILES];
    const int ti = (int)threadIdx.x / LT;
    if (ta + ti < tb) {
        s_row[threadIdx.x] = row_of(g.plan.order + (int64_t)ta * LT, threadIdx.x, g.T, g.ldy);
        if (l == 0) {
            s_slot[ti] = g.plan.tile_slot[ta + ti];
            s_count[ti] = g.plan.tile_count[ta + ti];
        }
    }
    __syncthreads();
    if (base >= g.C) return;
    uint16_t *const ycol = g.y + col;
    // a tile's adapter, -1: none, and the number of its tokens
    const auto slot_of = [&](int tile) {
        const int s = tile < tb ? __builtin_amdgcn_readfirstlane(s_slot[tile - ta]) : -1;
        return (uint32_t)s < (uint32_t)g.S ? s : -1;
    };
    const auto count_of = [&](int tile) {
        const int n = __builtin_amdgcn_readfirstlane(s_count[tile - ta]);
        return n < 1 ? 1 : (n < LT ? n : LT);
    };
    const auto read = [&](ExpandRows<RT> &r, int tile, int sub, int count) {
        const int64_t *const row = s_row + (tile - ta) * LT + sub * 16 + q * 4;
        const int in = count - sub * 16;  // places of the 16 that hold a token
        const int64_t place = (int64_t)tile * LT + sub * 16 + (c16 < in ? c16 : 0);
        if constexpr (MODE == EX_PARTS) {
            const float *const at = g.partial + place * (RT * 16) + q * 4;
            f32x4 v[RT];
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) v[rt] = *reinterpret_cast<const f32x4 *>(at + rt * 16);
#pragma unroll 2
            for (int p = 1; p < g.parts; ++p)
#pragma unroll
                for (int rt = 0; rt < RT; ++rt)
                    v[rt] += *reinterpret_cast<const f32x4 *>(at + p * g.places * (RT * 16) + rt * 16);
            row_operands<RT>(v, r.h);
        } else {
#pragma unroll
            for (int i = 0; i < RT; ++i)
                r.h[i] = reinterpret_cast<const u32x4 *>(g.h)[(place * RT + i) * 4 + q];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) r.at[i] = row[i];
#pragma unroll
        for (int i = 0; i < 4; ++i) r.y[i] = MODE == EX_ONCE ? ld16_once(ycol + r.at[i]) : ld16(ycol + r.at[i]);
    };
    int tile = ta, sub = 0, cur = -1, slot = slot_of(ta);
    if (slot < 0) return;
    int count = count_of(ta);
    Columns<RT> w_cols;
    bool finite = true;
    // one step: the next 16 places (or, at the end, these once more) into `next`, these out of `now`
    const auto step = [&](ExpandRows<RT> &now, ExpandRows<RT> &next) {
        int tile1 = tile, sub1 = sub + 1, slot1 = slot, count1 = count;
        if (sub1 * 16 >= count) {
            slot1 = slot_of(tile + 1);
            tile1 = tile + 1;
            sub1 = 0;
            if (slot1 >= 0) count1 = count_of(tile1);
        }
        const bool more = slot1 >= 0;
        if (slot != cur) {
            cur = slot;
            const auto rows_of = [&](int rt, u32x4 (&v)[4]) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = rt * 16 + q * 4 + i;
                    v[i] = ld16(g.w + ((int64_t)slot * g.R + (r < g.R ? r : 0)) * g.C + col);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (rt * 16 + q * 4 + i >= g.R) v[i] = u32x4{0, 0, 0, 0};
            };
            finite = read_columns<RT>(w_cols, rows_of);
        }
        if (MODE != EX_PARTS || more) read(next, more ? tile1 : tile, more ? sub1 : sub, more ? count1 : count);
        sched_fence();
        f32x4 acc[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] = f32x4{0, 0, 0, 0};
        multiply_rows<RT>(now.h, w_cols, finite, acc);
        if (!finite) cur = -1;  // read the adapter anew
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            u32x4 o;
#pragma unroll
            for (int d = 0; d < 4; ++d)
                o[d] = cast_pair(__uint_as_float(now.y[i][d] << 16) + acc[2 * d][i],
                                 __uint_as_float(now.y[i][d] & 0xFFFF0000u) + acc[2 * d + 1][i]);
            u32x4 *const to = reinterpret_cast<u32x4 *>(ycol + now.at[i]);
            if constexpr (MODE == EX_ONCE) __builtin_nontemporal_store(o, to);
            else *to = o;
        }
        tile = tile1, sub = sub1, slot = slot1, count = count1;
        return more;
    };
    ExpandRows<RT> even, odd;
    read(even, tile, 0, count);
    while (step(even, odd) && step(odd, even)) {
    }
}

// ---- outer: G_i = sum over i's tokens of u z^T ------------------------------------
struct OuterSide {
    const uint16_t *part[3];  // u: [Rp][place], its three parts
    const uint16_t *z;        // [tokens][ldz]
    int64_t ldz;
    float *out;               // [S][R][C]
    float *partial;           // [chunks][2][R][C]
    int32_t C;
    int32_t blocks;           // column blocks, one wave each
    int32_t q, chunks;        // tiles of a chunk
};

struct OuterArgs {
    OuterSide side[2];
    LoraPlan plan;
    int64_t places;
    int32_t T, R, S, max_tiles;
    int32_t accumulate, wg0;  // wg0: workgroups of side 0 per chunk
    int32_t clear;            // set where k_lora_outer_sum does not follow: zero the adapters without tokens
    int32_t groups;           // of a workgroup's four waves, those that share its columns: one for two rank tiles
    const uint16_t *w;        // FUSE: [S][R][C] what shrink multiplies z with
    float *sums;              // FUSE: [workgroups of a chunk][32 places][512 RT] their sums, as the lanes hold them
};

constexpr int OU_TILES = 32;  // most tiles of a chunk

// What 32 places need in outer: a lane's eight columns of eight rows, and u where
// the registers hold it twice (AHEAD).
template <int RT, bool AHEAD>
struct OuterRows {
    u32x4 z[8];
    u32x4 u[3][AHEAD ? RT : 1];
};

// A wave takes 128 columns, RT tiles of 16 ranks and one chunk of tiles, 32 places
// at a time; the next 32 places' rows are on their way meanwhile, into the other of
// two buffers.  The waves of a workgroup that differ in their ranks only read the
// same rows, three of four times from the nearest cache.  Matrix instruction: rows
// = ranks, columns = columns of z, 32 places.  Lane c of the column axis holds eight
// neighbouring columns of eight places, transposed in registers; instruction j takes
// its column j, once for each part of u (rows that are not all finite: the lower parts
// with ones for infinities; finding that out is 64 vector instructions of a step, which
// waits for its rows).  A chunk may cover several adapters and an
// adapter several chunks: a run that lies in one chunk goes straight to the output,
// the others to the chunk's partial sums (0: continues an earlier chunk's run, 1:
// begins here), which k_lora_outer_sum adds in order.
// 16384 x 4096 at rank 16: 31 us, 4.3 TB/s.
// FUSE: z is dy, and the same read serves dh = s B dy: the rows go through LDS
// into the order that shrink multiplies them in, the eight waves' sums over 128
// columns each are added there, and k_lora_join adds the workgroups'.  16384 x 14336
// at rank 16: 106 us, 4.4 TB/s, and 5.5 us for the join (dy read twice: 137 + 105 us);
// leaving out either product changes nothing, it waits for the rows.
template <int RT, bool FUSE>
__global__ __launch_bounds__(FUSE ? 512 : 256, FUSE ? 1 : 2) void k_lora_outer(OuterArgs g) {
    constexpr int NW = FUSE ? 8 : 4, W = 8;
    constexpr bool AHEAD = RT == 1;
    typedef OuterRows<RT, AHEAD> Rows;
    __shared__ int64_t s_row[OU_TILES * LT];
    __shared__ int32_t s_slot[OU_TILES], s_count[OU_TILES];
    __shared__ u32x4 s_stage[FUSE ? NW : 1][FUSE ? 512 : 1];
    __shared__ f32x4 s_sum[FUSE ? 2 : 1][FUSE ? NW : 1][FUSE ? 128 * RT : 1];
    const int w = __builtin_amdgcn_readfirstlane(wave_id()), l = lane_id(), c16 = l & 15, q = l >> 4;
    const int sd = (int)blockIdx.x >= g.wg0 ? 1 : 0;
    const OuterSide &s = g.side[sd];
    const int chunk = blockIdx.y, ta = chunk * s.q;
    const int ntiles = *g.plan.ntiles < g.max_tiles ? *g.plan.ntiles : g.max_tiles;
    const int tb = ta + s.q < ntiles ? ta + s.q : ntiles;
    if (chunk >= s.chunks || (ta >= tb && !g.clear)) return;
    for (int i = threadIdx.x; i < (tb - ta) * LT; i += NW * kWave) {
        s_row[i] = row_of(g.plan.order + (int64_t)ta * LT, i, g.T, s.ldz);
        if (i < tb - ta) {
            s_slot[i] = g.plan.tile_slot[ta + i];
            s_count[i] = g.plan.tile_count[ta + i];
        }
    }
    __syncthreads();
    const int groups = FUSE ? 1 : g.groups, r0 = w % groups * RT * 16;  // the wave's first rank
    const int cb = ((int)blockIdx.x - (sd ? g.wg0 : 0)) * (NW / groups) + w / groups, base = cb * 128, col = base + c16 * 8;
    if (!FUSE && (cb >= s.blocks || r0 >= g.R)) return;  // (FUSE: the wave still meets the others at their barriers)
    int64_t urow[RT];  // the lane's rank of each tile in u; past u's last tile: that one's
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) urow[rt] = (int64_t)((r0 + rt * 16 < g.R ? r0 + rt * 16 : r0) + c16) * g.places;
    const bool colok = col < s.C;
    const uint16_t *const zcol = s.z + (colok ? col : (base < s.C ? base : 0));
    const auto slot_of = [&](int tile) {
        const int v = tile < tb ? __builtin_amdgcn_readfirstlane(s_slot[tile - ta]) : -1;
        return (uint32_t)v < (uint32_t)g.S ? v : -1;
    };
    const auto count_of = [&](int tile) {
        const int n = __builtin_amdgcn_readfirstlane(s_count[tile - ta]);
        return n < 1 ? 1 : (n < LT ? n : LT);
    };
    if (g.clear && chunk == 0) {  // one chunk only: the adapters without a token have no other launch
        for (int a = 0; a < g.S; ++a) {
            if (g.plan.slot_tile[a] != g.plan.slot_tile[a + 1]) continue;
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = r0 + rt * 16 + q * 4 + i;
                    float *p = s.out + ((int64_t)a * g.R + r) * s.C + col;
                    if (r < g.R && colok) {
                        *reinterpret_cast<f32x4 *>(p) = f32x4{0, 0, 0, 0};
                        *reinterpret_cast<f32x4 *>(p + 4) = f32x4{0, 0, 0, 0};
                    }
                }
        }
    }
    f32x4 acc[RT][W];
    const auto flush = [&](int slot) __attribute__((always_inline)) {
        const int t0 = g.plan.slot_tile[slot], t1 = g.plan.slot_tile[slot + 1];
        const bool direct = t0 / s.q == (t1 - 1) / s.q;
        float *o = direct ? s.out + (int64_t)slot * g.R * s.C
                          : s.partial + ((int64_t)chunk * 2 + (t0 >= ta ? 1 : 0)) * g.R * s.C;
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = r0 + rt * 16 + q * 4 + i;
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
    const auto read = [&](Rows &r, int tile, int half) __attribute__((always_inline)) {
        const int64_t *const row = s_row + (tile - ta) * LT + half * 32 + q * 8;
        const int64_t place = (int64_t)tile * LT + half * 32 + q * 8;
        int64_t at[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) at[i] = row[i];
#pragma unroll
        for (int i = 0; i < 8; ++i) r.z[i] = ld16_once(zcol + at[i]);
        if constexpr (AHEAD) {
#pragma unroll
            for (int p = 0; p < 3; ++p)
#pragma unroll
                for (int rt = 0; rt < RT; ++rt)
                    r.u[p][rt] = ld16(s.part[p] + urow[rt] + place);
        }
    };
    if (ta >= tb) return;
    int tile = ta, half = 0, cur = -1, slot = slot_of(ta), buf = 0;
    if (slot < 0) return;
    int count = count_of(ta);
    u32x4 wf[FUSE ? 4 : 1][RT];
    // one step: the next 32 places (or, at the end, these once more) into `next`, these out of `now`
    const auto step = [&](Rows &now, Rows &next) __attribute__((always_inline)) {
        int tile1 = tile, half1 = 1, slot1 = slot, count1 = count;
        if (half == 1 || count <= 32) {
            tile1 = tile + 1;
            half1 = 0;
            slot1 = slot_of(tile1);
            if (slot1 >= 0) count1 = count_of(tile1);
        }
        const bool more = slot1 >= 0;
        if (slot != cur) {
            if (cur >= 0) flush(cur);
            cur = slot;
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                for (int j = 0; j < W; ++j) acc[rt][j] = f32x4{0, 0, 0, 0};
            if constexpr (FUSE) {
#pragma unroll
                for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int r = rt * 16 + c16, c = base + (k * 4 + q) * 8;
                        wf[k][rt] = u32x4{0, 0, 0, 0};
                        if (r < g.R && c < s.C) wf[k][rt] = ld16(g.w + ((int64_t)slot * g.R + r) * s.C + c);
                    }
            }
        }
        u32x4 u[3][RT];
#pragma unroll
        for (int p = 0; p < 3; ++p)
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                if constexpr (AHEAD) u[p][rt] = now.u[p][rt];
                else u[p][rt] = ld16(s.part[p] + urow[rt] + (int64_t)tile * LT + half * 32 + q * 8);
            }
        read(next, more ? tile1 : tile, more ? half1 : half);
        sched_fence();
        const int left = count - half * 32;
        if (left < 32) {  // empty places: no row, and past the last 16 that hold a token no u
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (q * 8 + i >= left) now.z[i] = u32x4{0, 0, 0, 0};
            const bool none = q * 8 >= (left + 15) / 16 * 16;
#pragma unroll
            for (int p = 0; p < 3; ++p)
#pragma unroll
                for (int rt = 0; rt < RT; ++rt)
                    if (none) u[p][rt] = u32x4{0, 0, 0, 0};
        }
        if constexpr (FUSE) {
            if (base + 128 > s.C && !colok) {
#pragma unroll
                for (int i = 0; i < 8; ++i) now.z[i] = u32x4{0, 0, 0, 0};
            }
            u32x4 *const st = s_stage[w];
            __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
#pragma unroll
            for (int i = 0; i < 8; ++i) st[staged(q * 8 + i, c16)] = now.z[i];
            __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
        }
        u32x4 zt[W];
#pragma unroll
        for (int j = 0; j < W; ++j)
#pragma unroll
            for (int d = 0; d < 4; ++d)
                zt[j][d] = __builtin_amdgcn_perm(now.z[2 * d + 1][j >> 1], now.z[2 * d][j >> 1],
                                                 (j & 1) ? 0x07060302u : 0x05040100u);
        const auto part = [&](int p) __attribute__((always_inline)) {
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                for (int j = 0; j < W; ++j)
                    acc[rt][j] =
                        __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf(u[p][rt]), as_bf(zt[j]), acc[rt][j], 0, 0, 0);
        };
        part(0);
        uint32_t most = 0;
#pragma unroll
        for (int j = 0; j < W; ++j)
#pragma unroll
            for (int d = 0; d < 4; ++d) most = most_of(most, zt[j][d]);
        if (__ballot(not_finite(most))) {
#pragma unroll
            for (int j = 0; j < W; ++j)
#pragma unroll
                for (int d = 0; d < 4; ++d) zt[j][d] = ones_for_infinities(zt[j][d]);
        }
        part(1);
        part(2);
        if constexpr (FUSE) {
            u32x4 *const st = s_stage[w];
            f32x4 sum[2][RT];
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) sum[m][rt] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    const u32x4 zv = st[staged(m * 16 + c16, k * 4 + q)];
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt)
                        sum[m][rt] =
                            __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf(wf[k][rt]), as_bf(zv), sum[m][rt], 0, 0, 0);
                }
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) s_sum[buf][w][(m * RT + rt) * kWave + l] = sum[m][rt];
            lds_barrier();  // the one barrier of a step: the other buffer's sums were read before it
            const float *in = reinterpret_cast<const float *>(&s_sum[buf][0][0]);
            float *out = g.sums + ((int64_t)blockIdx.x * (g.max_tiles * 2) + tile * 2 + half) * (512 * RT);
#pragma unroll
            for (int k = 0; k < RT; ++k) {
                const int e = k * 512 + (int)threadIdx.x;
                float v = in[e];
#pragma unroll
                for (int p = 1; p < NW; ++p) v += in[p * 512 * RT + e];
                out[e] = v;
            }
            buf ^= 1;
        }
        tile = tile1, half = half1, slot = slot1, count = count1;
        return more;
    };
    Rows even, odd;
    read(even, tile, 0);
    while (step(even, odd) && step(odd, even)) {
    }
    flush(cur);
}

// dh of 32 places from the fused pass's sums, a workgroup's after the other.
template <int RT>
__global__ __launch_bounds__(128 * RT) void k_lora_join(const float *__restrict__ sums, int32_t parts,
                                                        const float *__restrict__ scales, LoraPlan plan, LoraHidden h,
                                                        int32_t max_tiles, int32_t S, int32_t R) {
    const int tile = blockIdx.x >> 1, half = blockIdx.x & 1, slot = plan.tile_slot[tile];
    if ((uint32_t)slot >= (uint32_t)S) return;
    const int left = plan.tile_count[tile] - half * 32;
    if (left <= 0) return;
    const f32x4 *in = reinterpret_cast<const f32x4 *>(sums) + (int64_t)blockIdx.x * (128 * RT) + threadIdx.x;
    const float scale = scales[slot];
    f32x4 v = {0, 0, 0, 0};
#pragma unroll 8
    for (int p = 0; p < parts; ++p) v += in[(int64_t)p * (max_tiles * 2) * (128 * RT)];
    const int lane = threadIdx.x & 63, c = threadIdx.x >> 6, place = c / RT * 16 + (lane & 15);
    const int r = c % RT * 16 + (lane >> 4) * 4;
    v = place < left && r < R ? v * scale : f32x4{0, 0, 0, 0};
    store_hidden(h, (int64_t)blockIdx.x * 32 + place, (int64_t)max_tiles * LT, RT * 16, r, v);
}

// The gradients of adapters that lie in several chunks: their partial sums in
// the chunks' order; adapters without tokens: zero.
__global__ __launch_bounds__(256) void k_lora_outer_sum(OuterArgs g) {
    const OuterSide &s = g.side[blockIdx.z];
    const int slot = blockIdx.y;
    const int t0 = g.plan.slot_tile[slot], t1 = g.plan.slot_tile[slot + 1];
    const int64_t n = (int64_t)g.R * s.C;
    const int64_t e = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (e >= n || (t1 > t0 && t0 / s.q == (t1 - 1) / s.q) || (t1 == t0 && g.accumulate)) return;
    float *o = s.out + (int64_t)slot * n + e;
    f32x4 v = {0, 0, 0, 0};
    if (t1 > t0) {
        const int c0 = t0 / s.q, c1 = (t1 - 1) / s.q < s.chunks ? (t1 - 1) / s.q : s.chunks - 1;
        if (g.accumulate) v = *reinterpret_cast<const f32x4 *>(o);
#pragma unroll 4
        for (int c = c0 < 0 ? 0 : c0; c <= c1; ++c)
            v += *reinterpret_cast<const f32x4 *>(s.partial + ((int64_t)c * 2 + (c == c0 ? 1 : 0)) * n + e);
    }
    *reinterpret_cast<f32x4 *>(o) = v;
}

// ---- launches ---------------------------------------------------------------------
int64_t lora_outer_blocks(int64_t C) { return (C + 127) / 128; }

// Waves that share a column block: one for each two rank tiles (three: a fourth stays idle).
int lora_outer_groups(int64_t R) { return R <= 32 ? 1 : (R <= 64 ? 2 : 4); }

// Tiles of a chunk in outer: up to 1024 waves in all, one workgroup a compute unit
// (16384 x 4096 at rank 16: 29 us with 232 workgroups, 40 with 296, 41 with 512),
// and enough tokens that the partial sums, 4 R bytes a column, weigh no more than
// the rows, 2 bytes a token and column; up to 6 tiles one chunk, which needs no sum.
int lora_chunk(int64_t T, int64_t S, int64_t R, int64_t waves) {
    const int64_t mt = lora_max_tiles(T, S), q = (mt * waves + 1023) / 1024;
    const int64_t least = mt <= 6 ? 6 : (R > 64 ? R / 32 : 2);
    return (int)(q < least ? least : (q > OU_TILES ? OU_TILES : q));
}

// The backward pass reads dy once, for dh and dB together, where that saves more
// than it costs: from 64 MB of dy on (below, dy comes from the caches the second
// time and the launch more is felt), and to rank 32 (two rank tiles: the sums of
// more leave no registers to read ahead).  Backward with it and without, ranks 16 and
// 32: 16384 tokens, 4096 to 14336, 204 us and 303, 236 and 345; 4096 tokens of 4
// adapters, 14336 to 8200, 101 and 125, 129 and 152; 2100 tokens, 4096 to 16392, 56 and
// 63, 69 and 81; at 64 MB, 8192 tokens, 4096 to 4096, 79 and 77, 96 and 94 for one
// adapter, 79 and 84, 106 and 105 for 16.
bool lora_fused(int64_t T, int64_t N, int64_t R) { return R <= 32 && T * N >= (int64_t)1 << 25; }

int64_t lora_fused_groups(int64_t N) { return (N + 1023) / 1024; }

// Tiles of a chunk in the fused pass: one workgroup a compute unit, in one or two
// rounds, whichever comes to fewer tiles one after the other.
int lora_fused_chunk(int64_t T, int64_t S, int64_t N) {
    const int64_t mt = lora_max_tiles(T, S), groups = lora_fused_groups(N);
    int64_t best = OU_TILES, cost = INT64_MAX;
    for (int64_t rounds = 1; rounds <= 2; ++rounds) {
        const int64_t chunks = 256 * rounds / groups > 1 ? 256 * rounds / groups : 1, q = (mt + chunks - 1) / chunks;
        if (q <= OU_TILES && q * rounds < cost) best = q, cost = q * rounds;
    }
    return (int)best;
}

int64_t lora_chunks(int64_t T, int64_t S, int q) { return (lora_max_tiles(T, S) + q - 1) / q; }

// Most chunks of this T and every smaller one.  Outer alone: 2 tiles each, and what
// makes 1024 waves, or OU_TILES tiles each.  Fused: two rounds, or OU_TILES tiles.
int64_t lora_most_chunks(int64_t T, int64_t S, int64_t waves) {
    const int64_t mt = lora_max_tiles(T, S), a = mt / 2 + 1, b = 1024 / waves + 2, c = mt / OU_TILES + 1;
    const int64_t m = a < b ? a : b;
    return m > c ? m : c;
}

int64_t lora_most_fused_chunks(int64_t T, int64_t S, int64_t N) {
    const int64_t a = 512 / lora_fused_groups(N) + 1, b = lora_max_tiles(T, S) / OU_TILES + 1;
    return a > b ? a : b;
}

template <int RT, int MT, int MODE>
void launch_shrink_rt(const ShrinkArgs &g, int parts, hipStream_t stream) {
    const dim3 grid((unsigned)(MT == 1 ? g.max_groups : g.max_tiles * (4 / MT)), (unsigned)parts);
    k_lora_shrink<RT, MT, MODE><<<grid, dim3(SH_WAVES * kWave), 0, stream>>>(g);
}

// (one rank tile always takes 16 places, and eight leave room in LDS for no more)
template <int MT, int MODE>
void launch_shrink(const ShrinkArgs &g, int parts, int rt, hipStream_t stream) {
    switch (rt) {
    case 1: launch_shrink_rt<1, 1, MODE>(g, parts, stream); break;
    case 2: launch_shrink_rt<2, MT, MODE>(g, parts, stream); break;
    case 3: launch_shrink_rt<3, MT, MODE>(g, parts, stream); break;
    case 4: launch_shrink_rt<4, MT, MODE>(g, parts, stream); break;
    case 5: launch_shrink_rt<5, MT, MODE>(g, parts, stream); break;
    case 6: launch_shrink_rt<6, MT, MODE>(g, parts, stream); break;
    case 7: launch_shrink_rt<7, MT, MODE>(g, parts, stream); break;
    default: launch_shrink_rt<8, 1, MODE>(g, parts, stream);
    }
}

template <int MODE>
void launch_expand(const ExpandArgs &g, int rt, hipStream_t stream) {
    const int64_t blocks = ((int64_t)g.C + 511) / 512;
    const dim3 grid((unsigned)(blocks * g.groups)), block(256);
    switch (rt) {
    case 1: k_lora_expand<1, MODE><<<grid, block, 0, stream>>>(g); break;
    case 2: k_lora_expand<2, MODE><<<grid, block, 0, stream>>>(g); break;
    case 3: k_lora_expand<3, MODE><<<grid, block, 0, stream>>>(g); break;
    case 4: k_lora_expand<4, MODE><<<grid, block, 0, stream>>>(g); break;
    case 5: k_lora_expand<5, MODE><<<grid, block, 0, stream>>>(g); break;
    case 6: k_lora_expand<6, MODE><<<grid, block, 0, stream>>>(g); break;
    case 7: k_lora_expand<7, MODE><<<grid, block, 0, stream>>>(g); break;
    default: k_lora_expand<8, MODE><<<grid, block, 0, stream>>>(g); break;
    }
}

// Workgroups that share the long axis in a forward pass that keeps no h: as many
// as bring the groups of 16 places that hold a token to about 256, one step a wave
// or more.  Each writes its own part of h, which expand adds up.
int lora_parts(int64_t T, int64_t S, int64_t C, int64_t R) {
    const int64_t groups = (T + 15) / 16 + (S < T ? S : T);
    const int64_t waves = SH_WAVES, cols = shrink_cols((int)((R + 15) / 16), 1);
    const int64_t most = (C + cols - 1) / cols / waves, parts = 256 / groups < most ? 256 / groups : most;
    return (int)(parts < 1 ? 1 : (parts > 8 ? 8 : parts));
}

void launch_outer(const OuterArgs &g, int64_t wgs, int64_t chunks, hipStream_t stream) {
    const dim3 grid((unsigned)wgs, (unsigned)chunks), block(256);
    if (g.R <= 16) k_lora_outer<1, false><<<grid, block, 0, stream>>>(g);
    else k_lora_outer<2, false><<<grid, block, 0, stream>>>(g);
}

// Bytes of h's parts, for this T and every smaller one.  Parts are made where the
// groups of 16 places come to 128 or fewer: then there are 128 tiles or fewer, and
// groups times parts come to 256 or fewer, of at most 64 places each.
int64_t lora_parts_size(int64_t T, int64_t S, int64_t R) {
    const int64_t rp = (R + 15) / 16 * 16, mt = lora_max_tiles(T, S), n = mt * 8 < 256 ? mt * 8 : 256;
    return n * LT * rp * 4;
}

int64_t round256(int64_t n) { return (n + 255) / 256 * 256; }

}  // namespace pulse

using namespace pulse;

extern "C" int64_t pulse_lora_plan_size(int64_t T, int64_t S) { return lora_plan_size(T, S); }

extern "C" int64_t pulse_lora_hidden_size(int64_t T, int64_t S, int64_t R) { return lora_hidden_size(T, S, R, true); }

// Workspace: h of a forward pass, whole or in parts, or in a backward pass dh, the
// partial sums of dA and dB, and of dh where it comes from the fused pass.
struct LoraWs {
    int64_t da, db, sums, bytes;
};

LoraWs lora_ws(int64_t T, int64_t K, int64_t N, int64_t R, int64_t S, bool train) {
    LoraWs w{};
    int64_t n = round256(lora_hidden_size(T, S, R, train));
    if (n < lora_parts_size(T, S, R)) n = round256(lora_parts_size(T, S, R));
    if (train) {
        const bool fused = lora_fused(T, N, R);
        const int64_t each = lora_outer_groups(R), k = lora_outer_blocks(K) * each;
        const int64_t both = lora_most_chunks(T, S, k + lora_outer_blocks(N) * each);
        const int64_t da = fused ? lora_most_chunks(T, S, k) : both, db = fused ? lora_most_fused_chunks(T, S, N) : 0;
        w.da = n;
        n += round256(da * 2 * R * K * 4);  // (fewer column blocks, more chunks: da >= both)
        w.db = n;
        n += round256((both > db ? both : db) * 2 * R * N * 4);
        w.sums = n;
        if (fused) n += lora_fused_groups(N) * lora_max_tiles(T, S) * LT * ((R + 15) / 16 * 16) * 4;
    }
    w.bytes = n;
    return w;
}

extern "C" int64_t pulse_lora_ws_size(int64_t T, int64_t K, int64_t N, int64_t R, int64_t S, int32_t train) {
    return lora_ws(T, K, N, R, S, train != 0).bytes;
}

extern "C" int pulse_launch_lora_plan(const int32_t *ids, int64_t T, int32_t S, void *plan, uint32_t *d_status,
                                      hipStream_t stream) {
    // sixteen waves where their counts of all adapters stay below 64 KB of LDS
    const LoraPlan p = lora_plan_parts(plan, T, S);
    const int32_t mt = (int32_t)lora_max_tiles(T, S), mg = (int32_t)lora_max_groups(T, S);
    if (S <= 512)
        k_lora_plan<16><<<dim3(1), dim3(1024), (size_t)19 * S * 4, stream>>>(ids, (int32_t)T, S, p, mt, mg, d_status);
    else k_lora_plan<8><<<dim3(1), dim3(512), (size_t)11 * S * 4, stream>>>(ids, (int32_t)T, S, p, mt, mg, d_status);
    return hipGetLastError() == hipSuccess ? 0 : -5;
}

namespace {

ShrinkArgs shrink_args(const uint16_t *x, int64_t ldx, const uint16_t *a, const float *scales, const LoraPlan &plan,
                       const LoraHidden &h, int64_t T, int64_t C, int64_t R, int64_t S) {
    ShrinkArgs g{};
    g.max_tiles = (int32_t)lora_max_tiles(T, S);
    g.max_groups = (int32_t)lora_max_groups(T, S);
    g.x = x;
    g.ldx = ldx;
    g.a = a;
    g.scales = scales;
    g.plan = plan;
    g.h = h;
    g.places = (int64_t)g.max_tiles * LT;
    g.T = (int32_t)T;
    g.S = (int32_t)S;
    g.C = (int32_t)C;
    g.R = (int32_t)R;
    return g;
}

// h goes to its forms, or with parts > 1 to `partial`
void shrink(const uint16_t *x, int64_t ldx, const uint16_t *a, const float *scales, const LoraPlan &plan,
            const LoraHidden &h, float *partial, int parts, int64_t T, int64_t C, int64_t R, int64_t S,
            hipStream_t stream) {
    const int rt = (int)((R + 15) / 16);
    ShrinkArgs g = shrink_args(x, ldx, a, scales, plan, h, T, C, R, S);
    g.partial = partial;
    // 32 places a workgroup, so that the adapter is read half as often, once that still makes a workgroup
    // for each of the 256 compute units and few adapters end in the first half of a tile: 8192 x 5120 at
    // rank 64 37 us with 16 places, 27 with 32; at rank 16 or less the adapter weighs little (16384 x 4096
    // at rank 16: 29 us, 39)
    if (parts > 1) launch_shrink<1, SH_PARTS>(g, parts, rt, stream);
    else if (rt >= 2 && T / 32 >= 256 && T / S >= 128) launch_shrink<2, SH_WHOLE>(g, 1, rt, stream);
    else launch_shrink<1, SH_WHOLE>(g, 1, rt, stream);
}

// Workgroups of 16 places in SH_APPLY, or 0 where h and y take a launch each: for
// more than 256 groups or 4 blocks of 128 columns a wave (the second launch then
// spreads over more of the chip), where the adapter, which every workgroup reads,
// comes to more than 48 MB in all (96 tokens of 64 adapters, 5120 to 7168, rank 32:
// 69 MB, 16.4 us against 14.6; 64 tokens, 4096 to 4096, rank 16: 18 MB, 9.1 us
// against 9.8 and one launch less), and where h's long axis can be shared and one
// workgroup would read long (4 tokens, 4096 to 4096, rank 128: 1 MB, 22 us against 14).
// Both ways at 190 sizes (1 to 600 tokens of 8 to 64 adapters, ranks 8 to 128, five pairs
// of widths): the rule's choice is within an eighth of the better one but for 17, the
// largest of them 14336 to 4096 at rank 8 (224 KB; 12 us against 9, 600 tokens 23 against
// 14) and 64 adapters of rank 128 (4096 to 14336, two launches: 51 us against 41).
int64_t lora_apply_groups(int64_t T, int64_t S, int64_t C, int64_t N, int64_t R, bool shared) {
    const int64_t groups = lora_max_groups(T, S), waves = SH_WAVES;
    if (groups > 256 || (shared && R * C * 2 > 384 << 10)) return 0;
    const int64_t blocks = (N + 127) / 128, most = (blocks + waves - 1) / waves;
    const int64_t n = 256 / groups < most ? 256 / groups : most;
    return blocks <= n * waves * 4 && groups * n * R * C * 2 <= 48 << 20 ? n : 0;
}

// h and y += W^T h in one launch
void apply(const uint16_t *x, int64_t ldx, const uint16_t *a, const float *scales, const LoraPlan &plan,
           const LoraHidden &h, const uint16_t *w, uint16_t *y, int64_t ldy, int64_t groups, int64_t T, int64_t C,
           int64_t N, int64_t R, int64_t S, hipStream_t stream) {
    ShrinkArgs g = shrink_args(x, ldx, a, scales, plan, h, T, C, R, S);
    g.w = w;
    g.y = y;
    g.ldy = ldy;
    g.N = (int32_t)N;
    launch_shrink<1, SH_APPLY>(g, (int)groups, (int)((R + 15) / 16), stream);
}

void expand(const uint16_t *h, const float *partial, int parts, const uint16_t *w, uint16_t *y, int64_t ldy,
            const LoraPlan &plan, int64_t T, int64_t C, int64_t R, int64_t S, hipStream_t stream) {
    ExpandArgs g{};
    g.h = h;
    g.partial = partial;
    g.w = w;
    g.y = y;
    g.ldy = ldy;
    g.plan = plan;
    g.T = (int32_t)T;
    g.S = (int32_t)S;
    g.C = (int32_t)C;
    g.R = (int32_t)R;
    g.parts = parts;
    g.max_tiles = (int32_t)lora_max_tiles(T, S);
    g.places = (int64_t)g.max_tiles * LT;
    // tiles of a workgroup, whose adapter is then read and transposed once: up to EX_TILES, 2048 workgroups or more
    const int64_t per = g.max_tiles * ((C + 511) / 512) / 2048;
    g.per = (int32_t)(per < 1 ? 1 : (per > EX_TILES ? EX_TILES : per));
    g.groups = (g.max_tiles + g.per - 1) / g.per;
    const int rt = (int)((R + 15) / 16);
    // From 128 MB on y would not be in the last-level cache any more when the next kernel reads it, and
    // its lines would wait there to be written back: 8192 x 27648 at rank 64 173 us, past the cache 162;
    // forward and backward of 16384 x 14336 at rank 16 446 us, 434.
    if (parts > 1) launch_expand<EX_PARTS>(g, rt, stream);
    else if (T * C >= (int64_t)1 << 26) launch_expand<EX_ONCE>(g, rt, stream);
    else launch_expand<EX_PLAIN>(g, rt, stream);
}

}  // namespace

extern "C" int pulse_launch_lora_forward(const uint16_t *x, int64_t ldx, const uint16_t *a, const uint16_t *b,
                                         const float *scales, const void *plan, int64_t T, int64_t K, int64_t N, int64_t R,
                                         int64_t S, uint16_t *y, int64_t ldy, void *h, void *ws, hipStream_t stream) {
    const LoraPlan p = lora_plan_parts(const_cast<void *>(plan), T, S);
    const LoraHidden hp = lora_hidden_parts(h ? h : ws, T, S, R, h != nullptr);
    const int parts = h ? 1 : lora_parts(T, S, K, R);
    if (const int64_t groups = lora_apply_groups(T, S, K, N, R, parts > 1)) {
        const LoraHidden keep = h ? hp : LoraHidden{};
        apply(x, ldx, a, scales, p, keep, b, y, ldy, groups, T, K, N, R, S, stream);
        return hipGetLastError() == hipSuccess ? 0 : -5;
    }
    float *partial = static_cast<float *>(ws);
    shrink(x, ldx, a, scales, p, hp, partial, parts, T, K, R, S, stream);
    expand(hp.rows, partial, parts, b, y, ldy, p, T, N, R, S, stream);
    return hipGetLastError() == hipSuccess ? 0 : -5;
}

extern "C" int pulse_launch_lora_backward(const uint16_t *x, int64_t ldx, const uint16_t *dy, int64_t lddy,
                                          const uint16_t *a, const uint16_t *b, const float *scales, const void *plan,
                                          int64_t T, int64_t K, int64_t N, int64_t R, int64_t S, const void *h,
                                          uint16_t *dx, int64_t lddx, float *da, float *db, int32_t accumulate,
                                          void *ws, hipStream_t stream) {
    const LoraPlan p = lora_plan_parts(const_cast<void *>(plan), T, S);
    const LoraWs at = lora_ws(T, K, N, R, S, true);
    char *const w = static_cast<char *>(ws);
    const LoraHidden dh = lora_hidden_parts(w, T, S, R, true), hp = lora_hidden_parts(const_cast<void *>(h), T, S, R, true);
    const int rt = (int)((R + 15) / 16);
    const auto outer_side = [&](const LoraHidden &u, const uint16_t *z, int64_t ldz, float *out, int64_t partial, int64_t C,
                                int q) {
        return OuterSide{{u.part[0], u.part[1], u.part[2]}, z, ldz, out, reinterpret_cast<float *>(w + partial), (int32_t)C,
                         (int32_t)lora_outer_blocks(C), q, (int32_t)lora_chunks(T, S, q)};
    };
    const bool fused = lora_fused(T, N, R);
    const int64_t kb = lora_outer_blocks(K), nb = lora_outer_blocks(N);
    const int groups = lora_outer_groups(R), per = 4 / groups;  // column blocks of a workgroup
    const int q = lora_chunk(T, S, R, (fused ? kb : kb + nb) * groups);
    OuterArgs g{};
    g.plan = p;
    g.max_tiles = (int32_t)lora_max_tiles(T, S);
    g.places = (int64_t)g.max_tiles * LT;
    g.T = (int32_t)T;
    g.R = (int32_t)R;
    g.S = (int32_t)S;
    g.accumulate = accumulate;
    g.side[0] = outer_side(dh, x, ldx, da, at.da, K, q);
    g.side[1] = outer_side(hp, dy, lddy, db, at.db, N, fused ? lora_fused_chunk(T, S, N) : q);
    if (fused) {
        g.w = b;
        g.sums = reinterpret_cast<float *>(w + at.sums);
        const int32_t parts = (int32_t)lora_fused_groups(N);
        const dim3 grid((unsigned)parts, (unsigned)g.side[1].chunks), tiles((unsigned)g.max_tiles * 2);
        if (rt == 1) {
            k_lora_outer<1, true><<<grid, dim3(512), 0, stream>>>(g);
            k_lora_join<1><<<tiles, dim3(128), 0, stream>>>(g.sums, parts, scales, p, dh, g.max_tiles, g.S, g.R);
        } else {
            k_lora_outer<2, true><<<grid, dim3(512), 0, stream>>>(g);
            k_lora_join<2><<<tiles, dim3(256), 0, stream>>>(g.sums, parts, scales, p, dh, g.max_tiles, g.S, g.R);
        }
    } else if (const int64_t n = dx ? lora_apply_groups(T, S, N, K, R, false) : 0) {
        apply(dy, lddy, b, scales, p, dh, a, dx, lddx, n, T, N, K, R, S, stream);
        dx = nullptr;
    } else {
        shrink(dy, lddy, b, scales, p, dh, nullptr, 1, T, N, R, S, stream);
    }
    if (dx) expand(dh.rows, nullptr, 1, a, dx, lddx, p, T, K, R, S, stream);
    g.groups = groups;
    g.wg0 = (g.side[0].blocks + per - 1) / per;
    const int wgs = g.wg0 + (fused ? 0 : (g.side[1].blocks + per - 1) / per);
    // one chunk of a few adapters: every sum is whole, and the launch that would add parts is left out
    const bool whole = !fused && g.side[0].chunks == 1 && S <= 64;
    g.clear = whole && !accumulate;
    launch_outer(g, wgs, g.side[0].chunks, stream);
    if (whole) return hipGetLastError() == hipSuccess ? 0 : -5;
    const int64_t most = R * (K > N ? K : N);
    k_lora_outer_sum<<<dim3((unsigned)((most / 4 + 255) / 256), (unsigned)S, 2), dim3(256), 0, stream>>>(g);
    return hipGetLastError() == hipSuccess ? 0 : -5;
}
