// fp8_gemm.hip -- products with the weights that the receiver keeps as E4M3 codes
// in 128 x 128 blocks, of rows whose codes have a scale for each 128 columns.
//
//   nt:  y[m, n]  = sum over blocks b of k of  sx[m, b] sw[n / 128, b]  sum_k x[m, k] w[n, k]   (+ bias[n])
//   nn:  dx[m, k] = sum over blocks b of n of  sx[m, b] sw[b, k / 128]  sum_n x[m, n] w[n, k]
// Both contract C in steps of 128, one matrix instruction deep, and write J columns:
// with W the matrix operand's rows and tokens its columns, a lane's four results are
// four neighbouring columns of one token, and both scales are one factor for them:
//   p = W_step x_step (matrix instruction from zero);  acc += (sx sw) p
// which takes four vector FMAs beside each instruction of 16 x 16 x 128.
#include "lds_load.hpp"

#include <algorithm>

namespace pulse {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x8 __attribute__((ext_vector_type(8)));
typedef int32_t i32x2 __attribute__((ext_vector_type(2)));

constexpr int GB = 128;  // columns of a step, and of a scale

// What is read through the scalar cache: a vector load would wait behind those into LDS.
typedef const __attribute__((address_space(4))) float *scalar_floats;

struct GemmArgs {
    const uint8_t *x, *w;
    const float *sx, *sw;
    const uint16_t *bias;
    uint16_t *y;
    f32x4 *parts;  // sums of the shared tiles: [tile][share][result of a lane][thread]
    int64_t ldy;
    int32_t M, J, C;        // tokens, columns of y, contraction
    int32_t K;              // columns of w
    int32_t gx, gwj, gwc;   // scales: blocks of a row of sx; strides of sw for a block of J, of C
    int32_t tiles_m, tiles_j, steps;
    int32_t whole;          // tiles [0, whole) have one workgroup each, the others
    int32_t shares, per;    // `shares`, of `per` steps
};

// ---- the tile kernel ----------------------------------------------------------------
// A workgroup makes BJ columns of BM tokens; its waves are WJ x WM, each with BJ / WJ
// columns and BM / WM tokens.  A step's 128 columns of W and x lie in one of STAGES
// buffers of LDS, STAGES - 1 steps ahead of the step that is multiplied.
//
// In LDS a row of 128 bytes is eight pieces of 16, and piece p of row r lies at
// p ^ swap(r).  A wave's matrix operand for four tiles of 16 columns takes row
// 16 a + 4 t + b of its 64 as row 4 a + b of tile t: a lane's results of the four tiles
// are then 16 neighbouring columns.  Within a tile, a and b vary, and swap() goes by
// their low three bits.
__device__ __forceinline__ int swap_piece(int r) { return (r & 3) | ((r >> 2) & 4); }

// nn: rows are steps of the contraction, BJ bytes of columns each; piece p of row r lies
// at p ^ (r & 7), so that the eight rows of a transposing read are in eight places.
// The i-th of n when the workgroups 8 k + x, of XCD x, are to have neighbouring numbers
__device__ __forceinline__ int spread(int i, int n) {
    const int x = i & 7, k = i >> 3, whole = n >> 3, rest = n & 7;
    return x * whole + (x < rest ? x : rest) + k;
}

template <int BM, int BJ>
__device__ __forceinline__ void tile_origin(int tile, int tiles_m, int tiles_j, int &m0, int &j0) {
    const int band = 8 * tiles_j, b0 = tile / band * 8, rows = tiles_m - b0 < 8 ? tiles_m - b0 : 8;
    const int in = tile % band;
    m0 = (b0 + in % rows) * BM;
    j0 = in / rows * BJ;
}

// Result `j` (tile of 16 columns), `m` (tile of 16 tokens) of a thread: its token and the first of
// its four columns within a workgroup's tile
template <typename T, bool NN>
__device__ __forceinline__ void result_place(int thread, int j, int m, int &row, int &col) {
    const int lane = thread & 63, wave = thread / kWave, c16 = lane & 15, q = lane >> 4;
    row = wave % T::wm * T::tm + m * 16 + c16;
    col = wave / T::wm * T::tj + (j >> 2) * 64 + (NN ? (j & 3) * 16 + q * 4 : q * 16 + (j & 3) * 4);
}

// four columns of y from float32 sums
__device__ __forceinline__ void store_result(const GemmArgs &g, int row, int col, f32x4 v) {
    uint16_t *const out = g.y + (int64_t)row * g.ldy + col;
    if (g.bias)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (col + i < g.J) v[i] += __uint_as_float((uint32_t)g.bias[col + i] << 16);
    const u32x2 o = {cast_pair(v[0], v[1]), cast_pair(v[2], v[3])};
    if (col + 3 < g.J && g.ldy % 4 == 0) {
        *reinterpret_cast<u32x2 *>(out) = o;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (col + i < g.J) out[i] = (uint16_t)(o[i >> 1] >> (16 * (i & 1)));
    }
}

template <bool NN, int BM, int BJ, int WM, int WJ, int STAGES>
struct Tile {
    static constexpr int wm = WM;
    static constexpr int waves = WM * WJ, threads = waves * kWave;
    static constexpr int tm = BM / WM, tj = BJ / WJ;      // of a wave
    static constexpr int mt = tm / 16, jg = tj / 64;      // tiles of 16 tokens, groups of 64 columns
    static constexpr int results = mt * jg * 4;           // of a lane, four values each
    static constexpr int x_bytes = BM * GB, w_bytes = BJ * GB, s_bytes = BM * 4;
    static constexpr int stage = x_bytes + w_bytes + ((s_bytes + 255) / 256) * 256;
    static constexpr int xi = x_bytes / 1024 / waves, wi = w_bytes / 1024 / waves;  // loads of a wave
    static constexpr int si = (BM / kWave + waves - 1) / waves;  // (a wave beyond the last repeats the last one)
    static constexpr int loads = xi + wi + si;
    static_assert(x_bytes % (1024 * waves) == 0 && w_bytes % (1024 * waves) == 0, "whole loads");
    static_assert(BM % kWave == 0 && tj % 64 == 0 && GB % tj == 0 && (STAGES - 2) * loads <= 63, "tile");
};

template <bool NN, int BM, int BJ, int WM, int WJ, int STAGES>
__global__ __launch_bounds__(WM *WJ *kWave) void k_fp8_tile(GemmArgs g) {
    using T = Tile<NN, BM, BJ, WM, WJ, STAGES>;
    __shared__ __attribute__((aligned(1024))) uint8_t s_mem[STAGES * T::stage];
    const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(wave_id());
    const int c16 = lane & 15, q = lane >> 4;

    // A tile and its share of the contraction.  Workgroups go round the XCDs: each XCD takes a run of
    // tiles, which go through eight rows of tiles of tokens at a time.
    const int wg = blockIdx.x, tiles = g.tiles_m * g.tiles_j;
    int tile, share = 0, s0 = 0, s1 = g.steps;
    if (wg < g.whole) {
        tile = spread(wg, g.whole);
    } else {
        const int at = spread(wg - g.whole, (tiles - g.whole) * g.shares);
        tile = g.whole + at / g.shares;
        share = at % g.shares;
        s0 = share * g.per;
        s1 = s0 + g.per < g.steps ? s0 + g.per : g.steps;
    }
    int m0, j0;
    tile_origin<BM, BJ>(tile, g.tiles_m, g.tiles_j, m0, j0);
    // bases of the first step, and each load's offset from them
    const int64_t c0 = (int64_t)s0 * GB;
    const uint8_t *xb = load_base(g.x + (int64_t)m0 * g.C + c0);
    const uint8_t *wb = load_base(NN ? g.w + c0 * g.K + j0 : g.w + (int64_t)j0 * g.K + c0);
    const float *sb = load_base(g.sx + (int64_t)m0 * g.gx + s0);
    uint32_t xo[T::xi], wo[T::wi], so[T::si];
    constexpr int per_row = BJ / 16, rows_w = 64 / per_row;  // nn: pieces of a row, rows of a load
    const auto clamped = [](int r, int n) { return r < n ? r : n - 1; };
#pragma unroll
    for (int i = 0; i < T::xi; ++i) {
        const int r = (wave * T::xi + i) * 8 + (lane >> 3);
        xo[i] = (uint32_t)(clamped(m0 + r, g.M) - m0) * (uint32_t)g.C + ((lane & 7) ^ swap_piece(r)) * 16;
    }
#pragma unroll
    for (int i = 0; i < T::wi; ++i) {
        if constexpr (NN) {
            const int r = (wave * T::wi + i) * rows_w + lane / per_row;
            int p = (lane % per_row) ^ (r & 7);
            if (j0 + p * 16 >= g.J) p = 0;  // columns past the last are not written
            wo[i] = (uint32_t)r * (uint32_t)g.K + p * 16;
        } else {
            const int r = (wave * T::wi + i) * 8 + (lane >> 3);
            wo[i] = (uint32_t)(clamped(j0 + r, g.J) - j0) * (uint32_t)g.K + ((lane & 7) ^ swap_piece(r)) * 16;
        }
    }
#pragma unroll
    for (int i = 0; i < T::si; ++i) {
        int at = wave * T::si + i;
        if (at >= BM / kWave) at = BM / kWave - 1;
        so[i] = (uint32_t)(clamped(m0 + at * kWave + lane, g.M) - m0) * (uint32_t)g.gx * 4;
    }
    const uint32_t mem = __builtin_amdgcn_readfirstlane(lds_at(s_mem));
    // a step's loads into its buffer; in the last step of a ragged contraction pieces past its end are
    // taken from its first ones (x's are cleared there before they are multiplied)
    const auto issue = [&](int s) {
        const uint32_t at = mem + (uint32_t)((s - s0) % STAGES) * T::stage;
        const int left = g.C - s * GB;  // columns from this step's first on
        if (left < GB) {
#pragma unroll
            for (int i = 0; i < T::xi; ++i) {
                const int p = (lane & 7) ^ swap_piece((wave * T::xi + i) * 8 + (lane >> 3));
                if (p * 16 >= left) xo[i] -= p * 16;
            }
#pragma unroll
            for (int i = 0; i < T::wi; ++i) {
                if constexpr (NN) {
                    const int r = (wave * T::wi + i) * rows_w + lane / per_row;
                    if (r >= left) wo[i] -= (uint32_t)r * (uint32_t)g.K;
                } else {
                    const int p = (lane & 7) ^ swap_piece((wave * T::wi + i) * 8 + (lane >> 3));
                    if (p * 16 >= left) wo[i] -= p * 16;
                }
            }
        }
#pragma unroll
        for (int i = 0; i < T::xi; ++i) load_lds16(at + (wave * T::xi + i) * 1024, xb, xo[i]);
#pragma unroll
        for (int i = 0; i < T::wi; ++i) load_lds16(at + T::x_bytes + (wave * T::wi + i) * 1024, wb, wo[i]);
#pragma unroll
        for (int i = 0; i < T::si; ++i) {
            int n = wave * T::si + i;
            if (n >= BM / kWave) n = BM / kWave - 1;
            load_lds4(at + T::x_bytes + T::w_bytes + n * 256, sb, so[i]);
        }
        xb += GB;
        wb += NN ? (int64_t)GB * g.K : GB;
        sb += 1;
    };

    const int wm = wave % WM, wj = wave / WM;
    f32x4 acc[T::jg * 4][T::mt];
#pragma unroll
    for (int j = 0; j < T::jg * 4; ++j)
#pragma unroll
        for (int m = 0; m < T::mt; ++m) acc[j][m] = f32x4{0, 0, 0, 0};
    // a wave's columns lie in one block of 128
    const scalar_floats sw = (scalar_floats)(uint64_t)g.sw + (int64_t)((j0 + wj * T::tj) / GB) * g.gwj;

    for (int s = s0; s < s0 + STAGES - 1 && s < s1; ++s) issue(s);
    for (int s = s0; s < s1; ++s) {
        if (s + STAGES - 2 < s1) wait_loads<(STAGES - 2) * T::loads>();
        else wait_loads<0>();
        lds_barrier();  // this step is there, and the last one's buffer is free
        uint8_t *const buf = s_mem + ((s - s0) % STAGES) * T::stage;
        if (g.C - s * GB < GB) {  // the ragged end
            const int left = (g.C - s * GB) / 16, gone = 8 - left;
            for (int i = threadIdx.x; i < BM * gone; i += T::threads) {
                const int r = i / gone, p = left + i % gone;
                *reinterpret_cast<u32x4 *>(buf + r * GB + (p ^ swap_piece(r)) * 16) = u32x4{0, 0, 0, 0};
            }
            lds_barrier();
        }
        if (s + STAGES - 1 < s1) issue(s + STAGES - 1);
        const uint8_t *const bx = buf, *const bw = buf + T::x_bytes;
        const float *const bs = reinterpret_cast<const float *>(buf + T::x_bytes + T::w_bytes);
        const float sws = sw[(int64_t)s * g.gwc];
        i32x8 xf[T::mt];
        float f[T::mt];
#pragma unroll
        for (int m = 0; m < T::mt; ++m) {
            const int r = wm * T::tm + m * 16 + c16;
            const u32x4 lo = *reinterpret_cast<const u32x4 *>(bx + r * GB + (q ^ swap_piece(r)) * 16);
            const u32x4 hi = *reinterpret_cast<const u32x4 *>(bx + r * GB + ((q + 4) ^ swap_piece(r)) * 16);
#pragma unroll
            for (int i = 0; i < 4; ++i) xf[m][i] = lo[i], xf[m][i + 4] = hi[i];
            f[m] = bs[r] * sws;
        }
        // Tile j's products are on their way while those of tile j - 1 are added and the operand of
        // tile j + 1 is read.
        constexpr int JT = T::jg * 4;
        i32x8 wf[2];
        f32x4 p[2][T::mt];
        const auto operand = [&](int j) {
            i32x8 v;
            if constexpr (NN) {
                typedef __attribute__((address_space(3))) i32x2 *lds2;
                const int col = wj * (T::tj / 16) + j;
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    const int r = (h >> 1) * 64 + q * 16 + (h & 1) * 8 + (c16 >> 1);
                    const i32x2 u = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
                        (lds2)(uintptr_t)lds_at(bw + r * BJ + (col ^ (r & 7)) * 16 + (c16 & 1) * 8));
                    v[2 * h] = u[0], v[2 * h + 1] = u[1];
                }
            } else {
                const int r = wj * T::tj + (j >> 2) * 64 + (c16 >> 2) * 16 + (j & 3) * 4 + (c16 & 3);
                const u32x4 lo = *reinterpret_cast<const u32x4 *>(bw + r * GB + (q ^ swap_piece(r)) * 16);
                const u32x4 hi = *reinterpret_cast<const u32x4 *>(bw + r * GB + ((q + 4) ^ swap_piece(r)) * 16);
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = lo[i], v[i + 4] = hi[i];
            }
            return v;
        };
        const auto add = [&](int j, int m) {
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[j][m][i] = __builtin_fmaf(f[m], p[j & 1][m][i], acc[j][m][i]);
        };
        wf[0] = operand(0);
#pragma unroll
        for (int j = 0; j < JT; ++j) {
            if (j + 1 < JT) wf[(j + 1) & 1] = operand(j + 1);
#pragma unroll
            for (int m = 0; m < T::mt; ++m) {
                p[j & 1][m] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wf[j & 1], xf[m], f32x4{0, 0, 0, 0}, 0, 0,
                                                                               0, 0, 0, 0);
                if (j > 0) add(j - 1, m);
            }
            // in this order: the operand's reads, then four FMAs behind each matrix instruction
            __builtin_amdgcn_sched_group_barrier(0x100, NN ? 4 : 2, 0);
#pragma unroll
            for (int m = 0; m < T::mt; ++m) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);
            }
            sched_fence();
        }
#pragma unroll
        for (int m = 0; m < T::mt; ++m) add(JT - 1, m);
    }

#pragma unroll
    for (int m = 0; m < T::mt; ++m)
#pragma unroll
        for (int j = 0; j < T::jg * 4; ++j) {
            int row, col;
            result_place<T, NN>(threadIdx.x, j, m, row, col);
            if (m0 + row >= g.M) continue;
            if (wg < g.whole)
                store_result(g, m0 + row, j0 + col, acc[j][m]);
            else
                g.parts[(((int64_t)(tile - g.whole) * g.shares + share) * T::results + m * T::jg * 4 + j) * T::threads +
                        threadIdx.x] = acc[j][m];
        }
}

// y of the shared tiles: the sum of their shares, in order; a workgroup takes one result of every thread
template <bool NN, int BM, int BJ, int WM, int WJ, int STAGES>
__global__ __launch_bounds__(WM *WJ *kWave) void k_fp8_join(GemmArgs g) {
    using T = Tile<NN, BM, BJ, WM, WJ, STAGES>;
    const int tile = g.whole + blockIdx.y, result = blockIdx.x;
    int m0, j0, row, col;
    tile_origin<BM, BJ>(tile, g.tiles_m, g.tiles_j, m0, j0);
    result_place<T, NN>(threadIdx.x, result % (T::jg * 4), result / (T::jg * 4), row, col);
    if (m0 + row >= g.M || j0 + col >= g.J) return;
    const f32x4 *part = g.parts + ((int64_t)blockIdx.y * g.shares * T::results + result) * T::threads + threadIdx.x;
    f32x4 v = part[0];
    for (int s = 1; s < g.shares; ++s) v += part[(int64_t)s * T::results * T::threads];
    store_result(g, m0 + row, j0 + col, v);
}

// The tile, and how the work is shared: one round of workgroups after the other as long as each
// fills the chip; the tiles that are left over share the chip among them.
constexpr int kUnits = 256;  // compute units

struct GemmPlan {
    int bm, bj, whole, shares, per;
    int64_t tiles_m, tiles_j;
};

inline GemmPlan gemm_plan(int64_t M, int64_t J, int64_t C) {
    GemmPlan p;
    const int64_t big = ((M + 255) / 256) * ((J + 255) / 256);
    p.bm = M > 128 && big >= 128 ? 256 : M > 64 ? 128 : 64;
    p.bj = p.bm == 256 ? 256 : 128;
    p.tiles_m = (M + p.bm - 1) / p.bm;
    p.tiles_j = (J + p.bj - 1) / p.bj;
    const int64_t tiles = p.tiles_m * p.tiles_j, steps = (C + GB - 1) / GB, slots = kUnits * (p.bm == 128 ? 2 : 1);
    const int64_t rest = tiles % slots;
    int64_t shares = rest ? std::min<int64_t>(slots / rest, steps) : 1;
    p.per = (int)((steps + shares - 1) / shares);
    p.shares = (int)((steps + p.per - 1) / p.per);
    p.whole = (int)(p.shares > 1 ? tiles - rest : tiles);
    return p;
}

template <bool NN, int BM, int BJ, int WM, int WJ, int STAGES>
inline void launch_tiles(const GemmArgs &g, hipStream_t stream) {
    using T = Tile<NN, BM, BJ, WM, WJ, STAGES>;
    const int64_t rest = (int64_t)g.tiles_m * g.tiles_j - g.whole;
    k_fp8_tile<NN, BM, BJ, WM, WJ, STAGES><<<dim3((unsigned)(g.whole + rest * g.shares)), dim3(T::threads), 0, stream>>>(g);
    if (rest)
        k_fp8_join<NN, BM, BJ, WM, WJ, STAGES><<<dim3(T::results, (unsigned)rest), dim3(T::threads), 0, stream>>>(g);
}

}  // namespace pulse

using namespace pulse;

extern "C" {

int64_t pulse_fp8_gemm_ws_size(int64_t M, int64_t J, int64_t C) {
    const GemmPlan p = gemm_plan(M, J, C);
    return (p.tiles_m * p.tiles_j - p.whole) * p.shares * p.bm * p.bj * 4;
}

int pulse_launch_fp8_gemm(const uint8_t *x, const float *sx, const uint8_t *w, const float *sw, const uint16_t *bias,
                          int32_t nn, int64_t M, int64_t n, int64_t k, uint16_t *y, int64_t ldy, void *ws,
                          hipStream_t stream) {
    const int64_t J = nn ? k : n, C = nn ? n : k, gk = (k + GB - 1) / GB;
    const GemmPlan p = gemm_plan(M, J, C);
    const GemmArgs g{x, w, sx, sw, bias, y, static_cast<f32x4 *>(ws), ldy, (int32_t)M, (int32_t)J, (int32_t)C, (int32_t)k,
                     (int32_t)((C + GB - 1) / GB), nn ? 1 : (int32_t)gk, nn ? (int32_t)gk : 1, (int32_t)p.tiles_m,
                     (int32_t)p.tiles_j, (int32_t)((C + GB - 1) / GB), p.whole, p.shares, p.per};
    if (p.bm == 256) {
        if (nn) launch_tiles<true, 256, 256, 4, 2, 2>(g, stream);
        else launch_tiles<false, 256, 256, 4, 2, 2>(g, stream);
    } else if (p.bm == 128) {
        if (nn) launch_tiles<true, 128, 128, 2, 2, 2>(g, stream);
        else launch_tiles<false, 128, 128, 2, 2, 2>(g, stream);
    } else {
        if (nn) launch_tiles<true, 64, 128, 2, 2, 4>(g, stream);
        else launch_tiles<false, 64, 128, 2, 2, 4>(g, stream);
    }
    return hipGetLastError() == hipSuccess ? 0 : -5;
}
}
