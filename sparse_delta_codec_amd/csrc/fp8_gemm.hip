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

struct GemmArgs {
    const uint8_t *x, *w;
    const float *sx, *sw;
    const uint16_t *bias;
    uint16_t *y;
    float *parts;  // [splits][M][J], or null: y is written
    int64_t ldy;
    int32_t M, J, C;        // tokens, columns of y, contraction
    int32_t K;              // columns of w
    int32_t gx, gwj, gwc;   // scales: blocks of a row of sx; strides of sw for a block of J, of C
    int32_t tiles_m, tiles_j, steps, per_split;
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
template <bool NN, int BM, int BJ, int WM, int WJ, int STAGES>
struct Tile {
    static constexpr int waves = WM * WJ, threads = waves * kWave;
    static constexpr int tm = BM / WM, tj = BJ / WJ;      // of a wave
    static constexpr int mt = tm / 16, jg = tj / 64;      // tiles of 16 tokens, groups of 64 columns
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

    // workgroups go round the XCDs: each takes a run of tiles, eight rows of tiles of tokens at a time
    const int tiles = g.tiles_m * g.tiles_j;
    const int per = (tiles + 7) / 8;
    const int id = (int)(blockIdx.x & 7) * per + (int)(blockIdx.x >> 3);
    if ((int)(blockIdx.x >> 3) >= per || id >= tiles) return;
    const int band = 8 * g.tiles_j, b0 = id / band * 8, rows = g.tiles_m - b0 < 8 ? g.tiles_m - b0 : 8;
    const int m0 = (b0 + id % band % rows) * BM, j0 = id % band / rows * BJ;

    const int s0 = (int)blockIdx.y * g.per_split, s1 = s0 + g.per_split < g.steps ? s0 + g.per_split : g.steps;
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
#pragma unroll
        for (int i = 0; i < T::xi; ++i) {
            uint32_t o = xo[i];
            if (left < GB) {
                const int r = (wave * T::xi + i) * 8 + (lane >> 3), p = (lane & 7) ^ swap_piece(r);
                if (p * 16 >= left) o -= p * 16;
            }
            load_lds16(at + (wave * T::xi + i) * 1024, xb, o);
        }
#pragma unroll
        for (int i = 0; i < T::wi; ++i) {
            uint32_t o = wo[i];
            if (left < GB) {
                if constexpr (NN) {
                    const int r = (wave * T::wi + i) * rows_w + lane / per_row;
                    if (r >= left) o -= (uint32_t)r * (uint32_t)g.K;
                } else {
                    const int r = (wave * T::wi + i) * 8 + (lane >> 3), p = (lane & 7) ^ swap_piece(r);
                    if (p * 16 >= left) o -= p * 16;
                }
            }
            load_lds16(at + T::x_bytes + (wave * T::wi + i) * 1024, wb, o);
        }
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
    const float *const sw = g.sw + (int64_t)((j0 + wj * T::tj) / GB) * g.gwj;

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
#pragma unroll
        for (int j = 0; j < T::jg * 4; ++j) {
            i32x8 wf;
            if constexpr (NN) {
                // columns 16 a + 4 t + b of the group's 64 as row 4 a + b of tile t: see below
                typedef __attribute__((address_space(3))) i32x2 *lds2;
                const int col = wj * T::tj + j * 16;
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    const int r = (h >> 1) * 64 + q * 16 + (h & 1) * 8 + (c16 >> 1);
                    const int p = col / 16 ^ (r & 7);
                    const i32x2 v = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
                        (lds2)(uintptr_t)lds_at(bw + r * BJ + p * 16 + (c16 & 1) * 8));
                    wf[2 * h] = v[0], wf[2 * h + 1] = v[1];
                }
            } else {
                const int r = wj * T::tj + (j >> 2) * 64 + (c16 >> 2) * 16 + (j & 3) * 4 + (c16 & 3);
                const u32x4 lo = *reinterpret_cast<const u32x4 *>(bw + r * GB + (q ^ swap_piece(r)) * 16);
                const u32x4 hi = *reinterpret_cast<const u32x4 *>(bw + r * GB + ((q + 4) ^ swap_piece(r)) * 16);
#pragma unroll
                for (int i = 0; i < 4; ++i) wf[i] = lo[i], wf[i + 4] = hi[i];
            }
#pragma unroll
            for (int m = 0; m < T::mt; ++m) {
                const f32x4 p = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wf, xf[m], f32x4{0, 0, 0, 0}, 0, 0, 0,
                                                                                 0, 0, 0);
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[j][m][i] = __builtin_fmaf(f[m], p[i], acc[j][m][i]);
            }
        }
    }

    // a lane's columns of group jg, tile t, result i: nt 64 jg + 16 q + 4 t + i, nn 64 jg + 16 t + 4 q + i
#pragma unroll
    for (int m = 0; m < T::mt; ++m) {
        const int row = m0 + wm * T::tm + m * 16 + c16;
        if (row >= g.M) continue;
#pragma unroll
        for (int j = 0; j < T::jg * 4; ++j) {
            const int col = j0 + wj * T::tj + (j >> 2) * 64 + (NN ? (j & 3) * 16 + q * 4 : q * 16 + (j & 3) * 4);
            f32x4 v = acc[j][m];
            if (g.parts) {
                float *const out = g.parts + ((int64_t)blockIdx.y * g.M + row) * g.J + col;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (col + i < g.J) out[i] = v[i];
            } else {
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
        }
    }
}

// y = the sum of the parts, in their order (+ bias): a thread takes one value
__global__ __launch_bounds__(256) void k_fp8_join(const float *__restrict__ parts, int32_t splits, int64_t M, int64_t J,
                                                  const uint16_t *__restrict__ bias, uint16_t *__restrict__ y,
                                                  int64_t ldy) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= M * J) return;
    float v = 0;
    for (int s = 0; s < splits; ++s) v += parts[s * M * J + i];
    const int64_t m = i / J, j = i - m * J;
    if (bias) v += __uint_as_float((uint32_t)bias[j] << 16);
    y[m * ldy + j] = (uint16_t)cast_pair(v, 0.0f);
}

// How the contraction is shared
struct GemmPlan {
    int bm, bj, splits, per_split;
};

inline GemmPlan gemm_plan(int64_t M, int64_t J, int64_t C) {
    GemmPlan p;
    const int64_t big = ((M + 255) / 256) * ((J + 255) / 256);
    p.bm = M > 128 && big >= 128 ? 256 : M > 64 ? 128 : 64;
    p.bj = p.bm == 256 ? 256 : 128;
    const int64_t tiles = ((M + p.bm - 1) / p.bm) * ((J + p.bj - 1) / p.bj), steps = (C + GB - 1) / GB;
    int64_t splits = p.bm == 256 ? 1 : std::min<int64_t>(steps, std::max<int64_t>(1, 512 / tiles));
    p.per_split = (int)((steps + splits - 1) / splits);
    p.splits = (int)((steps + p.per_split - 1) / p.per_split);
    return p;
}

}  // namespace pulse

using namespace pulse;

extern "C" {

int64_t pulse_fp8_gemm_ws_size(int64_t M, int64_t J, int64_t C) {
    const GemmPlan p = gemm_plan(M, J, C);
    return p.splits > 1 ? (int64_t)p.splits * M * J * 4 : 0;
}

int pulse_launch_fp8_gemm(const uint8_t *x, const float *sx, const uint8_t *w, const float *sw, const uint16_t *bias,
                          int32_t nn, int64_t M, int64_t n, int64_t k, uint16_t *y, int64_t ldy, void *ws,
                          hipStream_t stream) {
    const int64_t J = nn ? k : n, C = nn ? n : k, gk = (k + GB - 1) / GB;
    const GemmPlan p = gemm_plan(M, J, C);
    GemmArgs g{x, w, sx, sw, bias, y, p.splits > 1 ? static_cast<float *>(ws) : nullptr, ldy, (int32_t)M, (int32_t)J,
               (int32_t)C, (int32_t)k, (int32_t)((C + GB - 1) / GB), nn ? 1 : (int32_t)gk, nn ? (int32_t)gk : 1,
               (int32_t)((M + p.bm - 1) / p.bm), (int32_t)((J + p.bj - 1) / p.bj), (int32_t)((C + GB - 1) / GB),
               p.per_split};
    const int64_t tiles = (int64_t)g.tiles_m * g.tiles_j;
    const dim3 grid((unsigned)((tiles + 7) / 8 * 8), (unsigned)p.splits);
    if (p.bm == 256) {
        if (nn) k_fp8_tile<true, 256, 256, 4, 2, 2><<<grid, dim3(512), 0, stream>>>(g);
        else k_fp8_tile<false, 256, 256, 4, 2, 2><<<grid, dim3(512), 0, stream>>>(g);
    } else if (p.bm == 128) {
        if (nn) k_fp8_tile<true, 128, 128, 2, 2, 2><<<grid, dim3(256), 0, stream>>>(g);
        else k_fp8_tile<false, 128, 128, 2, 2, 2><<<grid, dim3(256), 0, stream>>>(g);
    } else {
        if (nn) k_fp8_tile<true, 64, 128, 2, 2, 4><<<grid, dim3(256), 0, stream>>>(g);
        else k_fp8_tile<false, 64, 128, 2, 2, 4><<<grid, dim3(256), 0, stream>>>(g);
    }
    if (g.parts)
        k_fp8_join<<<dim3((unsigned)((M * J + 255) / 256)), dim3(256), 0, stream>>>(g.parts, p.splits, M, J, bias, y, ldy);
    return hipGetLastError() == hipSuccess ? 0 : -5;
}
}
