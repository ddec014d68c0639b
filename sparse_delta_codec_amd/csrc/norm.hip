// norm.hip -- the root-mean-square norm in front of a projection, with the
// residual's addition before it and E4M3 codes behind it; its backward pass; and
// the group quantiser for the rows that no norm makes (attention's output, an
// MLP's activation, gradients).
//
// For a row of n columns:
//   s = bf16(x + residual), or x         (what later layers and the backward pass read)
//   r = 1 / sqrt(mean(s^2) + eps),  y = s r w
//   dx = r (dy w - s r mean(dy w s r)) + dres,  dw = sum over rows of dy s r
// Every byte is read and written once, so the large calls are bound by HBM (5.2 to 5.5 TB/s where
// a copy has 5.1: more is read than written) and the small ones by the launch and the chain
// load - sum - barrier - store.  A row stays in the registers of one workgroup between its sum
// and its output: 8 columns (16 bytes) a lane, so that 16 lanes hold a quantisation group and
// 64 lanes read 1024 contiguous bytes.
#include "e4m3.hpp"

#include <algorithm>
#include <type_traits>

namespace pulse {

typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int NP = 512;         // columns of a wave's piece
constexpr int NORM_WAVES = 16;  // most waves of a workgroup
constexpr int NORM_PIECES = 8;  // most pieces of a lane, with at most four waves then
constexpr int NORM_BACK_WAVES = 8;  // of the backward pass, whose lanes hold dw too
constexpr int norm_threads(int pieces) { return (pieces <= 4 ? NORM_WAVES : 4) * kWave; }

struct NormArgs {
    const uint16_t *x, *w;
    uint16_t *residual, *y;
    uint8_t *codes;
    float *scales, *rstd;
    int64_t ldx, ldr, ldy;
    int32_t cols;
    float eps;
};

// the row's sum in every thread; s: LDS of a float a wave
__device__ __forceinline__ float row_sum(float v, float *s) {
    v = wave_reduce_sum(v);
    const int nw = blockDim.x / kWave;
    if (nw == 1) return v;
    if (lane_id() == 0) s[wave_id()] = v;
    lds_barrier();
    v = s[0];
    for (int i = 1; i < nw; ++i) v += s[i];
    return v;
}

// A workgroup takes one row, wave w its pieces w, w + waves, ...
template <int P, bool RES>
__global__ __launch_bounds__(norm_threads(P)) void k_rms_norm(NormArgs g) {
    __shared__ float s_sum[NORM_WAVES];
    const int64_t row = blockIdx.x;
    const int nt = blockDim.x;
    const uint16_t *const x = g.x + row * g.ldx;
    uint16_t *const res = RES ? g.residual + row * g.ldr : nullptr;
    u32x4 v[P], r[RES ? P : 1], w[P];
#pragma unroll
    for (int p = 0; p < P; ++p) {
        const int c = (p * nt + (int)threadIdx.x) * 8;
        v[p] = u32x4{0, 0, 0, 0};
        if (RES) r[p] = u32x4{0, 0, 0, 0};
        if (c < g.cols) {
            v[p] = *reinterpret_cast<const u32x4 *>(x + c);
            if (RES) r[p] = *reinterpret_cast<const u32x4 *>(res + c);
        }
    }
#pragma unroll
    for (int p = 0; p < P; ++p) {
        const int c = (p * nt + (int)threadIdx.x) * 8;
        w[p] = u32x4{0, 0, 0, 0};
        if (c < g.cols) w[p] = *reinterpret_cast<const u32x4 *>(g.w + c);
    }
    float sum = 0;
#pragma unroll
    for (int p = 0; p < P; ++p) {
        float a[8];
        widen8(v[p], a);
        if (RES) {
            float b[8];
            widen8(r[p], b);
#pragma unroll
            for (int i = 0; i < 8; ++i) a[i] += b[i];
            v[p] = narrow8(a);
            const int c = (p * nt + (int)threadIdx.x) * 8;
            if (c < g.cols) *reinterpret_cast<u32x4 *>(res + c) = v[p];
            widen8(v[p], a);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) sum = __builtin_fmaf(a[i], a[i], sum);
    }
    const float rstd = 1.0f / sqrtf(row_sum(sum, s_sum) / (float)g.cols + g.eps);
    if (g.rstd && threadIdx.x == 0) g.rstd[row] = rstd;
    const int64_t groups = (g.cols + QG - 1) / QG;
#pragma unroll
    for (int p = 0; p < P; ++p) {
        const int c = (p * nt + (int)threadIdx.x) * 8;
        float a[8], b[8];
        widen8(v[p], a);
        widen8(w[p], b);
#pragma unroll
        for (int i = 0; i < 8; ++i) a[i] = a[i] * rstd * b[i];
        if (g.y && c < g.cols) *reinterpret_cast<u32x4 *>(g.y + row * g.ldy + c) = narrow8(a);
        if (g.codes) {
            float s;
            const u32x2 q = group_codes(a, &s);  // (lanes past the last column hold zeros)
            if (c < g.cols) {
                *reinterpret_cast<u32x2 *>(g.codes + row * g.cols + c) = q;
                if (c % QG == 0) g.scales[row * groups + c / QG] = s;
            }
        }
    }
}

struct NormBackArgs {
    const uint16_t *s, *w, *dy, *dres;
    const float *rstd;
    uint16_t *dx;
    float *parts;  // [workgroups][cols]: sums of dy s r over a workgroup's rows
    int64_t lds, lddy, lddres, lddx, rows;
    int32_t cols;
};

// A workgroup takes the rows blockIdx.x, + gridDim.x, ... and keeps its share of dw in registers.
template <int P, bool RES>
__global__ __launch_bounds__(NORM_BACK_WAVES *kWave) void k_rms_norm_back(NormBackArgs g) {
    __shared__ float s_sum[2][NORM_BACK_WAVES];
    const int nt = blockDim.x;
    float dw[P][8];
    u32x4 w[P];
#pragma unroll
    for (int p = 0; p < P; ++p) {
        const int c = (p * nt + (int)threadIdx.x) * 8;
        w[p] = u32x4{0, 0, 0, 0};
        if (c < g.cols) w[p] = *reinterpret_cast<const u32x4 *>(g.w + c);
#pragma unroll
        for (int i = 0; i < 8; ++i) dw[p][i] = 0;
    }
    // a row's s, dy and dres; the next row's are on their way while a row is worked on (dres only
    // where the registers hold it)
    constexpr bool AHEAD = RES && P < 4;
    struct Row {
        u32x4 s[P], dy[P], dres[P];
        float rstd;
    };
    const auto load = [&](int64_t row, Row &r) {
        r.rstd = g.rstd[row];
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const int c = (p * nt + (int)threadIdx.x) * 8;
            r.s[p] = r.dy[p] = r.dres[p] = u32x4{0, 0, 0, 0};
            if (c < g.cols) {
                r.s[p] = *reinterpret_cast<const u32x4 *>(g.s + row * g.lds + c);
                r.dy[p] = *reinterpret_cast<const u32x4 *>(g.dy + row * g.lddy + c);
                if (AHEAD) r.dres[p] = *reinterpret_cast<const u32x4 *>(g.dres + row * g.lddres + c);
            }
        }
    };
    int turn = 0;
    Row now, next;
    load(blockIdx.x, now);
    for (int64_t row = blockIdx.x; row < g.rows; row += gridDim.x, turn ^= 1, now = next) {
        if (row + gridDim.x < g.rows) load(row + gridDim.x, next);
        float sum = 0;
#pragma unroll
        for (int p = 0; p < P; ++p) {
            float a[8], b[8], f[8];
            widen8(now.s[p], a);
            widen8(now.dy[p], b);
            widen8(w[p], f);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float hat = a[i] * now.rstd;
                dw[p][i] = __builtin_fmaf(b[i], hat, dw[p][i]);
                sum = __builtin_fmaf(b[i] * f[i], hat, sum);
            }
        }
        if (!g.dx) continue;
        // (the other half of s_sum next time: a wave still reads this one)
        const float mean = row_sum(sum, s_sum[turn]) / (float)g.cols;
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const int c = (p * nt + (int)threadIdx.x) * 8;
            if (c >= g.cols) continue;
            float a[8], b[8], f[8], o[8];
            widen8(now.s[p], a);
            widen8(now.dy[p], b);
            widen8(w[p], f);
            if (AHEAD) widen8(now.dres[p], o);
            else if (RES) widen8(*reinterpret_cast<const u32x4 *>(g.dres + row * g.lddres + c), o);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float t = __builtin_fmaf(a[i] * now.rstd, -mean, b[i] * f[i]);
                o[i] = RES ? __builtin_fmaf(t, now.rstd, o[i]) : t * now.rstd;
            }
            *reinterpret_cast<u32x4 *>(g.dx + row * g.lddx + c) = narrow8(o);
        }
    }
#pragma unroll
    for (int p = 0; p < P; ++p) {
        const int c = (p * nt + (int)threadIdx.x) * 8;
        if (c >= g.cols) continue;
        float *const out = g.parts + (int64_t)blockIdx.x * g.cols + c;
        *reinterpret_cast<f32x4 *>(out) = f32x4{dw[p][0], dw[p][1], dw[p][2], dw[p][3]};
        *reinterpret_cast<f32x4 *>(out + 4) = f32x4{dw[p][4], dw[p][5], dw[p][6], dw[p][7]};
    }
}

// dw = the sum of the workgroups' parts, in a fixed order: 16 columns a workgroup, so that there are
// enough of them; thread (r, c) takes the parts r, r + 64, ...
constexpr int SUM_COLS = 16;

__global__ __launch_bounds__(1024) void k_rms_norm_sum(const float *__restrict__ parts, int32_t n, int32_t cols,
                                                       float *__restrict__ dw, int32_t accumulate) {
    __shared__ float s[64][SUM_COLS];
    const int k = threadIdx.x % SUM_COLS, r = threadIdx.x / SUM_COLS, c = blockIdx.x * SUM_COLS + k;
    float sum = 0;
    if (c < cols) {
#pragma unroll 4
        for (int i = r; i < n; i += 64) sum += parts[(int64_t)i * cols + c];
    }
    s[r][k] = sum;
    for (int half = 32; half > 0; half /= 2) {
        __syncthreads();
        if (r < half) s[r][k] += s[r + half][k];
    }
    if (r == 0 && c < cols) dw[c] = accumulate ? dw[c] + s[0][k] : s[0][k];
}

struct GroupQuantArgs {
    const uint16_t *x;
    uint8_t *codes;
    float *scales;
    int64_t ldx, pieces;
    int32_t cols, per_row;
};

// pieces of a wave, all read before the first is worked on.  With 1, 2 and 4: 8191 x 28672 129, 119
// (5.9 TB/s) and 123 us, 1024 x 5120 5.3, 5.7 and 6.2, 96 x 27648 with silu 5.2, 5.3 and 6.2.
constexpr int GQ = 2;

// A wave takes GQ pieces of 512 columns, one after the other through the rows; GLU: silu(x[c]) x[cols + c],
// in the form for all gates only where a lane has one that needs it (8192 x 28672: 214 us; that
// form for all of them 250).
template <bool GLU>
__global__ __launch_bounds__(256) void k_group_quant(GroupQuantArgs g) {
    const int64_t first = ((int64_t)blockIdx.x * 4 + wave_id()) * GQ;
    const int lane = lane_id();
    u32x4 v[GQ], u[GLU ? GQ : 1];
    int64_t row[GQ];
    int c[GQ];
    int64_t r = first / g.per_row;
    int p = (int)(first - r * g.per_row);
#pragma unroll
    for (int i = 0; i < GQ; ++i) {
        row[i] = r;
        c[i] = p * NP + lane * 8;
        if (first + i >= g.pieces) c[i] = g.cols;
        if (++p == g.per_row) p = 0, ++r;
        v[i] = u32x4{0, 0, 0, 0};
        if (GLU) u[i] = u32x4{0, 0, 0, 0};
        if (c[i] < g.cols) {
            const uint16_t *const at = g.x + row[i] * g.ldx + c[i];
            v[i] = *reinterpret_cast<const u32x4 *>(at);
            if (GLU) u[i] = *reinterpret_cast<const u32x4 *>(at + g.cols);
        }
    }
    const int64_t groups = (g.cols + QG - 1) / QG;
#pragma unroll
    for (int i = 0; i < GQ; ++i) {
        float a[8], s;
        widen8(v[i], a);
        if (GLU) {
            float b[8], low = 0;
            widen8(u[i], b);
#pragma unroll
            for (int j = 0; j < 8; ++j) low = fminf(low, a[j]);
            if (__any(low < kFarGate)) {
#pragma unroll
                for (int j = 0; j < 8; ++j) a[j] = silu(a[j]) * b[j];
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) a[j] = silu<false>(a[j]) * b[j];
            }
        }
        const u32x2 q = group_codes(a, &s);
        if (c[i] < g.cols) {
            *reinterpret_cast<u32x2 *>(g.codes + row[i] * g.cols + c[i]) = q;
            if (c[i] % QG == 0) g.scales[row[i] * groups + c[i] / QG] = s;
        }
    }
}

// Waves of a row's workgroup and pieces of a wave: with many rows few waves, of which more rows
// are under way at once, with few rows many.  With codes and a residual, new rows for each call, up to 4 and
// 16 waves: 512 x 5120 8.2 and 8.1 us (the call's own time), 1024 x 5120 11.8 and 13.0, 4099 x 4096 24.8
// and 26.8, 8192 x 5120 56.9 and 57.1 (5.2 TB/s), 8192 x 16384 172 and 168.
struct NormShape {
    int waves, pieces;
};

inline NormShape norm_shape(int64_t cols, int most) {
    const int n = (int)((cols + NP - 1) / NP);
    int pieces = (n + most - 1) / most;
    for (int p : {1, 2, 3, 4, 6, NORM_PIECES})
        if (p >= pieces) {
            pieces = p;
            break;
        }
    return {(n + pieces - 1) / pieces, pieces};
}

// f with the pieces of norm_shape as a constant
template <typename F>
inline void with_pieces(int pieces, F &&f) {
    switch (pieces) {
    case 1: return f(std::integral_constant<int, 1>{});
    case 2: return f(std::integral_constant<int, 2>{});
    case 3: return f(std::integral_constant<int, 3>{});
    case 4: return f(std::integral_constant<int, 4>{});
    case 6: return f(std::integral_constant<int, 6>{});
    default: return f(std::integral_constant<int, NORM_PIECES>{});
    }
}

// Workgroups of the backward pass, a part of dw each: 8192 x 5120 with 256, 512 and 1024 of them 66, 71 and
// 78 us, 2000 x 1024 12.3, 10.0 and 10.3.
inline int64_t norm_parts(int64_t rows, int64_t cols) { return std::min<int64_t>(rows, cols > 2048 ? 256 : 512); }

}  // namespace pulse

using namespace pulse;

extern "C" {

int64_t pulse_rms_norm_ws_size(int64_t rows, int64_t cols) { return norm_parts(rows, cols) * cols * (int64_t)sizeof(float); }

int pulse_launch_rms_norm(const uint16_t *x, int64_t ldx, const uint16_t *w, double eps, uint16_t *residual,
                          int64_t ldr, uint16_t *y, int64_t ldy, uint8_t *codes, float *scales, float *rstd,
                          int64_t rows, int64_t cols, hipStream_t stream) {
    const NormArgs g{x, w, residual, y, codes, scales, rstd, ldx, ldr, ldy, (int32_t)cols, (float)eps};
    const NormShape n = norm_shape(cols, rows >= 1024 ? 4 : NORM_WAVES);
    with_pieces(n.pieces, [&](auto p) {
        constexpr int P = decltype(p)::value;
        const dim3 grid((unsigned)rows), block((unsigned)(n.waves * kWave));
        if (residual) k_rms_norm<P, true><<<grid, block, 0, stream>>>(g);
        else k_rms_norm<P, false><<<grid, block, 0, stream>>>(g);
    });
    return hipGetLastError() == hipSuccess ? 0 : -5;
}

int pulse_launch_rms_norm_backward(const uint16_t *s, int64_t lds, const uint16_t *w, const float *rstd,
                                   const uint16_t *dy, int64_t lddy, const uint16_t *dres, int64_t lddres,
                                   uint16_t *dx, int64_t lddx, float *dw, int32_t accumulate, int64_t rows,
                                   int64_t cols, void *ws, hipStream_t stream) {
    float *const parts = static_cast<float *>(ws);
    const NormBackArgs g{s, w, dy, dres, rstd, dx, parts, lds, lddy, lddres, lddx, rows, (int32_t)cols};
    const NormShape n = norm_shape(cols, NORM_BACK_WAVES);  // (four: 4099 x 8192 76 instead of 56 us)
    const int64_t wgs = norm_parts(rows, cols);
    with_pieces(n.pieces, [&](auto p) {
        constexpr int P = decltype(p)::value < 4 ? decltype(p)::value : 4;  // (eight waves: no more)
        const dim3 grid((unsigned)wgs), block((unsigned)(n.waves * kWave));
        if (dres) k_rms_norm_back<P, true><<<grid, block, 0, stream>>>(g);
        else k_rms_norm_back<P, false><<<grid, block, 0, stream>>>(g);
    });
    k_rms_norm_sum<<<dim3((unsigned)((cols + SUM_COLS - 1) / SUM_COLS)), dim3(1024), 0, stream>>>(parts, (int32_t)wgs,
                                                                                       (int32_t)cols, dw, accumulate);
    return hipGetLastError() == hipSuccess ? 0 : -5;
}

int pulse_launch_group_quant(const uint16_t *x, int64_t ldx, int64_t rows, int64_t cols, int32_t glu, uint8_t *codes,
                             float *scales, hipStream_t stream) {
    GroupQuantArgs g{x, codes, scales, ldx, 0, (int32_t)cols, (int32_t)((cols + NP - 1) / NP)};
    g.pieces = rows * g.per_row;
    const dim3 grid((unsigned)((g.pieces + 4 * GQ - 1) / (4 * GQ)));
    if (glu) k_group_quant<true><<<grid, dim3(256), 0, stream>>>(g);
    else k_group_quant<false><<<grid, dim3(256), 0, stream>>>(g);
    return hipGetLastError() == hipSuccess ? 0 : -5;
}
}
