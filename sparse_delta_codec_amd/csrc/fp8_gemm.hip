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
// The instruction keeps fewer bits than float32 inside: of eight neighbouring products each is cut to a
// multiple of about 2^-13 of the largest.  That is the price of its rate, twice that of codes widened to BF16,
// whose products stay whole.  Few tokens, whose time is W's and not the instruction's, go through it too, so that
// a token's results in a small batch and in a large one differ by the order of their sums alone.
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

// ---- tiles ----------------------------------------------------------------------------
// A workgroup makes BJ columns of BM tokens; its waves are WM x 2, each with BM / WM tokens
// and 64 columns of every 128 (which have one scale a step).  A step's 128 columns of x and
// W lie in LDS, put there while earlier steps are multiplied.
//
// In LDS a row of 128 bytes is eight pieces of 16, and piece p of row r lies at p ^ swap(r):
// two rows fill the 64 banks, and the sixteen rows that a matrix operand takes at one piece are
// to be in sixteen places.
//  x: rows 16 m .. 16 m + 15, so swap goes by bits 1 to 3.
//  W: a wave's operand for four tiles of 16 columns takes row 16 a + 4 t + b of its 64 as row
//     4 a + b of tile t, which makes a lane's results of the four tiles 16 neighbouring columns; a
//     and b vary within a tile, so swap goes by bits 1, 4 and 5.
//  W (nn): rows are steps of the contraction, and a transposing read takes eight of them.
// (By bits 0, 1 and 4 for both, reads of x met in banks four at a time: 8192 x [55296, 5120] 2280 us.)
__device__ __forceinline__ int swap_x(int r) { return (r >> 1) & 7; }
template <bool NN>
__device__ __forceinline__ int swap_w(int r) { return NN ? r & 7 : ((r >> 1) & 1) | ((r >> 3) & 6); }

template <int BM_, int BJ_, int WM_>
struct Tile {
    static constexpr int BM = BM_, BJ = BJ_, WM = WM_, WJ = 2;
    static constexpr int waves = WM * WJ, threads = waves * kWave;
    static constexpr int tm = BM / WM, mt = tm / 16;  // tokens of a wave, in tiles of 16
    static constexpr int parts = BJ / GB;             // of 128 columns
    static constexpr int results = mt * parts * 4;    // of a lane, four values each
    static constexpr int x_bytes = BM * GB, w_bytes = GB * GB;  // of a step (w: of a part)
    static constexpr int s_bytes = BM * 16;           // scales of four steps
    static constexpr int xi = x_bytes / 1024 / waves, wi = w_bytes / 1024 / waves;  // loads of a wave
    static constexpr int si = (BM / kWave + waves - 1) / waves;  // (a wave beyond the last repeats the last one)
    static_assert(x_bytes % (1024 * waves) == 0 && w_bytes % (1024 * waves) == 0, "whole loads");
    static_assert(BM % kWave == 0 && BJ % GB == 0 && tm % 16 == 0, "tile");
};

// The i-th of n when the workgroups 8 k + x, of XCD x, are to have neighbouring numbers
__device__ __forceinline__ int spread(int i, int n) {
    const int x = i & 7, k = i >> 3, whole = n >> 3, rest = n & 7;
    return x * whole + (x < rest ? x : rest) + k;
}

// Where a tile lies: tiles go through eight rows of tiles of tokens at a time.
template <typename T>
__device__ __forceinline__ void tile_origin(const GemmArgs &g, int tile, int &m0, int &j0) {
    const int band = 8 * g.tiles_j, b0 = tile / band * 8, rows = g.tiles_m - b0 < 8 ? g.tiles_m - b0 : 8;
    const int in = tile % band;
    m0 = (b0 + in % rows) * T::BM;
    j0 = in / rows * T::BJ;
}

// A workgroup's tile and its share of the contraction.  Workgroups go round the XCDs: each XCD
// takes a run of tiles.
struct Work {
    int tile, share, s0, s1;
};

__device__ __forceinline__ Work work_of(const GemmArgs &g) {
    const int wg = blockIdx.x;
    if (wg < g.whole) return {spread(wg, g.whole), 0, 0, g.steps};
    const int at = spread(wg - g.whole, (g.tiles_m * g.tiles_j - g.whole) * g.shares);
    const int share = at % g.shares, s0 = share * g.per;
    return {g.whole + at / g.shares, share, s0, s0 + g.per < g.steps ? s0 + g.per : g.steps};
}

// Result j (part and tile of 16 columns) and m (tile of 16 tokens) of a thread: its token and the
// first of its four columns within a workgroup's tile
template <typename T, bool NN>
__device__ __forceinline__ void result_place(int thread, int j, int m, int &row, int &col) {
    const int lane = thread & 63, wave = thread / kWave, c16 = lane & 15, q = lane >> 4;
    row = wave % T::WM * T::tm + m * 16 + c16;
    col = (j >> 2) * GB + wave / T::WM * 64 + (NN ? (j & 3) * 16 + q * 4 : q * 16 + (j & 3) * 4);
}

// four columns of y from float32 sums
template <bool BIAS>
__device__ __forceinline__ void store_result(const GemmArgs &g, int row, int col, f32x4 v) {
    uint16_t *const out = g.y + (int64_t)row * g.ldy + col;
    const bool whole = col + 3 < g.J && g.ldy % 4 == 0;
    if (BIAS)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (col + i < g.J) v[i] += __uint_as_float((uint32_t)g.bias[col + i] << 16);
    const u32x2 o = {cast_pair(v[0], v[1]), cast_pair(v[2], v[3])};
    if (whole) {
        *reinterpret_cast<u32x2 *>(out) = o;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (col + i < g.J) out[i] = (uint16_t)(o[i >> 1] >> (16 * (i & 1)));
    }
}

template <typename T, bool NN>
__device__ __forceinline__ void store_results(const GemmArgs &g, const Work &k, int m0, int j0,
                                              const f32x4 (&acc)[T::parts * 4][T::mt]) {
    int thread = threadIdx.x;
    asm volatile("" : "+v"(thread));  // as rare_lane
    f32x4 *const part = g.parts + ((int64_t)(k.tile - g.whole) * g.shares + k.share) * T::results * T::threads + thread;
    const auto each = [&](auto &&f) {
#pragma unroll
        for (int m = 0; m < T::mt; ++m)
#pragma unroll
            for (int j = 0; j < T::parts * 4; ++j) {
                int row, col;
                result_place<T, NN>(thread, j, m, row, col);
                if (m0 + row < g.M) f(m * T::parts * 4 + j, m0 + row, j0 + col, acc[j][m]);
            }
    };
    if (k.tile >= g.whole) each([&](int n, int, int, const f32x4 &v) { part[n * T::threads] = v; });
    else if (g.bias) each([&](int, int row, int col, const f32x4 &v) { store_result<true>(g, row, col, v); });
    else each([&](int, int row, int col, const f32x4 &v) { store_result<false>(g, row, col, v); });
}

// y of the shared tiles: the sum of their shares, in order; a workgroup takes one result of every thread
template <typename T, bool NN>
__global__ __launch_bounds__(T::threads) void k_fp8_join(GemmArgs g) {
    const int result = blockIdx.x;
    int m0, j0, row, col;
    tile_origin<T>(g, g.whole + blockIdx.y, m0, j0);
    result_place<T, NN>(threadIdx.x, result % (T::parts * 4), result / (T::parts * 4), row, col);
    if (m0 + row >= g.M || j0 + col >= g.J) return;
    const f32x4 *part = g.parts + ((int64_t)blockIdx.y * g.shares * T::results + result) * T::threads + threadIdx.x;
    f32x4 v = part[0];
#pragma unroll 4
    for (int s = 1; s < g.shares; ++s) v += part[(int64_t)s * T::results * T::threads];
    if (g.bias) store_result<true>(g, m0 + row, j0 + col, v);
    else store_result<false>(g, m0 + row, j0 + col, v);
}

// A wave's loads of x and of the parts of W, as offsets from the bases of a step, and of the scales
// of four steps (one by one, a request for each row's and step's, they took 7% of the time).
// Rows past the last are the last one's, columns (nn) past the last the first ones': their
// results are not written.
template <typename T, bool NN>
struct Loads {
    uint32_t x[T::xi], w[T::parts][T::wi], s[T::si];

    static __device__ __forceinline__ int row(int lane, int i, int n) { return (uniform_wave() * n + i) * 8 + (lane >> 3); }
    static __device__ __forceinline__ int uniform_wave() { return __builtin_amdgcn_readfirstlane(wave_id()); }
    static __device__ __forceinline__ int piece(int lane, int r, bool w) {
        return (lane & 7) ^ (w ? swap_w<NN>(r) : swap_x(r));
    }
    // The lane's number for what only a last step needs: the compiler does not see that it could be
    // worked out before the loop, and held in registers that the loop does not have.
    static __device__ __forceinline__ int rare_lane() {
        int lane = lane_id();
        asm volatile("" : "+v"(lane));
        return lane;
    }
    static __device__ __forceinline__ int scale_row(int i) {
        int n = uniform_wave() * T::si + i;
        return n < T::BM / kWave ? n : T::BM / kWave - 1;
    }

    __device__ __forceinline__ Loads(const GemmArgs &g, int m0, int j0) {
        const int lane = lane_id();
        const auto clamped = [](int r, int n) { return (uint32_t)(r < n ? r : n - 1); };
#pragma unroll
        for (int i = 0; i < T::xi; ++i) {
            const int r = row(lane, i, T::xi);
            x[i] = (clamped(m0 + r, g.M) - m0) * (uint32_t)g.C + piece(lane, r, false) * 16;
        }
#pragma unroll
        for (int p = 0; p < T::parts; ++p)
#pragma unroll
            for (int i = 0; i < T::wi; ++i) {
                const int r = row(lane, i, T::wi);
                if constexpr (NN) {
                    const int c = p * GB + piece(lane, r, true) * 16;
                    w[p][i] = (uint32_t)r * (uint32_t)g.K + (j0 + c < g.J ? c : 0);
                } else {
                    w[p][i] = (clamped(j0 + p * GB + r, g.J) - j0) * (uint32_t)g.K + piece(lane, r, true) * 16;
                }
            }
#pragma unroll
        for (int i = 0; i < T::si; ++i)
            s[i] = (clamped(m0 + scale_row(i) * kWave + lane, g.M) - m0) * (uint32_t)g.gx * 4;
    }

    // whether a tile from row m0 on has a row with one of the array's last four scales
    static __device__ __forceinline__ bool near_end(const GemmArgs &g, int m0) { return m0 + T::BM + 4 > g.M; }

    // The scales of steps 4 n .. 4 n + 3 of row r are four neighbours in memory, from its (4 n)th one
    // on (what is behind a row's last one is not used); at the array's end they are its last four,
    // and row r's first one is late() places further on.  An array of less than four is written by hand.
    static __device__ __forceinline__ int late(const GemmArgs &g, int row, int s) {
        const int64_t all = (int64_t)g.M * g.gx, at = (int64_t)(row < g.M ? row : g.M - 1) * g.gx + (s & ~3);
        return all >= 4 && at > all - 4 ? (int)(at - (all - 4)) : 0;
    }

    // for a last step of `left` columns: pieces past its end are taken from its beginning (x's are
    // cleared in LDS before they are multiplied)
    __device__ __forceinline__ void end_x(int left) {
        const int lane = rare_lane();
#pragma unroll
        for (int i = 0; i < T::xi; ++i) {
            const int p = piece(lane, row(lane, i, T::xi), false) * 16;
            if (p >= left) x[i] -= p;
        }
    }
    __device__ __forceinline__ void end_w(const GemmArgs &g, int part, int left) {
        const int lane = rare_lane();
#pragma unroll
        for (int i = 0; i < T::wi; ++i) {
            const int r = row(lane, i, T::wi), p = piece(lane, r, true) * 16;
            if (NN && r >= left) w[part][i] -= (uint32_t)r * (uint32_t)g.K;
            if (!NN && p >= left) w[part][i] -= p;
        }
    }

    __device__ __forceinline__ void load_x(uint32_t lds, const uint8_t *base) const {
#pragma unroll
        for (int i = 0; i < T::xi; ++i) load_lds16(lds + (uniform_wave() * T::xi + i) * 1024, base, x[i]);
    }
    template <bool ONCE>
    __device__ __forceinline__ void load_w(uint32_t lds, const uint8_t *base, int part) const {
#pragma unroll
        for (int i = 0; i < T::wi; ++i) {
            const uint32_t to = lds + (uniform_wave() * T::wi + i) * 1024;
            if constexpr (ONCE) load_lds16_once(to, base, w[part][i]);
            else load_lds16(to, base, w[part][i]);
        }
    }
    __device__ __forceinline__ void load_s(const GemmArgs &g, int m0, int s4, uint8_t *to, uint32_t lds) const {
        if ((int64_t)g.M * g.gx < 4) {
            for (int r = threadIdx.x; r < T::BM; r += T::threads)
                for (int i = 0; i < 4; ++i)
                    reinterpret_cast<float *>(to)[r * 4 + i] = i < g.gx ? g.sx[(r < g.M ? r : g.M - 1) * g.gx + i] : 0.0f;
            return;
        }
        // (offsets from a base are not negative: it lies four back where the array has begun by then)
        const int64_t from = (int64_t)m0 * g.gx + s4;
        const int back = from >= 4 ? 4 : 0;
        const float *const base = g.sx + (from - back);
        const bool end = near_end(g, m0);
#pragma unroll
        for (int i = 0; i < T::si; ++i) {
            uint32_t o = s[i] + 4 * back;
            if (end) o -= 4 * late(g, m0 + scale_row(i) * kWave + lane_id(), s4);
            load_lds16(lds + scale_row(i) * 1024, base, o);
        }
    }
};

// the pieces of x from column `left` of a step on are zero (and a barrier behind that)
template <typename T>
__device__ __forceinline__ void clear_end(uint8_t *x, int left) {
    const int from = left / 16, gone = 8 - from;
    int thread = threadIdx.x;
    asm volatile("" : "+v"(thread));  // as rare_lane
    for (int i = thread; i < T::BM * gone; i += T::threads) {
        const int r = i / gone, p = from + i % gone;
        *reinterpret_cast<u32x4 *>(x + r * GB + (p ^ swap_x(r)) * 16) = u32x4{0, 0, 0, 0};
    }
    lds_barrier();
}

// Row r of a step as a matrix operand: lane group q has columns 16 q .. + 15 and 64 + 16 q .. + 15.
__device__ __forceinline__ i32x8 row_operand(const uint8_t *at, int r, int swap) {
    const int q = lane_id() >> 4;
    const u32x4 lo = *reinterpret_cast<const u32x4 *>(at + r * GB + (q ^ swap) * 16);
    const u32x4 hi = *reinterpret_cast<const u32x4 *>(at + r * GB + ((q + 4) ^ swap) * 16);
    i32x8 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = lo[i], v[i + 4] = hi[i];
    return v;
}

// Tile t of a wave's 64 columns of W.  nn: a transposing read takes eight rows of 16 columns from
// sixteen lanes and gives each lane a column; the rows are those that row_operand's lanes have.
template <bool NN>
__device__ __forceinline__ i32x8 w_operand(const uint8_t *at, int wj, int t) {
    const int c16 = lane_id() & 15, q = lane_id() >> 4;
    if constexpr (NN) {
        typedef __attribute__((address_space(3))) i32x2 *lds2;
        i32x8 v;
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            const int r = (h >> 1) * 64 + q * 16 + (h & 1) * 8 + (c16 >> 1);
            const i32x2 u = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
                (lds2)(uintptr_t)lds_at(at + r * GB + ((wj * 4 + t) ^ swap_w<NN>(r)) * 16 + (c16 & 1) * 8));
            v[2 * h] = u[0], v[2 * h + 1] = u[1];
        }
        return v;
    } else {
        const int r = wj * 64 + (c16 >> 2) * 16 + t * 4 + (c16 & 3);
        return row_operand(at, r, swap_w<NN>(r));
    }
}

// acc += f * (W x): products are added LAG matrix instructions after theirs was issued, while the
// next tile's operand is read beside this tile's products.
template <typename T, bool NN>
__device__ __forceinline__ void multiply(const uint8_t *w, int wj, const i32x8 &first, const i32x8 (&x)[T::mt], const float (&f)[T::parts][T::mt],
                                         f32x4 (&acc)[T::parts * 4][T::mt]) {
    constexpr int LAG = T::mt < 3 ? T::mt : 3, N = T::parts * 4 * T::mt;
    i32x8 wf[2];
    f32x4 p[LAG + 1];
    const auto add = [&](int n) {
        f32x4 &a = acc[n / T::mt][n % T::mt];
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = __builtin_fmaf(f[n / T::mt / 4][n % T::mt], p[n % (LAG + 1)][i], a[i]);
    };
    const auto operand = [&](int t) { return w_operand<NN>(w + (t >> 2) * T::w_bytes, wj, t & 3); };
    wf[0] = first;
#pragma unroll
    for (int t = 0; t < T::parts * 4; ++t) {
        if (t + 1 < T::parts * 4) wf[(t + 1) & 1] = operand(t + 1);
#pragma unroll
        for (int m = 0; m < T::mt; ++m) {
            const int n = t * T::mt + m;
            p[n % (LAG + 1)] =
                __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wf[t & 1], x[m], f32x4{0, 0, 0, 0}, 0, 0, 0, 0, 0, 0);
            if (n >= LAG) add(n - LAG);
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
    for (int n = N - LAG; n < N; ++n) add(n);
    // the sums are made here, not where the compiler would move them, behind the next wait
#pragma unroll
    for (int n = 0; n < N; ++n) asm volatile("" : "+v"(acc[n / T::mt][n % T::mt]));
}

// STAGES buffers of a step: it is loaded STAGES - 1 steps before it is multiplied.
// 8192 x [5120, 55296] takes 2200 to 2280 us (2030 to 2110 TFLOP/s): 27 rounds of 40 steps of 2.0 to 2.1 us, of which
// the instructions take 1.4 at the rate that products of this card reach.  A unit's registers and LDS hold one such
// workgroup, so that nothing runs beside its waits, its barrier and a step's first reads.
// With few tokens the loads are all: 96 x [5120, 55296] 60 us, W at 4.8 TB/s with x beside it, through the
// same path into LDS.
// (Eight waves: with four, and all registers for one wave a SIMD, the compiler puts products
// into accumulation registers, which an FMA cannot read.)
// ONCE: one row of tiles, so W is read once and goes past the caches (96 x [5120, 27648] 44.0 and
// 40.0 us, 40 x [7168, 5120] 16.9 and 14.7).
template <typename T, bool NN, int STAGES, bool ONCE>
__global__ __launch_bounds__(T::threads) void k_fp8_tile(GemmArgs g) {
    constexpr int stage = T::x_bytes + T::parts * T::w_bytes, loads = T::xi + T::parts * T::wi, s_at = STAGES * stage;
    static_assert((STAGES - 2) * loads <= 63 && STAGES <= 5, "buffers: two for the scales of four steps");
    __shared__ __attribute__((aligned(1024))) uint8_t s_mem[s_at + 2 * T::s_bytes];
    const int wave = __builtin_amdgcn_readfirstlane(wave_id()), c16 = lane_id() & 15;
    const int wm = wave % T::WM, wj = wave / T::WM;
    const Work k = work_of(g);
    int m0, j0;
    tile_origin<T>(g, k.tile, m0, j0);
    const int64_t c0 = (int64_t)k.s0 * GB, w_step = NN ? (int64_t)GB * g.K : GB;
    const uint8_t *xb = load_base(g.x + (int64_t)m0 * g.C + c0);
    const uint8_t *wb = load_base(NN ? g.w + c0 * g.K + j0 : g.w + (int64_t)j0 * g.K + c0);
    const int blocks = (g.J + GB - 1) / GB;
    Loads<T, NN> l(g, m0, j0);
    const uint32_t mem = __builtin_amdgcn_readfirstlane(lds_at(s_mem));
    const auto issue = [&](int s) {
        const uint32_t at = mem + (uint32_t)((s - k.s0) % STAGES) * stage;
        const int left = g.C - s * GB;
        if (s == k.s0 || s % 4 == 0) {
            const int to = s_at + (s / 4 & 1) * T::s_bytes;
            l.load_s(g, m0, s & ~3, s_mem + to, mem + to);
        }
        if (left < GB) {
            l.end_x(left);
#pragma unroll
            for (int p = 0; p < T::parts; ++p) l.end_w(g, p, left);
        }
        l.load_x(at, xb);
#pragma unroll
        for (int p = 0; p < T::parts; ++p) l.template load_w<ONCE>(at + T::x_bytes + p * T::w_bytes, wb, p);
        xb += GB, wb += w_step;
    };
    f32x4 acc[T::parts * 4][T::mt];
#pragma unroll
    for (int t = 0; t < T::parts * 4; ++t)
#pragma unroll
        for (int m = 0; m < T::mt; ++m) acc[t][m] = f32x4{0, 0, 0, 0};

    for (int s = k.s0; s < k.s0 + STAGES - 1 && s < k.s1; ++s) issue(s);
    // W's scales of 64 steps, a lane's each: a step takes its own without waiting for a load
    float sw[T::parts];
    const bool end = Loads<T, NN>::near_end(g, m0);
    for (int s = k.s0; s < k.s1; ++s) {
        if (((s - k.s0) & 63) == 0) {
            const int64_t at = s + lane_id() < g.steps ? s + lane_id() : g.steps - 1;
#pragma unroll
            for (int p = 0; p < T::parts; ++p)  // (a tile's last part may lie past the last column)
                sw[p] = g.sw[(int64_t)(j0 / GB + p < blocks ? j0 / GB + p : blocks - 1) * g.gwj + at * g.gwc];
#pragma unroll
            for (int p = 0; p < T::parts; ++p) asm volatile("" : "+v"(sw[p]));  // waited for here, not in every step
        }
        int place[T::mt];
#pragma unroll
        for (int m = 0; m < T::mt; ++m) {
            const int r = wm * T::tm + m * 16 + c16;
            place[m] = r * 4 + (s & 3);
            if (end) place[m] += Loads<T, NN>::late(g, m0 + r, s);
        }
        // (a step may have loaded scales too, as its first load: that is then waited for as well)
        if (s + STAGES - 2 < k.s1) wait_loads<(STAGES - 2) * loads>();
        else wait_loads<0>();
        lds_barrier();  // this step is there, and the last one's buffer is free
        uint8_t *const at = s_mem + ((s - k.s0) % STAGES) * stage;
        if (g.C - s * GB < GB) clear_end<T>(at, g.C - s * GB);
        sched_fence();
        const float *const scale = reinterpret_cast<const float *>(s_mem + s_at + (s / 4 & 1) * T::s_bytes);
        i32x8 x[T::mt];
        float f[T::parts][T::mt];
        const i32x8 w0 = w_operand<NN>(at + T::x_bytes, wj, 0);
#pragma unroll
        for (int m = 0; m < T::mt; ++m) {
            const int r = wm * T::tm + m * 16 + c16;
            x[m] = row_operand(at, r, swap_x(r));
        }
#pragma unroll
        for (int m = 0; m < T::mt; ++m) f[0][m] = scale[place[m]];
        sched_fence();
        if (s + STAGES - 1 < k.s1) issue(s + STAGES - 1);  // (behind the reads, which the products wait for)
        sched_fence();
#pragma unroll
        for (int p = T::parts - 1; p >= 0; --p) {
            const float b = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(sw[p]), (s - k.s0) & 63));
#pragma unroll
            for (int m = 0; m < T::mt; ++m) f[p][m] = f[0][m] * b;
        }
        multiply<T, NN>(at + T::x_bytes, wj, w0, x, f, acc);
    }
    store_results<T, NN>(g, k, m0, j0, acc);
}

// ---- up to 16 tokens -------------------------------------------------------------------
// The time is that of reading W, a wave's share of it through LDS buffers of its own and
// without a barrier: a workgroup has RT times 16 rows of W, and its NW waves take their steps of
// 128 columns in turn, each D - 1 of its steps ahead (with x's and the scales).  The waves' sums
// are added through LDS, in their order.  Each workgroup reads x again, out of L2, so that 32 rows
// halve what 16 rows' reads cost: x [55296, 5120], 8 tokens 45.3 -> 42.2 us, 16 tokens 57.6 -> 47.8;
// one token 40.7 -> 41.0, x [28672, 5120] 22.8 -> 23.6.  Where they are too few for the chip,
// workgroups have 16 rows and more waves (kRows).
template <int NX, int NW, int D, int RT>
__global__ __launch_bounds__(NW *kWave) void k_fp8_rows(GemmArgs g) {
    constexpr int w_bytes = RT * 16 * GB, x_bytes = NX * GB, stage = w_bytes + x_bytes + 256;
    constexpr int wi = RT * 2, xi = x_bytes / 1024, loads = wi + xi + 1;
    static_assert(NX % 8 == 0 && NX <= 16 && (D - 1) * loads <= 63, "rows of x");
    __shared__ __attribute__((aligned(1024))) uint8_t s_mem[NW * D * stage];
    const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(wave_id()), c16 = lane & 15, q = lane >> 4;
    const int n0 = (int)blockIdx.x * RT * 16;
    const auto clamped = [](int r, int n) { return (uint32_t)(r < n ? r : n - 1); };
    const uint8_t *const wb = load_base(g.w + (int64_t)n0 * g.K), *const xb = load_base(g.x);
    const float *const sb = load_base(g.sx);
    const scalar_floats sw = (scalar_floats)(uint64_t)g.sw + (int64_t)(n0 / GB) * g.gwj;
    const int r8 = lane >> 3, pieces[2] = {(lane & 7) ^ swap_x(r8), (lane & 7) ^ swap_x(r8 + 8)};  // of rows r8 and r8 + 8
    uint32_t wo[wi];
#pragma unroll
    for (int i = 0; i < wi; ++i) wo[i] = (clamped(n0 + i * 8 + r8, g.J) - n0) * (uint32_t)g.K;
    const uint32_t xo[2] = {clamped(r8, g.M) * (uint32_t)g.K, clamped(r8 + 8, g.M) * (uint32_t)g.K};
    const uint32_t so = clamped(c16, g.M) * (uint32_t)g.gx * 4;
    uint8_t *const mine = s_mem + wave * D * stage;
    const uint32_t mem = __builtin_amdgcn_readfirstlane(lds_at(mine));
    const auto issue = [&](int s, int turn) {
        const uint32_t at = mem + (uint32_t)(turn % D) * stage;
        const int left = g.K - s * GB;
        uint32_t c[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) c[i] = (uint32_t)(s * GB + (pieces[i] * 16 < left ? pieces[i] * 16 : 0));
#pragma unroll
        for (int i = 0; i < wi; ++i) load_lds16_once(at + i * 1024, wb, wo[i] + c[i & 1]);
#pragma unroll
        for (int i = 0; i < xi; ++i) load_lds16(at + w_bytes + i * 1024, xb, xo[i] + c[i]);
        load_lds4(at + w_bytes + x_bytes, sb, so + (uint32_t)s * 4);
    };
    f32x4 acc[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) acc[t] = f32x4{0, 0, 0, 0};
    int ahead = wave, turns = 0, turn = 0;
    for (int i = 0; i < D - 1; ++i, ahead += NW)
        if (ahead < g.steps) issue(ahead, turns++);
    for (int s = wave; s < g.steps; s += NW, ++turn) {
        if (ahead < g.steps) {
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the last step's reads are done: its buffer is free
            issue(ahead, turns++);
            ahead += NW;
            wait_loads<(D - 1) * loads>();
        } else {
            wait_loads<0>();
        }
        uint8_t *const at = mine + (turn % D) * stage;
        if (g.K - s * GB < GB) {  // the pieces of x past the end are zero
            const int from = (g.K - s * GB) / 16, gone = 8 - from;
            for (int i = lane; i < NX * gone; i += kWave) {
                const int r = i / gone, p = from + i % gone;
                *reinterpret_cast<u32x4 *>(at + w_bytes + r * GB + (p ^ swap_x(r)) * 16) = u32x4{0, 0, 0, 0};
            }
        }
        const auto operand = [&](const uint8_t *m, int r) { return row_operand(m, r, swap_x(r)); };
        const float f = reinterpret_cast<const float *>(at + w_bytes + x_bytes)[lane] * sw[(int64_t)s * g.gwc];
        const i32x8 x = operand(at + w_bytes, c16 % NX);
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            const f32x4 p = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(operand(at, t * 16 + c16), x,
                                                                             f32x4{0, 0, 0, 0}, 0, 0, 0, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[t][i] = __builtin_fmaf(f, p[i], acc[t][i]);
        }
    }
    __syncthreads();
    f32x4 *const sums = reinterpret_cast<f32x4 *>(s_mem);
#pragma unroll
    for (int t = 0; t < RT; ++t) sums[(t * NW + wave) * kWave + lane] = acc[t];
    __syncthreads();
    if (wave >= RT || c16 >= g.M) return;  // wave t joins tile t
    f32x4 all = sums[wave * NW * kWave + lane];
    for (int i = 1; i < NW; ++i) all += sums[(wave * NW + i) * kWave + lane];
    const int col = n0 + wave * 16 + q * 4;
    if (g.bias) store_result<true>(g, c16, col, all);
    else store_result<false>(g, c16, col, all);
}

// The form, and how the work is shared: one round of workgroups after the other as long as each
// fills the chip; the tiles that are left over share the chip among them, in as many shares as pay.
constexpr int kUnits = 256;  // compute units

struct GemmPlan {
    int kind, bm, bj, whole, shares, per;
    int64_t tiles_m, tiles_j;
};

// The form is the one that takes the least time by this estimate.  Microseconds of a step while
// the chip is full, measured with 256 tiles of 64 steps, or, where one row of tiles reads W once,
// with 55296 x 5120 and 5120 x 27648; a second launch, a share in it and a float32 value written and
// read again as measured for the shared tiles of 1 to 512 rows.  By kind, in microseconds:
//   [2048, 8192] x [8192, 4096]   94.6   80.2  101   147
//   [4096, 8192] x [8192, 4096]  129    163    204   292
//   [96, 5120] x [5120, 55296]     -     60.0   75.9  99.0
//   [96, 27648] x [27648, 5120]    -     36.7   40.4  50.7
//   [24, 27648] x [27648, 5120]    -     33.7   35.7  29.3
//   [128, 14336] x [14336, 4096]   -     29.8   24.5  27.2
// (256 x 128 in place of 128 x 256: 85.9 and 165 of 2048 and 4096 rows, 104 of 96 rows x
// [5120, 55296], whose tiles are half empty then.)  Shares: one row x [27200, 128] in 213 of them
// 58.3 us, in 43 12.1; 100 rows 35.2 and 13.5.
struct GemmKind {
    int bm, bj;
    float step, once;
};

constexpr GemmKind kKinds[] = {{256, 256, 2.03f, 2.03f}, {128, 256, 1.28f, 1.45f}, {128, 128, 0.81f, 0.95f}, {64, 128, 0.62f, 0.74f}};

// k_fp8_rows: rows of W and waves of a workgroup; microseconds of a turn (a step of each wave) with
// up to 8 tokens and up to 16.  W comes in at 6.9 and 6.0 TB/s at most.  Microseconds in 32 rows, in 16
// rows and in tiles (nn has no such form: W's rows are what it contracts):
//                    one token            16 tokens
//   [7168, 5120]      7.8   7.8  12.8      9.2  11.8  13.3
//   [4096, 14336]    13.3  10.9  16.6     17.8  13.9  17.1
//   [5120, 27648]    24.4  28.6  28.1     33.0  44.2  28.8
//   [55296, 5120]    41.0  40.7  50.9     47.8  57.6  52.1
//   [128, 27200]     25.2  14.7  12.1     36.0  24.6  12.7
struct RowsKind {
    int rows, waves;
    float turn[2];
};

constexpr RowsKind kRows[] = {{32, 4, {0.46f, 0.62f}}, {16, 8, {0.5f, 0.85f}}};
constexpr int kRowsFrom = 4;  // kind of the first of them

inline GemmPlan gemm_plan(int64_t M, int64_t J, int64_t C, bool nn) {
    const int64_t steps = (C + GB - 1) / GB;
    GemmPlan best{};
    float least = 0;
    const auto consider = [&](const GemmPlan &p, float t) {
        if (best.per == 0 || t < least) best = p, least = t;
    };
    if (!nn && M <= 16)
        for (int i = 0; i < 2; ++i) {
            const RowsKind &k = kRows[i];
            const int64_t wgs = (J + k.rows - 1) / k.rows, turns = (steps + k.waves - 1) / k.waves;
            const float t = (float)((wgs + kUnits - 1) / kUnits * turns) * k.turn[M > 8];
            const float bytes = (float)(J * C) / (M > 8 ? 6.0e6f : 6.9e6f);
            consider({kRowsFrom + i, 16, k.rows, (int)wgs, 1, (int)steps, 1, wgs}, std::max(t, bytes) + 2.5f);
        }
    for (int kind = 0; kind < 4; ++kind) {
        const GemmKind &k = kKinds[kind];
        const int64_t tiles_m = (M + k.bm - 1) / k.bm, tiles_j = (J + k.bj - 1) / k.bj, tiles = tiles_m * tiles_j;
        const int64_t rest = tiles % kUnits;
        const float step = M <= k.bm ? k.once : k.step;
        for (int64_t most = rest ? std::min<int64_t>(kUnits / rest, steps) : 1; most >= 1; most /= 2) {
            GemmPlan p{kind, k.bm, k.bj, 0, 1, (int)((steps + most - 1) / most), tiles_m, tiles_j};
            p.shares = (int)((steps + p.per - 1) / p.per);
            p.whole = (int)(p.shares > 1 ? tiles - rest : tiles);
            float t = (float)((p.whole + kUnits - 1) / kUnits * steps) * step + 2.0f;
            if (p.shares > 1)  // the shared tiles, and the launch that joins them
                t += (float)p.per * step + 4.0f + 0.07f * (float)p.shares +
                     (float)(rest * p.shares * std::min<int64_t>(M, k.bm) * k.bj) * 8.0f / 5e6f;
            consider(p, t);
        }
    }
    return best;
}

// Bytes that hold the shared tiles of every plan for up to M rows: at most 128 tiles, whose shares
// are at most 256 and no more than their steps, of the largest kind (256 rows only beyond 128: below, its plan
// is that of 128 rows at a longer step).  The plans themselves rise and fall with M.
inline int64_t gemm_ws_bound(int64_t M, int64_t J, int64_t C) {
    const int64_t steps = (C + GB - 1) / GB;
    int64_t most = 0;
    for (const GemmKind &k : kKinds) {
        if (steps < 2 || (k.bm > 128 && M <= 128)) continue;
        const int64_t tiles = std::min<int64_t>((M + k.bm - 1) / k.bm * ((J + k.bj - 1) / k.bj), kUnits / 2);
        most = std::max(most, std::min<int64_t>(kUnits, tiles * steps) * k.bm * k.bj * 4);
    }
    return most;
}

template <typename T, bool NN, int STAGES>
inline void launch_tiles(const GemmArgs &g, hipStream_t stream) {
    const int64_t rest = (int64_t)g.tiles_m * g.tiles_j - g.whole;
    const dim3 grid((unsigned)(g.whole + rest * g.shares)), block(T::threads);
    if (T::BM <= 128 && g.tiles_m == 1) k_fp8_tile<T, NN, STAGES, T::BM <= 128><<<grid, block, 0, stream>>>(g);
    else k_fp8_tile<T, NN, STAGES, false><<<grid, block, 0, stream>>>(g);
    if (rest) k_fp8_join<T, NN><<<dim3(T::results, (unsigned)rest), block, 0, stream>>>(g);
}

template <int NW, int RT>
inline void launch_rows(const GemmArgs &g, hipStream_t stream) {
    const dim3 grid((unsigned)g.tiles_j), block(NW * kWave);
    if (g.M <= 8) k_fp8_rows<8, NW, 3, RT><<<grid, block, 0, stream>>>(g);
    else k_fp8_rows<16, NW, 3, RT><<<grid, block, 0, stream>>>(g);
}

template <bool NN>
inline void launch_gemm(const GemmPlan &p, const GemmArgs &g, hipStream_t stream) {
    switch (p.kind) {
    case 0: return launch_tiles<Tile<256, 256, 4>, NN, 2>(g, stream);
    case 1: return launch_tiles<Tile<128, 256, 4>, NN, 3>(g, stream);
    case 2: return launch_tiles<Tile<128, 128, 4>, NN, 4>(g, stream);
    default: return launch_tiles<Tile<64, 128, 4>, NN, 5>(g, stream);
    }
}

}  // namespace pulse

using namespace pulse;

extern "C" {

int64_t pulse_fp8_gemm_ws_size(int64_t M, int64_t J, int64_t C) { return gemm_ws_bound(M, J, C); }

int32_t pulse_fp8_gemm_shares(int64_t M, int64_t J, int64_t C, int32_t nn) { return gemm_plan(M, J, C, nn).shares; }

int pulse_launch_fp8_gemm(const uint8_t *x, const float *sx, const uint8_t *w, const float *sw, const uint16_t *bias,
                          int32_t nn, int64_t M, int64_t n, int64_t k, uint16_t *y, int64_t ldy, void *ws,
                          hipStream_t stream) {
    const int64_t J = nn ? k : n, C = nn ? n : k, gk = (k + GB - 1) / GB;
    const GemmPlan p = gemm_plan(M, J, C, nn);
    const GemmArgs g{x, w, sx, sw, bias, y, static_cast<f32x4 *>(ws), ldy, (int32_t)M, (int32_t)J, (int32_t)C, (int32_t)k,
                     (int32_t)((C + GB - 1) / GB), nn ? 1 : (int32_t)gk, nn ? (int32_t)gk : 1, (int32_t)p.tiles_m,
                     (int32_t)p.tiles_j, (int32_t)((C + GB - 1) / GB), p.whole, p.shares, p.per};
    if (p.kind == kRowsFrom) launch_rows<4, 2>(g, stream);
    else if (p.kind > kRowsFrom) launch_rows<8, 1>(g, stream);
    else if (nn) launch_gemm<true>(p, g, stream);
    else launch_gemm<false>(p, g, stream);
    return hipGetLastError() == hipSuccess ? 0 : -5;
}
}
