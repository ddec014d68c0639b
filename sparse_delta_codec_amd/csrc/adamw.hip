// adamw.hip -- the trainer's step in front of the codec: the norm of a list of
// gradients with the factor that clips them, and one AdamW step over a list of
// tensors that writes the served BF16 view and, where asked, the sparse patch
// of the view's changed elements.
//
// The mathematics, per element, in float32 with every operation rounded once
// (no fused multiply-add: the library is built with -ffp-contract=off), so a
// step is bit for bit the same wherever an element lies in a launch:
//   g  = grad * scale
//   m' = b1 m + (1 - b1) g          v' = b2 v + (1 - b2) (g g)
//   u  = sqrt(v')
//   p' = p (1 - lr wd) - (lr / (1 - b1^t)) (m' / (u / sqrt(1 - b2^t) + eps))
//   with lr wd below 2^-23: p' = p - ((lr / (1 - b1^t)) (...) + p (lr wd)), for the
//   float32 numbers below 1 are 2^-24 apart, and 1 - lr wd would be off by a third of
//   lr wd or more: at lr = 2e-6 and wd = 0.01 it is 1 and nothing ever decays
//   b' = bf16(p')                   patch: the elements where b' != b
// States in 8 bits: m and u, in blocks of 256 elements of one tensor, as
// E4M3 codes times amax / 448.  u rather than v is kept because a square root
// halves the exponents: 18 binades of u are 36 of v.  Codes are rounded up or
// down at random, with the chance that makes the expectation exact: at
// b2 = 0.999 a step lowers u by at most 0.05%, far below half a code's spacing
// (3% to 6%), so rounding to nearest would never let a code come down.  The random
// bits are a mix of the element's place, its tensor's number and the caller's
// seed.  A u above zero gets at least the smallest code: a zero would divide
// the next update by eps alone.
#include "tiles.hpp"

namespace pulse {

struct AdamSeg {  // the layout of pulse_adamw_segment
    float *p;
    const void *g;
    void *m;
    void *v;
    float *m_scale;
    float *v_scale;
    uint16_t *b;
    int64_t n;
    int64_t tile0;
    float lr_mult;
    float weight_decay;
};

struct GradSeg {  // the layout of pulse_grad_segment
    const void *g;
    int64_t n;
    int64_t tile0;
};

struct AdamArgs {
    const AdamSeg *segs;
    const uint32_t *tile_seg;
    const float *d_scale;
    int32_t nseg;
    uint32_t npieces;
    uint32_t seed;
    float lr, b1, omb1, b2, omb2, eps, inv_bc1, inv_sqrt_bc2;
    // the patch (PATCH only)
    int32_t *idx;
    uint16_t *val;
    int64_t cap;
    int64_t *seg_offsets;
    uint32_t *d_status;
    uint32_t *counts;  // [step's waves] changed elements
    uint32_t *flags;   // [tiles][512] a bit per element of a tile, in order
};

constexpr int AW_BLOCK = 256;  // elements of a state block: one group of a wave
constexpr float kLargest = 0x1.FFFFFEp127f;
constexpr float kTinyBlock = 0x1p-96f;  // blocks below are stored as zero (448 / amax would overflow)

// 32 well-mixed bits of x: xor-shifts and products with odd constants (the
// fractional bits of the square roots of 2 and 3).
__device__ __forceinline__ uint32_t aw_mix(uint32_t x) {
    x ^= x >> 16;
    x *= 0x6A09E667u;
    x ^= x >> 15;
    x *= 0xBB67AE85u;
    return x ^ (x >> 16);
}

// |x| * inv (at most 448 and a rounding) to an E4M3 code: the bits below the
// code's last one are added to 20 random bits, the carry rounds up.  Below
// 2^-6 the codes are evenly spaced, which adding 2^-6 turns into the spacing
// of the binade above it.
__device__ __forceinline__ uint32_t aw_code(float x, float inv, uint32_t rnd20) {
    const float y = __builtin_fabsf(x) * inv;
    const bool small = y < 0x1p-6f;
    const float t = y + (small ? 0x1p-6f : 0.0f);
    const uint32_t c = ((__float_as_uint(t) + rnd20) >> 20) - (small ? 968u : 960u);
    return c < 126u ? c : 126u;
}

// wave-wide maximum of the absolute values' bits, in every lane (a NaN, whose
// bits exceed every number's, wins)
__device__ __forceinline__ uint32_t aw_wave_max(uint32_t v) {
    v = wave_incl_max(v);
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

template <bool BF16G>
struct GradVec;
template <>
struct GradVec<false> {
    typedef u32x4 T;
};
template <>
struct GradVec<true> {
    typedef u32x2 T;
};

template <bool BF16G>
__device__ __forceinline__ float grad_of(const typename GradVec<BF16G>::T &v, int k) {
    if constexpr (BF16G) return __uint_as_float((k & 1) ? (v[k >> 1] & 0xFFFF0000u) : (v[k >> 1] << 16));
    else return __uint_as_float(v[k]);
}

// Four consecutive elements of E bytes each at element e of a tensor of n
// (FULL: all inside), as 32-bit words; elements past n read as zero.
template <bool FULL, typename V>
__device__ __forceinline__ V load4(const void *p, int64_t e, int64_t n) {
    constexpr int E = sizeof(V) / 4;
    const char *q = static_cast<const char *>(p) + e * E;
    if (FULL || e + 3 < n) return __builtin_nontemporal_load(reinterpret_cast<const V *>(q));
    union {
        V v;
        uint8_t c[sizeof(V)];
    } u = {};
#pragma unroll
    for (int k = 0; k < 3; ++k)
        if (e + k < n) {
            if constexpr (E == 4) reinterpret_cast<uint32_t *>(u.c)[k] = reinterpret_cast<const uint32_t *>(q)[k];
            else if constexpr (E == 2) reinterpret_cast<uint16_t *>(u.c)[k] = reinterpret_cast<const uint16_t *>(q)[k];
            else u.c[k] = reinterpret_cast<const uint8_t *>(q)[k];
        }
    return u.v;
}

template <bool FULL, typename V>
__device__ __forceinline__ void store4v(void *p, int64_t e, int64_t n, V v) {
    constexpr int E = sizeof(V) / 4;
    char *q = static_cast<char *>(p) + e * E;
    if (FULL || e + 3 < n) {
        __builtin_nontemporal_store(v, reinterpret_cast<V *>(q));
        return;
    }
    union {
        V v;
        uint8_t c[sizeof(V)];
    } u;
    u.v = v;
#pragma unroll
    for (int k = 0; k < 3; ++k)
        if (e + k < n) {
            if constexpr (E == 4) reinterpret_cast<uint32_t *>(q)[k] = reinterpret_cast<uint32_t *>(u.c)[k];
            else if constexpr (E == 2) reinterpret_cast<uint16_t *>(q)[k] = reinterpret_cast<uint16_t *>(u.c)[k];
            else reinterpret_cast<uint8_t *>(q)[k] = u.c[k];
        }
}

// What one wave needs of its tensor.
struct AdamTensor {
    AdamSeg s;
    float scale, decay, rate, size;  // decay: the factor, or 1 and the rate apart
    uint32_t key;
};

// G groups of 256 elements of one wave (lane l: elements 4l .. 4l+3 of each
// group, the first group at element e0 of the tensor): the step, its stores,
// and the changed flags (bit 4g+k) for the patch.
template <int G, bool FULL, bool BF16G, bool EIGHT, bool PATCH>
__device__ __forceinline__ uint32_t aw_chunk(const AdamArgs &a, const AdamTensor &t, int64_t e0) {
    typedef typename GradVec<BF16G>::T GV;
    const int64_t n = t.s.n;
    const int64_t el = e0 + 4 * lane_id();
    u32x4 pv[G];
    GV gv[G];
    u32x4 mv[G], vv[G];
    uint32_t mc[G], vc[G];
    u32x2 ov[G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
        const int64_t e = el + g * 256;
        pv[g] = load4<FULL, u32x4>(t.s.p, e, n);
        gv[g] = load4<FULL, GV>(t.s.g, e, n);
        if constexpr (EIGHT) {
            mc[g] = load4<FULL, uint32_t>(t.s.m, e, n);
            vc[g] = load4<FULL, uint32_t>(t.s.v, e, n);
        } else {
            mv[g] = load4<FULL, u32x4>(t.s.m, e, n);
            vv[g] = load4<FULL, u32x4>(t.s.v, e, n);
        }
        if constexpr (PATCH) ov[g] = load4<FULL, u32x2>(t.s.b, e, n);
    }
    // the blocks' scales: lane g of the wave holds block e0 / 256 + g
    float ms = 0.0f, vs = 0.0f;
    if constexpr (EIGHT) {
        const int64_t blk = e0 / AW_BLOCK + (lane_id() & (G - 1));
        if (FULL || blk * AW_BLOCK < n) {
            ms = t.s.m_scale[blk];
            vs = t.s.v_scale[blk];
        }
    }
    uint32_t flags = 0, mmax[G], umax[G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
        float m4[4], v4[4];
        if constexpr (EIGHT) {
            const float sm = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(ms), g));
            const float sv = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(vs), g));
            const f32x2_t m01 = __builtin_amdgcn_cvt_pk_f32_fp8((int)mc[g], false);
            const f32x2_t m23 = __builtin_amdgcn_cvt_pk_f32_fp8((int)mc[g], true);
            const f32x2_t u01 = __builtin_amdgcn_cvt_pk_f32_fp8((int)vc[g], false);
            const f32x2_t u23 = __builtin_amdgcn_cvt_pk_f32_fp8((int)vc[g], true);
            m4[0] = m01.x * sm, m4[1] = m01.y * sm, m4[2] = m23.x * sm, m4[3] = m23.y * sm;
            v4[0] = u01.x * sv, v4[1] = u01.y * sv, v4[2] = u23.x * sv, v4[3] = u23.y * sv;
#pragma unroll
            for (int k = 0; k < 4; ++k) v4[k] = v4[k] * v4[k];
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) m4[k] = __uint_as_float(mv[g][k]), v4[k] = __uint_as_float(vv[g][k]);
        }
        float p4[4], u4[4];
        uint32_t mm = 0, um = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float gr = grad_of<BF16G>(gv[g], k) * t.scale;
            m4[k] = m4[k] * a.b1 + gr * a.omb1;
            v4[k] = v4[k] * a.b2 + (gr * gr) * a.omb2;
            u4[k] = sqrtf(v4[k]);
            const float upd = m4[k] / (u4[k] * a.inv_sqrt_bc2 + a.eps);
            const float p = __uint_as_float(pv[g][k]), step = upd * t.size;
            // one of decay = 1 and rate = 0 holds: a zero added to the step changes nothing (a master that is
            // infinite stays so, as the largest number stands for it in the product)
            p4[k] = p * t.decay - (step + __builtin_amdgcn_fmed3f(p, -kLargest, kLargest) * t.rate);
            if constexpr (EIGHT) {
                const uint32_t mb = __float_as_uint(m4[k]) & 0x7FFFFFFFu, ub = __float_as_uint(u4[k]) & 0x7FFFFFFFu;
                mm = mb > mm ? mb : mm;
                um = ub > um ? ub : um;
            }
        }
        const int64_t e = el + g * 256;
        store4v<FULL, u32x4>(t.s.p, e, n, u32x4{__float_as_uint(p4[0]), __float_as_uint(p4[1]), __float_as_uint(p4[2]),
                                                __float_as_uint(p4[3])});
        if (t.s.b) {
            const uint32_t q0 = cast_pair(p4[0], p4[1]), q1 = cast_pair(p4[2], p4[3]);
            store4v<FULL, u32x2>(t.s.b, e, n, u32x2{q0, q1});
            if constexpr (PATCH) {
                uint32_t f = (uint32_t)pair_flags(q0 ^ ov[g].x, q1 ^ ov[g].y);
                if (!FULL) {
                    const int64_t left = n - e;
                    f &= left >= 4 ? 0xFu : (left > 0 ? (1u << left) - 1u : 0u);
                }
                flags |= f << (4 * g);
            }
        }
        if constexpr (EIGHT) {
#pragma unroll
            for (int k = 0; k < 4; ++k) mv[g][k] = __float_as_uint(m4[k]), vv[g][k] = __float_as_uint(u4[k]);
            mmax[g] = aw_wave_max(mm);
            umax[g] = aw_wave_max(um);
        } else {
            store4v<FULL, u32x4>(t.s.m, e, n, u32x4{__float_as_uint(m4[0]), __float_as_uint(m4[1]),
                                                    __float_as_uint(m4[2]), __float_as_uint(m4[3])});
            store4v<FULL, u32x4>(t.s.v, e, n, u32x4{__float_as_uint(v4[0]), __float_as_uint(v4[1]),
                                                    __float_as_uint(v4[2]), __float_as_uint(v4[3])});
        }
    }
    if constexpr (EIGHT) {
        // the eight blocks' scales in one pass of divisions: lane 2g + (0: m, 1: u)
        const int q = lane_id() & 7;
        uint32_t ab = 0;
#pragma unroll
        for (int g = 0; g < G; ++g) {
            ab = q == 2 * g ? mmax[g] : ab;
            ab = q == 2 * g + 1 ? umax[g] : ab;
        }
        const float amax = __uint_as_float(ab);
        const bool live = !(amax < kTinyBlock);
        const float scale = live ? amax / 448.0f : 0.0f;
        const float inv = live ? 448.0f / amax : 0.0f;
        const int64_t blk = e0 / AW_BLOCK + (q >> 1);
        if (lane_id() < 2 * G && (FULL || blk * AW_BLOCK < n)) ((q & 1) ? t.s.v_scale : t.s.m_scale)[blk] = scale;
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const int64_t e = el + g * 256;
            const float im = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(inv), 2 * g));
            const float iu = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(inv), 2 * g + 1));
            uint32_t cm = 0, cu = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t r = aw_mix((uint32_t)e + (uint32_t)k + t.key);
                const float m = __uint_as_float(mv[g][k]), u = __uint_as_float(vv[g][k]);
                const uint32_t c = aw_code(m, im, r & 0xFFFFFu) | ((mv[g][k] >> 24) & 0x80u);
                uint32_t d = aw_code(u, iu, r >> 12);
                if (d == 0 && u > 0.0f && iu > 0.0f) d = 1;
                cm |= c << (8 * k);
                cu |= d << (8 * k);
            }
            store4v<FULL, uint32_t>(t.s.m, e, n, cm);
            store4v<FULL, uint32_t>(t.s.v, e, n, cu);
        }
    }
    return flags;
}

// A wave's changed flags of 1024 elements (lane l: bit 4 g + k for element 256 g +
// 4 l + k) as 32 words in element order: lane 8 j + g, g < 4, gets word 8 g + j.
__device__ __forceinline__ uint32_t pack_flags(uint32_t f) {
    using namespace dppc;
    uint32_t word[4];
#pragma unroll
    for (int g = 0; g < 4; ++g) {  // the nibbles of eight lanes, in the first of them
        uint32_t v = (f >> (4 * g)) & 0xFu;
        v |= dpp_mov<kRowShl1, 0xf, 0xf>(0u, v) << 4;
        v |= dpp_mov<kRowShl2, 0xf, 0xf>(0u, v) << 8;
        word[g] = v | dpp_mov<kRowShl4, 0xf, 0xf>(0u, v) << 16;
    }
    const uint32_t w1 = dpp_mov<kRowShr1, 0xf, 0xf>(0u, word[1]), w2 = dpp_mov<kRowShr2, 0xf, 0xf>(0u, word[2]);
    const uint32_t w3 = dpp_mov<0x113 /*row shift right by 3*/, 0xf, 0xf>(0u, word[3]);
    const int g = lane_id() & 3;
    return g == 0 ? word[0] : (g == 1 ? w1 : (g == 2 ? w2 : w3));
}

// One workgroup of four waves per piece, E elements a wave (4096: a piece is a whole
// tile; 1024 and 256: a quarter and a sixteenth).  With a patch each wave leaves its changed flags and
// their number for k_adamw_patch.  Bound by HBM: 487.6M elements with 32-bit states,
// 28 bytes each, 2.56 ms (5.3 TB/s, as a large copy); 218M with 8-bit states and the
// flags, 20 bytes each, 0.74 ms (5.9 TB/s); 475K elements 4.4 us.
template <int E, bool BF16G, bool EIGHT, bool PATCH>
__global__ __launch_bounds__(CD_THREADS) void k_adamw(AdamArgs a) {
    constexpr int kPerTile = CD_TILE / (4 * E), G = E < 1024 ? E / 256 : 4, CH = E / (256 * G);
    const uint32_t piece = blockIdx.x, tile = piece / kPerTile;
    const uint32_t s = (uint32_t)__builtin_amdgcn_readfirstlane((int)a.tile_seg[tile]);
    AdamTensor t{};
    if (s < (uint32_t)a.nseg) t.s = a.segs[s];
    const int64_t lt = (int64_t)tile - t.s.tile0;
    const uintptr_t all = reinterpret_cast<uintptr_t>(t.s.p) | reinterpret_cast<uintptr_t>(t.s.g) |
                          reinterpret_cast<uintptr_t>(t.s.m) | reinterpret_cast<uintptr_t>(t.s.v) |
                          reinterpret_cast<uintptr_t>(t.s.b);
    const bool ok = s < (uint32_t)a.nseg && t.s.n >= 1 && t.s.n <= 2147483647ll && lt >= 0 && lt * CD_TILE < t.s.n &&
                    (all & 15u) == 0 && t.s.p && t.s.g && t.s.m && t.s.v && (!PATCH || t.s.b) &&
                    (!EIGHT || (t.s.m_scale && t.s.v_scale));
    t.scale = a.d_scale ? *a.d_scale : 1.0f;
    const float lr = a.lr * t.s.lr_mult, rate = lr * t.s.weight_decay;
    const bool apart = __builtin_fabsf(rate) < 0x1p-23f;
    t.decay = apart ? 1.0f : 1.0f - rate;
    t.rate = apart ? rate : 0.0f;
    t.size = lr * a.inv_bc1;
    t.key = aw_mix(a.seed + (s + 1u) * 0x9E3779B1u);
    const bool skip = !(__builtin_fabsf(t.scale) <= 3.402823466e38f);  // NaN or infinite: no step
    const int w = __builtin_amdgcn_readfirstlane(wave_id()), l = lane_id();
    const int64_t wbase = lt * CD_TILE + (int64_t)(piece % kPerTile) * (4 * E) + (int64_t)w * E;
    uint64_t flags = 0;
    if (ok && !skip && wbase < t.s.n) {
        if (wbase + E <= t.s.n) {
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                flags |= (uint64_t)aw_chunk<G, true, BF16G, EIGHT, PATCH>(a, t, wbase + c * 1024) << (16 * c);
                sched_fence();
            }
        } else {
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                if (wbase + c * 1024 < t.s.n)
                    flags |= (uint64_t)aw_chunk<G, false, BF16G, EIGHT, PATCH>(a, t, wbase + c * 1024) << (16 * c);
                sched_fence();
            }
        }
    }
    if constexpr (PATCH) {
        const int64_t wave = (int64_t)piece * 4 + w;
        const uint32_t count = wave_reduce_sum((uint32_t)__builtin_popcountll(flags));
        if (l == 0) a.counts[wave] = count;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const uint32_t word = pack_flags((uint32_t)(flags >> (16 * c)));
            if ((l & 7) < G) a.flags[(wave * CH + c) * (8 * G) + (l & 7) * 8 + (l >> 3)] = word;
        }
    }
    if (!ok && threadIdx.x == 0) or_agent32(a.d_status, 0x10u /*PULSE_DS_BADSEGMENT*/);
}

// The patch: a workgroup takes a run of units of 4096 elements, whose first entry
// is the sum of the counts before it; each of its waves goes through its share, 64
// consecutive elements a lane, so that one scan ranks a unit's entries and a lane
// picks its own bit by bit.  The step has no place in the patch to wait for:
// placing a piece's entries by a ticket and a look-back within the step itself cost
// 23 ns a piece, one after the other, and 41 us before the first 1800 pieces had
// begun (5.2M elements: 57 us, with this kernel 28 + 6; 218M with 8-bit states: 895
// us, 741 + 47).  Ranked with ballots, four for every 256 elements as in the codec's
// passes, it was bound by its instructions: 85 to 119 us.
template <int E>
__global__ __launch_bounds__(CD_THREADS) void k_adamw_patch(AdamArgs a) {
    constexpr int kCounts = 4096 / E;  // the step's waves of a unit
    constexpr int kAtOnce = 4;       // entries whose values are on their way together
    __shared__ uint64_t s_sum[CD_THREADS / kWave];
    const int w = __builtin_amdgcn_readfirstlane(wave_id()), l = lane_id();
    const int64_t nu = (int64_t)a.npieces * E / 1024;
    const int64_t u0 = nu * blockIdx.x / gridDim.x, u1 = nu * (blockIdx.x + 1) / gridDim.x;
    const int64_t first = u0 + (u1 - u0) * w / 4, last = u0 + (u1 - u0) * (w + 1) / 4;
    const uint64_t *const flags = reinterpret_cast<const uint64_t *>(a.flags) + l;
    uint64_t next = first < last ? flags[first * kWave] : 0;
    uint64_t sum = 0;
    const u32x4 *c4 = reinterpret_cast<const u32x4 *>(a.counts);
    const int64_t before = u0 * kCounts;
    for (int64_t i = threadIdx.x; i < before / 4; i += CD_THREADS) {
        const u32x4 c = c4[i];
        sum += (uint64_t)c.x + c.y + ((uint64_t)c.z + c.w);
    }
    if (threadIdx.x < (before & 3)) sum += a.counts[before / 4 * 4 + threadIdx.x];
    sum = wave_reduce_sum(sum);
    if (l == 0) s_sum[w] = sum;
    __syncthreads();
    uint64_t run = s_sum[0] + s_sum[1] + s_sum[2] + s_sum[3];
    uint32_t mine = 0;
    for (int64_t i = before + l; i < first * kCounts; i += kWave) mine += a.counts[i];
    run += wave_reduce_sum(mine);
    // the tensor of the current unit, and the tiles it has
    const uint16_t *b = nullptr;
    int64_t tile0 = 0, tile1 = 0;
    for (int64_t i = first; i < last; ++i) {
        uint64_t bits = next;
        if (i + 1 < last) next = flags[(i + 1) * kWave];
        const int64_t tile = i / 4;
        if (tile >= tile1) {
            const uint32_t s = (uint32_t)__builtin_amdgcn_readfirstlane((int)a.tile_seg[tile]);
            b = nullptr;
            tile0 = tile;
            tile1 = tile + 1;
            if (s < (uint32_t)a.nseg) {
                const AdamSeg &seg = a.segs[s];
                const int64_t t1 = seg.tile0 + (seg.n + CD_TILE - 1) / CD_TILE;
                if (tile >= seg.tile0 && tile < t1) {
                    b = seg.b;
                    tile0 = seg.tile0;
                    tile1 = t1;
                }
                if (l == 0 && i % 4 == 0 && tile == seg.tile0) a.seg_offsets[s] = (int64_t)run;
            }
        }
        const uint32_t count = (uint32_t)__builtin_popcountll(bits), incl = wave_incl_sum(count);
        const uint32_t total = (uint32_t)__builtin_amdgcn_readlane((int)incl, 63);
        int64_t at = (int64_t)(run + incl - count);
        run += total;
        if (total == 0 || !b) continue;
        const int32_t e0 = (int32_t)((i - tile0 * 4) * 4096) + l * 64;
        while (__ballot(bits != 0)) {
            int32_t e[kAtOnce];
            uint16_t v[kAtOnce];
            int n = 0;
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) {
                e[k] = -1;
                if (bits) {
                    e[k] = e0 + __builtin_ctzll(bits);
                    v[k] = b[e[k]];
                    bits &= bits - 1;
                    n = k + 1;
                }
            }
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k)
                if (e[k] >= 0 && at + k < a.cap) {
                    a.idx[at + k] = e[k];
                    a.val[at + k] = v[k];
                }
            at += n;
        }
    }
    if (last == nu && first < last && l == 0) {
        a.seg_offsets[a.nseg] = (int64_t)run;
        if ((int64_t)run > a.cap) or_agent32(a.d_status, 1u /*PULSE_DS_CAPACITY*/);
    }
}

// ---- the norm of a list of gradients --------------------------------------------
// Squares are summed in float64 (a float32 square overflows at 1.8e19 and
// underflows below 1e-22), each workgroup's sum over its tiles goes to its own
// slot, and the workgroup that finishes last adds the slots in their order: no
// atomic's order reaches the result.
constexpr int GN_THREADS = 512;
constexpr int GN_MAX_BLOCKS = 512;

struct NormArgs {
    const GradSeg *segs;
    const uint32_t *tile_seg;
    int32_t nseg;
    uint32_t npieces;
    double mul, max_norm;
    float *out;
    uint32_t *done;    // workgroups finished; the last one sets it back to zero
    double *partial;
};

// 16 bytes of a tensor of n elements at element e (FULL: all inside); elements past n read as zero.
template <bool FULL, bool BF16G>
__device__ __forceinline__ u32x4 grad16(const void *p, int64_t e, int64_t n) {
    constexpr int kPer = BF16G ? 8 : 4;
    if (FULL || e + kPer <= n)
        return __builtin_nontemporal_load(
            reinterpret_cast<const u32x4 *>(static_cast<const char *>(p) + e * (16 / kPer)));
    union {
        u32x4 v;
        uint32_t w[4];
        uint16_t h[8];
    } u = {};
#pragma unroll
    for (int k = 0; k < kPer - 1; ++k)
        if (e + k < n) {
            if constexpr (BF16G) u.h[k] = static_cast<const uint16_t *>(p)[e + k];
            else u.w[k] = static_cast<const uint32_t *>(p)[e + k];
        }
    return u.v;
}

// A thread takes V 16-byte pieces of every gridDim-th part of a tile; the next
// part's are read while these are added, so that a workgroup has its loads in
// flight all the time (waiting for each part alone reached 2.7 to 4 TB/s): 975 MB in
// 144 us, 6.8 TB/s; 1.9 MB in 5.3 us.
template <int V, bool BF16G>
__global__ __launch_bounds__(GN_THREADS) void k_grad_norm(NormArgs a) {
    constexpr int kPer = BF16G ? 8 : 4, kPart = V * GN_THREADS * kPer, kParts = CD_TILE / kPart;
    __shared__ double s_sum[GN_THREADS / kWave];
    __shared__ uint32_t s_last;
    double sum[4] = {0.0, 0.0, 0.0, 0.0};
    const auto fetch = [&](uint32_t piece, u32x4 *v) {
        const uint32_t tile = piece / kParts;
        const uint32_t s = (uint32_t)__builtin_amdgcn_readfirstlane((int)a.tile_seg[tile]);
        GradSeg d{};
        if (s < (uint32_t)a.nseg) d = a.segs[s];
        const int64_t lt = (int64_t)tile - d.tile0;
        if (!(d.g && (reinterpret_cast<uintptr_t>(d.g) & 15u) == 0 && lt >= 0 && lt * CD_TILE < d.n)) {
            sum[0] = __builtin_nan("");  // a broken table entry: the norm is not a number
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = u32x4{0, 0, 0, 0};
            return;
        }
        const int64_t base = lt * CD_TILE + (int64_t)(piece % kParts) * kPart, e = base + kPer * (int)threadIdx.x;
        if (base + kPart <= d.n) {
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = grad16<true, BF16G>(d.g, e + i * (GN_THREADS * kPer), d.n);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = grad16<false, BF16G>(d.g, e + i * (GN_THREADS * kPer), d.n);
        }
    };
    u32x4 v[V], next[V];
    uint32_t piece = blockIdx.x;
    if (piece < a.npieces) fetch(piece, v);
    while (piece < a.npieces) {
        piece += gridDim.x;
        if (piece < a.npieces) fetch(piece, next);
        sched_fence();
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if constexpr (BF16G) {
                    const double x = (double)__uint_as_float(v[i][k] << 16);
                    const double y = (double)__uint_as_float(v[i][k] & 0xFFFF0000u);
                    sum[k] = __builtin_fma(x, x, sum[k]);
                    sum[k] = __builtin_fma(y, y, sum[k]);
                } else {
                    const double x = (double)__uint_as_float(v[i][k]);
                    sum[k] = __builtin_fma(x, x, sum[k]);
                }
            }
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = next[i];
    }
    double acc = (sum[0] + sum[1]) + (sum[2] + sum[3]);
    acc = wave_reduce_sum(acc);
    if (lane_id() == 0) s_sum[wave_id()] = acc;
    __syncthreads();
    if (threadIdx.x == 0) {
        double t = 0.0;
#pragma unroll
        for (int w = 0; w < GN_THREADS / kWave; ++w) t += s_sum[w];
        __hip_atomic_store(&a.partial[blockIdx.x], t, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        // the partial sum was written through to memory and has arrived there before the count goes
        // up: a release and acquire here would write back and invalidate the XCD's whole L2, and
        // 1024 of them took 50 us
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        s_last = add_agent32(a.done, 1u) == gridDim.x - 1;
    }
    __syncthreads();
    if (!s_last) return;
    double t = 0.0;
    for (uint32_t i = threadIdx.x; i < gridDim.x; i += GN_THREADS)
        t += __hip_atomic_load(&a.partial[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    t = wave_reduce_sum(t);
    if (lane_id() == 0) s_sum[wave_id()] = t;
    __syncthreads();
    if (threadIdx.x == 0) {
        double tot = 0.0;
#pragma unroll
        for (int w = 0; w < GN_THREADS / kWave; ++w) tot += s_sum[w];
        const double norm = __builtin_sqrt(tot) * a.mul;
        const double coef = a.max_norm / (norm + 1e-6);
        double scale = a.mul * (coef < 1.0 ? coef : 1.0);
        if (!(norm <= 1.7976931348623157e308)) scale = __builtin_nan("");
        a.out[0] = (float)scale;
        a.out[1] = (float)norm;
        st_agent32(a.done, 0u);
    }
}

}  // namespace pulse

using namespace pulse;

// A bit per element and a 4-byte count per wave of the step (4, 16 or 64 of a tile).
extern "C" size_t pulse_adamw_ws_bytes(int64_t ntiles) {
    return (size_t)(ntiles > 0 ? ntiles : 1) * (CD_TILE / 8 + 64 * sizeof(uint32_t));
}

extern "C" size_t pulse_grad_norm_ws_bytes(void) { return 256 + GN_MAX_BLOCKS * sizeof(double); }

namespace {

// Lists of fewer tiles than 4 per compute unit are cut into sixteenths of a tile, so
// that they spread over the chip (5.2M float32 elements: 23.8 us, in quarters 27.5;
// 0.48M with 8-bit states: 5.8 us, in quarters 8.5, for a wave's 1024 elements are
// 4 us of instructions).  With a patch only short lists are: every piece's counts
// are added up again by every workgroup of the patch (5.2M elements with 8-bit
// states: 32.7 us, in quarters 27.9; 1M: 12.4 and 12.7).
constexpr int64_t kWholeTiles = 1024, kPatchQuarterTiles = 64;
constexpr int64_t kPatchBlocks = 2048;

template <int E, bool BF16G, bool EIGHT, bool PATCH>
void launch_adamw(AdamArgs a, int64_t ntiles, hipStream_t stream) {
    a.npieces = (uint32_t)(ntiles * (CD_TILE / (4 * E)));
    k_adamw<E, BF16G, EIGHT, PATCH><<<dim3(a.npieces), dim3(CD_THREADS), 0, stream>>>(a);
    if constexpr (PATCH) {
        const int64_t units = ntiles * 4;
        k_adamw_patch<E><<<dim3((unsigned)(units < kPatchBlocks ? units : kPatchBlocks)), dim3(CD_THREADS), 0, stream>>>(a);
    }
}

template <bool BF16G, bool EIGHT>
void launch_adamw_sizes(const AdamArgs &a, int64_t ntiles, hipStream_t stream) {
    if (a.idx) {
        if (ntiles >= kWholeTiles) launch_adamw<4096, BF16G, EIGHT, true>(a, ntiles, stream);
        else if (ntiles >= kPatchQuarterTiles) launch_adamw<1024, BF16G, EIGHT, true>(a, ntiles, stream);
        else launch_adamw<256, BF16G, EIGHT, true>(a, ntiles, stream);
    } else {
        if (ntiles >= kWholeTiles) launch_adamw<4096, BF16G, EIGHT, false>(a, ntiles, stream);
        else launch_adamw<256, BF16G, EIGHT, false>(a, ntiles, stream);
    }
}

}  // namespace

extern "C" int pulse_launch_adamw(const void *segs, int32_t nseg, const uint32_t *tile_seg, int64_t ntiles,
                                  const float *hyper, uint32_t seed, int32_t grad_bf16, int32_t state_bits,
                                  const float *d_scale, int32_t *idx, uint16_t *val, int64_t cap,
                                  int64_t *seg_offsets, uint32_t *d_status, void *ws, hipStream_t stream) {
    AdamArgs a{};
    a.segs = static_cast<const AdamSeg *>(segs);
    a.tile_seg = tile_seg;
    a.d_scale = d_scale;
    a.nseg = nseg;
    a.seed = seed;
    a.lr = hyper[0];
    a.b1 = hyper[1];
    a.omb1 = hyper[2];
    a.b2 = hyper[3];
    a.omb2 = hyper[4];
    a.eps = hyper[5];
    a.inv_bc1 = hyper[6];
    a.inv_sqrt_bc2 = hyper[7];
    a.idx = idx;
    a.val = val;
    a.cap = cap;
    a.seg_offsets = seg_offsets;
    a.d_status = d_status;
    a.flags = static_cast<uint32_t *>(ws);
    a.counts = ws ? reinterpret_cast<uint32_t *>(static_cast<char *>(ws) + ntiles * (CD_TILE / 8)) : nullptr;
    const bool bf16 = grad_bf16 != 0, eight = state_bits == 8;
    if (bf16 && eight) launch_adamw_sizes<true, true>(a, ntiles, stream);
    else if (bf16) launch_adamw_sizes<true, false>(a, ntiles, stream);
    else if (eight) launch_adamw_sizes<false, true>(a, ntiles, stream);
    else launch_adamw_sizes<false, false>(a, ntiles, stream);
    return hipGetLastError() == hipSuccess ? 0 : -5;
}

extern "C" int pulse_launch_grad_norm(const void *segs, int32_t nseg, const uint32_t *tile_seg, int64_t ntiles,
                                      int32_t grad_bf16, double mul, double max_norm, float *out, void *ws,
                                      hipStream_t stream) {
    NormArgs a{};
    a.segs = static_cast<const GradSeg *>(segs);
    a.tile_seg = tile_seg;
    a.nseg = nseg;
    a.mul = mul;
    a.max_norm = max_norm;
    a.out = out;
    a.done = static_cast<uint32_t *>(ws);
    a.partial = reinterpret_cast<double *>(static_cast<char *>(ws) + 256);
    // 32 KB of gradients at a time, or in lists that would not give every workgroup one 16 KB
    const bool whole = ntiles >= kWholeTiles;
    const int64_t pieces = ntiles * (whole ? 1 : 2) * (grad_bf16 ? 1 : 2);
    a.npieces = (uint32_t)pieces;
    const dim3 grid((unsigned)(pieces < GN_MAX_BLOCKS ? pieces : GN_MAX_BLOCKS)), block(GN_THREADS);
    if (whole) {
        if (grad_bf16) k_grad_norm<4, true><<<grid, block, 0, stream>>>(a);
        else k_grad_norm<4, false><<<grid, block, 0, stream>>>(a);
    } else {
        if (grad_bf16) k_grad_norm<2, true><<<grid, block, 0, stream>>>(a);
        else k_grad_norm<2, false><<<grid, block, 0, stream>>>(a);
    }
    return hipGetLastError() == hipSuccess ? 0 : -5;
}
