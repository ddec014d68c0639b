// compact.hpp -- the tiling of the calls over lists of tensors, and the compaction
// stage of the kernels that write a sparse patch in their own pass: a wave's
// changed elements, known as one flag bit per element and the new values in
// registers, are ranked with ballots, staged in LDS and written as one contiguous,
// ascending stretch of (int32 index, BF16 value) entries.
// A: any struct with the patch's idx, val and cap.
#pragma once

#include "device.hpp"

namespace pulse {

constexpr int CD_THREADS = 256;
constexpr int CD_GROUPS = 16;
constexpr int CD_WAVE_ELEMS = CD_GROUPS * 256;                    // 4096
constexpr int CD_TILE = (CD_THREADS / kWave) * CD_WAVE_ELEMS;   // 16384

constexpr int CD_SB = 512;  // patch entries staged per wave before a coalesced flush

struct CdShared {
    uint32_t wtot[CD_THREADS / kWave];
    uint64_t prefix;
    int32_t sbi[CD_THREADS / kWave][CD_SB];
    uint16_t sbv[CD_THREADS / kWave][CD_SB];
};

// Writes the wave's staged entries [0, nb) to the patch at out (lanes write
// consecutive entries: full-width stores) and empties the buffer.
template <typename A>
__device__ __forceinline__ void cd_flush(const A &a, const int32_t *sbi, const uint16_t *sbv, uint32_t &nb,
                                         int64_t &out) {
    __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");  // the lanes' staged entries are visible to the wave
    for (uint32_t i = lane_id(); i < nb; i += kWave) {
        const int64_t pos = out + i;
        if (pos < a.cap) {
            a.idx[pos] = sbi[i];
            a.val[pos] = sbv[i];
        }
    }
    __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");  // reads done before the buffer is refilled
    out += nb;
    nb = 0;
}

// Pass 2 of one wave: each changed element is ranked with ballots and staged
// in the wave's LDS buffer at its rank; the buffer goes out with coalesced
// stores (the wave's entries are one contiguous stretch of the patch, the
// first at position run).
template <typename A>
__device__ __forceinline__ void cd_pass2(const A &a, uint64_t flags, const uint32_t nvp[], int64_t wbase,
                                         int lo, int64_t run, int32_t *sbi, uint16_t *sbv) {
    uint32_t nb = 0;
#pragma unroll
    for (int g = 0; g < CD_GROUPS; ++g) {
        const uint32_t f = (uint32_t)(flags >> (4 * g)) & 0xFu;
        const uint64_t m0 = __ballot(f & 1u), m1 = __ballot(f & 2u), m2 = __ballot(f & 4u), m3 = __ballot(f & 8u);
        const uint32_t gtot = __builtin_popcountll(m0) + __builtin_popcountll(m1) + __builtin_popcountll(m2) +
                              __builtin_popcountll(m3);
        if (gtot == 0) continue;
        if (nb + gtot > (uint32_t)CD_SB) cd_flush(a, sbi, sbv, nb, run);
        uint32_t r = nb + lanes_below(m0) + lanes_below(m1) + lanes_below(m2) + lanes_below(m3);
        const int32_t e = (int32_t)(wbase + g * 256 + lo);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (f & (1u << k)) {
                sbi[r] = e + k;
                sbv[r] = (uint16_t)(nvp[2 * g + (k >> 1)] >> (16 * (k & 1)));
                ++r;
            }
        }
        nb += gtot;
    }
    if (nb) cd_flush(a, sbi, sbv, nb, run);
}

// Ranks and stages the wave's changed elements in its LDS buffer without
// storing them (the caller guarantees they fit); nb becomes their number.
__device__ __forceinline__ void cd_stage(uint64_t flags, const uint32_t nvp[], int64_t wbase, int lo, int32_t *sbi,
                                         uint16_t *sbv, uint32_t &nb) {
#pragma unroll
    for (int g = 0; g < CD_GROUPS; ++g) {
        const uint32_t f = (uint32_t)(flags >> (4 * g)) & 0xFu;
        const uint64_t m0 = __ballot(f & 1u), m1 = __ballot(f & 2u), m2 = __ballot(f & 4u), m3 = __ballot(f & 8u);
        const uint32_t gtot = __builtin_popcountll(m0) + __builtin_popcountll(m1) + __builtin_popcountll(m2) +
                              __builtin_popcountll(m3);
        if (gtot == 0) continue;
        uint32_t r = nb + lanes_below(m0) + lanes_below(m1) + lanes_below(m2) + lanes_below(m3);
        const int32_t e = (int32_t)(wbase + g * 256 + lo);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (f & (1u << k)) {
                sbi[r] = e + k;
                sbv[r] = (uint16_t)(nvp[2 * g + (k >> 1)] >> (16 * (k & 1)));
                ++r;
            }
        }
        nb += gtot;
    }
}

}  // namespace pulse
