// tiles.hpp -- the tiling of the calls over lists of tensors: a workgroup of four waves
// takes 16384 elements of one tensor, each wave 4096 as 16 groups of 256.
#pragma once

#include "device.hpp"

namespace pulse {

constexpr int CD_THREADS = 256;
constexpr int CD_GROUPS = 16;
constexpr int CD_WAVE_ELEMS = CD_GROUPS * 256;                    // 4096
constexpr int CD_TILE = (CD_THREADS / kWave) * CD_WAVE_ELEMS;   // 16384

}  // namespace pulse
