// lds_load.hpp -- loads from memory into LDS, past the registers.
#pragma once

#include "device.hpp"

namespace pulse {

// One instruction brings 16 (or 4) bytes of every lane, from base + its offset, to 64
// consecutive places of LDS from `lds` on (M0 holds it, which takes one wait state).
// The compiler does not count these loads: a reader waits for vmcnt itself.
__device__ __forceinline__ uint32_t lds_at(const void *p) {
    return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const uint8_t *)p;
}

// M0 is named as overwritten, so that the compiler expects no value of its own there behind such a
// load; it warns of that, for M0 is not one of the registers in which it keeps a program's values.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void load_lds16(uint32_t lds, const void *base, uint32_t off) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds), "v"(off), "s"(base)
                 : "m0", "memory");
}
__device__ __forceinline__ void load_lds16_once(uint32_t lds, const void *base, uint32_t off) {  // not read again
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2 nt" ::"s"(lds), "v"(off), "s"(base)
                 : "m0", "memory");
}
__device__ __forceinline__ void load_lds4(uint32_t lds, const void *base, uint32_t off) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, %2" ::"s"(lds), "v"(off), "s"(base)
                 : "m0", "memory");
}
#pragma clang diagnostic pop

template <int N>
__device__ __forceinline__ void wait_loads() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// A value that is the same in all lanes, in scalar registers.
template <typename T>
__device__ __forceinline__ T uniform(T v) {
    if constexpr (sizeof(T) == 8) {
        const uint64_t u = __builtin_bit_cast(uint64_t, v);
        const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)u);
        const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(u >> 32));
        return __builtin_bit_cast(T, (uint64_t)hi << 32 | lo);
    } else {
        return __builtin_bit_cast(T, __builtin_amdgcn_readfirstlane(__builtin_bit_cast(uint32_t, v)));
    }
}

// A base address for the loads above.  A vector instruction may have written its scalar
// registers, which a load may read five wait states later; the compiler does not see one here.
template <typename T>
__device__ __forceinline__ T *load_base(T *p) {
    uint64_t a = (uint64_t)uniform(p);
    asm volatile("s_nop 4" : "+s"(a));
    return reinterpret_cast<T *>(a);
}

}  // namespace pulse
