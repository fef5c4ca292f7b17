// block_dma.h -- direct global->LDS loads through a buffer resource, for the
// products of the block: 16 bytes a lane from a base that advances as a scalar, a
// 32-bit offset a lane that stays, and zeros where a lane's offset is kNone (the
// resource ends below it).  Inline assembly for the reason given in lds_dma.h: the
// compiler would wait for every outstanding load before each LDS read.  The
// statements have no outputs; landed_barrier waits for them.
#pragma once

#include "device_common.h"
#include "lds_dma.h"

namespace moe_lora {

typedef __attribute__((address_space(3))) char lds_char;

constexpr uint32_t kNone = 0xfffffff0u;

// LDS byte address of a __shared__ array, wave-uniform
__device__ __forceinline__ uint32_t lds_base(const void *p)
{
    return __builtin_amdgcn_readfirstlane((uint32_t)reinterpret_cast<uintptr_t>((const lds_char *)p));
}

// Raw buffer over [base, base + 2^31): offsets of a step stay below that.
__device__ __forceinline__ u32x4 buffer_resource(const char *base)
{
    const uint64_t b = reinterpret_cast<uint64_t>(base);
    return u32x4{(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)b),
                 (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(b >> 32)) & 0xffffu, 0x80000000u, 0x00027000u};
}

// 16 bytes of each lane to lds + 16 lane
__device__ __forceinline__ void buffer_load_lds16(u32x4 resource, uint32_t offset, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %2\n\t" MOE_LORA_M0_WAIT "buffer_load_dwordx4 %0, %1, 0 offen lds"
                 :
                 : "v"(offset), "s"(resource), "s"(lds)
                 : "memory", "m0");
}

// At most N of this wave's loads are still to land and its LDS reads are done; then
// the block meets.
template <int N>
__device__ __forceinline__ void landed_barrier()
{
    static_assert(N < 64, "the counter has 6 bits");
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" : : "n"(N) : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// LDS that only this wave uses: its stores are done before its loads that follow (the
// hardware keeps a wave's LDS operations in order; this keeps the compiler's).
__device__ __forceinline__ void lds_order()
{
    __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
}

} // namespace moe_lora
