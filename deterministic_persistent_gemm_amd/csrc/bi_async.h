// bi_async.h -- direct-to-LDS loads and the waits that go with them, for the
// kernels that stream their operands through an LDS ring.
//
// A direct-to-LDS load takes no destination register: lane i's bytes land at
// LDS byte address `lds` + i * (bytes per lane), with the wave's base in M0.
// The loads are inline assembly so that the compiler does not order each
// after the previous one (it would treat every load as an aliasing LDS write);
// what a consumer needs is waited for explicitly with async_wait / async_wait_later.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "bi_device.h"

namespace bi {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ uint32_t uniform(uint32_t v) { return (uint32_t)__builtin_amdgcn_readfirstlane((int)v); }

// A wave-uniform pointer in scalar registers (nothing is emitted where it
// already is).
__device__ __forceinline__ const void* uniform_ptr(const void* p)
{
    const uint64_t v = (uint64_t)(uintptr_t)p;
    return (const void*)(uintptr_t)((uint64_t)uniform((uint32_t)(v >> 32)) << 32 | uniform((uint32_t)v));
}

// 16 bytes per lane: a wave-uniform base, a 32-bit byte offset per lane.
__device__ __forceinline__ void async16(uint32_t voff, const void* sbase, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" : : "v"(voff), "s"(uniform_ptr(sbase)), "s"(lds)
                 : "memory", "m0");
}

// 4 bytes per lane.
__device__ __forceinline__ void async4(uint32_t voff, const void* sbase, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dword %0, %1" : : "v"(voff), "s"(uniform_ptr(sbase)), "s"(lds)
                 : "memory", "m0");
}

__device__ __forceinline__ uint32_t lds_byte(const void* p)
{
    return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void*)p;
}

// s_waitcnt with vmcnt <= N (N < 64), other counters untouched
template <int N>
__device__ __forceinline__ void async_wait()
{
    static_assert(N >= 0 && N < 64, "vmcnt holds six bits");
    __builtin_amdgcn_s_waitcnt((N & 0xF) | (0x7 << 4) | (0xF << 8) | ((N >> 4) << 14));
}

// vmcnt <= later * LW for a runtime later in [0, C]
template <int LW, int C>
__device__ __forceinline__ void async_wait_later(int later)
{
    if constexpr (C <= 0) {
        async_wait<0>();
    } else {
        if (later >= C)
            async_wait<C * LW>();
        else
            async_wait_later<LW, C - 1>(later);
    }
}

// A workgroup barrier without the fence of __syncthreads (whose release would
// wait for every outstanding load); callers wait for exactly what the other
// side needs first.
__device__ __forceinline__ void wg_barrier() { asm volatile("s_barrier" : : : "memory"); }

// The same after this wave's LDS reads have landed in registers.
__device__ __forceinline__ void wg_barrier_reads_done() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" : : : "memory"); }

// Transposing LDS read: in each group of 16 lanes, lane i points at 8 bytes
// (four bf16) of row i / 4 of a 4-row block, and receives the four rows'
// elements of column i -- column c being element c % 4 of the 8 bytes that
// lane c / 4 of each row pointed at.
__device__ __forceinline__ s16x4 lds_read_tr(const unsigned char* p)
{
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (__attribute__((address_space(3))) s16x4*)(const __attribute__((address_space(3))) void*)p);
}

}  // namespace bi
