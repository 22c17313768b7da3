// wq_device.h -- device-side helpers shared by the kernels (included by the
// .hip sources only; the host-side ABI layer needs none of it).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace wq {

// Workgroup barrier that orders LDS only: waits for this wave's LDS operations,
// then s_barrier. Unlike __syncthreads() it does not wait for outstanding global
// loads, so prefetched registers stay in flight across the barrier. (The two
// builtins touch no memory in the compiler's eyes: the empty statements keep LDS
// accesses on their side.)
__device__ __forceinline__ void lds_barrier()
{
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xC07F);        // lgkmcnt(0); vmcnt and expcnt untouched
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// Raw buffer descriptor over [p, p + bytes) (bytes < 2^32). Dword 3 selects
// 32-bit untyped data (raw buffer loads ignore the format otherwise).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void *p, uint64_t bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), 0, (int)(uint32_t)bytes, 0x00020000);
}

typedef _Float16 half2_t __attribute__((ext_vector_type(2)));

// Two values as sums of two binary16 parts each, x = hi + lo to 22 bits: hi rounded
// to nearest, the remainder exact in fp32 (v_fma_mix_f32 takes hi as it is packed: 4
// instructions for two values instead of 8). Both are made opaque first: contracted
// with the product that made it, the hi that is subtracted could be rounded
// differently from the hi that is kept. Neither may be a matrix instruction's
// result as such (the compiler's waits for those do not reach into the asm).
__device__ __forceinline__ void split2(float x, float y, half2_t &hi, half2_t &lo)
{
    typedef float f2 __attribute__((ext_vector_type(2)));
    asm("" : "+v"(x), "+v"(y));
    hi = __builtin_convertvector((f2{x, y}), half2_t);
    float a, b;
    asm("v_fma_mix_f32 %0, %1, -1.0, %2 op_sel_hi:[1,0,0]" : "=v"(a) : "v"(hi), "v"(x));
    asm("v_fma_mix_f32 %0, %1, -1.0, %2 op_sel:[1,0,0] op_sel_hi:[1,0,0]" : "=v"(b) : "v"(hi), "v"(y));
    lo = __builtin_convertvector((f2{a, b}), half2_t);
}

}  // namespace wq
