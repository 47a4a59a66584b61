// Direct loads from memory to LDS, and the pipeline barrier that waits for them.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

// LDS-DMA issued through inline assembly.  The compiler does not see these
// loads, so it inserts no waits for them (it cannot track many in-flight
// LDS-DMA stores and would otherwise wait for all of them before every LDS
// read); the pipeline waits for them explicitly with pipe_barrier.  The
// buffer resource (base, stride 0, 2^31-1 records) makes offsets >= 2^31 read
// zeros.  buffer_load_dwordx4 ... lds writes lane l's 16 bytes at M0 + 16 l;
// buffer_load_dword ... lds writes lane l's 4 bytes at M0 + 4 l.
typedef __attribute__((ext_vector_type(4))) int i32x4;

__device__ __forceinline__ i32x4 make_rsrc(const void* p) {
    uint64_t a = (uint64_t)p;
    i32x4 r;
    r[0] = __builtin_amdgcn_readfirstlane((int)(uint32_t)a);
    r[1] = __builtin_amdgcn_readfirstlane((int)(uint32_t)(a >> 32));
    r[2] = 0x7fffffff;
    r[3] = 0x00020000;
    return r;
}

// LDS byte address of a shared-memory pointer (the low 32 bits of the
// generic address; the LDS aperture is 4 GiB aligned), as a uniform value.
__device__ __forceinline__ uint32_t lds_u32(const void* p) {
    return __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)p);
}

// (M0 is a register that the compiler reserves: it keeps nothing there over other
// instructions, writes it right before an instruction of its own that reads it, and
// takes no clobber of it.  These kernels have no such instruction.)
__device__ __forceinline__ void dma16(const i32x4& rs, uint32_t voff, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                 ::"s"(lds), "v"(voff), "s"(rs) : "memory");
}

__device__ __forceinline__ void dma4(const i32x4& rs, uint32_t voff, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds"
                 ::"s"(lds), "v"(voff), "s"(rs) : "memory");
}

// Pipeline barrier: wait until at most N vector-memory loads (LDS-DMA batches
// of later K steps) are outstanding and all LDS accesses are done, then
// synchronize the workgroup.  __syncthreads() would also fence global memory,
// which waits for every outstanding load and so drains the look-ahead.
// The compiler does not see the waits inside the asm: the trailing
// s_waitcnt lgkmcnt(0) (free, the counter is already zero) tells it that
// every earlier LDS read has completed, so it does not hold back the MFMAs
// after the barrier for reads that landed long ago.
template <int N>
__device__ __forceinline__ void pipe_barrier() {
    static_assert(N >= 0 && N < 64, "vmcnt range");
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
    __builtin_amdgcn_s_waitcnt(0xC07F);   // vmcnt(63) expcnt(7) lgkmcnt(0)
}

__device__ __forceinline__ i32x4 rsrc_at(uint64_t base, int nrec) {
    i32x4 r;
    r[0] = __builtin_amdgcn_readfirstlane((int)(uint32_t)base);
    r[1] = __builtin_amdgcn_readfirstlane((int)(uint32_t)(base >> 32));
    r[2] = __builtin_amdgcn_readfirstlane(nrec);
    r[3] = 0x00020000;
    return r;
}

// A load whose lanes keep their offsets while uniform values (the resource,
// the scalar offset) move.
struct Dma { i32x4 rs; uint32_t soff; };

__device__ __forceinline__ void dma16(const Dma& d, uint32_t voff, uint32_t lds) {
    // (5 wait states from a vector write of the resource's registers)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                 ::"s"(lds), "v"(voff), "s"(d.rs), "s"(d.soff) : "memory");
}

}  // namespace moe
