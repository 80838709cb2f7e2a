// More inline-PTX wrappers for sm_100a, used by the token-by-token kernels: 16-column
// tensor-memory loads, the election of one lane, the split of registers between
// warpgroups.  Written from the public PTX ISA description of these instructions.
#pragma once

#include "ptx.cuh"

namespace attn {

// tmem_ld32 for 16 consecutive columns.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

// One lane of a converged warp.  A branch on it, unlike one on a lane index, tells
// the compiler that a single thread runs what follows: the products' operands
// then stay in uniform registers (8 products of N = 64 with A in tensor memory:
// 265 cycles, against 431 behind lane == 0).
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// Registers per thread of the calling warpgroup, down or up; the launch's total (its
// threads times its registers per thread) bounds the sum over all warpgroups.
template <int N>
__device__ __forceinline__ void regs_down() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_up() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

}  // namespace attn
