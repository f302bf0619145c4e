// Inline-PTX wrappers that the key/value cache's kernels need beside those of ptx.cuh (kept apart: the
// contraction kernels' committed counters are keyed to that file).
#pragma once

#include "ptx.cuh"

namespace mmq {
namespace ptx {

// Adds one and returns what was there; releases what this thread has seen (the CTA's writes, after a barrier) and
// acquires what the threads that counted before have released.
__device__ __forceinline__ uint32_t atom_inc_acq_rel(unsigned* p) {
    uint32_t v;
    asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(v) : "l"(p) : "memory");
    return v;
}

// True in one lane, always the same, of a converged warp.  Single-thread instructions whose operands
// are warp-uniform issue from uniform registers inside such a branch; behind a lane comparison every
// operand is moved there one instruction at a time.
__device__ __forceinline__ bool elect_one() {
    uint32_t on;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(on));
    return on != 0;
}

// As umma_f16 with A in TMEM: lane = row, each 32-bit column two consecutive k.
__device__ __forceinline__ void umma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                            uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// 32 lanes x 16 consecutive 32-bit columns written: thread i of the warp gives lane (base + i).
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

}  // namespace ptx
}  // namespace mmq
