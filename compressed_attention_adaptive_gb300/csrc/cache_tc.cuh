// What the kernels over the 4-bit cache that run on tcgen05 share (cache_tile.cu, cache_weigh_tile.cu):
// bounded waits that end together, and accesses to tensor memory.
#pragma once

#include "cache_walk.cuh"

namespace mita {

// Instruction descriptor of kind::f16 with half A and B and fp32 accumulate.
constexpr uint32_t idesc_half(int M, int N, int a_mn, int b_mn) {
    return (1u << 4) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) | ((uint32_t)(N >> 3) << 17) |
           ((uint32_t)(M >> 4) << 24);
}

struct Abort {
    int flag;   // a role has given up
    int limit;  // what a wait takes at most, in kSpinTest (from shared memory: as the kernel's
                // parameter it took operands out of the uniform registers, 263.8 us against 261.4)
};
// Bounded wait that also ends when another role has given up.
__device__ __forceinline__ bool tile_wait(uint64_t* bar, uint32_t parity, volatile Abort* abort) {
    if (tc::mbar_try_wait(bar, parity)) return true;
    const long long t0 = clock64();
    while (!tc::mbar_try_wait(bar, parity)) {
        if (abort->flag) return false;
        if (clock64() - t0 > abort->limit * tc::kSpinTest) {
            abort->flag = 1;
            return false;
        }
    }
    return true;
}
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile Abort* abort) {
    return __all_sync(0xffffffffu, tile_wait(bar, parity, abort));
}
// For what this block has issued to the asynchronous units, whatever the abort flag says.
__device__ __forceinline__ void drain(uint64_t* bar, uint32_t parity, int* status, long long lim) {
    (void)tc::mbar_wait(bar, parity, status, lim);
}

// (No memory clobber: loads may move across. fence_proxy_async() orders it.)
__device__ __forceinline__ void st_shared16(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d));
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float* v) {
    uint32_t* r = reinterpret_cast<uint32_t*>(v);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float* v) {
    uint32_t* r = reinterpret_cast<uint32_t*>(v);
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}
// Registers {a0, a1, a2, a3} of an m16n8k16 step's A, twice (two steps): 16 lanes, 16 columns.
__device__ __forceinline__ void tmem_st_frag(uint32_t taddr, const uint32_t* r) {
    asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
// One lane of a whole warp. (Behind a branch on this the compiler keeps the products'
// operands in uniform registers; behind one on the lane's number it moves each there.)
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r));
    return r != 0;
}

}  // namespace mita
