// Helpers of the attention kernels on the tensor cores (kernels_attn.cu,
// kernels_paged_wide.cu).
#pragma once

#include "common.cuh"

namespace tpk {

// Two float32 operations per instruction, and a maximum of three.
__device__ __forceinline__ uint64_t f2_pack(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void f2_unpack(uint64_t v, float& a, float& b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// mbar_wait in two halves: a try in line, and the bounded wait out of line, which keeps the loops' code short.
__device__ __forceinline__ bool mbar_try_at(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
static __device__ __noinline__ bool mbar_wait_slow(uint32_t bar, uint32_t parity, volatile int* abort, int* status) {
    const uint64_t t0 = global_ns();
    while (true) {
        if (mbar_try_at(bar, parity)) return true;
        if (*abort) return false;
        if (global_ns() - t0 > kWaitLimitNs) {
            *abort = 1;
            set_status(status, TP_ERR_TIMEOUT);
            return false;
        }
    }
}

__device__ __forceinline__ bool at_wait(uint64_t* bar, uint32_t parity, volatile int* abort, int* status) {
    const uint32_t b = smem_u32(bar);
    return mbar_try_at(b, parity) || mbar_wait_slow(b, parity, abort, status);
}

__device__ __forceinline__ uint64_t at_desc_add(uint64_t d, uint32_t bytes) { return d + (bytes >> 4); }

// A value that is the same in every lane, in a form that lets the compiler know.
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }

// 16-byte units of four lanes' rows, transposed: lane i of four gets unit i of the rows of all four, so that a store of the
// warp writes eight runs of 64 bytes and not 32 of 16.
__device__ __forceinline__ void transpose4(uint4 (&u)[4], int lane) {
    auto swap = [&](uint4& a, uint4& b, int off) {       // b of the lower lane for a of the upper
        const bool up = lane & off;
        uint4 give = up ? a : b;
        give.x = __shfl_xor_sync(0xffffffffu, give.x, off);
        give.y = __shfl_xor_sync(0xffffffffu, give.y, off);
        give.z = __shfl_xor_sync(0xffffffffu, give.z, off);
        give.w = __shfl_xor_sync(0xffffffffu, give.w, off);
        if (up) a = give;
        else b = give;
    };
    __syncwarp();
    swap(u[0], u[1], 1);
    swap(u[2], u[3], 1);
    swap(u[0], u[2], 2);
    swap(u[1], u[3], 2);
}

}  // namespace tpk
