// q4.cuh -- the 4-bit cache format of include/dash_cache.h: descriptor, addressing, conversions.
#pragma once
#include "dash_common.cuh"
#include "../../include/dash_cache.h"

namespace dash {

constexpr int kGrp = 32;   // elements that share a scale

// What the kernels see of a dash_q4_kv.
struct Q4 {
    uint8_t *kc, *ks, *vc, *vs;
    long long kcp, ksp, vcp, vsp;
    const int* pt;
    int pmax, psz, npages;
    int kexp, vexp;
};

// Page of token t of sequence b, or -1 where none is mapped.
__device__ __forceinline__ int q4_page(const Q4& c, int b, int t)
{
    const int slot = t / c.psz;
    if (t < 0 || slot >= c.pmax) return -1;
    const int pg = __ldg(c.pt + (long long)b * c.pmax + slot);
    return pg >= 0 && pg < c.npages ? pg : -1;
}

// Two e4m3 bytes (low byte first) as f16x2; exact, the code 0x7f gives a NaN.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two)
{
    uint32_t r;
    asm("{\n\t.reg .b16 h;\n\tcvt.u16.u32 h, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}\n" : "=r"(r) : "r"(two));
    return r;
}
__device__ __forceinline__ float e4m3_to_f32(uint32_t byte)
{
    float f;
    asm("{\n\t.reg .b16 h, lo, hi;\n\t.reg .b32 v;\n\tcvt.u16.u32 h, %1;\n\tcvt.rn.f16x2.e4m3x2 v, h;\n\t"
        "mov.b32 {lo, hi}, v;\n\tcvt.f32.f16 %0, lo;\n\t}\n"
        : "=f"(f)
        : "r"(byte & 0xffu));
    return f;
}
// x >= 0 (or NaN) as e4m3: round to nearest even, at most 448.
__device__ __forceinline__ uint32_t f32_to_e4m3(float x)
{
    uint32_t r;
    asm("{\n\t.reg .b16 h;\n\tcvt.rn.satfinite.e4m3x2.f32 h, %1, %2;\n\tcvt.u32.u16 %0, h;\n\t}\n"
        : "=r"(r)
        : "f"(0.f), "f"(x));
    return r & 0xffu;
}

// 2^e as a float, |e| <= 126
__device__ __forceinline__ float exp2i(int e) { return __int_as_float((127 + e) << 23); }

}  // namespace dash
