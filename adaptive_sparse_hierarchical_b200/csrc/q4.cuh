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

// An entry of the page table: an ordinary load (the kernel ahead may have been writing the table when this one started,
// which rules the read-only path out), but one that the compiler may place freely.  That is safe because nobody writes
// the table once the kernel ahead has ended, and `p` has to depend on a length read after that (as it does wherever a
// token's number is checked against one).
__device__ __forceinline__ int table_entry(const int* p)
{
    int v;
    asm("ld.global.s32 %0, [%1];" : "=r"(v) : "l"(__cvta_generic_to_global(p)));
    return v;
}

// Page of token t of sequence b, or -1 where none is mapped.
template <typename F>
__device__ __forceinline__ int q4_page(const Q4& c, int b, int t, F entry)
{
    const int slot = t / c.psz;
    if (t < 0 || slot >= c.pmax) return -1;
    const int pg = entry(c.pt + (long long)b * c.pmax + slot);
    return pg >= 0 && pg < c.npages ? pg : -1;
}

__device__ __forceinline__ int q4_page(const Q4& c, int b, int t)
{
    return q4_page(c, b, t, [](const int* e) { return table_entry(e); });
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
