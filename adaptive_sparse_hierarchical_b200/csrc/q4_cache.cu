// q4_cache.cu -- writing and reading the 4-bit cache: append (quantisation fused with the Stage 0
// summaries) and load.  Format and layout: include/dash_cache.h.
//
// Quantisation of a group of 32 elements x (4 lanes of 8): s = e4m3(max|x| 2^-e / 7), u = round(x
// 2^-e / s) + 8, both with the quotients' exact ties.  With s rounded to nearest, max|x| / s < 7.5, so
// nothing is clipped by more than half a step while s is a normal e4m3 number below 448; the clamp
// acts below 2^-6 and at 448.  Neither quotient needs a division:
//   - max|x| / 7 has an 8-bit dividend, so it is a midpoint of e4m3 (5 bits) exactly or at least 2^-8
//     of it away; the product with 1/7 is off by 2^-23, and rounding it to f16 (11 bits) first
//     restores the midpoints and makes no new ones;
//   - x has 8 significant bits and s has 4, so x / s is k + 1/2 exactly or at least (k + 1/2) / 256 away
//     from it; x * (2^-e / s) is off by 2^-22 of itself, and rounding it to f16 first does the same.
// Adding 1032 in f16 (two values at a time; the spacing there is 1) then leaves the code in the low bits,
// and the sums are added up, shifted, with what their upper bits contribute taken off once.
//
// Bound: HBM for a prompt (2 bytes read and 17/32 written per element) with the instruction rate close
// behind; launch latency for single tokens.
#include <cuda_fp16.h>

#include "q4.cuh"

namespace dash {
namespace {

constexpr int kBulkWarps = 4;

// Lanes of one row: 8 elements (16 bytes of bf16, one word of codes) each.
template <int D>
struct Row {
    static constexpr int LPK = D / 8, KPI = 32 / LPK;
};

// Scale byte of a group from its largest |x| (two bf16 bit patterns, either may be it), the factor 2^-e / s
// of its elements (inv_e = 2^-e; 0 where s is 0), and whether its quotients may have to be clamped (a
// subnormal or the largest scale).
__device__ __forceinline__ float group_scale(uint32_t top2, float inv_e, uint32_t* scale, bool* edge)
{
    const uint32_t top = max(top2 << 16, top2 & 0xffff0000u);   // as fp32 bits
    const float f = top < 0x7f800000u ? __uint_as_float(top) * inv_e * (1.f / 7.f) : __int_as_float(0x7fffffff);
    uint32_t sb, h;
    float r;
    asm("{\n\t.reg .b16 b;\n\tcvt.rn.f16x2.f32 %1, %2, %2;\n\tcvt.rn.satfinite.e4m3x2.f16x2 b, %1;\n\t"
        "cvt.u32.u16 %0, b;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}\n"
        : "=r"(sb), "=r"(h)
        : "f"(f));
    const float s = __half2float(__ushort_as_half((unsigned short)h));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
    *scale = sb & 0xffu;
    *edge = (sb & 0xffu) - 1u < 7u || (sb & 0xffu) == 0x7eu;
    return s == 0.f ? 0.f : r * inv_e;
}

// The word of codes of 8 elements (r: group_scale's factor; clamp: whether any quotient may need it).
__device__ __forceinline__ uint32_t codes8(const float* x, float r, bool clamp)
{
    __half2 y[4];   // elements i and i + 4
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = __floats2half2_rn(x[i] * r, x[i + 4] * r);
    if (clamp) {
        const __half2 lo = __float2half2_rn(-7.f), hi = __float2half2_rn(7.f);
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = __hmin2(__hmax2(y[i], lo), hi);
    }
    uint32_t w = 0u - 0x64006400u * 0x1111u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 u = __hadd2(y[i], __float2half2_rn(1032.f));
        w += *reinterpret_cast<const uint32_t*>(&u) << (4 * i);
    }
    return w;
}

// Codes of the 8 elements x of this lane (raw: their bf16 bits) and its group's scale byte (equal in the
// group's 4 lanes).  Every lane of the warp takes part.
__device__ __forceinline__ uint32_t quant8(uint4 raw, const float* x, float inv_e, uint32_t* scale)
{
    // |x| as bf16 bits: ordered as integers, infinities and NaNs on top
    uint32_t t = __vmaxu2(__vmaxu2(raw.x & 0x7fff7fffu, raw.y & 0x7fff7fffu),
                          __vmaxu2(raw.z & 0x7fff7fffu, raw.w & 0x7fff7fffu));
    t = __vmaxu2(t, __shfl_xor_sync(0xffffffffu, t, 1));
    t = __vmaxu2(t, __shfl_xor_sync(0xffffffffu, t, 2));
    bool edge;
    const float r = group_scale(t, inv_e, scale, &edge);
    return codes8(x, r, __any_sync(0xffffffffu, edge));
}

// Place of a key row's word `sub` (elements 8 sub ..): word j = sub % 4 of group sub / 4.
template <int D>
__device__ __forceinline__ int key_word(int sub) { return (sub & 3) * (D / kGrp) + (sub >> 2); }

// Online softmax over keys, base 2, of one lane group (8 elements per lane).
struct Sum {
    float m, l, a[8];
    __device__ void init()
    {
        m = -INFINITY;
        l = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) a[e] = 0.f;
    }
    __device__ void push(float z, const float* k)
    {
        const float mn = fmaxf(m, z), sc = exp2f(m - mn), p = exp2f(z - mn);
        l = fmaf(l, sc, p);
#pragma unroll
        for (int e = 0; e < 8; ++e) a[e] = fmaf(a[e], sc, p * k[e]);
        m = mn;
    }
};

struct Append {
    const __nv_bfloat16 *K, *V;
    int n_new;
    const int* counts;
    const float* qbar;
    float *kbar, *state;
    int* seqlens;
};

// Length before the call and number of tokens that sequence b takes (0 where there is nothing to do).
__device__ __forceinline__ void span(const Shape& s, const Append& a, int b, int* L, int* n)
{
    *L = a.seqlens[b];
    int c = a.counts ? min(a.counts[b], a.n_new) : a.n_new;
    c = min(c, s.n - *L);
    *n = *L < 0 || c < 0 ? 0 : c;
}

template <int D>
__device__ __forceinline__ void write_row(uint8_t* codes, uint8_t* scales, long long row, int sub, int word, uint32_t w,
                                          uint32_t sc)
{
    *reinterpret_cast<uint32_t*>(codes + row * (D / 2) + word * 4) = w;
    if ((sub & 3) == 0) scales[row * (D / kGrp) + (sub >> 2)] = (uint8_t)sc;
}

template <int D>
__device__ __forceinline__ void write_state(float* st, int sub, const Sum& r)
{
#pragma unroll
    for (int e = 0; e < 8; ++e) st[sub * 8 + e] = r.a[e];
    if (sub == 0) { st[D] = r.m; st[D + 1] = r.l; }
}
template <int D>
__device__ __forceinline__ void write_summary(float* out, int sub, const Sum& r)
{
    const float inv = 1.f / r.l;
#pragma unroll
    for (int e = 0; e < 8; ++e) out[sub * 8 + e] = r.a[e] * inv;
}

// Many tokens: a warp per (touched chunk, KV head, sequence) quantises the chunk's new keys and sums them
// up in one pass, another one the values.  Four lanes share a row: lane q holds the q-th quarter of every
// scale group.  The groups' maxima are reduced so that each lane is left with one group, whose scale it
// computes for all four (the scale is a third of the work when every lane does it); loads stay 64 bytes
// contiguous and a key's words come out in storage order.  The eight rows' sums of a warp are added by a
// reduce-scatter.  2 x 65536 tokens x 2 heads x 128 (134 MB in, 36 MB out): 41 us,
// 4.1 TB/s; with 8 elements and a scale per lane 50 us.
// The warp of the first chunk also takes the chunk left open at the end, so that the state is read and
// written by one warp, in that order.
template <int NG>
struct RowQuant {
    uint32_t word[NG];
    uint32_t scale;   // byte of the group that this lane owns: q for 4 groups, q / 2 for 2

    __device__ __forceinline__ void operator()(const uint4* raw, const float (*x)[8], float inv_e)
    {
        const int q = threadIdx.x & 3;
        // |x| as bf16 bits, two at a time: ordered as integers, infinities and NaNs on top
        uint32_t t[NG];
#pragma unroll
        for (int i = 0; i < NG; ++i)
            t[i] = __vmaxu2(__vmaxu2(raw[i].x & 0x7fff7fffu, raw[i].y & 0x7fff7fffu),
                            __vmaxu2(raw[i].z & 0x7fff7fffu, raw[i].w & 0x7fff7fffu));
        uint32_t own;
        if constexpr (NG == 4) {
            const bool b1 = q & 2, b0 = q & 1;
            uint32_t k0 = b1 ? t[2] : t[0], k1 = b1 ? t[3] : t[1];
            k0 = __vmaxu2(k0, __shfl_xor_sync(0xffffffffu, b1 ? t[0] : t[2], 2));
            k1 = __vmaxu2(k1, __shfl_xor_sync(0xffffffffu, b1 ? t[1] : t[3], 2));
            own = __vmaxu2(b0 ? k1 : k0, __shfl_xor_sync(0xffffffffu, b0 ? k0 : k1, 1));
        } else {
            const bool b1 = q & 2;
            own = __vmaxu2(b1 ? t[1] : t[0], __shfl_xor_sync(0xffffffffu, b1 ? t[0] : t[1], 2));
            own = __vmaxu2(own, __shfl_xor_sync(0xffffffffu, own, 1));
        }
        bool edge;
        const float r = group_scale(own, inv_e, &scale, &edge);
        edge = __any_sync(0xffffffffu, edge);
#pragma unroll
        for (int i = 0; i < NG; ++i)
            word[i] = codes8(x[i], __shfl_sync(0xffffffffu, r, (threadIdx.x & 28) | (NG == 4 ? i : 2 * i)), edge);
    }
};

template <int D>
__global__ void __launch_bounds__(32 * kBulkWarps, 4)
append_bulk_kernel(Shape s, Q4 c, Append a, int chunks, long long warps)
{
    constexpr int NG = D / kGrp, N = NG * 8;   // elements of a row per lane: group i, elements 8 q .. 8 q + 7
    pdl_wait();
    pdl_launch_dependents();
    __shared__ __align__(16) float qsm[kBulkWarps][D];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, q = lane & 3, slot = lane >> 2;
    const long long wid = (long long)blockIdx.x * kBulkWarps + warp;
    if (wid >= warps) return;
    const int chunk_i = (int)(wid % chunks), rest = (int)(wid / chunks);
    const bool val = rest & 1;
    const int r = (rest >> 1) % s.hkv, b = (rest >> 1) / s.hkv;
    int L, n;
    span(s, a, b, &L, &n);
    if (n == 0) return;
    const int end = L + n, first = L / s.B, ci = first + chunk_i, open = end / s.B;
    if ((long long)ci * s.B >= end || (ci == open && ci != first)) return;
    const float inv_e = exp2i(val ? -c.vexp : -c.kexp);
    const long long ld = val ? s.vs[1] : s.ks[1];
    const __nv_bfloat16* src = (val ? a.V + (long long)b * s.vs[0] + (long long)r * s.vs[2]
                                    : a.K + (long long)b * s.ks[0] + (long long)r * s.ks[2]) + q * 8;
    float* st = a.state + ((long long)b * s.hkv + r) * (D + 2);
    const float* qrow = qsm[warp];
    if (!val) {
        for (int d = lane; d < D; d += 32) qsm[warp][d] = a.qbar[r * D + d] * (kLog2e * rsqrtf((float)D));
        __syncwarp();
    }

    auto chunk = [&](int cc, bool with_state) {
        const int t0 = max(cc * s.B, L), len = min((cc + 1) * s.B, end) - t0;
        const __nv_bfloat16* p = src + (long long)(t0 - L + slot) * ld;
        uint4 nx[NG];
        auto load = [&](int row) {   // the rows after the last one read as zeros
#pragma unroll
            for (int i = 0; i < NG; ++i) {
                nx[i] = make_uint4(0u, 0u, 0u, 0u);
                if (row < len) nx[i] = __ldcs(reinterpret_cast<const uint4*>(p + i * kGrp));
            }
            p += 8 * ld;
        };
        load(slot);   // on its way before the page is known
        const int pg = q4_page(c, b, t0);
        const long long page = pg >= 0 ? pg : 0, row0 = (long long)r * c.psz + t0 % c.psz + slot;
        uint8_t* codes = (val ? c.vc + page * c.vcp : c.kc + page * c.kcp) + row0 * (D / 2);
        uint8_t* scales = (val ? c.vs + page * c.vsp : c.ks + page * c.ksp) + row0 * NG;
        // sums of this lane's elements over its slot's rows, relative to ref (which follows the maximum m of
        // the logits at a distance of 8 at most)
        float m = -INFINITY, ref = -INFINITY, l = 0.f, acc[N];
#pragma unroll
        for (int e = 0; e < N; ++e) acc[e] = 0.f;
        for (int row = slot; row - slot < len; row += 8) {
            uint4 raw[NG];
            float x[NG][8];
#pragma unroll
            for (int i = 0; i < NG; ++i) {
                raw[i] = nx[i];
                Vec<__nv_bfloat16>::cvt(raw[i], x[i]);
            }
            load(row + 8);
            if (!val) {
                float z = 0.f;
#pragma unroll
                for (int i = 0; i < NG; ++i)
#pragma unroll
                    for (int e = 0; e < 8; e += 4) {
                        const float4 w = *reinterpret_cast<const float4*>(qrow + i * kGrp + q * 8 + e);
                        z = fmaf(w.x, x[i][e], fmaf(w.y, x[i][e + 1], fmaf(w.z, x[i][e + 2], fmaf(w.w, x[i][e + 3], z))));
                    }
                z += __shfl_xor_sync(0xffffffffu, z, 1);
                z += __shfl_xor_sync(0xffffffffu, z, 2);
                if (row >= len) z = -INFINITY;
                m = fmaxf(m, z);
                if (__any_sync(0xffffffffu, z > ref + 8.f)) {
                    const float to = z > ref + 8.f ? z : ref, f = to == -INFINITY ? 1.f : exp2f(ref - to);
                    ref = to;
                    l *= f;
#pragma unroll
                    for (int e = 0; e < N; ++e) acc[e] *= f;
                }
                const float w = exp2f(z - (ref == -INFINITY ? 0.f : ref));   // 0 for rows that are not there
                l += w;
#pragma unroll
                for (int e = 0; e < N; ++e) acc[e] = fmaf(w, x[e >> 3][e & 7], acc[e]);
            }
            RowQuant<NG> out;
            out(raw, x, inv_e);
            if (row < len && pg >= 0) {
                if (val) {
#pragma unroll
                    for (int i = 0; i < NG; ++i) *reinterpret_cast<uint32_t*>(codes + (4 * i + q) * 4) = out.word[i];
                } else if constexpr (NG == 4) {
                    *reinterpret_cast<uint4*>(codes + q * 16) = make_uint4(out.word[0], out.word[1], out.word[2], out.word[3]);
                } else {
                    *reinterpret_cast<uint2*>(codes + q * 8) = make_uint2(out.word[0], out.word[1]);
                }
                if (NG == 4 || !(q & 1)) scales[NG == 4 ? q : q >> 1] = (uint8_t)out.scale;
            }
            codes += 8 * (D / 2);
            scales += 8 * NG;
        }
        if (val) return;
        // one reference for the warp (and the state it continues), then the sums
        float M = m;
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        const float m0 = with_state ? st[D] : -INFINITY;
        M = fmaxf(M, m0);
        const float base = M == -INFINITY ? 0.f : M;
        // a slot without a reference holds zeros, or NaNs that have to stay
        const float f = ref == -INFINITY ? 1.f : exp2f(ref - base), f0 = m0 == -INFINITY ? 0.f : exp2f(m0 - base);
        l *= f;
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
#pragma unroll
        for (int e = 0; e < N; ++e) acc[e] *= f;
#pragma unroll
        for (int h = N / 2; h >= NG; h >>= 1) {   // halves go to lanes 16, 8 and 4 apart
            const int o = 16 * h / (N / 2);
            const bool up = lane & o;
#pragma unroll
            for (int e = 0; e < h; ++e)
                acc[e] = (up ? acc[e + h] : acc[e]) + __shfl_xor_sync(0xffffffffu, up ? acc[e] : acc[e + h], o);
        }
        // lane bits 4, 3, 2 number the piece of NG elements that is left
        const int piece = ((lane >> 4) & 1) * 4 + ((lane >> 3) & 1) * 2 + ((lane >> 2) & 1), e0 = piece * NG;
        const int d0 = (e0 >> 3) * kGrp + q * 8 + (e0 & 7);
        if (with_state) {
            l = fmaf(st[D + 1], f0, l);
#pragma unroll
            for (int e = 0; e < NG; ++e) acc[e] = fmaf(st[d0 + e], f0, acc[e]);
            __syncwarp();   // the state is read before it is written
        }
        if ((cc + 1) * s.B <= end) {
            float* out = a.kbar + (((long long)b * s.hkv + r) * s.T + cc) * D + d0;
            const float inv = 1.f / l;
#pragma unroll
            for (int e = 0; e < NG; ++e) out[e] = acc[e] * inv;
        } else {
#pragma unroll
            for (int e = 0; e < NG; ++e) st[d0 + e] = acc[e];
            if (lane == 0) { st[D] = M; st[D + 1] = l; }
        }
    };
    chunk(ci, ci == first && L % s.B != 0);
    if (chunk_i == 0) {
        if (end % s.B != 0) {
            if (open != first) chunk(open, false);
        } else if (!val) {
            __syncwarp();
            for (int d = lane; d < D + 2; d += 32) st[d] = d == D ? -INFINITY : 0.f;
        }
    }
}

__global__ void append_len_kernel(Shape s, Append a)
{
    pdl_wait();   // the append reads the lengths
    pdl_launch_dependents();
    for (int b = threadIdx.x; b < s.batch; b += blockDim.x) {
        int L, n;
        span(s, a, b, &L, &n);
        a.seqlens[b] = L + n;
    }
}

// A few tokens: one block per sequence, a warp per KV head (in turn where there are more heads than
// warps), the two halves (or quarters) of a warp quantise the key and the value row.  One launch:
// the block advances the length itself.
template <int D>
__global__ void append_few_kernel(Shape s, Q4 c, Append a)
{
    using R = Row<D>;
    pdl_wait();
    pdl_launch_dependents();   // the decode routing that follows waits for this grid itself
    const int b = blockIdx.x, lane = threadIdx.x & 31, grp = lane / R::LPK, sub = lane % R::LPK;
    int L, n;
    span(s, a, b, &L, &n);
    for (int r = threadIdx.x >> 5; r < s.hkv && n > 0; r += blockDim.x >> 5) {
        float qv[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) qv[e] = a.qbar[r * D + sub * 8 + e] * (kLog2e * rsqrtf((float)D));
        float* st = a.state + ((long long)b * s.hkv + r) * (D + 2);
        Sum run;
        run.init();
        if (L % s.B != 0) {
#pragma unroll
            for (int e = 0; e < 8; ++e) run.a[e] = st[sub * 8 + e];
            run.m = st[D];
            run.l = st[D + 1];
        }
        const bool val = grp & 1;
        const __nv_bfloat16* src = val ? a.V + (long long)b * s.vs[0] + (long long)r * s.vs[2]
                                       : a.K + (long long)b * s.ks[0] + (long long)r * s.ks[2];
        const long long ld = val ? s.vs[1] : s.ks[1];
        const float inv_e = exp2i(val ? -c.vexp : -c.kexp);
        for (int j = 0; j < n; ++j) {
            const int t = L + j, pg = q4_page(c, b, t);
            const uint4 raw = *reinterpret_cast<const uint4*>(src + j * ld + sub * 8);
            float k[8], z = 0.f;
            Vec<__nv_bfloat16>::cvt(raw, k);
#pragma unroll
            for (int e = 0; e < 8; ++e) z = fmaf(qv[e], k[e], z);
#pragma unroll
            for (int o = R::LPK / 2; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
            uint32_t sc;
            const uint32_t w = quant8(raw, k, inv_e, &sc);
            if (pg >= 0 && grp < 2) {
                const long long row = (long long)r * c.psz + t % c.psz;
                if (val) write_row<D>(c.vc + pg * c.vcp, c.vs + pg * c.vsp, row, sub, sub, w, sc);
                else write_row<D>(c.kc + pg * c.kcp, c.ks + pg * c.ksp, row, sub, key_word<D>(sub), w, sc);
            }
            if (grp == 0) {
                run.push(z, k);
                if ((t + 1) % s.B == 0) {
                    write_summary<D>(a.kbar + (((long long)b * s.hkv + r) * s.T + t / s.B) * D, sub, run);
                    run.init();
                }
            }
        }
        __syncwarp();   // every lane has read the state
        if (grp == 0) write_state<D>(st, sub, run);
    }
    __syncthreads();
    if (threadIdx.x == 0 && n > 0) a.seqlens[b] = L + n;
}

// Reading back: a lane turns one word of codes into 16 bytes of bf16.  (u - 8) s 2^e is exact:
// 128 + u is a bf16 with the code in its low bits, 136 comes off exactly, and the product has at
// most 7 significant bits.  HBM-bound by its writes: 2 x 65536 tokens x 2 heads x 128 (36 MB in, 134 MB out) take
// 31 us, 5.4 TB/s.  Four rows of a lane are on their way at a time.
struct Load {
    __nv_bfloat16 *K, *V;
    const int *start, *seqlens;
    int offset, n;
};

constexpr int kLoadWarps = 8, kLoadRows = 4;

__device__ __forceinline__ uint32_t bf2(uint32_t pair, __nv_bfloat162 s)
{
    uint32_t w;   // (pair & 0x000f000f) | 0x43004300 in one instruction
    asm("lop3.b32 %0, %1, 0x000f000f, %2, 0xea;" : "=r"(w) : "r"(pair), "r"(0x43004300u));
    __nv_bfloat162 v = *reinterpret_cast<__nv_bfloat162*>(&w);
    v = __hmul2(__hsub2(v, __float2bfloat162_rn(136.f)), s);
    return *reinterpret_cast<uint32_t*>(&v);
}

template <int D>
__global__ void __launch_bounds__(32 * kLoadWarps) load_kernel(Shape s, Q4 c, Load a)
{
    using R = Row<D>;
    pdl_wait();
    pdl_launch_dependents();
    const int b = blockIdx.z, r = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int grp = lane / R::LPK, sub = lane % R::LPK;
    const long long first = (a.start ? (long long)a.start[b] : 0) + a.offset;
    const int len = min(a.seqlens[b], s.n);
    const int j0 = (blockIdx.x * kLoadWarps + warp) * R::KPI * kLoadRows + grp;
    // the lane's tokens are KPI apart: together at most as far as a page is long, so one division will do
    static_assert(R::KPI * kLoadRows <= 16, "pages hold at least 16 tokens");
    const long long t0 = first + j0;
    const int q0 = t0 >= 0 && t0 < len ? (int)t0 : 0, slot0 = q0 / c.psz, in0 = q0 - slot0 * c.psz;
    const int* table = c.pt + (long long)b * c.pmax;
    uint32_t kw[kLoadRows], vw[kLoadRows], kq[kLoadRows], vq[kLoadRows];
#pragma unroll
    for (int u = 0; u < kLoadRows; ++u) {
        kw[u] = vw[u] = kq[u] = vq[u] = 0;   // scale 0: the value 0
        const long long t = t0 + u * R::KPI;
        if (j0 + u * R::KPI >= a.n || t < 0 || t >= len) continue;
        int slot = slot0, in = in0 + u * R::KPI;
        if (t0 < 0) {   // the first token lies before the sequence
            slot = (int)t / c.psz;
            in = (int)t - slot * c.psz;
        } else if (in >= c.psz) {
            ++slot;
            in -= c.psz;
        }
        const int pg = slot < c.pmax ? table_entry(table + slot) : -1;
        if (pg < 0 || pg >= c.npages) continue;
        const long long row = (long long)r * c.psz + in;
        kw[u] = *reinterpret_cast<const uint32_t*>(c.kc + pg * c.kcp + row * (D / 2) + key_word<D>(sub) * 4);
        vw[u] = *reinterpret_cast<const uint32_t*>(c.vc + pg * c.vcp + row * (D / 2) + sub * 4);
        kq[u] = c.ks[pg * c.ksp + row * (D / kGrp) + (sub >> 2)];
        vq[u] = c.vs[pg * c.vsp + row * (D / kGrp) + (sub >> 2)];
    }
    const float ke = exp2i(c.kexp), ve = exp2i(c.vexp);
    auto put = [&](__nv_bfloat16* out, uint32_t w, uint32_t sb, float e) {
        const __nv_bfloat162 sc = __float2bfloat162_rn(e4m3_to_f32(sb) * e);
        uint32_t p[4];   // element pairs (i, i + 4)
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = bf2(w >> (4 * i), sc);
        uint4 o;
        o.x = __byte_perm(p[0], p[1], 0x5410);
        o.y = __byte_perm(p[2], p[3], 0x5410);
        o.z = __byte_perm(p[0], p[1], 0x7632);
        o.w = __byte_perm(p[2], p[3], 0x7632);
        *reinterpret_cast<uint4*>(out) = o;
    };
    __nv_bfloat16* ko = a.K + (long long)b * s.ks[0] + (long long)j0 * s.ks[1] + (long long)r * s.ks[2] + sub * 8;
    __nv_bfloat16* vo = a.V + (long long)b * s.vs[0] + (long long)j0 * s.vs[1] + (long long)r * s.vs[2] + sub * 8;
#pragma unroll
    for (int u = 0; u < kLoadRows; ++u) {
        if (j0 + u * R::KPI >= a.n) break;
        put(ko, kw[u], kq[u], ke);
        put(vo, vw[u], vq[u], ve);
        ko += R::KPI * s.ks[1];
        vo += R::KPI * s.vs[1];
    }
}

template <int D>
cudaError_t append_d(const Shape& s, const Q4& c, const Append& a, cudaStream_t st)
{
    // Up to this many tokens a warp walks them one after another (about 1 us each) and saves the
    // second launch (2 to 3 us of the call).
    if (a.n_new <= 4)
        return launch_after(append_few_kernel<D>, dim3(s.batch), dim3(32 * (s.hkv < 16 ? s.hkv : 16)), 0, st, s, c, a);
    const int chunks = (a.n_new + s.B - 2) / s.B + 1;
    const long long warps = 2ll * chunks * s.hkv * s.batch;
    const cudaError_t e = launch_after(append_bulk_kernel<D>, dim3((unsigned)((warps + kBulkWarps - 1) / kBulkWarps)),
                                       dim3(32 * kBulkWarps), 0, st, s, c, a, chunks, warps);
    if (e != cudaSuccess) return e;
    return launch_after(append_len_kernel, dim3(1), dim3(s.batch < 256 ? (s.batch + 31) / 32 * 32 : 256), 0, st, s, a);
}

}  // namespace

cudaError_t launch_append_q4(const Shape& s, const Q4& c, const void* K, const void* V, int n_new, const int* counts,
                             const float* qbar, float* kbar, float* state, int* seqlens, cudaStream_t st)
{
    const Append a{(const __nv_bfloat16*)K, (const __nv_bfloat16*)V, n_new, counts, qbar, kbar, state, seqlens};
    return s.d == 128 ? append_d<128>(s, c, a, st) : append_d<64>(s, c, a, st);
}

cudaError_t launch_load_q4(const Shape& s, const Q4& c, const int* start, int offset, int n, const int* seqlens,
                           void* K, void* V, cudaStream_t st)
{
    const Load a{(__nv_bfloat16*)K, (__nv_bfloat16*)V, start, seqlens, offset, n};
    const int per = kLoadWarps * kLoadRows * (256 / s.d);
    const dim3 grid((unsigned)(((long long)n + per - 1) / per), s.hkv, s.batch);
    return launch_after(s.d == 128 ? load_kernel<128> : load_kernel<64>, grid, dim3(32 * kLoadWarps), 0, st, s, c, a);
}

}  // namespace dash
