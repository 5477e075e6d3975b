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

// Codes of the 8 elements x of this lane (raw: their bf16 bits) and its group's scale byte (equal in the
// group's 4 lanes).  inv_e = 2^-e.  Every lane of the warp takes part.
__device__ __forceinline__ uint32_t quant8(uint4 raw, const float* x, float inv_e, uint32_t* scale)
{
    // |x| as bf16 bits: ordered as integers, infinities and NaNs on top
    uint32_t t = __vmaxu2(__vmaxu2(raw.x & 0x7fff7fffu, raw.y & 0x7fff7fffu),
                          __vmaxu2(raw.z & 0x7fff7fffu, raw.w & 0x7fff7fffu));
    t = __vmaxu2(t, __shfl_xor_sync(0xffffffffu, t, 1));
    t = __vmaxu2(t, __shfl_xor_sync(0xffffffffu, t, 2));
    const uint32_t top = max(t << 16, t & 0xffff0000u);   // as fp32 bits
    const float f = top < 0x7f800000u ? __uint_as_float(top) * inv_e * (1.f / 7.f) : __int_as_float(0x7fffffff);
    uint32_t sb, h;
    float s, r;
    asm("{\n\t.reg .b16 b;\n\tcvt.rn.f16x2.f32 %1, %2, %2;\n\tcvt.rn.satfinite.e4m3x2.f16x2 b, %1;\n\t"
        "cvt.u32.u16 %0, b;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}\n"
        : "=r"(sb), "=r"(h)
        : "f"(f));
    s = __half2float(__ushort_as_half((unsigned short)h));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
    r = s == 0.f ? 0.f : r * inv_e;
    *scale = sb = sb & 0xffu;
    __half2 y[4];   // elements i and i + 4
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = __floats2half2_rn(x[i] * r, x[i + 4] * r);
    if (__any_sync(0xffffffffu, sb - 1u < 7u || sb == 0x7eu)) {   // a subnormal or the largest scale in the warp
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
    __device__ void merge(float m2, float l2, const float* a2)
    {
        const float mn = fmaxf(m, m2);
        if (mn == -INFINITY) return;
        const float s1 = exp2f(m - mn), s2 = exp2f(m2 - mn);
        l = l * s1 + l2 * s2;
#pragma unroll
        for (int e = 0; e < 8; ++e) a[e] = a[e] * s1 + a2[e] * s2;
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

// One block of four warps per (touched chunk, KV head, sequence): the chunk's new keys and values
// are quantised and its keys summarised in one pass; the warps' sums merge in order.  The block of
// the first chunk also takes the chunk left open at the end, so that the state is read and written
// by one block, in that order.
template <int D>
__global__ void __launch_bounds__(32 * kBulkWarps, 4)
append_bulk_kernel(Shape s, Q4 c, Append a)
{
    using R = Row<D>;
    pdl_launch_dependents();
    __shared__ float part[kBulkWarps][D + 2];
    const int b = blockIdx.z, r = blockIdx.y;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, grp = lane / R::LPK, sub = lane % R::LPK;
    int L, n;
    span(s, a, b, &L, &n);
    if (n == 0) return;
    const int end = L + n, first = L / s.B, ci = first + blockIdx.x, open = end / s.B;
    if (ci * s.B >= end || (ci == open && ci != first)) return;
    float qv[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) qv[e] = a.qbar[r * D + sub * 8 + e] * (kLog2e * rsqrtf((float)D));
    const float ke = exp2i(-c.kexp), ve = exp2i(-c.vexp);
    float* st = a.state + ((long long)b * s.hkv + r) * (D + 2);
    const __nv_bfloat16* kb = a.K + (long long)b * s.ks[0] + (long long)r * s.ks[2] + sub * 8;
    const __nv_bfloat16* vb = a.V + (long long)b * s.vs[0] + (long long)r * s.vs[2] + sub * 8;

    auto chunk = [&](int cc, bool with_state) {
        const int t0 = max(cc * s.B, L), t1 = min((cc + 1) * s.B, end);
        // This lane's rows are first_row + i STEP of the chunk; the first ones are on their way before the page
        // is known, the next ones before the present ones are worked on.
        constexpr int U = 4, STEP = kBulkWarps * R::KPI;
        const int first_row = warp * R::KPI + grp;
        const __nv_bfloat16* kp = kb + (long long)(t0 - L + first_row) * s.ks[1];
        const __nv_bfloat16* vp = vb + (long long)(t0 - L + first_row) * s.vs[1];
        const long long kstep = STEP * s.ks[1], vstep = STEP * s.vs[1];
        int left = t1 - t0 - first_row;   // row i is there while left > i STEP
        uint4 kr[U], vr[U];
        auto load = [&](int rows) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                kr[u] = vr[u] = make_uint4(0u, 0u, 0u, 0u);
                if (rows > u * STEP) {
                    kr[u] = *reinterpret_cast<const uint4*>(kp);
                    vr[u] = *reinterpret_cast<const uint4*>(vp);
                }
                kp += kstep;
                vp += vstep;
            }
        };
        load(left);
        const int pg = q4_page(c, b, t0);
        const bool all = pg >= 0;
        const long long row = (long long)r * c.psz + t0 % c.psz + first_row, page = all ? pg : 0;
        uint8_t* kc = c.kc + page * c.kcp + row * (D / 2) + key_word<D>(sub) * 4;
        uint8_t* vc = c.vc + page * c.vcp + row * (D / 2) + sub * 4;
        uint8_t* ks = c.ks + page * c.ksp + row * (D / kGrp) + (sub >> 2);
        uint8_t* vs = c.vs + page * c.vsp + row * (D / kGrp) + (sub >> 2);
        Sum run;
        run.init();
        for (; __any_sync(0xffffffffu, left > 0); left -= U * STEP) {
            float k[U][8], z[U], top = run.m;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                Vec<__nv_bfloat16>::cvt(kr[u], k[u]);
                z[u] = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) z[u] = fmaf(qv[e], k[u][e], z[u]);
#pragma unroll
                for (int o = R::LPK / 2; o > 0; o >>= 1) z[u] += __shfl_xor_sync(0xffffffffu, z[u], o);
                if (left <= u * STEP) z[u] = -INFINITY;
                top = fmaxf(top, z[u]);
            }
            const float ref = top == -INFINITY ? 0.f : top, sc = exp2f(run.m - ref);
            run.m = top;
            run.l *= sc;
#pragma unroll
            for (int e = 0; e < 8; ++e) run.a[e] *= sc;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const float p = exp2f(z[u] - ref);   // 0 for rows that are not there (their keys are zeros)
                run.l += p;
#pragma unroll
                for (int e = 0; e < 8; ++e) run.a[e] = fmaf(p, k[u][e], run.a[e]);
                uint32_t sb;
                const uint32_t w = quant8(kr[u], k[u], ke, &sb);
                if (all && left > u * STEP) {
                    *reinterpret_cast<uint32_t*>(kc + u * STEP * (D / 2)) = w;
                    if ((sub & 3) == 0) ks[u * STEP * (D / kGrp)] = (uint8_t)sb;
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float v[8];
                Vec<__nv_bfloat16>::cvt(vr[u], v);
                uint32_t sb;
                const uint32_t w = quant8(vr[u], v, ve, &sb);
                if (all && left > u * STEP) {
                    *reinterpret_cast<uint32_t*>(vc + u * STEP * (D / 2)) = w;
                    if ((sub & 3) == 0) vs[u * STEP * (D / kGrp)] = (uint8_t)sb;
                }
            }
            kc += U * STEP * (D / 2);
            vc += U * STEP * (D / 2);
            ks += U * STEP * (D / kGrp);
            vs += U * STEP * (D / kGrp);
            load(left - U * STEP);
        }
#pragma unroll
        for (int o = R::LPK; o < 32; o <<= 1) {
            const float m2 = __shfl_xor_sync(0xffffffffu, run.m, o), l2 = __shfl_xor_sync(0xffffffffu, run.l, o);
            float a2[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) a2[e] = __shfl_xor_sync(0xffffffffu, run.a[e], o);
            run.merge(m2, l2, a2);
        }
        if (grp == 0) write_state<D>(part[warp], sub, run);
        __syncthreads();
        if (warp == 0 && grp == 0) {
            for (int w = 1; w < kBulkWarps; ++w) run.merge(part[w][D], part[w][D + 1], part[w] + sub * 8);
            if (with_state) {
                float old[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) old[e] = st[sub * 8 + e];
                run.merge(st[D], st[D + 1], old);
            }
            __syncwarp((1ull << R::LPK) - 1);   // the state is read by these lanes before it is written
            if ((cc + 1) * s.B <= end)
                write_summary<D>(a.kbar + (((long long)b * s.hkv + r) * s.T + cc) * D, sub, run);
            else
                write_state<D>(st, sub, run);
        }
        __syncthreads();   // `part` is used again
    };
    chunk(ci, ci == first && L % s.B != 0);
    if (blockIdx.x == 0) {
        if (end % s.B == 0) {
            if (warp == 0 && grp == 0) {
                Sum none;
                none.init();
                write_state<D>(st, sub, none);
            }
        } else if (open != first) {
            chunk(open, false);
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
// most 7 significant bits.
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
        const int pg = slot < c.pmax ? __ldg(table + slot) : -1;
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
    // second launch.
    if (a.n_new <= 4) {
        append_few_kernel<D><<<s.batch, 32 * (s.hkv < 16 ? s.hkv : 16), 0, st>>>(s, c, a);
        return cudaGetLastError();
    }
    const int chunks = (a.n_new + s.B - 2) / s.B + 1;
    append_bulk_kernel<D><<<dim3(chunks, s.hkv, s.batch), 32 * kBulkWarps, 0, st>>>(s, c, a);
    cudaError_t e = cudaGetLastError();
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
    if (s.d == 128) load_kernel<128><<<grid, 32 * kLoadWarps, 0, st>>>(s, c, a);
    else load_kernel<64><<<grid, 32 * kLoadWarps, 0, st>>>(s, c, a);
    return cudaGetLastError();
}

}  // namespace dash
