// q4_route.cuh -- pieces of Stage 1 that the 4-bit decode's routing kernels share (mathematics: q4_route.cu).
#pragma once
#include "entmax.cuh"
#include "q4.cuh"
#include "stage2_mma.cuh"

namespace dash {

// (hi, mid, lo) bf16 pairs with hi + mid + lo == (x0, x1) exactly, by truncation.
__device__ __forceinline__ void split3(float2 x, uint32_t& hi, uint32_t& mid, uint32_t& lo)
{
    const float h0 = __uint_as_float(__float_as_uint(x.x) & 0xffff0000u), h1 = __uint_as_float(__float_as_uint(x.y) & 0xffff0000u);
    const float r0 = x.x - h0, r1 = x.y - h1;
    const float m0 = __uint_as_float(__float_as_uint(r0) & 0xffff0000u), m1 = __uint_as_float(__float_as_uint(r1) & 0xffff0000u);
    hi = __byte_perm(__float_as_uint(h0), __float_as_uint(h1), 0x7632);
    mid = __byte_perm(__float_as_uint(m0), __float_as_uint(m1), 0x7632);
    lo = __byte_perm(__float_as_uint(r0 - m0), __float_as_uint(r1 - m1), 0x7632);
}

// Complete chunks before the query's own (a length beyond the capacity counts as the capacity).
__device__ __forceinline__ int chunks_of(const Shape& s, const int* seqlens, int b)
{
    return max(0, (min(seqlens[b], s.n) - 1) / s.B);
}

// The chunks' summaries of one 8-chunk tile: this lane's elements of chunk g8 (on: it is there).
template <int D>
__device__ __forceinline__ void load_tile(float2 (&u)[D / 16][2], const float* p, bool on)
{
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
        u[kk][0] = on ? *reinterpret_cast<const float2*>(p + kk * 16) : make_float2(0.f, 0.f);
        u[kk][1] = on ? *reinterpret_cast<const float2*>(p + kk * 16 + 8) : make_float2(0.f, 0.f);
    }
}
// acc += q u^T: heads g8 and g8 + 8, chunks 2 t4 and 2 t4 + 1
template <int D>
__device__ __forceinline__ void tile_logits(float* acc, const uint32_t (&qf)[D / 16][4], const float2 (&u)[D / 16][2])
{
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
        uint32_t h0, m0, l0, h1, m1, l1;
        split3(u[kk][0], h0, m0, l0);
        split3(u[kk][1], h1, m1, l1);
        mma_bf16(acc, qf[kk], l0, l1);
        mma_bf16(acc, qf[kk], m0, m1);
        mma_bf16(acc, qf[kk], h0, h1);
    }
}

// u^p for u >= 0 (or a NaN, which stays), kept out of line: alpha other than 1.5 and 2 is rare, and code that is only passed over
// has to be fetched too (these kernels run once per call, from a cold instruction cache).
static __device__ __noinline__ float power(float u, float p) { return u > 0.f ? exp2f(p * __log2f(u)) : u; }

// Weight [x]_+^p of a logit x less the threshold.  The solve passes over NaNs; here they come back.
__device__ __forceinline__ float weight_of(float x, float p, int mode)
{
    const float u = x < 0.f ? 0.f : x;
    return mode == 2 ? u * u : mode == 1 ? u : power(u, p);
}
// A chunk's group weight, from the heads' in order.  A summary that is not finite gives every head a NaN: the weight is
// one too, the chunk is routed, and the mean of the logarithms carries it to all of the pair's biases and outputs.  A
// query that is not finite gives them to its own head alone, whose output they reach anyway: the others go without it.
struct GroupWeight {
    float sum = 0.f;
    bool any = false;
    __device__ __forceinline__ void add(float w)
    {
        if (w == w) {
            sum += w;
            any = true;
        }
    }
    __device__ __forceinline__ float mean(float inv_g) const { return any ? sum * inv_g : __int_as_float(0x7fffffff); }
};
__device__ __forceinline__ bool routed(float w) { return !(w <= 0.f); }

// f = sum u^p, fd = sum u^(p-1) over the entries u = v - t > 0 of this thread.
template <int V>
__device__ __forceinline__ void sums(const float* v, float t, float p, int mode, float& f, float& fd)
{
    if (mode == 2) {
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const float u = fmaxf(v[k] - t, 0.f);
            fd += u;
            f = fmaf(u, u, f);
        }
    } else if (mode == 1) {
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const float u = fmaxf(v[k] - t, 0.f);
            f += u;
            fd += u > 0.f ? 1.f : 0.f;
        }
    } else {
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const float u = fmaxf(v[k] - t, 0.f);
            if (u > 0.f) { f += power(u, p); fd += power(u, p - 1.f); }
        }
    }
}

// The solve's start on a row that its maximum has been taken off: the threshold lies in [-1, -nv^-(alpha-1)].  (Entries
// near the maximum differ from it exactly, so the threshold is as fine as a weight whatever the logits' size; solved on
// the logits themselves it would have their spacing: weights off by 2% at logits of 1e5, and none left from 2^24 on.)
__device__ __forceinline__ void bracket(float& lo, float& t, float& hi, float alpha, int nv)
{
    lo = t = -1.f;
    hi = -exp2f(-(alpha - 1.f) * __log2f((float)nv));
}

// One Newton step of the threshold solve (ent_step of entmax.cuh without its closed forms, on the fast
// divide and square root: a step corrects what the one before was off by).  f, fd: sums of u^p and u^(p-1).
__device__ __forceinline__ bool newton(float f, float fd, float& t, float& lo, float& hi, float alpha, int mode)
{
    if (f >= 1.f) lo = t;
    else hi = t;
    float tn = 0.5f * (lo + hi);
    if (fd > 0.f && f > 0.f) {
        float g;
        if (mode == 2) asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(g) : "f"(f));
        else g = mode == 1 ? f : exp2f((alpha - 1.f) * __log2f(f));
        tn = t + __fdividef((g - 1.f) * f, g * fd);
    }
    if (fabsf(tn - t) <= 2e-7f * fmaxf(1.f, fabsf(t)) || fabsf(f - 1.f) <= 1e-6f) {
        t = tn;
        return true;
    }
    t = tn > lo && tn < hi ? tn : 0.5f * (lo + hi);
    return false;
}

// Rows of at most 32 V chunks by one block of V warps or more: routes of pair br, whose query has nv complete chunks
// before its own.  The tiles are shared by the warps, the logits stay in shared memory (x [16][32 V + 4], sums [2 V]),
// and a head is one warp's, whose Newton steps need no barrier.
template <int D, int V>
__device__ __forceinline__ void route_row(const Shape& s, const __nv_bfloat16* q, const float* kbar, const Routes& rt, int br,
                                          int nv, float* x, float* sums_of)
{
    constexpr int LD = 32 * V + 4;   // floats per head
    float* lsum = sums_of;
    int* csum = reinterpret_cast<int*>(sums_of + V);
    const int b = br / s.hkv, r = br % s.hkv, G = s.g, warps = blockDim.x >> 5;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g8 = lane >> 2, t4 = lane & 3;
    if (warp * 8 < nv) {
        uint32_t qf[D / 16][4];
        const __nv_bfloat16* qb = q + ((long long)b * s.hq + r * G) * D;
        load_q_frags<D>(qf, [&](int h) -> const __nv_bfloat16* { return h < G ? qb + (long long)h * D : nullptr; });
        const float scale = (s.alpha - 1.f) * s.gamma * rsqrtf((float)D);
        for (int c0 = warp * 8; c0 < nv; c0 += warps * 8) {
            float2 u[D / 16][2];
            load_tile<D>(u, kbar + ((long long)br * s.T + c0 + g8) * D + 2 * t4, c0 + g8 < nv);
            float acc[4] = {0.f, 0.f, 0.f, 0.f};
            tile_logits<D>(acc, qf, u);
#pragma unroll
            for (int e = 0; e < 4; ++e) x[(g8 + (e >> 1) * 8) * LD + c0 + 2 * t4 + (e & 1)] = acc[e] * scale;
        }
    }
    __syncthreads();

    // ---- thresholds; a head's weights take its logits' place ------------------------------------------
    const float p = 1.f / (s.alpha - 1.f);
    const int mode = ent_mode(s.alpha);
    for (int h = warp; h < G && nv > 0; h += warps) {
        float v[V], mx = -INFINITY;
#pragma unroll
        for (int k = 0; k < V; ++k) {
            v[k] = lane + 32 * k < nv ? x[h * LD + lane + 32 * k] : -INFINITY;
            mx = fmaxf(mx, v[k]);
        }
        mx = warp_max(mx);
#pragma unroll
        for (int k = 0; k < V; ++k) v[k] -= mx;
        float lo, t, hi;
        bracket(lo, t, hi, s.alpha, nv);
        for (int it = 0; it < kMaxIter; ++it) {
            float f = 0.f, fd = 0.f;
            sums<V>(v, t, p, mode, f, fd);
            f = warp_sum(f);
            fd = warp_sum(fd);
            if (newton(f, fd, t, lo, hi, s.alpha, mode)) break;
        }
#pragma unroll
        for (int k = 0; k < V; ++k) x[h * LD + lane + 32 * k] = weight_of(v[k] - t, p, mode);
    }
    __syncthreads();

    // ---- group weights, a warp per 32 chunks; ascending lists -----------------------------------------
    float w = 0.f, lw = 0.f;
    uint32_t m = 0;
    if (warp < V && warp * 32 < nv) {
        if (tid < nv) {
            GroupWeight sum;
            for (int k = 0; k < G; ++k) sum.add(x[k * LD + tid]);
            w = sum.mean(1.f / G);
        }
        m = __ballot_sync(0xffffffffu, routed(w));
        lw = routed(w) ? __logf(w) : 0.f;
        const float sl = warp_sum(lw);
        if (lane == 0) { lsum[warp] = sl; csum[warp] = __popc(m); }
    } else if (warp < V && lane == 0) {
        lsum[warp] = 0.f;
        csum[warp] = 0;
    }
    __syncthreads();
    float all = 0.f;
    int total = 0, at = 0;
#pragma unroll
    for (int k = 0; k < V; ++k) {
        all += lsum[k];
        at += k < warp ? csum[k] : 0;
        total += csum[k];
    }
    if (m >> lane & 1) {
        const long long j = (long long)br * rt.cap + at + __popc(m & ((1u << lane) - 1u));
        rt.idx[j] = tid;
        rt.bias[j] = (lw - all / total) * s.inv_sigma;
    }
    if (tid == 0) rt.counts[br] = total;
    if (rt.bitmask && lane == 0 && warp < rt.words) rt.bitmask[(long long)br * rt.words + warp] = warp < V ? m : 0u;
}

}  // namespace dash
