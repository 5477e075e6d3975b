// q4_route.cu -- Stage 1 of decoding for the 4-bit cache's decode: chunk logits over the whole GPU, then
// thresholds of the heads and the pairs' route lists.
//
// The quantities are those of stage1_decode.cu (Eq. 6 and Proposition 4.1):
//   x_c^(h) = (alpha-1) gamma <q^(h), kbar_c>/sqrt(d),  what = [x - tau]_+^{1/(alpha-1)},  w = mean over heads,
//   R = {w > 0},  bias_c = (log w_c - mean_R log w)/sigma
// and the logits are the same numbers (the same MMAs on the exact three-plane split of kbar).  There one
// cluster does all of it for a (sequence, KV head), which leaves most SMs idle while the summaries are read
// and has every head's threshold solved on a list that crosses blocks.  Here
//   1. a warp takes 16 chunks of a pair, reads their summaries once (all loads in flight together) and
//      writes the group's logits: HBM-bound, 4 d bytes per chunk;
//   2. a block per (pair, head) holds the head's row in registers, less its maximum: a Newton step is one pass over them
//      and one block barrier.  The weights take the logits' place (in L2).  Rows of more than 16384 chunks are read again
//      at every step instead (one pair of 57600 chunks: 55 us a call);
//   3. in a cluster of 4 blocks per pair each block adds up the heads' weights for a quarter of the chunks, and
//      the blocks tell each other their counts and sums of logarithms.
// Short rows take one block and one launch instead (route_short_kernel; in the shortest caches the attending block
// does it, see q4_decode.cu).
// Measured: with cold caches 16 pairs of 2047 chunks and 16 heads of 128 take 10 us for the logits (16.8 MB, 1.7
// TB/s: a read of this size is latency); one cluster for everything takes 25 to 26 us there.  Whole calls: steps 2
// and 3 in one kernel, with the heads spread over the cluster's blocks, are 1 us slower there (36.3 against
// 35.3) and 15 us with 128 pairs (79.6 against 64.1): a launch costs less than a cluster barrier, and blocks of
// one head fill the GPU.  Clusters of 8 are slower: 15 of 16 fit.
#include <cooperative_groups.h>

#include "q4_route.cuh"

namespace cg = cooperative_groups;

namespace dash {
namespace {

constexpr int kLogitWarps = 8, kTiles = 2;   // 8-chunk tiles per warp
constexpr int kCl = 4, kThr = 512, kWarps = kThr / 32, kMaxVals = 32, kLong = 8;

// X [pair][head][T]: the logits of the complete chunks before each query's own.
template <int D>
__global__ void __launch_bounds__(32 * kLogitWarps) route_logits_kernel(Shape s, const __nv_bfloat16* q, const float* kbar,
                                                                        const int* seqlens, float* X)
{
    pdl_wait();   // the append of this step
    pdl_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g8 = lane >> 2, t4 = lane & 3, G = s.g;
    const unsigned per = (s.T + 8 * kTiles - 1) / (8 * kTiles);
    const unsigned unit = blockIdx.x * kLogitWarps + warp;   // at most 2048 pairs x 57600 chunks / 16
    if (unit >= (unsigned)(s.batch * s.hkv) * per) return;
    const int br = unit / per, c0 = (unit % per) * 8 * kTiles, b = br / s.hkv, r = br % s.hkv;
    const int nv = chunks_of(s, seqlens, b);
    if (c0 >= nv) return;
    const float* kb = kbar + ((long long)br * s.T + c0 + g8) * D + 2 * t4;
    float2 u[kTiles][D / 16][2];
#pragma unroll
    for (int t = 0; t < kTiles; ++t) load_tile<D>(u[t], kb + t * 8 * D, c0 + t * 8 + g8 < nv);
    uint32_t qf[D / 16][4];
    const __nv_bfloat16* qb = q + ((long long)b * s.hq + r * G) * D;
    load_q_frags<D>(qf, [&](int h) -> const __nv_bfloat16* { return h < G ? qb + (long long)h * D : nullptr; });
    const float xs = (s.alpha - 1.f) * s.gamma * rsqrtf((float)D);
    float* out = X + (long long)br * G * s.T;
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
        float acc[4] = {0.f, 0.f, 0.f, 0.f};
        tile_logits<D>(acc, qf, u[t]);
        const int c = c0 + t * 8 + 2 * t4;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int h = g8 + (e >> 1) * 8;
            if (h < G && c + (e & 1) < nv) out[(long long)h * s.T + c + (e & 1)] = acc[e] * xs;
        }
    }
}

struct Cross {     // what a block tells the others of its cluster about its quarter of the chunks
    float slog;    // sum of log w over the routed ones
    int cnt;
};

// Warps of a head: as few (a power of two) as leave 16 entries or less per thread.
inline int warps_per_head(int T)
{
    int w = 1;
    while (w < kWarps && T > 16 * 32 * w) w *= 2;
    return w;
}

// Chunks per block in the last phase: whole 32-chunk words.
__host__ __device__ inline int quarter(int nv) { return ((nv + kCl - 1) / kCl + 31) / 32 * 32; }

// Thresholds: a block per (pair, head).  The head's weights [x - tau]_+^p take its logits' place in X.  V: entries per
// thread, held in registers; 0: rows of any length, read again (from L1 and L2) at every step, kLong at a time.
template <int V>
__global__ void __launch_bounds__(kThr) route_tau_kernel(Shape s, float* X, const int* seqlens, int* status)
{
    __shared__ float red[kWarps];
    __shared__ float2 part[2][kWarps];
    pdl_wait();
    pdl_launch_dependents();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, step = blockDim.x, warps = step >> 5;
    if (blockIdx.x == 0 && tid == 0) *status = 0;
    const int nv = chunks_of(s, seqlens, blockIdx.x / (s.g * s.hkv));
    if (nv == 0) return;
    const float p = 1.f / (s.alpha - 1.f);
    const int mode = ent_mode(s.alpha);
    constexpr int N = V ? V : kLong;
    float v[N], mx = -INFINITY;
    float* row = X + (long long)blockIdx.x * s.T;
    auto load = [&](int c0) {
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] = c0 + k * step < nv ? row[c0 + k * step] : -INFINITY;
    };
    auto relative = [&] {
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] -= mx;
    };
    // f on every part of the row, less its maximum (one part where it is in registers)
    auto parts = [&](auto f) {
        if constexpr (V != 0) {
            f(tid);
        } else {
            for (int c0 = tid; c0 < nv; c0 += N * step) {
                load(c0);
                relative();
                f(c0);
            }
        }
    };
    for (int c0 = tid; c0 < (V ? tid + 1 : nv); c0 += N * step) {
        load(c0);
#pragma unroll
        for (int k = 0; k < N; ++k) mx = fmaxf(mx, v[k]);
    }
    mx = warp_max(mx);
    if (warps > 1) {
        if (lane == 0) red[warp] = mx;
        __syncthreads();
        for (int k = 0; k < warps; ++k) mx = fmaxf(mx, red[k]);
    }
    if constexpr (V != 0) relative();
    // Newton steps from the maximum - 1, at most one barrier each
    float lo, t, hi;
    bracket(lo, t, hi, s.alpha, nv);
    for (int it = 0; it < kMaxIter; ++it) {
        float f = 0.f, fd = 0.f;
        parts([&](int) { sums<N>(v, t, p, mode, f, fd); });
        f = warp_sum(f);
        fd = warp_sum(fd);
        if (warps > 1) {
            if (lane == 0) part[it & 1][warp] = make_float2(f, fd);
            __syncthreads();   // a buffer is written again two steps, and a barrier, later
            f = fd = 0.f;
#pragma unroll
            for (int k = 0; k < kWarps; ++k) {
                if (k >= warps) break;
                const float2 o = part[it & 1][k];
                f += o.x;
                fd += o.y;
            }
        }
        if (newton(f, fd, t, lo, hi, s.alpha, mode)) break;   // the same numbers in every thread
    }
    parts([&](int c0) {
#pragma unroll
        for (int k = 0; k < N; ++k)
            if (c0 + k * step < nv) __stcg(row + c0 + k * step, weight_of(v[k] - t, p, mode));
    });
}

// Group weights and lists: a cluster of 4 blocks per pair, a quarter of the chunks each.
__global__ void __cluster_dims__(kCl, 1, 1) __launch_bounds__(kThr, 1)
    route_list_kernel(Shape s, const float* X, const int* seqlens, Routes rt)
{
    extern __shared__ float keep[];   // the weights of this block's quarter of the chunks
    __shared__ float lsum[kWarps];
    __shared__ int csum[kWarps];
    __shared__ Cross cx;
    cg::cluster_group cl = cg::this_cluster();
    pdl_wait();
    pdl_launch_dependents();
    const int rank = (int)cl.block_rank(), br = blockIdx.x / kCl, G = s.g;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int nv = chunks_of(s, seqlens, br / s.hkv);

    // ---- group weights of this block's quarter of the chunks, in whole 32-chunk words --------------
    const int per = quarter(nv), c_lo = min(nv, rank * per), c_hi = min(nv, c_lo + per);
    const int each = ((c_hi - c_lo + kWarps - 1) / kWarps + 31) / 32 * 32;   // a warp's part, in words too
    const int w_lo = min(c_hi, c_lo + warp * each), w_hi = min(c_hi, w_lo + each);
    const float inv_g = 1.f / G;
    const float* wrow = X + (long long)br * G * s.T;
    auto weight = [&](int c) {   // the heads in order; the reads are on their way before the first is added
        float a[16];
        GroupWeight sum;
#pragma unroll
        for (int k = 0; k < 16; ++k) a[k] = k < G ? __ldcg(wrow + (long long)k * s.T + c) : __int_as_float(0x7fffffff);
#pragma unroll
        for (int k = 0; k < 16; ++k) sum.add(a[k]);
        return sum.mean(inv_g);
    };
    float sl = 0.f;
    int cn = 0;
#pragma unroll 1
    for (int c = w_lo + lane; c < w_hi; c += 32) {
        const float w = weight(c);
        keep[c - c_lo] = w;
        if (routed(w)) { sl += __logf(w); ++cn; }
    }
    sl = warp_sum(sl);
    cn = warp_isum(cn);
    if (lane == 0) { lsum[warp] = sl; csum[warp] = cn; }
    __syncthreads();
    if (tid == 0) {
        float a = 0.f;
        int n = 0;
        for (int k = 0; k < kWarps; ++k) { a += lsum[k]; n += csum[k]; }
        cx.slog = a;
        cx.cnt = n;
    }
    cl.sync();
    float tot_log = 0.f;
    int tot = 0, at = 0;
    for (int k = 0; k < kCl; ++k) {
        const Cross* o = cl.map_shared_rank(&cx, k);
        tot_log += o->slog;
        if (k < rank) at += o->cnt;
        tot += o->cnt;
    }
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");   // done with the others' memory
    for (int k = 0; k < warp; ++k) at += csum[k];
    const float mu = tot > 0 ? tot_log / tot : 0.f;

    // ---- ascending lists ---------------------------------------------------------------------------
    int* idx = rt.idx + (long long)br * rt.cap;
    float* bias = rt.bias + (long long)br * rt.cap;
    uint32_t* mrow = rt.bitmask ? rt.bitmask + (long long)br * rt.words : nullptr;
#pragma unroll 1
    for (int c0 = w_lo; c0 < w_hi; c0 += 32) {
        const int c = c0 + lane;
        const float w = c < w_hi ? keep[c - c_lo] : 0.f;
        const bool on = routed(w);
        const uint32_t m = __ballot_sync(0xffffffffu, on);
        if (on) {
            const int j = at + __popc(m & ((1u << lane) - 1u));
            idx[j] = c;
            bias[j] = (__logf(w) - mu) * s.inv_sigma;
        }
        if (mrow && lane == 0) mrow[c0 >> 5] = m;
        at += __popc(m);
    }
    if (rank == 0) {
        if (tid == 0) rt.counts[br] = tot;
        if (mrow)
            for (int wd = ((nv + 31) >> 5) + tid; wd < rt.words; wd += kThr) mrow[wd] = 0u;
    }
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");   // no block leaves while its memory is read
}

template <int D, int V>
__global__ void __launch_bounds__(512) route_short_kernel(Shape s, const __nv_bfloat16* q, const float* kbar,
                                                          const int* seqlens, Routes rt, int* status)
{
    __shared__ float x[16 * (32 * V + 4)], sums_of[2 * V];
    pdl_wait();   // the append of this step
    pdl_launch_dependents();
    if (blockIdx.x == 0 && threadIdx.x == 0) *status = 0;
    route_row<D, V>(s, q, kbar, rt, blockIdx.x, chunks_of(s, seqlens, blockIdx.x / s.hkv), x, sums_of);
}

// Where one block does it all.  Up to 512 chunks (16 entries per lane), and as long as reading the summaries with
// one SM costs less than the launch and the cluster barriers that it saves: d = 64, 24 chunks 16.4 -> 12.3 us
// a call, 500 chunks 21.2 -> 17.6; d = 128, 127 chunks 25.4 -> 22.3, 255 chunks 26.7 -> 25.1, 300 chunks 21.1 ->
// 19.7, but 511 chunks 29.7 -> 30.5.
bool short_row(const Shape& s) { return s.T <= 512 && s.T * s.d <= 40960; }

template <int D, int V>
cudaError_t short_t(const Shape& s, const void* q, const float* kbar, const int* seqlens, const Routes& rt, int* status,
                    cudaStream_t st)
{
    // a warp per head, per 32 chunks, and (up to 16) per tile
    int warps = s.g > V ? s.g : V;
    while (warps < 16 && warps * 8 < s.T) warps *= 2;
    return launch_after(route_short_kernel<D, V>, dim3(s.batch * s.hkv), dim3(32 * warps), 0, st, s,
                        (const __nv_bfloat16*)q, kbar, seqlens, rt, status);
}
template <int V>
cudaError_t short_v(const Shape& s, const void* q, const float* kbar, const int* seqlens, const Routes& rt, int* status,
                    cudaStream_t st)
{
    return s.d == 128 ? short_t<128, V>(s, q, kbar, seqlens, rt, status, st) : short_t<64, V>(s, q, kbar, seqlens, rt, status, st);
}

template <int V>
cudaError_t tau_t(const Shape& s, float* X, const int* seqlens, int* status, cudaStream_t st)
{
    return launch_after(route_tau_kernel<V>, dim3(s.batch * s.hkv * s.g), dim3(32 * warps_per_head(s.T)), 0, st, s, X, seqlens,
                        status);
}

}  // namespace

// Rows that a block's registers hold, longer ones as long as a pair's logits (the heads' rows) stay within 225 KB.
bool route_q4_supported(const Shape& s) { return s.T > 0 && (s.T <= kMaxVals * kThr || (long long)s.g * s.T <= 57600); }

cudaError_t launch_route_q4(const Shape& s, const void* q, const float* kbar, const int* seqlens, const Routes& rt,
                            float* X, int* status, cudaStream_t st)
{
    if (short_row(s))
        return s.T <= 128 ? short_v<4>(s, q, kbar, seqlens, rt, status, st)
                          : s.T <= 256 ? short_v<8>(s, q, kbar, seqlens, rt, status, st) : short_v<16>(s, q, kbar, seqlens, rt, status, st);
    const long long units = (long long)s.batch * s.hkv * ((s.T + 8 * kTiles - 1) / (8 * kTiles));
    const dim3 grid((unsigned)((units + kLogitWarps - 1) / kLogitWarps));
    cudaError_t e = launch_after(s.d == 128 ? route_logits_kernel<128> : route_logits_kernel<64>, grid,
                                       dim3(32 * kLogitWarps), 0, st, s, (const __nv_bfloat16*)q, kbar, seqlens, X);
    if (e != cudaSuccess) return e;
    e = s.T <= 16 * kThr         ? tau_t<16>(s, X, seqlens, status, st)
        : s.T <= kMaxVals * kThr ? tau_t<kMaxVals>(s, X, seqlens, status, st)
                                 : tau_t<0>(s, X, seqlens, status, st);
    if (e != cudaSuccess) return e;
    const int keep = quarter(s.T) * 4;   // at most 57.6 KB (T <= 57600)
    if (keep > 48 * 1024 &&
        (e = cudaFuncSetAttribute(route_list_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, keep)) != cudaSuccess)
        return e;
    return launch_after(route_list_kernel, dim3(kCl * s.batch * s.hkv), dim3(kThr), keep, st, s, (const float*)X, seqlens, rt);
}

}  // namespace dash
