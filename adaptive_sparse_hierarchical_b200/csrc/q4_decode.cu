// q4_decode.cu -- decode attention over a K/V cache held in 4 bits (format: include/dash_cache.h).
//
// One query per sequence, g heads of a KV head share the keys (Proposition 4.1):
//   o = sum_j 2^(z_j) v_j / sum_j 2^(z_j),  z_j = <q, k_j> log2(e)/sqrt(d) + bias_j log2(e)
// over the routed chunks (bias of the chunk) and the query's own chunk (bias 0); gamma = 0 takes
// every chunk with bias 0.
//
// Work is cut into granules of 32 tokens (16 for chunks of 16).  The granules of all (sequence, KV head) pairs form one
// list that the blocks share evenly; a block's warps take its granules in turn, each with its own
// online softmax and its own ring of cp.async stages (a granule is used by one warp only, so no
// barrier is involved), and merge at the end of a pair.  A pair inside one block is finished there;
// pieces of a pair that spans blocks are merged by a second kernel, in block order.  Short caches give each pair a
// block of its own, which routes the pair as well (SOLO).
//
// A warp computes S^T = K q^T and O^T = V^T P^T: 16 tokens (then 16 of the d_h elements) are the
// 16 rows of m16n8k16 MMAs and the heads the 8 columns, so groups of up to 8 heads fill the tile.
//   K: the f16 number with the bits of a code u in its lowest bits is u 2^-24, in the next four 16 u
//      2^-24 (subnormals: linear, and exact in the MMA): two masks, a shift and two masks turn a word
//      of 8 codes into operands, straight from a 16-byte load (key rows are stored in the operand's
//      order).  The query, scaled by a power of two to have its largest element in 2^14..2^15, is
//      exact in f16 (its elements for the upper masks divided by 16) down to 2^-27 of the largest.
//      Each scale group's sum is multiplied by the key's scale in fp32.  The codes' offset of 8 is one
//      more MMA: the tokens' scales times -8 sum(q) of each group (two f16 numbers, 22 bits).
//   V: ldmatrix turns the rows: a register holds the codes 4 g .. 4 g + 3 of a group for two tokens, and masks
//      and one byte permutation make four operands u_0, u_0 + 16 u_1, u_2, u_2 + 16 u_3 of it (subnormals again;
//      the difference of a pair's sums is taken at the end).  The 16 rows of a tile belong to one scale group, so
//      the scale goes to the other side: P s in f16, one product per group, token pair and head.  The offset is
//      8 times the sum of P s, kept by one more MMA for two groups (A = the scales, B = P).
//   P is rounded to f16 (2^-12 relative; sums of P are taken before the rounding, in fp32), turned from S^T's
//   accumulator layout into an operand by movmatrix, and P s is rounded to f16 once more (2^-12, of terms with codes
//   up to 15).  P is 2^room at the reference and at most 2^(room + 6), and P s stays below 2^15: room is 9 while the
//   value scales s met so far are below 1, then 8 - floor(log2 s) of the largest (0 from 256 on), so small scales do not
//   push P s below f16's normals.  The reference moves only when a logit exceeds room by more than 6, or when room shrinks.
//
// Bound: 17/32 bytes of HBM per element are few enough for the unpacking to count: per 16 tokens of 128
// elements and 8 heads a warp issues some 260 instructions, of them 56 masks, 16 shifts and permutations, 14
// conversions (all integer pipe), 19 MMAs, and 25 for the copies and their addresses.
// Measured (L2 flushed): 48 pairs of 50021 tokens and fewer, 8 heads, all of it 283 MB: 60 us a call in short runs
// (4.7 TB/s, 72% of a copy; 58% of the issue slots, 56% of the integer pipe's and 34% of the tensor pipe's
// cycles), 64 to 66 in long ones, where the GPU's 1000 W hold the clock at 1.8 GHz.  A kernel without its loads takes
// 2 us less: it is the instructions.  16 pairs of 131072 tokens, 16 heads, a quarter routed, 91 MB: 36 us of a
// call's 54.8, some 7 of them the start and the merge.  Three sequences of 777 tokens and fewer, routed: 7.8 us a
// call, one launch.
// The values' scales on the weights' side instead of in every operand, with rows of one group per tile: 2% with
// the copies as they were, 8% with what it made possible (the byte permutation, two conversions at once).  No
// gain: shifts as multiplications (FMA pipe), 16 warps in one block, shares weighted by a block's place on its SM.
#include <cuda_fp16.h>

#include "q4_route.cuh"

namespace dash {
namespace {

constexpr int kMaxPairs = 2048;
constexpr int kSoloWords = 4;     // a block that has a pair to itself: at most 128 chunks (see q4_solo)
constexpr int kMeta = 64;         // granule descriptors per warp (two halves of 32)

// Descriptor of a granule: where its codes and scales lie, its chunk's bias, tokens | mapped << 8.
struct Meta {
    ulonglong2 kv[kMeta], sc[kMeta];
    float bias[kMeta];
    int nv[kMeta];
};

// Eight warps per block and as many blocks per SM as the registers of NT head tiles allow (128 and 255 per
// thread).  Two blocks merge and start at different times; one block of 16 warps is as fast.
template <int NT> struct Cfg { static constexpr int W = 8, BLOCKS = NT == 1 ? 2 : 1; };

// Granules of 16 U tokens (U = 2 wherever the chunk allows: descriptors, waits and votes are paid once for
// twice the tokens, and the warp has two independent chains to issue from); the ring holds 64 tokens.
template <int D, int U>
struct Stage {
    static constexpr int GRAN = 16 * U, N = 4 / U;
    static constexpr int CODES = GRAN * D / 2, SCALES = GRAN * D / kGrp;
    static constexpr int K = 0, V = CODES, KS = 2 * CODES, VS = 2 * CODES + SCALES, BYTES = 2 * (CODES + SCALES);
    static constexpr int OLD = D + 4;   // row length of the merge buffer [8 NT][OLD] that reuses a warp's ring
};

struct Attend {
    const __nv_bfloat16* q;
    const int* seqlens;
    int dense;        // every chunk before the query's own, bias 0 (no route lists)
    float* part;      // [block][first, last][g][D + 2]: partial o, reference, sum
    int2* span;       // [pairs]: first and last block of each pair (0, -1: no granules)
    __nv_bfloat16* O;
    const float* kbar;   // SOLO: the summaries, where the block routes its pair itself (else null)
};

__device__ __forceinline__ void mma_f16(float* c, const uint32_t* a, uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
                 "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void prefetch_l2(const char* p) { asm volatile("prefetch.global.L2 [%0];\n" ::"l"(p)); }
__device__ __forceinline__ uint32_t h2(__half2 v) { return *reinterpret_cast<uint32_t*>(&v); }
__device__ __forceinline__ __half2 h2(uint32_t v) { return *reinterpret_cast<__half2*>(&v); }
// d = a b, k = 8
__device__ __forceinline__ void mma_f16_k8(float* d, uint32_t a0, uint32_t a1, uint32_t b)
{
    asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5}, {%6}, {%7,%7,%7,%7};\n"
                 : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3]) : "r"(a0), "r"(a1), "r"(b), "f"(0.f));
}
// d = a b
__device__ __forceinline__ void mma_f16_0(float* d, const uint32_t* a, uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
                 "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};\n"
                 : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
// (c0, c1) + a (b0, b1) in one instruction
__device__ __forceinline__ void fma2(float& c0, float& c1, float a, float b0, float b1)
{
    asm("{\n\t.reg .b64 a, b, c;\n\tmov.b64 a, {%2, %2};\n\tmov.b64 b, {%3, %4};\n\tmov.b64 c, {%0, %1};\n\t"
        "fma.rn.f32x2 c, a, b, c;\n\tmov.b64 {%0, %1}, c;\n\t}\n"
        : "+f"(c0), "+f"(c1)
        : "f"(a), "f"(b0), "f"(b1));
}
// Four e4m3 bytes as two f16x2
__device__ __forceinline__ void e4m3x4_to_f16x4(uint32_t four, uint32_t& a, uint32_t& b)
{
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\tcvt.rn.f16x2.e4m3x2 %1, hi;\n\t}\n" : "=r"(a), "=r"(b) : "r"(four));
}
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t movm_t(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi)
{
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
// Length of sequence b as the kernels use it.
__device__ __forceinline__ int len_of(const Shape& s, const int* seqlens, int b) { return min(max(seqlens[b], 0), s.n); }

// SOLO: block x has pair x to itself: it routes it first, and there is nothing to merge.
template <int D, int NT, int U, bool SOLO>
__global__ void __launch_bounds__(32 * Cfg<NT>::W, Cfg<NT>::BLOCKS) q4_attend_kernel(Shape s, Q4 c, Routes rt, Attend a)
{
    constexpr int W = Cfg<NT>::W, NG = D / kGrp, MT = D / 16;
    using St = Stage<D, U>;
    constexpr int OLD = St::OLD, kGran = St::GRAN, kStages = St::N;
    static_assert(8 * NT * OLD * 4 <= kStages * St::BYTES, "the merge buffer reuses a warp's ring");
    extern __shared__ __align__(128) char smem[];
    __shared__ int pre[kMaxPairs + 1], at[kMaxPairs + 1], range[3];
    __shared__ float mrg_m[W][8 * NT], mrg_l[W][8 * NT], mrg_s[W][8 * NT], tot_m[8 * NT], tot_l[8 * NT];

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
    const int BR = s.batch * s.hkv, G = s.g, NB = s.B / kGran;
    {   // the page table and the query on their way to L2 while the routing still runs
        const long long at = ((long long)blockIdx.x * (32 * W) + threadIdx.x) * 128;
        if (at < (long long)s.batch * c.pmax * 4) prefetch_l2((const char*)c.pt + at);
        if (at < (long long)s.batch * s.hq * D * 2) prefetch_l2((const char*)a.q + at);
    }
    pdl_wait();   // the routes and the appended tokens of this step
    pdl_launch_dependents();
    auto granules = [&](int x) {
        const int L = len_of(s, a.seqlens, x / s.hkv);
        const int full = L > 0 ? (a.dense ? (L - 1) / s.B : rt.counts[x]) : 0;
        return L > 0 ? full * NB + ((L - 1) % s.B) / kGran + 1 : 0;
    };
    if constexpr (SOLO) {
        const int x = blockIdx.x;
        if (a.kbar) {
            float* scratch = reinterpret_cast<float*>(smem);   // 16 rows of 132 logits, 8 sums: the rings come later
            route_row<D, kSoloWords>(s, a.q, a.kbar, rt, x, chunks_of(s, a.seqlens, x / s.hkv), scratch, scratch + 16 * 132);
            __syncthreads();   // the routes are there, the scratch is free
        }
        const int n = granules(x);
        if (n == 0) {   // an empty sequence: zeros
            __nv_bfloat16* o = a.O + ((long long)(x / s.hkv) * s.hq + x % s.hkv * G) * D;
            for (int v = threadIdx.x; v < G * D / 8; v += 32 * W) reinterpret_cast<uint4*>(o)[v] = make_uint4(0u, 0u, 0u, 0u);
            return;
        }
        if (threadIdx.x == 0) {
            range[0] = pre[x] = 0;
            range[1] = pre[x + 1] = n;
            range[2] = x;
        }
    } else {
        for (int x = threadIdx.x; x < BR; x += 32 * W) pre[x + 1] = granules(x);
    }
    __syncthreads();
    if (!SOLO && warp == 0) {
        auto scan = [&](int* v, auto f) {   // v[x + 1] = f(0) + .. + f(x), v[0] = 0; returns the sum
            int run = 0;
            for (int x0 = 0; x0 < BR; x0 += 32) {
                const int x = x0 + lane;
                int n = x < BR ? f(x) : 0;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int u = __shfl_up_sync(0xffffffffu, n, o);
                    if (lane >= o) n += u;
                }
                if (x < BR) v[x + 1] = run + n;
                run += __shfl_sync(0xffffffffu, n, 31);
            }
            if (lane == 0) v[0] = 0;
            __syncwarp();
            return run;
        };
        auto last_le = [&](const int* v, int k) {   // the x with v[x] <= k < v[x + 1]
            int l = 0, h = BR;
            while (l < h) {
                const int m = (l + h) >> 1;
                if (v[m + 1] <= k) l = m + 1;
                else h = m;
            }
            return l;
        };
        const int total = scan(pre, [&](int x) { return pre[x + 1]; }), nb = (int)gridDim.x;
        // every warp of a block in use has a granule
        int used = min(nb, (total + W - 1) / W), x = 0, lo = 0, hi = 0;
        const int blk = (int)blockIdx.x;
        // Where one round of a block's warps is enough, pairs get blocks of their own: a pair that starts
        // inside a block costs it a merge, a descriptor chase and an empty ring (three short sequences: 17.4
        // us so, 18.9 with even shares; with more rounds even shares are as good or better).
        if (BR <= nb && total <= nb * W && scan(at, [&](int x) { return (pre[x + 1] - pre[x] + W - 1) / W; }) <= nb) {
            used = at[BR];
            if (blk < used) {
                x = last_le(at, blk);
                lo = pre[x] + (blk - at[x]) * W;
                hi = min(lo + W, pre[x + 1]);
            }
        } else if (blk < used) {
            // Even shares of the list, in which a pair starts with kPad granules that stand for that cost (four
            // rounds; three to five measure alike in the two large cases above, two 1 us more, none 3 to 4).
            constexpr int kPad = 4 * W;
            const int all = scan(at, [&](int x) { return pre[x + 1] > pre[x] ? pre[x + 1] - pre[x] + kPad : 0; });
            const int share = all / used, more = all - share * used;
            const int v0 = blk * share + min(blk, more), v1 = v0 + share + (blk < more);
            auto place = [&](int v, int y) { return pre[y] + max(0, v - at[y] - kPad); };
            x = last_le(at, v0);
            lo = place(v0, x);
            hi = place(v1, last_le(at, v1));
        }
        if (lane == 0) {
            range[0] = lo;
            range[1] = blk < used ? hi : 0;
            range[2] = x;
        }
    }
    if (!SOLO) __syncthreads();
    if (!SOLO && blockIdx.x == 0)
        for (int x = threadIdx.x; x < BR; x += 32 * W)
            if (pre[x] == pre[x + 1]) a.span[x] = make_int2(0, -1);
    const int lo = range[0], hi = range[1];
    if (hi == 0) return;   // a block without work
    int x = range[2];

    char* ring = smem + warp * (kStages * St::BYTES);
    const uint32_t ring_a = smem_u32(ring);
    Meta& meta = *reinterpret_cast<Meta*>(smem + W * kStages * St::BYTES + warp * sizeof(Meta));
    // the operands carry the codes times 2^-24
    const float scale2 = kLog2e * rsqrtf((float)D) * exp2i(c.kexp) * 16777216.f;
    const float out_scale = exp2i(24 + c.vexp);
    // This lane's row of the 8 x 8 matrices of 16 bits that ldmatrix takes from the value rows: token
    // (lane & 7) + 8 (lane >> 3 & 1), groups lane >> 4 and (D = 128) 2 more.  The groups of a row are
    // swizzled so that eight tokens' pieces of one group lie in different banks.
    auto v_at = [&](int group) {
        const int tok = (lane & 7) + ((lane >> 3) & 1) * 8;
        return (uint32_t)(St::V + tok * (D / 2) + (group ^ ((D == 128 ? tok >> 1 : tok >> 2) & (NG - 1))) * 16);
    };
    const uint32_t va0 = v_at(lane >> 4), va1 = v_at((lane >> 4) + (D == 128 ? 2 : 0));

    for (; x < BR && pre[x] < hi; ++x) {
        const int p0 = pre[x], p1 = pre[x + 1];
        const int s_lo = max(lo, p0), s_hi = min(hi, p1);
        if (s_lo >= s_hi) continue;
        const int b = x / s.hkv, r = x % s.hkv, i = len_of(s, a.seqlens, b) - 1;
        const int full = p1 - p0 - ((i % s.B) / kGran + 1);   // granules of routed chunks
        const int nm = max(0, (s_hi - s_lo - warp + W - 1) / W);

        // ---- granule descriptors, 32 at a time (page, row and number of tokens, bias) ----------------
        ulonglong2 f_kv = {}, f_sc = {};
        float f_b = 0.f;
        int f_nv = 0;
        auto fetch = [&](int m0) {
            const int m = m0 + lane;
            if (m >= nm) return;
            const int t = s_lo - p0 + warp + m * W;
            int tok, nv = kGran;
            f_b = 0.f;
            if (t < full) {
                int ch = t / NB;
                if (!a.dense) {
                    f_b = rt.bias[(long long)x * rt.cap + ch] * kLog2e;
                    ch = rt.idx[(long long)x * rt.cap + ch];
                }
                tok = ch * s.B + (t % NB) * kGran;
            } else {
                tok = (i / s.B) * s.B + (t - full) * kGran;
                nv = min(kGran, i + 1 - tok);
            }
            // Behind launches of the routing this kernel starts when all blocks of the last one have begun, which they do
            // after everything before that launch has ended: nobody writes the table any more, and the read-only path
            // holds (routed 128K 54.8 us, 55.9 without it).
            const int pg = q4_page(c, b, tok, [&](const int* e) { return !SOLO && !a.dense ? __ldg(e) : table_entry(e); });
            const long long p = pg >= 0 ? pg : 0, row = (long long)r * c.psz + tok % c.psz;
            f_kv.x = (unsigned long long)(c.kc + p * c.kcp + row * (D / 2));
            f_kv.y = (unsigned long long)(c.vc + p * c.vcp + row * (D / 2));
            f_sc.x = (unsigned long long)(c.ks + p * c.ksp + row * NG);
            f_sc.y = (unsigned long long)(c.vs + p * c.vsp + row * NG);
            f_nv = nv | (pg >= 0 ? 1 << 8 : 0);
        };
        auto publish = [&](int m0) {
            const int k = (m0 & 32) + lane;
            meta.kv[k] = f_kv;
            meta.sc[k] = f_sc;
            meta.bias[k] = f_b;
            meta.nv[k] = f_nv;
            __syncwarp();
        };
        constexpr int SP = St::SCALES / 16;
        const int lane16 = lane * 16, vlane16 = (lane ^ ((lane >> 3) & (NG - 1))) * 16;
        auto issue = [&](int m, uint32_t dst) {
            if (m < nm) {
                const int k = m & (kMeta - 1);
                const ulonglong2 kv = meta.kv[k];
                const unsigned long long sc = reinterpret_cast<const unsigned long long*>(&meta.sc[k])[(lane / SP) & 1];
                const int use = meta.nv[k];
                const uint32_t kd = dst + lane16, vd = dst + vlane16;
                const unsigned long long ka = kv.x + lane16, va = kv.y + lane16, sa = sc + lane16 % (SP * 16);
                const int have = lane < 2 * SP;
#define Q4_COPY(OFF) "cp.async.cg.shared.global [%0 + " #OFF "], [%2 + " #OFF "], 16, p;\n\t" \
                     "cp.async.cg.shared.global [%1 + %8 + " #OFF "], [%3 + " #OFF "], 16, p;\n\t"
#define Q4_COPIES(PIECES) asm volatile("{\n\t.reg .pred p, q;\n\tsetp.lt.s32 p, %5, 256;\n\tsetp.ne.s32 q, %7, 0;\n\t" \
                     PIECES "@q cp.async.cg.shared.global [%0 + %6], [%4], 16, p;\n\t}\n" \
                     ::"r"(kd), "r"(vd), "l"(ka), "l"(va), "l"(sa), "r"(use), "n"(St::KS), "r"(have), "n"(St::V))
                if constexpr (St::CODES == 2048) Q4_COPIES(Q4_COPY(0) Q4_COPY(512) Q4_COPY(1024) Q4_COPY(1536));
                else if constexpr (St::CODES == 1024) Q4_COPIES(Q4_COPY(0) Q4_COPY(512));
                else Q4_COPIES(Q4_COPY(0));
#undef Q4_COPIES
#undef Q4_COPY
            }
            cp_async_commit();
        };
        uint4 raw[NT][NG];   // the query: this lane's eight elements of each scale group, heads 8 nt + g
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int gg = 0; gg < NG; ++gg) {
                raw[nt][gg] = make_uint4(0u, 0u, 0u, 0u);
                if (nt * 8 + g < G)
                    raw[nt][gg] = *reinterpret_cast<const uint4*>(
                        a.q + ((long long)b * s.hq + r * G + nt * 8 + g) * D + gg * kGrp + t4 * 8);
            }
        fetch(0);
        publish(0);
#pragma unroll
        for (int k = 0; k < kStages - 1; ++k) issue(k, ring_a + k * St::BYTES);

        // ---- the query: operand B of S^T (columns = heads), in the order of the key words ------------
        uint32_t qf[NT][NG][4];   // elements (0, 4), (1, 5) / 16, (2, 6), (3, 7) / 16 of the lane's word
        uint32_t qs[NT];          // -2^-13 sum(q) of groups 2 (t4 % 2) and + 1: rounded to f16, and the rest
        float fac[NT][2];         // logit per accumulated unit of heads 2 t4 and 2 t4 + 1
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            uint32_t top = 0;
#pragma unroll
            for (int gg = 0; gg < NG; ++gg) {
                const uint4 w = raw[nt][gg];
                top = __vmaxu2(top, __vmaxu2(__vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu),
                                             __vmaxu2(w.z & 0x7fff7fffu, w.w & 0x7fff7fffu)));
            }
            top = max(top & 0xffffu, top >> 16);
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            // the power of two; a head with a NaN or an infinity becomes NaN as a whole
            const int ce = min(141 - (int)(top >> 7), 120);
            const float up = top >= 0x7f80u ? __int_as_float(0x7fffffff) : exp2i(ce);
            const float down = scale2 * exp2i(-ce);
            fac[nt][0] = __shfl_sync(0xffffffffu, down, 8 * t4);
            fac[nt][1] = __shfl_sync(0xffffffffu, down, 8 * t4 + 4);
            float sum[NG];
#pragma unroll
            for (int gg = 0; gg < NG; ++gg) {
                float v[8];
                Vec<__nv_bfloat16>::cvt(raw[nt][gg], v);
                sum[gg] = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) sum[gg] += v[e] * up;
                sum[gg] += __shfl_xor_sync(0xffffffffu, sum[gg], 1);
                sum[gg] += __shfl_xor_sync(0xffffffffu, sum[gg], 2);   // over t4: head g's sum
                const float up16 = up * 0.0625f;
                qf[nt][gg][0] = pack_f16(v[0] * up, v[4] * up);
                qf[nt][gg][1] = pack_f16(v[1] * up16, v[5] * up16);
                qf[nt][gg][2] = pack_f16(v[2] * up, v[6] * up);
                qf[nt][gg][3] = pack_f16(v[3] * up16, v[7] * up16);
            }
            // rows of the offset's operand: D = 128 has the rounded sums in lanes t4 = 0, 1 and the rests in
            // t4 = 2, 3; D = 64 in t4 = 0 and t4 = 1
            const bool second = D == 128 && (t4 & 1), rest = D == 128 ? t4 >= 2 : t4 == 1;
            const float x0 = -0.0001220703125f * (second ? sum[NG - 2] : sum[0]);
            const float x1 = -0.0001220703125f * (second ? sum[NG - 1] : sum[1]);
            const uint32_t hi = pack_f16(x0, x1);
            const float2 hf = __half22float2(h2(hi));
            qs[nt] = rest ? pack_f16(x0 - hf.x, x1 - hf.y) : D == 128 || t4 == 0 ? hi : 0u;
        }
        // o: tile 2 G + i holds rows of group G, elements 4 g + 2 i (rows g) and, 16 times as large, 4 g + 2 i + 1
        // (rows g + 8); off: sums of P s for groups 2 k (rows g, all alike) and 2 k + 1 (rows g + 8)
        float o[NT][MT][4], off[NT][NG / 2][4], ref[NT][2], l[NT][2];
        float room = 9.f;                   // P is 2^room at the reference's logit ...
        uint32_t above = 0x48484848u;       // ... + a scale byte: bit 7 where it is too large for that
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            ref[nt][0] = ref[nt][1] = -INFINITY;
            l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
            for (int m = 0; m < MT; ++m) o[nt][m][0] = o[nt][m][1] = o[nt][m][2] = o[nt][m][3] = 0.f;
#pragma unroll
            for (int k = 0; k < NG / 2; ++k) off[nt][k][0] = off[nt][k][1] = off[nt][k][2] = off[nt][k][3] = 0.f;
        }

        // The last granule of a pair may end before its last token: FULL = false.
        uint32_t cur = 0, nxt = (kStages - 1) * St::BYTES;   // ring offsets of granule m and of the one to load
        auto step = [&](int m, auto full_c) {
            constexpr bool FULL = decltype(full_c)::value;
            if ((m & 31) == 0) fetch(m + 32);
            if ((m & 31) == 16) publish(m + 16);
            cp_async_wait<kStages - 2>();
            __syncwarp();
            issue(m + kStages - 1, ring_a + nxt);
            const char* stg = ring + cur;
            const uint32_t stg_a = ring_a + cur;
            nxt = cur;
            cur = cur == (kStages - 1) * St::BYTES ? 0 : cur + St::BYTES;
            const int nv = FULL ? kGran : meta.nv[m & (kMeta - 1)] & 255;
            const float bias2 = meta.bias[m & (kMeta - 1)];

            // ---- S^T: rows 16 u + (tok_of(g), + 8), columns heads 2 t4, 2 t4 + 1 -------------------------
            float z[U][NT][4];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const char* ks = stg + St::K + u * 8 * D;
                const char* sc = stg + St::KS + u * 16 * NG;
                uint32_t ka[NG], kb[NG], sa, sb;
                if constexpr (D == 128) {
                    const uint4 x4 = *reinterpret_cast<const uint4*>(ks + g * 64 + t4 * 16);
                    const uint4 y4 = *reinterpret_cast<const uint4*>(ks + (g + 8) * 64 + t4 * 16);
                    ka[0] = x4.x; ka[1] = x4.y; ka[2] = x4.z; ka[3] = x4.w;
                    kb[0] = y4.x; kb[1] = y4.y; kb[2] = y4.z; kb[3] = y4.w;
                    sa = *reinterpret_cast<const uint32_t*>(sc + g * 4);
                    sb = *reinterpret_cast<const uint32_t*>(sc + (g + 8) * 4);
                } else {
                    const uint2 x2 = *reinterpret_cast<const uint2*>(ks + g * 32 + t4 * 8);
                    const uint2 y2 = *reinterpret_cast<const uint2*>(ks + (g + 8) * 32 + t4 * 8);
                    ka[0] = x2.x; ka[1] = x2.y;
                    kb[0] = y2.x; kb[1] = y2.y;
                    sa = *reinterpret_cast<const uint16_t*>(sc + g * 2);
                    sb = *reinterpret_cast<const uint16_t*>(sc + (g + 8) * 2);
                }
                uint32_t fa[NG / 2], fb[NG / 2];   // scales of this lane's two tokens, f16x2
                if constexpr (D == 128) {
                    e4m3x4_to_f16x4(sa, fa[0], fa[NG / 2 - 1]);
                    e4m3x4_to_f16x4(sb, fb[0], fb[NG / 2 - 1]);
                } else {
                    fa[0] = e4m3x2_to_f16x2(sa);
                    fb[0] = e4m3x2_to_f16x2(sb);
                }
                {
                    const uint32_t ua = (t4 & 1) ? fa[NG / 2 - 1] : fa[0], ub = (t4 & 1) ? fb[NG / 2 - 1] : fb[0];
                    const __half2 e8 = __float2half2_rn(0.00390625f);   // 2^-8: with the sums' 2^-13, 8 times 2^-24
                    const uint32_t f[2] = {h2(__hmul2(h2(ua), e8)), h2(__hmul2(h2(ub), e8))};
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma_f16_k8(z[u][nt], f[0], f[1], qs[nt]);
                }
#pragma unroll
                for (int gg = 0; gg < NG; ++gg) {
                    const uint32_t w = ka[gg], v = kb[gg], w8 = w >> 8, v8 = v >> 8;
                    const uint32_t f0[4] = {w & 0x000f000fu, v & 0x000f000fu, w & 0x00f000f0u, v & 0x00f000f0u};
                    const uint32_t f1[4] = {w8 & 0x000f000fu, v8 & 0x000f000fu, w8 & 0x00f000f0u, v8 & 0x00f000f0u};
                    const float2 pa = __half22float2(h2(fa[gg / 2])), pc = __half22float2(h2(fb[gg / 2]));
                    const float xa = gg & 1 ? pa.y : pa.x, xb = gg & 1 ? pc.y : pc.x;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float d[4];
                        mma_f16_0(d, f0, qf[nt][gg][0], qf[nt][gg][1]);
                        mma_f16(d, f1, qf[nt][gg][2], qf[nt][gg][3]);
                        fma2(z[u][nt][0], z[u][nt][1], xa, d[0], d[1]);
                        fma2(z[u][nt][2], z[u][nt][3], xb, d[2], d[3]);
                    }
                }
            }
            // logits relative to the reference; before the first one it is -inf and they are +inf
            float most = -INFINITY, tz[U][NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const float c0 = bias2 - ref[nt][0], c1 = bias2 - ref[nt][1];
#pragma unroll
                for (int u = 0; u < U; ++u) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) tz[u][nt][e] = fmaf(z[u][nt][e], fac[nt][e & 1], e & 1 ? c1 : c0);
                    if (!FULL) {
                        if (16 * u + g >= nv) tz[u][nt][0] = tz[u][nt][1] = -INFINITY;
                        if (16 * u + g + 8 >= nv) tz[u][nt][2] = tz[u][nt][3] = -INFINITY;
                    }
                    most = fmaxf(most, fmaxf(fmaxf(tz[u][nt][0], tz[u][nt][1]), fmaxf(tz[u][nt][2], tz[u][nt][3])));
                }
            }
            // the value scales of the granule, a word per lane (some lanes alike)
            constexpr int SW = St::SCALES / 4, TPW = 4 / NG;   // words, tokens per word
            uint32_t sw = *reinterpret_cast<const uint32_t*>(stg + St::VS + lane % SW * 4);
            if (!FULL) {
                const int left = nv - lane % SW * TPW;
                if (left < TPW) sw = left > 0 ? sw & 0xffffu : 0u;
            }
            if (__any_sync(0xffffffffu, most > room + 6.f || ((sw + above) & 0x80808080u))) {
                uint32_t top = 0;   // the largest scale byte that is a number
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t byte = (sw >> (8 * k)) & 0x7fu;
                    if (byte != 0x7fu) top = max(top, byte);
                }
                const float now = fminf(room, 15.f - (float)(__reduce_max_sync(0xffffffffu, top) >> 3));
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float mx = ref[nt][e] + room;   // the largest logit that moved the reference so far
#pragma unroll
                        for (int u = 0; u < U; ++u) {
                            float y0 = fmaf(z[u][nt][e], fac[nt][e], bias2), y1 = fmaf(z[u][nt][e + 2], fac[nt][e], bias2);
                            if (!FULL && 16 * u + g >= nv) y0 = -INFINITY;
                            if (!FULL && 16 * u + g + 8 >= nv) y1 = -INFINITY;
                            tz[u][nt][e] = y0;
                            tz[u][nt][e + 2] = y1;
                            mx = fmaxf(mx, fmaxf(y0, y1));
                        }
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                        const float base = mx == -INFINITY ? 0.f : mx - now, cr = exp2f(ref[nt][e] - base);
                        ref[nt][e] = mx == -INFINITY ? mx : base;
                        l[nt][e] *= cr;
#pragma unroll
                        for (int u = 0; u < U; ++u) { tz[u][nt][e] -= base; tz[u][nt][e + 2] -= base; }
#pragma unroll
                        for (int k = 0; k < MT; ++k) { o[nt][k][e] *= cr; o[nt][k][e + 2] *= cr; }
#pragma unroll
                        for (int k = 0; k < NG / 2; ++k) { off[nt][k][e] *= cr; off[nt][k][e + 2] *= cr; }
                    }
                room = now;
                above = (uint32_t)(8.f * room) * 0x01010101u;
            }
            uint32_t pb[U][NT][2];
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const float q0 = ex2(tz[u][nt][0]), q1 = ex2(tz[u][nt][1]), q2 = ex2(tz[u][nt][2]), q3 = ex2(tz[u][nt][3]);
                    l[nt][0] += q0 + q2;
                    l[nt][1] += q1 + q3;
                    pb[u][nt][0] = movm_t(pack_f16(q0, q1));
                    pb[u][nt][1] = movm_t(pack_f16(q2, q3));
                }

            // ---- O^T -----------------------------------------------------------------------------------
#pragma unroll
            for (int u = 0; u < U; ++u) {
                // codes 4 g .. 4 g + 3 of each group, tokens 2 t4 and 2 t4 + 1 in the halves (b: + 8)
                uint32_t a[NG], b[NG];
                const uint32_t row = stg_a + u * 8 * D;
                ldsm_x4_t(row + va0, a[0], b[0], a[1], b[1]);
                if constexpr (D == 128) ldsm_x4_t(row + va1, a[2], b[2], a[3], b[3]);
                uint32_t sl[NG], sh[NG];   // scales of these tokens, f16x2
                {
                    const char* sc = stg + St::VS + (16 * u + 2 * t4) * NG;
                    uint32_t w[2][NG / 2];   // bytes (2 t4, G), (2 t4 + 1, G), (2 t4, G + 1), (2 t4 + 1, G + 1)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        uint32_t x, y;
                        if constexpr (D == 128) {
                            const uint2 v = *reinterpret_cast<const uint2*>(sc + 8 * k * NG);
                            x = v.x;
                            y = v.y;
                        } else {
                            x = *reinterpret_cast<const uint32_t*>(sc + 8 * k * NG);
                            y = x >> 16;
                        }
                        if (!FULL) {   // beyond the query: whatever the page holds counts as 0
                            if (16 * u + 2 * t4 + 8 * k >= nv) x = 0u;
                            if (16 * u + 2 * t4 + 8 * k + 1 >= nv) y = 0u;
                        }
                        w[k][0] = __byte_perm(x, y, 0x5140);
                        if constexpr (D == 128) w[k][1] = __byte_perm(x, y, 0x7362);
                    }
#pragma unroll
                    for (int k = 0; k < NG / 2; ++k) {
                        e4m3x4_to_f16x4(w[0][k], sl[2 * k], sl[2 * k + 1]);
                        e4m3x4_to_f16x4(w[1][k], sh[2 * k], sh[2 * k + 1]);
                    }
                }
#pragma unroll
                for (int k = 0; k < NG / 2; ++k) {
                    const uint32_t f[4] = {sl[2 * k], sl[2 * k + 1], sh[2 * k], sh[2 * k + 1]};
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma_f16(off[nt][k], f, pb[u][nt][0], pb[u][nt][1]);
                }
#pragma unroll
                for (int gg = 0; gg < NG; ++gg) {
                    const uint32_t a8 = __byte_perm(a[gg], 0u, 0x4341), b8 = __byte_perm(b[gg], 0u, 0x4341);
                    const uint32_t f0[4] = {a[gg] & 0x000f000fu, a[gg] & 0x00ff00ffu, b[gg] & 0x000f000fu, b[gg] & 0x00ff00ffu};
                    const uint32_t f1[4] = {a8 & 0x000f000fu, a8, b8 & 0x000f000fu, b8};
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const uint32_t p0 = h2(__hmul2(h2(pb[u][nt][0]), h2(sl[gg]))), p1 = h2(__hmul2(h2(pb[u][nt][1]), h2(sh[gg])));
                        mma_f16(o[nt][2 * gg], f0, p0, p1);
                        mma_f16(o[nt][2 * gg + 1], f1, p0, p1);
                    }
                }
            }
        };
        // the pair's last granule, where it is partly filled, is this warp's last one or another warp's
        const bool part = nm > 0 && s_lo - p0 + warp + (nm - 1) * W == p1 - p0 - 1 && (i + 1) % kGran != 0;
        for (int m = 0; m < nm - part; ++m) step(m, std::true_type());
        if (part) step(nm - 1, std::false_type());

        // ---- merge the warps (fixed order), each through its own drained ring -----------------------
        cp_async_wait<0>();
        __syncwarp();
        float* ob = reinterpret_cast<float*>(ring);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float v = l[nt][e];
                v += __shfl_xor_sync(0xffffffffu, v, 4);
                v += __shfl_xor_sync(0xffffffffu, v, 8);
                v += __shfl_xor_sync(0xffffffffu, v, 16);
                if (g == 0) {
                    mrg_m[warp][nt * 8 + 2 * t4 + e] = ref[nt][e];
                    mrg_l[warp][nt * 8 + 2 * t4 + e] = v;
                }
#pragma unroll
                for (int gg = 0; gg < NG; ++gg) {
                    // the codes' offset: 8 P s, in the accumulators' unit of 2^-24
                    const float c8 = 4.76837158203125e-7f * off[nt][gg / 2][e + 2 * (gg & 1)];
                    const float* a0 = o[nt][2 * gg];
                    const float* a1 = o[nt][2 * gg + 1];
                    *reinterpret_cast<float4*>(ob + (nt * 8 + 2 * t4 + e) * OLD + gg * kGrp + g * 4) = make_float4(
                        a0[e] - c8, fmaf(a0[e + 2] - a0[e], 0.0625f, -c8), a1[e] - c8, fmaf(a1[e + 2] - a1[e], 0.0625f, -c8));
                }
            }
        }
        __syncthreads();
        if (threadIdx.x < 8 * NT) {
            const int h = threadIdx.x;
            float M = -INFINITY, sum = 0.f;
            for (int w = 0; w < W; ++w) M = fmaxf(M, mrg_m[w][h]);
            for (int w = 0; w < W; ++w) {
                const float f = mrg_m[w][h] == -INFINITY ? 0.f : exp2f(mrg_m[w][h] - M);
                mrg_s[w][h] = f;
                // a warp without granules, or whose logits were all NaN, has no reference
                sum += mrg_m[w][h] == -INFINITY ? mrg_l[w][h] : mrg_l[w][h] * f;
            }
            tot_m[h] = M;
            tot_l[h] = sum;
        }
        __syncthreads();
        const bool whole = SOLO || (s_lo == p0 && s_hi == p1);
        float* pb = a.part + ((long long)blockIdx.x * 2 + (s_lo > p0 ? 0 : 1)) * G * (D + 2);
        for (int v = threadIdx.x; v < G * (D / 4); v += 32 * W) {
            const int h = v / (D / 4), dd = v % (D / 4) * 4;
            float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
            for (int w = 0; w < W; ++w) {
                const float f = mrg_s[w][h];
                const float4 u = *reinterpret_cast<const float4*>(smem + w * (kStages * St::BYTES) + (h * OLD + dd) * 4);
                t.x = fmaf(u.x, f, t.x); t.y = fmaf(u.y, f, t.y); t.z = fmaf(u.z, f, t.z); t.w = fmaf(u.w, f, t.w);
            }
            if (whole) {
                const float inv = out_scale / tot_l[h];
                uint2 res;
                res.x = pack_bf16(t.x * inv, t.y * inv);
                res.y = pack_bf16(t.z * inv, t.w * inv);
                *reinterpret_cast<uint2*>(a.O + ((long long)b * s.hq + r * G + h) * D + dd) = res;
            } else {
                float* row = pb + h * (D + 2) + dd;   // rows of D + 2 floats: 8-byte aligned
                *reinterpret_cast<float2*>(row) = make_float2(t.x, t.y);
                *reinterpret_cast<float2*>(row + 2) = make_float2(t.z, t.w);
            }
        }
        if (!SOLO && threadIdx.x == 0) {
            if (s_lo == p0) a.span[x].x = blockIdx.x;
            if (s_hi == p1) a.span[x].y = blockIdx.x;
        }
        if (!whole && threadIdx.x < G) {
            pb[threadIdx.x * (D + 2) + D] = tot_m[threadIdx.x];
            pb[threadIdx.x * (D + 2) + D + 1] = tot_l[threadIdx.x];
        }
        __syncthreads();   // the rings and mrg_* are used again
    }
}

// Pairs that span blocks (and zeros for empty sequences): kMergeY groups of D threads (one per column)
// take the pieces in turn, each with a running reference, and are then added in order.
constexpr int kMergeY = 4;

template <int D>
__global__ void __launch_bounds__(D * kMergeY) q4_merge_kernel(Shape s, Attend a, int vexp)
{
    __shared__ float acc[kMergeY][D], ms[kMergeY], ls[kMergeY];
    pdl_wait();
    const int x = blockIdx.x, G = s.g, col = threadIdx.x % D, y = threadIdx.x / D;
    const int2 sp = a.span[x];
    const int c0 = sp.x, n = sp.y - sp.x + 1;
    if (n == 1) return;   // finished in its block
    const int b = x / s.hkv, r = x % s.hkv;
    __nv_bfloat16* out = a.O + ((long long)b * s.hq + r * G) * D;
    const long long stride = (long long)G * (D + 2);
    for (int h = blockIdx.y; h < G; h += gridDim.y) {
        // piece j: the last one of block c0 (j = 0), the first one of block c0 + j
        const float* base = a.part + (long long)h * (D + 2);
        float M = -INFINITY, L = 0.f, t = 0.f;
        for (int j0 = y; j0 < n; j0 += 4 * kMergeY) {
            float m[4], l[4], v[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int j = j0 + u * kMergeY;
                const float* p = base + ((long long)(c0 + j) * 2 + (j == 0 ? 1 : 0)) * stride;
                m[u] = j < n ? p[D] : -INFINITY;
                l[u] = j < n ? p[D + 1] : 0.f;
                v[u] = j < n ? p[col] : 0.f;
            }
            float top = M;
#pragma unroll
            for (int u = 0; u < 4; ++u) top = fmaxf(top, m[u]);
            const float f = M == -INFINITY ? 1.f : exp2f(M - top);   // nothing but NaNs so far: they stay
            L *= f;
            t *= f;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const float w = m[u] == -INFINITY ? 1.f : exp2f(m[u] - top);   // no reference: zeros or NaNs
                L = fmaf(l[u], w, L);
                t = fmaf(v[u], w, t);
            }
            M = top;
        }
        acc[y][col] = t;
        if (col == 0) { ms[y] = M; ls[y] = L; }
        __syncthreads();
        if (y == 0) {
            float top = M;
#pragma unroll
            for (int k = 1; k < kMergeY; ++k) top = fmaxf(top, ms[k]);
            float sum = 0.f;
            t = 0.f;
#pragma unroll
            for (int k = 0; k < kMergeY; ++k) {
                const float w = ms[k] == -INFINITY ? 1.f : exp2f(ms[k] - top);
                sum = fmaf(ls[k], w, sum);
                t = fmaf(acc[k][col], w, t);
            }
            out[h * D + col] = __float2bfloat16_rn(n ? t * exp2i(24 + vexp) / sum : 0.f);
        }
        __syncthreads();
    }
}

}  // namespace

// Short caches: a block per pair, which routes and attends in one launch.  A round of a block's warps takes 0.6 (D =
// 64) to 1.1 us, the merge and its launch 2 to 3, and the other blocks could have shared the rounds.  Dense, D = 64,
// 6 pairs: 500 tokens 7.9 -> 5.6 us a call, 1000 8.5 -> 6.9, but 2000 8.8 -> 9.3; D = 128, 6 pairs: 1000 9.6 ->
// 9.0, but 2000 9.9 -> 13.2; 192 pairs: 2000 25.8 -> 20.3.  Routed calls save the routing's launches too, and walk
// some of the chunks: D = 64, 6 pairs: 2000 tokens 13.2 -> 8.4, 3500 13.7 -> 9.2; D = 128: 1750 14.5 -> 10.1, but with
// 16 heads (rounds a quarter longer) 17.2 -> 19.5.  The limit of 16 bounds what lengths that differ can cost, and the
// chunks: 4096 tokens in chunks of 32 or more, 2048 in chunks of 16.
bool q4_solo(const Shape& s, bool routed)
{
    static_assert(Cfg<1>::W == 8 && Cfg<2>::W == 8 && kSoloWords * 32 >= 16 * 8 * 32 / 32 && kSoloWords * 32 >= 16 * 8 * 16 / 16,
                  "the routing of a block takes all chunks");
    const long long round = 8 * (s.B % 32 == 0 ? 32 : 16), rounds = (s.n + round - 1) / round;
    const long long cost = rounds * (s.d / 64) + (s.g > 8 ? rounds * (s.d / 64) / 4 : 0);
    const int pairs = s.batch * s.hkv, blocks = (s.g <= 8 ? Cfg<1>::BLOCKS : Cfg<2>::BLOCKS) * dec_tma_blocks();
    return pairs <= blocks && cost <= 16 && (routed || cost * (blocks - pairs) <= 7 * blocks);
}

namespace {

template <int D, int NT, int U, bool SOLO>
cudaError_t attend_k(const Shape& s, const Q4& c, const Routes& rt, const Attend& a, int blocks, cudaStream_t st)
{
    auto k = q4_attend_kernel<D, NT, U, SOLO>;
    const size_t smem = (size_t)Cfg<NT>::W * (Stage<D, U>::N * Stage<D, U>::BYTES + sizeof(Meta));
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    return e != cudaSuccess ? e : launch_after(k, dim3(blocks), dim3(32 * Cfg<NT>::W), smem, st, s, c, rt, a);
}

template <int D, int NT, int U>
cudaError_t attend_t(const Shape& s, const Q4& c, const Routes& rt, const Attend& a, cudaStream_t st)
{
    const int pairs = s.batch * s.hkv, blocks = Cfg<NT>::BLOCKS * dec_tma_blocks();
    if (q4_solo(s, !a.dense)) return attend_k<D, NT, U, true>(s, c, rt, a, pairs, st);
    const cudaError_t e = attend_k<D, NT, U, false>(s, c, rt, a, blocks, st);
    if (e != cudaSuccess) return e;
    return launch_after(q4_merge_kernel<D>, dim3(pairs, pairs * s.g <= 1024 ? s.g : 1), dim3(D * kMergeY), 0, st, s, a, c.vexp);
}

template <int D>
cudaError_t attend_d(const Shape& s, const Q4& c, const Routes& rt, const Attend& a, cudaStream_t st)
{
    if (s.B % 32 == 0) return s.g <= 8 ? attend_t<D, 1, 2>(s, c, rt, a, st) : attend_t<D, 2, 2>(s, c, rt, a, st);
    return s.g <= 8 ? attend_t<D, 1, 1>(s, c, rt, a, st) : attend_t<D, 2, 1>(s, c, rt, a, st);
}

}  // namespace

int q4_max_pairs() { return kMaxPairs; }

size_t q4_part_floats(const Shape& s) { return (size_t)2 * dec_tma_blocks() * 2 * s.g * (s.d + 2); }

cudaError_t launch_attend_q4(const Shape& s, const Q4& c, const void* q, const int* seqlens, const float* kbar,
                             const Routes& rt, bool dense, float* part, int* span, void* O, cudaStream_t st)
{
    const Attend a{(const __nv_bfloat16*)q, seqlens, dense ? 1 : 0, part, reinterpret_cast<int2*>(span), (__nv_bfloat16*)O,
                   kbar};
    return s.d == 128 ? attend_d<128>(s, c, rt, a, st) : attend_d<64>(s, c, rt, a, st);
}

}  // namespace dash
