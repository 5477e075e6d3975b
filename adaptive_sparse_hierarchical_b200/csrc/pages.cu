// pages.cu -- operations on the pages of a cache (include/dash_cache.h): copy, reserve, fork, free,
// compact.
//
// Each operation that moves data is two launches.  A plan (one block: the lists are short and the
// results must not depend on timing) checks the request, picks pages in ascending order with block
// scans over the reference counts, and leaves a list of (source, destination) pages in the
// workspace; the mover spreads the list's bytes over the whole GPU.  A request that fails its
// checks leaves an empty list, so nothing changes.  The mover is bound by HBM (2 bytes moved per
// byte of a page); small requests by the two launches, which overlap (programmatic dependent
// launch).  A copy of at most kFew pages needs no plan: every mover block checks the list itself.
//
// Measured: 1111 pages of 65.5 KB in each of 8 pools, 1.16 GB read and written: 188 us, 6.2 TB/s (a copy kernel
// reaches 6.5).  Compaction of 8192 pages, half of them in use (537 MB): 98.7 us, of which the plan is 8.  Pools of 4
// bits have pages of 16 KB (codes) and 1 KB (scales), less than a piece: 2.9 to 3.3 TB/s.  32 children of 8 rows of 32K
// tokens (84 MB): 26 us.  Three pages: 5.9 us, the call itself.  The plans are one
// block's work: reserving 131072 tokens for each of 64 rows (65536 slots) takes 0.32 ms, freeing them (a block
// per row) 18 us; a decode step's reserve finds its few slots in one step of the block.
#include "q4.cuh"
#include "pages.cuh"

namespace dash {
namespace {

constexpr int kPlan = 1024;             // threads of a plan block
constexpr int kMove = 256;              // threads of a mover block
// A mover block takes pieces of VEC 16-byte vectors per thread, all of them in flight before the first
// store: 8 (32 KB) reach 6.1 TB/s of pages moved where 2 reach 5.4 (1.16 GB); requests of less than
// two such pieces per SM are spread thinner, in pieces of 8 KB.
constexpr long long kPiece = 16ll * kMove;
constexpr int kSlots = 1024;            // table entries it takes at a time
constexpr int kFew = 256;               // a list short enough for every block to check
constexpr int kHeld = 16;               // table entries of a fork's destination that a lane looks at per step
constexpr int kMarks = 4096;            // rows whose marks fit a plan's shared memory

// Workspace header, then the lists (see PagesWs).
struct Plan {
    int pairs;      // pages to copy
    int ok;         // the request passed its checks (rows and tables may change)
    int used;       // compaction: pages in use
    int pad;
};

__device__ __forceinline__ void fail(int* status, int code)
{
    if (status) atomicCAS(status, 0, code);
}

// The lowest failure code that any thread of the plan block has in its mask (bit = code), stored;
// 0 if there is none.  Called by the whole block.
__device__ int first_failure(unsigned mask, int* status)
{
    __shared__ unsigned all;
    if (threadIdx.x == 0) all = 0;
    __syncthreads();
    if (mask) atomicOr(&all, mask);
    __syncthreads();
    const int code = all ? __ffs(all) - 1 : 0;
    if (code && threadIdx.x == 0) fail(status, code);
    __syncthreads();
    return code;
}

// Exclusive prefix of v over the block's threads in order; *total = the block's sum.
__device__ int block_scan(int v, int* total)
{
    __shared__ int ws[kPlan / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += u;
    }
    if (lane == 31) ws[warp] = x;
    __syncthreads();
    if (warp == 0) {
        int y = ws[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, y, o);
            if (lane >= o) y += u;
        }
        ws[lane] = y;
    }
    __syncthreads();
    const int before = warp ? ws[warp - 1] : 0;
    *total = ws[kPlan / 32 - 1];
    __syncthreads();
    return before + x - v;
}

constexpr int kPer = 8;   // pages a thread looks at per step

// Bit k: page p0 + kPer * thread + k is free.
__device__ __forceinline__ unsigned free_mask(const int* refs, int pages, int p0)
{
    const int p = p0 + threadIdx.x * kPer;
    unsigned m = 0;
#pragma unroll
    for (int k = 0; k < kPer; ++k)
        if (p + k < pages && refs[p + k] == 0) m |= 1u << k;
    return m;
}

// The `want` lowest pages with refs == 0, ascending, into list; returns how many there are (at most
// want).  Called by the whole plan block; first = free_mask of the first step, loaded ahead.
__device__ int lowest_free(const int* refs, int pages, int want, int* list, unsigned first)
{
    int found = 0;
    for (int p0 = 0; p0 < pages && found < want; p0 += kPlan * kPer) {
        unsigned m = p0 ? free_mask(refs, pages, p0) : first;
        int total;
        int at = found + block_scan(__popc(m), &total);
        for (; m; m &= m - 1, ++at)
            if (at < want) list[at] = p0 + threadIdx.x * kPer + __ffs(m) - 1;
        found += total;
    }
    __syncthreads();
    return min(found, want);
}

// ---- plans ------------------------------------------------------------------------------------------
// copy: destinations distinct and not sources.  mark[page] = the entry that writes it; a stale or
// foreign mark is recognised by looking the entry up, so the marks need no clearing.
__global__ void __launch_bounds__(kPlan) plan_copy_kernel(PageTab t, const int* src, const int* dst, int n, int* status,
                                                          PagesWs w)
{
    pdl_wait();
    pdl_launch_dependents();
    Plan* plan = reinterpret_cast<Plan*>(w.head);
    unsigned bad = 0;
    for (int i = threadIdx.x; i < n; i += kPlan) {
        const int s = src[i], d = dst[i];
        if (s < 0 || s >= t.num_pages || d < 0 || d >= t.num_pages) bad |= 1u << DASH_PAGES_INDEX;
        else w.mark[d] = i;
    }
    int code = first_failure(bad, status);
    if (!code) {
        for (int i = threadIdx.x; i < n; i += kPlan) {
            const int s = src[i], d = dst[i], k = w.mark[s];
            if (w.mark[d] != i) bad |= 1u << DASH_PAGES_TWICE;
            // a page that some entry writes is read: only fine where that entry copies it onto itself
            if (k >= 0 && k < n && dst[k] == s && src[k] != s) bad |= 1u << DASH_PAGES_TWICE;
            w.src[i] = s;
            w.dst[i] = d;
        }
        code = first_failure(bad, status);
    }
    if (threadIdx.x == 0) { plan->pairs = code ? 0 : n; plan->ok = !code; }
}

// reserve: the slots that the rows are to have (from the one that holds the next token on) form one list,
// in the order of rows and slots; those without a page get the lowest free pages, if there are enough.
__global__ void __launch_bounds__(kPlan) reserve_kernel(PageTab t, const int* counts, int count, int* status, PagesWs w)
{
    __shared__ int ends[kMarks], begins[kMarks];
    pdl_wait();
    pdl_launch_dependents();
    const unsigned first = free_mask(t.refs, t.num_pages, 0);
    // slots of the rows up to and including b; the first of them in b's table row
    int *end = t.batch <= kMarks ? ends : w.row, *begin = t.batch <= kMarks ? begins : w.own;
    unsigned bad = 0;
    int width = 0;
    for (int b0 = 0; b0 < t.batch; b0 += kPlan) {
        const int b = b0 + threadIdx.x, add = b < t.batch ? (counts ? counts[b] : count) : 0;
        int n = 0, from = 0, total;
        if (add > 0) {
            const int L = t.seqlens[b];
            const long long to = (long long)L + add;
            if (L < 0 || to > (long long)t.max_pages * t.page_size) bad |= 1u << DASH_PAGES_LENGTH;
            else {
                from = L / t.page_size;
                n = (int)((to + t.page_size - 1) / t.page_size) - from;
            }
        }
        const int at = block_scan(n, &total);
        if (b < t.batch) {
            end[b] = width + at + n;
            begin[b] = from;
        }
        width += total;
    }
    if (first_failure(bad, status)) return;   // (a barrier: `end` is there)
    // one slot per thread where they are enough, else kPer consecutive ones per thread and step
    const int per = width <= kPlan ? 1 : kPer;
    int* at[kPer];   // the table entries behind this thread's slots
    auto lacking = [&](int i0) {   // bit k: slot k of this thread has no page
        const int i = i0 + (int)threadIdx.x * per;
        if (i >= width) return 0u;
        int l = 0, h = t.batch - 1;   // the row with end[l - 1] <= i < end[l]
        while (l < h) {
            const int m = (l + h) >> 1;
            if (end[m] <= i) l = m + 1;
            else h = m;
        }
        int* e = t.page_table + (long long)l * t.max_pages + begin[l] + (i - (l ? end[l - 1] : 0));
        at[0] = e;
        if (per == 1) return *e < 0 ? 1u : 0u;
#pragma unroll
        for (int k = 1; k < kPer; ++k) {
            ++e;
            if (i + k < width && i + k == end[l]) {   // on to the next row with slots
                do ++l;
                while (end[l] <= i + k);
                e = t.page_table + (long long)l * t.max_pages + begin[l];
            }
            at[k] = e;
        }
        int v[kPer];
#pragma unroll
        for (int k = 0; k < kPer; ++k) v[k] = *(i + k < width ? at[k] : at[0]);
        unsigned m = 0;
#pragma unroll
        for (int k = 0; k < kPer; ++k)
            if (i + k < width && v[k] < 0) m |= 1u << k;
        return m;
    };
    const unsigned m0 = lacking(0);
    int want;
    block_scan(__popc(m0), &want);
    for (int i0 = kPlan * per; i0 < width; i0 += kPlan * per) {
        int total;
        block_scan(__popc(lacking(i0)), &total);
        want += total;
    }
    if (want == 0) return;
    if (want > t.num_pages || lowest_free(t.refs, t.num_pages, want, w.dst, first) < want) {
        if (threadIdx.x == 0) fail(status, DASH_PAGES_FULL);
        return;
    }
    int done = 0;
    for (int i0 = 0; i0 < width; i0 += kPlan * per) {
        // (with several steps `at` is another step's by now)
        const unsigned m = width <= kPlan * per ? m0 : lacking(i0);
        int total;
        int j = done + block_scan(__popc(m), &total);
#pragma unroll
        for (int k = 0; k < kPer; ++k)
            if (m >> k & 1) {
                const int pg = w.dst[j++];
                *at[k] = pg;
                t.refs[pg] = 1;
            }
        done += total;
    }
}

// fork: checks, a page for every child whose parent ends inside one.  Leaves the parent's length
// (w.row) and the child's own page (w.own, -1) per entry: the mover writes tables and lengths.  One
// thread per entry (n <= kPlan).
__global__ void __launch_bounds__(kPlan) plan_fork_kernel(PageTab t, const int* src, const int* dst, int n, int* status,
                                                          PagesWs w)
{
    __shared__ int marks[kMarks], fresh[kPlan];
    pdl_wait();
    pdl_launch_dependents();
    Plan* plan = reinterpret_cast<Plan*>(w.head);
    // the entry that writes a row; rows without one hold anything, which the look-up below recognises
    int* mark = t.batch <= kMarks ? marks : w.mark;
    const int i = threadIdx.x;
    const bool on = i < n;
    const int s = on ? src[i] : 0, d = on ? dst[i] : 0;
    const unsigned first = free_mask(t.refs, t.num_pages, 0);
    const bool inside = s >= 0 && s < t.batch && d >= 0 && d < t.batch;
    unsigned bad = 0;
    int L = 0;
    if (on && !inside) bad |= 1u << DASH_PAGES_INDEX;
    if (on && inside) {
        mark[d] = i;
        L = t.seqlens[s];
        if (L < 0 || L > (long long)t.max_pages * t.page_size) bad |= 1u << DASH_PAGES_LENGTH;
        else if (t.seqlens[d] != 0) bad |= 1u << DASH_PAGES_BUSY;
    }
    // no slot of a destination may hold a page: a warp per entry, kHeld slots of a lane on their way at a time
    for (int j = threadIdx.x >> 5; j < n; j += kPlan / 32) {
        const int to = dst[j];
        if (to < 0 || to >= t.batch) continue;
        const int* row = t.page_table + (long long)to * t.max_pages;
        int top = -1;
        for (int s0 = threadIdx.x & 31; s0 < t.max_pages; s0 += 32 * kHeld) {
            int e[kHeld];
#pragma unroll
            for (int k = 0; k < kHeld; ++k) e[k] = s0 + 32 * k < t.max_pages ? row[s0 + 32 * k] : -1;
#pragma unroll
            for (int k = 0; k < kHeld; ++k) top = max(top, e[k]);
        }
        if (top >= 0) bad |= 1u << DASH_PAGES_BUSY;
    }
    int code = first_failure(bad, status), want = 0, at = 0, part = 0;
    if (!code) {
        int pg = -1;
        if (on) {
            const int k = mark[s];
            if (mark[d] != i || (k >= 0 && k < n && dst[k] == s)) bad |= 1u << DASH_PAGES_TWICE;
            part = L % t.page_size != 0;
            if (part) {
                pg = t.page_table[(long long)s * t.max_pages + L / t.page_size];
                if (pg < 0 || pg >= t.num_pages) bad |= 1u << DASH_PAGES_INDEX;
            }
        }
        at = block_scan(part, &want);
        if (part) w.src[at] = pg;
        code = first_failure(bad, status);
    }
    if (!code && want && (want > t.num_pages || lowest_free(t.refs, t.num_pages, want, fresh, first) < want))
        code = first_failure(1u << DASH_PAGES_FULL, status);
    if (!code && on) {
        w.row[i] = L;
        w.own[i] = part ? fresh[at] : -1;
        if (part) {
            w.dst[at] = fresh[at];
            t.refs[fresh[at]] = 1;
        }
    }
    if (i == 0) { plan->pairs = code ? 0 : want; plan->ok = !code; }
}

// compact: U = pages in use; the k-th free page below U receives the k-th used page from U on.
__global__ void __launch_bounds__(kPlan) plan_compact_kernel(PageTab t, int* used, PagesWs w)
{
    pdl_wait();
    pdl_launch_dependents();
    Plan* plan = reinterpret_cast<Plan*>(w.head);
    const unsigned first = free_mask(t.refs, t.num_pages, 0);   // of the first step's pages
    const int here = max(0, min(kPer, t.num_pages - (int)threadIdx.x * kPer));
    int U = here - __popc(first);
    for (int p = kPlan * kPer + threadIdx.x; p < t.num_pages; p += kPlan) U += t.refs[p] != 0;
    {
        int total;
        block_scan(U, &total);
        U = total;
    }
    int holes = 0, movers = 0;
    for (int p0 = 0; p0 < t.num_pages; p0 += kPlan * kPer) {
        const int p = p0 + threadIdx.x * kPer;
        const unsigned none = p0 ? free_mask(t.refs, t.num_pages, p0) : first;
        unsigned h = 0, m = 0;
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            if (p + k >= t.num_pages) continue;
            const bool on = !(none >> k & 1);
            if (p + k < U && !on) h |= 1u << k;
            if (p + k >= U && on) m |= 1u << k;
            if (p + k >= U && !on) w.mark[p + k] = p + k;   // table entries of pages without a count stay
        }
        int total;   // both counts in one scan: at most 8192 of each per step
        const int at = block_scan(__popc(h) | __popc(m) << 16, &total);
        int a = holes + (at & 0xffff), c = movers + (at >> 16);
        for (; h; h &= h - 1) w.dst[a++] = p + __ffs(h) - 1;
        for (; m; m &= m - 1) w.src[c++] = p + __ffs(m) - 1;
        holes += total & 0xffff;
        movers += total >> 16;
    }
    __syncthreads();
    for (int k = threadIdx.x; k < movers; k += kPlan) {
        const int s = w.src[k], d = w.dst[k];
        w.mark[s] = d;
        t.refs[d] = t.refs[s];
        t.refs[s] = 0;
    }
    if (threadIdx.x == 0) {
        plan->pairs = movers;
        plan->ok = 1;
        plan->used = U;
        if (used) *used = U;
    }
}

// ---- mover --------------------------------------------------------------------------------------------
// Work of one launch, taken unit by unit: first the listed pages of up to CAP arrays (pieces of
// SEG bytes), then, for a fork, the rows of up to CAP row arrays, then the tables.
enum { MOVE_PAGES = 0, MOVE_FORK = 1, MOVE_COMPACT = 2 };

template <int CAP, int VEC>
struct Move {
    static constexpr long long SEG = VEC * kPiece;
    MoveArray pages[CAP];
    MoveRows rows[CAP];
    int np, nr, segs;               // arrays, row arrays, pieces per page over all arrays
    long long row_units;            // pieces per forked row over all row arrays
    int op, n;                      // fork: entries
    const int *src, *dst;           // fork: the row lists
    int tables;                     // this launch writes the tables
};

template <int VEC>
__device__ __forceinline__ void copy_bytes(char* dst, const char* src, long long bytes, bool wide)
{
    if (wide) {
        const int n = (int)(bytes >> 4);
        const uint4* s = reinterpret_cast<const uint4*>(src);
        uint4* d = reinterpret_cast<uint4*>(dst);
        uint4 v[VEC];
#pragma unroll
        for (int k = 0; k < VEC; ++k)
            if ((int)threadIdx.x + k * kMove < n) v[k] = __ldcs(s + threadIdx.x + k * kMove);
#pragma unroll
        for (int k = 0; k < VEC; ++k)
            if ((int)threadIdx.x + k * kMove < n) __stcs(d + threadIdx.x + k * kMove, v[k]);
    } else {
        const int n = (int)(bytes >> 2);
        for (int i = threadIdx.x; i < n; i += kMove)
            reinterpret_cast<uint32_t*>(dst)[i] = reinterpret_cast<const uint32_t*>(src)[i];
    }
}

// Piece q of page `from` to page `to`.
template <int CAP, int VEC>
__device__ __forceinline__ void copy_piece(const Move<CAP, VEC>& mv, int from, int to, int q)
{
    int a = 0;
    while (q >= mv.pages[a].segs) q -= mv.pages[a++].segs;
    const MoveArray& m = mv.pages[a];
    const long long off = q * mv.SEG;
    copy_bytes<VEC>(m.data + (long long)to * m.stride + off, m.data + (long long)from * m.stride + off,
                    min(mv.SEG, m.bytes - off), true);
}

// Copy of n <= kFew pages: every block checks the whole list (the rules of plan_copy_kernel).
template <int CAP, int VEC>
__global__ void __launch_bounds__(kMove) copy_few_kernel(PageTab t, const int* src, const int* dst, int n, int* status,
                                                         const __grid_constant__ Move<CAP, VEC> mv)
{
    __shared__ int from[kFew], to[kFew];
    __shared__ unsigned all;
    pdl_wait();
    pdl_launch_dependents();
    const int i = threadIdx.x;
    static_assert(kFew <= kMove, "one thread per entry");
    if (i == 0) all = 0;
    if (i < n) { from[i] = src[i]; to[i] = dst[i]; }
    __syncthreads();
    if (i < n) {
        const int s = from[i], d = to[i];
        unsigned bad = s < 0 || s >= t.num_pages || d < 0 || d >= t.num_pages ? 1u << DASH_PAGES_INDEX : 0u;
        for (int k = 0; k < n; ++k)
            if ((k != i && to[k] == d) || (to[k] == s && from[k] != s)) bad |= 1u << DASH_PAGES_TWICE;
        if (bad) atomicOr(&all, bad);
    }
    __syncthreads();
    if (all) {
        if (blockIdx.x == 0 && i == 0) fail(status, __ffs(all) - 1);
        return;
    }
    for (long long u = blockIdx.x; u < (long long)n * mv.segs; u += gridDim.x)
        copy_piece(mv, from[u / mv.segs], to[u / mv.segs], (int)(u % mv.segs));
}

template <int CAP, int VEC>
__global__ void __launch_bounds__(kMove) move_kernel(PageTab t, PagesWs w, const __grid_constant__ Move<CAP, VEC> mv)
{
    pdl_wait();   // the plan
    pdl_launch_dependents();
    const Plan* plan = reinterpret_cast<const Plan*>(w.head);
    if (!plan->ok) return;
    const long long page_units = (long long)plan->pairs * mv.segs;
    const long long row_units = mv.op == MOVE_FORK ? mv.row_units * mv.n : 0;
    const int per_row = (t.max_pages + kSlots - 1) / kSlots;
    const long long tab_rows = !mv.tables ? 0 : mv.op == MOVE_FORK ? mv.n : t.batch;
    const long long total = page_units + row_units + tab_rows * per_row;
    for (long long u = blockIdx.x; u < total; u += gridDim.x) {
        if (u < page_units) {
            const int k = (int)(u / mv.segs);
            copy_piece(mv, w.src[k], w.dst[k], (int)(u % mv.segs));
        } else if (u < page_units + row_units) {
            const long long v = u - page_units;
            const int k = (int)(v / mv.row_units);
            long long q = v % mv.row_units;
            int a = 0;
            while (q >= (long long)mv.rows[a].heads * mv.rows[a].segs) {
                q -= (long long)mv.rows[a].heads * mv.rows[a].segs;
                ++a;
            }
            const MoveRows& m = mv.rows[a];
            const int h = (int)(q / m.segs);
            const long long off = q % m.segs * mv.SEG;
            const int in_use = m.unit_tokens > 0 ? min(m.max_units, w.row[k] / m.unit_tokens) : m.max_units;
            const long long left = in_use * m.unit_bytes - off;
            if (left > 0) {
                const long long at = h * m.head_stride + off;
                copy_bytes<VEC>(m.data + mv.dst[k] * m.row_stride + at, m.data + mv.src[k] * m.row_stride + at,
                           min(mv.SEG, left), m.wide);
            }
        } else {
            const long long v = u - page_units - row_units;
            const int k = (int)(v / per_row), s0 = (int)(v % per_row) * kSlots, s1 = min(t.max_pages, s0 + kSlots);
            if (mv.op == MOVE_FORK) {
                const int L = w.row[k], full = L / t.page_size, own = w.own[k];
                const int* from = t.page_table + (long long)mv.src[k] * t.max_pages;
                int* to = t.page_table + (long long)mv.dst[k] * t.max_pages;
                for (int s = s0 + threadIdx.x; s < s1; s += kMove) {
                    int e = -1;
                    if (s < full) {
                        e = from[s];
                        if (e >= 0 && e < t.num_pages) atomicAdd(t.refs + e, 1);
                    } else if (s == full) {
                        e = own;
                    }
                    to[s] = e;
                }
                if (s0 == 0 && threadIdx.x == 0) t.seqlens[mv.dst[k]] = L;
            } else {
                for (int s = s0 + threadIdx.x; s < s1; s += kMove) {
                    int* e = t.page_table + (long long)k * t.max_pages + s;
                    const int p = *e;
                    if (p >= plan->used && p < t.num_pages) *e = w.mark[p];
                }
            }
        }
    }
}

// free: one block per (entry, part of its row); of equal entries the first acts.
template <int CAP>
struct Clear {
    MoveRows rows[CAP];
    int n, tables;
};
template <int CAP>
__global__ void __launch_bounds__(kMove) free_kernel(PageTab t, const int* rows, int n, int* status,
                                                     const __grid_constant__ Clear<CAP> c)
{
    pdl_wait();
    pdl_launch_dependents();
    const int i = blockIdx.x, b = rows[i];
    if (b < 0 || b >= t.batch) {
        if (threadIdx.x == 0) fail(status, DASH_PAGES_INDEX);
        return;
    }
    bool again = false;
    for (int j = threadIdx.x; j < i; j += kMove) again = again || rows[j] == b;
    if (__syncthreads_or(again)) return;
    const int s0 = blockIdx.y * kSlots, s1 = min(t.max_pages, s0 + kSlots);
    if (s0 == 0)
        for (int a = 0; a < c.n; ++a) {
            const MoveRows& m = c.rows[a];
            const long long words = m.max_units * m.unit_bytes / 4;
            for (int h = 0; h < m.heads; ++h)
                for (long long k = threadIdx.x; k < words; k += kMove)
                    reinterpret_cast<uint32_t*>(m.data + b * m.row_stride + h * m.head_stride)[k] =
                        m.clear == DASH_ROW_STATE && k == words - 2 ? 0xff800000u : 0u;   // -inf
        }
    if (!c.tables) return;
    for (int s = s0 + threadIdx.x; s < s1; s += kMove) {
        int* e = t.page_table + (long long)b * t.max_pages + s;
        const int p = *e;
        *e = -1;
        if (p >= 0 && p < t.num_pages) atomicSub(t.refs + p, 1);
    }
    if (s0 == 0 && threadIdx.x == 0) t.seqlens[b] = 0;
}

MoveRows rows_of(const dash_row_array& p, long long seg)
{
    MoveRows m;
    m.data = (char*)p.data;
    m.row_stride = p.row_stride;
    m.head_stride = p.head_stride;
    m.unit_bytes = p.unit_bytes;
    m.heads = p.heads;
    m.max_units = p.max_units;
    m.unit_tokens = p.unit_tokens;
    m.clear = p.clear;
    m.segs = (int)((p.max_units * p.unit_bytes + seg - 1) / seg);
    m.wide = (reinterpret_cast<uintptr_t>(p.data) | (uintptr_t)p.row_stride | (uintptr_t)p.head_stride |
              (uintptr_t)p.unit_bytes) % 16 == 0;
    return m;
}

// Enough blocks for 8 per SM, or one per unit of a small request.
dim3 move_grid(long long units)
{
    const long long most = 8ll * dec_tma_blocks();
    return dim3((unsigned)(units < 1 ? 1 : units < most ? units : most));
}

// The mover's launches: the arrays in groups of CAP.
template <int CAP, int VEC>
cudaError_t move_groups(const PageTab& t, const PagesWs* w, const dash_pages* pg, int op, int n, const int* src,
                        const int* dst, int* status, long long most_pairs, cudaStream_t st)
{
    int a = 0, r = 0;
    bool first = true;
    const int nr = op == MOVE_FORK ? pg->num_rows : 0;
    while (first || a < pg->num_arrays || r < nr) {
        Move<CAP, VEC> mv = {};
        mv.op = op;
        mv.n = n;
        mv.src = src;
        mv.dst = dst;
        mv.tables = first && op != MOVE_PAGES;
        for (; a < pg->num_arrays && mv.np < CAP; ++a) {
            const dash_page_array& p = pg->arrays[a];
            if (p.page_bytes == 0) continue;
            MoveArray& m = mv.pages[mv.np++];
            m.data = (char*)p.data;
            m.bytes = p.page_bytes;
            m.stride = p.page_stride;
            m.segs = (int)((p.page_bytes + mv.SEG - 1) / mv.SEG);
            mv.segs += m.segs;
        }
        for (; r < nr && mv.nr < CAP; ++r) {
            const dash_row_array& p = pg->rows[r];
            if (p.unit_bytes == 0 || p.heads == 0 || p.max_units == 0) continue;
            const MoveRows& m = mv.rows[mv.nr++] = rows_of(p, mv.SEG);
            mv.row_units += (long long)m.heads * m.segs;
        }
        cudaError_t e;
        if (!w) {
            if (mv.segs == 0) break;
            e = launch_after(copy_few_kernel<CAP, VEC>, move_grid(most_pairs * mv.segs), dim3(kMove), 0, st, t, src, dst, n,
                             status, mv);
        } else {
            const long long tab = mv.tables ? (long long)(op == MOVE_FORK ? n : t.batch) * ((t.max_pages + kSlots - 1) / kSlots) : 0;
            e = launch_after(move_kernel<CAP, VEC>, move_grid(most_pairs * mv.segs + mv.row_units * n + tab), dim3(kMove), 0, st,
                             t, *w, mv);
        }
        if (e != cudaSuccess) return e;
        first = false;
    }
    return cudaSuccess;
}

// w: the plan's lists; null for a copy without a plan (src, dst are its lists).
cudaError_t launch_move(const PageTab& t, const PagesWs* w, const dash_pages* pg, int op, int n, const int* src,
                        const int* dst, int* status, long long most_pairs, cudaStream_t st)
{
    long long bytes = 0;
    for (int a = 0; a < pg->num_arrays; ++a) bytes += most_pairs * pg->arrays[a].page_bytes;
    for (int r = 0; r < (op == MOVE_FORK ? pg->num_rows : 0); ++r)
        bytes += (long long)n * pg->rows[r].heads * pg->rows[r].max_units * pg->rows[r].unit_bytes;
    const bool large = bytes >= 2 * 8 * kPiece * dec_tma_blocks();
    // few arrays travel in a small argument block: the launch is cheaper
    if (pg->num_arrays <= kFewArrays && pg->num_rows <= kFewArrays)
        return large ? move_groups<kFewArrays, 8>(t, w, pg, op, n, src, dst, status, most_pairs, st)
                     : move_groups<kFewArrays, 2>(t, w, pg, op, n, src, dst, status, most_pairs, st);
    return large ? move_groups<kArrays, 8>(t, w, pg, op, n, src, dst, status, most_pairs, st)
                 : move_groups<kArrays, 2>(t, w, pg, op, n, src, dst, status, most_pairs, st);
}

template <int CAP>
cudaError_t free_groups(const PageTab& t, const dash_pages* pg, const int* rows, int n, int* status, cudaStream_t st)
{
    int r = 0;
    for (bool first = true; first || r < pg->num_rows; first = false) {
        Clear<CAP> c = {};
        c.tables = first;
        for (; r < pg->num_rows && c.n < CAP; ++r)
            if (pg->rows[r].clear) c.rows[c.n++] = rows_of(pg->rows[r], kPiece);
        if (!first && c.n == 0) break;
        const cudaError_t e = launch_after(free_kernel<CAP>, dim3(n, first ? (t.max_pages + kSlots - 1) / kSlots : 1),
                                           dim3(kMove), 0, st, t, rows, n, status, c);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace

int pages_max_fork() { return kPlan; }

size_t pages_ws(const PageTab& t, char* base, PagesWs* w)
{
    size_t at = 256;
    auto take = [&](size_t ints) {
        int* p = reinterpret_cast<int*>(base + at);
        at += (ints * 4 + 255) / 256 * 256;
        return p;
    };
    const size_t big = t.num_pages > t.batch ? t.num_pages : t.batch;
    w->head = base;
    w->src = take(big);
    w->dst = take(big);
    w->mark = take(big);
    w->row = take(t.batch);
    w->own = take(t.batch);
    return at;
}

cudaError_t launch_pages_copy(const PageTab& t, const dash_pages* pg, const int* src, const int* dst, int n, int* status,
                              const PagesWs& w, cudaStream_t st)
{
    if (n <= kFew) return launch_move(t, nullptr, pg, MOVE_PAGES, n, src, dst, status, n, st);
    const cudaError_t e = launch_after(plan_copy_kernel, dim3(1), dim3(kPlan), 0, st, t, src, dst, n, status, w);
    return e != cudaSuccess ? e : launch_move(t, &w, pg, MOVE_PAGES, 0, nullptr, nullptr, nullptr, n, st);
}

cudaError_t launch_pages_reserve(const PageTab& t, const int* counts, int count, int* status, const PagesWs& w,
                                 cudaStream_t st)
{
    return launch_after(reserve_kernel, dim3(1), dim3(kPlan), 0, st, t, counts, count, status, w);
}

cudaError_t launch_pages_fork(const PageTab& t, const dash_pages* pg, const int* src, const int* dst, int n, int* status,
                              const PagesWs& w, cudaStream_t st)
{
    const cudaError_t e = launch_after(plan_fork_kernel, dim3(1), dim3(kPlan), 0, st, t, src, dst, n, status, w);
    return e != cudaSuccess ? e : launch_move(t, &w, pg, MOVE_FORK, n, src, dst, nullptr, n, st);
}

cudaError_t launch_pages_free(const PageTab& t, const dash_pages* pg, const int* rows, int n, int* status, cudaStream_t st)
{
    return pg->num_rows <= kFewArrays ? free_groups<kFewArrays>(t, pg, rows, n, status, st)
                                      : free_groups<kArrays>(t, pg, rows, n, status, st);
}

cudaError_t launch_pages_compact(const PageTab& t, const dash_pages* pg, int* used, const PagesWs& w, cudaStream_t st)
{
    const cudaError_t e = launch_after(plan_compact_kernel, dim3(1), dim3(kPlan), 0, st, t, used, w);
    return e != cudaSuccess ? e : launch_move(t, &w, pg, MOVE_COMPACT, 0, nullptr, nullptr, nullptr, t.num_pages / 2, st);
}

}  // namespace dash
