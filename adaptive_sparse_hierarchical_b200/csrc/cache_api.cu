// cache_api.cu -- the entry points of include/dash_cache.h: argument checks, workspace layout and
// launch sequences.  No allocation, no synchronisation.
#include "pages.cuh"
#include "q4.cuh"

using namespace dash;

namespace dash {

cudaError_t launch_append_q4(const Shape& s, const Q4& c, const void* K, const void* V, int n_new, const int* counts,
                             const float* qbar, float* kbar, float* state, int* seqlens, cudaStream_t st);
cudaError_t launch_load_q4(const Shape& s, const Q4& c, const int* start, int offset, int n, const int* seqlens,
                           void* K, void* V, cudaStream_t st);
// kbar: the summaries, for caches whose blocks route their pairs themselves (q4_solo); else null
cudaError_t launch_attend_q4(const Shape& s, const Q4& c, const void* q, const int* seqlens, const float* kbar,
                             const Routes& rt, bool dense, float* part, int* span, void* O, cudaStream_t st);
bool q4_solo(const Shape& s, bool routed);
bool route_q4_supported(const Shape& s);
cudaError_t launch_route_q4(const Shape& s, const void* q, const float* kbar, const int* seqlens, const Routes& rt,
                            float* X, int* status, cudaStream_t st);
int q4_max_pairs();
size_t q4_part_floats(const Shape& s);

}  // namespace dash

namespace {

constexpr size_t kAlign = 256;
size_t up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }
bool on(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
int status_of(cudaError_t e) { return e == cudaSuccess ? DASH_OK : DASH_ELAUNCH; }

constexpr int kMaxGridYZ = 65535;
// Sizes of page and row arrays: the movers number 8 KB pieces of a page, and of a row's run, in 32 bits.
constexpr long long kMaxPageBytes = 1ll << 36, kMaxRunBytes = 1ll << 42;

int check_q4(const dash_params* p, const dash_q4_kv* kv)
{
    const int rc = check_params(p);
    if (rc != DASH_OK) return rc;
    if (!kv || !kv->k_codes || !kv->k_scales || !kv->v_codes || !kv->v_scales || !kv->page_table) return DASH_EINVAL;
    if (kv->page_size <= 0 || kv->max_pages <= 0 || kv->num_pages <= 0) return DASH_EINVAL;
    if (kv->k_exp < -32 || kv->k_exp > 32 || kv->v_exp < -32 || kv->v_exp > 32) return DASH_EINVAL;
    if ((long long)kv->max_pages * kv->page_size < p->seqlen) return DASH_EINVAL;
    if (p->dtype != DASH_BF16 || p->chunk == 1 || kv->page_size % p->chunk) return DASH_EUNSUPPORTED;
    if (p->h_kv > kMaxGridYZ || p->batch > kMaxGridYZ) return DASH_EUNSUPPORTED;
    const long long codes = (long long)p->h_kv * kv->page_size * p->d_h / 2, scales = codes / 16;
    if (kv->k_code_page < codes || kv->v_code_page < codes || kv->k_scale_page < scales || kv->v_scale_page < scales)
        return DASH_EINVAL;
    if ((kv->k_code_page | kv->v_code_page | kv->k_scale_page | kv->v_scale_page) % 16) return DASH_EALIGN;
    if (!on(kv->k_codes, 16) || !on(kv->v_codes, 16) || !on(kv->k_scales, 16) || !on(kv->v_scales, 16) ||
        !on(kv->page_table, 4))
        return DASH_EALIGN;
    return DASH_OK;
}

bool rows_ok(const long long st[3])
{
    for (int k = 0; k < 3; ++k)
        if (st[k] < 0 || (st[k] * 2) % 16) return false;
    return true;
}

// Whether the tokens and heads of an output [batch, n, h_kv, d] have places of their own.
bool apart(const dash_params* p, const long long st[3], int n)
{
    return (p->batch == 1 || st[0]) && (n == 1 || st[1]) && (p->h_kv == 1 || st[2]);
}

Shape shape_of(const dash_params* p)
{
    Shape s = {};
    s.batch = p->batch; s.n = p->seqlen; s.hq = p->h_q; s.hkv = p->h_kv; s.g = p->h_q / p->h_kv;
    s.d = p->d_h; s.B = p->chunk; s.T = p->seqlen / p->chunk;
    s.alpha = p->alpha; s.gamma = p->gamma; s.inv_sigma = p->inv_sigma;
    for (int k = 0; k < 3; ++k) { s.ks[k] = p->k_strides[k]; s.vs[k] = p->v_strides[k]; }
    return s;
}

Q4 cache_of(const dash_q4_kv* kv)
{
    Q4 c;
    c.kc = (uint8_t*)kv->k_codes; c.ks = (uint8_t*)kv->k_scales;
    c.vc = (uint8_t*)kv->v_codes; c.vs = (uint8_t*)kv->v_scales;
    c.kcp = kv->k_code_page; c.ksp = kv->k_scale_page; c.vcp = kv->v_code_page; c.vsp = kv->v_scale_page;
    c.pt = kv->page_table; c.pmax = kv->max_pages; c.psz = kv->page_size; c.npages = kv->num_pages;
    c.kexp = kv->k_exp; c.vexp = kv->v_exp;
    return c;
}

struct Q4Layout { size_t part, span, counts, idx, bias, x, err, total; };
Q4Layout q4_layout(const dash_params* p)
{
    Q4Layout L;
    const Shape s = shape_of(p);
    const size_t bh = (size_t)s.batch * s.hkv, T = s.T > 0 ? s.T : 1;
    L.part = 0;
    L.span = L.part + up(q4_part_floats(s) * 4);
    L.counts = L.span + up(bh * 8);
    L.idx = L.counts + up(bh * 4);
    L.bias = L.idx + up(bh * T * 4);
    L.x = L.bias + up(bh * T * 4);
    L.err = L.x + up(bh * s.g * T * 4);
    L.total = L.err + kAlign;
    return L;
}

int check_pages(const dash_pages* pg)
{
    if (!pg || pg->batch < 1 || pg->max_pages < 1 || pg->page_size < 1 || pg->num_pages < 1) return DASH_EINVAL;
    if (!pg->page_table || !pg->refs || !pg->seqlens) return DASH_EINVAL;
    if (!on(pg->page_table, 4) || !on(pg->refs, 4) || !on(pg->seqlens, 4)) return DASH_EALIGN;
    if ((long long)pg->max_pages * pg->page_size > 0x7fffffffll) return DASH_EINVAL;
    // the table's slots are numbered in 32 bits, its rows' parts are the y blocks of a launch
    if ((long long)pg->max_pages * pg->batch > 1ll << 30 || pg->max_pages > 1 << 25) return DASH_EUNSUPPORTED;
    if (pg->num_arrays < 0 || pg->num_rows < 0 || (pg->num_arrays && !pg->arrays) || (pg->num_rows && !pg->rows))
        return DASH_EINVAL;
    for (int i = 0; i < pg->num_arrays; ++i) {
        const dash_page_array& a = pg->arrays[i];
        if (!a.data || a.page_bytes < 0 || a.page_stride < a.page_bytes) return DASH_EINVAL;
        if (a.page_bytes > kMaxPageBytes) return DASH_EUNSUPPORTED;
        if (!on(a.data, 16) || a.page_bytes % 16 || a.page_stride % 16) return DASH_EALIGN;
    }
    for (int i = 0; i < pg->num_rows; ++i) {
        const dash_row_array& r = pg->rows[i];
        if (!r.data || r.unit_bytes < 0 || r.heads < 0 || r.max_units < 0 || r.unit_tokens < 0 ||
            r.row_stride < 0 || r.head_stride < 0 || r.clear < DASH_ROW_KEPT || r.clear > DASH_ROW_STATE)
            return DASH_EINVAL;
        if (r.unit_bytes > kMaxRunBytes / (r.max_units ? r.max_units : 1) ||
            r.head_stride > (1ll << 62) / (r.heads ? r.heads : 1) - kMaxRunBytes)
            return DASH_EUNSUPPORTED;
        if (!on(r.data, 4) || (r.unit_bytes | r.row_stride | r.head_stride) % 4) return DASH_EALIGN;
        // a row's runs must not reach into each other or into the next row
        const long long run = r.unit_bytes * r.max_units;
        if (r.heads > 1 && r.head_stride < run) return DASH_EINVAL;
        if (r.heads > 0 && pg->batch > 1 && r.row_stride < r.head_stride * (r.heads - 1) + run) return DASH_EINVAL;
    }
    return DASH_OK;
}

PageTab table_of(const dash_pages* pg)
{
    return PageTab{pg->batch, pg->max_pages, pg->page_size, pg->num_pages, pg->page_table, pg->refs, pg->seqlens};
}

int check_ws(const dash_pages* pg, void* ws, size_t bytes, PagesWs* w)
{
    if (!ws || bytes < pages_ws(table_of(pg), (char*)ws, w)) return DASH_EWORKSPACE;
    return on(ws, kAlign) ? DASH_OK : DASH_EALIGN;
}

}  // namespace

extern "C" {

size_t dash_q4_workspace_size(const dash_params* p)
{
    return check_params(p) == DASH_OK ? q4_layout(p).total : 0;
}

int dash_append_q4(const dash_params* p, const dash_q4_kv* kv, const void* K_new, const void* V_new, int n_new,
                   const int* counts, const float* qbar, float* kbar_cache, float* partial_state, int* seqlens,
                   void* stream)
{
    const int rc = check_q4(p, kv);
    if (rc != DASH_OK) return rc;
    if (n_new < 0 || (n_new && (!K_new || !V_new)) || !qbar || !partial_state || !seqlens) return DASH_EINVAL;
    if (!kbar_cache && p->seqlen >= p->chunk) return DASH_EINVAL;   // (shorter caches have no summaries)
    if (n_new > p->seqlen) n_new = p->seqlen;                       // the others would be dropped
    if (!on(K_new, 16) || !on(V_new, 16) || !rows_ok(p->k_strides) || !rows_ok(p->v_strides)) return DASH_EALIGN;
    if (!on(qbar, 4) || !on(kbar_cache, 4) || !on(partial_state, 4) || !on(seqlens, 4) || !on(counts, 4)) return DASH_EALIGN;
    if (n_new == 0) return DASH_OK;
    return status_of(launch_append_q4(shape_of(p), cache_of(kv), K_new, V_new, n_new, counts, qbar, kbar_cache,
                                      partial_state, seqlens, (cudaStream_t)stream));
}

int dash_load_q4(const dash_params* p, const dash_q4_kv* kv, const int* start, int offset, int n, const int* seqlens,
                 void* K, void* V, void* stream)
{
    const int rc = check_q4(p, kv);
    if (rc != DASH_OK) return rc;
    if (n < 0 || (n && (!K || !V)) || !seqlens) return DASH_EINVAL;
    if (!on(K, 16) || !on(V, 16) || !rows_ok(p->k_strides) || !rows_ok(p->v_strides)) return DASH_EALIGN;
    if (!on(start, 4) || !on(seqlens, 4)) return DASH_EALIGN;
    if (n == 0) return DASH_OK;
    if (n > 1 << 30) return DASH_EUNSUPPORTED;   // the blocks' rows are numbered in 32 bits, the last block's spare ones too
    if (!apart(p, p->k_strides, n) || !apart(p, p->v_strides, n)) return DASH_EINVAL;
    return status_of(launch_load_q4(shape_of(p), cache_of(kv), start, offset, n, seqlens, K, V, (cudaStream_t)stream));
}

int dash_decode_q4(const dash_params* p, const dash_q4_kv* kv, const void* q, const float* kbar_cache,
                   const int* seqlens, void* O, const dash_route_out* route, void* workspace, size_t ws_bytes,
                   void* stream)
{
    int rc = check_q4(p, kv);
    if (rc != DASH_OK) return rc;
    // a cache shorter than a chunk has nothing to route
    const bool none = p->seqlen < p->chunk, dense = p->gamma == 0.f || none, routed = !none && (!dense || route);
    if (!q || !seqlens || !O || (routed && !kbar_cache)) return DASH_EINVAL;
    if (!on(q, 16) || !on(O, 16) || !on(kbar_cache, 16) || !on(seqlens, 4)) return DASH_EALIGN;
    if ((long long)p->batch * p->h_kv > q4_max_pairs()) return DASH_EUNSUPPORTED;
    const Shape s = shape_of(p);
    // the pairs' granules (16 tokens or more), and what stands for a pair's start, are numbered in 32 bits
    if ((long long)p->batch * p->h_kv * (p->seqlen / 16 + 33ll) > 0x7fffffffll) return DASH_EUNSUPPORTED;
    if (routed && !route_q4_supported(s)) return DASH_EUNSUPPORTED;
    const Q4Layout L = q4_layout(p);
    if (!workspace || ws_bytes < L.total) return DASH_EWORKSPACE;
    if (!on(workspace, kAlign)) return DASH_EALIGN;
    char* ws = (char*)workspace;
    Routes rt = {};
    rt.counts = route && route->counts ? route->counts : (int*)(ws + L.counts);
    rt.idx = route && route->chunk_idx ? route->chunk_idx : (int*)(ws + L.idx);
    rt.bias = route && route->bias ? route->bias : (float*)(ws + L.bias);
    rt.bitmask = route ? route->bitmask : nullptr;
    rt.cap = s.T;
    rt.words = (s.T + 31) / 32;
    if (!on(rt.counts, 4) || !on(rt.idx, 4) || !on(rt.bias, 4) || !on(rt.bitmask, 4)) return DASH_EALIGN;
    const bool ahead = routed && !q4_solo(s, !dense);   // routing in launches of its own
    if (ahead) {
        float* X = (float*)(ws + L.x);
        int* err = (int*)(ws + L.err);
        rc = status_of(launch_route_q4(s, q, kbar_cache, seqlens, rt, X, err, (cudaStream_t)stream));
        if (rc != DASH_OK) return rc;
    }
    if (none && route) {
        const size_t bh = (size_t)p->batch * p->h_kv;
        if ((rc = status_of(cudaMemsetAsync(rt.counts, 0, bh * 4, (cudaStream_t)stream))) != DASH_OK) return rc;
    }
    return status_of(launch_attend_q4(s, cache_of(kv), q, seqlens, routed && !ahead ? kbar_cache : nullptr, rt, dense,
                                      (float*)(ws + L.part), (int*)(ws + L.span), O, (cudaStream_t)stream));
}

size_t dash_pages_workspace_size(const dash_pages* pg)
{
    if (check_pages(pg) != DASH_OK) return 0;
    PagesWs w;
    return pages_ws(table_of(pg), nullptr, &w);
}

int dash_pages_copy(const dash_pages* pg, const int* src, const int* dst, int n, int* status, void* workspace,
                    size_t ws_bytes, void* stream)
{
    int rc = check_pages(pg);
    if (rc != DASH_OK) return rc;
    if (n < 0 || n > pg->num_pages || (n && (!src || !dst))) return DASH_EINVAL;
    if (!on(src, 4) || !on(dst, 4) || !on(status, 4)) return DASH_EALIGN;
    PagesWs w;
    if ((rc = check_ws(pg, workspace, ws_bytes, &w)) != DASH_OK) return rc;
    if (n == 0) return DASH_OK;
    return status_of(launch_pages_copy(table_of(pg), pg, src, dst, n, status, w, (cudaStream_t)stream));
}

int dash_pages_reserve(const dash_pages* pg, const int* counts, int count, int* status, void* workspace,
                       size_t ws_bytes, void* stream)
{
    int rc = check_pages(pg);
    if (rc != DASH_OK) return rc;
    if (!on(counts, 4) || !on(status, 4)) return DASH_EALIGN;
    PagesWs w;
    if ((rc = check_ws(pg, workspace, ws_bytes, &w)) != DASH_OK) return rc;
    return status_of(launch_pages_reserve(table_of(pg), counts, count, status, w, (cudaStream_t)stream));
}

int dash_pages_fork(const dash_pages* pg, const int* src, const int* dst, int n, int* status, void* workspace,
                    size_t ws_bytes, void* stream)
{
    int rc = check_pages(pg);
    if (rc != DASH_OK) return rc;
    if (n < 0 || n > pg->batch || (n && (!src || !dst))) return DASH_EINVAL;
    if (n > pages_max_fork()) return DASH_EUNSUPPORTED;
    if (!on(src, 4) || !on(dst, 4) || !on(status, 4)) return DASH_EALIGN;
    PagesWs w;
    if ((rc = check_ws(pg, workspace, ws_bytes, &w)) != DASH_OK) return rc;
    if (n == 0) return DASH_OK;
    return status_of(launch_pages_fork(table_of(pg), pg, src, dst, n, status, w, (cudaStream_t)stream));
}

int dash_pages_free(const dash_pages* pg, const int* rows, int n, int* status, void* stream)
{
    const int rc = check_pages(pg);
    if (rc != DASH_OK) return rc;
    if (n < 0 || (n && !rows)) return DASH_EINVAL;
    if (!on(rows, 4) || !on(status, 4)) return DASH_EALIGN;
    if (n == 0) return DASH_OK;
    return status_of(launch_pages_free(table_of(pg), pg, rows, n, status, (cudaStream_t)stream));
}

int dash_pages_compact(const dash_pages* pg, int* used, void* workspace, size_t ws_bytes, void* stream)
{
    int rc = check_pages(pg);
    if (rc != DASH_OK) return rc;
    if (!on(used, 4)) return DASH_EALIGN;
    PagesWs w;
    if ((rc = check_ws(pg, workspace, ws_bytes, &w)) != DASH_OK) return rc;
    return status_of(launch_pages_compact(table_of(pg), pg, used, w, (cudaStream_t)stream));
}

}  // extern "C"
