/*
 * dash_cache.h -- caches for serving: keys and values held in 4 bits on pages, and operations on
 * the pages of a cache.  Extends dash.h (same library, conventions and status codes): device
 * pointers, caller-owned buffers and workspaces, everything enqueued on `stream`, arguments
 * checked before any launch, no allocation, no synchronisation.
 */
#ifndef DASH_CACHE_H
#define DASH_CACHE_H

#include "dash.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- K/V caches in 4 bits -----------------------------------------------------------------------
 * Format.  The d_h elements of one (token, KV head) form groups of 32 consecutive elements.  A
 * group x holds one scale s = e4m3(max|x| 2^-e / 7) (round to nearest even, at most 448) and a
 * 4-bit code u = round(x 2^-e / s) + 8 per element (nearest even, clamped to 1..15; 8 where s is
 * 0); the code stands for (u - 8) s 2^e, which bf16 holds exactly.  e is the cache's k_exp /
 * v_exp (-32..32): it moves the range of the scales, 2^-9..448, to the data's.  A group with a NaN
 * or an infinity gets the scale NaN and stands for NaNs.  17/32 bytes per element in all.
 * Layout.  Token t of sequence b sits in page page_table[b * max_pages + t / page_size], row
 * t % page_size.  A page of a code pool is uint8 [h_kv][page_size][d_h / 2], of a scale pool uint8
 * [h_kv][page_size][d_h / 32]; pages lie *_page bytes apart.  A row of codes is d_h / 8 words of
 * 32 bits with element i of the word in bits 4i..4i+3.  A value row keeps its words in order; a
 * key row stores the j-th word of group G at place j * (d_h / 32) + G (the order in which the
 * decode kernel's tensor-core operands want them).
 * Requirements: bf16 tensors, d_h 64 or 128, chunk 16, 32, 64 or 128, page_size a multiple of the
 * chunk, max_pages * page_size >= p->seqlen; pools 16-byte aligned, page strides multiples of 16
 * bytes.  A page id outside [0, num_pages) is never dereferenced: tokens on such a page are not
 * stored, and read as zeros. */
typedef struct {
    void *k_codes, *k_scales, *v_codes, *v_scales;
    long long k_code_page, k_scale_page, v_code_page, v_scale_page; /* bytes between pages */
    const int* page_table;                                          /* device int32 [batch, max_pages] */
    int max_pages, page_size, num_pages;
    int k_exp, v_exp;
} dash_q4_kv;

/* Append tokens.  K_new, V_new [batch, n_new, h_kv, d_h] (bf16, element strides p->k_strides /
 * p->v_strides) hold up to n_new tokens per sequence, counts (device int32 [batch], NULL: n_new
 * for all; clamped to 0..n_new) how many of them are there.  Sequence b's tokens go to positions
 * L_b = seqlens[b] and on, in 4 bits; the summaries (Eq. 4) are taken from the bf16 keys: every
 * chunk they complete is written to kbar_cache, the chunk they leave open to partial_state (the
 * buffers of dash_summary_append; the state is not read while L_b is a multiple of the chunk).
 * seqlens[b] becomes L_b + counts[b].  Tokens beyond the capacity p->seqlen are dropped.  (Rows that share pages
 * share filled ones: a caller that sets seqlens[b] back below them would write what the other row reads.) */
int dash_append_q4(const dash_params* p, const dash_q4_kv* kv, const void* K_new, const void* V_new, int n_new,
                   const int* counts, const float* qbar, float* kbar_cache, float* partial_state, int* seqlens,
                   void* stream);

/* Read back: K, V [batch, n, h_kv, d_h] (bf16, strides p->k_strides / p->v_strides) receive
 * positions start_b .. start_b + n - 1 of every sequence, start_b = (start ? start[b] : 0) +
 * offset.  Positions outside 0..seqlens[b]-1 or on unmapped pages give zeros.  n <= 2^30. */
int dash_load_q4(const dash_params* p, const dash_q4_kv* kv, const int* start, int offset, int n, const int* seqlens,
                 void* K, void* V, void* stream);

/* dash_decode over a 4-bit cache: q, O [batch, h_q, d_h] (bf16, contiguous), the query of sequence
 * b at position seqlens[b] - 1.  gamma = 0 attends over every cached token (dense attention, bias
 * 0); kbar_cache may then be NULL unless `route` is given (and for every call on a cache that is shorter
 * than a chunk).  A sequence of length 0 gives zeros.  batch * h_kv <= 2048; query elements up to 2^88
 * (beyond, logits of about that size overflow).  A query that is not finite makes its head's output NaN; a chunk whose
 * summary is not finite is routed, and makes the outputs of its KV head's group NaN.  Workspace:
 * dash_q4_workspace_size(p), 256-byte aligned. */
size_t dash_q4_workspace_size(const dash_params* p);
int dash_decode_q4(const dash_params* p, const dash_q4_kv* kv, const void* q, const float* kbar_cache,
                   const int* seqlens, void* O, const dash_route_out* route, void* workspace, size_t ws_bytes,
                   void* stream);

/* ---- pages of a cache -----------------------------------------------------------------------------
 * A pool of num_pages pages shared by `batch` rows (sequences).  page_table [batch, max_pages]
 * (-1: no page), refs [num_pages] (how many table entries hold the page; 0: free) and seqlens
 * [batch] are device int32 and are changed on the stream.  `arrays` (host) lists everything that
 * a page id addresses: the K and V pools of every layer, code and scale pools of 4-bit caches;
 * `rows` (host) what a row number addresses: the summary caches and incomplete-chunk states.
 * Pages that a sequence has filled are never written again, so rows may share them.
 * The lowest-numbered free pages are given out first, in the order of rows and slots: results do
 * not depend on timing.  A call that cannot be carried out changes nothing but *status.
 * status (device int32, may be NULL) is left alone on success; the first failure stores its code:
 *   1 an index outside its range, or an unmapped page where one is needed
 *   2 a destination that occurs twice, or that is also a source
 *   3 a destination row that is not empty
 *   4 not enough free pages
 *   5 a length beyond the row's pages */
enum { DASH_PAGES_INDEX = 1, DASH_PAGES_TWICE = 2, DASH_PAGES_BUSY = 3, DASH_PAGES_FULL = 4, DASH_PAGES_LENGTH = 5 };

typedef struct {                       /* page i: page_bytes at data + i * page_stride (multiples of 16) */
    void* data;
    long long page_bytes, page_stride;
} dash_page_array;

/* Row i holds `heads` runs of up to max_units units of unit_bytes (a multiple of 4) each, run j at
 * data + i * row_stride + j * head_stride; a row of length L has floor(L / unit_tokens) of them in
 * use (all max_units where unit_tokens is 0).  clear says what freeing a row leaves in its runs:
 *   DASH_ROW_KEPT   what was there (summaries: never read beyond a row's length)
 *   DASH_ROW_ZERO   zeros (the lengths that further layers keep for themselves)
 *   DASH_ROW_STATE  the state of an empty chunk: each run is one d_h + 2 floats, zeros but for the
 *                   maximum in the last but one, -inf */
enum { DASH_ROW_KEPT = 0, DASH_ROW_ZERO = 1, DASH_ROW_STATE = 2 };
typedef struct {
    void* data;
    long long row_stride, head_stride, unit_bytes;
    int heads, max_units, unit_tokens, clear;
} dash_row_array;

typedef struct {
    int batch, max_pages, page_size, num_pages;
    int *page_table, *refs, *seqlens;
    const dash_page_array* arrays;
    const dash_row_array* rows;
    int num_arrays, num_rows;
} dash_pages;

size_t dash_pages_workspace_size(const dash_pages* pg);

/* Contents of page src[i] copied to page dst[i] for i < n (device int32 lists) in every array.
 * A source may occur several times.  Tables and counts are not touched. */
int dash_pages_copy(const dash_pages* pg, const int* src, const int* dst, int n, int* status, void* workspace,
                    size_t ws_bytes, void* stream);

/* Gives every row b the free pages it lacks for positions seqlens[b] .. seqlens[b] + add_b - 1, add_b =
 * counts ? counts[b] : count (rows with add_b <= 0 are left alone).  Slots before the one of position
 * seqlens[b] stay as they are: where one is unmapped its tokens were not stored, and a page given to it now
 * would put what the page held before in their place. */
int dash_pages_reserve(const dash_pages* pg, const int* counts, int count, int* status, void* workspace,
                       size_t ws_bytes, void* stream);

/* Row dst[i] (empty: length 0 and no pages) becomes a copy of row src[i], i < n (device int32): it
 * shares the pages that src has filled, gets its own copy of the page that src has filled in part,
 * and copies of src's entries in `rows`.  A source may occur several times.  At most 1024 entries
 * per call. */
int dash_pages_fork(const dash_pages* pg, const int* src, const int* dst, int n, int* status, void* workspace,
                    size_t ws_bytes, void* stream);

/* Rows rows[i], i < n (device int32), give up their pages: counts go down, the table rows become
 * -1, the lengths 0, the `rows` what their `clear` says.  A row listed twice is freed once.  Indices out of
 * range are skipped (and reported). */
int dash_pages_free(const dash_pages* pg, const int* rows, int n, int* status, void* stream);

/* The used pages move together: with U used pages, those numbered U and above move, in order, into
 * the free pages below U, in order; the tables and counts follow.  used (device int32, may be
 * NULL) receives U: pages U and above are then free. */
int dash_pages_compact(const dash_pages* pg, int* used, void* workspace, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* DASH_CACHE_H */
