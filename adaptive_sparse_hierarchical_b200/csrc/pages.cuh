// pages.cuh -- internal structures and launchers of the page operations (include/dash_cache.h).
#pragma once
#include "dash_common.cuh"
#include "../../include/dash_cache.h"

namespace dash {

constexpr int kArrays = 64, kFewArrays = 8;   // arrays per mover launch (they travel as kernel arguments)

struct PageTab {
    int batch, max_pages, page_size, num_pages;
    int *page_table, *refs, *seqlens;
};

struct MoveArray {
    char* data;
    long long bytes, stride;
    int segs;
};
struct MoveRows {
    char* data;
    long long row_stride, head_stride, unit_bytes;
    int heads, max_units, unit_tokens, segs, clear;
    bool wide;
};

// Lists in the workspace: pages to copy (src, dst), marks or the page map (mark), per entry of a row
// list the parent's length or, for reserve, the pages given out before (row) and the child's own
// page (own).
struct PagesWs {
    char* head;
    int *src, *dst, *mark, *row, *own;
};
int pages_max_fork();   // entries of one fork call
size_t pages_ws(const PageTab& t, char* base, PagesWs* w);   // carves `base` up; returns the bytes needed

cudaError_t launch_pages_copy(const PageTab& t, const dash_pages* pg, const int* src, const int* dst, int n, int* status,
                              const PagesWs& w, cudaStream_t st);
cudaError_t launch_pages_reserve(const PageTab& t, const int* counts, int count, int* status, const PagesWs& w,
                                 cudaStream_t st);
cudaError_t launch_pages_fork(const PageTab& t, const dash_pages* pg, const int* src, const int* dst, int n, int* status,
                              const PagesWs& w, cudaStream_t st);
cudaError_t launch_pages_free(const PageTab& t, const dash_pages* pg, const int* rows, int n, int* status,
                              cudaStream_t st);
cudaError_t launch_pages_compact(const PageTab& t, const dash_pages* pg, int* used, const PagesWs& w, cudaStream_t st);

}  // namespace dash
