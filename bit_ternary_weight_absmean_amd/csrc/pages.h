// Arguments of the page kernels (csrc/pages.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace bt {

struct PagesArgs {
    int *table, *length, *refs, *first;  // [B, W], [B], [P], [1]
    const int *q_start;                  // grow
    const int *parent;                   // fork
    int *rows, *positions, *granted;     // grow: [T], [T], [B]
    int *ws;
    char *pool;
    int64_t layer_stride, page_bytes;    // bytes
    int B, W, P, T, layers, page_shift;
};

size_t pages_workspace_bytes(int64_t B, int64_t W, int64_t P);
hipError_t launch_pages_grow(const PagesArgs &a, hipStream_t s);
hipError_t launch_pages_fork(const PagesArgs &a, hipStream_t s);
hipError_t launch_pages_compact(const PagesArgs &a, hipStream_t s);
hipError_t launch_pages_copy(const PagesArgs &a, const int *src, const int *dst, int64_t n, hipStream_t s);

}  // namespace bt
