// ripe_paged_launch.h -- host-side launchers of the paged-cache kernels (internal).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

struct PagedArgs;

// The current device's error word for calls without err_dev.
cudaError_t paged_error_word(int32_t** word);

// A tensor map of the pages at `base`: boxes of `rows` positions of one page and head and
// `chunks` times 32 channels, 64-byte swizzle (false: the driver refused it).
bool paged_kv_map(void* map, const void* base, const PagedArgs& a, int rows, int chunks);

// The attention on the tensor cores, with the join of its partials: `grid` CTAs.
cudaError_t launch_paged_tc(PagedArgs a, int grid, cudaStream_t st);
// The other attention kernels: `grid` CTAs, partials for launch_paged_merge.
cudaError_t launch_paged_decode(PagedArgs a, int grid, cudaStream_t st);
cudaError_t launch_paged_simt(PagedArgs a, int dtype, int grid, cudaStream_t st);
// Joins the partials of the items that were cut, those of the two kernels before.
cudaError_t launch_paged_merge(const PagedArgs& a, int dtype, int grid, cudaStream_t st);

cudaError_t launch_paged_append(const PagedArgs& a, const char* K, const char* V, int64_t row_stride, int esize,
                                cudaStream_t st);
