// Shared by the paged-cache kernels' host sides: the checks of a cache
// description and the copy that mk_export_kv makes.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/mk.h"

namespace mkv {

// MK_OK, or the argument error of a cache description
int check_cache(const mk_paged_kv *kv);

// Enqueue the append of rows 0 .. count-1 of bf16 keys and values [count][heads][d]
// (element strides `row` and `head`) to slots slot0 .. of sequence `seq`, without
// norm or rotation; *status as for mk_paged_append.
int append_range(const mk_paged_kv *kv, const void *k, const void *v, int64_t row, int64_t head, int32_t count,
                 int32_t seq, int32_t slot0, int32_t *status, cudaStream_t stream);

// multiprocessors of the current device (looked up once per device); < 0: a CUDA error
int sm_count(int *device);

}  // namespace mkv
