// Host-side pieces shared by the C ABI's implementation files: size limits, tensor
// checks, TMA descriptors of fa_tensor and the process-wide watchdog setting.
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>

#include "flexattn.h"
#include "tmap.cuh"

namespace fa {

constexpr int64_t kMaxLen = (int64_t(1) << 31) - 256;  // q_len / kv_len bound (int32 tile coordinates)
constexpr size_t kWorkspaceBytes = 256;

uint64_t watchdog_ns();  // fa_set_watchdog_ms

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline int sm_count()
{
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    return n;
}

// A [B, H, S, D] bf16 tensor usable as a TMA source / 16-byte-vector target.  A
// stride of 0 (a broadcast, expanded dimension) is accepted only on a dimension of
// size 1: the tiles are addressed by coordinates, so an expanded dimension would
// read other data than the caller's.
inline int check_tensor(const fa_tensor* t)
{
    if (!t) return FA_ERR_INVALID_ARG;
    bool empty = false;
    for (int i = 0; i < 4; ++i) {
        if (t->dims[i] < 0) return FA_ERR_INVALID_ARG;
        empty |= t->dims[i] == 0;
    }
    if (empty) return FA_OK;  // never accessed
    if (!t->data) return FA_ERR_INVALID_ARG;
    if (t->strides[3] != 1) return FA_ERR_INVALID_ARG;
    for (int i = 0; i < 3; ++i) {
        if (t->strides[i] < 0 || (t->strides[i] % 8) != 0) return FA_ERR_INVALID_ARG;
        if (t->strides[i] == 0 && t->dims[i] > 1) return FA_ERR_INVALID_ARG;
    }
    if (!aligned16(t->data)) return FA_ERR_INVALID_ARG;
    return FA_OK;
}

inline bool tmap_for(CUtensorMap* map, const fa_tensor* t)
{
    // dims innermost first: (D, S, H, B); strides of S, H, B in bytes
    uint64_t dims[4] = {(uint64_t)t->dims[3], (uint64_t)t->dims[2], (uint64_t)t->dims[1], (uint64_t)t->dims[0]};
    uint64_t st[3] = {(uint64_t)t->strides[2] * 2, (uint64_t)t->strides[1] * 2, (uint64_t)t->strides[0] * 2};
    // the CUDA driver wants every stride nonzero: give size-1 dimensions (the only
    // ones check_tensor lets have stride 0) a legal one
    for (int i = 0; i < 3; ++i)
        if (st[i] == 0) st[i] = 16;
    return fa::make_tmap_bf16_4d(map, t->data, dims, st, 128);
}

} // namespace fa
