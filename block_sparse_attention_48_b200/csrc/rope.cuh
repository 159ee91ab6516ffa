// Launch interface of the rotary kernels: rotary positions on Q and K, and the
// append of new keys and values to a paged cache with the rotation on the way.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace fa {

// One tensor of a launch: H heads per token read from x and written to y, or, when
// `paged`, to the token's slot of the page pool y [num_pages, H, 128, D].
struct RopeGroup {
    const uint16_t* x;
    int64_t x_st0, x_st1, x_st2;  // batch, head, token
    uint16_t* y;
    int64_t y_st0, y_st1, y_st2;  // batch or page, head, token or slot
    int32_t H;
    int32_t rotate;
    int32_t paged;
};

constexpr int kRopeGroups = 3;

struct RopeParams {
    RopeGroup g[kRopeGroups];  // groups with H == 0 are absent
    int32_t first_chunk[kRopeGroups + 1];  // grid y blocks [first_chunk[i], first_chunk[i + 1]) serve group i
    int32_t heads_per_thread;

    int32_t B;
    int64_t S, tokens;         // tokens = B * S
    const double* inv_freq;    // [rotary / 2], radians per position
    int32_t rotary;            // rotated elements of a head, a multiple of 16
    int32_t interleaved;
    float amplitude;
    float sin_sign;            // -1: the inverse rotation

    // position of token (b, s): positions[b * pos_stride + s], or pos_offset + s
    const int32_t* positions;
    int64_t pos_stride;
    int64_t pos_offset;

    // paged append (cache_lens set): position cache_lens[b] + s, rows s >= new_lens[b]
    // (when given) left alone
    const int32_t* cache_lens;
    const int32_t* new_lens;
    const int32_t* page_table;
    int64_t pt_stride, pt_width;
    int32_t num_pages;
    int* status;
};

cudaError_t launch_rope(RopeParams& p, int D, int sms, cudaStream_t stream);

} // namespace fa
