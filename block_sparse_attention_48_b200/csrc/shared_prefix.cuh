// Launch interface of decoding behind a shared prefix: the prefix and the sequences' own
// parts in one kernel, and their join.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "paged_decode.cuh"
#include "shared_walk.cuh"

namespace fa {

struct SpParams {
    CUtensorMap tm_k;  // page pools [num_pages, Hkv, 128, D], box 64 x 128
    CUtensorMap tm_v;

    const uint16_t* q;  // [B, Hq, q_len, D] bf16
    int64_t q_st0, q_st1, q_st2;
    int32_t B, Hkv, G, q_len, rows;  // rows = G * q_len
    const int32_t* seq_lens;         // [B]
    const int32_t* prefix_row;       // the shared entries of the page table
    int32_t num_pages;

    float scale;
    float softcap, softcap_in;
    const float* slopes;

    SpGeom geom;
    int32_t sms;     // shared out between the prefix and the sequences' own pages
    int32_t* split;  // CTAs that took a share of the list, for the join
    // Partial results: of CTA c's piece of column col (counted over the heads) and stream
    // s, slot 2 (col + c) + s
    float* part_o;   // [slot][D / 4][128][4] fp32, unnormalised
    float* part_ml;  // [slot][128][2]: running max (log2 units), sum

    // join
    uint16_t* o;
    int64_t o_st0, o_st1, o_st2;
    float* lse;            // [B, Hq, q_len] or null
    const float* own_o;    // [B][Hkv][rows][D] fp32, unnormalised
    const float* own_ml;   // [B][Hkv][rows][2]
    int32_t pt_width;

    int* status;
    uint64_t watchdog_ns;
};

cudaError_t launch_shared_decode(const SpParams& p, const PdParams& own, int D, int score_kind, cudaStream_t stream);
cudaError_t launch_shared_join(const SpParams& p, int D, cudaStream_t stream);

} // namespace fa
