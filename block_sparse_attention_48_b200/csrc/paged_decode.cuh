// Launch interface of decoding against a paged cache (each sequence with its own
// length), and the walk over its work list.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace fa {

constexpr int kPdTeams = 2;                       // of a CTA, each with a share of the work
constexpr int kPdWarps = 4;                       // compute warps of a team, 32 keys of a page each
constexpr int kPdThreads = 32 * kPdTeams * (kPdWarps + 1);  // and a TMA producer warp each
constexpr int kPdMaxRows = 16;                    // query rows of a kv head's group: G * q_len

struct PdParams {
    CUtensorMap tm_k;  // page pools [num_pages, Hkv, 128, D], box 64 x 128
    CUtensorMap tm_v;

    const uint16_t* q;  // [B, Hq, q_len, D] bf16
    int64_t q_st0, q_st1, q_st2;
    uint16_t* o;
    int64_t o_st0, o_st1, o_st2;
    float* lse;         // [B, Hq, q_len] or null

    int32_t B, Hq, Hkv, G, q_len, rows;
    int32_t teams;              // at most so many have work
    const int32_t* seq_lens;    // [B]
    const int32_t* page_table;  // row b at b * pt_stride, pt_width entries
    int64_t pt_stride;
    int32_t pt_width, num_pages;
    int32_t prefix_pages;       // leading table entries whose keys are taken elsewhere; 0: none
    int32_t row0_pages;         // leading table entries that sequences reaching past them
                                // read from row 0 (a shared prefix taken page by page)
    int32_t has_window;
    int64_t window;

    float scale;
    float softcap, softcap_in;
    const float* slopes;

    // Work split: team c of those that have work takes the c-th share of the list of pages.  A segment
    // split over teams c0..c1 leaves partial results 2 c0 + 1 (its first piece, the end of
    // c0's share) and 2 c for c in (c0, c1] (the start of c's share)
    int32_t grid;         // CTAs, of kPdTeams teams each
    float* part_o;        // [2 * teams][rows][D] fp32, unnormalised
    float* part_ml;       // [2 * teams][rows][2]: running max (log2 units), sum
    unsigned* arrived;    // [team] pieces done of the segment whose first piece ends share c0;
                          // every call leaves zeros

    // With a shared prefix: the state (log2 max, sum, unnormalised O) of the rows whose
    // prefix is taken elsewhere, for the join
    float* own_o;         // [B][Hkv][rows][D] fp32
    float* own_ml;        // [B][Hkv][rows][2]

    int* status;
    uint64_t watchdog_ns;
};

cudaError_t launch_paged_decode(const PdParams& p, int D, int score_kind, cudaStream_t stream);

} // namespace fa
