// Decoding against a paged cache for sm_100a: a few query tokens per sequence,
// every sequence with its own length ("Flex Attention" paper review sec. 3.1, the
// decoding template, and sec. 4.5, paged attention; rocketrecap talk: the work is
// split along the KV dimension and the partial results are reduced at the end).
//
//   row (h, i) of sequence b sits at position len_b - q_len + i and attends the keys
//   at or before it (and within the window);  out = softmax(mod(q k^T scale)) v
//
// Bound: HBM (K and V of the pages are read once; 4 G flops per byte of them).
// Work split: the pages of all (sequence, kv head) segments form one list, and team c of
// two teams per SM takes its c-th equal share, so every SM streams the same number of
// bytes whatever the lengths are.  Each CTA finds its teams' shares by a scan of the
// lengths.  A team is a TMA producer warp, a ring of K and V tiles and four compute
// warps that take 32 keys of every page each, the query rows being the n = 8 side of
// m16n8k16 MMAs, with an online softmax of each warp's own.  The teams have nothing to
// wait for in one another: while one ends a segment or waits for a page, the other
// computes.  At the end of a piece of a segment a team's states are joined in shared
// memory.  A piece that is a whole segment is written out at once; else its state goes to
// the workspace and, at the end of the share, the team that completes the segment (a
// counter, which wraps back to zero) joins the pieces in list order, so that results do
// not depend on who comes last.
//
// Measured on a B200 (back to back, inputs not in L2): 8 sequences of 24k to 32k keys, Hkv 8
// D 128, 138 us = 6.55 TB/s; 16 ragged ones up to 8191 keys 45 us; 24 with four drafted
// tokens, a window of 4096 and capped scores, Hkv 8 D 64, 40 us; one of 700 keys 8.3 us.
// What the short ones are over their bytes is the start (the lengths, the table and the
// first pages one after the other, 4 us), unequal shares of the memory's bandwidth (the
// last SM ends 5 us after the first) and the join of split segments (4 us).  Tried and
// slower: eight warps of 16 keys on every page (0.85 us a page, more than the 32 KB of one
// at D = 64 need); an eighth of the list left open and taken by teams as they get done; two
// groups of warps on alternate pages of one share (they wait for one
// another at every segment's end); more than 192 KB in flight per SM.
//
// Places outside a row's keys may hold anything (a page's slots behind the last key
// are not initialised, and masked keys may hold infinities or NaN): their scores are
// replaced, not added to, and values that no row attends are zeroed before the product.
#include <mutex>
#include <vector>

#include <cuda_runtime.h>

#include "context.cuh"
#include "dependent_launch.cuh"
#include "paged_decode_impl.cuh"

namespace fa {

namespace {

template <int D, int SCORE, int NR>
__global__ void __launch_bounds__(kPdThreads, 1) paged_decode_kernel(const __grid_constant__ PdParams p)
{
    extern __shared__ uint8_t smem_raw[];
    __shared__ pd::Shared sh;
    __shared__ long long scratch[kPdThreads / 32];
    static_assert(pd::Cfg<D>::SMEM + sizeof(sh) + sizeof(scratch) <= 227 * 1024, "shared memory beyond 227 KB per CTA");
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    wait_prerequisites();
    launch_dependents();
    bool bad = false;
    const pd::Scan scan = pd::scan_lengths<kPdThreads>(p, scratch, bad);
    pd::decode_cta<D, SCORE, NR, kPdThreads>(p, sh, smem, blockIdx.x, gridDim.x, scan, bad);
}

template <int D, int SCORE, int NR>
cudaError_t launch_variant(const PdParams& p, cudaStream_t stream)
{
    static std::mutex mu;
    static std::vector<CtxKey> done;
    auto kern = paged_decode_kernel<D, SCORE, NR>;
    {
        CtxKey key;
        std::lock_guard<std::mutex> lock(mu);
        bool have = false;
        if (current_ctx(&key))
            for (const CtxKey& k : done) have |= k == key;
        if (!have) {
            cudaError_t e =
                cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, pd::Cfg<D>::SMEM);
            if (e != cudaSuccess) return e;
            if (current_ctx(&key)) done.push_back(key);
        }
    }
    return launch_after(kern, dim3((unsigned)p.grid), kPdThreads, pd::Cfg<D>::SMEM, stream, p);
}

} // namespace

cudaError_t launch_paged_decode(const PdParams& p, int D, int score_kind, cudaStream_t stream)
{
#define FA_PD_CASE(DD, SS)                    \
    if (D == DD && score_kind == SS)          \
        return p.rows > 8 ? launch_variant<DD, SS, 2>(p, stream) : launch_variant<DD, SS, 1>(p, stream);
    FA_PD_CASE(64, FA_SCORE_NONE) FA_PD_CASE(64, FA_SCORE_ALIBI) FA_PD_CASE(64, FA_SCORE_SOFTCAP)
    FA_PD_CASE(128, FA_SCORE_NONE) FA_PD_CASE(128, FA_SCORE_ALIBI) FA_PD_CASE(128, FA_SCORE_SOFTCAP)
#undef FA_PD_CASE
    return cudaErrorInvalidValue;
}

} // namespace fa
