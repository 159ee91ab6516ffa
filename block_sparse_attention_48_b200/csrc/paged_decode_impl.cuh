// The paged decode's CTA (see paged_decode.cu, which runs it on all SMs; the shared prefix's
// kernel runs it on some of them beside the prefix).
#pragma once

#include <climits>

#include <cuda_runtime.h>

#include "dependent_launch.cuh"
#include "flex_fwd.cuh"
#include "flexattn.h"
#include "paged_decode.cuh"
#include "paged_walk.cuh"
#include "ptx.cuh"
#include "score_math.cuh"

namespace fa {

namespace pd {

constexpr int kBox = 16384;  // 128 rows of 64 columns
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescale = 8.f;  // log2 of the growth that moves the running maximum

template <int D>
struct Cfg {
    static constexpr int TILE = 128 * D * 2;       // K or V of one page and kv head
    static constexpr int NT = D == 128 ? 3 : 6;    // tiles of a team's ring, 96 KB
    static constexpr int OROW = D + 4;             // padded row of the joining buffer (bank spread)
    static constexpr int JOIN = kPdWarps * 8 * OROW * 4;  // eight rows of every warp at a time
    static constexpr int OFF_JOIN = kPdTeams * NT * TILE;
    static constexpr int SMEM = OFF_JOIN + kPdTeams * JOIN + 1024;
};

struct __align__(16) Shared {
    uint64_t full[kPdTeams][6], empty[kPdTeams][6];
    PdWalk start[kPdTeams];                   // where a team's share starts
    int last[kPdTeams][2];                    // this team completed the split segment
    uint16_t row_at[kPdMaxRows];              // a query row's head in its group * 256 + its token
    float m[kPdTeams][kPdWarps][8], l[kPdTeams][kPdWarps][8];  // of eight rows
};

// The compute warps of a team.
__device__ __forceinline__ void team_sync(int team)
{
    asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "n"(32 * kPdWarps) : "memory");
}

// A cache policy for data that a call reads once: the first to leave L2, so that what every
// call reads again (code, tables, queries, partial results) stays.  16 ragged sequences 45.5
// us instead of 46.9, 64 behind 4096 shared keys with 500 to 3000 of their own 85 instead of
// 92; pages that several sequences share are found in L2 as before.
__device__ __forceinline__ uint64_t read_once_policy()
{
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
    return p;
}

// tma_load_4d with a cache policy.
__device__ __forceinline__ void tma_load_4d_once(void* smem_dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1,
                                                 int c2, int c3, uint64_t policy)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %3, %4, %5}], [%6], %7;" ::"r"(smem_u32(smem_dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_u32(bar)), "l"(policy)
        : "memory");
}

__device__ __forceinline__ uint32_t movmatrix_t(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// Address of 16-byte unit `unit` of key row `key` in a tile loaded with the
// 128-byte swizzle (64-column chunks of 16 KB).
__device__ __forceinline__ uint32_t swz(uint32_t base, int key, int unit)
{
    return base + (uint32_t)((unit >> 3) * kBox + key * 128 + (((unit & 7) ^ (key & 7)) << 4));
}

// An infinity or NaN among the two bf16 of a register.
__device__ __forceinline__ bool nonfinite2(uint32_t w)
{
    return (w & 0x7F80u) == 0x7F80u || (w & 0x7F800000u) == 0x7F800000u;
}

// Team of the work split: the first teams of all CTAs come before the second ones, so
// that a short list is spread over the SMs.
__device__ __forceinline__ int team_of(int block, int ctas, int team)
{
    return block < ctas ? block + ctas * team : INT_MAX;
}

// A thread's view of the lengths' sums (pd_weight): those of its sequences [lo, hi), of
// the sequences before them, and of all.
struct Scan {
    int lo, hi;
    long long mine, before, total;
    __device__ __forceinline__ static int pages(long long x) { return (int)(x & ((1ll << kPdCount) - 1)); }
    __device__ __forceinline__ static int sequences(long long x) { return (int)(x >> kPdCount); }
};

// All THREADS threads of the CTA.
template <int THREADS, class P>
__device__ __forceinline__ Scan scan_lengths(const P& p, long long* scratch, bool& bad)
{
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int per = (p.B + THREADS - 1) / THREADS;
    Scan s;
    s.lo = min(p.B, tid * per);
    s.hi = min(p.B, s.lo + per);
    s.mine = 0;
    for (int b = s.lo; b < s.hi; ++b) s.mine += pd_weight(pd_range(p, p.seq_lens[b], bad));
    long long inc = s.mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xFFFFFFFFu, inc, o);
        if (lane >= o) inc += y;
    }
    if (lane == 31) scratch[warp] = inc;
    __syncthreads();
    s.before = inc - s.mine;
    s.total = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
        s.before += w < warp ? scratch[w] : 0;
        s.total += scratch[w];
    }
    return s;
}

// One CTA's part, `block` of `ctas`, of the paged decode; all THREADS threads of the CTA
// call it (those past the teams' only help with the lengths).
template <int D, int SCORE, int NR, int THREADS>
__device__ __forceinline__ void decode_cta(const PdParams& p, Shared& sh, uint8_t* smem, int block, int ctas,
                                           const Scan& scan, bool bad)
{
    using C = Cfg<D>;
    constexpr int KD = D / 16;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    Watchdog wd{p.watchdog_ns, false};

    const int T = Scan::pages(scan.total) * p.Hkv, used = min(T, min(ctas * kPdTeams, p.teams));
    if (threadIdx.x == 0) {
        for (int t = 0; t < kPdTeams; ++t)
            for (int i = 0; i < C::NT; ++i) {
                mbar_init(&sh.full[t][i], 1);
                mbar_init(&sh.empty[t][i], kPdWarps);
            }
        mbar_fence_init();
    }
    if (threadIdx.x < p.rows)
        sh.row_at[threadIdx.x] = (uint16_t)(threadIdx.x / p.q_len * 256 + threadIdx.x % p.q_len);
#pragma unroll
    for (int t = 0; t < kPdTeams; ++t) {
        if (team_of(block, ctas, t) >= used) continue;
        const int x0 = pd_share(T, team_of(block, ctas, t), used), at = Scan::pages(scan.before);
        if (p.Hkv * at <= x0 && x0 < p.Hkv * (at + Scan::pages(scan.mine)))
            pd_find(p, x0, scan.lo, scan.hi, at, sh.start[t], bad);
    }
    __syncthreads();
    if (threadIdx.x >= kPdThreads) {
        if (bad) atomicOr(p.status, STATUS_BAD_BLOCKMASK);
        return;
    }
    const int team = warp < kPdTeams * kPdWarps ? warp / kPdWarps : warp - kPdTeams * kPdWarps;
    const int me = team_of(block, ctas, team);
    uint64_t *full = sh.full[team], *empty = sh.empty[team];
    uint8_t* ring = smem + team * C::NT * C::TILE;
    const bool works = me < used;
    const int x0 = works ? pd_share(T, me, used) : 0;
    const int count = works ? pd_share(T, me + 1, used) - x0 : 0;
    PdWalk w{0, 0, 0, {0, 0, 0, 0}};
    if (works) w = sh.start[team];

    if (warp >= kPdTeams * kPdWarps) {
        // TMA producer: K and V of every page of the share.  Lane l holds the page of the
        // (t & ~31) + l-th page of the segment's range.
        const uint64_t policy = read_once_policy();
        uint32_t issued = 0;  // tiles
        bool ok = true;
        int page_lane = 0, chunk = -1;
        auto load = [&](const CUtensorMap* tm, int hk, int page) {
            const uint32_t slot = issued % C::NT, use = issued / C::NT;
            ok = ok && __all_sync(0xFFFFFFFFu, mbar_wait(&empty[slot], (use & 1) ^ 1, wd));
            if (!ok) return;
            if (elect_one_sync()) {
                mbar_arrive_expect_tx(&full[slot], C::TILE);
#pragma unroll
                for (int c = 0; c < D / 64; ++c)
                    tma_load_4d_once(ring + slot * C::TILE + c * kBox, tm, &full[slot], c * 64, 0, hk, page, policy);
            }
            __syncwarp();
            ++issued;
        };
        for (int i = 0; ok && i < count; ++i) {
            if (chunk != (w.t & ~31)) {
                chunk = w.t & ~31;
                const int tt = chunk + lane;
                const int row = w.r.lo + tt < p.row0_pages && w.r.len - p.q_len >= 128 * p.row0_pages ? 0 : w.b;
                page_lane = tt < w.r.n ? p.page_table[row * p.pt_stride + w.r.lo + tt] : 0;
            }
            const int page = pd_page(__shfl_sync(0xFFFFFFFFu, page_lane, w.t & 31), p.num_pages, bad);
            load(&p.tm_k, w.hk, page);
            load(&p.tm_v, w.hk, page);
            if (i + 1 < count) {
                const int b = w.b;
                pd_advance(p, w, bad);
                if (w.b != b) chunk = -1;
            }
        }
        // copies in flight land before the CTA exits (bounded)
        Watchdog dw{wd.failed ? 1000000ull : wd.limit_ns, false};
        for (uint32_t j = 0; j < (uint32_t)C::NT && j < issued; ++j) {
            const uint32_t last = issued - 1 - j;
            dw.failed = false;
            mbar_wait(&full[last % C::NT], (last / C::NT) & 1, dw);
        }
        if (lane == 0 && (wd.failed || !ok)) atomicOr(p.status, STATUS_TIMEOUT);
        if (__any_sync(0xFFFFFFFFu, bad) && lane == 0) atomicOr(p.status, STATUS_BAD_BLOCKMASK);
        return;
    }

    // ---- compute warps: S^T = K Q^T for two tiles of 16 keys, O^T += V^T P^T.  Thread
    // (g, tq) = (lane / 4, lane % 4) holds S^T at keys g, g + 8 of a tile and query rows
    // 2 tq, 2 tq + 1 (+ 8 per row tile).
    const int tid = threadIdx.x % (32 * kPdWarps), tw = warp % kPdWarps;  // within the team
    const int g = lane >> 2, tq = lane & 3, m4 = lane >> 3;
    const int key0 = 32 * tw;  // the warp's first key of a page
    int tok[NR][2];      // the token of each of the thread's rows
    bool rvalid[NR][2];
    int hq_g[NR][2];     // and its head within the group
#pragma unroll
    for (int nt = 0; nt < NR; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int r = 8 * nt + 2 * tq + j;
            rvalid[nt][j] = r < p.rows;
            tok[nt][j] = rvalid[nt][j] ? r % p.q_len : 0;
            hq_g[nt][j] = rvalid[nt][j] ? r / p.q_len : 0;
        }
    float slope[NR][2];
    uint32_t qb[NR][KD][2];
    int64_t q_off[NR];  // the B fragment's column: a query row's place in a sequence's and head's Q
    bool q_in[NR];
#pragma unroll
    for (int nt = 0; nt < NR; ++nt) {
        const int r = 8 * nt + g;
        q_in[nt] = r < p.rows;
        q_off[nt] = q_in[nt] ? (int64_t)(r / p.q_len) * p.q_st1 + (int64_t)(r % p.q_len) * p.q_st2 + 2 * tq : 0;
    }
    auto load_segment = [&](int b, int hk) {
        const uint16_t* seg = p.q + (int64_t)b * p.q_st0 + (int64_t)(hk * p.G) * p.q_st1;
#pragma unroll
        for (int nt = 0; nt < NR; ++nt) {
#pragma unroll
            for (int j = 0; j < 2; ++j)
                slope[nt][j] = SCORE == FA_SCORE_ALIBI ? p.slopes[hk * p.G + hq_g[nt][j]] * kLog2e : 0.f;
#pragma unroll
            for (int kk = 0; kk < KD; ++kk) {
                const uint16_t* src = seg + q_off[nt] + 16 * kk;
                qb[nt][kk][0] = q_in[nt] ? *reinterpret_cast<const uint32_t*>(src) : 0u;
                qb[nt][kk][1] = q_in[nt] ? *reinterpret_cast<const uint32_t*>(src + 8) : 0u;
            }
        }
    };
    float oacc[KD][NR][4];
    float m_run[NR][2], l_run[NR][2];  // log2 units; l: this thread's keys only
    auto reset = [&]() {
#pragma unroll
        for (int mt = 0; mt < KD; ++mt)
#pragma unroll
            for (int nt = 0; nt < NR; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) oacc[mt][nt][e] = 0.f;
#pragma unroll
        for (int nt = 0; nt < NR; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                m_run[nt][j] = -INFINITY;
                l_run[nt][j] = 0.f;
            }
    };
    float* join = reinterpret_cast<float*>(smem + C::OFF_JOIN + team * C::JOIN);  // [warp][row][OROW]

    // One output row element group (four columns at d of row r): O / l and LSE, or the
    // state that joins the shared prefix's.  (Divisions by q_len and of list positions are
    // kept out of the pieces' code: it is run a few times a CTA, and fetching it from a
    // busy memory takes longer than running it.)
    auto write_out = [&](int b, int hk, int r, int d, bool shared, float M, float L, const float (&v)[4]) {
        if (shared) {
            const int64_t row = ((int64_t)b * p.Hkv + hk) * p.rows + r;
            *reinterpret_cast<float4*>(p.own_o + row * D + d) = make_float4(v[0], v[1], v[2], v[3]);
            if (d == 0) *reinterpret_cast<float2*>(p.own_ml + row * 2) = make_float2(M, L);
            return;
        }
        const bool some = L > 0.f && M != -INFINITY;
        const float inv = some ? 1.0f / L : 0.f;
        const int hq = hk * p.G + sh.row_at[r] / 256, i = sh.row_at[r] % 256;
        uint16_t* o = p.o + (int64_t)b * p.o_st0 + (int64_t)hq * p.o_st1 + (int64_t)i * p.o_st2 + d;
        // a row that attends nothing: O = 0
        *reinterpret_cast<uint2*>(o) =
            some || L != L ? make_uint2(pack_bf16x2(v[0] * inv, v[1] * inv), pack_bf16x2(v[2] * inv, v[3] * inv))
                           : make_uint2(0u, 0u);
        if (d == 0 && p.lse)
            p.lse[((int64_t)b * p.Hq + hq) * p.q_len + i] =
                some ? (M + __log2f(L)) * kLn2 : L != L ? L : -INFINITY;
    };

    // The end of a piece: the warps' states joined, and written out if it is a whole
    // segment, else left as partial result `part`.
    auto end_piece = [&](const PdWalk& at, int part) {
#pragma unroll
        for (int nt = 0; nt < NR; ++nt) {
            team_sync(team);  // the buffer's last states have been read
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float l = l_run[nt][j];  // sum over the eight key groups
                l += __shfl_xor_sync(0xFFFFFFFFu, l, 4);
                l += __shfl_xor_sync(0xFFFFFFFFu, l, 8);
                l += __shfl_xor_sync(0xFFFFFFFFu, l, 16);
                if (g == 0) {
                    sh.m[team][tw][2 * tq + j] = m_run[nt][j];
                    sh.l[team][tw][2 * tq + j] = l;
                }
                float* dst = join + (tw * 8 + 2 * tq + j) * C::OROW + g;
#pragma unroll
                for (int mt = 0; mt < KD; ++mt) {
                    dst[16 * mt] = oacc[mt][nt][j];
                    dst[16 * mt + 8] = oacc[mt][nt][2 + j];
                }
            }
            team_sync(team);
            const int items = min(8, p.rows - 8 * nt) * (D / 4);
            for (int it = tid; it < items; it += 32 * kPdWarps) {
                const int r8 = it / (D / 4), r = 8 * nt + r8, d = (it % (D / 4)) * 4;
                float M = -INFINITY;
#pragma unroll
                for (int k = 0; k < kPdWarps; ++k) M = fmaxf(M, sh.m[team][k][r8]);
                const float Mu = M == -INFINITY ? 0.f : M;
                float L = 0.f, v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int k = 0; k < kPdWarps; ++k) {
                    const float f = ex2_approx(sh.m[team][k][r8] - Mu);
                    const float4 x = *reinterpret_cast<const float4*>(join + (k * 8 + r8) * C::OROW + d);
                    L = fmaf(sh.l[team][k][r8], f, L);
                    v[0] = fmaf(x.x, f, v[0]);
                    v[1] = fmaf(x.y, f, v[1]);
                    v[2] = fmaf(x.z, f, v[2]);
                    v[3] = fmaf(x.w, f, v[3]);
                }
                if (part < 0) {
                    write_out(at.b, at.hk, r, d, at.r.shared, M, L, v);
                } else {
                    const int64_t row = (int64_t)part * p.rows + r;
                    __stcg(reinterpret_cast<float4*>(p.part_o + row * D + d), make_float4(v[0], v[1], v[2], v[3]));
                    if (d == 0) __stcg(reinterpret_cast<float2*>(p.part_ml + row * 2), make_float2(M, L));
                }
            }
        }
    };

    // The last piece of a split segment to arrive joins them all, in list order.  Only the
    // first piece of a share (the end or the middle of a segment) and the last (the start
    // of one) can be split; both arrive at the share's end, where the fence's and the
    // counters' latency holds up nothing.
    auto join_parts = [&](const PdWalk& at, int c0, int c1) {
        // Items under way together: all of up to 16 rows, and 16 loads of a thread (12 segments
        // of 12000 keys, 16 rows, D 128: 53.3 us one by one, 41.7 two by two, 40.6 so; 24 and
        // 32 loads: 41.8 and 42.9).  Up to 8 rows are mostly one item; two by two, their code
        // cost every call 0.7 us and more.
        constexpr int TH = 32 * kPdWarps, I = NR == 1 ? 1 : D / 32, U = NR == 1 ? 4 : 16 / I;
        const int items = p.rows * (D / 4);  // four columns of a row
        for (int it0 = tid; it0 < items; it0 += I * TH) {
            float M[I], L[I], v[I][4];
            int r[I], d[I];
#pragma unroll
            for (int i = 0; i < I; ++i) {
                const int it = it0 + i * TH < items ? it0 + i * TH : it0;
                r[i] = it / (D / 4);
                d[i] = (it % (D / 4)) * 4;
                M[i] = -INFINITY;
                L[i] = v[i][0] = v[i][1] = v[i][2] = v[i][3] = 0.f;
            }
#pragma unroll U  // the parts' loads do not wait for one another
            for (int c = c0; c <= c1; ++c) {
                const int64_t part = (2 * (int64_t)c + (c == c0)) * p.rows;
#pragma unroll
                for (int i = 0; i < I; ++i) {
                    const float2 w = reinterpret_cast<const float2*>(p.part_ml)[part + r[i]];
                    const float4 x = *reinterpret_cast<const float4*>(p.part_o + (part + r[i]) * D + d[i]);
                    const float m = fmaxf(M[i], w.x), Mu = m == -INFINITY ? 0.f : m;
                    const float f0 = ex2_approx(M[i] - Mu), f = ex2_approx(w.x - Mu);
                    M[i] = m;
                    L[i] = fmaf(w.y, f, L[i] * f0);
                    v[i][0] = fmaf(x.x, f, v[i][0] * f0);
                    v[i][1] = fmaf(x.y, f, v[i][1] * f0);
                    v[i][2] = fmaf(x.z, f, v[i][2] * f0);
                    v[i][3] = fmaf(x.w, f, v[i][3] * f0);
                }
            }
#pragma unroll
            for (int i = 0; i < I; ++i)
                if (it0 + i * TH < items) write_out(at.b, at.hk, r[i], d[i], at.r.shared, M[i], L[i], v[i]);
        }
    };

    const float F = SCORE == FA_SCORE_SOFTCAP ? p.softcap * kLog2e : p.scale * kLog2e;
    // One page: the warp's 32 keys, the first of them kv0.  K's slot is given back after its
    // products; V's tile is waited for when it is needed.
    auto page = [&](uint32_t kbase, uint32_t vbase, int kv0, int pos0, int pos1, bool edge, uint64_t* k_free,
                    uint64_t* v_full, uint32_t v_phase) {
        float sacc[2][NR][4], sodd[2][NR][4];  // two chains of products for each tile of keys
#pragma unroll
        for (int kt = 0; kt < 2; ++kt)
#pragma unroll
            for (int nt = 0; nt < NR; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) sacc[kt][nt][e] = sodd[kt][nt][e] = 0.f;
#pragma unroll
        for (int kk = 0; kk < KD; ++kk)
#pragma unroll
            for (int kt = 0; kt < 2; ++kt) {
                uint32_t ka[4];
                ldsm_x4(swz(kbase, key0 + 16 * kt + 8 * (m4 & 1) + (lane & 7), 2 * kk + (m4 >> 1)), ka);
#pragma unroll
                for (int nt = 0; nt < NR; ++nt)
                    mma_bf16_16816(kk & 1 ? sodd[kt][nt] : sacc[kt][nt], ka, qb[nt][kk][0], qb[nt][kk][1]);
            }
#pragma unroll
        for (int kt = 0; kt < 2; ++kt)
#pragma unroll
            for (int nt = 0; nt < NR; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) sacc[kt][nt][e] += sodd[kt][nt][e];
        __syncwarp();
        if (lane == 0) mbar_arrive(k_free);

        if constexpr (SCORE == FA_SCORE_SOFTCAP) {
            // tanh: the polynomial, and the far form where the warp has a far score
            bool far = false;
#pragma unroll
            for (int kt = 0; kt < 2; ++kt)
#pragma unroll
                for (int nt = 0; nt < NR; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        sacc[kt][nt][e] *= p.softcap_in;
                        far |= fabsf(sacc[kt][nt][e]) > kTanhPolyMax;
                    }
            const bool any = __any_sync(0xFFFFFFFFu, far);
#pragma unroll
            for (int kt = 0; kt < 2; ++kt)
#pragma unroll
                for (int nt = 0; nt < NR; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; e += 2) {
                        const float y0 = sacc[kt][nt][e], y1 = sacc[kt][nt][e + 1];
                        float t0, t1;
                        f2_unpack(tanh_poly2(f2_pack(y0, y1)), t0, t1);
                        if (any) {
                            const float u0 = tanh_far(y0), u1 = tanh_far(y1);
                            t0 = fabsf(y0) > kTanhPolyMax ? u0 : t0;
                            t1 = fabsf(y1) > kTanhPolyMax ? u1 : t1;
                        }
                        sacc[kt][nt][e] = t0;
                        sacc[kt][nt][e + 1] = t1;
                    }
        }
        // score_mod in log2 units; masked scores are replaced
        float mt_[NR][2];
#pragma unroll
        for (int nt = 0; nt < NR; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) mt_[nt][j] = -INFINITY;
#pragma unroll
        for (int nt = 0; nt < NR; ++nt)
#pragma unroll
            for (int kt = 0; kt < 2; ++kt)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int j = e & 1;
                    const int kv = kv0 + 16 * kt + g + 8 * (e >> 1);
                    const int pos = pos0 + tok[nt][j];
                    bool adm = rvalid[nt][j];
                    if (edge) adm = adm && kv <= pos && (!p.has_window || (int64_t)pos - kv <= p.window);
                    float x = sacc[kt][nt][e];
                    if constexpr (SCORE == FA_SCORE_SOFTCAP) x = x * F;  // capped above
                    else if constexpr (SCORE == FA_SCORE_ALIBI) x = fmaf(slope[nt][j], (float)(kv - pos), x * F);
                    else x = x * F;
                    x = adm ? x : -INFINITY;
                    sacc[kt][nt][e] = x;
                    mt_[nt][j] = fmaxf(mt_[nt][j], x);
                }
        // The running maximum moves only when a score exceeds it by 2^8 (the first score of
        // all does), so that most pages need neither the reductions nor the rescaling.
        bool grows = false;
#pragma unroll
        for (int nt = 0; nt < NR; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) grows |= mt_[nt][j] > m_run[nt][j] + kRescale;
        if (__any_sync(0xFFFFFFFFu, grows)) {
            float alpha[NR][2];
#pragma unroll
            for (int nt = 0; nt < NR; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float m = mt_[nt][j];
                    m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 4));
                    m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 8));
                    m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 16));
                    m = fmaxf(m_run[nt][j], m);
                    alpha[nt][j] = ex2_approx(m_run[nt][j] - (m == -INFINITY ? 0.f : m));  // 0 while nothing was admitted
                    m_run[nt][j] = m;
                    l_run[nt][j] *= alpha[nt][j];
                }
#pragma unroll
            for (int mt = 0; mt < KD; ++mt)
#pragma unroll
                for (int nt = 0; nt < NR; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) oacc[mt][nt][e] *= alpha[nt][e & 1];
        }
        float m_use[NR][2];
#pragma unroll
        for (int nt = 0; nt < NR; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) m_use[nt][j] = m_run[nt][j] == -INFINITY ? 0.f : m_run[nt][j];
        // P^T in bf16 (at most 2^-8 of each entry, as in every kernel here: the tensor
        // core's operand type); the sum is taken of the unrounded values
        uint32_t pb[2][NR][2];
#pragma unroll
        for (int kt = 0; kt < 2; ++kt)
#pragma unroll
            for (int nt = 0; nt < NR; ++nt) {
                float pv[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    pv[e] = ex2_approx(sacc[kt][nt][e] - m_use[nt][e & 1]);
                    l_run[nt][e & 1] += pv[e];
                }
                pb[kt][nt][0] = movmatrix_t(pack_bf16x2(pv[0], pv[1]));  // keys 0-7
                pb[kt][nt][1] = movmatrix_t(pack_bf16x2(pv[2], pv[3]));  // keys 8-15
            }
        // after a timeout V's tile may not have landed: whatever it holds
        __all_sync(0xFFFFFFFFu, mbar_wait(v_full, v_phase, wd));
        // V^T of 16 columns (mt) and 16 keys (kt)
        auto load_v = [&](int mt, int kt, uint32_t (&va)[4]) {
            ldsm_x4_trans(swz(vbase, key0 + 16 * kt + 8 * (m4 >> 1) + (lane & 7), 2 * mt + (m4 & 1)), va);
        };
        // register masks of V^T's keys 2 tq, 2 tq + 1 (low, high half) and the same + 8 that
        // a row at positions [from, to] may attend
        auto keep = [&](int kt, int from, int to, uint32_t (&k2)[2]) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int kv = kv0 + 16 * kt + 2 * tq + 8 * h;
                const bool a = kv <= to && (!p.has_window || (int64_t)from - kv <= p.window);
                const bool b = kv + 1 <= to && (!p.has_window || (int64_t)from - (kv + 1) <= p.window);
                k2[h] = (a ? 0x0000FFFFu : 0u) | (b ? 0xFFFF0000u : 0u);
            }
        };
        uint32_t k2[2][2] = {{~0u, ~0u}, {~0u, ~0u}};
        bool odd = false;
        if (edge) {
#pragma unroll
            for (int kt = 0; kt < 2; ++kt) keep(kt, pos0, pos1, k2[kt]);
            // an infinity or NaN that some rows attend and others may not
            if (p.q_len > 1) {
#pragma unroll 1
                for (int mt = 0; mt < KD; ++mt)
#pragma unroll
                    for (int kt = 0; kt < 2; ++kt) {
                        uint32_t vr[4];
                        load_v(mt, kt, vr);
#pragma unroll
                        for (int e = 0; e < 4; ++e) odd |= nonfinite2(vr[e] & k2[kt][e >> 1]);
                    }
                odd = __any_sync(0xFFFFFFFFu, odd);
            }
        }
        if (!odd) {
            // (masked on every page: a second copy of the products for the masked pages alone
            // took three times as long on them, most of it for fetching the code)
#pragma unroll
            for (int mt = 0; mt < KD; ++mt)
#pragma unroll
                for (int kt = 0; kt < 2; ++kt) {
                    uint32_t vr[4];
                    load_v(mt, kt, vr);
#pragma unroll
                    for (int e = 0; e < 4; ++e) vr[e] &= k2[kt][e >> 1];
#pragma unroll
                    for (int nt = 0; nt < NR; ++nt) mma_bf16_16816(oacc[mt][nt], vr, pb[kt][nt][0], pb[kt][nt][1]);
                }
        } else {
            // one product per token, each with its own keys, kept for its rows only
#pragma unroll 1
            for (int t = 0; t < p.q_len; ++t) {
#pragma unroll
                for (int kt = 0; kt < 2; ++kt) keep(kt, pos0 + t, pos0 + t, k2[kt]);
#pragma unroll
                for (int mt = 0; mt < KD; ++mt)
#pragma unroll
                    for (int kt = 0; kt < 2; ++kt) {
                        uint32_t vr[4];
                        load_v(mt, kt, vr);
#pragma unroll
                        for (int e = 0; e < 4; ++e) vr[e] &= k2[kt][e >> 1];
#pragma unroll
                        for (int nt = 0; nt < NR; ++nt) {
                            float d4[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) d4[e] = oacc[mt][nt][e];
                            mma_bf16_16816(d4, vr, pb[kt][nt][0], pb[kt][nt][1]);
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (tok[nt][e & 1] == t) oacc[mt][nt][e] = d4[e];
                        }
                    }
            }
        }
    };

    // the share's first and last piece where they are parts of a split segment, and the
    // list positions of those segments
    PdWalk head = w, tail = w;
    int xhead = -1, xtail = -1;
    if (count > 0) load_segment(w.b, w.hk);
    int xseg = x0 - w.t;  // list position of the segment's first page
    uint32_t slot = 0, phase = 0;  // of the next tile
    auto step = [&]() {
        if (++slot == C::NT) {
            slot = 0;
            phase ^= 1;
        }
    };
    for (int done = 0; done < count;) {
        // a piece: pages [w.t, w.t + n) of the segment
        const int n = min(w.r.n - w.t, count - done);
        const int pos0 = w.r.len - p.q_len, pos1 = w.r.len - 1;  // first and last query row's positions
        int kv0 = (w.r.lo + w.t) * 128 + key0;                   // the warp's first key
        reset();
        for (int i = 0; i < n; ++i, kv0 += 128) {
            // after a timeout the warp still walks its share (without computing), so that
            // the pieces' barriers and counters stay whole
            const bool ok = __all_sync(0xFFFFFFFFu, mbar_wait(&full[slot], phase, wd));
            const uint32_t ks = slot;
            step();
            if (ok) {
                const uint32_t kbase = smem_u32(ring + ks * C::TILE), vbase = smem_u32(ring + slot * C::TILE);
                // no row attends any of the warp's keys, or some row not all of them
                const bool none = kv0 > pos1 || (p.has_window && kv0 + 31 < pos0 - p.window);
                const bool edge = kv0 + 31 > pos0 || (p.has_window && kv0 < pos1 - p.window);
                if (!none) {
                    page(kbase, vbase, kv0, pos0, pos1, edge, &empty[ks], &full[slot], phase);
                } else {
                    if (lane == 0) mbar_arrive(&empty[ks]);
                    __all_sync(0xFFFFFFFFu, mbar_wait(&full[slot], phase, wd));
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&empty[slot]);
            }
            step();
        }
        done += n;
        PdWalk next = w;
        next.t += n - 1;
        if (done < count) {
            pd_advance(p, next, bad);
            load_segment(next.b, next.hk);  // its latency passes during the join
        }
        int part = -1;
        if (xseg < x0) {  // the segment's first piece is another team's
            head = w;
            xhead = xseg;
            part = 2 * me;
        } else if (xseg + w.r.n > x0 + count) {  // only its first piece is here
            tail = w;
            xtail = xseg;
            part = 2 * me + 1;
        }
        end_piece(w, part);
        xseg += w.r.n;
        w = next;
    }
    if (xhead >= 0 || xtail >= 0) {
        team_sync(team);
        const int h0 = xhead >= 0 ? pd_holder(T, xhead, used) : 0;
        const int h1 = xhead >= 0 ? pd_holder(T, xhead + head.r.n - 1, used) : 0;
        const int t1 = xtail >= 0 ? pd_holder(T, xtail + tail.r.n - 1, used) : 0;
        if (tid == 0) {
            __threadfence();
            unsigned h = 0, t = 0;  // the counters wrap to zero at the last piece
            if (xhead >= 0) h = atomicInc(p.arrived + h0, (unsigned)(h1 - h0));
            if (xtail >= 0) t = atomicInc(p.arrived + me, (unsigned)(t1 - me));
            sh.last[team][0] = xhead >= 0 && h == (unsigned)(h1 - h0);
            sh.last[team][1] = xtail >= 0 && t == (unsigned)(t1 - me);
            __threadfence();
        }
        team_sync(team);
        if (sh.last[team][0]) join_parts(head, h0, h1);
        if (sh.last[team][1]) join_parts(tail, me, t1);
    }
    // sequences without a key: O = 0, LSE = -inf
    for (int b = block; b < p.B; b += ctas) {
        if (pd_range(p, p.seq_lens[b], bad).n > 0) continue;
        const int per_head = p.q_len * (D / 8);
        for (int it = threadIdx.x; it < p.Hq * per_head; it += 32 * kPdWarps * kPdTeams) {
            const int h = it / per_head, i = it % per_head / (D / 8), u = it % (D / 8);
            uint16_t* o = p.o + (int64_t)b * p.o_st0 + (int64_t)h * p.o_st1 + (int64_t)i * p.o_st2;
            reinterpret_cast<uint4*>(o)[u] = make_uint4(0, 0, 0, 0);
            if (u == 0 && p.lse) p.lse[((int64_t)b * p.Hq + h) * p.q_len + i] = -INFINITY;
        }
    }
    if (bad) atomicOr(p.status, STATUS_BAD_BLOCKMASK);
    if (wd.failed && lane == 0) atomicOr(p.status, STATUS_TIMEOUT);
}

} // namespace pd

} // namespace fa
