// Decoding behind a shared prefix for sm_100a: the attention of every sequence's query
// rows to the keys that all of them share, taken as one matrix problem per kv head, and
// its join with the sequences' own parts (paged_decode.cu).
//
//   rows r = (b, h in group, i) of a kv head, R = B G q_len of them;
//   S = mod(Q K^T scale) over the prefix, m = row max, l = sum 2^(S - m),
//   O = 2^(S - m) V;   states (m, l, O) of two key ranges join to
//   m = max(m1, m2), l = l1 2^(m1 - m) + l2 2^(m2 - m), O alike;  out = O / l
//
// K and V of the prefix are read once for up to 256 rows, so the bound goes from HBM
// (few rows) to the tensor cores and the exponentials (4 D flops and one exponential per
// row and key).  A CTA per SM takes an equal share of the list of column entries
// (shared_walk.cuh).  K and V tiles arrive by TMA in one ring.  Two streams, each a tile
// of 128 rows with its own MMA warp and four softmax warps, run half a step apart: while
// one's scores are exponentiated, the other's products are on the tensor cores.  S, P
// (over S) and O live in tensor memory; a thread owns a row.  No key of the prefix is
// masked.  The running maximum moves only when a tile exceeds it by 2^8, so that O is
// rarely rescaled.
#include <mutex>
#include <vector>

#include <cuda_runtime.h>

#include "context.cuh"
#include "dependent_launch.cuh"
#include "flex_fwd.cuh"
#include "flexattn.h"
#include "ptx.cuh"
#include "score_math.cuh"
#include "shared_prefix.cuh"

namespace fa {

namespace {

constexpr int kBox = 16384;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescale = 8.f;       // log2 of the growth that moves the running maximum
constexpr int kLoadWarp = 8, kMmaWarp = 9;
constexpr int kSpThreads = 32 * 11;   // two streams of four softmax warps, loads, two MMA warps

template <int D>
struct SpCfg {
    static constexpr int TILE = 128 * D * 2;              // Q, K or V tile
    static constexpr int NS = D == 128 ? 5 : 12;          // ring slots
    static constexpr int OFF_RING = 2 * TILE;
    static constexpr int SMEM = OFF_RING + NS * TILE + 1024;
    static_assert(SMEM <= 227 * 1024, "shared memory beyond 227 KB per CTA");
    static constexpr uint32_t s_col(int s) { return 128u * s; }   // S, and P over it
    static constexpr uint32_t o_col(int s) { return 256u + 128u * s; }
};

struct __align__(16) SpShared {
    uint64_t full[12], empty[12];
    uint64_t q_full[2], s_full[2], p_full[2], o_full[2], o_empty[2], drain[2];
    uint32_t tmem_base;
};

// Ring positions of an entry's tiles for a stream: K at `k`, V at `v`.
struct SpSeq {
    uint32_t k, v;
};

// The walk of one stream over the CTA's share: `at` the ring position of the entry.
__device__ __forceinline__ uint32_t entry_tiles(const SpGeom& g, const SpPiece& p, int e)
{
    return p.one && 2 * (e + 1) <= g.pages ? 4u : 2u;
}

__device__ __forceinline__ SpSeq entry_seq(const SpGeom& g, const SpPiece& p, int e, int s, uint32_t at)
{
    if (!p.one) return {at, at + 1};
    const bool both = 2 * (e + 1) <= g.pages;
    return {at + s, at + (both ? 2 : 1) + s};
}

template <int D>
__device__ __forceinline__ void load_role(const SpParams& p, SpShared& sh, uint8_t* smem, long long x0, long long x1,
                                          Watchdog& wd)
{
    using C = SpCfg<D>;
    const int lane = threadIdx.x % 32;
    uint32_t seq = 0;
    bool ok = true, bad = false;
    // one tile of K (map tm_k) or V into the next slot
    auto load = [&](const CUtensorMap* tm, int hk, int page) {
        const uint32_t slot = seq % C::NS, use = seq / C::NS;
        ok = ok && __all_sync(0xFFFFFFFFu, mbar_wait(&sh.empty[slot], (use & 1) ^ 1, wd));
        if (!ok) return;
        if (elect_one_sync()) {
            uint8_t* dst = smem + C::OFF_RING + slot * C::TILE;
            mbar_arrive_expect_tx(&sh.full[slot], C::TILE);
#pragma unroll
            for (int c = 0; c < D / 64; ++c) tma_load_4d(dst + c * kBox, tm, &sh.full[slot], c * 64, 0, hk, page);
        }
        __syncwarp();
        ++seq;
    };
    int chunk = -1, page_lane = 0;
    // page t of the prefix
    auto page_at = [&](int t) {
        if (chunk != (t & ~31)) {
            chunk = t & ~31;
            page_lane = chunk + lane < p.geom.pages ? __ldg(p.prefix_row + chunk + lane) : 0;
        }
        return pd_page(__shfl_sync(0xFFFFFFFFu, page_lane, t & 31), p.num_pages, bad);
    };
    for (long long x = x0; ok && x < x1;) {
        const SpPiece pc = sp_piece(p.geom, x, x1);
        for (int e = pc.e0; ok && e < pc.e0 + pc.n; ++e) {
            if (!pc.one) {
                const int page = page_at(e);
                load(&p.tm_k, pc.hk, page);
                load(&p.tm_v, pc.hk, page);
            } else {
                const bool both = 2 * (e + 1) <= p.geom.pages;
                const int a = page_at(2 * e), b = both ? page_at(2 * e + 1) : 0;
                load(&p.tm_k, pc.hk, a);
                if (both) load(&p.tm_k, pc.hk, b);
                load(&p.tm_v, pc.hk, a);
                if (both) load(&p.tm_v, pc.hk, b);
            }
        }
        x += pc.n;
    }
    // copies in flight land before the CTA exits (bounded)
    Watchdog dw{wd.failed ? 1000000ull : wd.limit_ns, false};
    for (uint32_t j = 0; j < (uint32_t)C::NS && j < seq; ++j) {
        const uint32_t last = seq - 1 - j;
        dw.failed = false;
        mbar_wait(&sh.full[last % C::NS], (last / C::NS) & 1, dw);
    }
    if (lane == 0 && (wd.failed || !ok)) atomicOr(p.status, STATUS_TIMEOUT);
    if (__any_sync(0xFFFFFFFFu, bad) && lane == 0) atomicOr(p.status, STATUS_BAD_BLOCKMASK);
}

__device__ __forceinline__ uint64_t desc64(uint32_t hi, uint32_t lo) { return ((uint64_t)hi << 32) | lo; }

template <int D>
__device__ __forceinline__ void mma_role(const SpParams& p, SpShared& sh, uint8_t* smem, uint32_t tmem, int s,
                                         long long x0, long long x1, Watchdog& wd)
{
    using C = SpCfg<D>;
    const uint32_t hi_k = (uint32_t)(sdesc_sw128(0, 16, 1024) >> 32);
    const uint32_t hi_mn = (uint32_t)(sdesc_sw128(0, kBox, 1024) >> 32);
    const uint32_t qd = (uint32_t)sdesc_sw128(smem_u32(smem + s * C::TILE), 16, 1024);
    const uint32_t k0 = (uint32_t)sdesc_sw128(smem_u32(smem + C::OFF_RING), 16, 1024);
    const uint32_t v0 = (uint32_t)sdesc_sw128(smem_u32(smem + C::OFF_RING), kBox, 1024);
    constexpr uint32_t idesc_s = idesc_bf16_f32(128, 128, false, false);
    constexpr uint32_t idesc_o = idesc_bf16_f32(128, D, false, true);
    uint32_t at = 0, tile = 0, piece = 0;
    auto ready = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, wd)); };
    bool ok = true;
    for (long long x = x0; ok && x < x1;) {
        const SpPiece pc = sp_piece(p.geom, x, x1);
        const int n = sp_tiles(p.geom, pc, s);
        if (n > 0) ok = ready(&sh.q_full[s], piece & 1);
        for (int i = 0; ok && i < n; ++i, ++tile) {
            const SpSeq q = entry_seq(p.geom, pc, pc.e0 + i, s, at);
            at += entry_tiles(p.geom, pc, pc.e0 + i);
            const uint32_t ks = q.k % C::NS, vs = q.v % C::NS;
            if (!(ok = ready(&sh.full[ks], (q.k / C::NS) & 1))) break;
            tc_fence_after();
            if (elect_one_sync()) {
                const uint32_t kd = k0 + ks * (uint32_t)(C::TILE >> 4);
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    // 32 bytes per K step inside a 128-byte row, 16 KB per 64 columns
                    const uint32_t off = (uint32_t)(((k / 4) * kBox + (k % 4) * 32) >> 4);
                    umma_ss(tmem + C::s_col(s), desc64(hi_k, qd + off), desc64(hi_k, kd + off), idesc_s, k > 0);
                }
                umma_commit(&sh.empty[ks]);  // two arrivals free a slot: one of each stream, or
                if (pc.one) umma_commit(&sh.empty[ks]);  // both of the one that reads it
                umma_commit(&sh.s_full[s]);
            }
            __syncwarp();
            if (!(ok = ready(&sh.p_full[s], tile & 1))) break;
            if (i == 0 && piece > 0 && !(ok = ready(&sh.o_empty[s], (piece - 1) & 1))) break;
            if (!(ok = ready(&sh.full[vs], (q.v / C::NS) & 1))) break;
            tc_fence_after();
            if (elect_one_sync()) {
                const uint32_t vd = v0 + vs * (uint32_t)(C::TILE >> 4);
#pragma unroll
                for (int k = 0; k < 8; ++k)  // 16 keys (2 KB of V) per K step
                    umma_ts(tmem + C::o_col(s), tmem + C::s_col(s) + 8 * k, desc64(hi_mn, vd + (uint32_t)(k * 128)),
                            idesc_o, (i > 0 || k > 0) ? 1u : 0u);
                umma_commit(&sh.empty[vs]);
                if (pc.one) umma_commit(&sh.empty[vs]);
                if (i + 1 == n) umma_commit(&sh.o_full[s]);
            }
            __syncwarp();
        }
        for (int i = n; i < pc.n; ++i) at += entry_tiles(p.geom, pc, pc.e0 + i);
        if (n > 0) ++piece;
        x += pc.n;
    }
    // the products in flight end before tensor memory is given back (bounded)
    if (elect_one_sync()) umma_commit(&sh.drain[s]);
    __syncwarp();
    Watchdog dw{wd.failed ? 1000000ull : wd.limit_ns, false};
    mbar_wait(&sh.drain[s], 0, dw);
    if ((wd.failed || dw.failed) && threadIdx.x % 32 == 0) atomicOr(p.status, STATUS_TIMEOUT);
}

// P = exp2(x * F + b) of one row (128 scores) as bf16 to TMEM, and its sum.  P is off by
// at most 2^-8 of each entry (the tensor cores' operand type); the sum is taken of the
// unrounded values.
__device__ __forceinline__ float exp_row(const float (&x)[128], float F, float b, uint32_t p_addr)
{
    const uint64_t F2 = f2_pack(F, F), b2 = f2_pack(b, b);
    uint64_t la = f2_pack(0.f, 0.f), lb = la;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        uint32_t pk[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int e = 16 * c + 2 * j;
            float a0, a1;
            f2_unpack(f2_fma(f2_pack(x[e], x[e + 1]), F2, b2), a0, a1);
            const float e0 = ex2_approx(a0), e1 = ex2_approx(a1);
            if (j & 1) lb = f2_add(lb, f2_pack(e0, e1));
            else la = f2_add(la, f2_pack(e0, e1));
            pk[j] = pack_bf16x2(e0, e1);
        }
        tmem_st8(p_addr + 8 * c, pk);
    }
    float l0, l1;
    f2_unpack(f2_add(la, lb), l0, l1);
    return l0 + l1;
}

__device__ __forceinline__ float max_row(const float (&x)[128])
{
    float m[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        m[c] = max3(x[32 * c], x[32 * c + 1], x[32 * c + 2]);
#pragma unroll
        for (int j = 3; j < 31; j += 2) m[c] = max3(m[c], x[32 * c + j], x[32 * c + j + 1]);
        m[c] = fmaxf(m[c], x[32 * c + 31]);
    }
    return max3(m[0], m[1], fmaxf(m[2], m[3]));
}

template <int D, int SCORE>
__device__ __forceinline__ void softmax_role(const SpParams& p, SpShared& sh, uint8_t* smem, uint32_t tmem, int s,
                                             long long x0, long long x1, Watchdog& wd)
{
    using C = SpCfg<D>;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32 % 4, row = 32 * warp + lane;
    const uint32_t lanes = (uint32_t)(32 * warp) << 16;
    const uint32_t s_addr = tmem + C::s_col(s) + lanes, o_addr = tmem + C::o_col(s) + lanes;
    const uint32_t q_base = smem_u32(smem + s * C::TILE);
    uint32_t tile = 0, piece = 0;
    const float F = SCORE == FA_SCORE_SOFTCAP ? p.softcap * kLog2e : SCORE == FA_SCORE_ALIBI ? 1.f : p.scale * kLog2e;
    bool ok = true;
    for (long long x0p = x0; ok && x0p < x1;) {
        const SpPiece pc = sp_piece(p.geom, x0p, x1);
        const int n = sp_tiles(p.geom, pc, s);
        const long long col = (long long)pc.hk * sp_cols(p.geom) + pc.col;
        const long long slot = 2 * (col + blockIdx.x) + s;
        x0p += pc.n;
        float2* ml = reinterpret_cast<float2*>(p.part_ml) + slot * kSpRows + row;
        if (n == 0) {
            *ml = make_float2(-INFINITY, 0.f);
            continue;
        }
        const int first = 2 * kSpRows * pc.col + (pc.one ? 0 : kSpRows * s);  // row of the head
        // Q tile: 16-byte units, D / 8 lanes a row; rows past the last are zero.  The last
        // piece's products have read the tile (their scores were waited for).
#pragma unroll 4
        for (int k = 0; k < D / 8; ++k) {
            const int idx = k * 32 + lane, r = 32 * warp + idx / (D / 8), u = idx % (D / 8);
            const int R = first + r;
            uint4 v = make_uint4(0, 0, 0, 0);
            if (R < p.geom.rows) {
                const int b = R / p.rows, j = R % p.rows;
                v = __ldg(reinterpret_cast<const uint4*>(p.q + (int64_t)b * p.q_st0 +
                                                         (int64_t)(pc.hk * p.G + j / p.q_len) * p.q_st1 +
                                                         (int64_t)(j % p.q_len) * p.q_st2) + u);
            }
            sts128(q_base + (uint32_t)((u >> 3) * kBox + r * 128 + (((u & 7) ^ (r & 7)) << 4)), v.x, v.y, v.z, v.w);
        }
        fence_proxy_async_smem();
        mbar_arrive_warp(&sh.q_full[s]);

        float slope2 = 0.f;
        int pos = 0;
        if (SCORE == FA_SCORE_ALIBI && first + row < p.geom.rows) {
            const int b = (first + row) / p.rows, j = (first + row) % p.rows;
            slope2 = __ldg(p.slopes + pc.hk * p.G + j / p.q_len) * kLog2e;
            pos = __ldg(p.seq_lens + b) - p.q_len + j % p.q_len;
        }
        float m_run = -INFINITY, l_run = 0.f;
        for (int i = 0; i < n; ++i, ++tile) {
            ok = __all_sync(0xFFFFFFFFu, mbar_wait(&sh.s_full[s], tile & 1, wd));
            if (!ok) break;
            tc_fence_after();
            float x[128];
            {
                uint32_t raw[4][32];
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_ld32(s_addr + 32 * c, raw[c]);
                tmem_ld_wait();
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int j = 0; j < 32; ++j) x[32 * c + j] = __uint_as_float(raw[c][j]);
            }
            if constexpr (SCORE == FA_SCORE_ALIBI) {
                const int e = pc.e0 + i, kv0 = 128 * (pc.one ? 2 * e + s : e);
                const float f = p.scale * kLog2e, shift = (float)(kv0 - pos) * slope2;
                const uint64_t f2 = f2_pack(f, f), sl2 = f2_pack(slope2, slope2), sh2 = f2_pack(shift, shift);
#pragma unroll
                for (int j = 0; j < 128; j += 2)
                    f2_unpack(f2_fma(f2_pack(x[j], x[j + 1]), f2,
                                     f2_fma(f2_pack((float)j, (float)(j + 1)), sl2, sh2)), x[j], x[j + 1]);
            }
            if constexpr (SCORE == FA_SCORE_SOFTCAP) {
                // tanh: the polynomial, and per element its far form where a warp's 32
                // columns have one
                const uint64_t in2 = f2_pack(p.softcap_in, p.softcap_in);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    bool far = false;
#pragma unroll
                    for (int j = 32 * c; j < 32 * c + 32; j += 2) {
                        f2_unpack(f2_mul(f2_pack(x[j], x[j + 1]), in2), x[j], x[j + 1]);
                        far |= fmaxf(fabsf(x[j]), fabsf(x[j + 1])) > kTanhPolyMax;
                    }
                    const bool any = __any_sync(0xFFFFFFFFu, far);
#pragma unroll
                    for (int j = 32 * c; j < 32 * c + 32; j += 2) {
                        float t0, t1;
                        f2_unpack(tanh_poly2(f2_pack(x[j], x[j + 1])), t0, t1);
                        if (any) {
                            if (fabsf(x[j]) > kTanhPolyMax) t0 = tanh_far(x[j]);
                            if (fabsf(x[j + 1]) > kTanhPolyMax) t1 = tanh_far(x[j + 1]);
                        }
                        x[j] = t0;
                        x[j + 1] = t1;
                    }
                }
            }
            const float m_tile = max_row(x) * F;
            float alpha = 1.f;
            bool rescale = false;
            if (i == 0) {
                m_run = m_tile;
            } else if (m_tile > m_run + kRescale) {
                alpha = ex2_approx(m_run - m_tile);
                m_run = m_tile;
                l_run *= alpha;
                rescale = true;
            }
            l_run += exp_row(x, F, m_run == -INFINITY ? 0.f : -m_run, s_addr);
            if (__any_sync(0xFFFFFFFFu, rescale)) {
                // O is stable: this tile's scores were issued after the last tile's P V
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t ov[32];
                    tmem_ld32(o_addr + 32 * c, ov);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 32; ++j) ov[j] = __float_as_uint(__uint_as_float(ov[j]) * alpha);
                    tmem_st32(o_addr + 32 * c, ov);
                }
            }
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive_warp(&sh.p_full[s]);
        }
        if (!ok) break;
        ok = __all_sync(0xFFFFFFFFu, mbar_wait(&sh.o_full[s], piece & 1, wd));
        if (!ok) break;
        ++piece;
        tc_fence_after();
        *ml = make_float2(m_run, l_run);
        float4* dst = reinterpret_cast<float4*>(p.part_o) + (slot * (D / 8) * kSpRows + row) * 2;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
            uint32_t ov[32];
            tmem_ld32(o_addr + 32 * c, ov);
            tmem_ld_wait();
            if (c == D / 32 - 1) {
                tc_fence_before();
                mbar_arrive_warp(&sh.o_empty[s]);
            }
#pragma unroll
            for (int u = 0; u < 8; ++u)
                dst[((4 * c + u / 2) * kSpRows) * 2 + u % 2] =
                    make_float4(__uint_as_float(ov[4 * u]), __uint_as_float(ov[4 * u + 1]),
                                __uint_as_float(ov[4 * u + 2]), __uint_as_float(ov[4 * u + 3]));
        }
    }
    if (wd.failed && lane == 0) atomicOr(p.status, STATUS_TIMEOUT);
}

template <int D, int SCORE>
__global__ void __launch_bounds__(kSpThreads, 1) shared_prefix_kernel(const __grid_constant__ SpParams p)
{
    using C = SpCfg<D>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ SpShared sh;
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x / 32;
    launch_dependents();
    if (warp == kMmaWarp) {
        tmem_alloc(&sh.tmem_base, 512);
        tmem_relinquish();
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(&sh.q_full[s], 4);
            mbar_init(&sh.s_full[s], 1);
            mbar_init(&sh.p_full[s], 4);
            mbar_init(&sh.o_full[s], 1);
            mbar_init(&sh.o_empty[s], 4);
            mbar_init(&sh.drain[s], 1);
        }
        for (int i = 0; i < C::NS; ++i) {
            mbar_init(&sh.full[i], 1);
            mbar_init(&sh.empty[i], 2);
        }
        mbar_fence_init();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem_base;
    const long long T = (long long)p.Hkv * p.geom.per_head;
    const long long x0 = pd_share(T, blockIdx.x, p.used), x1 = pd_share(T, blockIdx.x + 1, p.used);
    Watchdog wd{p.watchdog_ns, false};
    if (warp < 8) softmax_role<D, SCORE>(p, sh, smem, tmem, warp / 4, x0, x1, wd);
    else if (warp == kLoadWarp) load_role<D>(p, sh, smem, x0, x1, wd);
    else mma_role<D>(p, sh, smem, tmem, warp - kMmaWarp, x0, x1, wd);
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

// The join: eight columns of a row a thread.  The prefix's pieces in list order, then the
// row's own part, whatever finished first.  Sequences that take no part in the sharing
// were written by the paged decode.
constexpr int kJoinThreads = 256;

template <int D>
__global__ void __launch_bounds__(kJoinThreads) shared_join_kernel(const __grid_constant__ SpParams p)
{
    wait_prerequisites();
    const long long t = (long long)blockIdx.x * kJoinThreads + threadIdx.x;
    const int u = (int)(t % (D / 8));
    const long long row = t / (D / 8);  // of [B][Hkv][rows]
    if (row >= (long long)p.B * p.Hkv * p.rows) return;
    const int j = (int)(row % p.rows), hk = (int)(row / p.rows % p.Hkv), b = (int)(row / p.rows / p.Hkv);
    const int64_t len = __ldg(p.seq_lens + b);
    if (len > (int64_t)p.pt_width * 128 ? (int64_t)p.pt_width * 128 - p.q_len < (int64_t)p.geom.pages * 128
                                        : len - p.q_len < (int64_t)p.geom.pages * 128)
        return;
    float M = -INFINITY, L = 0.f, v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    auto take = [&](float2 ml, const float4* o) {
        if (ml.x == -INFINITY && ml.y == 0.f) return;  // no key (its O may be unwritten)
        const float4 a = o[0], c = o[1];
        const float Mn = fmaxf(M, ml.x), Mu = Mn == -INFINITY ? 0.f : Mn;
        const float f0 = ex2_approx(M - Mu), f1 = ex2_approx(ml.x - Mu);
        M = Mn;
        L = fmaf(ml.y, f1, L * f0);
        const float w[8] = {a.x, a.y, a.z, a.w, c.x, c.y, c.z, c.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = fmaf(w[e], f1, v[e] * f0);
    };
    const int R = b * p.rows + j, col = R / (2 * kSpRows);
    const bool one = col >= p.geom.pairs;
    const int s0 = one ? 0 : R % (2 * kSpRows) / kSpRows, s1 = one ? 1 : s0;
    const long long T = (long long)p.Hkv * p.geom.per_head, start = sp_start(p.geom, hk, col);
    const int entries = one ? (p.geom.pages + 1) / 2 : p.geom.pages;
    const int c0 = pd_holder(T, start, p.used), c1 = pd_holder(T, start + entries - 1, p.used);
    const long long base = (long long)hk * sp_cols(p.geom) + col;
    for (int c = c0; c <= c1; ++c)
        for (int s = s0; s <= s1; ++s) {
            const long long slot = 2 * (base + c) + s;
            take(reinterpret_cast<const float2*>(p.part_ml)[slot * kSpRows + R % kSpRows],
                 reinterpret_cast<const float4*>(p.part_o) +
                     (slot * (D / 8) * kSpRows + u * kSpRows + R % kSpRows) * 2);
        }
    take(reinterpret_cast<const float2*>(p.own_ml)[row], reinterpret_cast<const float4*>(p.own_o + row * D) + 2 * u);
    const int hq = hk * p.G + j / p.q_len, i = j % p.q_len;
    const bool some = L > 0.f && M != -INFINITY;
    const float inv = some ? 1.f / L : L != L ? L : 0.f;
    uint16_t* o = p.o + (int64_t)b * p.o_st0 + (int64_t)hq * p.o_st1 + (int64_t)i * p.o_st2 + 8 * u;
    *reinterpret_cast<uint4*>(o) =
        inv != 0.f ? make_uint4(pack_bf16x2(v[0] * inv, v[1] * inv), pack_bf16x2(v[2] * inv, v[3] * inv),
                                pack_bf16x2(v[4] * inv, v[5] * inv), pack_bf16x2(v[6] * inv, v[7] * inv))
                   : make_uint4(0u, 0u, 0u, 0u);
    if (u == 0 && p.lse)
        p.lse[((int64_t)b * p.Hkv * p.G + hq) * p.q_len + i] = some ? (M + __log2f(L)) * kLn2 : L != L ? L : -INFINITY;
}

template <int D, int SCORE>
cudaError_t launch_variant(const SpParams& p, cudaStream_t stream)
{
    static std::mutex mu;
    static std::vector<CtxKey> done;
    auto kern = shared_prefix_kernel<D, SCORE>;
    {
        CtxKey key;
        std::lock_guard<std::mutex> lock(mu);
        bool have = false;
        if (current_ctx(&key))
            for (const CtxKey& k : done) have |= k == key;
        if (!have) {
            cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SpCfg<D>::SMEM);
            if (e != cudaSuccess) return e;
            if (current_ctx(&key)) done.push_back(key);
        }
    }
    kern<<<(unsigned)p.used, kSpThreads, SpCfg<D>::SMEM, stream>>>(p);
    return cudaGetLastError();
}

} // namespace

cudaError_t launch_shared_prefix(const SpParams& p, int D, int score_kind, cudaStream_t stream)
{
#define FA_SP_CASE(DD, SS) \
    if (D == DD && score_kind == SS) return launch_variant<DD, SS>(p, stream);
    FA_SP_CASE(64, FA_SCORE_NONE) FA_SP_CASE(64, FA_SCORE_ALIBI) FA_SP_CASE(64, FA_SCORE_SOFTCAP)
    FA_SP_CASE(128, FA_SCORE_NONE) FA_SP_CASE(128, FA_SCORE_ALIBI) FA_SP_CASE(128, FA_SCORE_SOFTCAP)
#undef FA_SP_CASE
    return cudaErrorInvalidValue;
}

cudaError_t launch_shared_join(const SpParams& p, int D, cudaStream_t stream)
{
    const long long threads = (long long)p.B * p.Hkv * p.rows * (D / 8);
    const dim3 grid((unsigned)((threads + kJoinThreads - 1) / kJoinThreads));
    return D == 64 ? launch_after(shared_join_kernel<64>, grid, kJoinThreads, 0, stream, p)
                   : launch_after(shared_join_kernel<128>, grid, kJoinThreads, 0, stream, p);
}

} // namespace fa
