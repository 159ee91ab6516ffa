// Decoding behind a shared prefix for sm_100a: the attention of every sequence's query
// rows to the keys that all of them share, taken as one matrix problem per kv head,
// beside the sequences' own parts (paged_decode_impl.cuh), and the join of both.
//
//   rows r = (b, h in group, i) of a kv head, R = B G q_len of them;
//   S = mod(Q K^T scale) over the prefix, m = row max, l = sum 2^(S - m),
//   O = 2^(S - m) V;   states (m, l, O) of two key ranges join to
//   m = max(m1, m2), l = l1 2^(m1 - m) + l2 2^(m2 - m), O alike;  out = O / l
//
// K and V of the prefix are read once for up to 256 rows, so the bound goes from HBM
// (few rows) to the tensor cores and the exponentials (4 D flops and one exponential per
// row and key).  CTA c of those that the prefix gets takes the c-th equal share of the
// list of column entries (shared_walk.cuh); the other SMs run the paged decode of the
// sequences' own pages, which is bound by HBM, meanwhile.
//
// K and V tiles arrive by TMA in one ring.  Two streams, each a tile of 128 rows with its
// own MMA warp and four softmax warps, share the tensor cores and the exponential units.
// S, P (over S) and O live in tensor memory; a thread owns a row.  A tile is taken in
// halves of 64 keys with a buffer each: while one half's scores are exponentiated, the
// other's P V and the scores of the half after it are on the tensor cores.  No key of the
// prefix is masked.  The running maximum moves only when a half exceeds it by 2^8, so that
// O is rarely rescaled.
//
// Measured on a B200, 128 sequences behind 16384 shared keys, Hq 32 Hkv 8 D 128, own parts of
// 128 to 777 keys: 82.6 us a call, 74 of them the kernel and 11 the join (under ncu).  A pair
// of tiles takes 3330 cycles, of which the products need 2050 (whole tiles with one buffer:
// 4280): 1.4 PFLOP/s over the prefix alone with all SMs.  Without the exponentials it would be
// 3200, without the products 2900, and 1750 with nothing but the barriers; a quarter of the
// exponentials by polynomial changed nothing.  One kernel after the other, each on all SMs,
// took 104 us (cold caches), side by side 96, in one kernel with the split by cost 80.
#include <mutex>
#include <vector>

#include <cuda_runtime.h>

#include "context.cuh"
#include "dependent_launch.cuh"
#include "paged_decode_impl.cuh"
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
    static constexpr uint32_t s_col(int s, int h) { return 128u * s + 64u * h; }  // S of 64 keys, and P over it
    static constexpr uint32_t o_col(int s) { return 256u + 128u * s; }
};

// Of the kernel, whose CTAs do one or the other.
template <int D>
struct SharedSmem {
    static constexpr int BYTES = SpCfg<D>::SMEM > pd::Cfg<D>::SMEM ? SpCfg<D>::SMEM : pd::Cfg<D>::SMEM;
};

struct __align__(16) SpShared {
    uint64_t full[12], empty[12];
    uint64_t q_full[2], s_full[2][2], p_full[2][2], pv_done[2], o_full[2], o_empty[2], drain[2];
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
__device__ __forceinline__ void load_role(const SpParams& p, SpShared& sh, uint8_t* smem, int x0, int x1,
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
            page_lane = chunk + lane < p.geom.pages ? p.prefix_row[chunk + lane] : 0;
        }
        return pd_page(__shfl_sync(0xFFFFFFFFu, page_lane, t & 31), p.num_pages, bad);
    };
    for (int x = x0; ok && x < x1;) {
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

template <int D, int s>
__device__ __forceinline__ void mma_role(const SpParams& p, SpShared& sh, uint8_t* smem, uint32_t tmem, int x0,
                                         int x1, Watchdog& wd)
{
    using C = SpCfg<D>;
    const uint32_t hi_k = (uint32_t)(sdesc_sw128(0, 16, 1024) >> 32);
    const uint32_t hi_mn = (uint32_t)(sdesc_sw128(0, kBox, 1024) >> 32);
    const uint32_t qd = (uint32_t)sdesc_sw128(smem_u32(smem + s * C::TILE), 16, 1024);
    const uint32_t k0 = (uint32_t)sdesc_sw128(smem_u32(smem + C::OFF_RING), 16, 1024);
    const uint32_t v0 = (uint32_t)sdesc_sw128(smem_u32(smem + C::OFF_RING), kBox, 1024);
    constexpr uint32_t idesc_s = idesc_bf16_f32(128, 64, false, false);
    constexpr uint32_t idesc_o = idesc_bf16_f32(128, D, false, true);
    constexpr uint32_t kHalf = 8192 >> 4;  // 64 keys of a 64-column box, in descriptor units
    uint32_t at = 0, tile = 0, piece = 0;
    bool ok = true;
    auto ready = [&](uint64_t* bar, uint32_t parity) {
        return ok = ok && __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, wd));
    };
    // A slot is free after an arrival of each stream.  In a column of one tile a stream
    // passes over the other's tiles: it waits for them too, since a barrier's parity tells
    // only its last phase and none may be skipped.
    auto pass = [&](uint32_t pos) {
        if (ready(&sh.full[pos % C::NS], (pos / C::NS) & 1) && elect_one_sync()) mbar_arrive(&sh.empty[pos % C::NS]);
        __syncwarp();
    };
    // S of one half of a tile whose K has landed
    auto scores = [&](uint32_t kpos, int h) {
        const uint32_t slot = kpos % C::NS, kd = k0 + slot * (uint32_t)(C::TILE >> 4) + h * kHalf;
        tc_fence_after();
        if (elect_one_sync()) {
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                // 32 bytes per K step inside a 128-byte row, 16 KB per 64 columns
                const uint32_t off = (uint32_t)(((k / 4) * kBox + (k % 4) * 32) >> 4);
                umma_ss(tmem + C::s_col(s, h), desc64(hi_k, qd + off), desc64(hi_k, kd + off), idesc_s, k > 0);
            }
            umma_commit(&sh.s_full[s][h]);
            if (h == 1) umma_commit(&sh.empty[slot]);
        }
        __syncwarp();
    };
    // O += P V of one half
    auto values = [&](uint32_t vpos, int h, uint32_t accumulate, bool last) {
        const uint32_t slot = vpos % C::NS, vd = v0 + slot * (uint32_t)(C::TILE >> 4) + h * kHalf;
        tc_fence_after();
        if (elect_one_sync()) {
#pragma unroll
            for (int k = 0; k < 4; ++k)  // 16 keys (2 KB of V) per K step
                umma_ts(tmem + C::o_col(s), tmem + C::s_col(s, h) + 8 * k, desc64(hi_mn, vd + (uint32_t)(k * 128)),
                        idesc_o, k > 0 ? 1u : accumulate);
            umma_commit(&sh.pv_done[s]);
            if (h == 1) umma_commit(&sh.empty[slot]);
            if (last) umma_commit(&sh.o_full[s]);
        }
        __syncwarp();
    };
    for (int x = x0; ok && x < x1;) {
        const SpPiece pc = sp_piece(p.geom, x, x1);
        const int n = sp_tiles(p.geom, pc, s);
        if (n > 0) {
            SpSeq cur = entry_seq(p.geom, pc, pc.e0, s, at);
            if (ready(&sh.q_full[s], piece & 1) && ready(&sh.full[cur.k % C::NS], (cur.k / C::NS) & 1)) {
                scores(cur.k, 0);
                scores(cur.k, 1);
            }
            for (int i = 0; ok && i < n; ++i, ++tile) {
                const uint32_t tiles = entry_tiles(p.geom, pc, pc.e0 + i);
                const bool both = pc.one && tiles == 4;  // the other stream has a tile of this entry
                // its K before the next K is waited for, which may go to that slot
                if (both) pass(at + 1 - s);
                at += tiles;
                const SpSeq nx = entry_seq(p.geom, pc, pc.e0 + i + 1, s, at);
                const bool more = i + 1 < n;
                ready(&sh.full[cur.v % C::NS], (cur.v / C::NS) & 1);
                if (!ready(&sh.p_full[s][0], tile & 1)) break;
                if (i == 0 && piece > 0 && !ready(&sh.o_empty[s], (piece - 1) & 1)) break;
                values(cur.v, 0, i > 0 ? 1u : 0u, false);
                if (more && !ready(&sh.full[nx.k % C::NS], (nx.k / C::NS) & 1)) break;
                if (more) scores(nx.k, 0);
                if (!ready(&sh.p_full[s][1], tile & 1)) break;
                values(cur.v, 1, 1u, !more);
                if (more) scores(nx.k, 1);
                if (both) pass(at - 1 - s);
                cur = nx;
            }
            ++piece;
        }
        if (ok && n < pc.n) {  // the last entry is the other stream's alone
            pass(at);
            pass(at + 1);
            at += 2;
        }
        x += pc.n;
    }
    // the products in flight end before tensor memory is given back (bounded)
    if (elect_one_sync()) umma_commit(&sh.drain[s]);
    __syncwarp();
    Watchdog dw{wd.failed ? 1000000ull : wd.limit_ns, false};
    mbar_wait(&sh.drain[s], 0, dw);
    if ((wd.failed || dw.failed) && threadIdx.x % 32 == 0) atomicOr(p.status, STATUS_TIMEOUT);
}

// P = exp2(x * F + b) of half a tile's row (64 scores) as bf16 to TMEM, and its sum.  P is
// off by at most 2^-8 of each entry (the tensor cores' operand type); the sum is taken of
// the unrounded values.
__device__ __forceinline__ float exp_row(const float (&x)[64], float F, float b, uint32_t p_addr)
{
    const uint64_t F2 = f2_pack(F, F), b2 = f2_pack(b, b);
    uint64_t la = f2_pack(0.f, 0.f), lb = la;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        uint32_t pk[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const int e = 32 * c + 2 * j;
            float a0, a1;
            f2_unpack(f2_fma(f2_pack(x[e], x[e + 1]), F2, b2), a0, a1);
            const float e0 = ex2_approx(a0), e1 = ex2_approx(a1);
            if (j & 1) lb = f2_add(lb, f2_pack(e0, e1));
            else la = f2_add(la, f2_pack(e0, e1));
            pk[j] = pack_bf16x2(e0, e1);
        }
        tmem_st16(p_addr + 16 * c, pk);
    }
    float l0, l1;
    f2_unpack(f2_add(la, lb), l0, l1);
    return l0 + l1;
}

__device__ __forceinline__ float max_row(const float (&x)[64])
{
    float m[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        m[c] = max3(x[16 * c], x[16 * c + 1], x[16 * c + 2]);
#pragma unroll
        for (int j = 3; j < 15; j += 2) m[c] = max3(m[c], x[16 * c + j], x[16 * c + j + 1]);
        m[c] = fmaxf(m[c], x[16 * c + 15]);
    }
    return max3(m[0], m[1], fmaxf(m[2], m[3]));
}

template <int D, int SCORE>
__device__ __forceinline__ void softmax_role(const SpParams& p, SpShared& sh, uint8_t* smem, uint32_t tmem, int s,
                                             int x0, int x1, Watchdog& wd)
{
    using C = SpCfg<D>;
    constexpr int U = D / 8;  // 16-byte units of a row
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32 % 4, row = 32 * warp + lane;
    const uint32_t lanes = (uint32_t)(32 * warp) << 16;
    const uint32_t o_addr = tmem + C::o_col(s) + lanes;
    const uint32_t q_base = smem_u32(smem + s * C::TILE);
    uint32_t tile = 0, piece = 0;
    const float F = SCORE == FA_SCORE_SOFTCAP ? p.softcap * kLog2e : SCORE == FA_SCORE_ALIBI ? 1.f : p.scale * kLog2e;
    bool ok = true;
    for (int x0p = x0; ok && x0p < x1;) {
        const SpPiece pc = sp_piece(p.geom, x0p, x1);
        const int n = sp_tiles(p.geom, pc, s);
        const long long col = (long long)pc.hk * sp_cols(p.geom) + pc.col;
        const long long slot = 2 * (col + blockIdx.x) + s;
        x0p += pc.n;
        float2* ml = reinterpret_cast<float2*>(p.part_ml) + slot * kSpRows + row;
        float4* dst = reinterpret_cast<float4*>(p.part_o) + slot * (D / 4) * kSpRows + row;
        if (n == 0) {
            *ml = make_float2(-INFINITY, 0.f);
            for (int c = 0; c < D / 4; ++c) dst[c * kSpRows] = make_float4(0.f, 0.f, 0.f, 0.f);
            continue;
        }
        // Q tile; rows past the last are zero.  The last piece's products have read the
        // tile (their end was waited for).
        const int R = 2 * kSpRows * pc.col + (pc.one ? 0 : kSpRows * s) + row;  // the thread's row of the head
        const bool valid = R < p.geom.rows;
        const int b = valid ? R / p.rows : 0, j = valid ? R - b * p.rows : 0, g = j / p.q_len, qi = j - g * p.q_len;
        const unsigned long long mine =
            valid ? reinterpret_cast<unsigned long long>(p.q + (int64_t)b * p.q_st0 +
                                                         (int64_t)(pc.hk * p.G + g) * p.q_st1 + (int64_t)qi * p.q_st2)
                  : 0ull;
        uint4 v[U];  // all loads in flight at once, ahead of the K and V tiles' traffic
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int idx = k * 32 + lane;
            const unsigned long long src = __shfl_sync(0xFFFFFFFFu, mine, idx / U);
            v[k] = src ? reinterpret_cast<const uint4*>(src)[idx % U] : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int idx = k * 32 + lane, r = 32 * warp + idx / U, u = idx % U;
            sts128(q_base + (uint32_t)((u >> 3) * kBox + r * 128 + (((u & 7) ^ (r & 7)) << 4)), v[k].x, v[k].y, v[k].z,
                   v[k].w);
        }
        fence_proxy_async_smem();
        mbar_arrive_warp(&sh.q_full[s]);

        float slope2 = 0.f;
        int pos = 0;
        if (SCORE == FA_SCORE_ALIBI && valid) {
            slope2 = p.slopes[pc.hk * p.G + g] * kLog2e;
            pos = pd_length(p, p.seq_lens[b]) - p.q_len + qi;
        }
        float m_run = -INFINITY, l_run = 0.f;
        // a warp without rows only passes the barriers on (its rows of P and O are nobody's)
        const bool rows = __any_sync(0xFFFFFFFFu, valid);
        for (int i = 0; ok && i < n; ++i, ++tile) {
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
                const uint32_t s_addr = tmem + C::s_col(s, h) + lanes;
                ok = __all_sync(0xFFFFFFFFu, mbar_wait(&sh.s_full[s][h], tile & 1, wd));
                if (!ok) break;
                if (!rows) {
                    mbar_arrive_warp(&sh.p_full[s][h]);
                    continue;
                }
                tc_fence_after();
                float x[64];
                {
                    uint32_t raw[2][32];
#pragma unroll
                    for (int c = 0; c < 2; ++c) tmem_ld32(s_addr + 32 * c, raw[c]);
                    tmem_ld_wait();
#pragma unroll
                    for (int c = 0; c < 2; ++c)
#pragma unroll
                        for (int k = 0; k < 32; ++k) x[32 * c + k] = __uint_as_float(raw[c][k]);
                }
                if constexpr (SCORE == FA_SCORE_ALIBI) {
                    const int e = pc.e0 + i, kv0 = 128 * (pc.one ? 2 * e + s : e) + 64 * h;
                    const float f = p.scale * kLog2e, shift = (float)(kv0 - pos) * slope2;
                    const uint64_t f2 = f2_pack(f, f), sl2 = f2_pack(slope2, slope2), sh2 = f2_pack(shift, shift);
#pragma unroll
                    for (int k = 0; k < 64; k += 2)
                        f2_unpack(f2_fma(f2_pack(x[k], x[k + 1]), f2,
                                         f2_fma(f2_pack((float)k, (float)(k + 1)), sl2, sh2)), x[k], x[k + 1]);
                }
                if constexpr (SCORE == FA_SCORE_SOFTCAP) {
                    // tanh: the polynomial, and per element its far form where a warp's 32
                    // columns have one
                    const uint64_t in2 = f2_pack(p.softcap_in, p.softcap_in);
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        bool far = false;
#pragma unroll
                        for (int k = 32 * c; k < 32 * c + 32; k += 2) {
                            f2_unpack(f2_mul(f2_pack(x[k], x[k + 1]), in2), x[k], x[k + 1]);
                            far |= fmaxf(fabsf(x[k]), fabsf(x[k + 1])) > kTanhPolyMax;
                        }
                        const bool any = __any_sync(0xFFFFFFFFu, far);
#pragma unroll
                        for (int k = 32 * c; k < 32 * c + 32; k += 2) {
                            float t0, t1;
                            f2_unpack(tanh_poly2(f2_pack(x[k], x[k + 1])), t0, t1);
                            if (any) {
                                if (fabsf(x[k]) > kTanhPolyMax) t0 = tanh_far(x[k]);
                                if (fabsf(x[k + 1]) > kTanhPolyMax) t1 = tanh_far(x[k + 1]);
                            }
                            x[k] = t0;
                            x[k + 1] = t1;
                        }
                    }
                }
                const float m_half = max_row(x) * F;
                float alpha = 1.f;
                bool rescale = false;
                if (i == 0 && h == 0) {
                    m_run = m_half;
                } else if (m_half > m_run + kRescale) {
                    alpha = ex2_approx(m_run - m_half);
                    m_run = m_half;
                    l_run *= alpha;
                    rescale = true;
                }
                l_run += exp_row(x, F, m_run == -INFINITY ? 0.f : -m_run, s_addr);
                if (__any_sync(0xFFFFFFFFu, rescale)) {
                    // O is stable once the P V before this half's is done.  The phase before
                    // that one has ended: this half's scores were issued after its P V.
                    ok = __all_sync(0xFFFFFFFFu, mbar_wait(&sh.pv_done[s], (2 * tile + h - 1) & 1, wd));
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t ov[32];
                        tmem_ld32(o_addr + 32 * c, ov);
                        tmem_ld_wait();
#pragma unroll
                        for (int k = 0; k < 32; ++k) ov[k] = __float_as_uint(__uint_as_float(ov[k]) * alpha);
                        tmem_st32(o_addr + 32 * c, ov);
                    }
                }
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive_warp(&sh.p_full[s][h]);
            }
        }
        if (!ok) break;
        // The piece's products are done.  (Not by pv_done: whether its last phase or the one
        // before it has ended, its parity cannot tell here.)
        ok = __all_sync(0xFFFFFFFFu, mbar_wait(&sh.o_full[s], piece & 1, wd));
        if (!ok) break;
        ++piece;
        tc_fence_after();
        if (valid) *ml = make_float2(m_run, l_run);
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
            uint32_t ov[32];
            tmem_ld32(o_addr + 32 * c, ov);
            tmem_ld_wait();
            if (c == D / 32 - 1) {
                tc_fence_before();
                mbar_arrive_warp(&sh.o_empty[s]);
            }
#pragma unroll
            for (int u = 0; u < 8 && valid; ++u)
                dst[(8 * c + u) * kSpRows] = make_float4(__uint_as_float(ov[4 * u]), __uint_as_float(ov[4 * u + 1]),
                                                         __uint_as_float(ov[4 * u + 2]), __uint_as_float(ov[4 * u + 3]));
        }
    }
    if (wd.failed && lane == 0) atomicOr(p.status, STATUS_TIMEOUT);
}

// CTA `block` of `ctas` that take the prefix.
template <int D, int SCORE>
__device__ __forceinline__ void prefix_cta(const SpParams& p, SpShared& sh, uint8_t* smem, int block, int ctas)
{
    using C = SpCfg<D>;
    const int warp = threadIdx.x / 32;
    if (warp == kMmaWarp) {
        tmem_alloc(&sh.tmem_base, 512);
        tmem_relinquish();
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(&sh.q_full[s], 4);
            for (int h = 0; h < 2; ++h) {
                mbar_init(&sh.s_full[s][h], 1);
                mbar_init(&sh.p_full[s][h], 4);
            }
            mbar_init(&sh.pv_done[s], 1);
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
    const int T = p.Hkv * p.geom.per_head, x0 = pd_share(T, block, ctas), x1 = pd_share(T, block + 1, ctas);
    Watchdog wd{p.watchdog_ns, false};
    if (warp < 8) softmax_role<D, SCORE>(p, sh, smem, tmem, warp / 4, x0, x1, wd);
    else if (warp == kLoadWarp) load_role<D>(p, sh, smem, x0, x1, wd);
    else if (warp == kMmaWarp) mma_role<D, 0>(p, sh, smem, tmem, x0, x1, wd);
    else mma_role<D, 1>(p, sh, smem, tmem, x0, x1, wd);
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

// The first CTAs take the prefix, the others the sequences' own pages; how many each from
// the lengths, on every CTA alike.
template <int D, int SCORE, int NR>
__global__ void __launch_bounds__(kSpThreads, 1)
shared_decode_kernel(const __grid_constant__ SpParams p, const __grid_constant__ PdParams own)
{
    extern __shared__ uint8_t smem_raw[];
    union State {
        SpShared sp;
        pd::Shared pd;
    };
    __shared__ __align__(16) uint8_t state[sizeof(State)];
    __shared__ long long scratch[kSpThreads / 32];
    static_assert(SharedSmem<D>::BYTES + sizeof(state) + sizeof(scratch) <= 227 * 1024,
                  "shared memory beyond 227 KB per CTA");
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    wait_prerequisites();
    launch_dependents();
    bool bad = false;
    const pd::Scan scan = pd::scan_lengths<kSpThreads>(own, scratch, bad);
    // An entry's softmax takes twice as long with the soft cap's tanh.  Entries at 16 / at 32
    // with it, us on a B200 with cold caches: 53.4 / 40.0 (B64 Hkv8 G4 D128, 4096 shared keys),
    // 77.5 / 53.4 (B64 Hkv16, 6 rows, D64, 4608), 40.7 / 43.9 (B40 Hkv4, 16 rows, D64, 8192).
    constexpr int kEntryCost = SCORE == FA_SCORE_SOFTCAP ? 32 : 16;
    const int ctas = sp_split(p.Hkv * p.geom.per_head, p.Hkv * sp_cols(p.geom), pd::Scan::pages(scan.total) * p.Hkv,
                              pd::Scan::sequences(scan.total) * p.Hkv, gridDim.x, kEntryCost);
    if ((int)blockIdx.x < ctas) {
        if (blockIdx.x == 0 && threadIdx.x == 0) *p.split = ctas;
        prefix_cta<D, SCORE>(p, reinterpret_cast<State*>(state)->sp, smem, blockIdx.x, ctas);
    } else {
        pd::decode_cta<D, SCORE, NR, kSpThreads>(own, reinterpret_cast<State*>(state)->pd, smem, blockIdx.x - ctas,
                                                 gridDim.x - ctas, scan, bad);
    }
}

// The join: a lane a row and a warp four columns of 32, so that the partial results are
// read in whole lines; no load waits for another part's.  The prefix's pieces come in
// list order, then the row's own part, whatever finished first.  Sequences that take no
// part in the sharing were written by the paged decode.
constexpr int kJoinWarps = 8, kJoinCols = 4 * kJoinWarps;

template <int D>
__global__ void __launch_bounds__(32 * kJoinWarps) shared_join_kernel(const __grid_constant__ SpParams p)
{
    __shared__ uint2 out[32][kJoinWarps + 1];
    __shared__ int64_t where[32];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int hk = blockIdx.y, R = blockIdx.x * 32 + lane;
    const int c4 = blockIdx.z * kJoinWarps + warp;  // the four columns
    const bool in = R < p.geom.rows;
    const int b = in ? R / p.rows : 0, j = in ? R - b * p.rows : 0;
    const int hq = hk * p.G + j / p.q_len, i = j % p.q_len;
    const int col = R / (2 * kSpRows), r = R % kSpRows;  // the same column and tile in all lanes
    const bool one = col >= p.geom.pairs;
    const int s0 = one ? 0 : R % (2 * kSpRows) / kSpRows;
    const int T = p.Hkv * p.geom.per_head, start = sp_start(p.geom, hk, col);
    const int entries = one ? (p.geom.pages + 1) / 2 : p.geom.pages;
    wait_prerequisites();
    const int used = *p.split;
    const bool takes = in && (int64_t)pd_length(p, p.seq_lens[b]) - p.q_len >= (int64_t)p.geom.pages * 128;
    const int c0 = pd_holder(T, start, used), c1 = pd_holder(T, start + entries - 1, used);
    const int parts = (c1 - c0 + 1) * (one ? 2 : 1);
    const int64_t step = one ? 1 : 2;  // slots from a part to the next
    const int64_t slot0 = 2 * ((int64_t)hk * sp_cols(p.geom) + col + c0) + s0;
    const float2* ml = reinterpret_cast<const float2*>(p.part_ml) + slot0 * kSpRows + r;
    const float4* po = reinterpret_cast<const float4*>(p.part_o) + (slot0 * (D / 4) + c4) * kSpRows + r;
    const int64_t own = ((int64_t)b * p.Hkv + hk) * p.rows + j;
    float M = -INFINITY, L = 0.f, v[4] = {0.f, 0.f, 0.f, 0.f};
    if (takes) {
        const float2 last = reinterpret_cast<const float2*>(p.own_ml)[own];
        const float4 x = reinterpret_cast<const float4*>(p.own_o + own * D)[c4];
        auto take = [&](float2 w, float4 y) {
            const float m = fmaxf(M, w.x), Mu = m == -INFINITY ? 0.f : m;
            const float f0 = ex2_approx(M - Mu), f = ex2_approx(w.x - Mu);
            M = m;
            L = fmaf(w.y, f, L * f0);
            v[0] = fmaf(y.x, f, v[0] * f0);
            v[1] = fmaf(y.y, f, v[1] * f0);
            v[2] = fmaf(y.z, f, v[2] * f0);
            v[3] = fmaf(y.w, f, v[3] * f0);
        };
        // Parts whose loads are issued together (which an unrolled loop alone does not bring
        // about: 5 sequences of 16 rows behind 300 shared pages 79.8 us, so 60.2; by four parts,
        // which leave the kernel 60 registers instead of 85, 82.5).
        constexpr int U = 8;
        for (int k = 0; k < parts; k += U) {
            float2 w[U];
            float4 y[U];
#pragma unroll
            for (int i = 0; i < U; ++i)
                if (k + i < parts) {
                    w[i] = ml[(k + i) * step * kSpRows];
                    y[i] = po[(k + i) * step * (D / 4) * kSpRows];
                }
#pragma unroll
            for (int i = 0; i < U; ++i)
                if (k + i < parts) take(w[i], y[i]);
        }
        take(last, x);
    }
    const bool some = L > 0.f && M != -INFINITY;
    const float inv = some ? 1.f / L : L != L ? L : 0.f;
    out[lane][warp] = inv != 0.f ? make_uint2(pack_bf16x2(v[0] * inv, v[1] * inv), pack_bf16x2(v[2] * inv, v[3] * inv))
                                 : make_uint2(0u, 0u);
    if (warp == 0) {
        where[lane] = takes ? (int64_t)b * p.o_st0 + (int64_t)hq * p.o_st1 + (int64_t)i * p.o_st2 : -1;
        if (takes && p.lse && blockIdx.z == 0)
            p.lse[((int64_t)b * p.Hkv * p.G + hq) * p.q_len + i] = some ? (M + __log2f(L)) * kLn2 : L != L ? L : -INFINITY;
    }
    __syncthreads();
    const int row = threadIdx.x / kJoinWarps, u = threadIdx.x % kJoinWarps;
    if (where[row] >= 0)
        *reinterpret_cast<uint2*>(p.o + where[row] + blockIdx.z * kJoinCols + 4 * u) = out[row][u];
}

template <int D, int SCORE, int NR>
cudaError_t launch_variant(const SpParams& p, const PdParams& own, cudaStream_t stream)
{
    static std::mutex mu;
    static std::vector<CtxKey> done;
    auto kern = shared_decode_kernel<D, SCORE, NR>;
    {
        CtxKey key;
        std::lock_guard<std::mutex> lock(mu);
        bool have = false;
        if (current_ctx(&key))
            for (const CtxKey& k : done) have |= k == key;
        if (!have) {
            cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SharedSmem<D>::BYTES);
            if (e != cudaSuccess) return e;
            if (current_ctx(&key)) done.push_back(key);
        }
    }
    return launch_after(kern, dim3((unsigned)p.sms), kSpThreads, SharedSmem<D>::BYTES, stream, p, own);
}

} // namespace

cudaError_t launch_shared_decode(const SpParams& p, const PdParams& own, int D, int score_kind, cudaStream_t stream)
{
#define FA_SP_CASE(DD, SS)                                                               \
    if (D == DD && score_kind == SS)                                                     \
        return p.rows > 8 ? launch_variant<DD, SS, 2>(p, own, stream) : launch_variant<DD, SS, 1>(p, own, stream);
    FA_SP_CASE(64, FA_SCORE_NONE) FA_SP_CASE(64, FA_SCORE_ALIBI) FA_SP_CASE(64, FA_SCORE_SOFTCAP)
    FA_SP_CASE(128, FA_SCORE_NONE) FA_SP_CASE(128, FA_SCORE_ALIBI) FA_SP_CASE(128, FA_SCORE_SOFTCAP)
#undef FA_SP_CASE
    return cudaErrorInvalidValue;
}

cudaError_t launch_shared_join(const SpParams& p, int D, cudaStream_t stream)
{
    const dim3 grid((unsigned)((p.geom.rows + 31) / 32), (unsigned)p.Hkv, (unsigned)(D / kJoinCols));
    return D == 64 ? launch_after(shared_join_kernel<64>, grid, 32 * kJoinWarps, 0, stream, p)
                   : launch_after(shared_join_kernel<128>, grid, 32 * kJoinWarps, 0, stream, p);
}

} // namespace fa
