// Rotary positions and the paged append for sm_100a.
//
// A token at position p turns the pair (a, b) of a head's elements by the angle
// p * f_j:  a' = A (a cos - b sin),  b' = A (b cos + a sin).  The pairs are elements
// (j, j + rotary / 2) in the half layout and (2 j, 2 j + 1) in the interleaved one,
// for the first `rotary` elements of a head; the rest is copied.  The gradient is
// the same with the angle negated (the matrix is A times an orthogonal one).
//
// Bound: HBM.  Every element is read once and written once, and the rest is kept
// small against that: a thread owns one pair of 16-byte vectors of a token and
// walks over heads, so the angle's cosine and sine (eight pairs) are computed once
// and serve all of them.  The angle is reduced in 64 bits, p * f / (2 pi) less its
// nearest whole number: at p = 10^6 a 32-bit product would be off by 0.06 radians.
//
// Measured on a B200, calls back to back on changing inputs: Q and K of 16383 tokens, Hq 32
// Hkv 8 D 128 half rotated, token-major, 54.9 us = 6.1 TB/s; four prompts of up to 4000 tokens
// appended with their rotated queries 34.2 us = 6.0 TB/s; Q and K of B4 H16 S2048 D64
// interleaved 13.7 us = 4.9 TB/s (a short kernel: its start and end are a fifth of it).  The
// first loads are under way while the angles are computed (55.9 and 35.3 us after them).
// Angles computed once per CTA, in shared memory: 70 us on the first.
#include <cuda_runtime.h>

#include "dependent_launch.cuh"
#include "flex_fwd.cuh"
#include "ptx.cuh"
#include "rope.cuh"

namespace fa {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeBatch = 4;  // heads whose loads are issued together

__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8])
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8])
{
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
}

// cos and sin of pos * f (radians), the angle reduced in 64 bits to [-pi, pi], where the
// fast functions are off by less than 2^-21 of the amplitude: little beside an output's
// rounding to bf16.  (With sincospif, Q and K of B4 H16 S2048 D64 take 16.8 us a launch.)
__device__ __forceinline__ void turn(double pos, double f, float amp, float sgn, float& c, float& s)
{
    const double t = pos * (f * 0.15915494309189533577);  // turns
    __sincosf((float)(t - rint(t)) * 6.28318530717958647693f, &s, &c);
    c *= amp;
    s *= amp * sgn;
}

// Work unit u of a head: two 16-byte vectors.  Half layout: vectors u and
// u + rotary / 16, whose elements pair up, then the copied vectors two by two.
// Interleaved: vectors u and u + D / 16, each with its own four pairs (so that a
// warp reads consecutive vectors), rotated when below rotary / 8.
template <int D, bool INTER>
__global__ void __launch_bounds__(kRopeThreads, 3) rope_kernel(const __grid_constant__ RopeParams p)
{
    wait_prerequisites();
    launch_dependents();
    constexpr int U = D / 16;                    // units per head
    constexpr int TOK = kRopeThreads / U;        // tokens per CTA
    const int u = threadIdx.x % U;
    const int64_t t = (int64_t)blockIdx.x * TOK + threadIdx.x / U;
    if (t >= p.tokens) return;
    int gi = 0;
    while (gi + 1 < kRopeGroups && (int)blockIdx.y >= p.first_chunk[gi + 1]) ++gi;
    const RopeGroup& g = p.g[gi];
    const int h0 = ((int)blockIdx.y - p.first_chunk[gi]) * p.heads_per_thread;
    const int h1 = min(g.H, h0 + p.heads_per_thread);

    const int64_t b = (uint32_t)t / (uint32_t)p.S, s = t - b * p.S;  // both below 2^31
    const uint16_t* src = g.x + b * g.x_st0 + s * g.x_st2;
    uint16_t* dst = g.y;
    int64_t pos;
    if (p.cache_lens) {
        const int32_t have = p.cache_lens[b];
        int32_t fresh = p.new_lens ? p.new_lens[b] : (int32_t)p.S;
        // a bad length or page is reported and its tokens are left out: no write
        // outside the pools
        bool bad = have < 0 || fresh < 0 || fresh > p.S;
        if (s >= fresh || have < 0) {
            if (bad && u == 0) atomicOr(p.status, STATUS_BAD_BLOCKMASK);
            return;
        }
        pos = (int64_t)have + s;
        const int64_t slot_page = pos / 128;
        int32_t page = -1;
        if (slot_page < p.pt_width) page = p.page_table[b * p.pt_stride + slot_page];
        const bool lost = page < 0 || page >= p.num_pages;
        if ((bad || lost) && u == 0) atomicOr(p.status, STATUS_BAD_BLOCKMASK);
        if (lost) return;
        dst += g.paged ? (int64_t)page * g.y_st0 + (pos % 128) * g.y_st2 : b * g.y_st0 + s * g.y_st2;
    } else {
        pos = p.positions ? (int64_t)p.positions[b * p.pos_stride + s] : p.pos_offset + s;
        dst += b * g.y_st0 + s * g.y_st2;
    }

    int va, vb;         // the unit's vectors
    bool ra, rb;        // rotated
    if (INTER) {
        va = u;
        vb = u + U;
        ra = g.rotate && va < p.rotary / 8;
        rb = g.rotate && vb < p.rotary / 8;
    } else {
        const int half = p.rotary / 16;
        ra = rb = g.rotate && u < half;
        va = u < half ? u : 2 * u;
        vb = u < half ? u + half : 2 * u + 1;
    }
    src += 8 * va;
    dst += 8 * va;
    const int64_t d_vb = 8 * (int64_t)(vb - va);
    uint4 xa[kRopeBatch], xb[kRopeBatch];
    auto load = [&](int h) {
#pragma unroll
        for (int k = 0; k < kRopeBatch; ++k)
            if (h + k < h1) {
                const uint16_t* q = src + (int64_t)(h + k) * g.x_st1;
                xa[k] = *reinterpret_cast<const uint4*>(q);
                xb[k] = *reinterpret_cast<const uint4*>(q + d_vb);
            }
    };
    load(h0);  // under way while the angles are computed
    float c[8], sn[8];
    {
        const double dp = (double)pos;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            c[i] = 1.f;
            sn[i] = 0.f;
        }
        if (INTER) {
            if (ra)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    turn(dp, p.inv_freq[4 * va + i], p.amplitude, p.sin_sign, c[i], sn[i]);
            if (rb)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    turn(dp, p.inv_freq[4 * vb + i], p.amplitude, p.sin_sign, c[4 + i], sn[4 + i]);
        } else if (ra) {
#pragma unroll
            for (int i = 0; i < 8; ++i) turn(dp, p.inv_freq[8 * u + i], p.amplitude, p.sin_sign, c[i], sn[i]);
        }
    }
    for (int h = h0; h < h1; h += kRopeBatch) {
        if (h > h0) load(h);
#pragma unroll
        for (int k = 0; k < kRopeBatch; ++k)
            if (h + k < h1) {
                if (ra || rb) {
                    float a[8], bb[8], ya[8], yb[8];
                    unpack8(xa[k], a);
                    unpack8(xb[k], bb);
                    if (INTER) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            ya[2 * i] = a[2 * i] * c[i] - a[2 * i + 1] * sn[i];
                            ya[2 * i + 1] = a[2 * i + 1] * c[i] + a[2 * i] * sn[i];
                            yb[2 * i] = bb[2 * i] * c[4 + i] - bb[2 * i + 1] * sn[4 + i];
                            yb[2 * i + 1] = bb[2 * i + 1] * c[4 + i] + bb[2 * i] * sn[4 + i];
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            ya[i] = a[i] * c[i] - bb[i] * sn[i];
                            yb[i] = bb[i] * c[i] + a[i] * sn[i];
                        }
                    }
                    if (ra) xa[k] = pack8(ya);
                    if (rb) xb[k] = pack8(yb);
                }
                uint16_t* y = dst + (int64_t)(h + k) * g.y_st1;
                *reinterpret_cast<uint4*>(y) = xa[k];
                *reinterpret_cast<uint4*>(y + d_vb) = xb[k];
            }
    }
}

} // namespace

cudaError_t launch_rope(RopeParams& p, int D, int sms, cudaStream_t stream)
{
    const int tok = kRopeThreads / (D / 16);
    const int64_t tiles = (p.tokens + tok - 1) / tok;
    // Heads per thread: many share one computed angle, few spread a small call over the
    // SMs.  At least three CTAs per SM, as many as fit one: Q and K of B4 H16 S2048 D64,
    // forward and inverse, take 27.4 us; with at least four (four heads a thread instead of
    // eight) 28.7.  In 64 registers four CTAs would fit: 16383 tokens then take 63.4 us
    // instead of 54.9.  Four heads' loads at a time: with eight the first case took 13 % more.
    int per = 16;
    auto chunks = [&](int n) {
        int c = 0;
        for (int i = 0; i < kRopeGroups; ++i) c += (p.g[i].H + n - 1) / n;
        return c;
    };
    while (per > 1 && tiles * chunks(per) < (int64_t)3 * sms) per /= 2;
    p.heads_per_thread = per;
    p.first_chunk[0] = 0;
    for (int i = 0; i < kRopeGroups; ++i) p.first_chunk[i + 1] = p.first_chunk[i] + (p.g[i].H + per - 1) / per;
    const dim3 grid((unsigned)tiles, (unsigned)p.first_chunk[kRopeGroups]);
    auto kern = D == 64 ? (p.interleaved ? rope_kernel<64, true> : rope_kernel<64, false>)
                        : (p.interleaved ? rope_kernel<128, true> : rope_kernel<128, false>);
    return launch_after(kern, grid, kRopeThreads, 0, stream, p);
}

} // namespace fa
