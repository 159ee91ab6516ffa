// Host build of the paged decode kernel's walk over its work list
// (csrc/paged_walk.cuh) and of the shared prefix's (csrc/shared_walk.cuh), for CPU unit tests: the device qualifiers are defined away
// and __ldg becomes a plain load.
#include <cstdint>

#define __device__
#define __forceinline__ inline
template <typename T>
static inline T __ldg(const T* p)
{
    return *p;
}

#include "paged_walk.cuh"
#include "shared_walk.cuh"

namespace {

// The fields the walk reads, as in the kernel's parameter block.
struct Params {
    int32_t B, Hkv, q_len, pt_width, has_window, prefix_pages;
    int64_t window;
    const int32_t* seq_lens;
};

} // namespace

// out = (len, lo, n, shared); returns whether the length was bad.
extern "C" int fa_host_pd_range(int32_t q_len, int32_t pt_width, int64_t window, int32_t prefix_pages, int32_t len,
                                int32_t* out)
{
    const Params p{1, 1, q_len, pt_width, window >= 0, prefix_pages, window >= 0 ? window : 0, nullptr};
    bool bad = false;
    const fa::PdRange r = fa::pd_range(p, len, bad);
    out[0] = r.len;
    out[1] = r.lo;
    out[2] = r.n;
    out[3] = r.shared;
    return bad;
}

// CTA c's entries of a list of T pages over `used` CTAs: count entries of (b, hk, t)
// from the position that the threads' ranges of sequences (per each) find.
extern "C" long long fa_host_pd_walk(int32_t B, int32_t Hkv, int32_t q_len, int32_t pt_width, int64_t window,
                                     int32_t prefix_pages, const int32_t* seq_lens, long long T, int c, int used,
                                     int threads, int32_t* out)
{
    const Params p{B, Hkv, q_len, pt_width, window >= 0, prefix_pages, window >= 0 ? window : 0, seq_lens};
    const long long x0 = fa::pd_share(T, c, used), n = fa::pd_share(T, c + 1, used) - x0;
    const int per = (B + threads - 1) / threads;
    bool bad = false, found = false;
    fa::PdWalk w{};
    long long before = 0;
    for (int t = 0; t < threads; ++t) {
        const int lo = t * per < B ? t * per : B, hi = lo + per < B ? lo + per : B;
        long long mine = 0;
        for (int b = lo; b < hi; ++b) mine += fa::pd_range(p, seq_lens[b], bad).n;
        if (Hkv * before <= x0 && x0 < Hkv * (before + mine)) {
            if (found) return -1;
            found = fa::pd_find(p, x0, lo, hi, before, w, bad);
            if (!found) return -2;
        }
        before += mine;
    }
    if (!found || Hkv * before != T) return -3;
    for (long long i = 0; i < n; ++i) {
        out[3 * i] = w.b;
        out[3 * i + 1] = w.hk;
        out[3 * i + 2] = w.t;
        if (i + 1 < n) fa::pd_advance(p, w, bad);
    }
    return n;
}

extern "C" int fa_host_pd_holder(long long T, long long x, int used) { return fa::pd_holder(T, x, used); }

extern "C" int fa_host_sp_split(int entries, int columns, int own_pages, int own_segments, int sms, int entry_cost)
{
    return fa::sp_split(entries, columns, own_pages, own_segments, sms, entry_cost);
}

extern "C" int fa_host_pd_page(int page, int num_pages, int32_t* bad)
{
    bool b = false;
    const int r = fa::pd_page(page, num_pages, b);
    *bad = b;
    return r;
}

// out = (pairs, single, per_head).
extern "C" void fa_host_sp_geom(long long R, int32_t pages, int32_t* out)
{
    const fa::SpGeom g = fa::sp_geom(R, pages);
    out[0] = g.pairs;
    out[1] = g.single;
    out[2] = g.per_head;
}

// CTA c's pieces: out rows of (hk, col, e0, n, one, tiles of stream 0, of stream 1).
extern "C" int fa_host_sp_pieces(long long R, int32_t pages, int32_t Hkv, int c, int used, int32_t* out)
{
    const fa::SpGeom g = fa::sp_geom(R, pages);
    const long long T = (long long)Hkv * g.per_head, x1 = fa::pd_share(T, c + 1, used);
    int n = 0;
    for (long long x = fa::pd_share(T, c, used); x < x1; ++n) {
        const fa::SpPiece p = fa::sp_piece(g, x, x1);
        int32_t* o = out + 7 * n;
        o[0] = p.hk;
        o[1] = p.col;
        o[2] = p.e0;
        o[3] = p.n;
        o[4] = p.one;
        o[5] = fa::sp_tiles(g, p, 0);
        o[6] = fa::sp_tiles(g, p, 1);
        if (fa::sp_start(g, p.hk, p.col) + p.e0 != x) return -1;
        x += p.n;
    }
    return n;
}
