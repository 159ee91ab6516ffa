// The paged decode kernel's walk over its work list: the pages of all (sequence, kv
// head) segments, in order.  Also built for the host by the unit tests.
#pragma once

#include <cstdint>

namespace fa {

// The pages a sequence needs: logical pages [lo, lo + n) of its table row.
struct PdRange {
    int32_t len;  // cached keys, the new tokens' among them
    int32_t lo, n;
    int32_t shared;  // the pages before lo are the shared prefix, taken elsewhere
};

// A sequence's length: one below zero or beyond the table's pages (whose keys are fewer than
// 2^31) is clamped.  The same in every kernel that reads it.
template <class P>
__device__ __forceinline__ int32_t pd_length(const P& p, int32_t raw_len)
{
    const int32_t most = p.pt_width * 128;
    return raw_len < 0 ? 0 : raw_len > most ? most : raw_len;
}

// A clamped length sets `bad`.
template <class P>
__device__ __forceinline__ PdRange pd_range(const P& p, int32_t raw_len, bool& bad)
{
    PdRange r;
    const int64_t len = r.len = pd_length(p, raw_len);
    bad |= r.len != raw_len;
    const int64_t pos = len - p.q_len;  // of the first query token
    // a prefix that every query token attends whole is left out; n > 0 all the same,
    // since pos >= 128 prefix_pages and q_len > 0
    r.shared = p.prefix_pages > 0 && pos >= (int64_t)p.prefix_pages * 128;
    r.lo = r.shared ? p.prefix_pages
                    : p.has_window && pos > p.window ? (int32_t)((pos - p.window) / 128) : 0;
    r.n = (int32_t)((len + 127) / 128) - r.lo;
    return r;
}

// A sequence's pages and, above kPdCount, whether it has any: sums of these hold both the
// pages (below 2^31) and the sequences.
constexpr int kPdCount = 44;

__device__ __forceinline__ long long pd_weight(const PdRange& r)
{
    return r.n > 0 ? r.n + (1ll << kPdCount) : 0;
}

// Worker c of the `used` workers that have work takes list entries
// [pd_share(T, c, used), pd_share(T, c + 1, used)), floor(c T / used) and on; used <= T, so
// no share is empty, and T < 2^31.  (Divisions of 64 bits would be most of the code that a
// CTA fetches before it can start.)
__device__ __forceinline__ int pd_share(int T, int c, int used)
{
    const uint32_t t = T, u = used;
    return (int)(t / u * c + t % u * c / u);
}

// The worker that holds list entry x: an estimate, off by one at most, put right.
__device__ __forceinline__ int pd_holder(int T, int x, int used)
{
    int c = (int)(((float)x + 1.f) * ((float)used / (float)T));
    c = c < used ? c : used - 1;
    while (pd_share(T, c, used) > x) --c;
    while (pd_share(T, c + 1, used) <= x) ++c;
    return c;
}

// A position in the work list: page t of the range of segment (b, hk).
struct PdWalk {
    int b, hk, t;
    PdRange r;
};

// Position x0 of the list, given that it lies in the segments of sequences [lo, hi)
// and that the sequences before lo have `before` pages a kv head.
template <class P>
__device__ __forceinline__ bool pd_find(const P& p, int x0, int lo, int hi, int before, PdWalk& w, bool& bad)
{
    for (int b = lo; b < hi; ++b) {
        const PdRange r = pd_range(p, p.seq_lens[b], bad);
        if (x0 < p.Hkv * (before + r.n)) {
            const int off = x0 - p.Hkv * before;
            w = PdWalk{b, off / r.n, off % r.n, r};
            return true;
        }
        before += r.n;
    }
    return false;
}

// The next list position; the caller knows that there is one.
template <class P>
__device__ __forceinline__ void pd_advance(const P& p, PdWalk& w, bool& bad)
{
    if (++w.t < w.r.n) return;
    w.t = 0;
    if (++w.hk < p.Hkv) return;
    w.hk = 0;
    do {
        if (w.b + 1 >= p.B) { w.r.n = 0; return; }
        ++w.b;
        w.r = pd_range(p, p.seq_lens[w.b], bad);
    } while (w.r.n == 0);
}

// A page of the table as one of the pool: one outside it is clamped and sets `bad`.
__device__ __forceinline__ int pd_page(int page, int num_pages, bool& bad)
{
    if (page >= 0 && page < num_pages) return page;
    bad = true;
    return page < 0 ? 0 : num_pages - 1;
}

} // namespace fa
