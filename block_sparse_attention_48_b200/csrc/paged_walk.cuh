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

// A length below zero or beyond the table's pages is clamped and sets `bad`.
template <class P>
__device__ __forceinline__ PdRange pd_range(const P& p, int32_t raw_len, bool& bad)
{
    PdRange r;
    int64_t len = raw_len;
    if (len < 0) { bad = true; len = 0; }
    if (len > (int64_t)p.pt_width * 128) { bad = true; len = (int64_t)p.pt_width * 128; }
    r.len = (int32_t)len;
    const int64_t pos = len - p.q_len;  // of the first query token
    // a prefix that every query token attends whole is left out; n > 0 all the same,
    // since pos >= 128 prefix_pages and q_len > 0
    r.shared = p.prefix_pages > 0 && pos >= (int64_t)p.prefix_pages * 128;
    r.lo = r.shared ? p.prefix_pages
                    : p.has_window && pos > p.window ? (int32_t)((pos - p.window) / 128) : 0;
    r.n = (int32_t)((len + 127) / 128) - r.lo;
    return r;
}

// CTA c of the `used` CTAs that have work takes list entries
// [pd_share(T, c, used), pd_share(T, c + 1, used)); used <= T, so no share is empty.
__device__ __forceinline__ long long pd_share(long long T, int c, int used)
{
    return (T / used) * c + (T % used) * c / used;
}

// The CTA that holds list entry x.
__device__ __forceinline__ int pd_holder(long long T, long long x, int used)
{
    return (int)(((x + 1) * used - 1) / T);
}

// A position in the work list: page t of the range of segment (b, hk).
struct PdWalk {
    int b, hk, t;
    PdRange r;
};

// Position x0 of the list, given that it lies in the segments of sequences [lo, hi)
// and that the sequences before lo have `before` pages a kv head.
template <class P>
__device__ __forceinline__ bool pd_find(const P& p, long long x0, int lo, int hi, long long before, PdWalk& w,
                                        bool& bad)
{
    for (int b = lo; b < hi; ++b) {
        const PdRange r = pd_range(p, __ldg(p.seq_lens + b), bad);
        if (x0 < p.Hkv * (before + r.n)) {
            const long long off = x0 - p.Hkv * before;
            w = PdWalk{b, (int)(off / r.n), (int)(off % r.n), r};
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
        w.r = pd_range(p, __ldg(p.seq_lens + w.b), bad);
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
