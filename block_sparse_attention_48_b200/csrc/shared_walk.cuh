// Geometry of the shared prefix's work (also built for the host by the unit tests).
//
// The query rows of all sequences of a kv head, R = B * G * q_len, are cut into columns
// of 256 rows; a column's two streams are tiles of 128 rows that read the same pages.  A
// last column of at most 128 rows has one tile, and its streams read alternate pages.
// The work list is, for every kv head and column, its entries in order: a page, or, for
// a column of one tile, two of them, so that every entry is two products of 128 rows by
// 128 keys.  It is shared out as the paged decode's list is (pd_share, pd_holder).
#pragma once

#include <cstdint>

#include "paged_walk.cuh"

namespace fa {

constexpr int kSpRows = 128;  // rows of a tile

struct SpGeom {
    int32_t pages;     // of the prefix
    int32_t rows;      // R
    int32_t pairs;     // columns of two tiles
    int32_t single;    // 1: and one of one tile
    int32_t per_head;  // list entries of a kv head
};

#ifdef __CUDACC__
#define FA_SP_FN __host__ __device__ inline
#else
#define FA_SP_FN inline
#endif

// The caller bounds R and pages so that per_head fits 32 bits.
FA_SP_FN SpGeom sp_geom(int64_t R, int32_t pages)
{
    SpGeom g;
    const int32_t rest = (int32_t)(R % (2 * kSpRows));
    g.pages = pages;
    g.rows = (int32_t)R;
    g.pairs = (int32_t)(R / (2 * kSpRows)) + (rest > kSpRows ? 1 : 0);
    g.single = rest > 0 && rest <= kSpRows ? 1 : 0;
    g.per_head = g.pairs * pages + (g.single ? (pages + 1) / 2 : 0);
    return g;
}

FA_SP_FN int sp_cols(const SpGeom& g) { return g.pairs + g.single; }

// A stretch of a column's entries.
struct SpPiece {
    int hk, col;   // kv head, column within it
    int e0, n;     // entries [e0, e0 + n) of the column
    bool one;      // a column of one tile
};

// The piece at list position x of a share that ends at x1 (x < x1).
FA_SP_FN SpPiece sp_piece(const SpGeom& g, long long x, long long x1)
{
    SpPiece p;
    p.hk = (int)(x / g.per_head);
    const int off = (int)(x % g.per_head);
    const int paired = g.pairs * g.pages;
    p.one = off >= paired;
    p.col = p.one ? g.pairs : off / g.pages;
    p.e0 = off - p.col * g.pages;
    const int left = (p.one ? (g.pages + 1) / 2 : g.pages) - p.e0;
    p.n = left < x1 - x ? left : (int)(x1 - x);
    return p;
}

// Tiles of stream s in the piece: all entries, but for a column of one tile's last
// entry when the pages are odd in number, which is stream 0's alone.
FA_SP_FN int sp_tiles(const SpGeom& g, const SpPiece& p, int s)
{
    return p.one && s == 1 && 2 * (p.e0 + p.n) > g.pages ? p.n - 1 : p.n;
}

// List position of a column's first entry.
FA_SP_FN long long sp_start(const SpGeom& g, int hk, int col) { return (long long)hk * g.per_head + (long long)col * g.pages; }

// SMs that take the prefix while the others take the sequences' own pages: in
// proportion to the two lists' costs (at D = 128, with one CTA per SM: an entry 2.1 us, a
// page 0.6 us), so that both end together.  The same on every CTA of both kernels.
FA_SP_FN int sp_split(long long entries, long long own_pages, int sms)
{
    const long long a = 7 * entries, b = 2 * own_pages;
    long long n = a + b > 0 ? (sms * a + (a + b) / 2) / (a + b) : 1;
    const long long most = entries < sms - 1 ? entries : sms - 1;
    n = n < most ? n : most;
    return n < 1 ? 1 : (int)n;
}

} // namespace fa
