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

// The caller bounds R and pages so that the list of all heads is below 2^31.
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
FA_SP_FN SpPiece sp_piece(const SpGeom& g, int x, int x1)
{
    SpPiece p;
    p.hk = x / g.per_head;
    const int off = x % g.per_head;
    const int paired = g.pairs * g.pages;
    p.one = off >= paired;
    p.col = p.one ? g.pairs : off / g.pages;
    p.e0 = off - p.col * g.pages;
    const int left = (p.one ? (g.pages + 1) / 2 : g.pages) - p.e0;
    p.n = left < x1 - x ? left : x1 - x;
    return p;
}

// Tiles of stream s in the piece: all entries, but for a column of one tile's last
// entry when the pages are odd in number, which is stream 0's alone.
FA_SP_FN int sp_tiles(const SpGeom& g, const SpPiece& p, int s)
{
    return p.one && s == 1 && 2 * (p.e0 + p.n) > g.pages ? p.n - 1 : p.n;
}

// List position of a column's first entry.
FA_SP_FN int sp_start(const SpGeom& g, int hk, int col) { return hk * g.per_head + col * g.pages; }

// SMs that take the prefix while the others take the sequences' own pages: in
// proportion to the two lists' costs, so that both end together, and if that is near a
// multiple of the columns, that multiple: no share then runs over two columns, whose end
// and start cost a CTA as much as four entries.  The same on every CTA of both kernels.
// In tenths of a microsecond of an SM: an entry `entry_cost`, a page 5, and 10 for a
// segment's start and end.
FA_SP_FN int sp_split(int entries, int columns, int own_pages, int own_segments, int sms, int entry_cost)
{
    const float a = (float)entry_cost * entries, b = 5.f * own_pages + 10.f * own_segments;
    const int most = entries < sms - 1 ? entries : sms - 1;
    int n = a > 0.f ? (int)(sms * (a / (a + b)) + 0.5f) : 1;
    n = n < most ? n : most;
    n = n < 1 ? 1 : n;
    int m = (n + columns / 2) / columns * columns;
    if (m > most) m -= columns;
    return m > 0 && 8 * (m > n ? m - n : n - m) <= n ? m : n;
}

} // namespace fa
