// The serving calls' choices between ways of one result, by sizes (also built for the unit
// tests).
#pragma once

#include <cmath>
#include <cstdint>

namespace fa {

// Whether a shared prefix is taken once, by the kernel made for it, or page by page for
// every sequence.  The first costs some 15 us more before it reads anything; the second
// reads (B - 1) Hkv prefix_pages pages again, most of them from L2, and is slower the more a
// page costs it.  Page by page / once, us on a B200: to 8 rows, D 128, 21.3 / 24.3 at 1976
// such pages, 30.3 / 30.4 at 3952, 33.8 / 31.0 at 4096; D 64, 24.8 / 28.6 at 3952, 30.5 / 30.1
// at 6016; to 16 rows, D 64, 26.2 / 28.1 at 1976, 36.1 / 29.8 at 3952.  To 16 rows, D 128, the
// two cross at some 200 pages where a prefix of more than four fills tiles of 128 rows (16
// sequences, 16 rows, 21.3 / 21.7 at 195, 27.0 / 23.8 at 390; over 14 cases of 192 and more rows
// the second takes 0.80 of the first, 1.08 at most); with fewer rows or pages either wins (10
// sequences of 14 rows with a soft cap 23.8 / 27.6 at 639, 4 of 16 rows 27.9 / 24.9 at 504, 32
// sequences behind 2 pages 26.4 / 30.3 at 496) until about 1024 (33.8 / 33.1).  Two sequences
// save one reading of two, and at D 128 lose by it: over 19 cases beyond those thresholds the
// second takes 1.13 of the first.
inline bool takes_prefix_once(int64_t B, int64_t Hkv, int64_t rows, int64_t D, int64_t prefix_pages)
{
    if (D == 128 && B == 2) return false;
    const int64_t wide = B * rows >= 192 && prefix_pages > 4 ? 256 : 1024;
    const int64_t least = D == 128 ? (rows > 8 ? wide : 4096) : rows > 8 ? 2048 : 6144;
    return (B - 1) * Hkv * prefix_pages >= least;
}

// Pages that a segment can have: those of the table, or that a window of `window` keys before
// the first of q_len query tokens reaches (window < 0: none).  Teams by the table alone / by
// this, us on a B200, 600 pages of table and a window of 16384: one sequence, 16 rows, D 128
// 27.8 / 23.8; 4 sequences, 8 rows, D 128 32.3 / 21.3; 2 of 4 rows, D 64 20.6 / 14.9.  (Behind a
// prefix that is taken once the table's width is kept: without the prefix's pages it made no
// difference, 102.8 / 102.9 and 95.3 / 95.7.)
inline int64_t pages_of_a_segment(int64_t pages_per_seq, int64_t window, int64_t q_len)
{
    if (window < 0 || window >= 128 * pages_per_seq) return pages_per_seq;
    const int64_t reach = (window + q_len + 126) / 128 + 1;
    return reach < pages_per_seq ? reach : pages_per_seq;
}

// Teams for `segments` segments of at most `pages` pages: all `most` of them, unless few
// segments would be cut into more pieces than pay.  With n teams a team takes about T / n us
// for T pages, and a segment's last team `cost` ns for each of its n / segments pieces: the
// sum is least at n^2 = 1000 T segments / cost.  The pieces are then of whole pages and as
// many for every segment, so that no share runs over two segments of equal length.  All / the
// fewer teams, us on a B200: one segment of 30000 keys (8 rows, D 128) 60.1 / 22.3; 2 of 8000 (4
// rows, D 64) 14.8 / 11.2; 2 of 60000 (16 rows, D 128) 52.0 / 34.8; 8 of 8000 (16 rows, D 128)
// 26.7 / 22.0; 9 of 5000 (4 rows, D 64) 16.4 / 10.7.  Unequal lengths gain less or lose, their
// shares running over two segments: 8 of 4000 to 8000 (16 rows, D 128) 34.7 / 30.1; 9 of 3746
// to 4998 (4 rows, D 64) 14.6 / 15.1; 6 of 2000 to 5700 (16 rows, D 128) 22.0 / 24.6; 9 of 1200
// to 2500 (16 rows, D 128) 15.5 / 21.6.  The table's width stands for the lengths, which are on
// the device, so tables wider than the sequences need lose the gain: the segment of 30000 keys
// takes 21.7 us with its 235 pages of table, 29.2 with 940, 57.1 with 7520.  (A rule on the
// lengths themselves, on the device, cost every call 0.3 us; all teams for unequal lengths with a team
// for every page, 0.1 us, and lost as often as it won: 15.4 -> 17.4, 13.6 -> 11.6.)
inline int32_t teams_that_pay(int64_t segments, int64_t pages, int64_t rows, int64_t D, int64_t most)
{
    const double cost = rows > 8 ? 50.0 * (double)D / 64 : 45.0 * (double)((rows * D + 511) / 512);
    const double pieces = std::sqrt(1000.0 * (double)pages / cost);  // of a segment
    if (!(pieces * (double)segments < (double)most) || pieces >= (double)pages) return (int32_t)most;
    const int64_t m = pieces < 1.0 ? 1 : (int64_t)pieces, share = (pages + m - 1) / m;
    return (int32_t)(segments * ((pages + share - 1) / share));
}

} // namespace fa
