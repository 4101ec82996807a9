// How the paged decode deals its work to CTAs. Plain C++, so that a CPU test can check the rule.
//
// A stage is 8 KB of keys and values of one KV head of one sequence; a chunk is up to 32 query rows of that head and all its
// stages, which the four warps of one CTA, or of the CTAs of a cluster, take in turn; or the chunks of all sequences form
// one row of stages, of which every resident CTA takes an equal share and whose partials a second kernel merges.
#pragma once

#include <algorithm>
#include <cmath>

namespace alibi {
namespace paged {

constexpr int kWarps = 4;          // of a CTA, two CTAs per SM
constexpr int kMostCluster = 16;

// us of a warp's step, one stage, of head size d with `groups` groups of 8 rows, where its SM has no other CTA: the
// chain of its own instructions, whatever memory gives (0.63 at d = 128 when last measured; 0.70 chooses no worse). The factors of
// two and four groups are estimates that the last rows of the table below check.
inline double step_us(int d, int groups)
{
    const double t = d == 128 ? 0.70 : d == 64 ? 0.72 : d == 32 ? 1.08 : 1.8;
    return t * (groups == 1 ? 1.0 : groups == 2 ? 1.2 : 1.8);
}

// CTAs of a chunk (1: whole chunks, more: clusters), or 0 for equal shares: the way with the least estimated time. `ctas`: that
// the device holds at once; fit[c]: clusters of c that it holds at once. A launch takes 3.3 us, with a cluster's merge 4.5, shares
// with theirs 9.5; memory gives a stage per 1.1 ns, a tenth less to clusters, and half of an SM's room takes
// a step 1.5 times as long. Measured, in us, launches in one graph over caches that together are larger than
// L2, whole / clusters of / shares, what is taken in brackets (sequences x KV heads (x G) x tokens x d):
//   1 x 1 x 8192 x 128           [S]   82.6 / 14.2 (8) 9.2 (16) / 8.1
//   1 x 32 x 2048 x 128          [6]   23.5 / 10.9 (4) 10.3 (6) 10.6 (8) / 14.4
//   1 x 40 x 8192 x 128          [6]   83.9 / 32.7 (3) 28.9 (5) 28.7 (6) / 34.2
//   1 x 8 (x 4) x 8192 x 128     [16]  83.9 / 19.1 (6) 13.9 (10) 12.7 (12) 12.0 (16) / 13.7
//   1 x 8 (x 4) x 32768 x 128    [S]   325 / 33.0 (12) 28.7 (16) / 28.9
//   1 x 4 (x 4) x 131071 x 128   [S]   1288 / 113 (12) 90.7 (16) / 49.4
//   4 x 8 (x 8) x 8192 x 128     [8]   84.4 / 27.0 (4) 25.4 (6) 25.2 (8) / 31.2
//   2 x 40 x 8192 x 128          [3]   84.3 / 53.5 (2) 52.9 (3) / 58.6
//   2 x 40 x 1024 x 128          [3]   14.0 / 11.6 (2) 11.3 (3) / 15.8
//   4 x 40 x 4096 x 128          [W]   52.2 /   -   / 58.3
//   16 x 8 (x 4) x 4097 x 128    [2]   46.0 / 45.1 (2) / 50.3
//   8 x 8 (x 4) x 16384 x 128    [4]   165 / 87.2 (2) 81.7 (3) 84.1 (4) / 88.5
//   8 x 8 (x 8) x 32768 x 128    [4]   326 / 155.5 (3) 160.6 (4) / 168.0
//   16 x 40 x 4096 x 128         [S]   207 /   -   / 202
//   9 x 37 x 8192 x 128          [S]   249 /   -   / 208
//   1 x 32 x 8192 x 64           [8]   44.6 / 16.2 (4) 15.6 (6) 15.5 (8) / 18.6
//   8 x 16 (x 2) x 4 new, 2048 x 64  [2]  15.0 / 15.2 (2) / 21.3
//   1 x 8 (x 8) x 16384 x 64     [16]  85.1 / 16.0 (8) 12.8 (12) 12.1 (16) / 13.3
//   1 x 32 x 16384 x 32          [8]   61.4 / 18.3 (6) 16.1 (8) / 20.9
// and with 16 and 32 rows of a KV head, d = 128 and then 64. Shares are taken for too little there, as their estimate is of memory's time
// alone and a step of four groups takes longer than that:
//   8 x 8 (x 4) x 4 new, 2048    [4]   29.4 / 19.5 (2) 17.1 (4) / 25.3
//   1 x 8 (x 4) x 4 new, 16384   [S]   200 / 31.5 (8) 24.0 (12) 21.6 (16) / 21.5
//   16 x 8 (x 8) x 2 new, 4096   [2]   55.4 / 47.2 (2) / 58.7
//   40 x 8 (x 4) x 4 new, 2048   [S]   76.6 /   -   / 74.2
//   8 x 8 (x 8) x 4 new, 2048    [S]   43.2 / 27.6 (3) 24.2 (4) / 36.9
//   8 x 8 (x 8) x 4 new, 8192    [S]   149 / 71.9 (3) 57.0 (4) / 70.2
//   1 x 8 (x 8) x 4 new, 32768   [S]   561 / 80.2 (8) 55.7 (16) / 37.3
//   64 x 8 (x 8) x 4 new, 2048   [W]   107 /   -   / 142
//   8 x 16 (x 2) x 8 new, 2048   [2]   17.9 / 16.4 (2) / 27.5
//   4 x 8 (x 4) x 8 new, 8192    [S]   83.6 / 27.1 (6) 23.3 (8) / 31.8
inline int ctas_of_chunk(long long units, int stages, int ctas, const int (&fit)[kMostCluster + 1], double step)
{
    constexpr double kStage = 0.0011;
    const int busy = (stages + kWarps - 1) / kWarps;  // CTAs that a chunk can keep busy
    const double memory = kStage * static_cast<double>(units) * stages;
    const double rounds = static_cast<double>(units) / ctas, whole = std::floor(rounds);
    double cost = 3.3 + whole * kStage * ctas * stages;
    if (rounds > whole) cost += std::max(step * busy * (whole == 0 && 2 * units > ctas ? 1.15 : 1.0), (rounds - whole) * kStage * ctas * stages);
    int best = 1;
    for (int c = 2; c <= kMostCluster && c <= busy; ++c) {
        if (units > fit[c]) continue;
        const double steps = std::ceil(static_cast<double>(stages) / (kWarps * c));
        const double t = 4.5 + std::max(steps * step * (2 * units * c > ctas ? 1.5 : 1.0 + 0.02 * c), 1.1 * memory);
        if (t < cost) cost = t, best = c;
    }
    if (busy > 1 && 9.5 + 1.07 * memory < cost) best = 0;
    return best;
}

}  // namespace paged
}  // namespace alibi
