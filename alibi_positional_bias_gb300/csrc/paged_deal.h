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
// chain of its own instructions, whatever memory gives.
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
//   1 x 1 x 8192 x 128           [S]   87.8 / 15.5 (8) 9.8 (16) / 8.2
//   1 x 32 x 2048 x 128          [6]   25.4 / 12.5 (4) 10.5 (6) 10.6 (8) / 14.4
//   1 x 40 x 8192 x 128          [6]   91.3 / 34.7 (3) 29.7 (5) 28.7 (6) / 33.8
//   1 x 8 (x 4) x 8192 x 128     [12]  93.7 / 20.6 (6) 15.4 (10) 14.3 (12) 13.5 (16) / 13.5
//   1 x 8 (x 4) x 32768 x 128    [S]   353 / 39.6 (12) 36.5 (16) / 28.9
//   1 x 4 (x 4) x 131071 x 128   [S]   1439 / 144 (12) 126 (16) / 49.0
//   4 x 8 (x 8) x 8192 x 128     [8]   95.4 / 33.4 (4) 25.9 (6) 25.6 (8) / 30.8
//   2 x 40 x 8192 x 128          [3]   90.5 / 58.8 (2) 52.6 (3) / 57.5
//   2 x 40 x 1024 x 128          [3]   14.4 / 11.8 (2) 11.6 (3) / 15.5
//   4 x 40 x 4096 x 128          [W]   52.8 /   -   / 57.5
//   16 x 8 (x 4) x 4097 x 128    [2]   48.9 / 45.1 (2) / 50.2
//   8 x 8 (x 4) x 16384 x 128    [4]   184 / 101.8 (2) 83.6 (3) 85.7 (4) / 87.1
//   8 x 8 (x 8) x 32768 x 128    [4]   366 / 161.5 (3) 169.5 (4) / 166.4
//   16 x 40 x 4096 x 128         [S]   207 /   -   / 200
//   9 x 37 x 8192 x 128          [S]   253 /   -   / 206
//   1 x 32 x 8192 x 64           [8]   49.7 / 18.7 (4) 16.5 (6) 15.7 (8) / 18.5
//   8 x 16 (x 2) x 4 new, 2048 x 64  [2]  15.8 / 15.7 (2) / 21.4
//   1 x 8 (x 8) x 16384 x 64     [S]   94.2 / 19.3 (8) 14.2 (12) 13.2 (16) / 13.4
//   1 x 32 x 16384 x 32          [8]   72.5 / 20.2 (6) 17.6 (8) / 20.5
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
