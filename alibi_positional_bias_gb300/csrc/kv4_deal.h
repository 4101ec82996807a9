// How the 4-bit decode deals its work to CTAs. Plain C++ (host and device), so that a CPU test can check that every
// stage of every sequence is taken once.
//
// A stage is 128 / D blocks of one KV head of one sequence; a chunk is up to 8 query rows of that head and all its stages.
// The chunks of all sequences, one after another, form one row of stages.
#pragma once

#include <cfloat>
#include <cmath>

#include "divide.h"
#include "kv4.h"

namespace alibi {
namespace kv4 {

constexpr int kWarps = 8;         // of a CTA
constexpr int kMostShares = 512;  // CTAs that share the work (two per SM)
constexpr int kMostCluster = 16;

KV4_HD constexpr int least(int a, int b) { return a < b ? a : b; }

// Where the work of a CTA lies.
struct Share {
    int left;          // stages that are left (slices: of the whole chunk)
    int b, unit, at;   // sequence, chunk of it and stage of that chunk that comes next (slices: number of the slice)
    int first, count;  // slices: the CTA that has the chunk's first slice, and their number
};

KV4_HD int divide(long long a, int b)
{
    return a < (1LL << 32) ? static_cast<int>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b)) : static_cast<int>(a / b);
}

using alibi::Divisor;

// Equal shares: share `i` of `ctas` of a row of `row` stages is [i row / n, (i + 1) row / n), n = least(ctas, row).
// Divisions in 32 bits where the row allows it (all but sequences of many millions of tokens in all).
struct Cut {
    long long row;
    int n;

    KV4_HD Cut(long long row_, int ctas) : row(row_), n(static_cast<int>(row_ < ctas ? row_ : ctas)) {}
    KV4_HD long long begin(int i) const
    {
        if (row < (1LL << 32) / (kMostShares + 1)) return static_cast<uint32_t>(i) * static_cast<uint32_t>(row) / static_cast<uint32_t>(n);
        return i * row / n;
    }
    // the last share that begins at or before stage `at`
    KV4_HD int holder(long long at) const { return static_cast<int>(((at + 1) * n + row - 1) / row - 1); }
};

// Slices: every chunk has CTAs of its own, in proportion to its weight, its stages + `extra`, with `extra` just large enough
// for the shortest chunk to have one. The chunk that begins at weight w of `all` has CTAs from floor(w ctas / all) on.
struct Slices {
    long long all;
    int extra, ctas;

    KV4_HD Slices(long long row, int units, int shortest, int ctas_) : ctas(ctas_)
    {
        const long long lack = row - static_cast<long long>(shortest) * ctas;
        extra = lack > 0 ? divide(lack + ctas - units - 1, ctas - units) : 0;
        all = row + static_cast<long long>(extra) * units;
    }
    KV4_HD int cta(long long w) const
    {
        if (all < (1LL << 32) / (kMostShares + 1)) return static_cast<uint32_t>(w) * static_cast<uint32_t>(ctas) / static_cast<uint32_t>(all);
        return static_cast<int>(w * ctas / all);
    }
    // the last weight whose CTA is i or before
    KV4_HD long long last(int i) const
    {
        if (all < (1LL << 32) / (kMostShares + 1))
            return (static_cast<uint32_t>(i + 1) * static_cast<uint32_t>(all) + ctas - 1) / static_cast<uint32_t>(ctas) - 1;
        return ((i + 1) * all + ctas - 1) / ctas - 1;
    }
    // CTA i's slice of the chunk of n stages that begins at weight w: of `count` slices, slice k has the stages k, k + count,
    // ... counted from the newest, so that each has its part of the near tokens, whose values count, and of the far
    // ones, whose values are skipped
    KV4_HD void place(int i, long long w, int n, Share &sh) const
    {
        sh.first = cta(w);
        sh.count = least(n, cta(w + n + extra) - sh.first);
        sh.at = i - sh.first;
        sh.left = sh.at < sh.count ? n : 0;
    }
};

enum class Deal { Whole, Clusters, Slices, Shares };

struct Plan {
    Deal deal;
    int count;  // Clusters: CTAs of a cluster
};

// Clusters of c CTAs that the device holds at once, at two CTAs per SM and at one. A cluster lies within a group of SMs, so
// that 152 SMs hold 38 clusters of 7 but 46 of 6.
struct ClusterFit {
    int two[kMostCluster + 1], one[kMostCluster + 1];
};

// The way with the least estimated time, in us. A CTA that has its SM to itself takes 0.11 for a stage (32 tokens of d =
// 128) of up to 8192 tokens, less of more, whose far values are skipped, and no less than memory gives it; two that share
// one take 0.15 to 0.2 each, the more the fuller the device; several rounds of whole chunks, and slices and shares, which
// fill it, run as fast as memory goes, whole chunks with a tail of the last round. A launch takes 3.4, the merge of a
// cluster 1.6 more, the partials and their merge kernel 4.9 (slices) or, with what a share pays to begin its next chunk,
// 9.6 (shares). The estimate was fitted at d = 128 with default slopes and knows neither the head size, the rows of a
// chunk nor the slopes; of all cases measured it takes the fastest way or one within 8% of it. Measured, in us, launches in
// one graph, caches colder than L2, whole / clusters of / slices / shares, the way taken first in brackets:
//   sequences x KV heads (x G) x tokens x d
//   1 x 32 x 2048 x 128        [8]   10.3 / 7.0 (8) 6.7 (4) 7.9 (5) / 9.7 / 9.9
//   1 x 40 x 8192 x 128        [6]   31.4 / 13.5 (6) 14.6 (3) / 15.6 / 19.8
//   1 x 8 (x 4) x 8192 x 128   [12]  29.7 / 7.1 (12) 7.9 (8) 8.6 (16) / 9.9 / 10.0
//   1 x 8 (x 4) x 32768 x 128  [12]  88.2 / 12.8 (12) 16.3 (8) 15.9 (16) / 14.3 / 15.4
//   1 x 4 (x 4) x 131071 x 128 [S]   320 / 27.3 (16) / 21.0 / 22.0
//   4 x 8 (x 8) x 8192 x 128   [8]   37.6 / 13.8 (8) 14.4 (4) / 16.5 / 21.3
//   2 x 40 x 8192 x 128        [3]   30.4 / 20.6 (3) 23.9 (2) / 25.1 / 27.2
//   2 x 40 x 1024 x 128        [W]   7.2 / 8.1 (2) 7.8 (3) / 10.7 / 13.5
//   4 x 40 x 4096 x 128        [W]   22.3 /    - /    - / 26.8
//   16 x 8 (x 4) x 4097 x 128  [2]   19.4 / 17.9 (2) / 21.4 / 24.3
//   8 x 8 (x 4) x 16384 x 128  [4]   51.5 / 27.0 (4) 31.0 (2) / 33.6 / 37.7
//   8 x 8 (x 8) x 32768 x 128  [4]   119.2 / 53.4 (4) / 60.7 / 61.6
//   9 x 37 x 16384 x 128       [E]   153.5 /    - /    - / 127.9
//   16 x 40 x 4096 x 128       [W]   64.5 /    - /    - / 68.3
//   64 x 40 x 8192 x 128       [W]   408 /    - /    - / 494 (of an earlier kernel)
//   1 x 32 x 8192 x 64         [8]   19.2 / 8.5 (8) 8.8 (4) / 11.4 / 13.9
//   8 x 16 (x 2) x 4 new, 2048 x 64  [W]  8.8 / 10.0 (2) / 15.4 / 18.3
//   1 x 8 (x 8) x 16384 x 64   [12]  35.9 / 7.8 (12) 8.7 (8) / 10.4 / 10.6
//   4 x 16 x 16384 x 64        [4]   32.3 / 16.3 (4) / 20.0 / 22.7
//   1 x 2 (x 4) x 131071 x 64  [S]   197 / 16.5 (16) / 13.0 / 13.5
//   1 x 32 x 16384 x 32        [8]   21.0 / 8.8 (8) / 11.8 / 14.2
//   8 x 8 (x 4) x 16384 x 32   [4]   21.5 / 12.5 (4) / 15.7 / 18.6
//   24 x 7 x 14336 x 32        [W]   28.1 /    - /    - / 27.4
//   1 x 4 (x 8) x 65536 x 32   [16]  81.3 / 9.7 (16) / 10.4 / 10.5
//   no bias:
//   1 x 40 x 8192 x 128        [6]   34.2 / 15.2 (6) 16.0 (3) / 17.6 / 20.1
//   2 x 40 x 8192 x 128        [3]   34.4 / 24.2 (3) / 27.8 / 27.7
//   16 x 8 (x 4) x 4097 x 128  [2]   19.7 / 20.3 (2) / 24.6 / 25.7
//   1 x 8 (x 8) x 32768 x 128  [12]  150 / 18.6 (12) / 17.3 / 17.8
inline Plan deal_of(long long units, int stages, int ctas, const ClusterFit &fit)
{
    if (stages <= kWarps) return {Deal::Whole, 1};
    const double rounds = static_cast<double>(units) / ctas, last = rounds - std::ceil(rounds) + 1;
    const double far = stages < 256 ? 0.11 : 0.08 + 0.03 * 256 / stages;
    const auto alone = [&](double full) { return far > 0.25 * full ? far : 0.25 * full; };  // full: of the places for CTAs
    Plan best = {Deal::Whole, 1};
    double cost = 3.4 + stages * (rounds <= 0.5 ? alone(rounds)
                                  : rounds <= 1 ? 0.148 + 0.1 * (rounds - 0.5)
                                                : 0.195 * rounds + 0.09 * (1 - last));
    const auto consider = [&](Deal deal, int count, double c) {
        if (c < cost) cost = c, best = {deal, count};
    };
    for (int c = 2; c <= kMostCluster; ++c)
        if (units <= fit.two[c]) {
            const double full = rounds * c, shared = 0.17 + 0.06 * (full > 0.5 ? full - 0.5 : 0);
            const double longest = std::ceil(stages / static_cast<double>(c));
            consider(Deal::Clusters, c, 5 + longest * (units <= fit.one[c] ? alone(full) : shared));
        }
    if (2 * units <= ctas)
        consider(Deal::Slices, 1, 8.3 + std::ceil(stages / std::floor(ctas / static_cast<double>(units))) * 0.2);
    consider(Deal::Shares, 1, 13 + stages * rounds * 0.21);
    return best;
}

}  // namespace kv4
}  // namespace alibi
