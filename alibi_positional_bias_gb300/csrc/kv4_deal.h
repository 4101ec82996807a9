// How the 4-bit decode deals its work to CTAs. Plain C++ (host and device), so that a CPU test can check that every
// stage of every sequence is taken once.
//
// A stage is 128 / D blocks of one KV head of one sequence; a chunk is up to 8 query rows of that head and all its stages.
// The chunks of all sequences, one after another, form one row of stages.
#pragma once

#include <cfloat>
#include <cmath>

#include "kv4.h"

namespace alibi {
namespace kv4 {

constexpr int kWarps = 8;         // of a CTA
constexpr int kMostShares = 512;  // CTAs that share the work (two per SM)
constexpr int kMostCluster = 16;
constexpr int kGroups = 8, kGroupCtas = 32;  // groups of SMs that hold a cluster, and resident CTAs of the smallest

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

// Division of 0 <= n < 2^31 by a number that the host knows, by multiplication (Granlund and Montgomery, 1994).
struct Divisor {
    uint32_t magic, shift;

    Divisor() = default;
    explicit Divisor(uint32_t d)
    {
        for (shift = 0; (1u << shift) < d;) ++shift;
        magic = static_cast<uint32_t>(((1ull << 32) * ((1ull << shift) - d)) / d + 1);
    }
    KV4_HD int of(int n) const
    {
        const uint32_t x = static_cast<uint32_t>(n);
        return static_cast<int>((static_cast<uint32_t>(static_cast<uint64_t>(x) * magic >> 32) + x) >> shift);
    }
};

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

// The way with the least estimated time of its slowest CTA, in stages of a CTA that shares its SM (0.23 us for 32 tokens of
// d = 128; one that has it to itself takes 0.58 of that). A launch is 27, the merge of a cluster 8 more (18 above
// 8 CTAs), the partials and their merge kernel 20 (slices) or 26 (shares), and a share that ends inside a chunk pays
// 20 to begin the next one. Several rounds of whole chunks run at 0.85 of that, as fast as memory goes, with a tail of
// 0.3. Clusters fit into groups of SMs, the smallest of which has 16 (40 clusters of 7 CTAs
// take a second round, 40 of 6 do not). Measured, in us, whole / clusters of / slices / shares:
//   sequences x KV heads (x G) x tokens x d   1 x 40 x 8192 x 128        35.2 / 18.7 (6) / 18.8 / 21.5
//                                             1 x 32 x 2048 x 128        14.6 / 10.6 (8) / 12.7 /    -
//                                             1 x 8 (x 4) x 8192 x 128   35.1 / 12.5 (8) / 12.8 /    -
//                                             1 x 8 (x 4) x 32768 x 128     - / 20.7 (8) / 16.9 / 18.9
//                                             1 x 4 (x 4) x 131071 x 128    - / 32.9 (16) / 21.5 / 25.1
//                                             4 x 8 (x 8) x 8192 x 128   39.3 / 16.7 (8) / 18.8 / 23.0
//                                             16 x 8 (x 4) x 4097 x 128  22.9 / 21.0 (2) / 25.0 / 27.1
//                                             8 x 8 (x 4) x 16384 x 128  57.6 / 33.1 (4) / 37.9 / 42.9
//                                             8 x 8 (x 8) x 32768 x 128   115 /    -     / 71.9 / 67.5
//                                             9 x 37 x 16384 x 128        152 /    -     /    - /  134
//                                             13 x 38 (x 4) x 16384 x 128 178 /    -     /    - /  199
//                                             16 x 40 x 4096 x 128       71.6 /    -     /    - / 74.3
//                                             64 x 40 x 8192 x 128        424 /    -     /    - /  494
inline Plan deal_of(long long units, int stages, int ctas)
{
    if (stages <= kWarps) return {Deal::Whole, 1};
    const double rounds = static_cast<double>(units) / ctas, alone = 0.58;
    Plan best = {Deal::Whole, 1};
    double cost = 27 + stages * (rounds <= 0.5 ? alone : rounds <= 1 ? 1 : 0.85 * rounds + 0.3);
    const auto consider = [&](Deal deal, int count, double c) {
        if (c < cost) cost = c, best = {deal, count};
    };
    for (int c = 2; c <= kMostCluster; ++c)
        if (units <= kGroups * (kGroupCtas / c))
            consider(Deal::Clusters, c,
                     27 + (c > 8 ? 18 : 8) + std::ceil(stages / static_cast<double>(c)) * (2 * units * c <= ctas ? alone : 1));
    if (2 * units <= ctas) consider(Deal::Slices, 1, 47 + std::ceil(stages / std::floor(ctas / static_cast<double>(units))));
    consider(Deal::Shares, 1, 53 + stages * rounds + 20);
    return best;
}

}  // namespace kv4
}  // namespace alibi
