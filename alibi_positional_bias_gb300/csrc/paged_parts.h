// How the prefill over pages cuts its work. Plain C++, so that a CPU test can check the rules.
//
// An item is up to 256 query rows of one head, in two tiles of 128, and all key tiles of 128 that they see; a persistent CTA per SM takes
// whole items, or parts of the tiles of those that do not fill a round.
#pragma once

#include <algorithm>
#include <cmath>

namespace alibi {
namespace paged {

constexpr int kMostParts = 16;
constexpr int kTileRows = 128;

// Parts into which the items of the last, incomplete round, the shortest, are cut: the number with the least estimated time of that
// round, in tiles of 256 rows and 128 keys (1.4 to 1.6 us): of the longest item where all parts run at once, else of the mean one.
// An item costs some four tiles beside its own; the merge, 1.6 and what reading each partial takes. Measured, in us, uncut /
// in 2 / 3 / 4 / 6 / 8 parts, what is taken in brackets (heads x new tokens of length):
//   2 x 6 x 100 of 999 (d = 64)  [4]  18.3 / 16.4 / 14.0 / 14.1 / 14.5 / 14.9
//   32 x 64 of 1024              [4]  18.3 / 15.8 / 14.5 / 13.9 / 18.6 / 18.7
//   6 x 100 of 500               [4]  13.1 / 12.6 / 13.1 / 13.0 / 13.0 / 13.1
//   6 x 1024 of 1024             [4]  20.6 / 18.2 / 16.8 / 17.2 / 17.4 / 21.7
//   4 x 8 x 128 of 4096          [4]  51.2 / 34.5 / 28.3 / 25.7 / 33.5 / 30.6
//   32 x 256 of 32768            [4]  405 / 211 / 146 / 113 / 154 / 122
//   40 x 512 of 8192             [3]  108 / 120 / 93.4 / 107 /  -  /  -
//   32 x 2048 of 32768           [4]  794 / 799 / 803 / 722 /  -  /  -
//   16 x 700 of 700              [1]  20.4 / 20.7 / 19.4 / 24.8 / 25.5 / 23.7
//   16 x 2048 of 2048            [1]  35.6 / 47.7 / 50.3 /  -  /  -  /  -
struct Parts {
    int parts;
    double cost;  // of the last round
};
inline Parts parts_of(int rest, int BH, int T, int head_rows, int L, int sms)  // head_rows: T, together G T
{
    const int before = L - std::min(T, L);
    const double blocks = static_cast<double>(rest) / BH, rows = std::min(head_rows, 256) / 256.0;
    const double mean = std::ceil((before + std::min<double>(T, 128 * (blocks + 1))) / 128);
    const double longest = std::ceil((before + std::min<double>(T, 256 * std::ceil(blocks))) / 128);
    const auto cost = [&](int parts) {
        const long long rounds = (static_cast<long long>(rest) * parts + sms - 1) / sms;
        return rounds * (std::ceil((rounds == 1 ? longest : mean) / parts) + 4) +
               (parts > 1 ? 1.6 + (0.02 + 0.008 * rows) * rest * parts : 0);
    };
    Parts best = {1, rest > 0 ? cost(1) : 0};
    for (int n = 2; n <= kMostParts && rest * n <= 3 * sms; ++n)
        if (rest > 0 && cost(n) < best.cost) best = {n, cost(n)};
    return best;
}

// Whether the rows of the heads of a group go together: of few tokens a query tile of 128 rows has room for those of several heads,
// which then pass the keys once, at the price of a bias that is computed element by element from the whole distance
// (1.25). Of up to 128 tokens, so that the rows of a block read the same pages either way. Measured, in us, apart / together, what is
// taken in brackets (heads (x G) x new tokens of length, d = 128):
//   8 x 8 (x 4) x 32 of 2048    [t]  54.8 / 28.2       8 x 8 (x 8) x 64 of 2048    [t]  97.1 / 42.7
//   8 x 8 (x 8) x 20 of 8192    [t]  312 / 78.3        64 x 8 (x 8) x 17 of 2048   [t]  648 / 139
//   32 x 8 (x 4) x 48 of 1000   [t]  106 / 48.5        1 x 8 (x 4) x 32 of 32768   [t]  95.5 / 41.6
//   16 x 4 (x 2) x 64 of 4096   [t]  51.3 / 41.8       16 x 8 (x 2) x 100 of 2048  [t]  55.1 / 42.4
//   1 x 8 (x 4) x 128 of 8192   [t]  34.0 / 31.4       4 x 8 (x 4) x 128 of 4096   [t]  51.9 / 49.6
//   1 x 8 (x 4) x 64 of 1024    [a]  14.1 / 15.8       2 x 2 (x 3) x 128 of 700    [a]  16.3 / 17.8
inline bool together(int BH, int G, int T, int L, int sms)  // BH: sequences times query heads, of which G share a KV head
{
    const int rows = G * T;
    if (G == 1 || T > kTileRows) return false;
    const double tiles = std::ceil(L / 128.0);
    const auto cost = [&](int items, int head_rows) {
        return static_cast<double>(items / sms) * (tiles + 4) + parts_of(items % sms, items, T, head_rows, L, sms).cost;
    };
    return 1.25 * cost(BH / G * ((rows + 255) / 256), rows) < cost(BH, T);
}

}  // namespace paged
}  // namespace alibi
