"""How the 4-bit decode deals its work (csrc/kv4_deal.h), on the host.

The header is plain C++; a small program compiled with g++ checks, over random batches (lengths of zero and
one, very unequal ones, row counts beyond 32-bit arithmetic, fewer stages than CTAs):

* equal shares: every stage of every chunk is in one share, a share leaves at most one partial of a chunk that
  began earlier and one of a chunk that goes on, and holder() names the share a chunk began in;
* slices: every chunk has a slice of its own at least, the CTAs of a chunk follow each other, no slice within the
  count is empty, and last() inverts cta();
* divisions by multiplication give the quotient;
* the plan: whole chunks for short sequences, clusters only as many as fit, slices only where every chunk can have two
  CTAs. No GPU involved."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "alibi_positional_bias_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include <map>
#include <random>
#include <utility>
#include <vector>
#include "kv4_deal.h"
using namespace alibi::kv4;
static int fails = 0;
#define EXPECT(c) do { if (!(c)) { if (++fails < 20) std::printf("FAIL line %d: %s\n", __LINE__, #c); } } while (0)
using ll = long long;

static void shares(const std::vector<ll> &n, int ctas)  // n: stages of every chunk
{
    std::vector<ll> start(n.size() + 1, 0);
    for (size_t u = 0; u < n.size(); ++u) start[u + 1] = start[u] + n[u];
    const ll row = start.back();
    const Cut cut(row, ctas);
    std::vector<ll> next(n.size(), 0);  // stages of the chunk that are taken so far
    std::vector<int> began(n.size(), -1);
    EXPECT(cut.begin(0) == 0 && cut.begin(cut.n) == row);
    for (int i = 0; i < cut.n; ++i) {
        ll at = cut.begin(i), left = cut.begin(i + 1) - at;
        EXPECT(left > 0);
        size_t u = std::upper_bound(start.begin(), start.end(), at) - start.begin() - 1;
        int earlier = 0, later = 0;
        while (left > 0) {
            const ll in = at - start[u], take = std::min(left, n[u] - in);
            EXPECT(in == next[u]);
            next[u] += take;
            if (in == 0) began[u] = i;
            if (take < n[u]) (in == 0 ? later : earlier)++;
            if (in + take == n[u]) EXPECT(cut.holder(start[u]) == began[u]);
            left -= take;
            at += take;
            ++u;
        }
        EXPECT(earlier <= 1 && later <= 1);
    }
    for (size_t u = 0; u < n.size(); ++u) EXPECT(next[u] == n[u]);
}

static void slices(const std::vector<ll> &n, int ctas)
{
    const int units = static_cast<int>(n.size());
    if (units >= ctas) return;
    ll row = 0, shortest = n[0];
    for (ll x : n) row += x, shortest = std::min(shortest, x);
    const Slices sl(row, units, static_cast<int>(shortest), ctas);
    EXPECT(sl.extra >= 0);
    std::vector<ll> w(units + 1, 0);
    for (int u = 0; u < units; ++u) w[u + 1] = w[u] + n[u] + sl.extra;
    EXPECT(w[units] == sl.all && sl.cta(0) == 0 && sl.cta(sl.all) == ctas);
    for (int u = 0; u < units; ++u) EXPECT(sl.cta(w[u + 1]) > sl.cta(w[u]));
    for (int i = 0; i < ctas; ++i) {
        const ll at = sl.last(i);
        EXPECT(at >= 0 && at < sl.all && sl.cta(at) <= i && (at + 1 == sl.all || sl.cta(at + 1) > i));
        const int u = static_cast<int>(std::upper_bound(w.begin(), w.end(), at) - w.begin() - 1);
        Share sh;
        sl.place(i, w[u], static_cast<int>(n[u]), sh);
        EXPECT(sh.first == sl.cta(w[u]) && sh.at == i - sh.first && sh.at >= 0 && sh.at < sl.cta(w[u + 1]) - sh.first);
        EXPECT(sh.count >= 1 && sh.count <= n[u] && sh.count == std::min<ll>(n[u], sl.cta(w[u + 1]) - sh.first));
        EXPECT((sh.left > 0) == (sh.at < sh.count));
    }
}

static void divisor(uint32_t d)
{
    const Divisor by(d);
    const auto check = [&](ll n) { if (n >= 0 && n < (1ll << 31)) EXPECT(by.of(static_cast<int>(n)) == n / d); };
    for (ll n = 0; n < 5000; ++n) check(n);
    for (ll k : {1ll, 2ll, 3ll, 1000ll, 65535ll, 1ll << 20, ((1ll << 31) - 1) / d})
        for (ll off : {-1ll, 0ll, 1ll}) check(k * d + off);
    check((1ll << 31) - 1);
}

int main()
{
    for (uint32_t d = 1; d < 5000; ++d) divisor(d);
    for (uint32_t d : {65535u, 65536u, 65537u, 131072u, (1u << 30) - 1, 1u << 30, (1u << 30) + 1, (1u << 31) - 1}) divisor(d);
    std::mt19937_64 rng(7);
    const auto pick = [&](ll lo, ll hi) { return lo + static_cast<ll>(rng() % static_cast<unsigned long long>(hi - lo + 1)); };
    for (int t = 0; t < 4000; ++t) {
        const int B = static_cast<int>(pick(1, 40)), U = static_cast<int>(pick(1, 12));
        const ll most = t % 5 == 0 ? 400000 : t % 5 == 1 ? 1 : t % 5 == 2 ? 5 : 300;
        std::vector<ll> n;
        for (int b = 0; b < B; ++b) {
            const ll len = rng() % 4 == 0 ? 1 : pick(1, most);
            for (int u = 0; u < U; ++u) n.push_back(len);
        }
        const int ctas[] = {1, 2, 7, 50, 264, 304, 512};
        shares(n, ctas[t % 7]);
        slices(n, ctas[(t / 7) % 7]);
    }
    // 152 SMs in groups of 20 and 12, and a device that holds no cluster
    ClusterFit some = {}, none = {};
    for (int c = 2; c <= kMostCluster; ++c) some.two[c] = 7 * (40 / c) + 24 / c, some.one[c] = 7 * (20 / c) + 12 / c;
    for (ll units : {1ll, 2ll, 8ll, 19ll, 32ll, 40ll, 64ll, 100ll, 152ll, 153ll, 304ll, 305ll, 2560ll, 71680ll})
        for (int stages = 1; stages <= 20000; stages = stages < 40 ? stages + 1 : stages * 5 / 4)
            for (int ctas : {2, 264, 304}) {
                EXPECT(deal_of(units, stages, ctas, none).deal != Deal::Clusters);
                const Plan p = deal_of(units, stages, ctas, some);
                if (stages <= kWarps) EXPECT(p.deal == Deal::Whole);
                EXPECT(p.deal == Deal::Clusters ? p.count >= 2 && p.count <= kMostCluster : p.count == 1);
                if (p.deal == Deal::Clusters) EXPECT(units <= some.two[p.count]);
                if (p.deal == Deal::Slices) EXPECT(2 * units <= ctas);
            }
    // the sizes of the GPU tests take every way
    for (ll stages : {313ll, 1024ll}) EXPECT(deal_of(168, static_cast<int>(stages), 304, some).deal == Deal::Shares);
    EXPECT(deal_of(160, 469, 304, some).deal == Deal::Shares);
    EXPECT(deal_of(50, 1000, 304, some).deal == Deal::Slices && deal_of(2, 1250, 304, some).deal == Deal::Slices);
    EXPECT(deal_of(1, 1250, 304, some).deal == Deal::Slices && deal_of(2, 938, 304, some).deal == Deal::Slices);
    EXPECT(deal_of(32, 64, 304, some).deal == Deal::Clusters && deal_of(8, 256, 304, some).deal == Deal::Clusters);
    EXPECT(deal_of(304, 128, 304, some).deal == Deal::Whole && deal_of(168, 112, 304, some).deal == Deal::Whole);
    std::printf(fails ? "%d failures\n" : "ok\n", fails);
    return fails != 0;
}
"""


def test_deal_on_host(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    src, exe = tmp_path / "deal.cpp", tmp_path / "deal"
    src.write_text("#include <algorithm>\n" + PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover", f"-I{CSRC}", str(src), "-o",
                    str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
