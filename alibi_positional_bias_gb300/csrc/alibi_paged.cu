// Appending new tokens to a paged KV cache, with the rotation of keys and queries by their positions where one is asked for.
//
// Token t < count_b of sequence b has position n = pos_b + t and goes to slot n % S of page table[b, n / S]. A rotation turns
// each pair (x, y) of elements, of frequency f_i, by the angle n f_i:
//   x' = x cos - y sin,  y' = y cos + x sin,
// in fp32, rounded once. The angle is reduced exactly: f_i / 2 pi is held as a 64-bit fraction of a turn (turns.h), and
// n times it modulo 2^64 is the fraction of a turn that is left, off by 2^-39 at most; its upper 32 bits go, as a float of half
// turns (off by 2^-26 of a turn), to sincospi. (In fp32 the angle of position 100000 would be off by 0.004.)
//
// What has to move: 2 bytes in and 2 bytes out of each element. A thread takes 16 bytes of a row; rows of consecutive tokens
// of one head follow one another, and a thread keeps its token from head to head, so that the page is looked up and the
// sines are computed once per thread. Four heads' loads are issued together, with a rotation before the sines are computed.
//
// Measured, launches in one graph over tensors colder than L2: prompts of 4 x 32 heads x 2048 tokens of d = 128 (268 MB) 42.7
// us, 6.3 TB/s, and with the keys and as many heads of queries rotated (403 MB) 66 us, 6.1 TB/s: bound by HBM. One token of
// 64 x 40 heads 2.1 us, 2 x (6 + 24) heads x 1001 tokens of d = 64 rotated (18 MB) 5.8 us: a launch, the way from length to
// page to row, one round of CTAs.

#include <algorithm>
#include <cmath>
#include <cuda_bf16.h>

#include "alibi.h"
#include "divide.h"
#include "pages.cuh"
#include "ptx.cuh"
#include "turns.h"

namespace alibi {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;  // heads whose loads are in flight at once
constexpr int kMostPairs = 64;

struct Rows {  // bf16 rows of new tokens; strides in elements
    const __nv_bfloat16 *data;
    long long batch, head, token;
};

struct AppendParams {
    Rows k, v, q;
    __nv_bfloat16 *q_out;  // [B, H, T, d]
    Pages pg;
    const int *pos, *count;
    uint32_t *status;
    int T, H;             // H: query heads
    int log_vec, log_tok; // log2 of the threads of a row and of the tokens of a CTA
    int group;            // heads of a CTA
    int kv_groups;        // CTAs (of the y axis) that take keys and values; those after them take queries
    int R, interleaved;
    Divisor by_blocks;    // blocks of tokens of a sequence
    uint64_t turn[kMostPairs];  // f_i / 2 pi in units of 2^-64
};

// Cosines and sines of a thread's eight elements at position n: halves, of elements 8 c .. 8 c + 7, negative sines for the
// first of each pair; interleaved, of pairs 4 c .. 4 c + 3.
struct Turn {
    float c[8], s[8];
};

// Lane that has the other elements of this lane's pairs (halves).
__device__ __forceinline__ int partner(const AppendParams &p, int vec, bool on)
{
    const int lane = threadIdx.x & 31, half = p.R / 16;
    return !on ? lane : vec < half ? lane + half : lane - half;
}

// All threads of the warp call it; `on`: this thread's elements turn.
__device__ __forceinline__ void turn_of(const AppendParams &p, int vec, int n, bool on, Turn &t)
{
    const bool upper = 16 * vec >= p.R;
    // a lane and its partner turn by the same eight angles: each computes four
    const int first = p.interleaved ? 4 * vec : upper ? 8 * vec - p.R / 2 + 4 : 8 * vec;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint64_t left = on ? p.turn[first + e] * static_cast<uint64_t>(n) : 0;
        sincospif(static_cast<float>(static_cast<int32_t>(left >> 32)) * 0x1p-31f, &t.s[e], &t.c[e]);
    }
    if (p.interleaved) return;
    const int other = partner(p, vec, on);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float c = __shfl_sync(0xffffffffu, t.c[e], other), s = __shfl_sync(0xffffffffu, t.s[e], other);
        t.c[4 + e] = upper ? t.c[e] : c;
        t.s[4 + e] = upper ? t.s[e] : -s;
        t.c[e] = upper ? c : t.c[e];
        t.s[e] = upper ? s : -t.s[e];
    }
}

__device__ __forceinline__ float lo_of(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_of(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// The thread's 16 bytes, rotated. All threads of the warp call it; `on`: this thread's elements turn.
__device__ __forceinline__ uint4 rotated(const AppendParams &p, uint4 x, int vec, bool on, const Turn &t)
{
    uint32_t w[4] = {x.x, x.y, x.z, x.w};
    if (p.interleaved) {
        if (on)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float a = lo_of(w[i]), b = hi_of(w[i]);
                w[i] = pack_bf16x2(fmaf(a, t.c[i], -b * t.s[i]), fmaf(b, t.c[i], a * t.s[i]));
            }
    } else {
        const int other = partner(p, vec, on);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t y = __shfl_sync(0xffffffffu, w[i], other);
            if (on)
                w[i] = pack_bf16x2(fmaf(lo_of(w[i]), t.c[2 * i], lo_of(y) * t.s[2 * i]),
                                   fmaf(hi_of(w[i]), t.c[2 * i + 1], hi_of(y) * t.s[2 * i + 1]));
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <bool ROTATE>
__global__ void __launch_bounds__(kThreads) paged_append_kernel(const __grid_constant__ AppendParams p)
{
    griddep_wait();
    const int vec = threadIdx.x & ((1 << p.log_vec) - 1), row = threadIdx.x >> p.log_vec;
    const int b = p.by_blocks.of(blockIdx.x);
    const int t = (p.by_blocks.rest(blockIdx.x) << p.log_tok) + (row & ((1 << p.log_tok) - 1));
    const int step = (kThreads >> p.log_vec) >> p.log_tok;  // heads that the CTA takes at once
    const int S = 1 << p.pg.shift, first = p.pos ? p.pos[b] : 0, count = p.count ? p.count[b] : p.T;
    if (first < 0 || count < 0 || count > p.T || first > p.pg.width * S - count) {
        if (threadIdx.x == 0 && p.by_blocks.rest(blockIdx.x) == 0 && blockIdx.y == 0) atomicOr(p.status, ALIBI_DEV_RANGE);
        return;
    }
    const int n = first + t;
    bool live = t < count;
    const bool queries = ROTATE && static_cast<int>(blockIdx.y) >= p.kv_groups;
    const int h0 = (queries ? blockIdx.y - p.kv_groups : blockIdx.y) * p.group + (row >> p.log_tok);
    const Rows from = queries ? p.q : p.k;
    const int heads = queries ? p.H : p.pg.heads, page = live && !queries ? p.pg.page_of(b, n) : 0, slot = p.pg.slot_of(n);
    if (page < 0) {
        atomicOr(p.status, ALIBI_DEV_RANGE);
        live = false;
    }
    const __nv_bfloat16 *src = from.data + b * from.batch + t * from.token + 8 * vec;
    const __nv_bfloat16 *vs = p.v.data + b * p.v.batch + t * p.v.token + 8 * vec;
    __nv_bfloat16 *dst = (queries ? p.q_out + (static_cast<size_t>(b) * p.H * p.T + t) * p.pg.d
                                  : p.pg.k + page * p.pg.k_page + slot * p.pg.k_slot) + 8 * vec;
    __nv_bfloat16 *vd = p.pg.v + page * p.pg.v_page + slot * p.pg.v_slot + 8 * vec;
    const long long dst_head = queries ? static_cast<long long>(p.T) * p.pg.d : p.pg.k_head;
    uint4 x[kUnroll], y[kUnroll];
    const auto load = [&](int i) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int o = i + u * step, h = h0 + o;
            x[u] = y[u] = make_uint4(0, 0, 0, 0);
            if (live && o < p.group && h < heads) {
                x[u] = __ldcs(reinterpret_cast<const uint4 *>(src + h * from.head));
                if (!queries) y[u] = __ldcs(reinterpret_cast<const uint4 *>(vs + h * p.v.head));
            }
        }
    };
    if (ROTATE) load(0);
    Turn turn;
    const bool on = ROTATE && 8 * vec < p.R;
    if (ROTATE) turn_of(p, vec, n, on && live, turn);  // while the first rows are on their way
    for (int i = 0; i < p.group; i += kUnroll * step) {
        if (!ROTATE || i > 0) load(i);
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int o = i + u * step, h = h0 + o;
            if (ROTATE) x[u] = rotated(p, x[u], vec, on, turn);
            if (live && o < p.group && h < heads) {
                *reinterpret_cast<uint4 *>(dst + h * dst_head) = x[u];
                if (!queries) *reinterpret_cast<uint4 *>(vd + h * p.pg.v_head) = y[u];
            }
        }
    }
}

int check_rows(const alibi_rows *r)
{
    if (!r || !r->data || (reinterpret_cast<uintptr_t>(r->data) & 15u)) return ALIBI_ERR_INVALID;
    for (const long long s : {r->batch, r->head, r->token})
        if (s < 0 || s % 8 != 0) return ALIBI_ERR_INVALID;
    return ALIBI_OK;
}

Rows rows_of(const alibi_rows *r) { return {static_cast<const __nv_bfloat16 *>(r->data), r->batch, r->head, r->token}; }

int log2_of(int n)  // of a power of two, or of the next one
{
    int l = 0;
    while ((1 << l) < n) ++l;
    return l;
}

}  // namespace
}  // namespace alibi

using namespace alibi;

extern "C" int alibi_paged_append(const alibi_rows *k, const alibi_rows *v, const alibi_pages *pages, const int *pos,
                                  const int *count, int B, int T, const alibi_rotation *rotation, const alibi_rows *q,
                                  void *q_out, int H, void *stream)
{
    int st = check_pages(pages);
    if (st != ALIBI_OK) return st;
    if (check_rows(k) != ALIBI_OK || check_rows(v) != ALIBI_OK) return ALIBI_ERR_INVALID;
    if (B < 1 || T < 1 || static_cast<long long>(T) > static_cast<long long>(pages->width) * pages->slots) return ALIBI_ERR_INVALID;
    if ((reinterpret_cast<uintptr_t>(pos) & 3u) || (reinterpret_cast<uintptr_t>(count) & 3u)) return ALIBI_ERR_INVALID;
    const int R = rotation ? rotation->dims : 0;
    if (R < 0 || R > pages->d || R % 16 != 0) return ALIBI_ERR_INVALID;
    if (rotation && rotation->interleaved != 0 && rotation->interleaved != 1) return ALIBI_ERR_INVALID;
    if (q) {
        if (R == 0 || !q_out || (reinterpret_cast<uintptr_t>(q_out) & 15u) || H < 1 || check_rows(q) != ALIBI_OK)
            return ALIBI_ERR_INVALID;
        if (H > kMaxQueryHeads) return ALIBI_ERR_UNSUPPORTED;
    }
    AppendParams p;
    p.R = R;
    p.interleaved = R ? rotation->interleaved : 0;
    for (int i = 0; i < R / 2; ++i) {
        const double f = rotation->freqs ? rotation->freqs[i] : std::pow(rotation->base, -2.0 * i / R);
        if (!std::isfinite(f) || std::fabs(f) > 1e6) return ALIBI_ERR_INVALID;
        p.turn[i] = turns_of(f);
    }
    p.k = rows_of(k);
    p.v = rows_of(v);
    p.q = q ? rows_of(q) : Rows{};
    p.q_out = static_cast<__nv_bfloat16 *>(q_out);
    p.pg = pages_of(pages);
    p.pos = pos;
    p.count = count;
    p.T = T;
    p.H = q ? H : 0;
    p.status = device_status_word();
    if (!p.status) return ALIBI_ERR_CUDA;
    p.log_vec = log2_of(pages->d / 8);
    const int rows = kThreads >> p.log_vec;
    p.log_tok = std::min(log2_of(T), log2_of(rows));
    const int step = rows >> p.log_tok, blocks = (T + (1 << p.log_tok) - 1) >> p.log_tok;
    const long long tokens = static_cast<long long>(B) * blocks;
    if (tokens > 0x7fffffffLL) return ALIBI_ERR_UNSUPPORTED;
    p.by_blocks = Divisor(static_cast<uint32_t>(blocks));
    // Heads of a CTA: as few as its threads take at once while that fills the device eight times, else up to sixteen times as
    // many; with a rotation, whose sines are computed once per CTA, twice (2 x (6 + 24) heads x 1001 tokens of d = 64 9.7 us
    // at two heads, 6.3 at eight, with the loads after the sines).
    const int most = std::max(pages->heads, p.H);
    p.group = step;
    while (p.group < most && p.group < 4 * kUnroll * step && tokens * ((most + p.group - 1) / p.group) > (R ? 2LL : 8LL) * num_sms())
        p.group *= 2;
    p.kv_groups = (pages->heads + p.group - 1) / p.group;
    const int q_groups = (p.H + p.group - 1) / p.group;
    const dim3 grid(static_cast<unsigned>(tokens), static_cast<unsigned>(p.kv_groups + q_groups));
    const cudaError_t e = launch_kernel(R ? paged_append_kernel<true> : paged_append_kernel<false>, grid, kThreads, 0,
                                        static_cast<cudaStream_t>(stream), p);
    return e == cudaSuccess ? ALIBI_OK : ALIBI_ERR_CUDA;
}
