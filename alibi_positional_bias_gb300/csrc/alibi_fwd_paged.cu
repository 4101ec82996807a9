// ALiBi attention of the tokens of a prompt, or of a part of one, over the pages that hold them and what came before, on the
// sm_103a tensor cores (tcgen05 + TMEM + TMA).
//
// Query t < count_b of sequence b and head h has position i = len_b - count_b + t and sees rows j <= i of KV head h / G:
//   x_ij = q_i.k_j / sqrt(d) - m_h (i - j),   O_i = sum_j softmax_j(x_ij) v_j,   LSE_i = ln sum_j exp(x_ij).
//
// The pipeline is that of the dense prefill (alibi_fwd_tc.cu): a persistent CTA per SM, work items of 256 query rows of one
// head in two slots of 128, K(u) and V(u - 1) behind one barrier in a ring of two units, S and P V on the tensor
// cores, the column part of the bias among them, the softmax a row per thread, key tiles of 128 from the newest down. What
// pages change:
//
//   loads     a tile of 128 keys is 128 / S boxes of S rows (of 128 rows of a larger page), one warp's lanes issue them, each
//             for the page whose number it read one tile ahead. A page past the length, or a number that is none, is
//             loaded from beyond the tensor, which fills zeros.
//   diagonal  positions begin anywhere in a tile, so a slot's rows end inside two tiles, and a row may see nothing of the first
//             tile that its slot visits.
//   values    that a row does not see meet a weight of zero, which an infinity or a NaN would turn into NaN. The loading warp
//             sets the values past the length to zero before it hands their tile over. If an output is not finite all the
//             same, the CTA takes its items once more: the warp then looks through the first tiles' values, those that some row
//             of the item does not see (up to three tiles), puts zeros in place of what is not finite and notes per column the
//             first such row, from which on the outputs are NaN. (Looking through them at once took 15% of the time of
//             prompts of 2048 tokens; two warps of their own for it, and what the MMA issuer had to say to them, 2%.)
//   rows      past count_b are left as they were: of a box of 32 rows that reaches there the lanes store their own.
//   parts     items that do not fill a round of one per SM are cut into parts of their tiles, which run one after another over
//             all SMs, part by part, so that the CTAs of a KV head pass its tiles at the same time; a part leaves its mean,
//             maximum and sum in scratch, and a second kernel merges them. (Equal shares of all items' tiles for every CTA, as the
//             decode has them, took longer than whole items: a CTA with many short items is late, whatever their tiles.)
//
// Of up to 128 tokens the rows of the G heads of a group may go together, as one head with G T rows of which each has its own
// slope and token (paged_parts.h): they pass the group's keys once and fill the tiles (64 x 8 (x 8) heads x 17 new of 2048 tokens
// 648 -> 139 us).
//
// Where some head is steep (a slope above 4 / log2(e)), the bias is taken element by element from the whole distance: the
// column part on the tensor core and the row part would cancel with a rounding of 2^-24 of 128 slopes.
//
// Measured (d = 128, launches in one graph): 16 heads x 16384 tokens 726 to 748 us (the dense prefill 695 to 710), 32 heads x 2048 new
// tokens of 32768 717 to 737 us (1447 to 1488 TFLOP/s), 4 x 32 prompts of up to 2048 133 us (895 TFLOP/s), 8 (x 4) heads x 256 new of
// 32768 113 us; 2 x 6 heads x 100 new of up to 999, d = 64, 13.4 to 14.2 us. What bounds it is what bounds the dense prefill: the chain from S
// over the softmax to P V (tensor pipe 63 to 65% of active cycles in long items, 48% in prompts of 2048), and the instruction
// cache, which the roles' code does not fit (0.6 to 0.8 cycles per issue without an instruction; the text of a second copy of
// the exponentials, or waits out of line, cost 2 to 6%).
// The place of the loops counts too, by whole lines of 128 bytes: with 0 to 7 instructions of 16 bytes at the end of the loading role
// 32 x 2048 of 32768 takes 741 / 739 / 739 / 737 / 720 / 721 / 737 / 756 us, 16 heads x 16384 749 / 757 / 753 / 747 / 732 / 742 / 760
// / 760, 4 x 32 prompts 134.8 / 134.2 / 134.6 / 134.4 / 132.4 / 132.9 / 135.3 / 135.6; four stand there. Measure again after any change
// to this kernel.

#include <algorithm>
#include <cmath>
#include <cuda.h>

#include "alibi.h"
#include "divide.h"
#include "fwd_tiles.cuh"
#include "paged_parts.h"
#include "pages.cuh"
#include "ptx.cuh"

namespace alibi {
namespace {

constexpr float kSteep = 4.0f;  // m log2(e)
using paged::kMostParts;

struct FwdPagedParams {
    CUtensorMap tq;      // [B H, T, d] bf16, box {64, 128, 1}, 128-byte swizzle
    CUtensorMap tk, tv;  // of encode_pages, boxes of min(slots, 128) slots, 128-byte swizzle
    CUtensorMap tout;    // [B H, T, d] bf16, box {32, 32, 1}, no swizzle (epilogue stores)
    Pages pg;
    const int *lens, *count;
    __nv_bfloat16 *out;
    float *lse;
    uint32_t *err;
    int T, L, BH, H, num_items, blocks;  // blocks of 256 rows of a head; together: BH and H count KV heads
    int rows, G;                         // rows of a head: T, together G T
    int whole, rest, parts;              // items that are not cut, those after them, parts of each of these
    int num_units;                       // whole + rest parts
    Divisor div_rest;
    float *part;                         // [rest][parts] partials
    Divisor div_bh, div_h, div_g;        // by B H, H and H / H_kv (together 1)
    Divisor div_t;                       // by T
    float c1;                            // log2(e) / sqrt(d)
    float slope[kMaxQueryHeads];         // m log2(e)
    uint64_t wait_ns;                    // limit of every bounded wait (the self-test's kernel; the others have kWaitLimitNs)
    int hold;                            // the self-test's barrier (HOLD_...), -1: none
};

// Barriers that the self-test of the failure path (the plain steep kernels carry it) makes wait for an arrival that nobody makes.
enum : int {
    HOLD_Q_FULL, HOLD_UNIT_FULL, HOLD_UNIT_EMPTY, HOLD_S_FULL, HOLD_P_FULL, HOLD_O_FULL, HOLD_O_EMPTY, HOLD_V_LANDED, HOLD_MET,
    HOLD_COUNT,
};

enum : uint32_t {
    SITE_PG_Q = 0x401, SITE_PG_UNIT = 0x402, SITE_PG_FIX = 0x403, SITE_PG_P = 0x404, SITE_PG_O = 0x405, SITE_PG_DONE = 0x406,
    SITE_PG_S = 0x407, SITE_PG_AGAIN = 0x408,
};

// A partial: D means of 256 rows, [D][256], then M and l of the rows, [2][256].
__host__ __device__ constexpr int paged_part_floats(int D) { return (D + 2) * 2 * BM; }

struct PagedItem {
    int bh, qb;
    int len, count;   // of the sequence
    int first;        // position of its query 0
    int top, n;       // newest key tile, and tiles visited: top, top - 1, ...
    int n_fix;        // of which the first are looked through
    int first0;       // iteration at which slot 0 begins
    bool q1valid, bad;
    int part;         // number of the partial it leaves, -1: whole
};

// Item idx, or false where its sequence has no rows there. Longest first: round r holds block blocks - 1 - r of every head.
// careful: n_fix is the tiles that some row does not see whole; else the one that the sequence ends in. TOGETHER: the rows are those
// of all heads of a KV head, T of each, which all end in the newest tiles.
template <bool TOGETHER>
__device__ __forceinline__ bool paged_item(const FwdPagedParams &p, int idx, bool careful, PagedItem &t)
{
    const int round = p.div_bh.of(idx);
    t.bh = idx - round * p.BH;
    t.qb = p.blocks - 1 - round;
    const int b = p.div_h.of(t.bh);
    t.len = p.lens ? p.lens[b] : p.L;
    t.count = p.count ? p.count[b] : p.T;
    t.bad = t.len < 0 || t.len > p.L || t.count < 0 || t.count > p.T;
    if (t.bad) {
        t.len = 0;
        if (t.count < 0 || t.count > p.T) t.count = p.T;
    }
    if (TOGETHER ? t.count == 0 : 256 * t.qb >= t.count) return false;
    t.first = t.len - t.count;
    if constexpr (TOGETHER) {
        t.q1valid = 256 * t.qb + BM < p.rows;
        t.top = max(0, t.len - 1) >> 7;
        t.n = t.top + 1;
        t.n_fix = careful ? max(1, t.top + 1 - ((max(t.first, 0) + 1) >> 7)) : (t.top + 1) * BN > t.len ? 1 : 0;
        t.first0 = 0;
        t.part = -1;
        return true;
    }
    t.q1valid = 256 * t.qb + BM < t.count;
    const int i0 = t.first + 256 * t.qb;  // position of the item's first row
    const int top0 = max(0, min(i0 + BM - 1, t.len - 1)) >> 7, top1 = max(0, min(i0 + 2 * BM - 1, t.len - 1)) >> 7;
    t.top = t.q1valid ? top1 : top0;
    t.n = t.top + 1;
    t.n_fix = careful ? max(1, t.top + 1 - ((max(i0, 0) + 1) >> 7)) : (t.top + 1) * BN > t.len ? 1 : 0;
    t.first0 = t.top - top0;
    t.part = -1;
    return true;
}

// Tiles of an item of n before its part `q` of `parts`. Not 1: slot 0 may begin at tile 1, and a part has tiles of both slots.
__device__ __forceinline__ int part_begin(int n, int q, int parts)
{
    const int c = static_cast<int>(static_cast<long long>(n) * q / parts);
    return c == 1 && n > 1 ? 0 : c;
}

// Token of a row of an item, and its head's place in the group.
template <bool TOGETHER>
__device__ __forceinline__ int token_of(const FwdPagedParams &p, int row, int &head)
{
    if constexpr (!TOGETHER) return row;
    row = min(row, p.rows - 1);
    head = p.div_t.of(row);
    return row - head * p.T;
}

// The items of a CTA, or its parts of items, one after another.
template <bool TOGETHER>
struct PagedWalk {
    int k = 0;

    __device__ __forceinline__ bool next(const FwdPagedParams &p, bool careful, PagedItem &t)
    {
        while (true) {
            const int G = gridDim.x, c = blockIdx.x, unit = (k & 1) ? (k + 1) * G - 1 - c : k * G + c;
            if (unit >= p.num_units) return false;
            ++k;
            const int q = unit < p.whole ? 0 : p.div_rest.of(unit - p.whole), i = unit - q * p.rest;  // part, item
            if (!paged_item<TOGETHER>(p, i, careful, t)) continue;
            if (unit < p.whole) return true;
            const int a = part_begin(t.n, q, p.parts), b = part_begin(t.n, q + 1, p.parts);
            if (a == b) continue;
            t.part = (i - p.whole) * p.parts + q;
            t.n = b - a;
            t.top -= a;
            t.n_fix = max(0, min(t.n_fix - a, t.n));
            if (a > 0) t.first0 = 0;
            return true;
        }
    }
};

// What a softmax warp keeps from item to item, and of an item until its tiles are done.
struct SoftmaxState {
    int k;                     // its walk
    int pass, items, outputs;  // of its CTA's, items begun, outputs written
    int part, bh, count, row0, first, flags;
};

// And the MMA issuer.
struct IssuerState {
    int k, pass, items;
    int outputs;  // parity of the outputs of each slot, bit s
};

__device__ __forceinline__ bool paged_active(const PagedItem &t, int s, int it) { return s == 1 ? t.q1valid : it >= t.first0; }

// A bounded wait of a role that other items may leave idle for long: the limit holds from one item of the MMA issuer, which
// it counts in `progress`, to the next. It sleeps between its looks, as a warp that polls
// takes issue slots of the softmax warps beside it.
__device__ __forceinline__ bool wait_idle(uint64_t *bar, uint32_t parity, const int *progress, uint32_t *err, uint32_t site)
{
    uint64_t t0 = 0;
    int seen = 0;
    uint32_t sleep = 20;
#pragma unroll 1
    for (uint32_t n = 0;; ++n) {
        if (mbar_test(bar, parity)) return true;
        __nanosleep(sleep);
        sleep = min(2 * sleep, 200u);
        if ((n & 255u) != 255u) continue;
        if (*(volatile uint32_t *)&cta_abort != 0u) return false;
        const uint64_t t = global_timer_ns();
        const int now = *reinterpret_cast<const volatile int *>(progress);
        if (t0 == 0 || now != seen) {
            t0 = t, seen = now;
        } else if (t - t0 > *(volatile uint64_t *)&cta_wait_ns) {
            report_error(err, ALIBI_DEV_TIMEOUT, site);
            *(volatile uint32_t *)&cta_abort = ALIBI_DEV_TIMEOUT;
            return false;
        }
    }
}

// The CTA's warps meet after a pass over its items: is there to be another one?
__device__ __forceinline__ bool again(uint64_t *met, const int *progress, const int *redo, uint32_t *err)
{
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(met);
    return __all_sync(0xffffffffu, wait_idle(met, 0, progress, err, SITE_PG_AGAIN)) && *reinterpret_cast<const volatile int *>(redo) != 0;
}

// After a wait that ran out: NaN for every row of the CTA's items, of which some were not computed, and for those that its parts go
// into (the merge would take whatever the scratch holds). `thread`: of 256.
template <int D, bool TOGETHER>
__device__ __forceinline__ void leave_nan(const FwdPagedParams &p, int thread)
{
    const float nan = __uint_as_float(0x7fc00000u);
    PagedWalk<TOGETHER> walk;
    PagedItem t;
#pragma unroll 1
    while (walk.next(p, false, t)) {
        if (t.part >= 0) {
            p.part[static_cast<size_t>(t.part) * paged_part_floats(D) + (D + 1) * 2 * BM + thread] = nan;
            continue;
        }
        int head = 0;
        const int row = 256 * t.qb + thread, token = token_of<TOGETHER>(p, row, head);
        if (token >= t.count || row >= p.rows) continue;
        const size_t at = static_cast<size_t>(t.bh) * p.rows + row;
#pragma unroll 1
        for (int e = 0; e < p.pg.d; e += 8)
            *reinterpret_cast<uint4 *>(p.out + at * p.pg.d + e) = make_uint4(0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u);
        if (p.lse) p.lse[at] = nan;
    }
}

template <int D, bool STEEP, bool TOGETHER>
__global__ void __launch_bounds__(kThreads, 1) fwd_paged_kernel(const __grid_constant__ FwdPagedParams p)
{
    using C = Cfg<D>;
    using PagedWalk = PagedWalk<TOGETHER>;
    static_assert(STEEP || !TOGETHER, "rows of several heads have no column part in common");
    extern __shared__ uint8_t smem_raw[];
    // of the items in flight, two at most: the first row of each column of V that is not finite, whether there is one, and
    // whether a page number is none
    __shared__ int odd_from[2][D];
    __shared__ int odd_any[2], lost[2], redo, progress;
    __shared__ SoftmaxState states[8];
    __shared__ IssuerState issuer;
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    // In static shared memory, whose addresses are constants: the softmax loop has no registers for them.
    __shared__ uint64_t q_full[1];      // both Q tiles of the item loaded
    __shared__ uint64_t q_empty[1];
    __shared__ uint64_t unit_full[2];   // ring unit of stage s loaded (K(u) and V(u - 1))
    __shared__ uint64_t unit_empty[2];  // ring unit of stage s read by the MMAs
    __shared__ uint64_t s_full[2];
    __shared__ uint64_t p_full[2];      // P of keys 0..63 written
    __shared__ uint64_t p_hi[2];        // P of keys 64..127 written
    __shared__ uint64_t o_full[2];
    __shared__ uint64_t o_empty[2];
    __shared__ uint64_t bias_full[1];   // column-bias operand of the item written
    __shared__ uint64_t v_landed[1];    // values to be looked through before their unit is handed over
    __shared__ uint64_t met[1];         // the warps after their first pass
    __shared__ uint64_t mma_done[1];
    __shared__ uint32_t tmem_slot[1];

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    uint32_t *err = p.err;

    if (threadIdx.x == 0) {
        const auto held = [&](int barrier) -> uint32_t { return STEEP && !TOGETHER && p.hold == barrier; };
        cta_err_init(STEEP && !TOGETHER ? p.wait_ns : kWaitLimitNs);
        cta_check_init(p.err, smem_raw, C::kSmem);
        redo = progress = 0;
        for (int s = 0; s < 2; ++s) {
            mbar_init(&unit_full[s], 1 + (s == 0 ? held(HOLD_UNIT_FULL) : 0));
            mbar_init(&unit_empty[s], 1 + (s == 1 ? held(HOLD_UNIT_EMPTY) : 0));
            mbar_init(&s_full[s], 1 + held(HOLD_S_FULL));
            mbar_init(&p_full[s], 4 + held(HOLD_P_FULL));  // one arrival per softmax warp
            mbar_init(&p_hi[s], 4);
            mbar_init(&o_full[s], 1 + held(HOLD_O_FULL));
            mbar_init(&o_empty[s], 4 + held(HOLD_O_EMPTY));
        }
        mbar_init(q_empty, 1);
        mbar_init(q_full, 1 + held(HOLD_Q_FULL));
        mbar_init(bias_full, 1);
        mbar_init(v_landed, 1 + held(HOLD_V_LANDED));
        mbar_init(mma_done, 1);
        mbar_init(met, 10 + held(HOLD_MET));  // of the loading, the issuing and the softmax warps
        fence_mbar_init();
        tma_prefetch_desc(&p.tq);
        tma_prefetch_desc(&p.tk);
        tma_prefetch_desc(&p.tv);
        tma_prefetch_desc(&p.tout);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, kTmemCols);
        tmem_relinquish();
    }
    if (threadIdx.x < 2 * BM) {
        // ones in logical 16-byte chunks 0-1 of every row (the A operand of the bias MMA)
        write_ones_chunk(smem + C::kAux, threadIdx.x >> 1, threadIdx.x & 1);
        fence_proxy_async_smem();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    if (p.parts > 1) griddep_launch_dependents();  // the merge kernel
    griddep_wait();  // the kernel before, which may have written what this one reads, is done

    if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsLow));
    if (warp == 0) {
        // ------------------------------------------------------ TMA producer
        const int box = min(1 << p.pg.shift, BN), boxes = BN / box;  // rows of a box, boxes of a tile
        const int copies = boxes == 1 ? 1 : C::kChunks;
        uint32_t uc = 0;  // ring units issued
        int kk = 0;       // items begun
        uint32_t looked = 0;
        bool ok = true;
        PagedWalk walk;
        for (int pass = 0; ok;) {
            PagedItem t;
            if (!walk.next(p, pass != 0, t)) {
                if (pass++ || !again(met, &progress, &redo, err)) break;
                walk = PagedWalk();
                continue;
            }
            const int b = p.div_h.of(t.bh), hk = p.div_g.of(p.div_h.rest(t.bh));
            // page of this lane's box of tile j
            const auto page_at = [&](int j) {
                const int at = j * BN + lane * box;
                return lane < boxes && j >= 0 && at < t.len ? p.pg.page_of(b, at) : p.pg.pages;
            };
            int page = page_at(t.top), before = p.pg.pages;
            ok = __all_sync(0xffffffffu, mbar_wait(q_empty, (kk & 1) ^ 1, err, SITE_PG_Q));
            if (!ok) break;
            if (lane == 0) {
                lost[kk & 1] = odd_any[kk & 1] = 0;
                mbar_arrive_expect_tx(q_full, 2 * C::kTileBytes);
                for (int s = 0; s < 2; ++s)
                    for (int c = 0; c < C::kChunks; ++c)
                        tma_load_3d(smem + C::kQ + s * C::kTileBytes + c * C::kChunkBytes, &p.tq, 64 * c, (2 * t.qb + s) * BM,
                                    t.bh, q_full);
            }
            if (pass != 0)
                for (int e = lane; e < D; e += 32) odd_from[kk & 1][e] = 0x7fffffff;
            __syncwarp();
            // Unit u = 0 .. n: K(u) (u < n) and V(u - 1) (u >= 1), consumed in the MMA issuer's iteration u - 1.
            for (int u = 0; u <= t.n; ++u) {
                const uint32_t st = uc % 2, ph = (uc / 2) & 1;
                // V(u - 1) goes by a barrier of its own, to be looked through; the first one of an item is asked for with K(0),
                // into a ring that is empty then.
                const bool look = u >= 1 && u <= t.n_fix, with_k0 = u == 0 && t.n_fix > 0;
                if (page < 0) lost[kk & 1] = 1, page = p.pg.pages;
                const int ahead = page_at(t.top - u - 1);
                ok = __all_sync(0xffffffffu, mbar_wait(&unit_empty[st], ph ^ 1, err, SITE_PG_UNIT));
                if (!ok) {
                    looked += u == 1 && look;  // V(0), asked for with K(0), is in flight
                    break;
                }
                if (lane == 0) {
                    if (with_k0 || (look && u > 1)) mbar_arrive_expect_tx(v_landed, C::kTileBytes);
                    if (look) {
                        if (u < t.n) mbar_expect_tx(&unit_full[st], C::kTileBytes);
                    } else {
                        mbar_arrive_expect_tx(&unit_full[st], (u < t.n ? C::kTileBytes : 0u) + (u >= 1 ? C::kTileBytes : 0u));
                    }
                }
                __syncwarp();
                uint8_t *const v = smem + C::kV + st * C::kTileBytes;
                if (lane < boxes) {
                    const int at = lane * box * 128;  // of the box in a swizzle atom
                    for (int c = 0; c < copies; ++c) {
                        if (u < t.n)
                            load_box<64>(smem + C::kK + st * C::kTileBytes + c * C::kChunkBytes + at, &p.tk, p.pg, box, C::kChunks / copies,
                                         p.pg.slot_of((t.top - u) * BN + lane * box), c, hk, page, &unit_full[st]);
                        if (with_k0)
                            load_box<64>(smem + C::kV + (st ^ 1) * C::kTileBytes + c * C::kChunkBytes + at, &p.tv, p.pg, box, C::kChunks / copies,
                                         p.pg.slot_of(t.top * BN + lane * box), c, hk, page, v_landed);
                        else if (u >= 1 && !(look && u == 1))
                            load_box<64>(v + c * C::kChunkBytes + at, &p.tv, p.pg, box, C::kChunks / copies,
                                         p.pg.slot_of((t.top - u + 1) * BN + lane * box), c, hk, before, look ? v_landed : &unit_full[st]);
                    }
                }
                __syncwarp();
                if (u == 0 && !STEEP) {
                    // the column-bias operand, whose last readers were the products of the item before
                    const float scale = p.slope[p.div_h.rest(t.bh)] / p.c1;
                    for (int r = lane; r < BN; r += 32) write_bias_row(smem + C::kAux, r, 0, scale * static_cast<float>(r));
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bias_full);
                }
                if (look) {
                    ok = __all_sync(0xffffffffu, mbar_wait(v_landed, looked++ & 1, err, SITE_PG_FIX));
                    constexpr int kPieces = D / 8;  // of 16 bytes of a row
                    const int row0 = (t.top - u + 1) * BN;
                    // in a first pass the slots past the length, in a second one all
                    for (int x = (pass == 0 ? t.len - row0 : 0) * kPieces + lane; x < BN * kPieces && ok; x += 32) {
                        const int row = x / kPieces, piece = x % kPieces;
                        uint4 *const at = reinterpret_cast<uint4 *>(v + piece / 8 * C::kChunkBytes + row * 128 + (((piece ^ row) & 7) << 4));
                        if (row0 + row >= t.len) {
                            *at = make_uint4(0, 0, 0, 0);
                            continue;
                        }
                        const uint4 y = *at;
                        // a half whose exponent is full overflows into bit 15 when one is added to it
                        const auto odd = [](uint32_t a) { return ((a & 0x7f807f80u) + 0x00800080u) & 0x80008000u; };
                        if ((odd(y.x) | odd(y.y) | odd(y.z) | odd(y.w)) == 0u) continue;
                        uint32_t a[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const uint32_t m = 0x7f80u << (16 * (e & 1));
                            if ((a[e / 2] & m) != m) continue;
                            a[e / 2] &= ~(0xffffu << (16 * (e & 1)));
                            atomicMin(&odd_from[kk & 1][8 * piece + e], row0 + row);
                            odd_any[kk & 1] = 1;
                        }
                        *at = make_uint4(a[0], a[1], a[2], a[3]);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&unit_full[st]);  // after an error too: the copies into the unit may be waited for
                }
                before = page;
                page = ahead;
                ++uc;
                if (!ok) break;
            }
            ++kk;  // after an error too: the item's Q was issued
        }
        // Drain (also after an error): the last Q load and the last load into each ring stage has landed before the CTA can
        // exit. Earlier loads into a stage were consumed, hence complete, before the stage was reused.
        if (kk > 0) mbar_wait(q_full, (kk - 1) & 1, err, SITE_PG_Q, true);
        if (looked > 0) mbar_wait(v_landed, (looked - 1) & 1, err, SITE_PG_FIX, true);
        for (uint32_t n = uc > 2 ? uc - 2 : 0; n < uc; ++n) mbar_wait(&unit_full[n % 2], (n / 2) & 1, err, SITE_PG_UNIT, true);
        // Four instructions of 16 bytes, run once: the loops of the roles that follow keep their best place (the head of this file).
#pragma unroll
        for (int i = 0; i < 4; ++i) __nanosleep(0);
    } else if (warp == 1) {
        // -------------------------------------------------------- MMA issuer (converged; one elected lane issues)
        constexpr uint32_t idS = idesc_bf16_f32(BM, BN, 0);
        constexpr uint32_t idO = idesc_bf16_f32(BM, D, 1);
        const uint32_t sQ = smem_u32(smem + C::kQ);
        const uint32_t sK = smem_u32(smem + C::kK);
        const uint32_t sV = smem_u32(smem + C::kV);
        const uint64_t auxd = smem_desc_sw128(smem_u32(smem + C::kAux), 16, 1024);
        uint32_t uc = 0;  // ring units consumed
        uint32_t p_cnt[2] = {0, 0};
        // As the softmax warps' state, what the loop over tiles does not need waits in shared memory.
        volatile IssuerState &st = issuer;
        if (lane == 0) st.k = st.pass = st.items = st.outputs = 0;
        __syncwarp();
        bool ok = true;
        while (ok) {
            PagedItem t;
            uint32_t outputs;  // parity of the outputs of each slot before the item, bit s
            {
                PagedWalk walk;
                walk.k = st.k;
                const int pass = st.pass, items = st.items;
                outputs = st.outputs;
                const bool more = walk.next(p, pass != 0, t);
                __syncwarp();
                if (!more) {
                    if (pass != 0 || !again(met, &progress, &redo, err)) break;
                    if (lane == 0) st.k = 0, st.pass = 1;
                    __syncwarp();
                    continue;
                }
                if (lane == 0) {
                    st.k = walk.k, st.items = items + 1, st.outputs = outputs ^ (t.q1valid ? 3 : 1);
                    *reinterpret_cast<volatile int *>(&progress) = items;
                }
                __syncwarp();
                ok = mbar_wait(q_full, items & 1, err, SITE_PG_Q);
                if (ok && !STEEP) ok = mbar_wait(bias_full, items & 1, err, SITE_PG_Q);
            }
            // an idle slot's epilogue of an earlier item reads what this item's values will overwrite (odd_from)
            if (ok && !t.q1valid) ok = mbar_wait(&o_empty[1], (outputs >> 1 & 1) ^ 1, err, SITE_PG_O);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;

            auto issue_S = [&](int s, uint32_t kst) {
                const uint64_t qd = smem_desc_sw128(sQ + s * C::kTileBytes, 16, 1024);
                const uint64_t kd = smem_desc_sw128(sK + kst * C::kTileBytes, 16, 1024);
                const uint32_t dst = tmem + s * 128;
#pragma unroll
                for (int m = 0; m < D / 16; ++m) {
                    const uint32_t step = ((m >> 2) * C::kChunkBytes + (m & 3) * 32) >> 4;
                    mma_ss_w(dst, qd + step, kd + step, idS, m > 0);
                }
                if (!STEEP) mma_ss_w(dst, auxd, auxd + 2, idS, 1u);
                mma_commit_w(&s_full[s]);
            };
            auto issue_PV_half = [&](int s, uint32_t vst, bool first, int half) {
                const uint64_t vd = smem_desc_sw128(sV + vst * C::kTileBytes, C::kChunkBytes, 1024);
                const uint32_t dst = tmem + 256 + s * 128, pa = tmem + s * 128;
#pragma unroll
                for (int k4 = 0; k4 < BN / 32; ++k4) {
                    const int m = half * (BN / 32) + k4;
                    mma_ts_w(dst, pa + m * 8, vd + ((m * 2048) >> 4), idO, (first && m == 0) ? 0u : 1u);
                }
            };

            bool first_pv[2] = {true, true};
            {
                const uint32_t st = uc % 2, ph = (uc / 2) & 1;  // unit 0: K(0)
                ok = __all_sync(0xffffffffu, mbar_wait(&unit_full[st], ph, err, SITE_PG_UNIT));
                if (!ok) break;
                for (int s = 0; s < 2; ++s)
                    if (paged_active(t, s, 0)) issue_S(s, st);
                mma_commit_w(&unit_empty[st]);
                ++uc;
            }
            for (int it = 0; it < t.n && ok; ++it) {
                // unit it + 1: V(it) and K(it + 1)
                const uint32_t vst = uc % 2, uph = (uc / 2) & 1;
                ok = __all_sync(0xffffffffu, mbar_wait(&unit_full[vst], uph, err, SITE_PG_UNIT));
                if (!ok) break;
                for (int s = 0; s < 2 && ok; ++s) {
                    if (paged_active(t, s, it)) {
                        ok = mbar_wait_spin(&p_full[s], p_cnt[s] & 1, err, SITE_PG_P);
                        if (ok && first_pv[s]) ok = mbar_wait(&o_empty[s], (outputs >> s & 1) ^ 1, err, SITE_PG_O);
                        ok = __all_sync(0xffffffffu, ok);
                        if (!ok) break;
                        tc_fence_after();
                        issue_PV_half(s, vst, first_pv[s], 0);
                        ok = __all_sync(0xffffffffu, mbar_wait_spin(&p_hi[s], p_cnt[s] & 1, err, SITE_PG_P));
                        ++p_cnt[s];
                        if (!ok) break;
                        tc_fence_after();
                        issue_PV_half(s, vst, first_pv[s], 1);
                        first_pv[s] = false;
                        if (it == t.n - 1) mma_commit_w(&o_full[s]);
                    }
                    if (it + 1 < t.n && paged_active(t, s, it + 1)) issue_S(s, vst);
                }
                mma_commit_w(&unit_empty[vst]);  // the unit's V and K have both been read
                ++uc;
            }
            mma_commit_w(q_empty);
        }
        // drain: every MMA issued above completes before TMEM is released
        mma_commit_w(mma_done);
        mbar_wait(mma_done, 0, err, SITE_PG_DONE, true);
    }
    } else {
        // ------------------------------------------------ softmax warpgroups
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsHigh));
        const int s = (warp - 4) >> 2;
        const int quad = warp & 3;  // TMEM lane quadrant this warp may access
        const int r = quad * 32 + lane;
        const uint32_t lane_addr = tmem + (static_cast<uint32_t>(quad * 32) << 16);
        // What the loop over tiles does not need waits in shared memory: the loop takes all registers.
        volatile SoftmaxState &st = states[warp - 4];
        if (lane == 0) st.k = st.pass = st.items = st.outputs = 0;
        __syncwarp();
        uint32_t s_phase = 0;
        bool ok = true;
        while (ok) {
            float di, sl2;  // of this row: position less that of the tile's first key; m log2(e)
            int left;       // tiles
            {
                PagedItem t;
                PagedWalk walk;
                walk.k = st.k;
                const int pass = st.pass, items = st.items;
                const bool more = walk.next(p, pass != 0, t);
                __syncwarp();
                if (!more) {
                    if (lane == 0) bulk_wait_all();  // the outputs of the first pass stand before those of the second
                    if (pass != 0 || !again(met, &progress, &redo, err)) break;
                    if (lane == 0) st.k = 0, st.pass = 1;
                    __syncwarp();
                    continue;
                }
                const int row0 = (2 * t.qb + s) * BM + quad * 32, it0 = s == 0 ? t.first0 : 0;
                if (lane == 0) {
                    st.k = walk.k, st.items = items + 1;
                    st.part = t.part, st.bh = t.bh, st.count = t.count, st.row0 = row0, st.first = t.first;
                    st.flags = t.bad;
                }
                __syncwarp();
                if (s == 1 && !t.q1valid) continue;
                int head = 0;
                const int token = token_of<TOGETHER>(p, row0 + lane, head);
                di = static_cast<float>(t.first + token - (t.top - it0) * BN);  // exact: below 2^24
                sl2 = p.slope[TOGETHER ? p.div_h.rest(t.bh) * p.G + head : p.div_h.rest(t.bh)];
                left = t.n - it0;
            }
            float M = 0.f, l = 0.f;
            if (s == 1) ok = __all_sync(0xffffffffu, wait_idle(&s_full[s], s_phase, &progress, err, SITE_PG_S));
            for (; left > 0 && ok; --left, di += static_cast<float>(BN)) {
                ok = __all_sync(0xffffffffu, mbar_wait(&s_full[s], s_phase, err, SITE_PG_S));  // converged for tcgen05.ld
                s_phase ^= 1;
                if (!ok) break;
                tc_fence_after();
                uint32_t sraw[BN];
#pragma unroll
                for (int c = 0; c < BN / 32; ++c)
                    tmem_ld32(lane_addr + s * 128 + c * 32, *reinterpret_cast<uint32_t(*)[32]>(&sraw[c * 32]));
                tmem_wait_ld();
                float x[BN];  // relative to the running maximum M
                if (!STEEP) {
                    const float2 c1v = make_float2(p.c1, p.c1);
                    const float rb = -sl2 * di - M;
                    const float2 rbv = make_float2(rb, rb);
#pragma unroll
                    for (int u = 0; u < BN / 2; ++u) {
                        const float2 xv = __ffma2_rn(
                            make_float2(__uint_as_float(sraw[2 * u]), __uint_as_float(sraw[2 * u + 1])), c1v, rbv);
                        x[2 * u] = xv.x;
                        x[2 * u + 1] = xv.y;
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < BN; ++c)
                        x[c] = fmaf(sl2, static_cast<float>(c) - di, fmaf(__uint_as_float(sraw[c]), p.c1, -M));
                }
                if (__any_sync(0xffffffffu, di < static_cast<float>(BN - 1))) {  // some row of the warp does not see all keys
#pragma unroll
                    for (int c = 0; c < BN; ++c) x[c] = static_cast<float>(c) > di ? -INFINITY : x[c];
                }
                const float mt = row_max128(x);
                // Raise the running maximum lazily, only when this tile exceeds it by 2^8, or where the row has seen nothing
                // so far (then M is 0, and there is nothing to rescale). O_s is quiescent here: S_s(it) completing implies that
                // the product before it has completed.
                const bool none = l == 0.f, need = mt > (none ? -INFINITY : kRescaleThreshold);
                if (__any_sync(0xffffffffu, need)) {
                    const float shift = need ? mt : 0.f, alpha = none ? 1.0f : ex2_approx(-shift);
                    M += shift;
                    l *= alpha;
                    const float2 negs = make_float2(-shift, -shift);
#pragma unroll
                    for (int u = 0; u < BN / 2; ++u) {
                        const float2 xv = __fadd2_rn(make_float2(x[2 * u], x[2 * u + 1]), negs);
                        x[2 * u] = xv.x;
                        x[2 * u + 1] = xv.y;
                    }
                    if (__any_sync(0xffffffffu, need && !none)) {
#pragma unroll 1
                        for (int c = 0; c < D / 32; ++c) {
                            uint32_t o[32];
                            tmem_ld32(lane_addr + 256 + s * 128 + c * 32, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int u = 0; u < 32; ++u) o[u] = __float_as_uint(__uint_as_float(o[u]) * alpha);
                            tmem_st32(lane_addr + 256 + s * 128 + c * 32, o);
                        }
                    }
                }
                float2 acc[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                // Two halves of 64 keys: the first half of P is handed to the MMA issuer while the second is exponentiated.
                uint32_t pk[BN / 2];
#pragma unroll
                for (int half = 0; half < 2; ++half) {
#pragma unroll
                    for (int u = half * (BN / 4); u < (half + 1) * (BN / 4); ++u) {
                        const float2 pv = make_float2(ex2_approx(x[2 * u]), ex2_approx(x[2 * u + 1]));
                        acc[u & 3] = __fadd2_rn(acc[u & 3], pv);
                        pk[u] = pack_bf16x2(pv.x, pv.y);
                    }
                    tmem_st32(lane_addr + s * 128 + half * 32, *reinterpret_cast<uint32_t(*)[32]>(&pk[half * 32]));
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(half == 0 ? &p_full[s] : &p_hi[s]);
                }
                const float2 a01 = __fadd2_rn(acc[0], acc[1]), a23 = __fadd2_rn(acc[2], acc[3]);
                const float2 a = __fadd2_rn(a01, a23);
                l += a.x + a.y;
            }
            if (!ok) break;
            // ------------------------------------------------------ epilogue
            const int outputs = st.outputs, buf = (st.items - 1) & 1;
            __syncwarp();
            if (lane == 0) st.outputs = outputs + 1;
            ok = mbar_wait(&o_full[s], outputs & 1, err, SITE_PG_O);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after();
            const float nan = __uint_as_float(0x7fc00000u);
            const int flags = st.flags, count = st.count, bh = st.bh, row0 = st.row0, pass = st.pass;
            const bool bad = (flags & 1) || *(volatile int *)&lost[buf];
            if (bad && quad == 0 && lane == 0) atomicOr(err, ALIBI_DEV_RANGE);
            const float inv_l = bad ? nan : l == 0.f ? 0.f : 1.0f / l;
            const bool odd = pass != 0 && *(volatile int *)&odd_any[buf] != 0;
            int head = 0;
            const int token = token_of<TOGETHER>(p, row0 + lane, head);
            const bool valid = token < count && (!TOGETHER || row0 + lane < p.rows);
            const int i = st.first + token;  // position
            const int dr = D == 64 ? p.pg.d : D;
            // O / l goes out through a per-warp staging box and bulk tensor stores, so that the warp does not wait for its
            // stores before its next tile; of a box that reaches past the sequence's rows each lane stores its own row.
            const bool box = TOGETHER ? __all_sync(0xffffffffu, valid) : row0 + 32 <= count, whole = st.part < 0;
            const bool none = TOGETHER ? !__any_sync(0xffffffffu, valid) : row0 >= count;
            float *part = whole ? nullptr : p.part + static_cast<size_t>(st.part) * paged_part_floats(D) + s * BM + r;
            float finite = 0.f;  // or NaN
            uint8_t *stg = smem + C::kStage + (warp - 4) * 2048;
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
                if (c * 32 >= dr || none) break;
                uint32_t o[32];
                tmem_ld32(lane_addr + 256 + s * 128 + c * 32, o);
                tmem_wait_ld();
                if (pass == 0) {
#pragma unroll
                    for (int u = 0; u < 32; ++u) finite = fmaf(__uint_as_float(o[u]), 0.f, finite);
                }
                if (!whole) {
#pragma unroll
                    for (int u = 0; u < 32; ++u) part[(c * 32 + u) * 2 * BM] = __uint_as_float(o[u]) * inv_l;
                    continue;
                }
                uint32_t y[16];
#pragma unroll
                for (int u = 0; u < 16; ++u)
                    y[u] = pack_bf16x2(__uint_as_float(o[2 * u]) * inv_l, __uint_as_float(o[2 * u + 1]) * inv_l);
                if (box) {
                    if (lane == 0) bulk_wait_read();  // the previous box has left the staging
                    __syncwarp();
                    uint4 *dst = reinterpret_cast<uint4 *>(stg + lane * 64);
#pragma unroll
                    for (int u = 0; u < 4; ++u) dst[u] = make_uint4(y[4 * u], y[4 * u + 1], y[4 * u + 2], y[4 * u + 3]);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        tma_store_3d(&p.tout, stg, c * 32, row0, bh);
                        bulk_commit();
                    }
                } else if (valid) {
                    uint4 *dst = reinterpret_cast<uint4 *>(p.out + (static_cast<size_t>(bh) * p.rows + row0 + lane) * dr + c * 32);
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        if (c * 32 + 8 * u < dr) dst[u] = make_uint4(y[4 * u], y[4 * u + 1], y[4 * u + 2], y[4 * u + 3]);
                }
            }
            if (odd) {  // NaN over what was stored
                if (lane == 0) bulk_wait_all();
                __syncwarp();
#pragma unroll 1
                for (int e = 0; e < dr; ++e) {
                    if (!valid || i < odd_from[buf][e]) continue;
                    if (whole)
                        p.out[(static_cast<size_t>(bh) * p.rows + row0 + lane) * dr + e] = __ushort_as_bfloat16(0x7fffu);
                    else
                        part[e * 2 * BM] = nan;
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&o_empty[s]);
            if (pass == 0 && valid && !bad && finite != 0.f) redo = 1;
            if (!whole) {
                part[D * 2 * BM] = M;
                part[(D + 1) * 2 * BM] = bad ? nan : l;
                continue;
            }
            if (valid && p.lse)
                p.lse[static_cast<size_t>(bh) * p.rows + row0 + lane] =
                    bad ? nan : l == 0.f ? -INFINITY : (M + __log2f(l)) * 0.69314718055994531f;
        }
    }

    if (warp >= 4 && lane == 0) bulk_wait_all();  // the epilogue's stores are done
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
    if (warp >= 4 && *(volatile uint32_t *)&cta_abort != 0u) leave_nan<D, TOGETHER>(p, threadIdx.x - 128);
}

// Merge of the parts of item whole + blockIdx.x, 32 rows and 8 COLS columns by CTA: lane r has row r, a warp COLS columns. As many
// parts are asked for at once as 64 registers hold (one part after another: 2 x 6 heads x 100 new of 999 tokens 16.1 us and not
// 15.0). The weights l 2^(M - max M) are normalised before they meet the means, so nothing overflows; a part that the row sees
// nothing of has l = 0 and means that do not count.
template <int D, int COLS, bool TOGETHER>
__global__ void __launch_bounds__(256) fwd_paged_merge_kernel(const __grid_constant__ FwdPagedParams p)
{
    constexpr int kPart = paged_part_floats(D), kRows = 2 * BM, kBatch = 64 / COLS;
    static_assert(kMostParts % kBatch == 0);
    __shared__ __align__(16) __nv_bfloat16 rows[32][8 * COLS + 8];
    griddep_wait();
    PagedItem t;
    if (!paged_item<TOGETHER>(p, p.whole + blockIdx.x, false, t)) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, row0 = 256 * t.qb + 32 * static_cast<int>(blockIdx.y);
    if (row0 >= (TOGETHER ? p.rows : t.count)) return;
    const auto valid = [&](int row) {
        int head;
        return token_of<TOGETHER>(p, row, head) < t.count && (!TOGETHER || row < p.rows);
    };
    const int col0 = 8 * COLS * static_cast<int>(blockIdx.z);
    const float *part = p.part + static_cast<size_t>(blockIdx.x) * p.parts * kPart + 32 * blockIdx.y + lane;
    // the parts that have tiles
    const uint32_t some = __ballot_sync(
        0xffffffffu, lane < p.parts && part_begin(t.n, lane, p.parts) < part_begin(t.n, lane + 1, p.parts));
    const auto in = [&](int q) { return (some >> q & 1) != 0; };
    float M[kMostParts], l[kMostParts], x[kBatch][COLS], top = -INFINITY, sum = 0.f, o[COLS] = {};
    uint32_t seen = 0;  // parts that the row sees something of: a NaN among their means stays one whatever its weight
    const auto load = [&](int q0) {
#pragma unroll
        for (int q = 0; q < kBatch; ++q)
#pragma unroll
            for (int c = 0; c < COLS; ++c) x[q][c] = in(q0 + q) ? __ldcg(part + (q0 + q) * kPart + (col0 + COLS * warp + c) * kRows) : 0.f;
    };
#pragma unroll
    for (int q = 0; q < kMostParts; ++q) {
        M[q] = in(q) ? __ldcg(part + q * kPart + D * kRows) : 0.f;
        l[q] = in(q) ? __ldcg(part + q * kPart + (D + 1) * kRows) : 0.f;
    }
    load(0);
#pragma unroll
    for (int q = 0; q < kMostParts; ++q)
        if (l[q] != 0.f) top = fmaxf(top, M[q]), seen |= 1u << q;
#pragma unroll
    for (int q = 0; q < kMostParts; ++q) {
        if (l[q] != 0.f) l[q] *= ex2_approx(M[q] - top);
        sum += l[q];
    }
    const float inv = sum == 0.f ? 0.f : 1.0f / sum;
#pragma unroll
    for (int q0 = 0; q0 < kMostParts; q0 += kBatch) {
        if (q0 >= p.parts) break;
        if (q0 > 0) load(q0);
#pragma unroll
        for (int q = 0; q < kBatch; ++q)
#pragma unroll
            for (int c = 0; c < COLS; ++c) o[c] = seen >> (q0 + q) & 1 ? fmaf(x[q][c], l[q0 + q] * inv, o[c]) : o[c];
    }
#pragma unroll
    for (int c = 0; c < COLS; c += 2) *reinterpret_cast<uint32_t *>(&rows[lane][COLS * warp + c]) = pack_bf16x2(o[c], o[c + 1]);
    if (warp == 0 && col0 == 0 && p.lse && valid(row0 + lane))
        p.lse[static_cast<size_t>(t.bh) * p.rows + row0 + lane] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.69314718055994531f;
    __syncthreads();
    const int d = p.pg.d;
    for (int i = threadIdx.x; i < 32 * COLS; i += 256) {  // pieces of 8 elements
        const int r = i / COLS, c = i % COLS * 8;
        if (valid(row0 + r) && col0 + c < d)
            *reinterpret_cast<uint4 *>(p.out + (static_cast<size_t>(t.bh) * p.rows + row0 + r) * d + col0 + c) =
                *reinterpret_cast<const uint4 *>(&rows[r][c]);
    }
}

template <int D, bool TOGETHER>
cudaError_t launch(FwdPagedParams &p, const alibi_pages *pages, const void *q, cudaStream_t stream)
{
    using C = Cfg<D>;
    const uint64_t d = static_cast<uint64_t>(pages->d);
    const uint32_t box = static_cast<uint32_t>(std::min(pages->slots, BN));
    if (!encode_tmap_bf16_3d(&p.tq, q, d, p.rows, p.BH, 64, BM) || !encode_tmap_bf16_3d(&p.tout, p.out, d, p.rows, p.BH, 32, 32, false) ||
        !encode_pages(&p.tk, &p.tv, pages, 64, box, box == static_cast<uint32_t>(BN)))
        return cudaErrorInvalidValue;
    const auto kern = [&] {
        if constexpr (TOGETHER) return &fwd_paged_kernel<D, true, true>;
        else return p.hold >= 0 || *std::max_element(p.slope, p.slope + p.H) > kSteep ? &fwd_paged_kernel<D, true, false> : &fwd_paged_kernel<D, false, false>;
    }();
    cudaError_t e = prepare_kernel(reinterpret_cast<const void *>(kern), C::kSmem, kLaunchRegs);
    if (e != cudaSuccess) return e;
    const int sms = num_sms();
    p.rest = p.num_items % sms;
    p.whole = p.num_items - p.rest;
    p.parts = paged::parts_of(p.rest, p.BH, p.T, p.rows, p.L, sms).parts;
    if (p.parts == 1) p.whole = p.num_items, p.rest = 0;
    p.num_units = p.whole + p.rest * p.parts;
    p.div_rest = Divisor(static_cast<uint32_t>(std::max(p.rest, 1)));
    p.part = nullptr;
    const dim3 grid(static_cast<unsigned>(std::min(p.num_units, sms)));
    if (p.parts == 1) return launch_kernel(kern, grid, kThreads, C::kSmem, stream, p);
    e = cudaMallocFromPoolAsync(reinterpret_cast<void **>(&p.part), static_cast<size_t>(p.rest) * p.parts * paged_part_floats(D) * sizeof(float),
                                decode_pool(), stream);
    if (e != cudaSuccess) return e;
    e = launch_kernel(kern, grid, kThreads, C::kSmem, stream, p);
    // Of few partials a warp merges four columns, of many its eighth of all (32 x 64 new of 1024 tokens 14.7 us in eighths and 14.1
    // in fours, 32 x 256 of 32768 112.5 and 116.3).
    const unsigned rows = std::min(8, (p.rows + 31) / 32), slices = static_cast<unsigned>(pages->d + 31) / 32;
    const bool few = p.rest * rows * slices <= 2u * sms;
    if (e == cudaSuccess)
        e = launch_kernel(few ? fwd_paged_merge_kernel<D, 4, TOGETHER> : fwd_paged_merge_kernel<D, D / 8, TOGETHER>,
                          dim3(static_cast<unsigned>(p.rest), rows, few ? slices : 1), 256, 0, stream, p);
    const cudaError_t f = cudaFreeAsync(p.part, stream);
    return e != cudaSuccess ? e : f;
}

bool aligned(const void *p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// hold, wait_ns: of the self-test, else -1 and the usual limit
int fwd_paged(const void *q, const alibi_pages *pages, const int *lens, const int *count, void *out, float *lse, int B, int H, int T,
              int L, const float *slopes, void *stream, int hold, uint64_t wait_ns)
{
    const int st = check_pages(pages);
    if (st != ALIBI_OK) return st;
    if (!q || !out || !aligned(q, 16) || !aligned(out, 16) || !aligned(lens, 4) || !aligned(count, 4) || !aligned(lse, 4))
        return ALIBI_ERR_INVALID;
    if (B < 1 || H < 1 || T < 1 || L < 1 || H % pages->heads != 0) return ALIBI_ERR_INVALID;
    if (static_cast<long long>(L) > static_cast<long long>(pages->width) * pages->slots) return ALIBI_ERR_INVALID;
    if (H > kMaxQueryHeads || T > (1 << 24)) return ALIBI_ERR_UNSUPPORTED;
    const int blocks = (T + 255) / 256;
    if (static_cast<long long>(B) * H * blocks > (1LL << 30)) return ALIBI_ERR_UNSUPPORTED;
    if (slopes)
        for (int h = 0; h < H; ++h)
            if (!std::isfinite(slopes[h]) || slopes[h] < 0.0f) return ALIBI_ERR_INVALID;
    FwdPagedParams p;
    if (slopes)
        for (int h = 0; h < H; ++h) p.slope[h] = static_cast<float>(static_cast<double>(slopes[h]) * 1.4426950408889634);
    else
        fill_slopes_log2e(H, p.slope);
    // A slope beyond 1e30 is 1e30: the bias of the next token is out of reach already, and its multiples stay finite.
    for (int h = 0; h < H; ++h) p.slope[h] = std::min(p.slope[h], 1e30f);
    p.pg = pages_of(pages);
    p.lens = lens;
    p.count = count;
    p.out = static_cast<__nv_bfloat16 *>(out);
    p.lse = lse;
    p.err = device_status_word();
    if (!p.err) return ALIBI_ERR_CUDA;
    p.T = T;
    p.L = L;
    p.BH = B * H;
    p.H = H;
    p.rows = T;
    p.G = H / pages->heads;
    p.blocks = blocks;
    p.hold = hold;
    p.wait_ns = wait_ns;
    const bool join = hold < 0 && paged::together(p.BH, p.G, T, L, num_sms());
    if (join) {
        p.BH = B * pages->heads;
        p.H = pages->heads;
        p.rows = p.G * T;
        p.blocks = (p.rows + 255) / 256;
    }
    p.num_items = p.BH * p.blocks;
    p.div_bh = Divisor(static_cast<uint32_t>(p.BH));
    p.div_h = Divisor(static_cast<uint32_t>(p.H));
    p.div_g = Divisor(static_cast<uint32_t>(p.H / pages->heads));
    p.div_t = Divisor(static_cast<uint32_t>(T));
    p.c1 = 1.4426950408889634f / sqrtf(static_cast<float>(pages->d));
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    const cudaError_t e = pages->d == 128 ? (join ? launch<128, true>(p, pages, q, cs) : launch<128, false>(p, pages, q, cs))
                                          : (join ? launch<64, true>(p, pages, q, cs) : launch<64, false>(p, pages, q, cs));
    return e == cudaSuccess ? ALIBI_OK : ALIBI_ERR_CUDA;
}

}  // namespace
}  // namespace alibi

using namespace alibi;

extern "C" int alibi_attn_fwd_paged(const void *q, const alibi_pages *pages, const int *lens, const int *count, void *out,
                                    float *lse, int B, int H, int T, int L, const float *slopes, void *stream)
{
    return fwd_paged(q, pages, lens, count, out, lse, B, H, T, L, slopes, stream, -1, kWaitLimitNs);
}

extern "C" int alibi_selftest_fwd_paged_timeout(const void *q, const alibi_pages *pages, const int *lens, const int *count, void *out,
                                                float *lse, int B, int H, int T, int L, int barrier, int wait_us, void *stream)
{
    if (barrier < 0 || barrier >= HOLD_COUNT || !selftest_wait(wait_us)) return ALIBI_ERR_INVALID;
    return fwd_paged(q, pages, lens, count, out, lse, B, H, T, L, nullptr, stream, barrier, static_cast<uint64_t>(wait_us) * 1000u);
}
