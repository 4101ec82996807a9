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
//   values    that some row of the item does not see meet a weight of zero, which an infinity or a NaN would turn into NaN: two
//             warps look through the first tiles' values, those that some row does not see whole (up to three of an item),
//             put zeros in place of what is not finite and note per column the first such row, from which on the
//             outputs are NaN. The scores and the softmax of the tile run meanwhile.
//   rows      past count_b are left as they were: of a box of 32 rows that reaches there the lanes store their own.
//
// Steep heads (slopes above 4 / log2(e)) take the bias element by element from the whole distance, where the column part on
// the tensor core and the row part would cancel with a rounding of 2^-24 of 128 slopes.

#include <algorithm>
#include <cmath>
#include <cuda.h>
#include <type_traits>

#include "alibi.h"
#include "divide.h"
#include "fwd_tiles.cuh"
#include "pages.cuh"
#include "ptx.cuh"

namespace alibi {
namespace {

constexpr float kSteep = 4.0f;  // m log2(e)

struct FwdPagedParams {
    CUtensorMap tq;      // [B H, T, d] bf16, box {64, 128, 1}, 128-byte swizzle
    CUtensorMap tk, tv;  // [pages, heads, slots, d] by strides, box {64, min(slots, 128), 1, 1}, 128-byte swizzle
    CUtensorMap tout;    // [B H, T, d] bf16, box {32, 32, 1}, no swizzle (epilogue stores)
    Pages pg;
    const int *lens, *count;
    __nv_bfloat16 *out;
    float *lse;
    uint32_t *err;
    int T, L, BH, H, num_items, blocks;  // blocks of 256 rows of a head
    Divisor div_bh, div_h, div_g;        // by B H, H and H / H_kv
    float c1;                            // log2(e) / sqrt(d)
    float slope[kMaxQueryHeads];         // m log2(e)
};

enum : uint32_t {
    SITE_PG_Q = 0x401, SITE_PG_UNIT = 0x402, SITE_PG_FIX = 0x403, SITE_PG_P = 0x404, SITE_PG_O = 0x405, SITE_PG_DONE = 0x406,
    SITE_PG_S = 0x407,
};

struct PagedItem {
    int bh, qb;
    int len, count;   // of the sequence
    int first;        // position of its query 0
    int top, n;       // newest key tile, and tiles visited: top, top - 1, ..., 0
    int n_fix;        // of which the first have keys that some row does not see
    int first0;       // iteration at which slot 0 begins
    bool q1valid, bad;
};

// Work item at position idx, or false where the sequence has no rows there. Longest first: round r holds block blocks - 1 - r
// of every head.
__device__ __forceinline__ bool paged_item(const FwdPagedParams &p, int idx, PagedItem &t)
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
    if (256 * t.qb >= t.count) return false;
    t.first = t.len - t.count;
    t.q1valid = 256 * t.qb + BM < t.count;
    const int i0 = t.first + 256 * t.qb;  // position of the item's first row
    const int top0 = max(0, min(i0 + BM - 1, t.len - 1)) >> 7, top1 = max(0, min(i0 + 2 * BM - 1, t.len - 1)) >> 7;
    t.top = t.q1valid ? top1 : top0;
    t.n = t.top + 1;
    t.n_fix = max(1, t.top + 1 - ((max(i0, 0) + 1) >> 7));
    t.first0 = t.top - top0;
    return true;
}

__device__ __forceinline__ int paged_index(int k)
{
    const int G = gridDim.x, c = blockIdx.x;
    return (k & 1) ? (k + 1) * G - 1 - c : k * G + c;
}

__device__ __forceinline__ bool paged_active(const PagedItem &t, int s, int it) { return s == 1 ? t.q1valid : it >= t.first0; }

template <int D>
__global__ void __launch_bounds__(kThreads, 1) fwd_paged_kernel(const __grid_constant__ FwdPagedParams p)
{
    using C = Cfg<D>;
    extern __shared__ uint8_t smem_raw[];
    // of the items in flight, two at most: the first row of each column of V that is not finite, whether each half of the
    // columns has one, and whether a page number is none
    __shared__ int odd_from[2][D];
    __shared__ int odd_any[2][2], lost[2];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::kBar);
    uint64_t *q_full = bars + 0;      // both Q tiles of the item loaded
    uint64_t *q_empty = bars + 1;
    uint64_t *unit_full = bars + 2;   // [2] ring unit of stage s loaded (K(u) and V(u - 1))
    uint64_t *unit_empty = bars + 4;  // [2] ring unit of stage s read by the MMAs
    uint64_t *s_full = bars + 6;      // [2]
    uint64_t *p_full = bars + 8;      // [2] P of keys 0..63 written
    uint64_t *p_hi = bars + 10;       // [2] P of keys 64..127 written
    uint64_t *o_full = bars + 12;     // [2]
    uint64_t *o_empty = bars + 14;    // [2]
    uint64_t *bias_full = bars + 16;  // [2] column-bias operand of item k written (buffer k & 1)
    uint64_t *v_ready = bars + 18;    // values that some row does not see have landed
    uint64_t *v_fixed = bars + 19;    // and are finite
    uint64_t *mma_done = bars + 20;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 21);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    uint32_t *err = p.err;

    if (threadIdx.x == 0) {
        cta_err_init(kWaitLimitNs);
        cta_check_init(p.err, smem_raw, C::kSmem);
        for (int s = 0; s < 2; ++s) {
            mbar_init(&unit_full[s], 1);
            mbar_init(&unit_empty[s], 1);
            mbar_init(&s_full[s], 1);
            mbar_init(&p_full[s], 4);  // one arrival per softmax warp
            mbar_init(&p_hi[s], 4);
            mbar_init(&o_full[s], 1);
            mbar_init(&o_empty[s], 4);
            mbar_init(&bias_full[s], 4);  // the slot-0 softmax warps
        }
        mbar_init(q_empty, 1);
        mbar_init(q_full, 1);
        mbar_init(v_ready, 1);
        mbar_init(v_fixed, 2);  // the two warps that look through them
        mbar_init(mma_done, 1);
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
    griddep_wait();  // the kernel before, which may have written what this one reads, is done

    if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsLow));
    if (warp == 0) {
        // ------------------------------------------------------ TMA producer
        const int box = min(1 << p.pg.shift, BN), boxes = BN / box;  // rows of a box, boxes of a tile
        uint32_t uc = 0;  // ring units issued
        int kk = 0;       // items begun
        bool ok = true;
        for (int k = 0; ok; ++k) {
            const int w = paged_index(k);
            if (w >= p.num_items) break;
            PagedItem t;
            if (!paged_item(p, w, t)) continue;
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
                lost[kk & 1] = 0;
                mbar_arrive_expect_tx(q_full, 2 * C::kTileBytes);
                for (int s = 0; s < 2; ++s)
                    for (int c = 0; c < C::kChunks; ++c)
                        tma_load_3d(smem + C::kQ + s * C::kTileBytes + c * C::kChunkBytes, &p.tq, 64 * c, (2 * t.qb + s) * BM,
                                    t.bh, q_full);
            }
            __syncwarp();
            // Unit u = 0 .. n: K(u) (u < n) and V(u - 1) (u >= 1), consumed in the MMA issuer's iteration u - 1.
            for (int u = 0; u <= t.n; ++u) {
                const uint32_t st = uc % 2, ph = (uc / 2) & 1;
                if (page < 0) lost[kk & 1] = 1, page = p.pg.pages;
                const int ahead = page_at(t.top - u - 1);
                ok = __all_sync(0xffffffffu, mbar_wait(&unit_empty[st], ph ^ 1, err, SITE_PG_UNIT));
                if (!ok) break;
                if (lane == 0)
                    mbar_arrive_expect_tx(&unit_full[st], (u < t.n ? C::kTileBytes : 0u) + (u >= 1 ? C::kTileBytes : 0u));
                __syncwarp();
                if (lane < boxes) {
                    const int at = lane * box * 128;  // of the box in a swizzle atom
                    for (int c = 0; c < C::kChunks; ++c) {
                        if (u < t.n)
                            tma_load_4d(smem + C::kK + st * C::kTileBytes + c * C::kChunkBytes + at, &p.tk, 64 * c,
                                        p.pg.slot_of((t.top - u) * BN + lane * box), hk, page, box * 128, &unit_full[st]);
                        if (u >= 1)
                            tma_load_4d(smem + C::kV + st * C::kTileBytes + c * C::kChunkBytes + at, &p.tv, 64 * c,
                                        p.pg.slot_of((t.top - u + 1) * BN + lane * box), hk, before, box * 128, &unit_full[st]);
                    }
                }
                before = page;
                page = ahead;
                ++uc;
            }
            ++kk;  // after an error too: the item's Q was issued
        }
        // Drain (also after an error): the last Q load and the last load into each ring stage has landed before the CTA can
        // exit. Earlier loads into a stage were consumed, hence complete, before the stage was reused.
        if (kk > 0) mbar_wait(q_full, (kk - 1) & 1, err, SITE_PG_Q, true);
        for (uint32_t n = uc > 2 ? uc - 2 : 0; n < uc; ++n) mbar_wait(&unit_full[n % 2], (n / 2) & 1, err, SITE_PG_UNIT, true);
    } else if (warp == 1) {
        // -------------------------------------------------------- MMA issuer (converged; one elected lane issues)
        constexpr uint32_t idS = idesc_bf16_f32(BM, BN, 0);
        constexpr uint32_t idO = idesc_bf16_f32(BM, D, 1);
        const uint32_t sQ = smem_u32(smem + C::kQ);
        const uint32_t sK = smem_u32(smem + C::kK);
        const uint32_t sV = smem_u32(smem + C::kV);
        const uint64_t auxd = smem_desc_sw128(smem_u32(smem + C::kAux), 16, 1024);
        uint32_t uc = 0;  // ring units consumed
        uint32_t p_cnt[2] = {0, 0}, o_cnt[2] = {0, 0}, f_cnt = 0;
        int kk = 0;
        bool ok = true;
        for (int k = 0; ok; ++k) {
            const int w = paged_index(k);
            if (w >= p.num_items) break;
            PagedItem t;
            if (!paged_item(p, w, t)) continue;
            const bool aux = p.slope[p.div_h.rest(t.bh)] <= kSteep;
            ok = mbar_wait(q_full, kk & 1, err, SITE_PG_Q);
            if (ok) ok = mbar_wait(&bias_full[kk & 1], (kk >> 1) & 1, err, SITE_PG_Q);
            // an idle slot's epilogue of an earlier item reads what this item's values will overwrite (odd_from)
            if (ok && !t.q1valid) ok = mbar_wait(&o_empty[1], (o_cnt[1] & 1) ^ 1, err, SITE_PG_O);
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
                if (aux) mma_ss_w(dst, auxd, auxd + 2 * (1 + (kk & 1)), idS, 1u);
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
                bool fix = it < t.n_fix;
                if (fix && lane == 0) mbar_arrive(v_ready);
                for (int s = 0; s < 2 && ok; ++s) {
                    if (paged_active(t, s, it)) {
                        ok = mbar_wait_spin(&p_full[s], p_cnt[s] & 1, err, SITE_PG_P);
                        if (ok && first_pv[s]) ok = mbar_wait(&o_empty[s], (o_cnt[s] & 1) ^ 1, err, SITE_PG_O);
                        if (ok && fix) {  // once a tile, whichever slot comes first
                            ok = mbar_wait(v_fixed, f_cnt++ & 1, err, SITE_PG_FIX);
                            fix = false;
                        }
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
                        if (it == t.n - 1) {
                            mma_commit_w(&o_full[s]);
                            ++o_cnt[s];
                        }
                    }
                    if (it + 1 < t.n && paged_active(t, s, it + 1)) issue_S(s, vst);
                }
                mma_commit_w(&unit_empty[vst]);  // the unit's V and K have both been read
                ++uc;
            }
            mma_commit_w(q_empty);
            ++kk;
        }
        // drain: every MMA issued above completes before TMEM is released
        mma_commit_w(mma_done);
        mbar_wait(mma_done, 0, err, SITE_PG_DONE, true);
    } else {
        // ------------------------------------ values that some row does not see: what is not finite becomes zero
        // Each of the two warps has half of the columns.
        constexpr int kPieces = D / 16;  // of 16 bytes of a row
        const int side = warp - 2;
        uint32_t uc = 0, r_cnt = 0;
        int kk = 0;
        bool ok = true;
        for (int k = 0; ok; ++k) {
            const int w = paged_index(k);
            if (w >= p.num_items) break;
            PagedItem t;
            if (!paged_item(p, w, t)) continue;
            int *from = odd_from[kk & 1];
            for (int it = 0; it < t.n_fix; ++it) {
                // The MMA issuer has seen the tile land; it is past the item before, and so are the epilogues of the item
                // before that, which read this item's buffers.
                ok = __all_sync(0xffffffffu, mbar_wait(v_ready, r_cnt++ & 1, err, SITE_PG_FIX));
                if (!ok) break;
                if (it == 0) {
                    for (int e = lane; e < D / 2; e += 32) from[side * (D / 2) + e] = 0x7fffffff;
                    if (lane == 0) odd_any[kk & 1][side] = 0;
                    __syncwarp();
                }
                const uint32_t st = (uc + it + 1) % 2;
                uint8_t *v = smem + C::kV + st * C::kTileBytes;
                const int row0 = (t.top - it) * BN;
#pragma unroll 4
                for (int x = lane; x < BN * kPieces; x += 32) {
                    const int row = x / kPieces, piece = side * kPieces + x % kPieces;
                    uint8_t *at = v + piece / 8 * C::kChunkBytes + row * 128 + (((piece ^ row) & 7) << 4);
                    const uint4 y = *reinterpret_cast<const uint4 *>(at);
                    // a half whose exponent is full overflows into bit 15 when one is added to it
                    const auto odd = [](uint32_t a) { return ((a & 0x7f807f80u) + 0x00800080u) & 0x80008000u; };
                    if ((odd(y.x) | odd(y.y) | odd(y.z) | odd(y.w)) == 0u) continue;
                    uint32_t a[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const uint32_t m = 0x7f80u << (16 * (e & 1));
                        if ((a[e / 2] & m) != m) continue;
                        a[e / 2] &= ~(0xffffu << (16 * (e & 1)));
                        if (row0 + row < t.len) {
                            atomicMin(&from[8 * piece + e], row0 + row);
                            odd_any[kk & 1][side] = 1;
                        }
                    }
                    *reinterpret_cast<uint4 *>(at) = make_uint4(a[0], a[1], a[2], a[3]);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(v_fixed);
            }
            uc += t.n + 1;
            ++kk;
        }
    }
    } else {
        // ------------------------------------------------ softmax warpgroups
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsHigh));
        const int s = (warp - 4) >> 2;
        const int quad = warp & 3;  // TMEM lane quadrant this warp may access
        const int r = quad * 32 + lane;
        const uint32_t lane_addr = tmem + (static_cast<uint32_t>(quad * 32) << 16);
        uint32_t s_cnt = 0, o_cnt = 0;
        int kk = 0, k_bias = 0, kk_bias = 0;  // items begun; of the bias operands, position of the next and number of it
        bool ok = true;
        for (int k = 0; ok; ++k) {
            const int w = paged_index(k);
            if (w >= p.num_items) break;
            PagedItem t;
            if (!paged_item(p, w, t)) continue;
            if (s == 0) {
                // Column-bias operand, one row per thread, one item ahead: every MMA that read that buffer for the item
                // before the last completed before this warp's epilogue of the last one.
                while (kk_bias <= kk + 1) {
                    const int wn = paged_index(k_bias++);
                    if (wn >= p.num_items) break;
                    PagedItem tn;
                    if (!paged_item(p, wn, tn)) continue;
                    const float m = p.slope[p.div_h.rest(tn.bh)];
                    write_bias_row(smem + C::kAux, r, kk_bias & 1, m <= kSteep ? m * static_cast<float>(r) / p.c1 : 0.0f);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bias_full[kk_bias & 1]);
                    ++kk_bias;
                }
            }
            const int buf = kk++ & 1;
            if (s == 1 && !t.q1valid) continue;
            const int row0 = (2 * t.qb + s) * BM + quad * 32;  // query token of the warp's first row
            const int i = t.first + row0 + lane;               // position of this thread's row
            const int i_warp = t.first + row0;
            const float sl2 = p.slope[p.div_h.rest(t.bh)];
            const bool steep = sl2 > kSteep;
            const int it0 = s == 0 ? t.first0 : 0;
            float M = 0.f, l = 0.f;
            for (int it = it0; it < t.n; ++it) {
                const int j = t.top - it;
                ok = mbar_wait(&s_full[s], s_cnt & 1, err, SITE_PG_S);
                ++s_cnt;
                ok = __all_sync(0xffffffffu, ok);  // keep the warp converged for tcgen05.ld
                if (!ok) break;
                tc_fence_after();
                uint32_t sraw[BN];
#pragma unroll
                for (int c = 0; c < BN / 32; ++c)
                    tmem_ld32(lane_addr + s * 128 + c * 32, *reinterpret_cast<uint32_t(*)[32]>(&sraw[c * 32]));
                tmem_wait_ld();
                // After a row's first tile x is relative to the running maximum M.
                const bool rel = it != it0;
                const float di = static_cast<float>(i - j * BN);  // exact: |i - k0| < 2^24
                float x[BN];
                if (!steep) {
                    const float2 c1v = make_float2(p.c1, p.c1);
                    const float rb = -sl2 * di - (rel ? M : 0.f);
                    const float2 rbv = make_float2(rb, rb);
#pragma unroll
                    for (int u = 0; u < BN / 2; ++u) {
                        const float2 xv = __ffma2_rn(
                            make_float2(__uint_as_float(sraw[2 * u]), __uint_as_float(sraw[2 * u + 1])), c1v, rbv);
                        x[2 * u] = xv.x;
                        x[2 * u + 1] = xv.y;
                    }
                } else {
                    const float less = rel ? -M : 0.f;
#pragma unroll
                    for (int c = 0; c < BN; ++c)
                        x[c] = fmaf(sl2, static_cast<float>(c) - di, fmaf(__uint_as_float(sraw[c]), p.c1, less));
                }
                if (j * BN + BN - 1 > i_warp) {  // some row of the warp does not see all keys
                    const int lim = i - j * BN;
#pragma unroll
                    for (int c = 0; c < BN; ++c) x[c] = c > lim ? -INFINITY : x[c];
                }
                const float mt = row_max128(x);
                // Raise the running maximum lazily, only when this tile exceeds it by 2^8, or where the row has seen nothing
                // so far (then M is 0 and O is 0). O_s is quiescent here: S_s(it) completing implies that the product
                // before it has completed.
                const bool none = l == 0.f;
                const bool need = rel && (mt > kRescaleThreshold || (none && mt > -INFINITY));
                if (it == it0) M = mt == -INFINITY ? 0.f : mt;
                if (__any_sync(0xffffffffu, need)) {
                    const float alpha = need && !none ? ex2_approx(-mt) : 1.0f;
                    if (need) {
                        M += mt;
                        l *= alpha;
                    }
#pragma unroll
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t o[32];
                        tmem_ld32(lane_addr + 256 + s * 128 + c * 32, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int u = 0; u < 32; ++u) o[u] = __float_as_uint(__uint_as_float(o[u]) * alpha);
                        tmem_st32(lane_addr + 256 + s * 128 + c * 32, o);
                    }
                }
                const float shift = rel ? (need ? mt : 0.f) : M;  // what the exponent still needs subtracted
                float2 acc[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                // Two halves of 64 keys: the first half of P is handed to the MMA issuer while the second is exponentiated.
                uint32_t pk[BN / 2];
                auto exps = [&](auto sub_c) {
                    const float2 negs = make_float2(-shift, -shift);
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
#pragma unroll
                        for (int u = half * (BN / 4); u < (half + 1) * (BN / 4); ++u) {
                            float2 dv = make_float2(x[2 * u], x[2 * u + 1]);
                            if (decltype(sub_c)::value) dv = __fadd2_rn(dv, negs);
                            const float2 pv = make_float2(ex2_approx(dv.x), ex2_approx(dv.y));
                            acc[u & 3] = __fadd2_rn(acc[u & 3], pv);
                            pk[u] = pack_bf16x2(pv.x, pv.y);
                        }
                        tmem_st32(lane_addr + s * 128 + half * 32, *reinterpret_cast<uint32_t(*)[32]>(&pk[half * 32]));
                        tmem_wait_st();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(half == 0 ? &p_full[s] : &p_hi[s]);
                    }
                };
                if (__any_sync(0xffffffffu, shift != 0.f))
                    exps(std::true_type{});
                else
                    exps(std::false_type{});
                const float2 a01 = __fadd2_rn(acc[0], acc[1]), a23 = __fadd2_rn(acc[2], acc[3]);
                const float2 a = __fadd2_rn(a01, a23);
                l += a.x + a.y;
            }
            if (!ok) break;
            // ------------------------------------------------------ epilogue
            ok = mbar_wait(&o_full[s], o_cnt & 1, err, SITE_PG_O);
            ++o_cnt;
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after();
            const float nan = __uint_as_float(0x7fc00000u);
            const bool bad = t.bad || *(volatile int *)&lost[buf];
            if (bad && quad == 0 && lane == 0) atomicOr(err, ALIBI_DEV_RANGE);
            const float inv_l = bad ? nan : l == 0.f ? 0.f : 1.0f / l;
            const bool odd = (*(volatile int *)&odd_any[buf][0] | *(volatile int *)&odd_any[buf][1]) != 0;
            const bool valid = row0 + lane < t.count;
            const int dr = D == 64 ? p.pg.d : D;
            // O / l goes out through a per-warp staging box and bulk tensor stores, so that the warp does not wait for its
            // stores before its next tile; of a box that reaches past the sequence's rows each lane stores its own row.
            const bool box = row0 + 32 <= t.count;
            uint8_t *stg = smem + C::kStage + (warp - 4) * 2048;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                if (c * 32 >= dr || row0 >= t.count) break;
                uint32_t o[32];
                tmem_ld32(lane_addr + 256 + s * 128 + c * 32, o);
                tmem_wait_ld();
                uint32_t y[16];
#pragma unroll
                for (int u = 0; u < 16; ++u)
                    y[u] = pack_bf16x2(__uint_as_float(o[2 * u]) * inv_l, __uint_as_float(o[2 * u + 1]) * inv_l);
                if (odd) {
#pragma unroll
                    for (int u = 0; u < 32; ++u)
                        if (i >= odd_from[buf][c * 32 + u]) y[u / 2] |= 0x7fc0u << (16 * (u & 1));
                }
                if (box) {
                    if (lane == 0) bulk_wait_read();  // the previous box has left the staging
                    __syncwarp();
                    uint4 *dst = reinterpret_cast<uint4 *>(stg + lane * 64);
#pragma unroll
                    for (int u = 0; u < 4; ++u) dst[u] = make_uint4(y[4 * u], y[4 * u + 1], y[4 * u + 2], y[4 * u + 3]);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        tma_store_3d(&p.tout, stg, c * 32, row0, t.bh);
                        bulk_commit();
                    }
                } else if (valid) {
                    uint4 *dst = reinterpret_cast<uint4 *>(p.out + (static_cast<size_t>(t.bh) * p.T + row0 + lane) * dr + c * 32);
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        if (c * 32 + 8 * u < dr) dst[u] = make_uint4(y[4 * u], y[4 * u + 1], y[4 * u + 2], y[4 * u + 3]);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&o_empty[s]);
            if (valid && p.lse)
                p.lse[static_cast<size_t>(t.bh) * p.T + row0 + lane] =
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
}

template <int D>
cudaError_t launch(FwdPagedParams &p, const alibi_pages *pages, const void *q, cudaStream_t stream)
{
    using C = Cfg<D>;
    const uint64_t d = static_cast<uint64_t>(pages->d);
    const uint32_t box = static_cast<uint32_t>(std::min(pages->slots, BN));
    if (!encode_tmap_bf16_3d(&p.tq, q, d, p.T, p.BH, 64, BM) || !encode_tmap_bf16_3d(&p.tout, p.out, d, p.T, p.BH, 32, 32, false) ||
        !encode_pages(&p.tk, &p.tv, pages, 64, box))
        return cudaErrorInvalidValue;
    const auto kern = &fwd_paged_kernel<D>;
    const cudaError_t e = prepare_kernel(reinterpret_cast<const void *>(kern), C::kSmem, kLaunchRegs);
    if (e != cudaSuccess) return e;
    return launch_kernel(kern, dim3(static_cast<unsigned>(std::min(p.num_items, num_sms()))), kThreads, C::kSmem, stream, p);
}

bool aligned(const void *p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

}  // namespace
}  // namespace alibi

using namespace alibi;

extern "C" int alibi_attn_fwd_paged(const void *q, const alibi_pages *pages, const int *lens, const int *count, void *out,
                                    float *lse, int B, int H, int T, int L, const float *slopes, void *stream)
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
    p.blocks = blocks;
    p.num_items = p.BH * blocks;
    p.div_bh = Divisor(static_cast<uint32_t>(p.BH));
    p.div_h = Divisor(static_cast<uint32_t>(H));
    p.div_g = Divisor(static_cast<uint32_t>(H / pages->heads));
    p.c1 = 1.4426950408889634f / sqrtf(static_cast<float>(pages->d));
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    const cudaError_t e = pages->d == 128 ? launch<128>(p, pages, q, cs) : launch<64>(p, pages, q, cs);
    return e == cudaSuccess ? ALIBI_OK : ALIBI_ERR_CUDA;
}
