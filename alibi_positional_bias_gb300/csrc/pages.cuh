// The paged KV cache as the kernels see it (include/alibi.h, alibi_pages), and the host's checks of it.
#pragma once

#include <cuda_bf16.h>

#include "alibi.h"
#include "internal.h"
#include "ptx.cuh"

namespace alibi {

struct Pages {
    __nv_bfloat16 *k, *v;
    long long k_page, k_head, k_slot, v_page, v_head, v_slot;  // strides in elements
    const int *table;                                          // [B, width]
    int pages, heads, shift, width, d;                         // shift: log2 of a page's slots

    __device__ __forceinline__ int slot_of(int j) const { return j & ((1 << shift) - 1); }
    // entry of the table for token j of sequence b
    __device__ __forceinline__ int number(int b, int j) const { return table[static_cast<size_t>(b) * width + (j >> shift)]; }
    // page of token j of sequence b, -1 for a number that is none of a page
    __device__ __forceinline__ int page_of(int b, int j) const
    {
        const int id = number(b, j);
        return static_cast<unsigned>(id) < static_cast<unsigned>(pages) ? id : -1;
    }
};

// Head sizes of the paged calls; a page has a power of two of 8 to 1024 slots.
inline int check_pages(const alibi_pages *p)
{
    const auto aligned = [](const void *a, unsigned n) { return (reinterpret_cast<uintptr_t>(a) & (n - 1)) == 0; };
    if (!p || !p->k || !p->v || !p->table) return ALIBI_ERR_INVALID;
    if (!aligned(p->k, 16) || !aligned(p->v, 16) || !aligned(p->table, 4)) return ALIBI_ERR_INVALID;
    if (p->pages < 1 || p->heads < 1 || p->slots < 1 || p->width < 1 || p->d < 1) return ALIBI_ERR_INVALID;
    if (!decode_supports(p->d)) return ALIBI_ERR_UNSUPPORTED;
    if (p->slots < 8 || p->slots > 1024 || (p->slots & (p->slots - 1)) != 0) return ALIBI_ERR_UNSUPPORTED;
    if (p->heads > kMaxQueryHeads || static_cast<long long>(p->width) * p->slots > (1LL << 24)) return ALIBI_ERR_UNSUPPORTED;
    for (const long long s : {p->k_page, p->k_head, p->k_slot, p->v_page, p->v_head, p->v_slot}) {
        if (s < p->d || s % 8 != 0) return ALIBI_ERR_INVALID;
        if (s >= (1LL << 38)) return ALIBI_ERR_UNSUPPORTED;  // 2^39 bytes
    }
    return ALIBI_OK;
}

// Limits that the self-tests of the failure paths take: the waits for copies and MMAs in flight have the same one, and these are to
// have ended before the kernel does.
inline bool selftest_wait(int wait_us) { return wait_us >= 1000 && wait_us <= 1000000; }

inline Pages pages_of(const alibi_pages *p)
{
    Pages g;
    g.k = static_cast<__nv_bfloat16 *>(p->k);
    g.v = static_cast<__nv_bfloat16 *>(p->v);
    g.k_page = p->k_page, g.k_head = p->k_head, g.k_slot = p->k_slot;
    g.v_page = p->v_page, g.v_head = p->v_head, g.v_slot = p->v_slot;
    g.table = p->table;
    g.pages = p->pages;
    g.heads = p->heads;
    g.shift = 0;
    while ((1 << g.shift) < p->slots) ++g.shift;
    g.width = p->width;
    g.d = p->d;
    return g;
}

// Load of one box of a page: `box` slots from `slot` on of head `head`, WIDTH elements of each from WIDTH `half` on (a row of fewer is
// filled up with zeros), of `halves` parts, as the map has them, one after the other. It completes on `bar`.
template <int WIDTH>
__device__ __forceinline__ void load_box(void *dst, const void *tmap, const Pages &pg, int box, int halves, int slot, int half, int head,
                                         int page, uint64_t *bar)
{
#ifdef ALIBI_CHECKS
    const int parts = pg.d > WIDTH ? pg.d / WIDTH : 1;
    if (!check::page_box(slot, half, head, page, box, halves, 1 << pg.shift, parts, pg.heads, pg.pages))
        return check_fail(check::PAGE_BOX, static_cast<uint32_t>(slot));
    if (!check_smem(smem_u32(dst), check::page_box_bytes(box, halves, WIDTH), check::page_box_align(box, WIDTH)))
        return check_fail(check::TMA_LOAD, smem_u32(dst));
#endif
    (void)pg, (void)box, (void)halves;
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(0), "r"(slot), "r"(half), "r"(head), "r"(page), "r"(smem_u32(bar))
        : "memory");
}

// Maps of the keys' and values' pools for boxes of `box` slots of one head of one page: rows of `width` elements, of one half of
// d = 128 or (`both`) of the one and then of the other: each copy that a warp issues takes it 40 cycles or more (64 x 40 x 8192
// tokens decoded in 1448 us with one half at a time, 1407 with both).
inline bool encode_pages(CUtensorMap *tk, CUtensorMap *tv, const alibi_pages *p, uint32_t width, uint32_t box, bool both)
{
    const uint64_t d = static_cast<uint64_t>(p->d), part = d < 64 ? d : 64;
    const uint64_t dims[5] = {part, static_cast<uint64_t>(p->slots), d / part, static_cast<uint64_t>(p->heads),
                              static_cast<uint64_t>(p->pages)};
    const uint64_t ks[4] = {2ull * p->k_slot, 128, 2ull * p->k_head, 2ull * p->k_page};
    const uint64_t vs[4] = {2ull * p->v_slot, 128, 2ull * p->v_head, 2ull * p->v_page};
    const uint32_t halves = both ? static_cast<uint32_t>(d / part) : 1;
    return encode_tmap_bf16_5d(tk, p->k, dims, ks, width, box, halves) && encode_tmap_bf16_5d(tv, p->v, dims, vs, width, box, halves);
}

}  // namespace alibi
