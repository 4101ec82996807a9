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
    // page of token j of sequence b, -1 for a number that is none of a page
    __device__ __forceinline__ int page_of(int b, int j) const
    {
        const int id = table[static_cast<size_t>(b) * width + (j >> shift)];
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

// 4-D tiled load of one box of `bytes` bytes, a power of two, into shared memory, completing on `bar`. It lies on a multiple of
// its size or of 1024, where the swizzle's pattern begins anew.
__device__ __forceinline__ void tma_load_4d(void *dst, const void *tmap, int x, int y, int z, int w, uint32_t bytes, uint64_t *bar)
{
#ifdef ALIBI_CHECKS
    if (!check::tma_x_aligned(x)) return check_fail(check::TMA_LOAD, static_cast<uint32_t>(x));
    if (!check_smem(smem_u32(dst), bytes, bytes < 1024 ? bytes : 1024)) return check_fail(check::TMA_LOAD, smem_u32(dst));
#endif
    (void)bytes;
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
        : "memory");
}

// Maps of the keys' and values' pools for boxes of `box0` elements of `box1` slots of one head of one page.
inline bool encode_pages(CUtensorMap *tk, CUtensorMap *tv, const alibi_pages *p, uint32_t box0, uint32_t box1)
{
    const uint64_t dims[4] = {static_cast<uint64_t>(p->d), static_cast<uint64_t>(p->slots), static_cast<uint64_t>(p->heads),
                              static_cast<uint64_t>(p->pages)};
    const uint64_t ks[3] = {2ull * p->k_slot, 2ull * p->k_head, 2ull * p->k_page};
    const uint64_t vs[3] = {2ull * p->v_slot, 2ull * p->v_head, 2ull * p->v_page};
    return encode_tmap_bf16_4d(tk, p->k, dims, ks, box0, box1) && encode_tmap_bf16_4d(tv, p->v, dims, vs, box0, box1);
}

}  // namespace alibi
