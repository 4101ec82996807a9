// ALiBi attention of the newest tokens of each sequence over its 4-bit KV cache.
//
// Row (h, t) of sequence b is the query of head h at position i = len_b - T + t, with
// len_b tokens in the cache (the new ones included), and h / G its KV head, G = H / H_kv:
//   x_j = q.k_j / sqrt(d) - m_h (i - j),  j <= i,   out = sum_j softmax_j(x) v_j,
// with k and v the values s (u - 8) that the cache's codes stand for (kv4.h).
//
// The G T rows of a KV head share its keys, so up to 8 rows form a chunk that one CTA
// takes over one slice of the sequence. Each warp streams stages of 4608 bytes (128 / D
// blocks) from HBM through a ring of its own in shared memory (cp.async.bulk, one
// mbarrier per stage, no synchronisation between warps) and works on tiles of 16 tokens:
//
//   scores   acc_n = (U_n - 8) Q_n^T per group n of 32 elements, mma.m16n8k16 with u - 8 and
//            q as fp16 operands, both exact: four bits under the exponent of 1024 are 1024 + u
//            (or 1024 + 16 u), and one add or fma per pair leaves u - 8; each group of
//            q is scaled to [2^14, 2^15), which holds elements down to 2^-32 of the group's largest.
//            kappa (s_jn 2^e_n) acc_n is the group's share of the logit: exact products summed in fp32, the
//            powers of two taking the scaling of q back. 2^e_n, a bf16 number of at most 2^-23 (2^-13 for rows of 2^117
//            and more), meets the scale first, exactly, so that the sum over n stays in range; kappa is
//            the row's: s_jn acc_n alone leaves fp32 from keys of 2^113 on.
//            (Masked bits without the 1024 are operands too, the subnormals u 2^-24 and u 2^-20,
//            but the tensor core aligns products by their nominal exponents, which costs 10 and 6
//            bits of the sum: errors of 2^-17 of 8 |s| were measured. Keys as 1024 + 16 u, with the
//            offset in the sum's start, save two operations in nine, but the start takes registers
//            that the loop does not have: 426 -> 440 us at 64 x 40 heads of 8192 tokens.)
//   softmax  in base 2: p_j = 2^(x_j - R), summed in fp32, with a reference R of each row, its first block's largest
//            x_j (so that a row that sees one token has its value exactly), which is raised by a whole number when some
//            x_j exceeds it by 8. A weight below 2^-126 of the row's largest counts as zero.
//   values   O^T += (U - 8)^T P^T per group, P_jn = p_j s_jn F_n as fp16, with a power of two F_n of each row
//            and group that puts the largest |p_j s_jn| so far at 2^7 or more and is lowered when one leaves
//            fp16's range then: a group's products are held relative to the largest of that group, however large
//            or small the other groups' values are (with one reference for all groups, those of 2^-32 of the
//            largest vanished). The rounding of P is the only one below fp32: off by at most 2^-11 of a product,
//            a quarter of the bf16 output's own step, or, below fp16's normal numbers, by 2^-32 of the
//            group's largest product. (bf16 weights would be off by as much as the output itself.) F_n is held
//            as a bf16 number, as the scale that it multiplies first, exactly. A block whose P all round to zero adds
//            nothing and its values are not multiplied.
//
// mma.sync and not tcgen05.mma: the operands are made in registers, where tcgen05 would have to be
// fed through shared or tensor memory, and at 8 columns the tensor pipe is 20% busy.
//
// What has to move: 1.125 d bytes per key and KV head, once. 64 x 40 heads of 8192 tokens, d = 128
// (3.0 GB): 408 to 413 us, 7.3 to 7.4 TB/s, 109 to 111% of the measured copy (which also writes); 565 instructions of a warp per block of 32
// tokens at 1 x 40 x 8192, start and merge included. With fewer CTAs than
// SMs' room a warp's own chain bounds a block (about 1300 cycles where the values are skipped and 1900 with them,
// at 2 warps per scheduler: 1 x 8 (x 4) x 8192 and 32768 tokens with a CTA each 30 and 88 us, 1 x 40 x 8192 without bias 34),
// and about 6 us of first loads, merge and an uneven last round of stages come on
// top: 1 x 40 x 8192, 47 MB, 13.2 us. 16 warps per SM are what 128 registers allow (of d = 128 the kernels of clusters and
// shares keep 4 to 32 bytes of a thread in local memory, that of whole chunks none); the ring of 3 stages
// per warp keeps 147 KB in flight.
//
// The work is dealt in one of four ways (deal_of), by lengths that only the device knows:
//   whole    a CTA takes one chunk: short sequences, and many chunks;
//   clusters a chunk's stages are dealt to the CTAs of a cluster, which merge through each other's shared memory;
//   slices   each of few chunks has several of the 2 x 152 resident CTAs, in proportion to its length, which take
//            its stages in turn;
//   shares   the chunks of all sequences, one after another, form one row of stages, of which each resident
//            CTA takes an equal share, whose ends may lie inside chunks.
// A chunk that slices or shares worked on leaves a partial from each, and a second kernel merges them in
// fp32. Each kernel begins while the one before it ends (16 x 8 (x 4) x 4097 tokens: 20.5 -> 18.0 us per call).

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <mutex>
#include <type_traits>

#include "alibi.h"
#include "kv4_deal.h"
#include "ptx.cuh"

namespace alibi {
namespace {

using namespace kv4;

constexpr int kStages = 3;          // ring depth of each warp
constexpr int kStageBytes = 4608;   // 128 / D blocks of 36 D bytes
constexpr int kRows = 8;            // query rows of a chunk, at most (the columns of an mma)
constexpr int kMergeThreads = 256;
constexpr int kSmem = kWarps * kStages * kStageBytes;
constexpr uint32_t kMostF = 253;    // exponent field of a value factor F_n, at most: 1 / F_n is a normal number too

struct HeadSlopes {
    float log2e[kMaxQueryHeads];
};

// What a share leaves behind for the merge: the partial of a chunk that began in an earlier share (0) and of one that
// goes on in a later one (1), each of kRows rows of D means and then (R, l) of each row.
KV4_HD constexpr int part_floats(int D) { return kRows * (D + 2); }

struct alignas(8) Header {  // of a chunk
    int first, last;  // the shares it begins and ends in, or -1 where one share did all of it
};

struct DecodeKv4Params {
    const __nv_bfloat16 *q;  // [B, H, T, d]: the G T rows of a KV head are consecutive
    const uint8_t *cache;    // [B, H_kv, C / 32, block]
    const int *lens;         // [B] or null
    __nv_bfloat16 *out;      // [B, H, T, d]
    float *lse;              // [B, H, T] or null
    float *part;             // [CTAs][2][part_floats], null: CTA i takes chunk i
    Header *head;            // [chunks of all sequences]
    uint32_t *status;
    int B, Hkv, G, T, L, blocks, d;  // G: H / H_kv, blocks: C / 32
    int rows, chunks;             // G T, ceil(G T / 8)
    kv4::Divisor by_chunks, by_U, by_T, by_count;  // U: chunks of a sequence
    bool slices;                  // Shares: every chunk has CTAs of its own; otherwise equal shares
    int count;                    // Cluster: CTAs of a cluster
    float c1;                     // log2(e) / sqrt(d)
    HeadSlopes slopes;
};

struct MergeParams {
    const float *part;
    const Header *head;
    __nv_bfloat16 *out;
    float *lse;
    int d, rows, chunks;
};

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// Floats at shared-memory address `a` of CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t map_cluster(uint32_t a, int rank)
{
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
    return r;
}
__device__ __forceinline__ float2 ld_cluster2(uint32_t a, int rank)
{
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(map_cluster(a, rank)) : "memory");
    return v;
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t a, int rank)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(map_cluster(a, rank))
                 : "memory");
    return v;
}

// Transpose of an 8 x 8 matrix of halves spread over the warp (lane 4 i + c: row i, columns 2c, 2c + 1).
__device__ __forceinline__ uint32_t transpose8(uint32_t a)
{
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi)
{
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// Product of the low halves of two bf16 pairs, or of the high ones, in fp32: exact, and in one operation of the fma pipe. (A
// product of pairs in bf16 and taking it apart takes half an operation there and one of the logic pipe, which has less
// room: 24 x 7 x 14336 tokens of d = 32 28.3 -> 27.1 us, 8 x 8 (x 8) x 32768 55.1 -> 52.7.)
template <int HALF>
__device__ __forceinline__ float bf16_product(uint32_t a, uint32_t b)
{
    float d;
    if constexpr (HALF == 0)
        asm("{\n\t.reg .b16 a0, a1, b0, b1;\n\t"
            "mov.b32 {a0, a1}, %1;\n\t"
            "mov.b32 {b0, b1}, %2;\n\t"
            "fma.rn.f32.bf16 %0, a0, b0, %3;\n\t}"
            : "=f"(d) : "r"(a), "r"(b), "f"(0.0f));
    else
        asm("{\n\t.reg .b16 a0, a1, b0, b1;\n\t"
            "mov.b32 {a0, a1}, %1;\n\t"
            "mov.b32 {b0, b1}, %2;\n\t"
            "fma.rn.f32.bf16 %0, a1, b1, %3;\n\t}"
            : "=f"(d) : "r"(a), "r"(b), "f"(0.0f));
    return d;
}

// The largest of |a|, |b| and |c|, NaN if one is.
__device__ __forceinline__ float max_abs3(float a, float b, float c)
{
    float d;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// 2^n for n <= 127, 0 below the normal numbers.
__device__ __forceinline__ float pow2(int n) { return n < -126 ? 0.0f : __uint_as_float(static_cast<uint32_t>(n + 127) << 23); }

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// N words (1, 2 or 4) of shared memory in one load
template <int N>
__device__ __forceinline__ void lds(uint32_t (&w)[N], const uint8_t *p)
{
    if constexpr (N == 4) {
        const uint4 x = *reinterpret_cast<const uint4 *>(p);
        w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
    } else if constexpr (N == 2) {
        const uint2 x = *reinterpret_cast<const uint2 *>(p);
        w[0] = x.x, w[1] = x.y;
    } else {
        w[0] = *reinterpret_cast<const uint32_t *>(p);
    }
}

__device__ __forceinline__ uint32_t hsub2(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c)
{
    uint32_t d;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}

// (w & mask) | k1024 as the one operation it is
__device__ __forceinline__ uint32_t under1024(uint32_t w, uint32_t mask)
{
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(w), "r"(mask), "r"(0x64006400u));
    return d;
}

// The codes of a word as four fp16 pairs: r[i] = (u_i - 8, u_{i+4} - 8). Bits under the exponent of 1024, or of 1024 over
// their place, as a number whose offset one operation takes off: the conversion published by Kim, Henry, Fahim and Hassan
// Awadalla, "Who Says Elephants Can't Run: Bringing Large Scale MoE Models into Cloud Scale Production" (2022). The order
// of the codes in a word is this cache's own (kv4.h).
__device__ __forceinline__ void unpack(uint32_t w, uint32_t (&r)[4])
{
    constexpr uint32_t k1032 = 0x64086408u, kSixteenth = 0x2c002c00u, kMinus72 = 0xd480d480u;
    const uint32_t t = w >> 8;
    r[0] = hsub2(under1024(w, 0x000f000fu), k1032);
    r[1] = hfma2(under1024(w, 0x00f000f0u), kSixteenth, kMinus72);
    r[2] = hsub2(under1024(t, 0x000f000fu), k1032);
    r[3] = hfma2(under1024(t, 0x00f000f0u), kSixteenth, kMinus72);
}

// State of one warp. KC = 2: the chunk's 8 rows are the mma's 8 columns, and a lane has rows 2c and 2c + 1. KC = 1: up to
// 4 rows, each in an even column, so that a lane has row c alone and does half the work per score.
template <int D, int KC>
struct State {
    static constexpr int NG = D / 32;
    uint32_t q[NG][4];      // B operands: column lane / 4, elements 32 n + 8 c + (i, i + 4)
    uint32_t unq[KC][NG > 1 ? NG / 2 : 1];  // bf16 pairs 2^e_n, as the key scales lie (D = 32: in the low half)
    float kappa[KC];        // from their sum to base-2 logits
    float slope[KC];        // m log2(e)
    float pos[KC];          // position less lane / 4
    float R[KC], l[KC];
    uint32_t F[KC][NG > 1 ? NG / 2 : 1];  // bf16 pairs, as the value scales lie (D = 32: in the high half)
    float acc[NG][2][4];    // elements 32 n + 4 g + (0, 2) in [0], + (1, 3) in [1]; columns 2c, 2c + 1
};

// One block of 32 tokens from j0: two tiles whose chains of products, exponentials and products overlap. MASK: some
// query does not see all of them.
template <int D, int KC, bool MASK>
__device__ __forceinline__ void block32(State<D, KC> &st, const uint8_t *blk, int j0, int lane)
{
    constexpr int NG = D / 32;
    const int g = lane >> 2, c = lane & 3;

    // logits: x[i][k] of token g + 8 i and row 2c + k; sv: the words of the tokens' value scales
    float x[4][KC];
    uint32_t sv[4][NG];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        uint32_t kw[2][NG];
        const uint8_t *kp = blk + (t * 16 + g) * (D / 2) + c * (D / 8);
        const uint8_t *sp = blk + 32 * D + (t * 16 + g) * (D / 8);
        lds<NG>(kw[0], kp);
        lds<NG>(kw[1], kp + 4 * D);
        lds<NG>(sv[2 * t], sp);
        lds<NG>(sv[2 * t + 1], sp + D);
#pragma unroll
        for (int n = 0; n < NG; ++n) {
            uint32_t k0[4], k1[4];
            unpack(kw[0][n], k0);
            unpack(kw[1][n], k1);
            float s[4] = {0.f, 0.f, 0.f, 0.f};
            mma16816(s, k0[0], k1[0], k0[1], k1[1], st.q[n][0], st.q[n][1]);
            mma16816(s, k0[2], k1[2], k0[3], k1[3], st.q[n][2], st.q[n][3]);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int k = 0; k < KC; ++k) {
                    const uint32_t w = sv[2 * t + h][n / 2];
                    const float sk = (n & 1) ? bf16_product<1>(w, st.unq[k][n / 2]) : bf16_product<0>(w, st.unq[k][n / 2]);
                    x[2 * t + h][k] = n == 0 ? sk * s[2 * h + k] : fmaf(sk, s[2 * h + k], x[2 * t + h][k]);
                }
            }
        }
    }
    // token less position, in whole numbers below 2^24: exact
    const auto behind = [&](int i, int k) { return static_cast<float>(j0 + 8 * i) - st.pos[k]; };  // pos is less g
    const auto seen = [&](int i, int k) { return !MASK || behind(i, k) <= 0.0f; };
#pragma unroll
    for (int k = 0; k < KC; ++k) {
        // Where all tokens are seen, from the nearest one on, so that no bias is off by more than two roundings of its own
        // size; else each by itself, so that the nearest one's is exact wherever it stands.
        const float nearest = st.slope[k] * behind(3, k);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if constexpr (MASK)
                x[i][k] = seen(i, k) ? fmaf(st.kappa[k], x[i][k], st.slope[k] * behind(i, k)) : -INFINITY;
            else
                x[i][k] = fmaf(st.kappa[k], x[i][k], i == 3 ? nearest : fmaf(8.0f * (i - 3), st.slope[k], nearest));
    }

    // scale of group n of token i: the word it lies in, and itself from that word (or the word's multiple)
    const auto scales = [&](int i, int n) { return sv[i][NG == 1 ? 0 : NG / 2 + n / 2]; };
    const auto scale = [](uint32_t word, int n) { return NG == 1 || (n & 1) ? bf16_hi(word) : bf16_lo(word); };
    const auto scaleF = [&](int i, int n, int k) {
        const uint32_t w = scales(i, n), F = st.F[k][n / 2];
        return NG == 1 || (n & 1) ? bf16_product<1>(w, F) : bf16_product<0>(w, F);
    };
    // p_j and P_jn; of a token that the row does not see zero, whatever its scale. Two rows' P are packed at once, which
    // holds them in half the registers.
    using Product = std::conditional_t<KC == 1, float, uint32_t>;
    const auto product = [](const float (&f)[KC]) -> Product {
        if constexpr (KC == 1)
            return f[0];
        else
            return pack_f16x2(f[0], f[1]);
    };
    float sum[KC] = {}, top = -INFINITY, most = 0.0f;
    Product pr[4][NG];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float p[KC];
#pragma unroll
        for (int k = 0; k < KC; ++k) {
            const float a = x[i][k] - st.R[k];
            top = fmaxf(top, a);
            p[k] = ex2_approx(a);
            sum[k] += p[k];
        }
#pragma unroll
        for (int n = 0; n < NG; ++n) {
            float f[KC];
#pragma unroll
            for (int k = 0; k < KC; ++k) f[k] = seen(i, k) ? p[k] * scaleF(i, n, k) : 0.0f;
            most = max_abs3(most, f[0], f[KC - 1]);
            pr[i][n] = product(f);
        }
    }
    // Every P_jn of the block rounds to zero, and no scale is NaN: nothing to add. With ALiBi most of a long sequence
    // ends here.
    if (!__any_sync(0xffffffffu, top > 8.0f || !(most <= 0x1p-25f))) {
#pragma unroll
        for (int k = 0; k < KC; ++k) st.l[k] += sum[k];
        return;
    }
    // References are moved where a P_jn leaves fp16's range; also where F_n times a scale overflows although the product
    // would not, and where a scale is NaN. With R at the largest x_j or above it p_j <= 1, and p_j s_jn is finite.
    if (__any_sync(0xffffffffu, top > 8.0f || !(most <= 65408.0f))) {
        constexpr int NW = NG > 1 ? NG / 2 : 1;
        float p[4][KC];
#pragma unroll
        for (int k = 0; k < KC; ++k) {
            float mx = -INFINITY;
#pragma unroll
            for (int i = 0; i < 4; ++i) mx = fmaxf(mx, x[i][k]);
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
            // the sum may round below mx, from 2^24 on
            const float was = st.R[k], r = fmaxf(was == -FLT_MAX ? was : was + ceilf(fmaxf(mx - was, 0.0f)), mx);
            const float up = fminf(r - was, 1000.0f);
            st.l[k] *= ex2_approx(-up);
            st.R[k] = r;
#pragma unroll
            for (int i = 0; i < 4; ++i) p[i][k] = ex2_approx(x[i][k] - r);
            sum[k] = (p[0][k] + p[1][k]) + (p[2][k] + p[3][k]);
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                // the largest |p_j s_jn| of each group, NaN left out: its exponent, in the upper bits of its half
                uint32_t tops = 0;
#pragma unroll
                for (int n = 2 * w; n < 2 * w + 2 && n < NG; ++n) {
                    float my = 0.0f;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (seen(i, k)) my = fmaxf(my, fabsf(p[i][k] * scale(scales(i, n), n)));
                    tops |= NG == 1 || (n & 1) ? __float_as_uint(my) & 0xffff0000u : __float_as_uint(my) >> 16;
                }
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) tops = __vmaxu2(tops, __shfl_xor_sync(0xffffffffu, tops, off));
                // the exponent fields of F_n: with R raised they grow by as much, and the sums stay, unless that is too large
                uint32_t F = 0;
#pragma unroll
                for (int n = 2 * w; n < 2 * w + 2 && n < NG; ++n) {
                    const int half = NG == 1 || (n & 1) ? 16 : 0;
                    const int old = static_cast<int>(st.F[k][w] >> (half + 7) & 0xffu);
                    const int e = static_cast<int>(tops >> (half + 7) & 0xffu);  // 2^(e - 127) F_n is 2^7
                    const int f = min(min(old + __float2int_rn(up), 261 - e), static_cast<int>(kMostF));
                    F |= static_cast<uint32_t>(f) << (half + 7);
                    const float down = ex2_approx(static_cast<float>(f - old) - up);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        st.acc[n][i][k] *= down;
                        st.acc[n][i][2 + k] *= down;
                    }
                }
                st.F[k][w] = F;
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int n = 0; n < NG; ++n) {
                float f[KC];
#pragma unroll
                for (int k = 0; k < KC; ++k)
                    f[k] = seen(i, k) ? p[i][k] * scale(scales(i, n), n) * scale(st.F[k][n / 2], n) : 0.0f;
                pr[i][n] = product(f);
            }
    }
#pragma unroll
    for (int k = 0; k < KC; ++k) st.l[k] += sum[k];

#pragma unroll
    for (int t = 0; t < 2; ++t) {
        uint32_t vw[NG][2];
        const uint8_t *vp = blk + 16 * D + t * 8 * D;
        if constexpr (NG == 1) {
            lds<2>(vw[0], vp + lane * 8);
        } else {
#pragma unroll
            for (int n = 0; n < NG; n += 2) {
                uint32_t w[4];
                lds<4>(w, vp + n * 256 + lane * 16);
                vw[n][0] = w[0], vw[n][1] = w[1], vw[n + 1][0] = w[2], vw[n + 1][1] = w[3];
            }
        }
#pragma unroll
        for (int n = 0; n < NG; ++n) {
            uint32_t pb[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if constexpr (KC == 1)
                    pb[h] = transpose8(pack_f16x2(pr[2 * t + h][n], 0.0f));
                else
                    pb[h] = transpose8(pr[2 * t + h][n]);
            }
            uint32_t v0[4], v1[4];
            unpack(vw[n][0], v0);
            unpack(vw[n][1], v1);
            mma16816(st.acc[n][0], v0[0], v0[2], v1[0], v1[2], pb[0], pb[1]);
            mma16816(st.acc[n][1], v0[1], v0[3], v1[1], v1[3], pb[0], pb[1]);
        }
    }
}

// Merge of n partials of 4 elements of a row: `rl(i)` gives partial i's R and l, `mean(i)` its mean. The weights
// l 2^(R - max R) are normalised before they meet the means, so nothing overflows. All of up to N partials are
// asked for before the first is used: those of a cluster's CTAs, one by one, took 3.5 us.
struct Merged {
    float R, l;
    float4 o;
};

template <int N, class RL, class Mean>
__device__ __forceinline__ Merged merge(int n, RL rl, Mean mean)
{
    Merged m = {-FLT_MAX, 0.0f, make_float4(0.f, 0.f, 0.f, 0.f)};
    float2 x[N];
    float4 v[N];
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = i < n ? rl(i) : make_float2(-FLT_MAX, 0.0f);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = i < n ? mean(i) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < N; ++i) m.R = fmaxf(m.R, x[i].x);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        x[i].y *= ex2_approx(x[i].x - m.R);
        m.l += x[i].y;
    }
    const float inv = m.l == 0.0f ? 0.0f : 1.0f / m.l;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float a = x[i].y * inv;
        m.o.x = fmaf(v[i].x, a, m.o.x), m.o.y = fmaf(v[i].y, a, m.o.y);
        m.o.z = fmaf(v[i].z, a, m.o.z), m.o.w = fmaf(v[i].w, a, m.o.w);
    }
    return m;
}

// One row's result: 4 elements of out, and lse by the thread of element 0.
__device__ __forceinline__ void finish(__nv_bfloat16 *out, float *lse, int d, size_t row, int e, const Merged &m, bool bad)
{
    const float nan = __uint_as_float(0x7fc00000u);
    if (e < d) {
        uint2 w;
        w.x = bad ? 0x7fc07fc0u : pack_bf16x2(m.o.x, m.o.y);
        w.y = bad ? 0x7fc07fc0u : pack_bf16x2(m.o.z, m.o.w);
        *reinterpret_cast<uint2 *>(out + row * d + e) = w;
    }
    if (e == 0 && lse) lse[row] = bad ? nan : m.l == 0.0f ? -INFINITY : (m.R + log2f(m.l)) * 0.6931471805599453f;
}

// Length of sequence b; one outside [0, L] counts as 0. Not by the read-only path: this kernel's life begins while the one
// that writes the lengths may still run.
__device__ __forceinline__ int length_of(const DecodeKv4Params &p, int b, bool &bad)
{
    const int n = p.lens ? p.lens[b] : p.L;
    bad = n < 0 || n > p.L;
    return bad ? 0 : n;
}

template <int SB>
__device__ __forceinline__ int stages_of(int len)  // at least one, so that every chunk has a place in the row of stages
{
    return max(1, (len + SB * kv4::kBlock - 1) / (SB * kv4::kBlock));
}

// Share or slice `i`, into `sh`; returns the row. All threads of the CTA.
template <int SB>
__device__ __forceinline__ long long share_of(const DecodeKv4Params &p, int i, Share &sh)
{
    const int U = p.Hkv * p.chunks, ctas = gridDim.x;
    const int units = p.slices ? p.B * U : 0;  // of shares there may be fewer than chunks, which `Slices` cannot take
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    bool bad;
    if (p.B <= 32) {  // one sequence per lane, in every warp
        const int n = lane < p.B ? stages_of<SB>(length_of(p, lane, bad)) : 0;
        int upto = n;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, upto, off);
            if (lane >= off) upto += v;
        }
        const long long row = static_cast<long long>(__shfl_sync(0xffffffffu, upto, 31)) * U;
        if (warp == 0) {
            const Cut cut(row, ctas);
            const Slices sl(row, units, static_cast<int>(__reduce_min_sync(0xffffffffu, n ? n : 0x7fffffff)), ctas);
            const long long weight = static_cast<long long>(upto) * U + static_cast<long long>(lane + 1) * U * sl.extra;
            const long long at = p.slices ? sl.last(i) : i < cut.n ? cut.begin(i) : 0;
            const int b = __popc(__ballot_sync(0xffffffffu, lane < p.B && (p.slices ? weight : static_cast<long long>(upto) * U) <= at));
            const int nb = __shfl_sync(0xffffffffu, n, b), before = __shfl_sync(0xffffffffu, upto, b) - nb;
            if (lane == 0) {
                sh.b = b;
                if (p.slices) {
                    const int step = nb + sl.extra;
                    const long long w0 = (before + static_cast<long long>(b) * sl.extra) * U;
                    sh.unit = min(U - 1, divide(at - w0, step));
                    sl.place(i, w0 + static_cast<long long>(sh.unit) * step, nb, sh);
                } else {
                    const long long rem = at - static_cast<long long>(before) * U;
                    sh.left = i < cut.n ? static_cast<int>(cut.begin(i + 1) - at) : 0;
                    sh.unit = divide(rem, nb);
                    sh.at = static_cast<int>(rem - static_cast<long long>(sh.unit) * nb);
                }
            }
        }
        __syncthreads();
        return row;
    }
    // sum of the sequences' stages, a run of sequences per thread; then the run that holds the beginning
    __shared__ long long warp_sum[kWarps];
    __shared__ int warp_min[kWarps];
    const int run = (p.B + kWarps * 32 - 1) / (kWarps * 32), b0 = min(p.B, static_cast<int>(threadIdx.x) * run), b1 = min(p.B, b0 + run);
    long long mine = 0;
    int least = 0x7fffffff;
    for (int b = b0; b < b1; ++b) {
        const int n = stages_of<SB>(length_of(p, b, bad));
        mine += n;
        least = min(least, n);
    }
    long long upto = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, upto, off);
        if (lane >= off) upto += v;
    }
    least = __reduce_min_sync(0xffffffffu, least);
    if (lane == 31) warp_sum[warp] = upto, warp_min[warp] = least;
    __syncthreads();
    long long before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += warp_sum[w];
        all += warp_sum[w];
        least = min(least, warp_min[w]);
    }
    before += upto - mine;
    const Cut cut(all * U, ctas);
    if (p.slices || i < cut.n) {
        const Slices sl(all * U, units, least, ctas);
        const int extra = p.slices ? sl.extra : 0;
        const long long at = p.slices ? sl.last(i) : cut.begin(i);
        long long w0 = (before + static_cast<long long>(b0) * extra) * U;
        if (at >= w0 && at < w0 + (mine + static_cast<long long>(b1 - b0) * extra) * U) {
            for (int b = b0; b < b1; ++b) {
                const int n = stages_of<SB>(length_of(p, b, bad)), step = n + extra;
                if (at < w0 + static_cast<long long>(step) * U) {
                    sh.b = b;
                    sh.unit = divide(at - w0, step);
                    w0 += static_cast<long long>(sh.unit) * step;
                    if (p.slices) {
                        sl.place(i, w0, n, sh);
                    } else {
                        sh.left = static_cast<int>(cut.begin(i + 1) - at);
                        sh.at = static_cast<int>(at - w0);
                    }
                    break;
                }
                w0 += static_cast<long long>(step) * U;
            }
        }
    } else if (threadIdx.x == 0) {
        sh.left = 0;
    }
    __syncthreads();
    return all * U;
}

// What a CTA takes: a chunk, a slice of a cluster's chunk, or share (or slice) i of the row of all stages.
enum class Mode { Chunk, Cluster, Shares };

template <int D, int KC, Mode MODE>
__global__ void __launch_bounds__(kWarps * 32, 2) decode_kv4_kernel(const __grid_constant__ DecodeKv4Params p)
{
    constexpr int NG = D / 32, SB = 128 / D, kBlk = 36 * D;
    constexpr bool SHARES = MODE == Mode::Shares, CLUSTER = MODE == Mode::Cluster;
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ __align__(8) uint64_t full[kWarps][kStages];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const int U = p.Hkv * p.chunks;

    if (MODE == Mode::Shares) griddep_launch_dependents();  // the merge kernel
    if (threadIdx.x == 0) {
        cta_err_init(kWaitLimitNs);
        cta_check_init(p.status, ring, kSmem);
    }
    if (lane == 0) {
        for (int i = 0; i < kStages; ++i) mbar_init(&full[warp][i], 1);
        fence_mbar_init();
    }
    __syncthreads();
    griddep_wait();  // the kernel before, which may have written what this one reads, is done

    // what is left of the share: kept in shared memory, out of the registers of the loop over blocks
    __shared__ Share sh;
    __shared__ long long row;
    // The second half of the CTAs, which join the first on their SMs, take the shares from the end: with them an SM has heads
    // from both ends of the row, steep slopes, whose far values are skipped, with flat ones.
    const int half = gridDim.x / 2;
    const int share = static_cast<int>(blockIdx.x) < half ? blockIdx.x : gridDim.x - 1 - (blockIdx.x - half);
    if constexpr (SHARES) {
        const long long all = share_of<SB>(p, share, sh);
        if (threadIdx.x == 0) row = all;
        if (sh.left <= 0) return;
    }

    uint8_t *mine = ring + warp * (kStages * kStageBytes);
    int slot = 0;
    uint32_t phase = 0;

    while (true) {
        const int all = CLUSTER ? p.by_count.of(blockIdx.x) : blockIdx.x;  // chunk of all sequences
        const int b = SHARES ? sh.b : p.by_U.of(all), unit = SHARES ? sh.unit : all - b * U;
        const int at = SHARES ? sh.at : CLUSTER ? blockIdx.x - all * p.count : 0;
        const int hk = p.by_chunks.of(unit), chunk = unit - hk * p.chunks;
        const size_t bk = static_cast<size_t>(b) * p.Hkv + hk;
        const int row0 = chunk * kRows, nrows = min(kRows, p.rows - row0);
        // This lane's slice of the row in column g: the 8 elements from 8 c of every group. Asked for before the first copies
        // of the cache, in whose queue it would stand otherwise (1 x 40 heads x 8192 tokens: the loop began 5.0 us after the
        // CTA, now 1.5).
        uint32_t qw[NG][4];
        {
            const int qr = KC == 2 ? g : g >> 1;
            const bool in = qr < nrows && (KC == 2 || (g & 1) == 0);
            const __nv_bfloat16 *qp = p.q + (bk * p.rows + row0 + (in ? qr : 0)) * p.d;
#pragma unroll
            for (int i = 0; i < NG; ++i) {
                uint4 w = make_uint4(0, 0, 0, 0);
                if (in && 32 * i + 8 * c < p.d) w = *reinterpret_cast<const uint4 *>(qp + 32 * i + 8 * c);
                qw[i][0] = w.x, qw[i][1] = w.y, qw[i][2] = w.z, qw[i][3] = w.w;
            }
        }
        bool bad;
        const int len = length_of(p, b, bad), n = stages_of<SB>(len);
        const int nblk = (len + kv4::kBlock - 1) / kv4::kBlock;
        const bool slices = CLUSTER || (SHARES && p.slices);
        const int count = CLUSTER ? p.count : slices ? sh.count : 1;  // slices of the chunk
        const int take = SHARES && !slices ? min(sh.left, n - at) : n;
        // This CTA's stages [s0, s1) of the chunk (slices: every count-th of all), dealt to its warps in turn from the
        // newest to the oldest: the bias falls on the way, so the references R and F_n settle in the first
        // tiles. (Oldest first, a steep head raises them at every tile.)
        const int s0 = slices ? 0 : at, s1 = min(s0 + take, (nblk + SB - 1) / SB);
        const int step = kWarps * count;
        const uint8_t *src = p.cache + bk * p.blocks * kBlk;
        if (bad && unit == 0 && threadIdx.x == 0) atomicOr(p.status, ALIBI_DEV_RANGE);

        auto fetch = [&](int s, int slot_) {
            const uint32_t bytes = static_cast<uint32_t>(min(SB, nblk - s * SB)) * kBlk;
            mbar_arrive_expect_tx(&full[warp][slot_], bytes);
            bulk_load(mine + slot_ * kStageBytes, src + static_cast<size_t>(s) * kStageBytes, bytes, &full[warp][slot_]);
        };
        int s = s1 - 1 - (slices ? at + warp * count : warp);  // this warp's stages: s, s - step, ...
        if (lane == 0)
            for (int i = 0, k = slot; i < kStages; ++i) {
                if (s - i * step >= s0) fetch(s - i * step, k);
                if (++k == kStages) k = 0;
            }

        State<D, KC> st;
        {
            uint32_t ex[NG], most = 14u;  // exponents of the groups' largest elements, and of the row's
#pragma unroll
            for (int i = 0; i < NG; ++i) {
                uint32_t top = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) top = __vmaxu2(top, qw[i][j] & 0x7fff7fffu);
                top = max(top & 0xffffu, top >> 16);
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                ex[i] = top >> 7;
                most = max(most, ex[i]);
            }
            const uint32_t m = min(most, 244u);  // kappa stays finite
            const float kappa = __uint_as_float((m + 9u) << 23) * p.c1;
            uint32_t unq[NG > 1 ? NG / 2 : 1] = {};
#pragma unroll
            for (int i = 0; i < NG; ++i) {
                // a group of less than 2^-103 of the row's largest element is scaled up less, so that 2^e_n is a normal number
                const uint32_t e = max(ex[i], max(m, 103u + 14u) - 103u);
                const float up = __uint_as_float((268u - e) << 23);  // 2^14 over the largest element's power of two
                unq[i / 2] |= (104u + e - m) << (i & 1 ? 23 : 7);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    st.q[i][j] = (j & 1) ? pack_f16x2(bf16_hi(qw[i][j / 2]) * up, bf16_hi(qw[i][2 + j / 2]) * up)
                                         : pack_f16x2(bf16_lo(qw[i][j / 2]) * up, bf16_lo(qw[i][2 + j / 2]) * up);
                    st.acc[i][0][j] = st.acc[i][1][j] = 0.0f;
                }
            }
#pragma unroll
            for (int k = 0; k < KC; ++k) {
                const int r = min(row0 + KC * c + k, p.rows - 1);
                st.kappa[k] = __shfl_sync(0xffffffffu, kappa, (2 * c + k) * 4);
#pragma unroll
                for (int i = 0; i < (NG > 1 ? NG / 2 : 1); ++i) st.unq[k][i] = __shfl_sync(0xffffffffu, unq[i], (2 * c + k) * 4);
                const int h = p.by_T.of(r);
                st.slope[k] = p.slopes.log2e[hk * p.G + h];
                st.pos[k] = static_cast<float>(len - p.T + r - h * p.T - g);
                st.R[k] = -FLT_MAX;
                st.l[k] = 0.0f;
#pragma unroll
                for (int i = 0; i < (NG > 1 ? NG / 2 : 1); ++i) st.F[k][i] = kMostF << 23 | kMostF << 7;
            }
        }

        for (; s >= s0; s -= step) {
            const bool ok = mbar_wait(&full[warp][slot], phase, p.status, 0x60);
            if (!__all_sync(0xffffffffu, ok)) break;
            const uint8_t *stage = mine + slot * kStageBytes;
            // Of one row per lane and d = 128 the masked form takes every block: a second copy of the loop's body costs more
            // there than the masks (64 x 40 x 8192 tokens 419 us with two copies, 412 with one; d = 32 28.0 and 29.2 at
            // 24 x 7 x 14336, two rows per lane 53.1 and 55.5 at 8 x 8 (x 8) x 32768; d = 64 57.4 and 57.6 at 8 x 38 x 16384).
            constexpr bool kOneForm = KC == 1 && D == 128;
#pragma unroll 1
            for (int t = SB - 1; t >= 0; --t) {
                const int j0 = (s * SB + t) * kv4::kBlock;
                if (j0 >= len) continue;
                if (kOneForm || j0 + kv4::kBlock > len - p.T + 1)
                    block32<D, KC, true>(st, stage + t * kBlk, j0, lane);
                else
                    block32<D, KC, false>(st, stage + t * kBlk, j0, lane);
            }
            __syncwarp();
            if (lane == 0 && s - kStages * step >= s0) fetch(s - kStages * step, slot);
            if (++slot == kStages) slot = 0, phase ^= 1u;
        }
        // a wait ran out (recorded): let the copies in flight land before the ring is reused
        for (int i = 0; i < kStages && s >= s0; ++i, s -= step) {
            mbar_wait(&full[warp][slot], phase, p.status, 0x61, true);
            if (++slot == kStages) slot = 0, phase ^= 1u;
        }

        // the warp's partial: reference R, l = sum of p, and the mean of v (never beyond the largest |v|)
        float *pw = reinterpret_cast<float *>(mine);  // [kRows][D + 4], then R and l of each row
        constexpr int kRowStride = D + 4;
#pragma unroll
        for (int k = 0; k < KC; ++k) {
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) st.l[k] += __shfl_xor_sync(0xffffffffu, st.l[k], off);
            const float inv = st.l[k] == 0.0f ? 0.0f : 1.0f / st.l[k];
            const int r = KC * c + k;
#pragma unroll
            for (int i = 0; i < NG; ++i) {
                // 1 / F_n, after the division by l: a mean is in range, the sum may not be
                const uint32_t F = st.F[k][i / 2] >> (NG == 1 || (i & 1) ? 23 : 7) & 0xffu;
                const float up = pow2(127 - static_cast<int>(F));
                const float4 o = make_float4(st.acc[i][0][k] * inv * up, st.acc[i][1][k] * inv * up,
                                             st.acc[i][0][2 + k] * inv * up, st.acc[i][1][2 + k] * inv * up);
                *reinterpret_cast<float4 *>(pw + r * kRowStride + 32 * i + 4 * g) = o;
            }
            if (g == 0)
                *reinterpret_cast<float2 *>(pw + kRows * kRowStride + 2 * r) = make_float2(st.R[k], st.l[k]);
        }
        __syncthreads();

        bool whole = true;
        float *to = nullptr;
        if constexpr (CLUSTER) {
            // into the second stage of the first warp's ring, which no partial lies in
            static_assert(part_floats(D) * sizeof(float) <= kStageBytes && kRows * (kRowStride + 2) * sizeof(float) <= kStageBytes,
                          "a warp's partial and the CTA's take a stage each");
            whole = false;
            to = reinterpret_cast<float *>(ring + kStageBytes);
        } else if constexpr (SHARES) {
            whole = p.slices ? sh.count == 1 : take == n;
            to = p.part + (static_cast<size_t>(share) * 2 + (sh.at == 0)) * part_floats(D);
        }
        for (int i = threadIdx.x; i < nrows * (D / 4); i += kWarps * 32) {
            const int r = i / (D / 4), e = i % (D / 4) * 4;
            const float *base = reinterpret_cast<const float *>(ring);
            constexpr int kStep = kStages * kStageBytes / 4;
            const Merged m = merge<kWarps>(
                kWarps,
                [&](int w) { return *reinterpret_cast<const float2 *>(base + w * kStep + kRows * kRowStride + 2 * r); },
                [&](int w) { return *reinterpret_cast<const float4 *>(base + w * kStep + r * kRowStride + e); });
            if (whole) {
                finish(p.out, p.lse, p.d, bk * p.rows + row0 + r, e, m, bad);
            } else {
                *reinterpret_cast<float4 *>(to + r * D + e) = m.o;
                if (e == 0) *reinterpret_cast<float2 *>(to + kRows * D + 2 * r) = make_float2(m.R, m.l);
            }
        }
        if constexpr (CLUSTER) {
            cluster_arrive();
            cluster_wait();
            // This CTA merges `per` of the rows' elements, fewer than it has threads.
            const int items = nrows * (D / 4), per = p.by_count.of(items + count - 1);
            const uint32_t base = smem_u32(to);
            const int i = at * per + threadIdx.x, r = i / (D / 4), e = i % (D / 4) * 4;
            const bool in = i < min(items, (at + 1) * per);
            Merged m;
            if (in) {
                const auto rl = [&](int k) { return ld_cluster2(base + (kRows * D + 2 * r) * 4, k); };
                const auto mean = [&](int k) { return ld_cluster4(base + (r * D + e) * 4, k); };
                m = count <= 8 ? merge<8>(count, rl, mean) : merge<kv4::kMostCluster>(count, rl, mean);
            }
            cluster_arrive();  // the other CTAs may still read this one's partial
            if (in) finish(p.out, p.lse, p.d, bk * p.rows + row0 + r, e, m, bad);
            cluster_wait();
        }
        if constexpr (!SHARES) return;
        if (p.slices) {
            if (threadIdx.x == 0 && sh.at == 0)
                p.head[static_cast<size_t>(sh.b) * U + sh.unit] =
                    sh.count == 1 ? Header{-1, -1} : Header{share, share + sh.count - 1};
            return;
        }
        fence_proxy_async_smem();  // the partials were written and read before the next copies overwrite them
        __syncthreads();
        if (threadIdx.x == 0) {
            sh.left -= take;
            sh.at += take;
            if (sh.at == n) {
                Header h = {-1, -1};
                if (take < n) {  // the share's first chunk, whose first stage lies n - take before the share's beginning
                    const Cut cut(row, gridDim.x);
                    h = {cut.holder(cut.begin(share) + take - n), share};
                }
                p.head[static_cast<size_t>(sh.b) * U + sh.unit] = h;
                sh.at = 0;
                if (++sh.unit == U) sh.unit = 0, ++sh.b;
            }
        }
        __syncthreads();
        if (sh.left <= 0) return;
    }
}

// Merge of the chunks that several shares worked on: CTA (i, r) looks at row r of chunk i. Its partials are slot 1 of the
// share it began in and slot 0 of the shares up to the one it ends in. The loads of a thread are issued
// together: with 76 partials the merge waits for three round trips to L2 and not for 76.
template <int D>
__global__ void __launch_bounds__(kMergeThreads) decode_kv4_merge_kernel(const __grid_constant__ MergeParams p)
{
    constexpr int kPart = part_floats(D), kItems = D / 4, kGroups = kMergeThreads / kItems, kDepth = 8;
    __shared__ float weight[kMostShares];
    __shared__ float red[2][kMergeThreads / 32];
    __shared__ float4 sum[kMergeThreads];
    griddep_wait();
    const int unit = blockIdx.x, r = blockIdx.y;
    const int2 h = __ldcg(reinterpret_cast<const int2 *>(p.head + unit));  // (first, last)
    if (h.x < 0) return;
    const int n = h.y - h.x + 1;
    const int bk = unit / p.chunks, row0 = (unit - bk * p.chunks) * kRows;
    if (row0 + r >= p.rows) return;
    const float *part0 = p.part + (static_cast<size_t>(h.x) * 2 + 1) * kPart;
    const auto from = [&](int k) { return part0 + (k == 0 ? 0 : (2 * k - 1) * kPart); };
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, item = threadIdx.x % kItems, group = threadIdx.x / kItems;
    // the first means are fetched while the weights are computed
    float4 v[kDepth];
#pragma unroll
    for (int i = 0; i < kDepth; ++i) {
        const int k = group + i * kGroups;
        if (k < n) v[i] = __ldcg(reinterpret_cast<const float4 *>(from(k) + r * D + 4 * item));
    }
    // weights l 2^(R - max R)
    float R = -FLT_MAX, l = 0.0f;
    float2 x[kMostShares / kMergeThreads];
#pragma unroll
    for (int i = 0; i < kMostShares / kMergeThreads; ++i) {
        const int k = threadIdx.x + i * kMergeThreads;
        x[i] = k < n ? __ldcg(reinterpret_cast<const float2 *>(from(k) + kRows * D + 2 * r)) : make_float2(-FLT_MAX, 0.0f);
        R = fmaxf(R, x[i].x);
    }
#pragma unroll
    for (int off = 16; off; off >>= 1) R = fmaxf(R, __shfl_xor_sync(0xffffffffu, R, off));
    if (lane == 0) red[0][warp] = R;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kMergeThreads / 32; ++w) R = fmaxf(R, red[0][w]);
#pragma unroll
    for (int i = 0; i < kMostShares / kMergeThreads; ++i) {
        const int k = threadIdx.x + i * kMergeThreads;
        const float w = x[i].y * ex2_approx(x[i].x - R);
        if (k < n) weight[k] = w;
        l += w;
    }
#pragma unroll
    for (int off = 16; off; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
    if (lane == 0) red[1][warp] = l;
    __syncthreads();
    l = 0.0f;
#pragma unroll
    for (int w = 0; w < kMergeThreads / 32; ++w) l += red[1][w];
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    Merged m = {R, l, make_float4(0.f, 0.f, 0.f, 0.f)};
    for (int k0 = group; k0 < n; k0 += kDepth * kGroups) {
#pragma unroll
        for (int i = 0; i < kDepth; ++i) {
            const int k = k0 + i * kGroups;
            if (k < n) {
                const float a = weight[k] * inv;
                m.o.x = fmaf(v[i].x, a, m.o.x), m.o.y = fmaf(v[i].y, a, m.o.y);
                m.o.z = fmaf(v[i].z, a, m.o.z), m.o.w = fmaf(v[i].w, a, m.o.w);
            }
        }
#pragma unroll
        for (int i = 0; i < kDepth; ++i) {
            const int k = k0 + (kDepth + i) * kGroups;
            if (k < n) v[i] = __ldcg(reinterpret_cast<const float4 *>(from(k) + r * D + 4 * item));
        }
    }
    sum[threadIdx.x] = m.o;
    __syncthreads();
    if (group != 0) return;
#pragma unroll
    for (int k = 1; k < kGroups; ++k) {
        const float4 y = sum[k * kItems + item];
        m.o.x += y.x, m.o.y += y.y, m.o.z += y.z, m.o.w += y.w;
    }
    finish(p.out, p.lse, p.d, static_cast<size_t>(bk) * p.rows + row0 + r, 4 * item, m, false);
}

bool aligned(const void *p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// What the current device holds of clusters of 8-warp CTAs with kSmem, asked for once; kAlone bytes are more than half of an
// SM's shared memory.
constexpr int kAlone = 120 << 10;

template <class Kernel>
cudaError_t cluster_fit(Kernel kernel, kv4::ClusterFit *fit)
{
    constexpr int kDevices = 64;  // a device beyond is asked every time
    static std::mutex mu;
    static kv4::ClusterFit known[kDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> g(mu);
    if (dev < kDevices && known[dev].two[0] != 0) {
        *fit = known[dev];
        return cudaSuccess;
    }
    kv4::ClusterFit f = {};
    for (int c = 2; c <= kv4::kMostCluster; ++c)
        for (int smem : {kSmem, kAlone}) {
            cudaLaunchAttribute attr = {};
            attr.id = cudaLaunchAttributeClusterDimension;
            attr.val.clusterDim.x = static_cast<unsigned>(c);
            attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(static_cast<unsigned>(c));
            cfg.blockDim = dim3(kWarps * 32);
            cfg.dynamicSmemBytes = static_cast<size_t>(smem);
            cfg.attrs = &attr;
            cfg.numAttrs = 1;
            e = cudaOccupancyMaxActiveClusters(smem == kSmem ? &f.two[c] : &f.one[c], kernel, &cfg);
            if (e != cudaSuccess) return e;
        }
    f.two[0] = 1;
    if (dev < kDevices) known[dev] = f;
    *fit = f;
    return cudaSuccess;
}

template <int D, int KC>
cudaError_t launch(DecodeKv4Params &p, long long units, cudaStream_t stream)
{
    const auto whole = &decode_kv4_kernel<D, KC, Mode::Chunk>;
    const auto clusters = &decode_kv4_kernel<D, KC, Mode::Cluster>;
    const auto shared = &decode_kv4_kernel<D, KC, Mode::Shares>;
    constexpr int kTokens = 128 / D * kv4::kBlock;  // of a stage
    const int stages = (p.L + kTokens - 1) / kTokens, ctas = std::min(2 * num_sms(), kMostShares);
    cudaError_t e = prepare_kernel(reinterpret_cast<const void *>(clusters), kAlone, 0, true);
    if (e != cudaSuccess) return e;
    kv4::ClusterFit fit;
    e = cluster_fit(clusters, &fit);
    if (e != cudaSuccess) return e;
    const Plan plan = deal_of(units, stages, ctas, fit);
    p.part = nullptr;
    p.head = nullptr;
    p.slices = false;
    p.count = plan.count;
    p.by_count = kv4::Divisor(plan.count);
    if (plan.deal == Deal::Whole || plan.deal == Deal::Clusters) {
        if (units * plan.count > 0x7fffffffLL) return cudaErrorInvalidValue;
        if (plan.count == 1) e = prepare_kernel(reinterpret_cast<const void *>(whole), kSmem, 0);
        if (e != cudaSuccess) return e;
        return launch_kernel(plan.count > 1 ? clusters : whole, dim3(static_cast<unsigned>(units * plan.count)),
                             kWarps * 32, kSmem, stream, p, plan.count);
    }
    e = prepare_kernel(reinterpret_cast<const void *>(shared), kSmem, 0);
    if (e != cudaSuccess) return e;
    const int per = (stages + kWarps - 1) / kWarps;  // CTAs that a chunk can keep busy
    const int shares = static_cast<int>(std::min<long long>(units * per, ctas));
    p.slices = plan.deal == Deal::Slices;
    const size_t bytes = static_cast<size_t>(shares) * 2 * part_floats(D) * sizeof(float);
    char *ws = nullptr;
    e = cudaMallocFromPoolAsync(reinterpret_cast<void **>(&ws), bytes + static_cast<size_t>(units) * sizeof(Header), decode_pool(), stream);
    if (e != cudaSuccess) return e;
    p.part = reinterpret_cast<float *>(ws);
    p.head = reinterpret_cast<Header *>(ws + bytes);
    e = launch_kernel(shared, dim3(static_cast<unsigned>(shares)), kWarps * 32, kSmem, stream, p);
    if (e == cudaSuccess && shares > 1) {
        MergeParams m = {p.part, p.head, p.out, p.lse, p.d, p.rows, p.chunks};
        e = launch_kernel(decode_kv4_merge_kernel<D>, dim3(static_cast<unsigned>(units), std::min(p.rows, kRows)),
                          kMergeThreads, 0, stream, m);
    }
    const cudaError_t f = cudaFreeAsync(ws, stream);
    return e != cudaSuccess ? e : f;
}

}  // namespace
}  // namespace alibi

using namespace alibi;

extern "C" int alibi_attn_decode_kv4(const void *q, const void *cache, const int *lens, void *out, float *lse, int B,
                                     int H, int Hkv, int T, int L, int C, int d, const float *slopes, void *stream)
{
    if (!q || !cache || !out) return ALIBI_ERR_INVALID;
    if (!aligned(q, 16) || !aligned(cache, 16) || !aligned(out, 16) || !aligned(lens, 4) || !aligned(lse, 4))
        return ALIBI_ERR_INVALID;
    if (B < 1 || H < 1 || Hkv < 1 || T < 1 || L < 1 || C < 1 || d < 1) return ALIBI_ERR_INVALID;
    if (H % Hkv != 0 || C % kv4::kBlock != 0 || L > C) return ALIBI_ERR_INVALID;
    if (!decode_supports(d) || H > kMaxQueryHeads || T > 16 || C > (1 << 24)) return ALIBI_ERR_UNSUPPORTED;
    if (static_cast<long long>(B) * H * T > (1LL << 31) - 1) return ALIBI_ERR_UNSUPPORTED;
    if (slopes)
        for (int h = 0; h < H; ++h)
            if (!std::isfinite(slopes[h]) || slopes[h] < 0.0f) return ALIBI_ERR_INVALID;
    DecodeKv4Params p;
    if (slopes)
        for (int h = 0; h < H; ++h) p.slopes.log2e[h] = static_cast<float>(static_cast<double>(slopes[h]) * 1.4426950408889634);
    else
        fill_slopes_log2e(H, p.slopes.log2e);
    p.q = static_cast<const __nv_bfloat16 *>(q);
    p.cache = static_cast<const uint8_t *>(cache);
    p.lens = lens;
    p.out = static_cast<__nv_bfloat16 *>(out);
    p.lse = lse;
    p.status = device_status_word();
    if (!p.status) return ALIBI_ERR_CUDA;
    p.B = B;
    p.Hkv = Hkv;
    p.T = T;
    p.G = H / Hkv;
    p.L = L;
    p.blocks = C / kv4::kBlock;
    p.d = d;
    p.rows = p.G * T;
    p.chunks = (p.rows + kRows - 1) / kRows;
    p.by_chunks = kv4::Divisor(p.chunks);
    p.by_U = kv4::Divisor(Hkv * p.chunks);
    p.by_T = kv4::Divisor(T);
    p.c1 = 1.4426950408889634f / sqrtf(static_cast<float>(d));
    // A slope beyond 1e30 is 1e30: the bias of the next token is out of reach already, and its multiples stay finite.
    for (int h = 0; h < H; ++h) p.slopes.log2e[h] = std::min(p.slopes.log2e[h], 1e30f);
    const long long units = static_cast<long long>(B) * Hkv * p.chunks;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool few = p.rows <= kRows / 2;  // one row per lane
    cudaError_t e;
    switch (kv4::padded(d)) {
        case 128: e = few ? launch<128, 1>(p, units, st) : launch<128, 2>(p, units, st); break;
        case 64: e = few ? launch<64, 1>(p, units, st) : launch<64, 2>(p, units, st); break;
        default: e = few ? launch<32, 1>(p, units, st) : launch<32, 2>(p, units, st); break;
    }
    return e == cudaSuccess ? ALIBI_OK : ALIBI_ERR_CUDA;
}
