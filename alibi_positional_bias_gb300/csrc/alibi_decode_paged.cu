// ALiBi attention of the newest tokens of each sequence over its pages.
//
// Row (h, t) of sequence b is the query of head h at position i = len_b - T + t, with len_b tokens in its pages (the new ones
// included), and h / G its KV head, G = H / H_kv:
//   x_j = q.k_j / sqrt(d) - m_h (i - j),  j <= i,   out = sum_j softmax_j(x) v_j.
//
// The G T rows of a KV head share its keys: a chunk of up to 8, 16 or 32 rows is what a CTA takes over all or a part of the
// sequence. Each warp streams stages of 8 KB (16 tokens' keys and values of d = 128) through a ring of its own in shared memory,
// by TMA: boxes of up to a page's slots of one head, swizzled as ldmatrix reads them, one mbarrier per stage and no
// synchronisation between warps. (cp.async of 16 bytes per lane took 200 instructions per stage, and a warp's step 1350
// cycles.) The slots past a sequence's length are loaded too, whatever they hold, and their values set to zero in shared
// memory. Per tile of 16 tokens:
//
//   scores   S^T = K Q^T, mma.m16n8k16 in bf16 with fp32 sums: exact products. The tokens are the 16 rows, so that 8 query
//            rows fill the 8 columns.
//   softmax  in base 2: p_j = 2^(x_j - R), summed in fp32, with a reference R of each row that is raised when some x_j exceeds
//            it by 8. A weight below 2^-126 of the row's largest counts as zero.
//   values   O^T += V^T P^T, with p as the sum of two bf16 numbers, off by at most 2^-16 of itself: the tensor pipe has
//            room for the second product (one mma per 2 cycles and SM were measured, 600 TFLOP/s), and the output has no
//            rounding but its own that counts.
//
// mma.sync and not tcgen05.mma: of 8 rows a tile of 128 would be empty but for 1/16.
//
// Measured, launches in one graph over caches that together are larger than L2: 64 x 40 heads x 8192 tokens of d = 128 (10.7 GB)
// 1407 to 1448 us, 7.4 to 7.6 TB/s, bound by HBM; 1 x 40 x 8192 29 us (5.8 TB/s), 16 x 8 (x 4) x 2049..4097 39 (5.7), 1 x 4
// (x 4) x 131071 47 (5.7): what a launch, the first loads and the merge take (4 to 8 us) over HBM's time; 8 x 16 (x 2) x 4
// new tokens of 1025..2048, d = 64, 13.5 us: a launch, up to eight stages one after another in each warp of a cluster of two,
// and the cluster's merge; 1 x 6 x 100 2.8 us: a launch. A warp's step (a stage
// of one row group at d = 128) is 1240 to 1350 cycles when L2 has the pages: 700 of copies and waits, 970 of products and
// softmax, partly at the same time; eight warps per SM keep up with HBM at 3000 cycles a step, four at 1500.

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cuda.h>
#include <cuda_bf16.h>
#include <mutex>

#include "alibi.h"
#include "kv4_deal.h"
#include "paged_deal.h"
#include "pages.cuh"
#include "ptx.cuh"
#include "split_merge.cuh"

namespace alibi {
namespace {

constexpr int kPgWarps = paged::kWarps;
constexpr int kPgStages = 3;       // ring depth of each warp
constexpr int kPgStageBytes = 8192;
constexpr int kPgRing = kPgWarps * kPgStages * kPgStageBytes;
constexpr int kMostRows = 32;      // query rows of a chunk

KV4_HD constexpr int pg_tokens(int D) { return 2048 / D; }  // of a stage
KV4_HD constexpr int pg_smem(int D, int NT) { return kPgRing + (NT > 2 ? kMostRows * D * 2 : 0) + 1024; }  // 1024: alignment

struct DecodePagedParams {
    CUtensorMap tk, tv;      // of encode_pages, boxes of min(slots, tokens of a stage) slots
    const __nv_bfloat16 *q;  // [B, H, T, d]: the G T rows of a KV head are consecutive
    Pages pg;
    const int *lens;         // [B] or null
    __nv_bfloat16 *out;      // [B, H, T, d]
    float *lse;              // [B, H, T] or null
    float *part;             // Shares: [CTAs][2][part_floats]
    Header *head;            // Shares: [chunks of all sequences]
    uint32_t *status;
    int B, Hkv, G, T, L;     // G: H / H_kv
    int rows, chunks;        // G T, chunks of a KV head
    Divisor by_chunks, by_U, by_T, by_count;  // U: chunks of a sequence
    int count;               // CTAs of a cluster
    int hold;                // 1: the self-test's, whose warps 0 wait for an arrival that nobody makes
    uint64_t wait_ns;        // limit of every bounded wait
    float c1;                // log2(e) / sqrt(d)
    HeadSlopes slopes;
};

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Byte of the 16-byte piece `piece` of row `row` of a tile of N bf16 rows of D elements, as TMA's swizzle leaves them: the
// eight rows that an ldmatrix reads lie in the eight 16-byte banks. D = 128: the first halves of all rows, then the second.
template <int D, int N>
__device__ __forceinline__ uint32_t place(int row, int piece)
{
    if constexpr (D == 128) return (piece >> 3) * (N * 128) + row * 128 + (((piece ^ row) & 7) << 4);
    const int turn = D >= 64 ? row & 7 : D == 32 ? (row >> 1) & 3 : (row >> 2) & 1;
    return static_cast<uint32_t>(row * (2 * D) + ((piece ^ turn) << 4));
}

// The same for pieces 2 m + i of a lane's row, from place(row, i): the swizzle turns only the lower bits, and m those above i.
template <int D, int N>
__device__ __forceinline__ uint32_t step(uint32_t at, int m)
{
    return D == 128 ? (at ^ ((m & 3) << 5)) + (m >> 2) * (N * 128) : at ^ (m << 5);
}

// State of one warp: NT groups of 8 rows; a lane has rows 8 n + 2 c + k.
template <int D, int NT>
struct Rows8 {
    float acc[D / 16][NT][4];  // elements 16 i + g of rows 2c, 2c + 1, then elements 16 i + g + 8
    float R[NT][2], l[NT][2];
    float slope[NT][2];        // m log2(e)
    float pos[NT][2];          // position less g
    uint32_t q[NT > 2 ? 1 : D / 16][NT][2];  // B operands; of more than 16 rows they stay in shared memory
};

// Values of 16 TT tokens whose rows see them unequally and of which some are infinite or NaN: of every query token the
// products by themselves, without the values that it does not see. The tile's values are overwritten.
template <int D, int NT, int TT>
__device__ __forceinline__ void add_values_apart(Rows8<D, NT> &st, uint32_t v, const uint32_t (&hi)[TT][NT][2],
                                              const uint32_t (&lo)[TT][NT][2], int j0, int last, int T, int lane)
{
    for (int i = last; i > last - T; --i) {  // positions of the query tokens
        for (int x = lane; x < 16 * TT * (D / 8); x += 32)
            if (j0 + x / (D / 8) > i)
                asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(v + place<D, 16 * TT>(x / (D / 8), x % (D / 8))), "r"(0)
                             : "memory");
        __syncwarp();
#pragma unroll
        for (int t = 0; t < TT; ++t)
#pragma unroll
            for (int m = 0; m < D / 16; ++m) {
                uint32_t a[4];
                ldmatrix4_trans(a, v + place<D, 16 * TT>(16 * t + (lane & 7) + (lane >> 4) * 8, 2 * m + ((lane >> 3) & 1)));
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float y[4] = {0.f, 0.f, 0.f, 0.f};
                    mma_bf16(y, a, lo[t][n][0], lo[t][n][1]);
                    mma_bf16(y, a, hi[t][n][0], hi[t][n][1]);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (st.pos[n][e & 1] + static_cast<float>(lane >> 2) == static_cast<float>(i)) st.acc[m][n][e] += y[e];
                }
            }
        __syncwarp();
    }
    fence_proxy_async_smem();  // the zeros before the next copies
    __syncwarp();
}

// 16 TT tokens from j0: keys at shared-memory address k, values at v.
template <int D, int NT, int TT>
__device__ __forceinline__ void tokens16(Rows8<D, NT> &st, uint32_t k, uint32_t v, uint32_t sq, float c1, int j0, int last,
                                         int T, int lane)
{
    constexpr int CH = TT * NT == 1 ? 2 : 1;  // chains of products
    constexpr int kRow = D < 64 ? 2 * D : 128;  // bytes from row to row
    const uint32_t ka = place<D, 16 * TT>(lane & 15, lane >> 4), va = place<D, 16 * TT>((lane & 7) + (lane >> 4) * 8, (lane >> 3) & 1);
    // Operands are read in batches, the products that take them after that: one by one, each would wait for its own read.
    constexpr int kBatch = NT > 2 ? (D < 64 ? D / 16 : 4) : D / 16;
    float s[TT][NT][CH][4] = {};
#pragma unroll
    for (int m0 = 0; m0 < D / 16; m0 += kBatch) {
        uint32_t a[TT][kBatch][4], b[kBatch][NT][2];
#pragma unroll
        for (int m = 0; m < kBatch; ++m) {
#pragma unroll
            for (int t = 0; t < TT; ++t) ldmatrix4(a[t][m], step<D, 16 * TT>(k + ka, m0 + m) + 16 * t * kRow);
            if constexpr (NT > 2) {
#pragma unroll
                for (int n = 0; n < NT; n += 2) {
                    uint32_t w[4];
                    ldmatrix4(w, sq + place<D, kMostRows>(8 * n + (lane & 7) + (lane >> 4) * 8, 2 * (m0 + m) + ((lane >> 3) & 1)));
                    b[m][n][0] = w[0], b[m][n][1] = w[1], b[m][n + 1][0] = w[2], b[m][n + 1][1] = w[3];
                }
            } else {
#pragma unroll
                for (int n = 0; n < NT; ++n) b[m][n][0] = st.q[m0 + m][n][0], b[m][n][1] = st.q[m0 + m][n][1];
            }
        }
#pragma unroll
        for (int m = 0; m < kBatch; ++m)
#pragma unroll
            for (int t = 0; t < TT; ++t)
#pragma unroll
                for (int n = 0; n < NT; ++n) mma_bf16(s[t][n][m % CH], a[t][m], b[m][n][0], b[m][n][1]);
    }
    // logits: element e of s is token 16 t + g + 8 (e / 2), row 2c + e % 2
    float top = -INFINITY;
    const bool masked = j0 + 16 * TT > last - T + 2;  // some row does not see all of them
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float behind0 = static_cast<float>(j0) - st.pos[n][i];  // whole numbers below 2^24: exact
#pragma unroll
            for (int t = 0; t < TT; ++t)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int e = 2 * h + i;
                    const float behind = behind0 + static_cast<float>(16 * t + 8 * h);
                    const float y = CH == 2 ? s[t][n][0][e] + s[t][n][CH - 1][e] : s[t][n][0][e];
                    float x = fmaf(y, c1, st.slope[n][i] * behind);
                    if (masked) x = behind <= 0.0f ? x : -INFINITY;
                    s[t][n][0][e] = x;
                    top = fmaxf(top, x - st.R[n][i]);
                }
        }
    if (__any_sync(0xffffffffu, top > 8.0f)) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float mx = -INFINITY;
#pragma unroll
                for (int t = 0; t < TT; ++t) mx = fmaxf(mx, fmaxf(s[t][n][0][i], s[t][n][0][2 + i]));
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
                const float r = fmaxf(st.R[n][i], mx);
                const float down = ex2_approx(st.R[n][i] - r);
                st.R[n][i] = r;
                st.l[n][i] *= down;
#pragma unroll
                for (int m = 0; m < D / 16; ++m) st.acc[m][n][i] *= down, st.acc[m][n][2 + i] *= down;
            }
    }
    uint32_t hi[TT][NT][2], lo[TT][NT][2];  // B operands of the values' products
#pragma unroll
    for (int t = 0; t < TT; ++t)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float p0 = ex2_approx(s[t][n][0][2 * h] - st.R[n][0]), p1 = ex2_approx(s[t][n][0][2 * h + 1] - st.R[n][1]);
                st.l[n][0] += p0;
                st.l[n][1] += p1;
                // cut, not rounded, and the rest not below 2^-126 where p is not zero: an infinite value times both is
                // infinite and not NaN
                const auto rest = [](float y) {
                    return fmaxf(y - __uint_as_float(__float_as_uint(y) & 0xffff0000u), fminf(y, FLT_MIN));
                };
                hi[t][n][h] = transpose8(__byte_perm(__float_as_uint(p0), __float_as_uint(p1), 0x7632));
                lo[t][n][h] = transpose8(pack_bf16x2(rest(p0), rest(p1)));
            }
    if (T > 1 && masked) {
        bool odd = false;
        for (int x = lane; x < 16 * TT * (D / 8); x += 32) {
            uint32_t w[4];
            asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(v + 16 * x) : "memory");
#pragma unroll
            for (int i = 0; i < 4; ++i) odd |= (w[i] & 0x7f80u) == 0x7f80u || (w[i] & 0x7f800000u) == 0x7f800000u;
        }
        if (__any_sync(0xffffffffu, odd)) return add_values_apart<D, NT, TT>(st, v, hi, lo, j0, last, T, lane);
    }
#pragma unroll
    for (int t = 0; t < TT; ++t)
#pragma unroll
        for (int m0 = 0; m0 < D / 16; m0 += kBatch) {
            uint32_t a[kBatch][4];
#pragma unroll
            for (int m = 0; m < kBatch; ++m)
                ldmatrix4_trans(a[m], step<D, 16 * TT>(v + va, m0 + m) + 16 * t * kRow);
#pragma unroll
            for (int m = 0; m < kBatch; ++m)
#pragma unroll
                for (int n = 0; n < NT; ++n) mma_bf16(st.acc[m0 + m][n], a[m], lo[t][n][0], lo[t][n][1]);
#pragma unroll
            for (int m = 0; m < kBatch; ++m)
#pragma unroll
                for (int n = 0; n < NT; ++n) mma_bf16(st.acc[m0 + m][n], a[m], hi[t][n][0], hi[t][n][1]);
        }
}

// Length of sequence b; one outside [0, L] counts as 0. Not by the read-only path: this kernel's life begins while the one
// that writes the lengths may still run.
__device__ __forceinline__ int length_of(const DecodePagedParams &p, int b, bool &bad)
{
    const int n = p.lens ? p.lens[b] : p.L;
    bad = n < 0 || n > p.L;
    return bad ? 0 : n;
}

template <int TK>
__device__ __forceinline__ int stages_of(int len)  // at least one, so that every chunk has a place in the row of stages
{
    return max(1, (len + TK - 1) / TK);
}

// Where share `i` of the row of all sequences' stages begins, into `sh`; returns the row's length. All threads of the CTA.
template <int TK>
__device__ __forceinline__ long long share_of(const DecodePagedParams &p, int i, kv4::Share &sh)
{
    constexpr int kThreads = kPgWarps * 32;
    __shared__ long long warp_sum[kPgWarps];
    const int U = p.Hkv * p.chunks, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int run = (p.B + kThreads - 1) / kThreads;  // sequences of a thread
    const int b0 = min(p.B, static_cast<int>(threadIdx.x) * run), b1 = min(p.B, b0 + run);
    bool bad;
    long long mine = 0;
    for (int b = b0; b < b1; ++b) mine += stages_of<TK>(length_of(p, b, bad));
    long long upto = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, upto, off);
        if (lane >= off) upto += v;
    }
    if (lane == 31) warp_sum[warp] = upto;
    if (threadIdx.x == 0) sh.left = 0;
    __syncthreads();
    long long before = upto - mine, all = 0;
#pragma unroll
    for (int w = 0; w < kPgWarps; ++w) {
        if (w < warp) before += warp_sum[w];
        all += warp_sum[w];
    }
    const kv4::Cut cut(all * U, gridDim.x);
    if (i < cut.n) {
        const long long at = cut.begin(i);
        long long w0 = before * U;
        if (at >= w0 && at < w0 + mine * U)
            for (int b = b0; b < b1; ++b) {
                const int n = stages_of<TK>(length_of(p, b, bad));
                if (at < w0 + static_cast<long long>(n) * U) {
                    sh.b = b;
                    sh.unit = kv4::divide(at - w0, n);
                    sh.at = static_cast<int>(at - w0 - static_cast<long long>(sh.unit) * n);
                    sh.left = static_cast<int>(cut.begin(i + 1) - at);
                    break;
                }
                w0 += static_cast<long long>(n) * U;
            }
    }
    __syncthreads();
    return all * U;
}

// What a CTA takes: a chunk (of a cluster's, every count-th stage), or share i of the row of all stages.
template <int D, int NT, bool SHARES>
__global__ void __launch_bounds__(kPgWarps * 32, 2) decode_paged_kernel(const __grid_constant__ DecodePagedParams p)
{
    constexpr int TK = pg_tokens(D), ROWS = 8 * NT, kRowStride = D + 4;
    constexpr int TT = D == 128 ? 1 : 2;           // tiles of 16 tokens taken at once
    static_assert(ROWS * kRowStride * 4 <= kPgStages * kPgStageBytes, "a warp's partial fits its ring");
    static_assert(D < 128 || (TK == 16 * TT), "a tile of halves is a stage");
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ __align__(8) uint64_t full[kPgWarps][kPgStages];
    __shared__ float2 merged_rl[kMostRows];
    __shared__ float2 warp_rl[kPgWarps][kMostRows];
    __shared__ kv4::Share sh;
    __shared__ long long row;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const int U = p.Hkv * p.chunks;

    if (SHARES) griddep_launch_dependents();  // the merge kernel
    if (threadIdx.x == 0) {
        cta_err_init(p.wait_ns);
        cta_check_init(p.status, smem_raw, pg_smem(D, NT));
        tma_prefetch_desc(&p.tk);
        tma_prefetch_desc(&p.tv);
    }
    if (lane == 0) {
        for (int i = 0; i < kPgStages; ++i) mbar_init(&full[warp][i], 1 + (warp == 0 && i == 0 ? p.hold : 0));
        fence_mbar_init();
    }
    __syncthreads();
    griddep_wait();  // the kernel before, which may have written what this one reads, is done
    // The second half of the CTAs, which join the first on their SMs, take the shares from the end.
    const int half = gridDim.x / 2;
    const int share = static_cast<int>(blockIdx.x) < half ? blockIdx.x : gridDim.x - 1 - (blockIdx.x - half);
    if constexpr (SHARES) {
        const long long all = share_of<TK>(p, share, sh);
        if (threadIdx.x == 0) row = all;
        if (sh.left <= 0) return;
    }
    uint8_t *const mine = smem + warp * (kPgStages * kPgStageBytes), *const queries = smem + kPgRing;
    const uint32_t ring = smem_u32(mine), sq = smem_u32(queries);
    // A stage is boxes of `box` slots; lanes i and 16 + i load box i of the keys and of the values.
    const int box = min(1 << p.pg.shift, TK), part = (lane & 15) * box, copies = box == TK ? 1 : (D + 63) / 64;
    int slot = 0;
    uint32_t phase = 0;

    while (true) {
        const int whole_chunk = p.by_count.of(blockIdx.x);  // chunk of all sequences
        const int b = SHARES ? sh.b : p.by_U.of(whole_chunk), unit = SHARES ? sh.unit : whole_chunk - b * U;
        const int at = SHARES ? sh.at : blockIdx.x - whole_chunk * p.count;
        const int hk = p.by_chunks.of(unit), chunk = unit - hk * p.chunks;
        const size_t bk = static_cast<size_t>(b) * p.Hkv + hk;
        const int row0 = chunk * ROWS, nrows = min(ROWS, p.rows - row0);
        const __nv_bfloat16 *q0 = p.q + (bk * p.rows + row0) * D;
        Rows8<D, NT> st;
        if constexpr (NT > 2) {
            for (int x = threadIdx.x; x < ROWS * (D / 8); x += kPgWarps * 32) {
                const int r = x / (D / 8), piece = x % (D / 8);
                uint4 w = make_uint4(0, 0, 0, 0);
                if (r < nrows) w = *reinterpret_cast<const uint4 *>(q0 + r * D + 8 * piece);
                *reinterpret_cast<uint4 *>(queries + place<D, kMostRows>(r, piece)) = w;
            }
        } else {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const bool in = 8 * n + g < nrows;
                const __nv_bfloat16 *qp = q0 + (in ? 8 * n + g : 0) * D + 2 * c;
#pragma unroll
                for (int m = 0; m < D / 16; ++m)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        st.q[m][n][i] = in ? *reinterpret_cast<const uint32_t *>(qp + 16 * m + 8 * i) : 0u;
            }
        }
        bool bad;
        const int len = length_of(p, b, bad), n = stages_of<TK>(len);
        const int count = SHARES ? 1 : p.count;
        const int take = SHARES ? min(sh.left, n - at) : n;
        // This CTA's stages [s0, s1) of the chunk (clusters: every count-th of all), dealt to its warps in turn from the newest
        // to the oldest: the bias falls on the way, so the references settle in the first tiles.
        const int s0 = SHARES ? at : 0, s1 = min(s0 + take, (len + TK - 1) / TK);
        const int step = kPgWarps * count;
        if (bad && unit == 0 && threadIdx.x == 0) atomicOr(p.status, ALIBI_DEV_RANGE);
        bool lost = false;  // a page number that is none

        // Page number of this lane's box of stage s, as the table has it: looked at when the copy is issued, a step after it was
        // asked for.
        const auto is_there = [&](int s) { return part < TK && s >= s0 && s * TK + part < len; };
        const auto page_at = [&](int s) { return is_there(s) ? p.pg.number(b, s * TK + part) : 0; };
        const auto fetch = [&](int s, int slot_, int page) {
            if (s < s0) return;
            const bool in = static_cast<unsigned>(page) < static_cast<unsigned>(p.pg.pages), there = is_there(s);
            lost |= there && !in;
            // past the length, and for a number that is none, one beyond the pool, whose box is filled with zeros
            if (!(there && in)) page = p.pg.pages;
            if (lane == 0) mbar_arrive_expect_tx(&full[warp][slot_], kPgStageBytes);
            __syncwarp();
            if (part < TK) {
                constexpr int W = D < 64 ? D : 64;  // elements of a box's row
                const bool values = lane >= 16;
                uint8_t *const to = mine + slot_ * kPgStageBytes + (values ? kPgStageBytes / 2 : 0) + part * (2 * W);
                for (int h = 0; h < copies; ++h)
                    load_box<W>(to + h * (TK * 2 * W), values ? &p.tv : &p.tk, p.pg, box, D / W / copies, p.pg.slot_of(s * TK + part),
                                h, hk, page, &full[warp][slot_]);
            }
        };
        int s = s1 - 1 - (SHARES ? warp : at + warp * count);  // this warp's stages: s, s - step, ...
        // after a wait that ran out in an earlier chunk the ring may be out of step: nothing more is loaded into it
        if (SHARES && *(volatile uint32_t *)&cta_abort != 0u) s = s0 - 1;
        for (int i = 0, k = slot; i < kPgStages; ++i) {
            fetch(s - i * step, k, page_at(s - i * step));
            if (++k == kPgStages) k = 0;
        }
        int page = page_at(s - kPgStages * step);  // of the stage to be fetched next, read an iteration ahead

#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int r = min(row0 + 8 * i + 2 * c + k, p.rows - 1), h = p.by_T.of(r);
                st.slope[i][k] = p.slopes.log2e[hk * p.G + h];
                st.pos[i][k] = static_cast<float>(len - p.T + r - h * p.T - g);
                st.R[i][k] = -FLT_MAX;
                st.l[i][k] = 0.0f;
            }
#pragma unroll
        for (int m = 0; m < D / 16; ++m)
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) st.acc[m][i][e] = 0.0f;
        if constexpr (NT > 2) __syncthreads();  // the queries in shared memory

        for (; s >= s0; s -= step) {
            const int next = s - kPgStages * step, ahead = page_at(next - step);
            if (!__all_sync(0xffffffffu, mbar_wait(&full[warp][slot], phase, p.status, 0x70))) break;
            const uint32_t k = ring + slot * kPgStageBytes, v = k + kPgStageBytes / 2;
            if ((s + 1) * TK > len) {  // slots past the length: their weights are zero, and so are to be their values
                for (int x = (len - s * TK) * (D / 8) + lane; x < TK * (D / 8); x += 32)
                    asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(v + place<D, TK>(x / (D / 8), x % (D / 8))), "r"(0)
                                 : "memory");
                fence_proxy_async_smem();
                __syncwarp();
            }
#pragma unroll 1
            for (int t = TK / (16 * TT) - 1; t >= 0; --t) {
                const int j0 = s * TK + t * 16 * TT;
                if (j0 < len)
                    tokens16<D, NT, TT>(st, k + t * (TT * 32 * D), v + t * (TT * 32 * D), sq, p.c1, j0, len - 1, p.T, lane);
            }
            __syncwarp();
            fetch(next, slot, page);
            page = ahead;
            if (++slot == kPgStages) slot = 0, phase ^= 1u;
        }
        // a wait ran out (recorded): let the copies in flight land before the ring is reused
        for (int i = 0; i < kPgStages && s >= s0; ++i, s -= step) {
            mbar_wait(&full[warp][slot], phase, p.status, 0x71, true);
            if (++slot == kPgStages) slot = 0, phase ^= 1u;
        }
        __syncwarp();

        // the warp's partial: reference R, l = sum of p, and the mean of v (never beyond the largest |v|)
        lost = __any_sync(0xffffffffu, lost);
        if (lost && lane == 0) atomicOr(p.status, ALIBI_DEV_RANGE);
        // after a wait that ran out, here or in an earlier chunk, what was summed is not all that there is
        lost |= *(volatile uint32_t *)&cta_abort != 0u;
        float *pw = reinterpret_cast<float *>(mine);  // [ROWS][D + 4]
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                float l = st.l[i][k];
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
                if (lost) l = __uint_as_float(0x7fc00000u);
                const float inv = l == 0.0f ? 0.0f : 1.0f / l;
                const int r = 8 * i + 2 * c + k;
#pragma unroll
                for (int m = 0; m < D / 16; ++m) {
                    pw[r * kRowStride + 16 * m + g] = st.acc[m][i][k] * inv;
                    pw[r * kRowStride + 16 * m + g + 8] = st.acc[m][i][2 + k] * inv;
                }
                if (g == 0) warp_rl[warp][r] = make_float2(st.R[i][k], l);
            }
        __syncthreads();

        // Merge of the warps' partials, into out, or into a partial of the chunk: Shares in memory, of a cluster's CTA in place of
        // the first warp's.
        const bool whole = SHARES ? take == n : count == 1;
        float *to = SHARES ? p.part + (static_cast<size_t>(share) * 2 + (at == 0)) * part_floats(D, ROWS) : nullptr;
        for (int i = threadIdx.x; i < nrows * (D / 4); i += kPgWarps * 32) {
            const int r = i / (D / 4), e = i % (D / 4) * 4;
            float *base = reinterpret_cast<float *>(smem) + r * kRowStride + e;
            constexpr int kStep = kPgStages * kPgStageBytes / 4;
            const Merged m = merge<kPgWarps>(kPgWarps, [&](int w) { return warp_rl[w][r]; },
                                             [&](int w) { return *reinterpret_cast<const float4 *>(base + w * kStep); });
            if (whole) {
                finish(p.out, p.lse, D, bk * p.rows + row0 + r, e, m, bad);
            } else if (SHARES) {
                *reinterpret_cast<float4 *>(to + r * D + e) = m.o;
                if (e == 0) *reinterpret_cast<float2 *>(to + ROWS * D + 2 * r) = make_float2(m.R, m.l);
            } else {
                *reinterpret_cast<float4 *>(base) = m.o;
                if (e == 0) merged_rl[r] = make_float2(m.R, m.l);
            }
        }
        if constexpr (!SHARES) {
            if (count == 1) return;
            cluster_arrive();
            cluster_wait();
            // This CTA merges `per` of the rows' elements.
            const int items = nrows * (D / 4), per = p.by_count.of(items + count - 1);
            const uint32_t means = smem_u32(smem), rls = smem_u32(merged_rl);
            for (int i = at * per + threadIdx.x; i < min(items, (at + 1) * per); i += kPgWarps * 32) {
                const int r = i / (D / 4), e = i % (D / 4) * 4;
                const auto rl = [&](int w) { return ld_cluster2(rls + r * 8, w); };
                const auto mean = [&](int w) { return ld_cluster4(means + (r * kRowStride + e) * 4, w); };
                const Merged m = count <= 8 ? merge<8>(count, rl, mean) : merge<kv4::kMostCluster>(count, rl, mean);
                finish(p.out, p.lse, D, bk * p.rows + row0 + r, e, m, bad);
            }
            cluster_arrive();  // the other CTAs may still read this one's partial
            cluster_wait();
            return;
        }
        fence_proxy_async_smem();  // the partials were written and read before the next copies overwrite them
        __syncthreads();           // and the share's place read before it changes
        if (threadIdx.x == 0) {
            sh.left -= take;
            sh.at += take;
            if (sh.at == n) {
                Header h = {-1, -1};
                if (take < n) {  // the share's first chunk, whose first stage lies n - take before the share's beginning
                    const kv4::Cut cut(row, gridDim.x);
                    h = {cut.holder(cut.begin(share) + take - n), share};
                }
                p.head[static_cast<size_t>(b) * U + unit] = h;
                sh.at = 0;
                if (++sh.unit == U) sh.unit = 0, ++sh.b;
            }
        }
        __syncthreads();
        if (sh.left <= 0) return;
    }
}

bool aligned(const void *p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Clusters of c CTAs that the current device holds at once, asked for once, with the most shared memory that any of the kernels
// takes: two CTAs per SM as with the least.
template <class Kernel>
cudaError_t cluster_fit(Kernel kernel, int smem, int (&fit)[paged::kMostCluster + 1])
{
    constexpr int kDevices = 64;  // a device beyond is asked every time
    static std::mutex mu;
    static int known[kDevices][paged::kMostCluster + 1];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> g(mu);
    if (dev >= kDevices || known[dev][1] == 0) {
        e = prepare_kernel(reinterpret_cast<const void *>(kernel), smem, 0, true);
        if (e != cudaSuccess) return e;
        fit[0] = 0, fit[1] = 1;
        for (int c = 2; c <= paged::kMostCluster; ++c) {
            cudaLaunchAttribute attr = {};
            attr.id = cudaLaunchAttributeClusterDimension;
            attr.val.clusterDim.x = static_cast<unsigned>(c);
            attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(static_cast<unsigned>(c));
            cfg.blockDim = dim3(kPgWarps * 32);
            cfg.dynamicSmemBytes = static_cast<size_t>(smem);
            cfg.attrs = &attr;
            cfg.numAttrs = 1;
            e = cudaOccupancyMaxActiveClusters(&fit[c], kernel, &cfg);
            if (e != cudaSuccess) return e;
        }
        if (dev < kDevices) std::copy(fit, fit + paged::kMostCluster + 1, known[dev]);
        return cudaSuccess;
    }
    std::copy(known[dev], known[dev] + paged::kMostCluster + 1, fit);
    return cudaSuccess;
}

template <int D, int NT>
cudaError_t launch(DecodePagedParams &p, const alibi_pages *pages, cudaStream_t stream)
{
    constexpr int ROWS = 8 * NT, smem = pg_smem(D, NT);
    p.chunks = (p.rows + ROWS - 1) / ROWS;
    p.by_chunks = Divisor(static_cast<uint32_t>(p.chunks));
    p.by_U = Divisor(static_cast<uint32_t>(p.Hkv * p.chunks));
    const long long units = static_cast<long long>(p.B) * p.Hkv * p.chunks;
    const int stages = (p.L + pg_tokens(D) - 1) / pg_tokens(D), ctas = std::min(2 * num_sms(), kv4::kMostShares);
    const int busy = (stages + kPgWarps - 1) / kPgWarps;  // CTAs that a chunk can keep busy
    const auto chunks = &decode_paged_kernel<D, NT, false>;
    const auto shared = &decode_paged_kernel<D, NT, true>;
    if (!encode_pages(&p.tk, &p.tv, pages, std::min(D, 64), std::min(pages->slots, pg_tokens(D)), pages->slots >= pg_tokens(D))) return cudaErrorInvalidValue;
    p.part = nullptr;
    p.head = nullptr;
    int fit[paged::kMostCluster + 1];
    cudaError_t e = cluster_fit(chunks, pg_smem(128, 4), fit);
    if (e != cudaSuccess) return e;
    const int count = paged::ctas_of_chunk(units, stages, ctas, fit, paged::step_us(D, NT));
    p.count = std::max(count, 1);
    p.by_count = Divisor(static_cast<uint32_t>(p.count));
    if (count > 0) {
        if (units * count > 0x7fffffffLL) return cudaErrorInvalidValue;
        e = prepare_kernel(reinterpret_cast<const void *>(chunks), pg_smem(128, 4), 0, true);
        if (e != cudaSuccess) return e;
        return launch_kernel(chunks, dim3(static_cast<unsigned>(units * count)), kPgWarps * 32, smem, stream, p, count);
    }
    e = prepare_kernel(reinterpret_cast<const void *>(shared), smem, 0);
    if (e != cudaSuccess) return e;
    const int shares = static_cast<int>(std::min<long long>(units * busy, ctas));
    const size_t bytes = static_cast<size_t>(shares) * 2 * part_floats(D, ROWS) * sizeof(float);
    char *ws = nullptr;
    e = cudaMallocFromPoolAsync(reinterpret_cast<void **>(&ws), bytes + static_cast<size_t>(units) * sizeof(Header), decode_pool(), stream);
    if (e != cudaSuccess) return e;
    p.part = reinterpret_cast<float *>(ws);
    p.head = reinterpret_cast<Header *>(ws + bytes);
    e = launch_kernel(shared, dim3(static_cast<unsigned>(shares)), kPgWarps * 32, smem, stream, p);
    if (e == cudaSuccess && shares > 1) {
        MergeParams m = {p.part, p.head, p.out, p.lse, D, p.rows, p.chunks};
        e = launch_kernel(split_merge_kernel<D, ROWS>, dim3(static_cast<unsigned>(units), std::min(p.rows, ROWS)), kMergeThreads, 0,
                          stream, m);
    }
    const cudaError_t f = cudaFreeAsync(ws, stream);
    return e != cudaSuccess ? e : f;
}

template <int D>
cudaError_t launch_rows(DecodePagedParams &p, const alibi_pages *pages, cudaStream_t stream)
{
    return p.rows <= 8 ? launch<D, 1>(p, pages, stream) : p.rows <= 16 ? launch<D, 2>(p, pages, stream) : launch<D, 4>(p, pages, stream);
}

// hold, wait_ns: of the self-test, else 0 and the usual limit
int decode_paged(const void *q, const alibi_pages *pages, const int *lens, void *out, float *lse, int B, int H, int T, int L,
                 const float *slopes, void *stream, int hold, uint64_t wait_ns)
{
    const int st = check_pages(pages);
    if (st != ALIBI_OK) return st;
    if (!q || !out || !aligned(q, 16) || !aligned(out, 16) || !aligned(lens, 4) || !aligned(lse, 4)) return ALIBI_ERR_INVALID;
    if (B < 1 || H < 1 || T < 1 || L < 1 || H % pages->heads != 0) return ALIBI_ERR_INVALID;
    if (static_cast<long long>(L) > static_cast<long long>(pages->width) * pages->slots) return ALIBI_ERR_INVALID;
    if (H > kMaxQueryHeads || T > 16) return ALIBI_ERR_UNSUPPORTED;
    if (static_cast<long long>(B) * H * T > (1LL << 31) - 1) return ALIBI_ERR_UNSUPPORTED;
    if (slopes)
        for (int h = 0; h < H; ++h)
            if (!std::isfinite(slopes[h]) || slopes[h] < 0.0f) return ALIBI_ERR_INVALID;
    DecodePagedParams p;
    if (slopes)
        for (int h = 0; h < H; ++h) p.slopes.log2e[h] = static_cast<float>(static_cast<double>(slopes[h]) * 1.4426950408889634);
    else
        fill_slopes_log2e(H, p.slopes.log2e);
    // A slope beyond 1e30 is 1e30: the bias of the next token is out of reach already, and its multiples stay finite.
    for (int h = 0; h < H; ++h) p.slopes.log2e[h] = std::min(p.slopes.log2e[h], 1e30f);
    p.q = static_cast<const __nv_bfloat16 *>(q);
    p.pg = pages_of(pages);
    p.lens = lens;
    p.out = static_cast<__nv_bfloat16 *>(out);
    p.lse = lse;
    p.status = device_status_word();
    if (!p.status) return ALIBI_ERR_CUDA;
    p.B = B;
    p.Hkv = pages->heads;
    p.T = T;
    p.G = H / pages->heads;
    p.L = L;
    p.rows = p.G * T;
    p.hold = hold;
    p.wait_ns = wait_ns;
    p.by_T = Divisor(static_cast<uint32_t>(T));
    p.c1 = 1.4426950408889634f / sqrtf(static_cast<float>(pages->d));
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    switch (pages->d) {
        case 128: e = launch_rows<128>(p, pages, cs); break;
        case 64: e = launch_rows<64>(p, pages, cs); break;
        case 32: e = launch_rows<32>(p, pages, cs); break;
        default: e = launch_rows<16>(p, pages, cs); break;
    }
    return e == cudaSuccess ? ALIBI_OK : ALIBI_ERR_CUDA;
}

}  // namespace
}  // namespace alibi

using namespace alibi;

extern "C" int alibi_attn_decode_paged(const void *q, const alibi_pages *pages, const int *lens, void *out, float *lse, int B,
                                       int H, int T, int L, const float *slopes, void *stream)
{
    return decode_paged(q, pages, lens, out, lse, B, H, T, L, slopes, stream, 0, kWaitLimitNs);
}

extern "C" int alibi_selftest_decode_paged_timeout(const void *q, const alibi_pages *pages, const int *lens, void *out, float *lse,
                                                   int B, int H, int T, int L, int wait_us, void *stream)
{
    if (!selftest_wait(wait_us)) return ALIBI_ERR_INVALID;
    return decode_paged(q, pages, lens, out, lse, B, H, T, L, nullptr, stream, 1, static_cast<uint64_t>(wait_us) * 1000u);
}
