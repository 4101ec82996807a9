// Joining the partial results of a softmax over slices of the keys: what the decodes over the 4-bit and the paged cache
// share. A partial of a row is its reference R (base 2), l = sum of 2^(x_j - R) and the mean of v under those weights.
#pragma once

#include <cfloat>
#include <cmath>
#include <cuda_bf16.h>

#include "kv4_deal.h"
#include "ptx.cuh"

namespace alibi {
namespace {

constexpr int kMergeThreads = 256;

struct HeadSlopes {
    float log2e[kMaxQueryHeads];
};

// What a share leaves behind for the merge: the partial of a chunk that began in an earlier share (0) and of one that
// goes on in a later one (1), each of `rows` rows of D means and then (R, l) of each row.
KV4_HD constexpr int part_floats(int D, int rows) { return rows * (D + 2); }

struct alignas(8) Header {  // of a chunk
    int first, last;  // the shares it begins and ends in, or -1 where one share did all of it
};

struct MergeParams {
    const float *part;
    const Header *head;
    __nv_bfloat16 *out;
    float *lse;
    int d, rows, chunks;
};

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

// Merge of the chunks that several shares worked on: CTA (i, r) looks at row r of chunk i. Its partials are slot 1 of the
// share it began in and slot 0 of the shares up to the one it ends in. The loads of a thread are issued
// together: with 76 partials the merge waits for three round trips to L2 and not for 76. At most 64 registers, so that a CTA
// finds room beside the two of a decode on its SM and waits there for their end: 1 x 4 (x 4) x 131071 tokens over pages 48.2 us (48.8
// with 8 means at once, 49.1 with 12 and 74 registers), 1 x 1 x 8192 7.2 (7.9), over the 4-bit cache 16.3 (17.0).
template <int D, int ROWS>
__global__ void __launch_bounds__(kMergeThreads, 4) split_merge_kernel(const __grid_constant__ MergeParams p)
{
    constexpr int kPart = part_floats(D, ROWS), kItems = D / 4, kGroups = kMergeThreads / kItems, kDepth = 10;
    __shared__ float weight[kv4::kMostShares];
    __shared__ float red[2][kMergeThreads / 32];
    __shared__ float4 sum[kMergeThreads];
    griddep_wait();
    const int unit = blockIdx.x, r = blockIdx.y;
    const int2 h = __ldcg(reinterpret_cast<const int2 *>(p.head + unit));  // (first, last)
    if (h.x < 0) return;
    const int n = h.y - h.x + 1;
    const int bk = unit / p.chunks, row0 = (unit - bk * p.chunks) * ROWS;
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
    float2 x[kv4::kMostShares / kMergeThreads];
#pragma unroll
    for (int i = 0; i < kv4::kMostShares / kMergeThreads; ++i) {
        const int k = threadIdx.x + i * kMergeThreads;
        x[i] = k < n ? __ldcg(reinterpret_cast<const float2 *>(from(k) + ROWS * D + 2 * r)) : make_float2(-FLT_MAX, 0.0f);
        R = fmaxf(R, x[i].x);
    }
#pragma unroll
    for (int off = 16; off; off >>= 1) R = fmaxf(R, __shfl_xor_sync(0xffffffffu, R, off));
    if (lane == 0) red[0][warp] = R;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kMergeThreads / 32; ++w) R = fmaxf(R, red[0][w]);
#pragma unroll
    for (int i = 0; i < kv4::kMostShares / kMergeThreads; ++i) {
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

}  // namespace
}  // namespace alibi
