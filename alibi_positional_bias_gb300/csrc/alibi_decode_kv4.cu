// ALiBi attention of the newest tokens of each sequence over its 4-bit KV cache.
//
// Row (h, t) of sequence b is the query of head h at position i = len_b - T + t, with
// len_b tokens in the cache (the new ones included), and h / (H / H_kv) its KV head:
//   x_j = q.k_j / sqrt(d) - m_h (i - j),  j <= i,   out = sum_j softmax_j(x) v_j,
// with k and v the values s (u - 8) that the cache's codes stand for (kv4.h).

#include <cmath>
#include <cuda_bf16.h>

#include "alibi.h"
#include "kv4.h"
#include "ptx.cuh"

namespace alibi {
namespace {

struct HeadSlopes {
    float log2e[kMaxHeads];
};

struct DecodeKv4Params {
    const __nv_bfloat16 *q;  // [B, H, T, d]
    const uint8_t *cache;    // [B, H_kv, C / 32, block]
    const int *lens;         // [B] or null
    __nv_bfloat16 *out;      // [B, H, T, d]
    float *lse;              // [B, H, T] or null
    uint32_t *status;
    int H, Hkv, T, L, C, d;
    float c1;  // log2(e) / sqrt(d)
    HeadSlopes slopes;
};

constexpr int kWarps = 4;

template <int D>
__global__ void __launch_bounds__(kWarps * 32) decode_kv4_kernel(const __grid_constant__ DecodeKv4Params p)
{
    constexpr int E = D / 32;  // elements per lane
    __shared__ float sm_m[kWarps], sm_l[kWarps], sm_o[kWarps][D];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int row = blockIdx.x;  // (b, h, t)
    const int t = row % p.T, bh = row / p.T, h = bh % p.H, b = bh / p.H;
    const int len = p.lens ? p.lens[b] : p.L;
    const bool bad = len < 0 || len > p.L;
    if (bad && h == 0 && t == 0 && threadIdx.x == 0) atomicOr(p.status, ALIBI_DEV_RANGE);
    const int at = bad ? -1 : len - p.T + t;
    const uint8_t *cache = p.cache + static_cast<size_t>(b * p.Hkv + h / (p.H / p.Hkv)) * (p.C / kv4::kBlock) *
                                         kv4::block_bytes(D);
    float q[E], o[E], m = -INFINITY, l = 0.0f;
#pragma unroll
    for (int i = 0; i < E; ++i) {
        const int e = E * lane + i;
        q[i] = e < p.d ? __bfloat162float(p.q[static_cast<size_t>(row) * p.d + e]) * p.c1 : 0.0f;
        o[i] = 0.0f;
    }
    for (int j = warp; j <= at; j += kWarps) {
        const uint8_t *blk = cache + static_cast<size_t>(j / kv4::kBlock) * kv4::block_bytes(D);
        const int r = j % kv4::kBlock;
        float x = 0.0f, v[E];
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const int e = E * lane + i, sh = 4 * (e & 1);
            const float sk = __uint_as_float(
                uint32_t(*reinterpret_cast<const uint16_t *>(blk + kv4::scale_byte(D, r, 0, e / 32))) << 16);
            const float sv = __uint_as_float(
                uint32_t(*reinterpret_cast<const uint16_t *>(blk + kv4::scale_byte(D, r, 1, e / 32))) << 16);
            x = fmaf(q[i], sk * (float((blk[kv4::key_byte(D, r, e & ~1)] >> sh) & 15) - 8.0f), x);
            v[i] = sv * (float((blk[kv4::value_byte(D, r, e & ~1)] >> sh) & 15) - 8.0f);
        }
#pragma unroll
        for (int off = 16; off; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
        x = fmaf(-p.slopes.log2e[h], static_cast<float>(at - j), x);
        const float mn = fmaxf(m, x), a = ex2_approx(m - mn), w = ex2_approx(x - mn);
        m = mn;
        l = fmaf(l, a, w);
#pragma unroll
        for (int i = 0; i < E; ++i) o[i] = fmaf(o[i], a, w * v[i]);
    }
    if (lane == 0) sm_m[warp] = m, sm_l[warp] = l;
#pragma unroll
    for (int i = 0; i < E; ++i) sm_o[warp][E * lane + i] = o[i];
    __syncthreads();
    float M = -INFINITY, Ls = 0.0f;
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm_m[w]);
    for (int w = 0; w < kWarps; ++w) Ls += sm_m[w] == -INFINITY ? 0.0f : sm_l[w] * ex2_approx(sm_m[w] - M);
    const float none = bad ? __uint_as_float(0x7fc00000u) : 0.0f;
    for (int e = threadIdx.x; e < p.d; e += kWarps * 32) {
        float O = 0.0f;
        for (int w = 0; w < kWarps; ++w) O += sm_m[w] == -INFINITY ? 0.0f : sm_o[w][e] * ex2_approx(sm_m[w] - M);
        p.out[static_cast<size_t>(row) * p.d + e] = __float2bfloat16_rn(at < 0 ? none : O / Ls);
    }
    if (p.lse && threadIdx.x == 0)
        p.lse[row] = bad ? none : at < 0 ? -INFINITY : (M + log2f(Ls)) * 0.6931471805599453f;
}

bool aligned(const void *p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

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
    if (!decode_supports(d) || H > kMaxHeads || T > 16 || C > (1 << 24)) return ALIBI_ERR_UNSUPPORTED;
    if (static_cast<long long>(B) * H * T > (1LL << 31) - 1) return ALIBI_ERR_UNSUPPORTED;
    if (slopes)
        for (int h = 0; h < H; ++h)
            if (!std::isfinite(slopes[h]) || slopes[h] < 0.0f) return ALIBI_ERR_INVALID;
    Slopes s;
    if (slopes)
        fill_slopes_from(H, slopes, &s);
    else
        fill_slopes(H, &s);
    DecodeKv4Params p;
    p.q = static_cast<const __nv_bfloat16 *>(q);
    p.cache = static_cast<const uint8_t *>(cache);
    p.lens = lens;
    p.out = static_cast<__nv_bfloat16 *>(out);
    p.lse = lse;
    p.status = device_status_word();
    if (!p.status) return ALIBI_ERR_CUDA;
    p.H = H;
    p.Hkv = Hkv;
    p.T = T;
    p.L = L;
    p.C = C;
    p.d = d;
    p.c1 = 1.4426950408889634f / sqrtf(static_cast<float>(d));
    for (int h = 0; h < H; ++h) p.slopes.log2e[h] = s.log2e[h];
    const unsigned grid = static_cast<unsigned>(B * H * T);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    switch (kv4::padded(d)) {
        case 128: decode_kv4_kernel<128><<<grid, kWarps * 32, 0, st>>>(p); break;
        case 64: decode_kv4_kernel<64><<<grid, kWarps * 32, 0, st>>>(p); break;
        default: decode_kv4_kernel<32><<<grid, kWarps * 32, 0, st>>>(p); break;
    }
    return cudaGetLastError() == cudaSuccess ? ALIBI_OK : ALIBI_ERR_CUDA;
}
