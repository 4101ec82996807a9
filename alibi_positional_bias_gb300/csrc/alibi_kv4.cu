// 4-bit KV cache: quantising new tokens as they are written, and reading rows back.
//
// A group is 32 consecutive elements x of one token's key or value row. Its element
// of largest magnitude x_m (the positive one when +x and -x tie) gives the scale
//   s = -x_m / 8,   u = min(15, floor(x / s + 8.5)),   value = s (u - 8),
// so x_m itself is code 0 and is held exactly, and all 16 codes are used. x is bf16,
// so s is a bf16 number exactly (below 2^-100 the group is stored as zeros), and the
// quotient of two 8-bit significands either is a multiple of 1/2 or is at least 2^-10
// away from one: x (1/s) in fp32, off by at most 2^-20, with 2^-12 added before the
// floor, decides every element as exact arithmetic does.

#include <cuda_bf16.h>

#include "alibi.h"
#include "kv4.h"
#include "ptx.cuh"

namespace alibi {
namespace {

struct Kv4Params {
    const void *k, *v;  // write: [B, H, T, d] bf16
    void *ko, *vo;      // read: [B, H, T, d] bf16 or fp32
    uint8_t *cache;
    const int *pos, *count;
    uint32_t *status;
    long long rows;     // B H T
    int H, T, C, d;
};

// The rows of sequence b: first row and number, or 0 rows after recording a span
// that does not fit the cache.
__device__ __forceinline__ int2 span_of(const Kv4Params &p, int b, bool report)
{
    const int first = p.pos ? p.pos[b] : 0, n = p.count ? p.count[b] : p.T;
    if (first < 0 || n < 0 || n > p.T || first > p.C - n) {
        if (report && p.status) atomicOr(p.status, ALIBI_DEV_RANGE);
        return make_int2(0, 0);
    }
    return make_int2(first, n);
}

// bf16 bits in order of magnitude, a positive number before the negative one of its magnitude.
__device__ __forceinline__ uint32_t order_key(uint32_t bits) { return ((bits << 1) & 0xfffeu) | (~(bits >> 15) & 1u); }

template <int D>
__global__ void __launch_bounds__(256) kv4_write_kernel(const __grid_constant__ Kv4Params p)
{
    constexpr int LPR = D / 8;  // lanes per row, 8 elements each
    griddep_launch_dependents();
    griddep_wait();
    const long long i = (static_cast<long long>(blockIdx.x) * 256 + threadIdx.x) / LPR;  // (row, key or value)
    const int l = threadIdx.x % LPR;
    const long long row = i >> 1;
    const int side = static_cast<int>(i & 1);
    const bool in = row < p.rows;
    const long long bh = in ? row / p.T : 0;
    const int t = in ? static_cast<int>(row - bh * p.T) : 0;
    const int2 sp = span_of(p, static_cast<int>(bh / p.H), in && t == 0 && l == 0 && bh % p.H == 0);
    const bool live = in && t < sp.y;

    uint32_t w[4] = {0, 0, 0, 0};
    if (live && 8 * l < p.d) {
        const uint4 x = *reinterpret_cast<const uint4 *>(static_cast<const char *>(side ? p.v : p.k) +
                                                         (row * p.d + 8 * l) * 2);
        w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
    }
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) top = max(top, order_key((w[j / 2] >> (16 * (j & 1))) & 0xffffu));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    if (!live) return;
    const uint32_t mag = top >> 1;
    float s = __uint_as_float((mag << 16) | ((top & 1u) ? 0x80000000u : 0u)) * 0.125f;
    float r = 0.0f;
    if (mag < 0x0d80u)  // below 2^-100
        s = 0.0f;
    else if (mag >= 0x7f80u)  // an infinity or a NaN: the group is NaN
        s = __uint_as_float(0x7fc00000u);
    else
        r = __frcp_rn(s);
    uint32_t code = 0;
#pragma unroll
    for (int j = 7; j >= 0; --j) {
        const float x = __uint_as_float((j & 1) ? (w[j / 2] & 0xffff0000u) : (w[j / 2] << 16));
        const float y = fminf(fmaf(x, r, 8.5f + 0x1p-12f), 15.5f);
        code = code * 16 + (__float_as_uint(__fadd_rd(y, 8388608.0f)) & 15u);
    }
    const int tok = sp.x + t, rr = tok % kv4::kBlock, e = 8 * l;
    uint8_t *blk = p.cache + (bh * (p.C / kv4::kBlock) + tok / kv4::kBlock) * kv4::block_bytes(D);
    if (side == 0) {
        *reinterpret_cast<uint32_t *>(blk + kv4::key_byte(D, rr, e)) = code;
    } else {
        *reinterpret_cast<uint16_t *>(blk + kv4::value_byte(D, rr, e)) = static_cast<uint16_t>(code);
        *reinterpret_cast<uint16_t *>(blk + kv4::value_byte(D, rr, e + 4)) = static_cast<uint16_t>(code >> 16);
    }
    if (l % 4 == 0)
        *reinterpret_cast<uint16_t *>(blk + kv4::scale_byte(D, rr, side, l / 4)) =
            static_cast<uint16_t>(__float_as_uint(s) >> 16);
}

template <int D, bool F32>
__global__ void __launch_bounds__(256) kv4_read_kernel(const __grid_constant__ Kv4Params p)
{
    constexpr int LPR = D / 8;
    griddep_launch_dependents();
    griddep_wait();
    const long long i = (static_cast<long long>(blockIdx.x) * 256 + threadIdx.x) / LPR;
    const int l = threadIdx.x % LPR;
    const long long row = i >> 1;
    const int side = static_cast<int>(i & 1);
    if (row >= p.rows || 8 * l >= p.d) return;
    const long long bh = row / p.T;
    const int t = static_cast<int>(row - bh * p.T);
    const int2 sp = span_of(p, static_cast<int>(bh / p.H), t == 0 && l == 0 && bh % p.H == 0);
    if (t >= sp.y) return;
    const int tok = sp.x + t, rr = tok % kv4::kBlock, e = 8 * l;
    const uint8_t *blk = p.cache + (bh * (p.C / kv4::kBlock) + tok / kv4::kBlock) * kv4::block_bytes(D);
    uint32_t code;
    if (side == 0)
        code = *reinterpret_cast<const uint32_t *>(blk + kv4::key_byte(D, rr, e));
    else
        code = *reinterpret_cast<const uint16_t *>(blk + kv4::value_byte(D, rr, e)) |
               (static_cast<uint32_t>(*reinterpret_cast<const uint16_t *>(blk + kv4::value_byte(D, rr, e + 4))) << 16);
    const float s = __uint_as_float(
        static_cast<uint32_t>(*reinterpret_cast<const uint16_t *>(blk + kv4::scale_byte(D, rr, side, l / 4))) << 16);
    float x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = s * (static_cast<float>((code >> (4 * j)) & 15u) - 8.0f);
    void *dst = side ? p.vo : p.ko;
    if (F32) {
        float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(dst) + row * p.d + e);
        o[0] = make_float4(x[0], x[1], x[2], x[3]);
        o[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
        __nv_bfloat162 h[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) h[j] = __floats2bfloat162_rn(x[2 * j], x[2 * j + 1]);
        *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(dst) + row * p.d + e) =
            *reinterpret_cast<const uint4 *>(h);
    }
}

bool aligned(const void *p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int check_sizes(int B, int H, int T, int C, int d)
{
    if (B < 1 || H < 1 || T < 1 || C < 1 || d < 1) return ALIBI_ERR_INVALID;
    if (C % kv4::kBlock != 0 || T > C) return ALIBI_ERR_INVALID;
    if (!decode_supports(d) || H > kMaxHeads || C > (1 << 24)) return ALIBI_ERR_UNSUPPORTED;
    const long long bh = static_cast<long long>(B) * H;
    if (bh > (1LL << 31) - 1 || bh * T > ((1LL << 31) - 1) * 4) return ALIBI_ERR_UNSUPPORTED;
    return ALIBI_OK;
}

template <int D>
cudaError_t launch(const Kv4Params &p, int op, cudaStream_t stream)
{
    const unsigned grid = static_cast<unsigned>((p.rows * 2 * (D / 8) + 255) / 256);
    return launch_overlapped(op == 0   ? kv4_write_kernel<D>
                             : op == 1 ? kv4_read_kernel<D, false>
                                       : kv4_read_kernel<D, true>,
                             dim3(grid), 256, 0, stream, p);
}

int run(Kv4Params &p, int B, int op, void *stream)
{
    p.status = device_status_word();
    if (!p.status) return ALIBI_ERR_CUDA;
    p.rows = static_cast<long long>(B) * p.H * p.T;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    switch (kv4::padded(p.d)) {
        case 128: e = launch<128>(p, op, s); break;
        case 64: e = launch<64>(p, op, s); break;
        default: e = launch<32>(p, op, s); break;
    }
    return e == cudaSuccess ? ALIBI_OK : ALIBI_ERR_CUDA;
}

}  // namespace
}  // namespace alibi

using namespace alibi;

extern "C" int alibi_kv4_block_bytes(int d)
{
    if (d < 1) return ALIBI_ERR_INVALID;
    if (!decode_supports(d)) return ALIBI_ERR_UNSUPPORTED;
    return kv4::block_bytes(kv4::padded(d));
}

extern "C" int alibi_kv4_write(const void *k, const void *v, void *cache, const int *pos, const int *count, int B,
                               int H, int T, int C, int d, void *stream)
{
    if (!k || !v || !cache) return ALIBI_ERR_INVALID;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(cache, 16) || !aligned(pos, 4) || !aligned(count, 4))
        return ALIBI_ERR_INVALID;
    const int st = check_sizes(B, H, T, C, d);
    if (st != ALIBI_OK) return st;
    Kv4Params p = {};
    p.k = k;
    p.v = v;
    p.cache = static_cast<uint8_t *>(cache);
    p.pos = pos;
    p.count = count;
    p.H = H;
    p.T = T;
    p.C = C;
    p.d = d;
    return run(p, B, 0, stream);
}

extern "C" int alibi_kv4_read(const void *cache, void *k, void *v, const int *pos, const int *count, int B, int H,
                              int T, int C, int d, int fp32, void *stream)
{
    if (!k || !v || !cache) return ALIBI_ERR_INVALID;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(cache, 16) || !aligned(pos, 4) || !aligned(count, 4))
        return ALIBI_ERR_INVALID;
    if (fp32 != 0 && fp32 != 1) return ALIBI_ERR_INVALID;
    const int st = check_sizes(B, H, T, C, d);
    if (st != ALIBI_OK) return st;
    Kv4Params p = {};
    p.ko = k;
    p.vo = v;
    p.cache = static_cast<uint8_t *>(const_cast<void *>(cache));
    p.pos = pos;
    p.count = count;
    p.H = H;
    p.T = T;
    p.C = C;
    p.d = d;
    return run(p, B, fp32 ? 2 : 1, stream);
}
