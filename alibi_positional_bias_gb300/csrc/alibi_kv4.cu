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

#include <algorithm>
#include <cuda_bf16.h>

#include "alibi.h"
#include "kv4.h"
#include "ptx.cuh"

namespace alibi {
namespace {

struct Kv4Params {
    const char *k, *v;  // write: [B, H, T, d] bf16
    char *ko, *vo;      // read: [B, H, T, d] bf16 or fp32
    uint8_t *cache;
    const int *pos, *count;
    uint32_t *status;
    int BH, H, T, blocks, d;  // blocks: C / 32
    int span;                 // blocks that T tokens can touch, from any row on
};

// The rows of sequence b: first row and number, or 0 rows after recording a span
// that does not fit the cache.
__device__ __forceinline__ int2 span_of(const Kv4Params &p, int b, bool report)
{
    const int first = p.pos ? p.pos[b] : 0, n = p.count ? p.count[b] : p.T;
    if (first < 0 || n < 0 || n > p.T || first > p.blocks * kv4::kBlock - n) {
        if (report) atomicOr(p.status, ALIBI_DEV_RANGE);
        return make_int2(0, 0);
    }
    return make_int2(first, n);
}

// Two bf16 numbers in order of magnitude, each in 16 bits, a positive one before the negative one of its magnitude.
__device__ __forceinline__ uint32_t order_keys(uint32_t w) { return ((w << 1) & 0xfffefffeu) | (~(w >> 15) & 0x00010001u); }

// From the largest order key of a group: bf16 bits of the scale s, and 1 / s (0 where all codes are 8).
struct Scale {
    uint32_t bits;
    float inverse;
};

__device__ __forceinline__ Scale scale_of(uint32_t key)
{
    const uint32_t mag = key >> 1;
    if (mag < 0x0d80u) return {0u, 0.0f};            // below 2^-100: zeros
    if (mag >= 0x7f80u) return {0x7fc0u, 0.0f};      // an infinity or a NaN: the group is NaN
    const uint32_t bits = (mag - (3u << 7)) | ((key & 1u) << 15);  // -x_m / 8
    return {bits, __frcp_rn(__uint_as_float(bits << 16))};
}

// Code of x in the low four bits (and more above them).
__device__ __forceinline__ uint32_t code_of(float x, float inverse)
{
    // 8.5 + x / s, and 2^-12 against the error of the product; the sum with 2^23 leaves its floor in the low bits
    return __float_as_uint(__fadd_rd(fminf(fmaf(x, inverse, 8.5f + 0x1p-12f), 15.5f), 8388608.0f));
}

// Codes of four bf16 numbers, 16 bits.
__device__ __forceinline__ uint32_t codes4(uint2 w, float inverse)
{
    uint32_t c = code_of(__uint_as_float(w.y & 0xffff0000u), inverse);
    c = c * 16 + code_of(__uint_as_float(w.y << 16), inverse);
    c = c * 16 + code_of(__uint_as_float(w.x & 0xffff0000u), inverse);
    c = c * 16 + code_of(__uint_as_float(w.x << 16), inverse);
    return c - 0x4b000000u * (1u + 16u + 256u + 4096u);  // the exponents of the four sums
}

// Values of four codes (the low 16 bits of w) times s.
__device__ __forceinline__ float4 values4(uint32_t w, float s)
{
    const auto value = [&](uint32_t u) { return s * (__uint_as_float(0x4b000000u | u) - 8388616.0f); };
    return make_float4(value(w & 15u), value(w >> 4 & 15u), value(w >> 8 & 15u), value(w >> 12 & 15u));
}

template <bool F32>
__device__ __forceinline__ void put4(char *row, int e, float4 x)
{
    if (F32) {
        *reinterpret_cast<float4 *>(row + 4 * e) = x;
    } else {
        const __nv_bfloat162 h[2] = {__floats2bfloat162_rn(x.x, x.y), __floats2bfloat162_rn(x.z, x.w)};
        *reinterpret_cast<uint2 *>(row + 2 * e) = *reinterpret_cast<const uint2 *>(h);
    }
}

__device__ __forceinline__ float bf16_at(const uint8_t *p)
{
    return __uint_as_float(static_cast<uint32_t>(*reinterpret_cast<const uint16_t *>(p)) << 16);
}

// A row's key or value per D / 8 lanes, 8 elements each: for few tokens per sequence, whose blocks are mostly
// other tokens'. Row i of the launch is token i % T of head i / T, keys (side 0) or values.
struct RowItem {
    int bh, t, side, l;
    bool in;
};

template <int D>
__device__ __forceinline__ RowItem row_item(const Kv4Params &p)
{
    constexpr int kRowsPerCta = 256 / (D / 8);
    const unsigned i = blockIdx.x * (kRowsPerCta / 2) + threadIdx.x / (2 * (D / 8));
    RowItem r;
    r.in = i < static_cast<unsigned>(p.BH) * static_cast<unsigned>(p.T);
    r.bh = r.in ? static_cast<int>(i / static_cast<unsigned>(p.T)) : 0;
    r.t = r.in ? static_cast<int>(i - static_cast<unsigned>(r.bh) * static_cast<unsigned>(p.T)) : 0;
    r.side = threadIdx.x / (D / 8) % 2;
    r.l = threadIdx.x % (D / 8);
    return r;
}

template <int D>
__global__ void __launch_bounds__(256) kv4_write_rows_kernel(const __grid_constant__ Kv4Params p)
{
    griddep_launch_dependents();
    griddep_wait();
    const RowItem r = row_item<D>(p);
    const int b = r.bh / p.H, e = 8 * r.l;
    const int2 sp = span_of(p, b, r.in && r.t == 0 && threadIdx.x % (2 * (D / 8)) == 0 && r.bh == b * p.H);
    const bool live = r.in && r.t < sp.y;
    uint4 w = make_uint4(0, 0, 0, 0);
    if (live && e < p.d)
        w = *reinterpret_cast<const uint4 *>((r.side ? p.v : p.k) + ((static_cast<size_t>(r.bh) * p.T + r.t) * p.d + e) * 2);
    uint32_t top = __vmaxu2(__vmaxu2(order_keys(w.x), order_keys(w.y)), __vmaxu2(order_keys(w.z), order_keys(w.w)));
    top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 2));
    if (!live) return;
    const Scale s = scale_of(max(top & 0xffffu, top >> 16));
    const uint32_t lo = codes4(make_uint2(w.x, w.y), s.inverse), hi = codes4(make_uint2(w.z, w.w), s.inverse);
    const int tok = sp.x + r.t, row = tok % kv4::kBlock;
    uint8_t *blk = p.cache + (static_cast<size_t>(r.bh) * p.blocks + tok / kv4::kBlock) * kv4::block_bytes(D);
    if (r.side == 0) {
        *reinterpret_cast<uint32_t *>(blk + kv4::key_byte(D, row, e)) = lo | hi << 16;
    } else {
        *reinterpret_cast<uint16_t *>(blk + kv4::value_byte(D, row, e)) = static_cast<uint16_t>(lo);
        *reinterpret_cast<uint16_t *>(blk + kv4::value_byte(D, row, e + 4)) = static_cast<uint16_t>(hi);
    }
    if (r.l % 4 == 0)
        *reinterpret_cast<uint16_t *>(blk + kv4::scale_byte(D, row, r.side, r.l / 4)) = static_cast<uint16_t>(s.bits);
}

template <int D, bool F32>
__global__ void __launch_bounds__(256) kv4_read_rows_kernel(const __grid_constant__ Kv4Params p)
{
    griddep_launch_dependents();
    griddep_wait();
    const RowItem r = row_item<D>(p);
    const int b = r.bh / p.H, e = 8 * r.l;
    const int2 sp = span_of(p, b, r.in && r.t == 0 && threadIdx.x % (2 * (D / 8)) == 0 && r.bh == b * p.H);
    if (!r.in || r.t >= sp.y || e >= p.d) return;
    const int tok = sp.x + r.t, row = tok % kv4::kBlock;
    const uint8_t *blk = p.cache + (static_cast<size_t>(r.bh) * p.blocks + tok / kv4::kBlock) * kv4::block_bytes(D);
    uint32_t code;
    if (r.side == 0)
        code = *reinterpret_cast<const uint32_t *>(blk + kv4::key_byte(D, row, e));
    else
        code = *reinterpret_cast<const uint16_t *>(blk + kv4::value_byte(D, row, e)) |
               (static_cast<uint32_t>(*reinterpret_cast<const uint16_t *>(blk + kv4::value_byte(D, row, e + 4))) << 16);
    const float s = bf16_at(blk + kv4::scale_byte(D, row, r.side, r.l / 4));
    char *out = (r.side ? p.vo : p.ko) + (static_cast<size_t>(r.bh) * p.T + r.t) * p.d * (F32 ? 4 : 2);
    put4<F32>(out, e, values4(code, s));
    put4<F32>(out, e + 4, values4(code >> 16, s));
}

// A block of the cache per CTA: half of the threads for the keys, half for the values. A thread takes the piece that lies
// together in the cache, 4 D / 32 bytes of a key row (8 elements of every group) or one lane's 16 bytes of a value tile
// (4 elements of up to two groups, of 4 tokens), so that the cache is read and written in whole 16-byte
// words without shared memory, and the rows in whole 64-byte segments.
struct BlockItem {
    int bh, first, n;  // head; token of the call in the block's row 0 (may be negative), tokens of the call
    uint8_t *blk;
};

template <int D>
__device__ __forceinline__ bool block_item(const Kv4Params &p, BlockItem &it)
{
    it.bh = blockIdx.x / p.span;
    const int i = blockIdx.x - it.bh * p.span, b = it.bh / p.H;
    const int2 sp = span_of(p, b, threadIdx.x == 0 && i == 0 && it.bh == b * p.H);
    const int block = sp.x / kv4::kBlock + i;
    it.first = block * kv4::kBlock - sp.x;
    it.n = sp.y;
    it.blk = p.cache + (static_cast<size_t>(it.bh) * p.blocks + block) * kv4::block_bytes(D);
    return it.first < it.n;  // the block has tokens of the call (it is inside the cache then)
}

constexpr int kHalf = 128;  // threads for the keys, and for the values
constexpr int kWriteCtas = 5, kReadCtas = 6;

template <int D>
__global__ void __launch_bounds__(2 * kHalf, kWriteCtas) kv4_write_block_kernel(const __grid_constant__ Kv4Params p)
{
    constexpr int NG = D / 32;
    griddep_launch_dependents();
    griddep_wait();
    BlockItem it;
    if (!block_item<D>(p, it)) return;
    const auto live = [&](int row) { return static_cast<unsigned>(it.first + row) < static_cast<unsigned>(it.n); };
    const auto at = [&](const char *x, int row) { return x + (static_cast<size_t>(it.bh) * p.T + it.first + row) * p.d * 2; };
    if (threadIdx.x < kHalf) {
        const int row = threadIdx.x / 4, c = threadIdx.x % 4;
        uint4 w[NG];
#pragma unroll
        for (int n = 0; n < NG; ++n) {
            w[n] = make_uint4(0, 0, 0, 0);
            if (live(row) && 32 * n + 8 * c < p.d) w[n] = *reinterpret_cast<const uint4 *>(at(p.k, row) + (32 * n + 8 * c) * 2);
        }
        uint32_t code[NG], bits[NG];
#pragma unroll
        for (int n = 0; n < NG; ++n) {
            uint32_t top = __vmaxu2(__vmaxu2(order_keys(w[n].x), order_keys(w[n].y)),
                                    __vmaxu2(order_keys(w[n].z), order_keys(w[n].w)));
            top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const Scale s = scale_of(max(top & 0xffffu, top >> 16));
            code[n] = codes4(make_uint2(w[n].x, w[n].y), s.inverse) | codes4(make_uint2(w[n].z, w[n].w), s.inverse) << 16;
            bits[n] = s.bits;
        }
        if (!live(row)) return;
        uint8_t *dst = it.blk + kv4::key_byte(D, row, 8 * c);
        if constexpr (NG == 4)
            *reinterpret_cast<uint4 *>(dst) = make_uint4(code[0], code[1], code[2], code[3]);
        else if constexpr (NG == 2)
            *reinterpret_cast<uint2 *>(dst) = make_uint2(code[0], code[1]);
        else
            *reinterpret_cast<uint32_t *>(dst) = code[0];
#pragma unroll
        for (int n = 0; n < NG; ++n)
            if (c == n) *reinterpret_cast<uint16_t *>(it.blk + kv4::scale_byte(D, row, 0, n)) = static_cast<uint16_t>(bits[n]);
    } else {
        constexpr int kChunks = NG > 2 ? NG / 2 : 1, NL = NG < 2 ? NG : 2;  // groups of a lane's piece
        const int i = threadIdx.x - kHalf, lane = i % 32, g = lane / 4, c = lane % 4;
        const int tile = i / 32 % 2, chunk = i / 64;
        if (chunk >= kChunks) return;  // whole warps
        uint32_t code[NL][2];
        uint2 w[NL][4];  // of the tokens 2c, 2c + 1, 2c + 8, 2c + 9 of the tile
#pragma unroll
        for (int m = 0; m < NL; ++m)
#pragma unroll
            for (int z = 0; z < 4; ++z) {
                const int row = 16 * tile + 8 * (z / 2) + 2 * c + z % 2, e = 64 * chunk + 32 * m + 4 * g;
                w[m][z] = make_uint2(0, 0);
                if (live(row) && e < p.d) w[m][z] = *reinterpret_cast<const uint2 *>(at(p.v, row) + e * 2);
            }
#pragma unroll
        for (int m = 0; m < NL; ++m) {
            uint32_t top[4];
#pragma unroll
            for (int z = 0; z < 4; ++z) {
                const uint32_t t = __vmaxu2(order_keys(w[m][z].x), order_keys(w[m][z].y));
                top[z] = max(t & 0xffffu, t >> 16);
            }
            uint32_t pair[2] = {top[0] | top[1] << 16, top[2] | top[3] << 16};
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) {
                pair[0] = __vmaxu2(pair[0], __shfl_xor_sync(0xffffffffu, pair[0], off));
                pair[1] = __vmaxu2(pair[1], __shfl_xor_sync(0xffffffffu, pair[1], off));
            }
#pragma unroll
            for (int z = 0; z < 4; ++z) {
                const int row = 16 * tile + 8 * (z / 2) + 2 * c + z % 2;
                const Scale s = scale_of(z % 2 ? pair[z / 2] >> 16 : pair[z / 2] & 0xffffu);
                const uint32_t u = codes4(w[m][z], s.inverse);
                code[m][z / 2] = z % 2 ? code[m][z / 2] | u << 16 : u;
                if (g == z && live(row))
                    *reinterpret_cast<uint16_t *>(it.blk + kv4::scale_byte(D, row, 1, 2 * chunk + m)) = static_cast<uint16_t>(s.bits);
            }
        }
        uint8_t *dst = it.blk + kv4::value_byte(D, 16 * tile + 2 * c, 64 * chunk + 4 * g);
        const int row = 16 * tile + 2 * c;
        if (live(row) && live(row + 9)) {  // and the tokens between
            if constexpr (NL == 2)
                *reinterpret_cast<uint4 *>(dst) = make_uint4(code[0][0], code[0][1], code[1][0], code[1][1]);
            else
                *reinterpret_cast<uint2 *>(dst) = make_uint2(code[0][0], code[0][1]);
        } else {
#pragma unroll
            for (int m = 0; m < NL; ++m)
#pragma unroll
                for (int z = 0; z < 4; ++z)
                    if (live(row + 8 * (z / 2) + z % 2))
                        *reinterpret_cast<uint16_t *>(dst + 8 * m + 2 * z) = static_cast<uint16_t>(code[m][z / 2] >> (16 * (z % 2)));
        }
    }
}

template <int D, bool F32>
__global__ void __launch_bounds__(2 * kHalf, kReadCtas) kv4_read_block_kernel(const __grid_constant__ Kv4Params p)
{
    constexpr int NG = D / 32;
    griddep_launch_dependents();
    griddep_wait();
    BlockItem it;
    if (!block_item<D>(p, it)) return;
    const auto live = [&](int row) { return static_cast<unsigned>(it.first + row) < static_cast<unsigned>(it.n); };
    const auto at = [&](char *x, int row) { return x + (static_cast<size_t>(it.bh) * p.T + it.first + row) * p.d * (F32 ? 4 : 2); };
    if (threadIdx.x < kHalf) {
        const int row = threadIdx.x / 4, c = threadIdx.x % 4;
        if (!live(row)) return;
        uint32_t code[NG];
        const uint8_t *src = it.blk + kv4::key_byte(D, row, 8 * c);
        if constexpr (NG == 4) {
            const uint4 x = *reinterpret_cast<const uint4 *>(src);
            code[0] = x.x, code[1] = x.y, code[2] = x.z, code[3] = x.w;
        } else if constexpr (NG == 2) {
            const uint2 x = *reinterpret_cast<const uint2 *>(src);
            code[0] = x.x, code[1] = x.y;
        } else {
            code[0] = *reinterpret_cast<const uint32_t *>(src);
        }
        char *out = at(p.ko, row);
#pragma unroll
        for (int n = 0; n < NG; ++n) {
            const int e = 32 * n + 8 * c;
            if (e >= p.d) continue;
            const float s = bf16_at(it.blk + kv4::scale_byte(D, row, 0, n));
            const float4 x = values4(code[n], s), y = values4(code[n] >> 16, s);
            if (F32) {
                put4<true>(out, e, x);
                put4<true>(out, e + 4, y);
            } else {
                const __nv_bfloat162 h[4] = {__floats2bfloat162_rn(x.x, x.y), __floats2bfloat162_rn(x.z, x.w),
                                             __floats2bfloat162_rn(y.x, y.y), __floats2bfloat162_rn(y.z, y.w)};
                *reinterpret_cast<uint4 *>(out + 2 * e) = *reinterpret_cast<const uint4 *>(h);
            }
        }
    } else {
        constexpr int kChunks = NG > 2 ? NG / 2 : 1, NL = NG < 2 ? NG : 2;
        const int i = threadIdx.x - kHalf, lane = i % 32, g = lane / 4, c = lane % 4;
        const int tile = i / 32 % 2, chunk = i / 64, row0 = 16 * tile + 2 * c;
        if (chunk >= kChunks) return;
        uint32_t code[NL][2];
        const uint8_t *src = it.blk + kv4::value_byte(D, row0, 64 * chunk + 4 * g);
        if constexpr (NL == 2) {
            const uint4 x = *reinterpret_cast<const uint4 *>(src);
            code[0][0] = x.x, code[0][1] = x.y, code[1][0] = x.z, code[1][1] = x.w;
        } else {
            const uint2 x = *reinterpret_cast<const uint2 *>(src);
            code[0][0] = x.x, code[0][1] = x.y;
        }
#pragma unroll
        for (int z = 0; z < 4; ++z) {
            const int row = row0 + 8 * (z / 2) + z % 2;
            if (live(row)) {
                char *out = at(p.vo, row);
#pragma unroll
                for (int m = 0; m < NL; ++m) {
                    const int n = 2 * chunk + m, e = 32 * n + 4 * g;
                    if (e < p.d)
                        put4<F32>(out, e, values4(code[m][z / 2] >> (16 * (z % 2)), bf16_at(it.blk + kv4::scale_byte(D, row, 1, n))));
                }
            }
        }
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

// Tokens per sequence from which a CTA takes a block and not single rows.
constexpr int kBlockTokens = 16;

template <int D>
cudaError_t launch(Kv4Params &p, int op, cudaStream_t stream)
{
    const long long rows = static_cast<long long>(p.BH) * p.T;
    if (p.T < kBlockTokens && rows < (1LL << 31)) {
        constexpr int kRowsPerCta = 256 / (D / 8) / 2;
        return launch_overlapped(op == 0   ? kv4_write_rows_kernel<D>
                                 : op == 1 ? kv4_read_rows_kernel<D, false>
                                           : kv4_read_rows_kernel<D, true>,
                                 dim3(static_cast<unsigned>((rows + kRowsPerCta - 1) / kRowsPerCta)), 256, 0, stream, p);
    }
    p.span = std::min(p.blocks, (p.T + 2 * kv4::kBlock - 2) / kv4::kBlock);
    const long long ctas = static_cast<long long>(p.BH) * p.span;
    if (ctas > 0x7fffffffLL) return cudaErrorInvalidValue;
    return launch_overlapped(op == 0   ? kv4_write_block_kernel<D>
                             : op == 1 ? kv4_read_block_kernel<D, false>
                                       : kv4_read_block_kernel<D, true>,
                             dim3(static_cast<unsigned>(ctas)), 2 * kHalf, 0, stream, p);
}

// op: 0 write, 1 read as bf16, 2 read as fp32
int run(Kv4Params p, int op, void *stream)
{
    p.status = device_status_word();
    if (!p.status) return ALIBI_ERR_CUDA;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    switch (kv4::padded(p.d)) {
        case 128: e = launch<128>(p, op, s); break;
        case 64: e = launch<64>(p, op, s); break;
        default: e = launch<32>(p, op, s); break;
    }
    return e == cudaSuccess ? ALIBI_OK : ALIBI_ERR_CUDA;
}

Kv4Params params(const void *cache, const int *pos, const int *count, int B, int H, int T, int C, int d)
{
    Kv4Params p = {};
    p.cache = static_cast<uint8_t *>(const_cast<void *>(cache));
    p.pos = pos;
    p.count = count;
    p.BH = B * H;
    p.H = H;
    p.T = T;
    p.blocks = C / kv4::kBlock;
    p.d = d;
    return p;
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
    Kv4Params p = params(cache, pos, count, B, H, T, C, d);
    p.k = static_cast<const char *>(k);
    p.v = static_cast<const char *>(v);
    return run(p, 0, stream);
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
    Kv4Params p = params(cache, pos, count, B, H, T, C, d);
    p.ko = static_cast<char *>(k);
    p.vo = static_cast<char *>(v);
    return run(p, fp32 ? 2 : 1, stream);
}
