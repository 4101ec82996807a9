// 4-bit KV cache: quantising new tokens as they are written, and reading rows back.
//
// A group is 32 consecutive elements x of one token's key or value row. Its element
// of largest magnitude x_m (the positive one when +x and -x tie) gives the scale
//   s = -x_m / 8,   u = min(15, floor(x / s + 8.5)),   value = s (u - 8),
// so x_m itself is code 0 and is held exactly, and all 16 codes are used. x is bf16,
// so s is a bf16 number exactly (below 2^-100 the group is stored as zeros), and the
// quotient of two 8-bit significands either is a multiple of 1/2 or is at least 2^-10
// away from one: x (1/s) in fp32, off by at most 2^-19, with 2^-12 added before the
// floor, decides every element as exact arithmetic does.
//
// What has to move: 4 d bytes of a token's key and value and 1.125 d of the cache. Prompts
// go a block per CTA, the cache in whole 16-byte words of a thread, the rows in 64-byte
// segments, no shared memory. Written and read back, calls in one graph over sets of tensors that together are larger
// than L2, in us and TB/s (the measured copy: 6.7):
//   4 x 32 heads x 2048 tokens, d = 128    28.2 (6.1)   26.4 (6.5)   as fp32 47.5 (6.5)
//   8 x 32 x 2048, d = 128                 53.0 (6.5)   50.3 (6.8)   91.5 (6.7)
//   8 x 32 x 4096, d = 64                  56.0 (6.1)   52.9 (6.5)   90.7 (6.7)
//   8 x 32 x 8192, d = 32                  66.2 (5.2)   61.3 (5.6)   93.3 (6.6)
//   64 x 40 x 1, d = 128                    3.0          3.3          3.4
// The write is bound by memory's latency and the logic pipe (59% busy, 68% of
// issue slots): 10 operations per element, of which the group's largest takes 1, the codes 4;
// one thread per 8 elements with 16-bit stores of the values took 161 us for the first case's two calls. A step's new
// token takes a launch's time. Every launch overlaps the end of the kernel before it (each kernel
// waits for that before it touches memory): the first case written and read in turn takes 54.3 and not 55.7 us, 64 x 40 x 16
// tokens 18.0 and not 19.3; a single token's two calls, 6.8 us, take 6.5 without.

#include <algorithm>
#include <cuda_bf16.h>

#include "alibi.h"
#include "kv4_deal.h"
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
    int run, runs;            // blocks of a CTA, and runs of so many that T tokens can touch from any row on
    kv4::Divisor by_runs, by_H, by_T;
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

// The largest element of each half of N words of two bf16 numbers, as keys in order of magnitude, a positive one before the
// negative one of its magnitude: the magnitude, and below it the sign, inverted. As signed 16-bit numbers the largest
// positive one comes first, as unsigned ones the largest negative one: one operation per word and sign.
template <int N>
__device__ __forceinline__ uint32_t top_keys(const uint32_t (&w)[N])
{
    uint32_t above = w[0], below = w[0];
#pragma unroll
    for (int i = 1; i < N; ++i) above = __vmaxs2(above, w[i]), below = __vmaxu2(below, w[i]);
    return __vmaxu2(__vmaxs2(above, 0u) * 2u + 0x00010001u, (below & 0x7fff7fffu) * 2u);
}

// The larger of the two halves.
__device__ __forceinline__ uint32_t fold(uint32_t keys) { return max(keys & 0xffffu, keys >> 16); }

// From the largest order key of a group: bf16 bits of the scale s, and 1 / (16 s) (0 where nothing is to be scaled). The
// reciprocal is the approximate one, good to 2^-23, as code_of allows for.
struct Scale {
    uint32_t bits;
    float inverse;
};

__device__ __forceinline__ Scale scale_of(uint32_t key)
{
    const uint32_t mag = key >> 1;
    const uint32_t bits = (mag - (3u << 7)) | ((key & 1u) << 15);  // -x_m / 8
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(__uint_as_float(bits << 16)));
    const bool plain = mag - 0x0d80u < 0x7f80u - 0x0d80u;  // 2^-100 and above, and finite
    return {plain ? bits : mag >= 0x7f80u ? 0x7fc0u : 0u, plain ? r * 0.0625f : 0.0f};
}

// min(15, floor(x / s + 8.5)) in the low bits, `inverse` being 1 / (16 s). The sum of a sixteenth, clamped to [0, 1], is off by
// 2^-23 at most; 2^-12 (in units of a code) stands against that and keeps ties above their integer, and the product with
// 16 (1 - 2^-22), added to 2^23 and rounded down, leaves the floor in the low bits, 15 for the clamped ones. Both are fma, on the pipe
// that has room: minimum, and, or, shift and permute share the other one, which bounds the kernel.
__device__ __forceinline__ uint32_t code_of(float x, float inverse)
{
    return __float_as_uint(__fmaf_rd(__saturatef(fmaf(x, inverse, (8.5f + 0x1p-12f) / 16.0f)), 16.0f - 0x1p-18f, 8388608.0f));
}

// A word of the cache: codes of four bf16 numbers in its low half, of four others in its high half.
__device__ __forceinline__ uint32_t code_word(uint2 lo, uint2 hi, float inverse_lo, float inverse_hi)
{
    const auto pair = [&](uint32_t a, uint32_t b) {
        return __byte_perm(code_of(__uint_as_float(a), inverse_lo), code_of(__uint_as_float(b), inverse_hi), 0x5410);
    };
    const uint32_t p0 = pair(lo.x << 16, hi.x << 16), p1 = pair(lo.x & 0xffff0000u, hi.x & 0xffff0000u);
    const uint32_t p2 = pair(lo.y << 16, hi.y << 16), p3 = pair(lo.y & 0xffff0000u, hi.y & 0xffff0000u);
    return ((p3 * 16u + p2) * 16u + p1) * 16u + p0;
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
    r.bh = r.in ? p.by_T.of(static_cast<int>(i)) : 0;
    r.t = r.in ? static_cast<int>(i) - r.bh * p.T : 0;
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
    const int b = p.by_H.of(r.bh), e = 8 * r.l;
    const int2 sp = span_of(p, b, r.in && r.t == 0 && threadIdx.x % (2 * (D / 8)) == 0 && r.bh == b * p.H);
    const bool live = r.in && r.t < sp.y;
    uint4 w = make_uint4(0, 0, 0, 0);
    if (live && e < p.d)
        w = *reinterpret_cast<const uint4 *>((r.side ? p.v : p.k) + ((static_cast<size_t>(r.bh) * p.T + r.t) * p.d + e) * 2);
    uint32_t top = top_keys<4>({w.x, w.y, w.z, w.w});
    top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 2));
    if (!live) return;
    const Scale s = scale_of(fold(top));
    const uint32_t code = code_word(make_uint2(w.x, w.y), make_uint2(w.z, w.w), s.inverse, s.inverse);
    const int tok = sp.x + r.t, row = tok % kv4::kBlock;
    uint8_t *blk = p.cache + (static_cast<size_t>(r.bh) * p.blocks + tok / kv4::kBlock) * kv4::block_bytes(D);
    if (r.side == 0) {
        *reinterpret_cast<uint32_t *>(blk + kv4::key_byte(D, row, e)) = code;
    } else {
        *reinterpret_cast<uint16_t *>(blk + kv4::value_byte(D, row, e)) = static_cast<uint16_t>(code);
        *reinterpret_cast<uint16_t *>(blk + kv4::value_byte(D, row, e + 4)) = static_cast<uint16_t>(code >> 16);
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
    const int b = p.by_H.of(r.bh), e = 8 * r.l;
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
constexpr int kHalf = 128;  // threads for the keys, and for the values
constexpr int kWriteCtas = 8, kReadCtas = 8;

struct BlockItem {
    int first, n;       // token of the call in the block's row 0 (may be negative), tokens of the call
    size_t row0;        // row of the call's tensors that is the block's row 0 (may wrap below the first one)
    uint8_t *blk;
};

// Blocks of a CTA: one of the larger head sizes, whose kernels are the faster without a loop.
template <int D>
__device__ __forceinline__ int run_of(const Kv4Params &p)
{
    return D < 64 ? p.run : 1;
}

// The first block of this CTA's run.
template <int D>
__device__ __forceinline__ BlockItem first_block(const Kv4Params &p)
{
    const int bh = p.by_runs.of(blockIdx.x), i = blockIdx.x - bh * p.runs, b = p.by_H.of(bh);
    const int2 sp = span_of(p, b, threadIdx.x == 0 && i == 0 && bh == b * p.H);
    const int block = sp.x / kv4::kBlock + i * run_of<D>(p);
    BlockItem it;
    it.first = block * kv4::kBlock - sp.x;
    it.n = sp.y;
    it.row0 = static_cast<size_t>(bh) * p.T + it.first;
    it.blk = p.cache + (static_cast<size_t>(bh) * p.blocks + block) * kv4::block_bytes(D);
    return it;
}

template <int D>
__device__ __forceinline__ void next_block(BlockItem &it)
{
    it.first += kv4::kBlock;
    it.row0 += kv4::kBlock;
    it.blk += kv4::block_bytes(D);
}

// ALL: every row of the block is a token of the call.
template <bool ALL>
__device__ __forceinline__ bool live(const BlockItem &it, int row)
{
    return ALL || static_cast<unsigned>(it.first + row) < static_cast<unsigned>(it.n);
}

// Pieces of a value tile: groups per lane, and 512-byte runs of lanes.
template <int D>
struct ValuePiece {
    static constexpr int kGroups = D < 64 ? 1 : 2, kRuns = D < 64 ? 1 : D / 64;
    int g, c, tile, run;

    __device__ __forceinline__ explicit ValuePiece(int i) : g(i % 32 / 4), c(i % 4), tile(i / 32 % 2), run(i / 64) {}
    __device__ __forceinline__ int row() const { return 16 * tile + 2 * c; }  // and row + 1, + 8, + 9
    static __device__ __forceinline__ constexpr int step(int z) { return 8 * (z / 2) + z % 2; }
    __device__ __forceinline__ int element() const { return 64 * run + 4 * g; }
    __device__ __forceinline__ uint8_t *in(uint8_t *blk) const { return blk + kv4::value_byte(D, row(), element()); }
};

template <int d, bool ALL>
__device__ __forceinline__ void write_keys(const Kv4Params &p, const BlockItem &it, int i)
{
    constexpr int D = kv4::padded(d), NG = D / 32;
    const int row = i / 4, c = i % 4;
    const char *src = p.k + (it.row0 + row) * (2 * d) + 16 * c;
    uint4 w[NG];
#pragma unroll
    for (int n = 0; n < NG; ++n) {
        w[n] = make_uint4(0, 0, 0, 0);
        if (live<ALL>(it, row) && (d >= 32 || 8 * c < d)) w[n] = *reinterpret_cast<const uint4 *>(src + 64 * n);
    }
    // lane c makes the scale of group c
    uint32_t code[NG], mine = 0;
#pragma unroll
    for (int n = 0; n < NG; ++n) {
        uint32_t top = top_keys<4>({w[n].x, w[n].y, w[n].z, w[n].w});
        top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 2));
        if (c == n) mine = top;
    }
    const Scale s = scale_of(fold(mine));
#pragma unroll
    for (int n = 0; n < NG; ++n) {
        const float inverse = __shfl_sync(0xffffffffu, s.inverse, n, 4);
        code[n] = code_word(make_uint2(w[n].x, w[n].y), make_uint2(w[n].z, w[n].w), inverse, inverse);
    }
    if (!live<ALL>(it, row)) return;
    uint8_t *dst = it.blk + kv4::key_byte(D, row, 8 * c);
    if constexpr (NG == 4)
        *reinterpret_cast<uint4 *>(dst) = make_uint4(code[0], code[1], code[2], code[3]);
    else if constexpr (NG == 2)
        *reinterpret_cast<uint2 *>(dst) = make_uint2(code[0], code[1]);
    else
        *reinterpret_cast<uint32_t *>(dst) = code[0];
    if (c < NG) *reinterpret_cast<uint16_t *>(it.blk + kv4::scale_byte(D, row, 0, c)) = static_cast<uint16_t>(s.bits);
}

template <int d, bool ALL>
__device__ __forceinline__ void write_values(const Kv4Params &p, const BlockItem &it, int i)
{
    constexpr int D = kv4::padded(d), NL = ValuePiece<D>::kGroups;
    const ValuePiece<D> v(i);
    if (v.run >= ValuePiece<D>::kRuns) return;  // whole warps
    const char *src = p.v + (it.row0 + v.row()) * (2 * d) + 2 * v.element();
    uint32_t code[NL][2], mine = 0;
    uint2 w[NL][4];  // of the piece's four tokens
#pragma unroll
    for (int m = 0; m < NL; ++m)
#pragma unroll
        for (int z = 0; z < 4; ++z) {
            w[m][z] = make_uint2(0, 0);
            if (live<ALL>(it, v.row() + v.step(z)) && (d >= 32 || v.element() < d))
                w[m][z] = *reinterpret_cast<const uint2 *>(src + v.step(z) * (2 * d) + 64 * m);
        }
    // largest keys of the tokens of a word; lane g makes the scale of group g / 4 and token g % 4
#pragma unroll
    for (int m = 0; m < NL; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint2 *x = w[m] + 2 * h;
            // the first token in the low halves, the second one in the high halves
            uint32_t pair = top_keys<4>({__byte_perm(x[0].x, x[1].x, 0x5410), __byte_perm(x[0].x, x[1].x, 0x7632),
                                         __byte_perm(x[0].y, x[1].y, 0x5410), __byte_perm(x[0].y, x[1].y, 0x7632)});
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) pair = __vmaxu2(pair, __shfl_xor_sync(0xffffffffu, pair, off));
            if (v.g / 2 == 2 * m + h) mine = pair;
        }
    const Scale s = scale_of(v.g % 2 ? mine >> 16 : mine & 0xffffu);
    const int own = v.row() + v.step(v.g % 4);
    if (v.g < 4 * NL && live<ALL>(it, own))
        *reinterpret_cast<uint16_t *>(it.blk + kv4::scale_byte(D, own, 1, 2 * v.run + v.g / 4)) = static_cast<uint16_t>(s.bits);
#pragma unroll
    for (int m = 0; m < NL; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int from = (4 * m + 2 * h) * 4 + v.c;
            code[m][h] = code_word(w[m][2 * h], w[m][2 * h + 1], __shfl_sync(0xffffffffu, s.inverse, from),
                                   __shfl_sync(0xffffffffu, s.inverse, from + 4));
        }
    uint8_t *dst = v.in(it.blk);
    if (live<ALL>(it, v.row()) && live<ALL>(it, v.row() + 9)) {  // and the tokens between
        if constexpr (NL == 2)
            *reinterpret_cast<uint4 *>(dst) = make_uint4(code[0][0], code[0][1], code[1][0], code[1][1]);
        else
            *reinterpret_cast<uint2 *>(dst) = make_uint2(code[0][0], code[0][1]);
    } else {
#pragma unroll
        for (int m = 0; m < NL; ++m)
#pragma unroll
            for (int z = 0; z < 4; ++z)
                if (live<ALL>(it, v.row() + v.step(z)))
                    *reinterpret_cast<uint16_t *>(dst + 8 * m + 2 * z) = static_cast<uint16_t>(code[m][z / 2] >> (16 * (z % 2)));
    }
}

template <int d>
__global__ void __launch_bounds__(2 * kHalf, kWriteCtas) kv4_write_block_kernel(const __grid_constant__ Kv4Params p)
{
    griddep_launch_dependents();
    griddep_wait();
    constexpr int D = kv4::padded(d);
    BlockItem it = first_block<D>(p);
#pragma unroll 1
    for (int k = 0; k < run_of<D>(p); ++k, next_block<D>(it)) {
        if (it.first >= it.n) return;  // no tokens of the call here (others are inside the cache)
        const bool all = it.first >= 0 && it.first + kv4::kBlock <= it.n;
        const int i = threadIdx.x % kHalf;
        if (threadIdx.x < kHalf)
            all ? write_keys<d, true>(p, it, i) : write_keys<d, false>(p, it, i);
        else
            all ? write_values<d, true>(p, it, i) : write_values<d, false>(p, it, i);
    }
}

template <int d, bool F32>
__device__ __forceinline__ void read_block(const Kv4Params &p, const BlockItem &it, int i)
{
    constexpr int D = kv4::padded(d), NG = D / 32, kSize = F32 ? 4 : 2;
    if (threadIdx.x < kHalf) {
        const int row = i / 4, c = i % 4;
        if (!live<false>(it, row) || (d < 32 && 8 * c >= d)) return;
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
        char *out = p.ko + (it.row0 + row) * (kSize * d);
#pragma unroll
        for (int n = 0; n < NG; ++n) {
            const int e = 32 * n + 8 * c;
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
        constexpr int NL = ValuePiece<D>::kGroups;
        const ValuePiece<D> v(i);
        if (v.run >= ValuePiece<D>::kRuns || (d < 32 && v.element() >= d)) return;
        uint32_t code[NL][2];
        if constexpr (NL == 2) {
            const uint4 x = *reinterpret_cast<const uint4 *>(v.in(it.blk));
            code[0][0] = x.x, code[0][1] = x.y, code[1][0] = x.z, code[1][1] = x.w;
        } else {
            const uint2 x = *reinterpret_cast<const uint2 *>(v.in(it.blk));
            code[0][0] = x.x, code[0][1] = x.y;
        }
        char *out = p.vo + (it.row0 + v.row()) * (kSize * d);
#pragma unroll
        for (int z = 0; z < 4; ++z) {
            const int row = v.row() + v.step(z);
            if (live<false>(it, row)) {
#pragma unroll
                for (int m = 0; m < NL; ++m)
                    put4<F32>(out + v.step(z) * (kSize * d), v.element() + 32 * m,
                              values4(code[m][z / 2] >> (16 * (z % 2)),
                                      bf16_at(it.blk + kv4::scale_byte(D, row, 1, 2 * v.run + m))));
            }
        }
    }
}

template <int d, bool F32>
__global__ void __launch_bounds__(2 * kHalf, kReadCtas) kv4_read_block_kernel(const __grid_constant__ Kv4Params p)
{
    griddep_launch_dependents();
    griddep_wait();
    constexpr int D = kv4::padded(d);
    BlockItem it = first_block<D>(p);
#pragma unroll 1
    for (int k = 0; k < run_of<D>(p); ++k, next_block<D>(it)) {
        if (it.first >= it.n) return;
        read_block<d, F32>(p, it, threadIdx.x % kHalf);
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

// Tokens per sequence from which a CTA takes a block and not single rows. (In us, rows / blocks, at odd rows of a cache of
// 2048 tokens, which touch two blocks: 64 x 40 heads of d = 128, 8 tokens written 7.5 / 11.7, read 7.4 / 7.6; 12 tokens
// 10.1 / 12.4 and 9.7 / 8.4; 16 tokens 12.6 / 13.1 and 12.2 / 9.2; 20 tokens 15.1 / 13.7 and 14.3 / 9.8; 24 tokens
// 17.5 / 14.4 and 16.7 / 10.6. 64 x 8 heads of d = 64: 16 tokens 2.8 / 3.2 and 2.7 / 2.5, 24 tokens 3.2 / 3.2 and 3.2 / 2.6.)
constexpr int kWriteBlocks = 20, kReadBlocks = 10;
// Blocks of a head that a CTA takes one after another where there are more than a CTA each that is resident: of d = 32 (and
// 16), where beginning a CTA costs as much as a block, 4 (8 x 32 x 8192 tokens written and read in 66 and 62 us, with one
// each in 92 and 81); of d = 64 one (8 x 32 x 4096 tokens written and read in 56.3 and 53.2 us, with two in 58.6 and 52.0).
constexpr int kRun = 4;

template <int d>
cudaError_t launch(Kv4Params &p, int op, cudaStream_t stream)
{
    constexpr int D = kv4::padded(d);
    const long long rows = static_cast<long long>(p.BH) * p.T;
    if (p.T < (op == 0 ? kWriteBlocks : kReadBlocks) && rows < (1LL << 31)) {
        constexpr int kRowsPerCta = 256 / (D / 8) / 2;
        return launch_kernel(op == 0   ? kv4_write_rows_kernel<D>
                                 : op == 1 ? kv4_read_rows_kernel<D, false>
                                           : kv4_read_rows_kernel<D, true>,
                                 dim3(static_cast<unsigned>((rows + kRowsPerCta - 1) / kRowsPerCta)), 256, 0, stream, p);
    }
    const int blocks = std::min(p.blocks, (p.T + 2 * kv4::kBlock - 2) / kv4::kBlock);
    const bool full = static_cast<long long>(p.BH) * blocks > kWriteCtas * num_sms();
    p.run = D < 64 && full ? kRun : 1;
    p.runs = (blocks + p.run - 1) / p.run;
    p.by_runs = kv4::Divisor(p.runs);
    const long long ctas = static_cast<long long>(p.BH) * p.runs;
    if (ctas > 0x7fffffffLL) return cudaErrorInvalidValue;
    return launch_kernel(op == 0   ? kv4_write_block_kernel<d>
                             : op == 1 ? kv4_read_block_kernel<d, false>
                                       : kv4_read_block_kernel<d, true>,
                             dim3(static_cast<unsigned>(ctas)), 2 * kHalf, 0, stream, p);
}

// op: 0 write, 1 read as bf16, 2 read as fp32
int run(Kv4Params p, int op, void *stream)
{
    p.status = device_status_word();
    if (!p.status) return ALIBI_ERR_CUDA;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    switch (p.d) {
        case 128: e = launch<128>(p, op, s); break;
        case 64: e = launch<64>(p, op, s); break;
        case 32: e = launch<32>(p, op, s); break;
        default: e = launch<16>(p, op, s); break;
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
    p.by_H = kv4::Divisor(H);
    p.by_T = kv4::Divisor(T);
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
