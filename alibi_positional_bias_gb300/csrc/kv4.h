// Layout of the 4-bit KV cache: which byte of a block holds which element. Plain
// C++ (host and device), shared by the kernels and a CPU test.
//
// A block holds 32 tokens of one head, keys and values: 36 D bytes with D =
// max(d, 32) (d = 16 is stored with 16 zero elements). Each row of D elements is cut
// into groups of 32 consecutive elements with one bf16 scale s and a 4-bit code u per
// element standing for s (u - 8). The order of the codes is the order in which the
// lanes of a warp need them as operands of mma.m16n8k16 (one 4-byte word is four
// half-register pairs), so that the decode reads a tile of 16 tokens with whole
// 16-byte shared-memory loads and unpacks it with masks alone:
//   keys    lane 4 g + c holds rows g and g + 8 of a tile, and of every group n the 8
//           consecutive elements from 8 c: a row's D/2 bytes are [c][n][4 bytes];
//   values  lane 4 g + c holds rows 2c, 2c + 1 (low and high half of a word) and 2c + 8,
//           2c + 9 (the next word) of a tile, and of every group the 4 consecutive
//           elements from 4 g: a tile's 8 D bytes are [n / 2][lane][n % 2][word][half].
// A byte holds an even element in its low four bits and the next one in its high
// ones, always of one token, so tokens are written without reading their neighbours.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define KV4_HD __host__ __device__ __forceinline__
#else
#define KV4_HD inline
#endif

namespace alibi {
namespace kv4 {

constexpr int kBlock = 32;  // tokens per block
constexpr int kGroup = 32;  // elements per scale
constexpr int kTile = 16;   // tokens per tile (the rows of one mma)

KV4_HD constexpr int padded(int d) { return d < kGroup ? kGroup : d; }
KV4_HD constexpr int block_bytes(int D) { return 36 * D; }

// Byte of key element e (even) of row r.
KV4_HD constexpr int key_byte(int D, int r, int e)
{
    return r * (D / 2) + (e % 32 / 8) * (D / 8) + 4 * (e / 32) + e % 8 / 2;
}

// Byte of value element e (even) of row r.
KV4_HD constexpr int value_byte(int D, int r, int e)
{
    const int n = e / 32, g = e % 32 / 4, c = r % 8 / 2;
    const int lane_bytes = D < 64 ? 8 : 16;
    return 16 * D + 8 * D * (r / kTile) + 512 * (n / 2) + (4 * g + c) * lane_bytes + 8 * (n % 2) +
           4 * (r % kTile / 8) + 2 * (r % 2) + e % 4 / 2;
}

// Byte of the bf16 scale of group n of row r, keys (0) or values (1).
KV4_HD constexpr int scale_byte(int D, int r, int values, int n)
{
    return 32 * D + r * (D / 8) + (values * (D / 32) + n) * 2;
}

}  // namespace kv4
}  // namespace alibi
