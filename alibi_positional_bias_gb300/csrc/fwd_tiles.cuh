// Tiles, shared-memory layout and register split of the tensor-core prefills (over dense tensors and over pages).
#pragma once

#include <cstdint>

namespace alibi {
namespace {

constexpr int BM = 128;  // query rows per tile (MMA M)
constexpr int BN = 128;  // keys per tile
constexpr int kThreads = 384;
constexpr int kKStages = 2;
constexpr int kVStages = 2;
constexpr uint32_t kTmemCols = 512;
constexpr float kRescaleThreshold = 8.0f;  // log2 units
// Register split: the kernel launches with kLaunchRegs per thread (384 threads,
// one CTA per SM); the producer/MMA warpgroup gives registers back and the two
// softmax warpgroups take them. The shares add up exactly to the launch total.
constexpr uint32_t kLaunchRegs = 168;
constexpr uint32_t kRegsLow = 88;    // warps 0-3
constexpr uint32_t kRegsHigh = 208;  // warps 4-11
static_assert(128 * kRegsLow + 256 * kRegsHigh == kThreads * kLaunchRegs, "register split must match launch");

template <int D>
struct Cfg {
    static constexpr int kChunks = D / 64;                 // 128-byte swizzle atoms along d
    static constexpr uint32_t kChunkBytes = BM * 128;      // one 64-column box: 16 KB
    static constexpr uint32_t kTileBytes = BM * D * 2;     // one 128 x D bf16 tile
    static constexpr uint32_t kQ = 0;                      // 2 Q tiles
    static constexpr uint32_t kK = 2 * kTileBytes;         // K tiles of the two ring stages
    static constexpr uint32_t kV = kK + kKStages * kTileBytes;  // V tiles of the two ring stages
    // One 128 x 64 swizzle atom of bias operands: ones (K-step 0, the A side), the
    // column bias m log2(e) c / c1 for the two items in flight (K-steps 1, 2, the B
    // side), and minus ones (K-step 3, the A side that turns the same column bias
    // into -m log2(e) c / c1 for keys after the rows, non-causal).
    static constexpr uint32_t kAux = kV + kVStages * kTileBytes;
    // Epilogue staging: 2 KB per softmax warp, one 32 x 32 bf16 box of O at a time.
    static constexpr uint32_t kStage = kAux + kChunkBytes;
    static constexpr uint32_t kBar = kStage + kChunkBytes;
    static constexpr uint32_t kSmem = kBar + 256 + 1024;   // barriers, TMEM slot, alignment slack
};

__device__ __forceinline__ float max3f(float a, float b, float c)
{
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Max of 128 values as 8 independent chains of three-input max (short dependency chains).
__device__ __forceinline__ float row_max128(const float (&x)[128])
{
    float m[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        m[k] = x[k];
#pragma unroll
        for (int t = 1; t + 1 < 16; t += 2) m[k] = max3f(m[k], x[k + 8 * t], x[k + 8 * (t + 1)]);
        m[k] = fmaxf(m[k], x[k + 8 * 15]);
    }
    return fmaxf(max3f(m[0], m[1], m[2]), max3f(max3f(m[3], m[4], m[5]), m[6], m[7]));
}

}  // namespace
}  // namespace alibi
