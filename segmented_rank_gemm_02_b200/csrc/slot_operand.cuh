// slot_operand.cuh -- the low-rank A operand of the GEMMs that add LoRA products in the
// tensor core (base_gemm.cu, mx_gemm.cu).
#pragma once

#include "ptx.cuh"

namespace mlora {

constexpr int kOperandRows = 128;   // rows of one operand (one tensor-memory lane each)

// Index of a rank bucket (8, 16, 32, 64) among a pool's TMA views.
__device__ __forceinline__ int bucket_index(int R) { return R <= 8 ? 0 : R <= 16 ? 1 : R <= 32 ? 2 : 3; }

// One row of the LoRA operand: s * H[row, 0:rank) (zeros past rank, all zeros for
// rank 0) as bf16 hi + lo parts in the K-major no-swizzle layout [RK/8][16][8][8].
// The row's loads are all issued before any is used.
template <int RK>
__device__ __forceinline__ void stage_operand(uint8_t *hi, uint8_t *lo, const float *hsrc, int rank, float sc, int r)
{
    float h[RK];
    if (rank == RK) {
#pragma unroll
        for (int i = 0; i < RK / 4; ++i) {
            const float4 v = reinterpret_cast<const float4 *>(hsrc)[i];
            h[4 * i] = v.x;
            h[4 * i + 1] = v.y;
            h[4 * i + 2] = v.z;
            h[4 * i + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int c = 0; c < RK; ++c) h[c] = c < rank ? hsrc[c] : 0.f;
    }
#pragma unroll
    for (int cg = 0; cg < RK / 8; ++cg) {
        uint4 vh, vl;
        uint32_t *ph = reinterpret_cast<uint32_t *>(&vh);
        uint32_t *pl = reinterpret_cast<uint32_t *>(&vl);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            float h0, l0, h1, l1;
            split_bf16(sc * h[8 * cg + 2 * c], h0, l0);
            split_bf16(sc * h[8 * cg + 2 * c + 1], h1, l1);
            ph[c] = pack_bf16x2(h0, h1);
            pl[c] = pack_bf16x2(l0, l1);
        }
        const int off = (cg * (kOperandRows / 8) + r / 8) * 128 + (r % 8) * 16;
        *reinterpret_cast<uint4 *>(hi + off) = vh;
        *reinterpret_cast<uint4 *>(lo + off) = vl;
    }
}

}  // namespace mlora
