// mx_gemm.cu -- the base projection of 4-bit microscaled operands and the LoRA delta.
//
// Y[t, o] = round( sum_b 2^(ex[t,b] + ew[o,b]) sum_{i in b} cx[t,i] cw[o,i]  +  s_a H[t, :] B_a[o, :]^T )
//
// over blocks b of 32 elements, with the codes and scales of mlora_mx_quantize; H = X A_a^T
// of the unquantised X comes from the library's segmented shrink, in fp32, as in
// base_gemm.cu.  Products of codes are exact and sums are fp32 in the tensor core
// (tcgen05.mma kind::mxf4, K = 64 per instruction, two scales per row and instruction); the
// low-rank product is a second accumulator (kind::f16, s H split into bf16 hi + lo) and the
// two are added in fp32 before the one rounding.
//
// Tile kernel: 128 rows x 128 columns of Y per cluster of `ksplit` CTAs, each CTA one part
// of d_in and every ksplit-th of the tile's adapter slots.  Warp roles:
//   warp 0     TMA: per 256-wide K block the codes of X and W (128 rows x 128 bytes each,
//              128-byte swizzle) and their scale tiles (1 KB each) into a ring; after the K
//              blocks the slots' B chunks
//   warp 1     tensor memory; one thread copies a stage's scale tiles into that stage's own
//              tensor-memory columns and issues the products
//   warps 2-5  stage the slots' rows of s H, then the epilogue
// With more than one CTA each leaves its fp32 part in shared memory; after a cluster
// barrier every CTA sums a share of the columns over the cluster in CTA order.
// Every mbarrier wait is bounded; on expiry the kernel flags a timeout and stores nothing.
#include <algorithm>

#include <cuda_fp16.h>

#include "kernels.cuh"
#include "ptx.cuh"
#include "slot_operand.cuh"

namespace mlora {

namespace {

constexpr int MR = kMxTileRows;            // rows per tile
constexpr int MC = 128;                    // columns per tile
constexpr int KB = 256;                    // K per stage: 128 bytes of codes per row
constexpr int OP_BYTES = MR * KB / 2;      // 16 KB: one operand's codes of a stage
constexpr int SF_BYTES = 1024;             // one operand's scale tiles of a stage
constexpr int STAGE = 2 * OP_BYTES + 2 * SF_BYTES;
constexpr int MX_WARPS = 6;
constexpr int MT = MX_WARPS * 32;
constexpr int kMaxStages = 6;
// tensor memory: accumulator, low-rank accumulator, 16 columns of scales per stage
constexpr int T_LORA = 128, T_SCALES = 256, T_COLS = 512;
constexpr int RED_PITCH = MC + 4;          // floats per row of the reduction buffer
constexpr uint64_t kMxWaitNs = 1000000000ull;
constexpr int kRowBar = 1;

// RK: 0 without LoRA, else 16 or 64, the largest rank bucket of the pool (at least 16).
template <int RK>
struct Shape {
    static constexpr int HOP = MR * RK * 2;            // one of hi / lo
    static constexpr int GS = RK == 64 ? 4 : 6;        // ring stages
    static constexpr int ZERO = RK ? 2048 : 0;         // the zero second half of a rank-8 B chunk
    static constexpr int SMEM = 1024 + GS * STAGE + 4 * HOP + ZERO;
    static_assert(SMEM + 1024 <= 227 * 1024, "shared memory");
    static_assert(MR * RED_PITCH * 4 <= GS * STAGE, "the reduction buffer reuses the ring");
    static_assert(GS <= kMaxStages && T_SCALES + 16 * GS <= T_COLS, "tensor memory");
    static_assert(STAGE % 1024 == 0 && MC * RK * 2 <= STAGE, "stage layout");
};

struct Ctl {
    uint64_t full[kMaxStages], empty[kMaxStages];
    uint64_t done;                 // every product of the tile is in tensor memory
    uint64_t hop_full[2], hop_empty[2];
    uint32_t tmem;
    volatile int fail;
};

__device__ __forceinline__ uint8_t *align_1024(uint8_t *p)
{
    return reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(p) + 1023) & ~uintptr_t(1023));
}

__device__ __forceinline__ bool mwait(const MxGemmParams &p, Ctl &ctl, uint64_t *bar, uint32_t parity)
{
    if (ctl.fail) return false;
    if (!mbar_wait_bounded(bar, parity, kMxWaitNs)) {
        ctl.fail = 1;
        atomicOr(p.status, kFlagTimeout);
        return false;
    }
    return true;
}

// Eight columns of a row, one rounding to the output's type.
__device__ __forceinline__ void store8(const MxGemmParams &p, int row, int col, const float (&f)[8])
{
    const int64_t at = (int64_t)row * p.ldy + col;
    if (p.y_type == 2) {
        float4 *y = reinterpret_cast<float4 *>(static_cast<float *>(p.Y) + at);
        y[0] = make_float4(f[0], f[1], f[2], f[3]);
        y[1] = make_float4(f[4], f[5], f[6], f[7]);
        return;
    }
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (p.y_type == 1) {
            const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        } else {
            w[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
        }
    }
    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.Y) + at) = make_uint4(w[0], w[1], w[2], w[3]);
}

}  // namespace

template <int RK>
__global__ void __launch_bounds__(MT, 1) mx_gemm_kernel(const __grid_constant__ MxGemmParams p)
{
    using S = Shape<RK>;
    constexpr int GS = S::GS, HOP = S::HOP;
    extern __shared__ __align__(128) uint8_t smem_raw[];
    __shared__ Ctl ctl;
    uint8_t *ring = align_1024(smem_raw);
    uint8_t *hop = ring + GS * STAGE;              // [2][hi, lo]
    uint8_t *zero = hop + 4 * HOP;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int ksplit = (int)cluster_size(), crank = (int)cluster_rank();
    const int tile = (int)blockIdx.x / ksplit;
    const int mb = tile % p.n_mblk, nb = tile / p.n_mblk;
    const int m0 = mb * MR, n0 = nb * MC;

    if (warp == 1) {
        tmem_alloc(&ctl.tmem, T_COLS);
        tmem_relinquish();
    }
    if (tid == 0) {
        for (int s = 0; s < GS; ++s) {
            mbar_init(&ctl.full[s], 1);
            mbar_init(&ctl.empty[s], 1);
        }
        mbar_init(&ctl.done, 1);
        for (int b = 0; b < 2; ++b) {
            mbar_init(&ctl.hop_full[b], 1);
            mbar_init(&ctl.hop_empty[b], 1);
        }
        fence_mbar_init();
        ctl.fail = 0;
    }
    if (RK > 0) {
        for (int i = tid; i < S::ZERO / 16; i += MT) reinterpret_cast<uint4 *>(zero)[i] = make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ctl.tmem;
    // this CTA's K blocks and adapter slots
    const int nkb = (p.d_in + KB - 1) / KB;
    const int kb0 = nkb * crank / ksplit, kb1 = nkb * (crank + 1) / ksplit;
    const int32_t *bs = RK ? p.block_slots + (int64_t)mb * kBlockSlotsPitch : nullptr;
    const int cnt = RK ? bs[0] : 0;

    if (warp == 0) {
        if (lane == 0) {
            uint32_t g = 0;
            for (int kb = kb0; kb < kb1; ++kb, ++g) {
                const int s = (int)(g % GS);
                if (g >= GS && !mwait(p, ctl, &ctl.empty[s], ((g / GS) - 1) & 1u)) break;
                uint8_t *st = ring + s * STAGE;
                mbar_arrive_expect_tx(&ctl.full[s], STAGE);
                tma_load_2d(st, &p.x_map, kb * (KB / 2), m0, &ctl.full[s]);
                tma_load_2d(st + OP_BYTES, &p.w_map, kb * (KB / 2), n0, &ctl.full[s]);
                bulk_load(st + 2 * OP_BYTES, p.x_scales + ((int64_t)mb * nkb + kb) * SF_BYTES, SF_BYTES, &ctl.full[s]);
                bulk_load(st + 2 * OP_BYTES + SF_BYTES, p.w_scales + ((int64_t)nb * nkb + kb) * SF_BYTES, SF_BYTES,
                          &ctl.full[s]);
            }
            for (int j = crank; j < cnt && !ctl.fail; j += ksplit, ++g) {
                const int slot = bs[1 + 2 * j], R = bs[2 + 2 * j];
                const int s = (int)(g % GS);
                if (g >= GS && !mwait(p, ctl, &ctl.empty[s], ((g / GS) - 1) & 1u)) break;
                // columns past d_out read as zeros
                mbar_arrive_expect_tx(&ctl.full[s], (uint32_t)R * MC * 2);
                tma_load_4d(ring + s * STAGE, &p.b_map[bucket_index(R)], 0, n0 / p.b_col_div, 0, slot, &ctl.full[s]);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        if (lane == 0) {
            uint32_t g = 0, hc = 0;
            bool ok = true;
            for (int kb = kb0; kb < kb1; ++kb, ++g) {
                const int s = (int)(g % GS);
                if (!mwait(p, ctl, &ctl.full[s], (g / GS) & 1u)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t xs = smem_addr(ring + s * STAGE), ws = xs + OP_BYTES, sf = xs + 2 * OP_BYTES;
                // the stage's own scale columns: their last readers finished before the stage was refilled
                const uint32_t sx = tmem + T_SCALES + 16 * s, sw = sx + 8;
                tmem_copy_scales(sx, sf);
                tmem_copy_scales(sx + 4, sf + 512);
                tmem_copy_scales(sw, sf + SF_BYTES);
                tmem_copy_scales(sw + 4, sf + SF_BYTES + 512);
                const int steps = min(4, (p.d_in - kb * KB + 63) / 64);
                for (int k = 0; k < steps; ++k)
                    umma_mxf4(tmem, umma_desc_sw128(xs + 32 * k), umma_desc_sw128(ws + 32 * k),
                              umma_idesc_mxf4(MR, MC, (k & 1) * 2, (k & 1) * 2), sx + 4 * (k >> 1), sw + 4 * (k >> 1),
                              kb > kb0 || k > 0 ? 1u : 0u);
                umma_commit(&ctl.empty[s]);
            }
            if (RK > 0 && ok) {
                const uint32_t idesc = umma_idesc_bf16(MR, MC);
                for (int j = crank; j < cnt; j += ksplit, ++g, ++hc) {
                    const int R = bs[2 + 2 * j];
                    const int s = (int)(g % GS), hb = (int)(hc & 1);
                    if (!mwait(p, ctl, &ctl.hop_full[hb], (hc >> 1) & 1u) || !mwait(p, ctl, &ctl.full[s], (g / GS) & 1u)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t a_hi = smem_addr(hop + hb * 2 * HOP), a_lo = a_hi + HOP;
                    const uint32_t b_s = smem_addr(ring + s * STAGE);
                    for (int st = 0; st < (R < 16 ? 16 : R) / 16; ++st) {
                        const uint32_t b0 = b_s + st * 2 * MC * 16;
                        // bucket 8: the second rank group of B is the zero block
                        const uint32_t lbo = R == 8 ? smem_addr(zero) - b0 : MC * 16;
                        const uint64_t bd = umma_desc_kmajor(b0, lbo, 128);
                        const uint32_t koff = st * 2 * (MR / 8) * 128;
                        umma_bf16(tmem + T_LORA, umma_desc_kmajor(a_hi + koff, (MR / 8) * 128, 128), bd, idesc,
                                  hc > 0 || st > 0 ? 1u : 0u);
                        umma_bf16(tmem + T_LORA, umma_desc_kmajor(a_lo + koff, (MR / 8) * 128, 128), bd, idesc, 1u);
                    }
                    umma_commit(&ctl.empty[s]);
                    umma_commit(&ctl.hop_empty[hb]);
                }
            }
            if (ok) umma_commit(&ctl.done);
        }
        __syncwarp();
    } else {
        const int r = tid - 64, quarter = warp & 3;
        bool alive = true;
        if constexpr (RK > 0) {
            // operand row r: this row's s H for one slot after the other (zeros for other slots' rows)
            const int row = m0 + r;
            int4 info = make_int4(-1, -1, 0, 0);
            if (cnt > 0 && row < p.n_rows) info = p.row_info[row];
            uint32_t hc = 0;
            for (int j = crank; j < cnt; j += ksplit, ++hc) {
                const int slot = bs[1 + 2 * j], R = bs[2 + 2 * j], hb = (int)(hc & 1);
                if (hc >= 2 && !named_sync_and(kRowBar, 128, mwait(p, ctl, &ctl.hop_empty[hb], ((hc >> 1) - 1) & 1u))) {
                    alive = false;
                    break;
                }
                const bool mine = info.x >= 0 && info.y == slot;
                const int rank = mine ? info.w : 0;
                const float sc = mine ? __int_as_float(info.z) : 0.f;
                const float *hsrc = p.H + (int64_t)(mine ? info.x : 0) * p.ldh;
                uint8_t *hi = hop + hb * 2 * HOP;
                if constexpr (RK == 16) {
                    stage_operand<16>(hi, hi + HOP, hsrc, rank, sc, r);
                } else {
                    if (R <= 16) stage_operand<16>(hi, hi + HOP, hsrc, rank, sc, r);
                    else if (R == 32) stage_operand<32>(hi, hi + HOP, hsrc, rank, sc, r);
                    else stage_operand<64>(hi, hi + HOP, hsrc, rank, sc, r);
                }
                fence_proxy_async_smem();
                named_sync(kRowBar, 128);
                if (r == 0) mbar_arrive(&ctl.hop_full[hb]);
            }
        }
        alive = named_sync_and(kRowBar, 128, alive && mwait(p, ctl, &ctl.done, 0));
        if (alive) {
            tc_fence_after();
            const int row = m0 + 32 * quarter + lane;
            const uint32_t tb = tmem + ((uint32_t)(32 * quarter) << 16);
            const bool lora = RK > 0 && cnt > crank;   // this CTA had a slot
            float *red = reinterpret_cast<float *>(ring) + (32 * quarter + lane) * RED_PITCH;
            for (int c = 0; c < MC; c += 32) {
                uint32_t v[32];
                tmem_ld32(tb + c, v);
                tmem_wait_ld();
                if (lora) {
                    uint32_t w[32];
                    tmem_ld32(tb + T_LORA + c, w);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) + __uint_as_float(w[i]));
                }
                if (row >= p.n_rows) continue;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float f[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(v[8 * q + i]);
                    if (ksplit > 1) {
                        reinterpret_cast<float4 *>(red + c + 8 * q)[0] = make_float4(f[0], f[1], f[2], f[3]);
                        reinterpret_cast<float4 *>(red + c + 8 * q)[1] = make_float4(f[4], f[5], f[6], f[7]);
                    } else if (n0 + c + 8 * q < p.d_out) {   // d_out is a multiple of 8
                        store8(p, row, n0 + c + 8 * q, f);
                    }
                }
            }
        }
    }

    if (ksplit > 1) {
        cluster_arrive_release();
        cluster_wait_acquire();
        // this CTA's share of the columns, summed over the cluster in CTA order
        int bad = 0;
        for (int c = 0; c < ksplit; ++c)
            bad |= __float_as_int(ld_dsmem_f32(map_to_rank(smem_addr((const void *)&ctl.fail), (uint32_t)c)));
        const int rows = min(MR, p.n_rows - m0), share = MC / ksplit / 8;   // 8-column groups
        for (int i = tid; i < rows * share && !bad; i += MT) {
            const int r = i / share, col = (crank * share + i % share) * 8;
            if (n0 + col >= p.d_out) continue;
            const uint32_t at = smem_addr(reinterpret_cast<float *>(ring) + r * RED_PITCH + col);
            float f[8] = {};
            for (int c = 0; c < ksplit; ++c) {
                const uint32_t src = map_to_rank(at, (uint32_t)c);
                const float4 a = ld_dsmem_f32x4(src), b = ld_dsmem_f32x4(src + 16);
                f[0] += a.x, f[1] += a.y, f[2] += a.z, f[3] += a.w;
                f[4] += b.x, f[5] += b.y, f[6] += b.z, f[7] += b.w;
            }
            store8(p, m0 + r, n0 + col, f);
        }
        cluster_arrive_release();
        cluster_wait_acquire();
    }
    __syncthreads();
    if (ctl.fail && tid == 0) {   // let copies in flight land
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < 2000000ull) {
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, T_COLS);
}

namespace {

template <int RK>
cudaError_t launch_tile(const MxGemmParams &p, int ksplit, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3((unsigned)(p.n_mblk * p.n_nblk * ksplit), 1, 1);
    cfg.blockDim = dim3(MT, 1, 1);
    cfg.dynamicSmemBytes = Shape<RK>::SMEM;
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)ksplit;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, mx_gemm_kernel<RK>, p);
}

template <int RK>
cudaError_t prepare_tile()
{
    cudaError_t e = cudaFuncSetAttribute(mx_gemm_kernel<RK>, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape<RK>::SMEM);
    if (e != cudaSuccess) return e;
    return cudaFuncSetAttribute(mx_gemm_kernel<RK>, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
}

}  // namespace

cudaError_t launch_mx_gemm(const MxGemmParams &p, int rank_bucket_max, cudaStream_t stream)
{
    // CTAs per tile: waves of resident CTAs (one per SM) times K blocks per CTA, plus what a
    // part costs beside its K blocks.
    const int nkb = (p.d_in + KB - 1) / KB;
    const int64_t tiles = (int64_t)p.n_mblk * p.n_nblk;
    int best = 1;
    int64_t best_cost = INT64_MAX;
    for (int ks = 1; ks <= 8 && ks <= nkb; ks *= 2) {
        const int64_t waves = (tiles * ks + 147) / 148;
        const int64_t cost = waves * ((nkb + ks - 1) / ks + 4) + (ks > 1 ? 2 : 0);
        if (cost < best_cost) {
            best_cost = cost;
            best = ks;
        }
    }
    if (rank_bucket_max == 0) return launch_tile<0>(p, best, stream);
    if (rank_bucket_max <= 16) return launch_tile<16>(p, best, stream);
    return launch_tile<64>(p, best, stream);
}

cudaError_t prepare_mx_gemm()
{
    cudaError_t e;
    if ((e = prepare_tile<0>()) != cudaSuccess) return e;
    if ((e = prepare_tile<16>()) != cudaSuccess) return e;
    return prepare_tile<64>();
}

}  // namespace mlora
