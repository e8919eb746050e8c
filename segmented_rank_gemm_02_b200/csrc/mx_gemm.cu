// mx_gemm.cu -- the base projection of 4-bit microscaled operands and the LoRA delta.
//
// Y[t, o] = round( sum_b 2^(ex[t,b] + ew[o,b]) sum_{i in b} cx[t,i] cw[o,i]  +  s_a H[t, :] B_a[o, :]^T )
//
// over blocks b of 32 elements, with the codes and scales of mlora_mx_quantize; H = X A_a^T
// of the unquantised X comes from the library's segmented shrink, in fp32, as in
// base_gemm.cu.  Products of codes are exact and sums are fp32 in the tensor core
// (tcgen05.mma kind::mxf4, K = 64 per instruction, two scales per row and instruction); the
// low-rank products (kind::f16, s H split into bf16 hi + lo) are added in fp32 before the one
// rounding.
//
// Two kernels.  Few rows are bound by the bytes of W and by latency: mx_tile_kernel, 128 x 128
// tiles with d_in split over a cluster, so that all SMs stream W.  Many rows are bound by the
// tensor core and the copies that feed it: mx_pair_kernel, 256 x 256 or 256 x 384 tiles
// on pairs of CTAs.
// Every mbarrier wait is bounded; on expiry a kernel flags a timeout and stores nothing.
#include <algorithm>
#include <mutex>

#include <cuda_fp16.h>

#include "kernels.cuh"
#include "ptx.cuh"
#include "slot_operand.cuh"

namespace mlora {

namespace {

constexpr int MR = kMxTileRows;            // rows per CTA (one tensor-memory lane each)
constexpr int KB = 256;                    // K per stage: 128 bytes of codes per row
constexpr int OP_BYTES = 128 * KB / 2;     // 16 KB: the codes of 128 rows, one stage
constexpr int SF_BYTES = 1024;             // their scale tiles (two of 512 bytes)
constexpr uint64_t kMxWaitNs = 1000000000ull;
constexpr int kRowBar = 1;                 // named barrier of the operand warps
constexpr int kEpiBar = 2;                 // named barrier of the epilogue warps (pair kernel)

__device__ __forceinline__ uint8_t *align_1024(uint8_t *p)
{
    return reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(p) + 1023) & ~uintptr_t(1023));
}

// Two values as the 16-bit output type.
template <int YT>
__device__ __forceinline__ uint32_t pack2(float a, float b)
{
    if constexpr (YT == 1) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    } else {
        return pack_bf16x2(a, b);
    }
}

// Eight columns of a row, one rounding to the output's type.
template <int YT>
__device__ __forceinline__ void store8(const MxGemmParams &p, int row, int col, const float (&f)[8])
{
    const int64_t at = (int64_t)row * p.ldy + col;
    if constexpr (YT == 2) {
        float4 *y = reinterpret_cast<float4 *>(static_cast<float *>(p.Y) + at);
        y[0] = make_float4(f[0], f[1], f[2], f[3]);
        y[1] = make_float4(f[4], f[5], f[6], f[7]);
    } else {
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.Y) + at) =
            make_uint4(pack2<YT>(f[0], f[1]), pack2<YT>(f[2], f[3]), pack2<YT>(f[4], f[5]), pack2<YT>(f[6], f[7]));
    }
}

__device__ __forceinline__ void store8(const MxGemmParams &p, int row, int col, const float (&f)[8])
{
    if (p.y_type == 2) store8<2>(p, row, col, f);
    else if (p.y_type == 1) store8<1>(p, row, col, f);
    else store8<0>(p, row, col, f);
}

// 8 x 8 transpose of 16-byte pieces across groups of eight lanes: lane k of a group ends up with
// piece k of the group's eight rows, so that a store instruction writes whole 128-byte lines.
__device__ __forceinline__ void transpose8(uint4 (&a)[8], int k)
{
#pragma unroll
    for (int sh = 4; sh >= 1; sh >>= 1) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (j & sh) continue;
            const bool upper = (k & sh) != 0;
            const uint4 send = upper ? a[j] : a[j | sh];
            uint4 recv;
            recv.x = __shfl_xor_sync(0xffffffffu, send.x, sh);
            recv.y = __shfl_xor_sync(0xffffffffu, send.y, sh);
            recv.z = __shfl_xor_sync(0xffffffffu, send.z, sh);
            recv.w = __shfl_xor_sync(0xffffffffu, send.w, sh);
            if (upper) a[j] = recv;
            else a[j | sh] = recv;
        }
    }
}

// 64 fp32 columns of this lane's row, rounded to 16 bits: eight 16-byte pieces.
template <int YT>
__device__ __forceinline__ void round64(const uint32_t (&v)[2][32], uint4 (&a)[8])
{
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i] = pack2<YT>(__uint_as_float(v[c][8 * q + 2 * i]), __uint_as_float(v[c][8 * q + 2 * i + 1]));
            a[4 * c + q] = make_uint4(w[0], w[1], w[2], w[3]);
        }
}

__device__ __forceinline__ void put64(const MxGemmParams &p, uint4 (&a)[8], int row0, int n0, int k)
{
    transpose8(a, k);
    const int col = n0 + 8 * k;
    if (col >= p.d_out) return;   // d_out is a multiple of 8
    uint16_t *y = static_cast<uint16_t *>(p.Y) + col;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (row0 + j < p.n_rows) *reinterpret_cast<uint4 *>(y + (int64_t)(row0 + j) * p.ldy) = a[j];
}

}  // namespace

// ------------------------------------------------------------------ few rows
// 128 rows x 128 columns of Y per cluster of `ksplit` CTAs, each CTA one part of d_in and every
// ksplit-th of the tile's adapter slots.  Warp roles:
//   warp 0     TMA: per 256-wide K block the codes of X and W (128 rows x 128 bytes each,
//              128-byte swizzle) and their scale tiles (1 KB each) into a ring; after the K
//              blocks the slots' B chunks
//   warp 1     tensor memory; one thread copies a stage's scale tiles into that stage's own
//              tensor-memory columns and issues the products; the low-rank products have an
//              accumulator of their own
//   warps 2-5  find the tile's rows in the segments and its distinct slots (while the K blocks
//              stream: no launch of its own), stage the rows' s H, then the epilogue
// The low-rank operand is every row's own s H; the products of one slot's B write the lanes of
// that slot's rows alone (the others are masked), so that it is staged once however many slots.
// With more than one CTA each leaves its fp32 part in shared memory; after a cluster
// barrier every CTA sums a share of the columns over the cluster in CTA order.
namespace {

constexpr int MC = 128;                    // columns per tile
constexpr int STAGE = 2 * OP_BYTES + 2 * SF_BYTES;
constexpr int MT = 6 * 32;
constexpr int kMaxStages = 6;
// tensor memory: accumulator, low-rank accumulator, 16 columns of scales per stage
constexpr int T_LORA = 128, T_SCALES = 256, T_COLS = 512;
constexpr int RED_PITCH = MC + 4;          // floats per row of the reduction buffer

// RK: 0 without LoRA, else 16 or 64, the largest rank bucket of the pool (at least 16).
template <int RK>
struct TileShape {
    static constexpr int HOP = MR * RK * 2;            // one of hi / lo
    static constexpr int GS = RK == 64 ? 5 : 6;        // ring stages
    static constexpr int ZERO = RK ? 2048 : 0;         // the zero second half of a rank-8 B chunk
    static constexpr int B_BYTES = MC * RK * 2;        // a slot's chunk of B
    static constexpr int SLOTS = RK ? STAGE / B_BYTES : 1;   // slots per ring stage
    static constexpr int SMEM = 1024 + GS * STAGE + 2 * HOP + ZERO;
    static_assert(SMEM + 6144 <= 227 * 1024, "shared memory");   // and TileCtl
    static_assert(MR * RED_PITCH * 4 <= GS * STAGE, "the reduction buffer reuses the ring");
    static_assert(GS <= kMaxStages && T_SCALES + 16 * GS <= T_COLS, "tensor memory");
    static_assert(STAGE % 1024 == 0 && SLOTS >= 1, "stage layout");
};

struct TileCtl {
    uint64_t full[kMaxStages], empty[kMaxStages];
    uint64_t done;                 // every product of the tile is in tensor memory
    uint64_t staged;               // the rows' s H are in place, the low-rank accumulator is zero
    uint64_t listed;               // the slot list is complete
    uint32_t tmem;
    volatile int fail;
    int count;                     // distinct slots of the tile's rows, and their
    alignas(16) int slot[MR];      // numbers,
    int bucket[MR];                // rank buckets
    uint32_t others[MR][4];        // and, a bit each, the rows of other slots
    int pos[MR];                   // each row's grouped position (-1: none)
    alignas(16) int row_slot[MR];  // and slot
    int part[4];
};

// Bounded wait; the flag of one that ran out is looked at only while waiting.
__device__ __forceinline__ bool mwait(const MxGemmParams &p, TileCtl &ctl, uint64_t *bar, uint32_t parity)
{
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = global_timer_ns();
    for (;;) {
        for (int i = 0; i < 32; ++i)
            if (mbar_try_wait(bar, parity)) return true;
        if (ctl.fail) return false;
        if (global_timer_ns() - t0 > kMxWaitNs) break;
    }
    ctl.fail = 1;
    atomicOr(p.status, kFlagTimeout);
    return false;
}

// The operand warps' 128 threads: row r's grouped position, slot, scale and rank (position -1:
// base only), and the distinct slots of the tile in order of first appearance.  The first CTA
// of the launch reports the segments' and rows' problems, as row_map_kernel does.
// records: shared memory for the segments' copy, free until this returns.
__device__ int4 find_rows(const TileParams &t, TileCtl &ctl, int4 *records, int capacity, int m0, int r, bool reporter)
{
    const int lane = r & 31, warp = r >> 5;
    ctl.pos[r] = -1;
    const SegmentTable segments = copy_segments(t, records, capacity, r, 128, reporter);
    named_sync(kRowBar, 128);
    claim_rows(t, segments, m0, MR, ctl.pos, r, 128, reporter);
    named_sync(kRowBar, 128);
    int4 info = make_int4(-1, -1, 0, 0);
    if (ctl.pos[r] >= 0) info = row_of_position(t, segments, ctl.pos[r]);
    ctl.row_slot[r] = info.y;
    named_sync(kRowBar, 128);
    const bool first = first_with_slot(ctl.row_slot, r, info.y);
    const unsigned m = __ballot_sync(0xffffffffu, first);
    if (lane == 0) ctl.part[warp] = __popc(m);
    named_sync(kRowBar, 128);
    int before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        before += w < warp ? ctl.part[w] : 0;
        total += ctl.part[w];
    }
    if (first) {
        const int i = before + __popc(m & ((1u << lane) - 1u));
        ctl.slot[i] = info.y;
        ctl.bucket[i] = rank_bucket(info.w);
    }
    if (r == 0) ctl.count = total;
#pragma unroll
    for (int i = 0; i < 4; ++i) ctl.others[r][i] = 0xffffffffu;
    named_sync(kRowBar, 128);
    if (info.x >= 0) atomicAnd(&ctl.others[slot_index(ctl.slot, total, info.y)][warp], ~(1u << lane));
    named_sync(kRowBar, 128);
    return info;
}

}  // namespace

template <int RK>
__global__ void __launch_bounds__(MT, 1)
    mx_tile_kernel(const __grid_constant__ MxGemmParams p, const __grid_constant__ MxSegments sg)
{
    using S = TileShape<RK>;
    constexpr int GS = S::GS, HOP = S::HOP;
    static_assert(sizeof(TileCtl) <= 6144, "shared memory");
    extern __shared__ __align__(128) uint8_t smem_raw[];
    __shared__ TileCtl ctl;
    uint8_t *ring = align_1024(smem_raw);
    uint8_t *hop = ring + GS * STAGE;              // s H: hi, lo
    uint8_t *zero = hop + 2 * HOP;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int ksplit = (int)cluster_size(), crank = (int)cluster_rank();
    const int tile = (int)blockIdx.x / ksplit;
    const int mb = tile % p.n_mblk, nb = tile / p.n_mblk;
    const int m0 = mb * MR, n0 = nb * MC;

    if (warp == 1) {
        tmem_alloc(&ctl.tmem, T_COLS);
        tmem_relinquish();
    }
    if (tid < 4) prefetch_map(tid == 0 ? &p.w_map : tid == 1 ? &p.x_map : tid == 2 ? &p.ws_map : &p.xs_map);
    // (the maps past the pool's largest bucket are not encoded)
    if (RK > 0 && tid >= 4 && tid < 8 && 8 << (tid - 4) <= p.rank_bucket_max) prefetch_map(&p.b_map[tid - 4]);
    if (tid == 0) {
        for (int s = 0; s < GS; ++s) {
            mbar_init(&ctl.full[s], 1);
            mbar_init(&ctl.empty[s], 1);
        }
        mbar_init(&ctl.done, 1);
        mbar_init(&ctl.staged, 1);
        mbar_init(&ctl.listed, 1);
        fence_mbar_init();
        ctl.fail = 0;
        ctl.count = 0;
    }
    if (RK > 0) {
        for (int i = tid; i < S::ZERO / 16; i += MT) reinterpret_cast<uint4 *>(zero)[i] = make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // this CTA's K blocks and adapter slots
    const int nkb = (p.d_in + KB - 1) / KB;
    const int kb0 = nkb * crank / ksplit, kb1 = nkb * (crank + 1) / ksplit;
    griddep_wait();   // from here on: what earlier kernels wrote
    const uint32_t tmem = ctl.tmem;

    if (warp == 0) {
        // (the whole warp walks the stages, one lane issues: see warp 1)
        const bool issuer = elect_one();
        uint32_t g = 0;
        bool ok = true;
        for (int kb = kb0; kb < kb1; ++kb, ++g) {
            const int s = (int)(g % GS);
            ok = g < GS || __all_sync(0xffffffffu, mwait(p, ctl, &ctl.empty[s], ((g / GS) - 1) & 1u));
            if (!ok) break;
            if (issuer) {
                uint8_t *st = ring + s * STAGE;
                mbar_arrive_expect_tx(&ctl.full[s], STAGE);
                tma_load_2d(st + OP_BYTES, &p.w_map, kb * (KB / 2), n0, &ctl.full[s]);
                tma_load_2d(st, &p.x_map, kb * (KB / 2), m0, &ctl.full[s]);
                tma_load_2d(st + 2 * OP_BYTES, &p.xs_map, kb * 256, mb, &ctl.full[s]);
                tma_load_2d(st + 2 * OP_BYTES + SF_BYTES, &p.ws_map, kb * 256, nb, &ctl.full[s]);
            }
            __syncwarp();
        }
        if (RK > 0 && ok && __all_sync(0xffffffffu, mwait(p, ctl, &ctl.listed, 0))) {
            const int mine = (ctl.count - crank + ksplit - 1) / ksplit;   // slots crank, + ksplit, ...
            for (int i0 = 0; i0 < mine; i0 += S::SLOTS, ++g) {
                const int s = (int)(g % GS), n = min(S::SLOTS, mine - i0);
                if (g >= GS && !__all_sync(0xffffffffu, mwait(p, ctl, &ctl.empty[s], ((g / GS) - 1) & 1u))) break;
                if (issuer) {
                    int ranks = 0;
                    for (int i = 0; i < n; ++i) ranks += ctl.bucket[crank + (i0 + i) * ksplit];
                    // columns past d_out read as zeros
                    mbar_arrive_expect_tx(&ctl.full[s], (uint32_t)ranks * MC * 2);
                    for (int i = 0; i < n; ++i) {
                        const int j = crank + (i0 + i) * ksplit;
                        tma_load_4d(ring + s * STAGE + i * S::B_BYTES, &p.b_map[bucket_index(ctl.bucket[j])], 0,
                                    n0 / p.b_col_div, 0, ctl.slot[j], &ctl.full[s]);
                    }
                }
                __syncwarp();
            }
        }
    } else if (warp == 1) {
        // The whole warp walks the stages, one lane of it issues: the descriptors then live in uniform
        // registers, where the products take them from.  (A lone lane spent about 110 cycles a
        // product on moving them there: a K block took 0.66 us instead of 0.33.)
        const bool issuer = elect_one();
        const uint64_t x0 = umma_desc_sw128(smem_addr(ring));
        uint32_t g = 0;
        bool ok = true;
        for (int kb = kb0; kb < kb1; ++kb, ++g) {
            const int s = (int)(g % GS);
            if (!__all_sync(0xffffffffu, mwait(p, ctl, &ctl.full[s], (g / GS) & 1u))) {
                ok = false;
                break;
            }
            tc_fence_after();
            const uint64_t xd = x0 + (uint32_t)s * (STAGE >> 4), wd = xd + (OP_BYTES >> 4);
            const uint32_t sf = smem_addr(ring) + (uint32_t)s * STAGE + 2 * OP_BYTES;
            // the stage's own scale columns: their last readers finished before the stage was refilled
            const uint32_t sx = tmem + T_SCALES + 16 * s, sw = sx + 8;
            const int steps = min(4, (p.d_in - kb * KB + 63) / 64);
            if (issuer) {
                tmem_copy_scales<1>(sx, sf);
                tmem_copy_scales<1>(sx + 4, sf + 512);
                tmem_copy_scales<1>(sw, sf + SF_BYTES);
                tmem_copy_scales<1>(sw + 4, sf + SF_BYTES + 512);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (k < steps)
                        umma_mxf4<1>(tmem, xd + 2 * k, wd + 2 * k, umma_idesc_mxf4(MR, MC, (k & 1) * 2, (k & 1) * 2),
                                     sx + 4 * (k >> 1), sw + 4 * (k >> 1), kb > kb0 || k > 0 ? 1u : 0u);
                umma_commit(&ctl.empty[s]);
            }
            __syncwarp();
        }
        if (RK > 0 && ok) ok = __all_sync(0xffffffffu, mwait(p, ctl, &ctl.listed, 0));
        if (RK > 0 && ok && ctl.count > crank) {
            ok = __all_sync(0xffffffffu, mwait(p, ctl, &ctl.staged, 0));
            constexpr uint32_t idesc = umma_idesc_bf16(MR, MC);
            const int mine = (ctl.count - crank + ksplit - 1) / ksplit;
            const uint32_t a_hi = smem_addr(hop);
            for (int i0 = 0; i0 < mine && ok; i0 += S::SLOTS, ++g) {
                const int s = (int)(g % GS), n = min(S::SLOTS, mine - i0);
                ok = __all_sync(0xffffffffu, mwait(p, ctl, &ctl.full[s], (g / GS) & 1u));
                if (!ok) break;
                tc_fence_after();
                const uint64_t ah = umma_desc_kmajor(a_hi, (MR / 8) * 128, 128), al = ah + (HOP >> 4);
                const uint64_t b_s = umma_desc_kmajor(smem_addr(ring) + (uint32_t)s * STAGE, MC * 16, 128);
                for (int i = 0; i < n; ++i) {
                    const int j = crank + (i0 + i) * ksplit, R = ctl.bucket[j];
                    const uint4 others = *reinterpret_cast<const uint4 *>(ctl.others[j]);
                    uint64_t bd = b_s + (uint32_t)i * (S::B_BYTES >> 4);
                    // bucket 8: the second rank group of B is the zero block
                    if (R == 8) {
                        const uint32_t b0 = smem_addr(ring) + (uint32_t)(s * STAGE + i * S::B_BYTES);
                        bd = umma_desc_kmajor(b0, smem_addr(zero) - b0, 128);
                    }
                    if (issuer) {
#pragma unroll
                        for (int st = 0; st < RK / 16; ++st) {
                            if (16 * st >= R) break;
                            umma_bf16_rows(tmem + T_LORA, ah + st * (2 * (MR / 8) * 128 >> 4), bd + st * (2 * MC), idesc,
                                           others);
                            umma_bf16_rows(tmem + T_LORA, al + st * (2 * (MR / 8) * 128 >> 4), bd + st * (2 * MC), idesc,
                                           others);
                        }
                    }
                    __syncwarp();
                }
                if (issuer) umma_commit(&ctl.empty[s]);
                __syncwarp();
            }
        }
        if (ok && issuer) umma_commit(&ctl.done);
        __syncwarp();
    } else {
        const int r = tid - 64, quarter = warp & 3;
        bool lora = false;
        if constexpr (RK > 0) {
            const int4 info = find_rows(sg.t, ctl, reinterpret_cast<int4 *>(hop), 2 * HOP / 16, m0, r, blockIdx.x == 0);
            if (r == 0) mbar_arrive(&ctl.listed);
            lora = ctl.count > crank;   // this CTA has a slot
            if (lora) {
                if (info.x >= 0) {
                    RowOperand<RK, 1> op;
                    op.load(sg.H + (int64_t)info.x * sg.ldh, info.w, __int_as_float(info.z), 0);
                    op.store(hop, r, 0);
                }
                // the low-rank accumulator starts at zero: no product writes all of its rows
                const uint32_t none[8] = {};
                for (int c = 0; c < MC; c += 8)
                    tmem_st8(tmem + ((uint32_t)(32 * quarter) << 16) + T_LORA + c, none);
                tmem_wait_st();
                tc_fence_before();
                fence_proxy_async_smem();
                named_sync(kRowBar, 128);
                if (r == 0) mbar_arrive(&ctl.staged);
            }
        }
        const bool alive = named_sync_and(kRowBar, 128, mwait(p, ctl, &ctl.done, 0));
        if (alive) {
            tc_fence_after();
            const int row = m0 + 32 * quarter + lane;
            const uint32_t tb = tmem + ((uint32_t)(32 * quarter) << 16);
            float *red = reinterpret_cast<float *>(ring) + (32 * quarter + lane) * RED_PITCH;
            const bool any = m0 + 32 * quarter < p.n_rows;   // a row of this warp exists
            const int k = lane & 7, row0 = row - lane + 8 * (lane >> 3);
            for (int c = 0; c < MC && any; c += 64) {
                uint32_t v[2][32];
                tmem_ld32(tb + c, v[0]);
                tmem_ld32(tb + c + 32, v[1]);
                if (lora) {
                    uint32_t w[2][32];
                    tmem_ld32(tb + T_LORA + c, w[0]);
                    tmem_ld32(tb + T_LORA + c + 32, w[1]);
                    tmem_wait_ld32(w[0]);
                    tmem_wait_ld32(w[1]);
                    tmem_wait_ld32(v[0]);
                    tmem_wait_ld32(v[1]);
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        v[0][i] = __float_as_uint(__uint_as_float(v[0][i]) + __uint_as_float(w[0][i]));
                        v[1][i] = __float_as_uint(__uint_as_float(v[1][i]) + __uint_as_float(w[1][i]));
                    }
                } else {
                    tmem_wait_ld32(v[0]);
                    tmem_wait_ld32(v[1]);
                }
                if (ksplit == 1 && p.y_type != 2) {
                    uint4 a[8];
                    if (p.y_type == 1) round64<1>(v, a);
                    else round64<0>(v, a);
                    put64(p, a, row0, n0 + c, k);
                } else if (row < p.n_rows) {
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        float f[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(v[q >> 2][8 * (q & 3) + i]);
                        if (ksplit > 1) {
                            reinterpret_cast<float4 *>(red + c + 8 * q)[0] = make_float4(f[0], f[1], f[2], f[3]);
                            reinterpret_cast<float4 *>(red + c + 8 * q)[1] = make_float4(f[4], f[5], f[6], f[7]);
                        } else if (n0 + c + 8 * q < p.d_out) {   // d_out is a multiple of 8
                            store8<2>(p, row, n0 + c + 8 * q, f);
                        }
                    }
                }
            }
        }
    }

    if (ksplit > 1) {
        cluster_arrive_release();
        cluster_wait_acquire();
        // this CTA's share of the columns, summed over the cluster in CTA order (all loads first)
        int bad = 0;
#pragma unroll
        for (int c = 0; c < 8; ++c)
            if (c < ksplit)
                bad |= __float_as_int(ld_dsmem_f32(map_to_rank(smem_addr((const void *)&ctl.fail), (uint32_t)c)));
        const int rows = min(MR, p.n_rows - m0), share = MC / ksplit / 8;   // 8-column groups
        for (int i = tid; i < rows * share; i += MT) {
            const int r = i / share, col = (crank * share + i % share) * 8;
            if (n0 + col >= p.d_out) continue;
            const uint32_t at = smem_addr(reinterpret_cast<float *>(ring) + r * RED_PITCH + col);
            float4 a[8], b[8];
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                if (c >= ksplit) break;
                const uint32_t src = map_to_rank(at, (uint32_t)c);
                a[c] = ld_dsmem_f32x4(src);
                b[c] = ld_dsmem_f32x4(src + 16);
            }
            float f[8] = {};
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                if (c >= ksplit) break;
                f[0] += a[c].x, f[1] += a[c].y, f[2] += a[c].z, f[3] += a[c].w;
                f[4] += b[c].x, f[5] += b[c].y, f[6] += b[c].z, f[7] += b[c].w;
            }
            if (!bad) store8(p, m0 + r, n0 + col, f);
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

// ------------------------------------------------------------------ many rows
// Persistent tiles of 256 rows x (NSUB x UN) columns on pairs of CTAs (a cluster of two on
// neighbouring SMs) with tcgen05.mma.cta_group::2: CTA c holds rows [128 c, +128) of the tile's X,
// half of the W rows of each sub-tile, and 128 rows of the fp32 accumulator.  The accumulator and
// the stages' scales fill tensor memory, so there is no second accumulator: the epilogue takes
// the tile out in one go, as 16-bit values in the registers of eight warps, hands it back and
// stores while the next tile's products run.
//   warp 0     TMA of both CTAs' codes onto the even one's barriers, as in base_gemm.cu
//   warp 2     the scales likewise: one box of X's and one of W's a stage
//   warp 1     even CTA: copies a stage's scales into that stage's own columns of tensor memory
//              and issues the pair's products; after the K blocks it waits for them before the
//              low-rank products, whose instruction kind differs, continue the same accumulator
//   warps 4-11 stage the rows' s H, the tile's slots and their rows' masks while the K blocks run,
//              then the epilogue: quarter = warp % 4 of the rows, half = (warp - 4) / 4 of the
//              ranks and of the columns
namespace {

constexpr int PT = 12 * 32;
constexpr int P_COLS = 512;
constexpr uint16_t kPairMask = 0x3;
constexpr int kGroupRows = 8;              // row blocks per group of tiles (see tile_at)
constexpr int kPairStages = 6;             // most ring stages of any shape

template <int RK, int NSUB>
struct PairShape {
    static constexpr int UN = NSUB == 1 ? 256 : 192;   // columns per product
    static constexpr int PN = NSUB * UN;               // columns per tile
    static constexpr int PH = UN / 2;                  // W rows (and B columns) per CTA and sub-tile
    static constexpr int W_BYTES = PH * KB / 2;        // a sub-tile's, a multiple of 1 KB
    static constexpr int NSF = 1 + PN / 128;           // scale blocks (128 rows each) of a stage
    static constexpr int SF_COLS = 8 * NSF;            // their columns of tensor memory
    static constexpr int STAGE = OP_BYTES + NSUB * W_BYTES + (NSF * SF_BYTES + 1023) / 1024 * 1024;
    static constexpr int HOP = MR * RK * 2;
    static constexpr int GS = NSUB == 2 ? 4 : RK ? 5 : 6;   // ring stages
    static constexpr int ZERO = RK ? 2048 : 0;
    static constexpr int B_BYTES = NSUB * PH * RK * 2; // a slot's chunk of B
    static constexpr int SLOTS = RK ? STAGE / B_BYTES : 1;   // slots per ring stage
    static constexpr int SMEM = 1024 + GS * STAGE + 2 * HOP + ZERO;
    static_assert(PN + SF_COLS * GS <= P_COLS && GS <= kPairStages, "tensor memory");
    static_assert(STAGE % 1024 == 0 && SLOTS >= 1, "stage layout");
};

struct PairCtl {
    // Ring stages, counted alike by all who use them (K blocks and slots' B chunks):
    uint64_t full[kPairStages];    // the copies have landed
    uint64_t empty[kPairStages];   // the products are done
    uint64_t acc_full, acc_empty;
    uint64_t k_done;               // the K blocks' products are complete
    uint64_t listed;               // the tile's slots are in this CTA's list,
    uint64_t staged;               // the rows' s H in both CTAs' shared memory
    uint32_t tmem;
    volatile int fail;
    alignas(16) int slot[2 * MR];  // a tile's distinct slots, their
    int bucket[2 * MR];            // rank buckets,
    uint32_t others[2 * MR][8];    // and, a bit each, the rows of other slots (the issuing CTA's)
};

// Bounded wait.  The flag of a wait that ran out, here or in the pair's other CTA (which is
// told), is looked at only while waiting: a satisfied wait costs one test.
__device__ __forceinline__ bool pwait(const MxGemmParams &p, PairCtl &ctl, uint64_t *bar, uint32_t parity)
{
    if (mbar_try_wait_cluster(bar, parity)) return true;
    const uint64_t t0 = global_timer_ns();
    for (;;) {
        for (int i = 0; i < 32; ++i)
            if (mbar_try_wait_cluster(bar, parity)) return true;
        if (ctl.fail) return false;
        if (global_timer_ns() - t0 > kMxWaitNs) break;
    }
    ctl.fail = 1;
    st_cluster_u32(map_to_rank(smem_addr((const void *)&ctl.fail), cluster_rank() ^ 1u), 1u);
    atomicOr(p.status, kFlagTimeout);
    return false;
}

// Tiles run in groups of kGroupRows row blocks, column-major inside a group, so that the pairs
// working at the same time share a few row blocks of X and column blocks of W in L2.
__device__ __forceinline__ void tile_at(const MxGemmParams &p, int t, int &mb, int &nb)
{
    const int per_group = kGroupRows * p.n_nblk;
    const int first_mb = (t / per_group) * kGroupRows;
    const int rows = min(kGroupRows, p.n_mblk - first_mb);
    const int local = t % per_group;
    mb = first_mb + local % rows;
    nb = local / rows;
}

// Distinct slots of a row block.
template <int RK>
__device__ __forceinline__ int slot_count(const MxSlots &sl, int mb)
{
    return RK > 0 ? sl.block_slots[(int64_t)mb * kBlockSlotsPitch] : 0;
}

__device__ __forceinline__ uint32_t leader_bar(const uint64_t *bar) { return map_to_rank(smem_addr(bar), 0); }

}  // namespace

// YT: 0 bf16, 1 fp16, 2 fp32 (an fp32 tile does not fit the epilogue's registers: it is stored
// from tensor memory chunk by chunk, and the accumulator handed back after the last).
template <int RK, int NSUB, int YT>
__global__ void __launch_bounds__(PT, 1)
    mx_pair_kernel(const __grid_constant__ MxGemmParams p, const __grid_constant__ MxSlots sl)
{
    using S = PairShape<RK, NSUB>;
    constexpr int GS = S::GS, HOP = S::HOP, UN = S::UN, PN = S::PN, PH = S::PH, SLOTS = S::SLOTS;
    static_assert(S::SMEM + sizeof(PairCtl) <= 227 * 1024, "shared memory");
    constexpr int SF_AT = OP_BYTES + NSUB * S::W_BYTES;   // scales in a stage: X's block, then W's
    extern __shared__ __align__(128) uint8_t smem_raw[];
    __shared__ PairCtl ctl;
    uint8_t *ring = align_1024(smem_raw);
    uint8_t *hop = ring + GS * S::STAGE;           // s H: hi, lo
    uint8_t *zero = hop + 2 * HOP;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int crank = (int)cluster_rank();         // 0 issues the pair's products
    const bool leader = crank == 0;
    const int n_clusters = (int)(gridDim.x / 2), first = (int)cluster_index();

    if (warp == 1) {
        tmem_alloc_pair(&ctl.tmem, P_COLS);
        tmem_relinquish_pair();
    }
    if (tid < 4) prefetch_map(tid == 0 ? &p.w_map : tid == 1 ? &p.x_map : tid == 2 ? &p.ws_map : &p.xs_map);
    if (tid == 0) {
        for (int s = 0; s < GS; ++s) {
            mbar_init(&ctl.full[s], 2);            // codes, scales
            mbar_init(&ctl.empty[s], 1);
        }
        mbar_init(&ctl.acc_full, 1);
        mbar_init(&ctl.acc_empty, 16);             // eight epilogue warps in each CTA
        mbar_init(&ctl.k_done, 1);
        mbar_init(&ctl.listed, 1);
        mbar_init(&ctl.staged, 2);                 // one arrival per CTA
        fence_mbar_init();
        ctl.fail = 0;
    }
    if (RK > 0) {
        for (int i = tid; i < S::ZERO / 16; i += PT) reinterpret_cast<uint4 *>(zero)[i] = make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();
    }
    tc_fence_before();
    __syncthreads();
    cluster_arrive_release();   // both CTAs' barriers exist before either signals the other's
    cluster_wait_acquire();
    tc_fence_after();
    // After a long-segment shrink only the operand warps wait for the grids before this one: that
    // shrink follows a plainly launched kernel, so all but H is complete when this one starts.
    if (!sl.early || warp >= 4) griddep_wait();
    const uint32_t tmem = ctl.tmem;
    const int n_tiles = p.n_mblk * p.n_nblk;
    const int nkb = (p.d_in + KB - 1) / KB;

    // Ring stages are counted by g: a tile's K blocks, then its slots' B chunks, SLOTS to a stage.
    // The warps that issue walk them whole, one lane issues: see mx_tile_kernel.
    if (warp == 0) {
        const bool issuer = elect_one();
        uint32_t g = 0, lc = 0;
        bool ok = true;
        for (int t = first; t < n_tiles && ok; t += n_clusters) {
            int mb, nb;
            tile_at(p, t, mb, nb);
            const int count = slot_count<RK>(sl, mb);   // (used after the K blocks)
            const int m0 = (2 * mb + crank) * MR, nc = nb * PN + PH * crank;
            for (int kb = 0; kb < nkb; ++kb, ++g) {
                const int s = (int)(g % GS);
                ok = g < GS || __all_sync(0xffffffffu, pwait(p, ctl, &ctl.empty[s], ((g / GS) - 1) & 1u));
                if (!ok) break;
                if (issuer) {
                    uint8_t *st = ring + s * S::STAGE;
                    if (leader) mbar_arrive_expect_tx(&ctl.full[s], 2u * SF_AT);
                    const uint32_t fb = leader_bar(&ctl.full[s]);
                    // rows past the end read as zeros
                    tma_load_2d_pair(st, &p.x_map, kb * (KB / 2), m0, fb);
#pragma unroll
                    for (int u = 0; u < NSUB; ++u)
                        tma_load_2d_pair(st + OP_BYTES + u * S::W_BYTES, &p.w_map, kb * (KB / 2), nc + u * UN, fb);
                }
                __syncwarp();
            }
            if (RK > 0 && ok && count > 0) {
                ok = __all_sync(0xffffffffu, pwait(p, ctl, &ctl.listed, lc++ & 1u));
                for (int i0 = 0; i0 < count && ok; i0 += SLOTS, ++g) {
                    const int s = (int)(g % GS), n = min(SLOTS, count - i0);
                    ok = g < GS || __all_sync(0xffffffffu, pwait(p, ctl, &ctl.empty[s], ((g / GS) - 1) & 1u));
                    if (!ok) break;
                    if (issuer) {
                        int ranks = 0;
                        for (int i = 0; i < n; ++i) ranks += ctl.bucket[i0 + i];
                        // columns past d_out read as zeros
                        if (leader) mbar_arrive_expect_tx(&ctl.full[s], 2u * NSUB * (uint32_t)ranks * PH * 2);
                        const uint32_t fb = leader_bar(&ctl.full[s]);
                        for (int i = 0; i < n; ++i)
#pragma unroll
                            for (int u = 0; u < NSUB; ++u)
                                tma_load_4d_pair(ring + s * S::STAGE + i * S::B_BYTES + u * PH * RK * 2,
                                                 &p.b_map[bucket_index(ctl.bucket[i0 + i])], 0,
                                                 (nc + u * UN) / p.b_col_div, 0, ctl.slot[i0 + i], fb);
                    }
                    __syncwarp();
                }
            }
        }
    } else if (warp == 2) {
        const bool issuer = elect_one();
        uint32_t g = 0;
        bool ok = true;
        for (int t = first; t < n_tiles && ok; t += n_clusters) {
            int mb, nb;
            tile_at(p, t, mb, nb);
            const int stages = nkb + (slot_count<RK>(sl, mb) + SLOTS - 1) / SLOTS;
            for (int kb = 0; kb < stages; ++kb, ++g) {
                const int s = (int)(g % GS);
                // (B chunks too: a waiter that skipped phases could not tell them apart by parity)
                ok = g < GS || __all_sync(0xffffffffu, pwait(p, ctl, &ctl.empty[s], ((g / GS) - 1) & 1u));
                if (!ok) break;
                if (issuer) {
                    if (kb >= nkb) {
                        if (leader) mbar_arrive(&ctl.full[s]);
                    } else {
                        // blocks past the last read as zeros
                        uint8_t *st = ring + s * S::STAGE + SF_AT;
                        if (leader) mbar_arrive_expect_tx(&ctl.full[s], 2u * S::NSF * SF_BYTES);
                        const uint32_t fb = leader_bar(&ctl.full[s]);
                        tma_load_2d_pair(st, &p.xs_map, kb * 256, 2 * mb + crank, fb);
                        tma_load_2d_pair(st + SF_BYTES, &p.ws_map, kb * 256, nb * (PN / 128), fb);
                    }
                }
                __syncwarp();
            }
        }
    } else if (warp == 1) {
        if (leader) {
            const bool issuer = elect_one();
            const uint64_t x0 = umma_desc_sw128(smem_addr(ring));
            uint32_t g = 0, tc = 0, lc = 0;
            bool ok = true, ready = false;   // ready: the next stage was full when last looked at
            for (int t = first; t < n_tiles && ok; t += n_clusters, ++tc) {
                int mb, nb;
                tile_at(p, t, mb, nb);
                const int count = slot_count<RK>(sl, mb);
                // the first stage is waited for before the accumulator, which comes later
                if (!ready) ready = __all_sync(0xffffffffu, pwait(p, ctl, &ctl.full[g % GS], (g / GS) & 1u));
                if (!ready || (tc > 0 && !__all_sync(0xffffffffu, pwait(p, ctl, &ctl.acc_empty, (tc - 1) & 1u)))) break;
                for (int kb = 0; kb < nkb; ++kb, ++g) {
                    const int s = (int)(g % GS);
                    if (!ready && !__all_sync(0xffffffffu, pwait(p, ctl, &ctl.full[s], (g / GS) & 1u))) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t xd = x0 + (uint32_t)s * (S::STAGE >> 4);   // (the address field, in 16 bytes)
                    const uint64_t wd = xd + (OP_BYTES >> 4);
                    // per 128 of K: X's four columns of scales, then W's (32 rows a column).  The stage's own:
                    // their last readers finished before it was refilled
                    const uint32_t sf = tmem + PN + S::SF_COLS * s;
                    const uint32_t sm = smem_addr(ring) + (uint32_t)s * S::STAGE + SF_AT;
                    const int steps = min(4, (p.d_in - kb * KB + 63) / 64);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t sx = sf + h * 4 * S::NSF, sw = sx + 4;
                        if (issuer) {
#pragma unroll
                            for (int i = 0; i < S::NSF; ++i)
                                tmem_copy_scales<2>(sx + 4 * i, sm + i * SF_BYTES + h * 512);
#pragma unroll
                            for (int k = 2 * h; k < 2 * h + 2; ++k) {
                                if (k >= steps) continue;
#pragma unroll
                                for (int u = 0; u < NSUB; ++u)
                                    umma_mxf4<2>(tmem + u * UN, xd + 2 * k, wd + u * (S::W_BYTES >> 4) + 2 * k,
                                                 umma_idesc_mxf4(2 * MR, UN, (k & 1) * 2, (k & 1) * 2), sx,
                                                 sw + u * UN / 32, kb > 0 || k > 0 ? 1u : 0u);
                            }
                        }
                        __syncwarp();
                        // a look at the next stage's barrier, while products are queued
                        if (h == 0)
                            ready = __all_sync(0xffffffffu, mbar_test_wait_cluster(&ctl.full[(g + 1) % GS],
                                                                                   ((g + 1) / GS) & 1u));
                    }
                    if (issuer) umma_commit_pair(&ctl.empty[s], kPairMask);
                    __syncwarp();
                }
                if (RK > 0 && ok && count > 0) {
                    if (issuer) umma_commit_pair(&ctl.k_done, kPairMask);
                    __syncwarp();
                    ready = false;
                    ok = __all_sync(0xffffffffu, pwait(p, ctl, &ctl.staged, lc & 1u) &&
                                                     pwait(p, ctl, &ctl.listed, lc & 1u) &&
                                                     pwait(p, ctl, &ctl.k_done, lc & 1u));
                    ++lc;
                    constexpr uint32_t idesc = umma_idesc_bf16(2 * MR, UN);
                    const uint32_t a_hi = smem_addr(hop);
                    for (int i0 = 0; i0 < count && ok; i0 += SLOTS, ++g) {
                        const int s = (int)(g % GS), n = min(SLOTS, count - i0);
                        ok = __all_sync(0xffffffffu, pwait(p, ctl, &ctl.full[s], (g / GS) & 1u));
                        if (!ok) break;
                        tc_fence_after();
                        const uint64_t ah = umma_desc_kmajor(a_hi, (MR / 8) * 128, 128), al = ah + (HOP >> 4);
                        const uint64_t b_s = umma_desc_kmajor(smem_addr(ring) + (uint32_t)s * S::STAGE, PH * 16, 128);
                        for (int i = 0; i < n; ++i) {
                            const int R = ctl.bucket[i0 + i];
                            const uint4 *others = reinterpret_cast<const uint4 *>(ctl.others[i0 + i]);
                            const uint4 o0 = others[0], o1 = others[1];
#pragma unroll
                            for (int u = 0; u < NSUB; ++u) {
                                uint64_t bd = b_s + (uint32_t)i * (S::B_BYTES >> 4) + u * (PH * RK * 2 >> 4);
                                // bucket 8: the second rank group of B is the zero block
                                if (R == 8) {
                                    const uint32_t b0 =
                                        smem_addr(ring) + (uint32_t)(s * S::STAGE + i * S::B_BYTES + u * PH * RK * 2);
                                    bd = umma_desc_kmajor(b0, smem_addr(zero) - b0, 128);
                                }
                                if (issuer) {
#pragma unroll
                                    for (int st = 0; st < RK / 16; ++st) {
                                        if (16 * st >= R) break;
                                        umma_bf16_rows_pair(tmem + u * UN, ah + st * (2 * (MR / 8) * 128 >> 4),
                                                            bd + st * (2 * PH), idesc, o0, o1);
                                        umma_bf16_rows_pair(tmem + u * UN, al + st * (2 * (MR / 8) * 128 >> 4),
                                                            bd + st * (2 * PH), idesc, o0, o1);
                                    }
                                }
                                __syncwarp();
                            }
                        }
                        if (issuer) umma_commit_pair(&ctl.empty[s], kPairMask);
                        __syncwarp();
                    }
                }
                if (ok && issuer) umma_commit_pair(&ctl.acc_full, kPairMask);
                __syncwarp();
            }
        }
        __syncwarp();
    } else if (warp >= 4) {
        const int quarter = warp & 3, half = (warp - 4) >> 2;
        const uint32_t empty_bar = leader_bar(&ctl.acc_empty);
        const uint32_t staged_bar = leader_bar(&ctl.staged);
        const int r = 32 * quarter + lane, k = lane & 7;
        constexpr int HC = PN / 2;                 // columns per thread
        uint32_t tc = 0;
        for (int t = first; t < n_tiles; t += n_clusters, ++tc) {
            int mb, nb;
            tile_at(p, t, mb, nb);
            const int row = (2 * mb + crank) * MR + r;
            const int count = slot_count<RK>(sl, mb);
            if constexpr (RK > 0) {
                if (count > 0) {
                    // This tile's operand, while its K blocks run (the last tile's products are done): this
                    // row, half of the ranks; and the list, an entry per thread.
                    const int i = tid - 128;
                    int4 info = make_int4(-1, -1, 0, 0);
                    if (row < p.n_rows) info = sl.row_info[row];
                    int its_slot = -1;   // of the block's row i
                    if (leader && 2 * mb * MR + i < p.n_rows) {
                        const int4 v = sl.row_info[2 * mb * MR + i];
                        if (v.x >= 0) its_slot = v.y;
                    }
                    if (i < count) {
                        const int32_t *entry = sl.block_slots + (int64_t)mb * kBlockSlotsPitch + 1 + 2 * i;
                        ctl.slot[i] = entry[0];
                        ctl.bucket[i] = entry[1];
                        uint4 *o = reinterpret_cast<uint4 *>(ctl.others[i]);
                        o[0] = o[1] = make_uint4(0xffffffffu, 0xffffffffu, 0xffffffffu, 0xffffffffu);
                    }
                    if (info.x >= 0) {
                        RowOperand<RK, 2> op;
                        op.load(sl.H + (int64_t)info.x * sl.ldh, info.w, __int_as_float(info.z), half);
                        op.store(hop, r, half);
                    }
                    fence_proxy_async_smem();
                    named_sync(kEpiBar, 256);
                    if (its_slot >= 0) atomicAnd(&ctl.others[slot_index(ctl.slot, count, its_slot)][i >> 5], ~(1u << (i & 31)));
                    named_sync(kEpiBar, 256);
                    if (i == 0) {
                        mbar_arrive(&ctl.listed);
                        mbar_arrive_cluster(staged_bar);
                    }
                }
            }
            if (!named_sync_and(kEpiBar, 256, pwait(p, ctl, &ctl.acc_full, tc & 1u))) break;
            tc_fence_after();
            const int n0 = nb * PN + HC * half;
            const int row0 = row - lane + 8 * (lane >> 3);
            const uint32_t tb = tmem + ((uint32_t)(32 * quarter) << 16) + HC * half;
            if constexpr (YT == 2) {
                for (int c = 0; c < HC; c += 32) {
                    uint32_t v[32];
                    tmem_ld32(tb + c, v);
                    tmem_wait_ld();
                    if (c == HC - 32) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_cluster(empty_bar);
                    }
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        float f[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(v[8 * q + i]);
                        if (row < p.n_rows && n0 + c + 8 * q < p.d_out) store8<2>(p, row, n0 + c + 8 * q, f);
                    }
                }
            } else {
                uint4 a[HC / 64][8];
                // each piece's loads run while the one before is rounded; the accumulator goes back
                // before the last piece is
                uint32_t v[2][2][32];
                tmem_ld32(tb, v[0][0]);
                tmem_ld32(tb + 32, v[0][1]);
#pragma unroll
                for (int h = 0; h < HC / 64; ++h) {
                    tmem_wait_ld32(v[h & 1][0]);
                    tmem_wait_ld32(v[h & 1][1]);
                    if (h + 1 < HC / 64) {
                        tmem_ld32(tb + 64 * (h + 1), v[(h + 1) & 1][0]);
                        tmem_ld32(tb + 64 * (h + 1) + 32, v[(h + 1) & 1][1]);
                    } else {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_cluster(empty_bar);
                    }
                    round64<YT>(v[h & 1], a[h]);
                }
#pragma unroll
                for (int h = 0; h < HC / 64; ++h) put64(p, a[h], row0, n0 + 64 * h, k);
            }
        }
    }

    // leave: tensor-core work done, copies landed, neither CTA still signals the other
    __syncthreads();
    if (ctl.fail && tid == 0) {
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < 2000000ull) {
        }
    }
    tc_fence_before();
    __syncthreads();
    cluster_arrive_release();
    cluster_wait_acquire();
    tc_fence_after();
    if (warp == 1) tmem_dealloc_pair(tmem, P_COLS);
}

// ------------------------------------------------------------------ launches
namespace {

cudaLaunchConfig_t config(unsigned ctas, unsigned threads, size_t smem, unsigned cluster, cudaStream_t stream,
                          cudaLaunchAttribute (&attr)[2])
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas, 1, 1);
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cfg;
}

template <int RK>
cudaError_t launch_tile(const MxGemmParams &p, const MxSegments &sg, int ksplit, cudaStream_t stream)
{
    cudaLaunchAttribute attr[2];
    const cudaLaunchConfig_t cfg =
        config((unsigned)(p.n_mblk * p.n_nblk * ksplit), MT, TileShape<RK>::SMEM, (unsigned)ksplit, stream, attr);
    return cudaLaunchKernelEx(&cfg, mx_tile_kernel<RK>, p, sg);
}

template <typename K>
cudaError_t allow_smem(K kernel, int bytes)
{
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    return cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
}

template <int RK, int NSUB>
cudaError_t prepare_pair()
{
    constexpr int smem = PairShape<RK, NSUB>::SMEM;
    cudaError_t e;
    if ((e = allow_smem(mx_pair_kernel<RK, NSUB, 0>, smem)) != cudaSuccess) return e;
    if ((e = allow_smem(mx_pair_kernel<RK, NSUB, 1>, smem)) != cudaSuccess) return e;
    return allow_smem(mx_pair_kernel<RK, NSUB, 2>, smem);
}

template <int RK>
cudaError_t prepare_rank()
{
    cudaError_t e;
    if ((e = allow_smem(mx_tile_kernel<RK>, TileShape<RK>::SMEM)) != cudaSuccess) return e;
    if ((e = prepare_pair<RK, 1>()) != cudaSuccess) return e;
    return prepare_pair<RK, 2>();
}

// Pairs resident at once on the current device (cached per device; every variant takes whole SMs).
cudaError_t active_pairs(int &active)
{
    static std::mutex mu;
    static int cached[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(mu);
    if (cached[dev] == 0) {
        cudaLaunchAttribute attr[2];
        cudaLaunchConfig_t cfg = config(2, PT, PairShape<0, 1>::SMEM, 2, nullptr, attr);
        cfg.numAttrs = 1;
        int n = 0;
        cudaError_t e = cudaOccupancyMaxActiveClusters(&n, mx_pair_kernel<0, 1, 0>, &cfg);
        if (e != cudaSuccess) return e;
        if (n <= 0) return cudaErrorInvalidConfiguration;
        cached[dev] = n;
    }
    active = cached[dev];
    return cudaSuccess;
}

template <int RK, int NSUB>
cudaError_t launch_pair_shape(const MxGemmParams &p, const MxSlots &sl, unsigned pairs, cudaStream_t stream)
{
    cudaLaunchAttribute attr[2];
    const cudaLaunchConfig_t cfg = config(2 * pairs, PT, PairShape<RK, NSUB>::SMEM, 2, stream, attr);
    if (p.y_type == 0) return cudaLaunchKernelEx(&cfg, mx_pair_kernel<RK, NSUB, 0>, p, sl);
    if (p.y_type == 1) return cudaLaunchKernelEx(&cfg, mx_pair_kernel<RK, NSUB, 1>, p, sl);
    return cudaLaunchKernelEx(&cfg, mx_pair_kernel<RK, NSUB, 2>, p, sl);
}

template <int RK>
cudaError_t launch_pair(const MxGemmParams &p, const MxSlots &sl, int cols, unsigned pairs, cudaStream_t stream)
{
    return cols == 256 ? launch_pair_shape<RK, 1>(p, sl, pairs, stream) : launch_pair_shape<RK, 2>(p, sl, pairs, stream);
}

}  // namespace

static int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// With adapters every CTA of the few-rows form walks the whole list of grouped positions, so its time
// grows with their square; the many-rows form has them looked up once.  Whole calls with adapters, few-rows
// against pair tiles, in us: 64 -> 64, 8192 rows 26 / 26, 16384 34 / 30, 60000 245 / 61; 512 -> 128
// 28 / 28, 36 / 32, 280 / 90; 4096 -> 128 38 / 40, 71 / 61, 382 / 167.
constexpr int kTileTokens = 8192;

MxPlan plan_mx_gemm(int n_rows, int d_in, int d_out, int n_tokens)
{
    // Each form's time in us, as measured on a B200 with 148 SMs (shapes of 1 to 4096 rows, d_in
    // 1024 to 14336): waves of resident CTAs or pairs times (what a tile costs + its K blocks), and
    // for a split tile the exchange of its parts.  E.g. 256 x 4096 -> 4096: 8.4 us with one CTA a
    // tile, 9.9 with two, 10.8 on pairs; 512 x 4096 -> 14336: 32.5, 63, 18.9; one row of
    // 4096 -> 4096: 8.0 with one, 7.3 with two or four.
    const int64_t nkb = ceil_div(d_in, KB);
    const int64_t tiles = ceil_div(n_rows, MR) * ceil_div(d_out, MC);
    MxPlan plan{MR, MC, 1};
    double best = 1e30;
    for (int ks = 1; ks <= 8 && ks <= nkb && n_tokens <= kTileTokens; ks *= 2) {
        const double exchange = ks > 1 ? 1.0 + 0.5 * ks + 0.02 * std::min(n_rows, MR) : 0.0;
        const double cost = (double)((tiles * ks + 147) / 148) * (3.1 + 0.31 * (double)((nkb + ks - 1) / ks) + exchange);
        if (cost < best) {
            best = cost;
            plan.ksplit = ks;
        }
    }
    for (int cols = 256; cols <= 384; cols += 128) {
        const int64_t pairs = ceil_div(n_rows, 2 * MR) * ceil_div(d_out, cols);
        const double tile = cols == 256 ? 2.2 + 0.3125 * (double)nkb : 2.8 + 0.43 * (double)nkb;
        const double cost = 3.9 + (double)((pairs + 73) / 74) * tile;
        if (cost < best) {
            best = cost;
            plan = MxPlan{2 * MR, cols, 1};
        }
    }
    return plan;
}

cudaError_t launch_mx_tile(const MxGemmParams &p, const MxSegments &sg, int ksplit, cudaStream_t stream)
{
    if (p.rank_bucket_max == 0) return launch_tile<0>(p, sg, ksplit, stream);
    if (p.rank_bucket_max <= 16) return launch_tile<16>(p, sg, ksplit, stream);
    return launch_tile<64>(p, sg, ksplit, stream);
}

cudaError_t launch_mx_pair(const MxGemmParams &p, const MxSlots &sl, int cols, cudaStream_t stream)
{
    int active = 0;
    cudaError_t e = active_pairs(active);
    if (e != cudaSuccess) return e;
    const unsigned pairs = (unsigned)std::min<int64_t>((int64_t)p.n_mblk * p.n_nblk, active);
    if (p.rank_bucket_max == 0) return launch_pair<0>(p, sl, cols, pairs, stream);
    if (p.rank_bucket_max <= 16) return launch_pair<16>(p, sl, cols, pairs, stream);
    return launch_pair<64>(p, sl, cols, pairs, stream);
}

cudaError_t prepare_mx_gemm()
{
    cudaError_t e;
    if ((e = prepare_rank<0>()) != cudaSuccess) return e;
    if ((e = prepare_rank<16>()) != cudaSuccess) return e;
    return prepare_rank<64>();
}

}  // namespace mlora
