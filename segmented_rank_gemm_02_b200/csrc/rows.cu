// rows.cu -- rows grouped by adapter slot on the device, and moved there and back.
//
// mlora_build_segments groups on the host; a router's choices, or a batch whose slots a
// captured graph computes, are known on the device only.  With N = n_rows * top_k choices
// (entry t * top_k + j is row t's j-th slot):
//
//   group     p -> order[p], the stable sort of the entries by slot, with segment metadata
//             (offsets, slots, ranks) of the non-empty slots in ascending order
//   gather    Xs[positions[t, j]] = X[t]
//   combine   Y[t] = sum_j w[t, j] Ys[positions[t, j]]
//   backward  dYs[positions[t, j]] = w[t, j] dY[t],  dw[t, j] = <dY[t], Ys[positions[t, j]]>
//
// gather's own gradient is combine without weights; combine's without weights is gather.
// The last three are bound by HBM: rows are read and written once, but for backward, which
// reads dY once for every four choices of a row.  Sums are fp32, one rounding at the end.  No
// atomics, so results do not vary from run to run.
#include "mlora.h"

#include <algorithm>
#include <cstdint>
#include <mutex>

#include <cuda_fp16.h>

#include "internal.h"
#include "kernels.cuh"
#include "ptx.cuh"

namespace mlora {

namespace {

// ------------------------------------------------------------------ group
// One cluster sorts the whole batch in one launch.  Every ranking warp owns a contiguous
// range of the entries and counts its slots in its own table in shared memory; the tables
// are summed over the warps of a CTA there and over the CTAs through distributed shared
// memory; then each warp walks its range again and places its entries.  Warps never share
// a counter, so the order is the entries' own (a stable sort) without atomics.  What it
// costs is latency: the metadata is a few hundred KB at most.
constexpr int kGroupMaxWarps = 32;
constexpr int kGroupMaxCluster = 8;
constexpr int kGroupSmem = 200 * 1024;
constexpr int kGroupTables = 4;   // besides the warps' tables: CTA totals, totals, first position, spare
constexpr int64_t kMaxEntries = (int64_t)1 << 30;   // 32-bit positions, with room for a block's stride

struct GroupParams {
    const int32_t *row_slots;
    int32_t n;                    // entries
    int32_t n_slots, n_segments;
    const int32_t *slot_rank;
    int32_t *offsets, *slots, *ranks, *order, *positions;
    unsigned int *status;
    int32_t warps;                // ranking warps per CTA
    int32_t range;                // entries per ranking warp (a multiple of 32)
};

// Bin of a slot: 0 for base rows (-1), slot + 1, or n_slots + 1 for what is no slot.
__device__ __forceinline__ int bin_of(int slot, int n_slots)
{
    return slot < -1 || slot >= n_slots ? n_slots + 1 : slot + 1;
}

__global__ void __launch_bounds__(1024, 1) group_kernel(const __grid_constant__ GroupParams p)
{
    extern __shared__ int32_t g_smem[];
    __shared__ int s_scan[2][32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nt = blockDim.x;
    const int bins = p.n_slots + 2;
    const uint32_t crank = cluster_rank(), csize = cluster_size();
    int32_t *cta_total = g_smem, *total = g_smem + bins, *first = g_smem + 2 * bins;
    int32_t *tables = g_smem + 3 * bins;              // [warps][bins]
    for (int i = tid; i < p.warps * bins; i += nt) tables[i] = 0;
    __syncthreads();

    // this warp's entries [lo, hi)
    int32_t *mine = tables + warp * bins;
    const int64_t lo64 = (int64_t)((int)crank * p.warps + warp) * p.range;
    const int lo = warp < p.warps ? (int)min(lo64, (int64_t)p.n) : p.n;
    const int hi = (int)min((int64_t)lo + p.range, (int64_t)p.n);
    for (int i0 = lo; i0 < hi; i0 += 128) {
        int b[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int i = i0 + 32 * u + lane;
            b[u] = i < hi ? bin_of(p.row_slots[i], p.n_slots) : -1;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const unsigned same = __match_any_sync(0xffffffffu, b[u]);
            if (b[u] >= 0 && lane == __ffs(same) - 1) mine[b[u]] += __popc(same);
            __syncwarp();
        }
    }
    __syncthreads();
    // per bin: each warp's entries before it in this CTA, and the CTA's total
    for (int b = tid; b < bins; b += nt) {
        int sum = 0;
        for (int w = 0; w < p.warps; ++w) {
            const int c = tables[w * bins + b];
            tables[w * bins + b] = sum;
            sum += c;
        }
        cta_total[b] = sum;
    }
    if (csize > 1) {
        cluster_arrive_release();
        cluster_wait_acquire();
    } else {
        __syncthreads();
    }
    // per bin over the cluster: the total, and what the CTAs before this one hold
    for (int b = tid; b < bins; b += nt) {
        int before = 0, sum = 0;
        const uint32_t at = smem_addr(cta_total + b);
        for (uint32_t c = 0; c < csize; ++c) {
            const int v = c == crank ? cta_total[b] : __float_as_int(ld_dsmem_f32(map_to_rank(at, c)));
            before += c < crank ? v : 0;
            sum += v;
        }
        total[b] = sum;
        first[b] = before;
    }
    __syncthreads();
    if (csize > 1) cluster_arrive_release();   // waited for before leaving: peers read cta_total

    // scan over the bins in order: the first position of each, and its segment
    int run_pos = 0, run_seg = 0;
    for (int b0 = 0; b0 < bins; b0 += nt) {
        const int b = b0 + tid;
        const int c = b < bins ? total[b] : 0;
        const int has = c > 0 && b <= p.n_slots;
        int ic = c, is = has;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int vc = __shfl_up_sync(0xffffffffu, ic, o), vs = __shfl_up_sync(0xffffffffu, is, o);
            if (lane >= o) {
                ic += vc;
                is += vs;
            }
        }
        if (lane == 31) {
            s_scan[0][warp] = ic;
            s_scan[1][warp] = is;
        }
        __syncthreads();
        int bc = 0, bs = 0, tc = 0, ts = 0;
        for (int w = 0; w < nt / 32; ++w) {
            const int vc = s_scan[0][w], vs = s_scan[1][w];
            bc += w < warp ? vc : 0;
            bs += w < warp ? vs : 0;
            tc += vc;
            ts += vs;
        }
        if (b < bins) {
            const int pos = run_pos + bc + ic - c;
            first[b] += pos;
            if (crank == 0 && has) {
                const int g = run_seg + bs + is - 1;   // < n_segments: at most min(n_slots + 1, n) bins are filled
                p.offsets[g] = pos;
                p.slots[g] = b - 1;
                if (p.ranks) p.ranks[g] = b > 0 ? p.slot_rank[b - 1] : 0;
            }
        }
        run_pos += tc;
        run_seg += ts;
        __syncthreads();
    }
    if (crank == 0) {
        // the remaining segments are empty base segments behind the last grouped entry
        const int bad = total[bins - 1], end = p.n - bad;
        for (int g = run_seg + tid; g < p.n_segments; g += nt) {
            p.offsets[g] = end;
            p.slots[g] = -1;
            if (p.ranks) p.ranks[g] = 0;
        }
        if (tid == 0) {
            p.offsets[p.n_segments] = end;
            if (bad > 0) atomicOr(p.status, kFlagBadSlot);
        }
    }
    for (int i0 = lo; i0 < hi; i0 += 128) {
        int b[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int i = i0 + 32 * u + lane;
            b[u] = i < hi ? bin_of(p.row_slots[i], p.n_slots) : -1;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const unsigned same = __match_any_sync(0xffffffffu, b[u]);
            const int i = i0 + 32 * u + lane;
            if (b[u] >= 0) {
                const int pos = first[b[u]] + mine[b[u]] + __popc(same & ((1u << lane) - 1u));
                p.order[pos] = i;
                p.positions[i] = b[u] <= p.n_slots ? pos : -1;
            }
            __syncwarp();
            if (b[u] >= 0 && lane == __ffs(same) - 1) mine[b[u]] += __popc(same);
            __syncwarp();
        }
    }
    if (csize > 1) cluster_wait_acquire();
}

// ------------------------------------------------------------------ rows there and back
// 16 bytes of a row as fp32.
template <typename T>
struct Vec;
template <>
struct Vec<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void unpack(const uint4 &v, float (&f)[8])
    {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ uint4 pack(const float (&f)[8])
    {
        return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                          pack_bf16x2(f[6], f[7]));
    }
};
template <>
struct Vec<__half> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void unpack(const uint4 &v, float (&f)[8])
    {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 two = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
            f[2 * i] = two.x;
            f[2 * i + 1] = two.y;
        }
    }
    static __device__ __forceinline__ uint4 pack(const float (&f)[8])
    {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <>
struct Vec<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void unpack(const uint4 &v, float (&f)[4])
    {
        f[0] = __uint_as_float(v.x);
        f[1] = __uint_as_float(v.y);
        f[2] = __uint_as_float(v.z);
        f[3] = __uint_as_float(v.w);
    }
    static __device__ __forceinline__ uint4 pack(const float (&f)[4])
    {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    }
};

struct RowParams {
    const int32_t *positions;   // [n_rows][top_k]
    const float *weights;       // [n_rows][top_k] or null (ones)
    const uint8_t *in, *grouped_in;   // rows in row order; grouped rows that are read
    uint8_t *out, *grouped_out;
    float *dweights;            // [n_rows][top_k] or null
    int64_t ld_in, ld_grouped_in, ld_out, ld_grouped_out;   // bytes
    int64_t vecs;               // 16-byte pieces of a row
    int32_t n_rows, top_k, n_tokens;
    unsigned int *status;
};

constexpr int kRowThreads = 256;
constexpr int kRowUnroll = 4;

// A position that may be used; -1 (an entry that was dropped) is silent, others are reported.
__device__ __forceinline__ int checked_position(const RowParams &p, int64_t e, int lane)
{
    const int q = p.positions[e];
    if (q >= 0 && q < p.n_tokens) return q;
    if (q != -1 && lane == 0) atomicOr(p.status, kFlagBadRow);
    return -1;
}

__device__ __forceinline__ uint4 load_row16(const uint8_t *p) { return __ldg(reinterpret_cast<const uint4 *>(p)); }

// TEAM threads per row; each reads its pieces of the row once and writes them top_k times.
template <int TEAM>
__global__ void __launch_bounds__(kRowThreads) gather_kernel(const __grid_constant__ RowParams p)
{
    const int lane = threadIdx.x % TEAM;
    const int64_t t = (int64_t)blockIdx.x * (kRowThreads / TEAM) + threadIdx.x / TEAM;
    if (t >= p.n_rows) return;
    const uint8_t *src = p.in + t * p.ld_in;
    for (int64_t v0 = lane; v0 < p.vecs; v0 += (int64_t)TEAM * kRowUnroll) {
        uint4 x[kRowUnroll];
#pragma unroll
        for (int u = 0; u < kRowUnroll; ++u)
            if (v0 + u * TEAM < p.vecs) x[u] = load_row16(src + 16 * (v0 + u * TEAM));
        for (int j = 0; j < p.top_k; ++j) {
            const int q = checked_position(p, t * p.top_k + j, lane);
            if (q < 0) continue;
            uint8_t *dst = p.grouped_out + (int64_t)q * p.ld_grouped_out;
#pragma unroll
            for (int u = 0; u < kRowUnroll; ++u)
                if (v0 + u * TEAM < p.vecs) *reinterpret_cast<uint4 *>(dst + 16 * (v0 + u * TEAM)) = x[u];
        }
    }
}

// K choices at a time (top_k itself for 1, 2, 4): all their pieces are loaded before the first is used.
template <typename T, int TEAM, int K>
__global__ void __launch_bounds__(kRowThreads) combine_kernel(const __grid_constant__ RowParams p)
{
    constexpr int U = K >= 4 ? 2 : 4;
    constexpr int N = Vec<T>::N;
    const int lane = threadIdx.x % TEAM;
    const int64_t t = (int64_t)blockIdx.x * (kRowThreads / TEAM) + threadIdx.x / TEAM;
    if (t >= p.n_rows) return;
    uint8_t *dst = p.out + t * p.ld_out;
    for (int64_t v0 = lane; v0 < p.vecs; v0 += (int64_t)TEAM * U) {
        float acc[U][N];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < N; ++i) acc[u][i] = 0.f;
        for (int j0 = 0; j0 < p.top_k; j0 += K) {
            int q[K];
            float w[K];
            uint4 x[K][U];
#pragma unroll
            for (int k = 0; k < K; ++k) {
                q[k] = j0 + k < p.top_k ? checked_position(p, t * p.top_k + j0 + k, lane) : -1;
                w[k] = q[k] >= 0 && p.weights ? p.weights[t * p.top_k + j0 + k] : 1.f;
            }
#pragma unroll
            for (int k = 0; k < K; ++k) {
                if (q[k] < 0) continue;
                const uint8_t *src = p.grouped_in + (int64_t)q[k] * p.ld_grouped_in;
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (v0 + u * TEAM < p.vecs) x[k][u] = load_row16(src + 16 * (v0 + u * TEAM));
            }
#pragma unroll
            for (int k = 0; k < K; ++k) {
                if (q[k] < 0) continue;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (v0 + u * TEAM >= p.vecs) continue;
                    float f[N];
                    Vec<T>::unpack(x[k][u], f);
#pragma unroll
                    for (int i = 0; i < N; ++i) acc[u][i] = fmaf(w[k], f[i], acc[u][i]);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (v0 + u * TEAM < p.vecs) *reinterpret_cast<uint4 *>(dst + 16 * (v0 + u * TEAM)) = Vec<T>::pack(acc[u]);
    }
}

// One pass over dY[t] per K choices: each piece of dY is scaled into the choices' grouped rows
// and multiplied with theirs; the products are summed over the row by the team.
template <typename T, int TEAM, int K>
__global__ void __launch_bounds__(kRowThreads) combine_backward_kernel(const __grid_constant__ RowParams p)
{
    constexpr int U = K >= 4 ? 2 : 4;
    constexpr int N = Vec<T>::N;
    constexpr int WARPS = TEAM / 32;
    __shared__ float s_dot[kRowThreads / 32][K];
    const int lane = threadIdx.x % TEAM;
    const int64_t t0 = (int64_t)blockIdx.x * (kRowThreads / TEAM) + threadIdx.x / TEAM;
    const bool in = t0 < p.n_rows;   // every thread stays for the barriers
    const int64_t t = in ? t0 : 0;
    const uint8_t *src = p.in + t * p.ld_in;
    for (int j0 = 0; j0 < p.top_k; j0 += K) {
        int q[K];
        float w[K], dot[K];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            q[k] = in && j0 + k < p.top_k ? checked_position(p, t * p.top_k + j0 + k, lane) : -1;
            w[k] = q[k] >= 0 && p.weights ? p.weights[t * p.top_k + j0 + k] : 1.f;
            dot[k] = 0.f;
        }
        for (int64_t v0 = lane; v0 < p.vecs; v0 += (int64_t)TEAM * U) {
            uint4 dy[U], y[K][U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (v0 + u * TEAM < p.vecs) dy[u] = load_row16(src + 16 * (v0 + u * TEAM));
            if (p.dweights) {
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    if (q[k] < 0) continue;
                    const uint8_t *row = p.grouped_in + (int64_t)q[k] * p.ld_grouped_in;
#pragma unroll
                    for (int u = 0; u < U; ++u)
                        if (v0 + u * TEAM < p.vecs) y[k][u] = load_row16(row + 16 * (v0 + u * TEAM));
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (v0 + u * TEAM >= p.vecs) continue;
                float f[N];
                Vec<T>::unpack(dy[u], f);
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    if (q[k] < 0) continue;
                    if (p.dweights) {
                        float g[N];
                        Vec<T>::unpack(y[k][u], g);
#pragma unroll
                        for (int i = 0; i < N; ++i) dot[k] = fmaf(f[i], g[i], dot[k]);
                    }
                    if (p.grouped_out) {
                        float g[N];
#pragma unroll
                        for (int i = 0; i < N; ++i) g[i] = w[k] * f[i];
                        *reinterpret_cast<uint4 *>(p.grouped_out + (int64_t)q[k] * p.ld_grouped_out +
                                                   16 * (v0 + u * TEAM)) = Vec<T>::pack(g);
                    }
                }
            }
        }
        if (p.dweights) {
#pragma unroll
            for (int k = 0; k < K; ++k) {
#pragma unroll
                for (int o = 16; o >= 1; o >>= 1) dot[k] += __shfl_xor_sync(0xffffffffu, dot[k], o);
                if (threadIdx.x % 32 == 0) s_dot[threadIdx.x / 32][k] = dot[k];
            }
            __syncthreads();
            if (in && lane < K && j0 + lane < p.top_k) {
                float sum = 0.f;
#pragma unroll
                for (int w2 = 0; w2 < WARPS; ++w2) sum += s_dot[threadIdx.x / TEAM * WARPS + w2][lane];
                p.dweights[t * p.top_k + j0 + lane] = sum;
            }
            __syncthreads();
        }
    }
}

// Threads per row: so many that each has about four pieces, a whole warp at least.
int row_team(int64_t vecs) { return vecs >= 1024 ? 256 : vecs >= 512 ? 128 : vecs >= 256 ? 64 : 32; }

template <int TEAM>
unsigned row_blocks(int n_rows)
{
    return (unsigned)(((int64_t)n_rows + kRowThreads / TEAM - 1) / (kRowThreads / TEAM));
}

template <typename T, int TEAM>
void launch_combine(const RowParams &p, cudaStream_t s)
{
    const unsigned b = row_blocks<TEAM>(p.n_rows);
    if (p.top_k == 1) combine_kernel<T, TEAM, 1><<<b, kRowThreads, 0, s>>>(p);
    else if (p.top_k == 2) combine_kernel<T, TEAM, 2><<<b, kRowThreads, 0, s>>>(p);
    else combine_kernel<T, TEAM, 4><<<b, kRowThreads, 0, s>>>(p);
}

template <typename T, int TEAM>
void launch_backward(const RowParams &p, cudaStream_t s)
{
    const unsigned b = row_blocks<TEAM>(p.n_rows);
    if (p.top_k == 1) combine_backward_kernel<T, TEAM, 1><<<b, kRowThreads, 0, s>>>(p);
    else if (p.top_k == 2) combine_backward_kernel<T, TEAM, 2><<<b, kRowThreads, 0, s>>>(p);
    else combine_backward_kernel<T, TEAM, 4><<<b, kRowThreads, 0, s>>>(p);
}

enum RowOp { ROW_GATHER, ROW_COMBINE, ROW_BACKWARD };

template <int TEAM>
cudaError_t launch_rows_team(RowOp op, int dtype, const RowParams &p, cudaStream_t s)
{
    if (op == ROW_GATHER) gather_kernel<TEAM><<<row_blocks<TEAM>(p.n_rows), kRowThreads, 0, s>>>(p);
    else if (dtype == MLORA_DTYPE_BF16)
        op == ROW_COMBINE ? launch_combine<__nv_bfloat16, TEAM>(p, s) : launch_backward<__nv_bfloat16, TEAM>(p, s);
    else if (dtype == MLORA_DTYPE_FP16)
        op == ROW_COMBINE ? launch_combine<__half, TEAM>(p, s) : launch_backward<__half, TEAM>(p, s);
    else
        op == ROW_COMBINE ? launch_combine<float, TEAM>(p, s) : launch_backward<float, TEAM>(p, s);
    return cudaGetLastError();
}

cudaError_t launch_rows(RowOp op, int dtype, const RowParams &p, cudaStream_t s)
{
    switch (row_team(p.vecs)) {
    case 256: return launch_rows_team<256>(op, dtype, p, s);
    case 128: return launch_rows_team<128>(op, dtype, p, s);
    case 64: return launch_rows_team<64>(op, dtype, p, s);
    default: return launch_rows_team<32>(op, dtype, p, s);
    }
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int dtype_size(int32_t dtype)
{
    return dtype == MLORA_DTYPE_BF16 || dtype == MLORA_DTYPE_FP16 ? 2 : dtype == MLORA_DTYPE_FP32 ? 4 : 0;
}

// What gather, combine and backward have in common: sizes, the pool's device and status.
mlora_status row_common(mlora_pool *pool, const int32_t *positions, int32_t n_rows, int32_t top_k, int32_t n_tokens,
                        int32_t d, int32_t dtype, RowParams &p, int &device)
{
    mlora_pool_view view;
    if (!mlora_pool_get_view(pool, &view)) return MLORA_ERR_INVALID_ARG;
    const int size = dtype_size(dtype);
    if (n_rows < 0 || top_k < 1 || n_tokens < 0 || d < 1 || size == 0) return MLORA_ERR_INVALID_ARG;
    if ((int64_t)n_rows * top_k > kMaxEntries) return MLORA_ERR_INVALID_ARG;
    if (((int64_t)d * size) % 16 != 0) return MLORA_ERR_UNSUPPORTED;   // rows of whole 16-byte vectors
    if (n_rows > 0 && positions == nullptr) return MLORA_ERR_INVALID_ARG;
    p.positions = positions;
    p.n_rows = n_rows;
    p.top_k = top_k;
    p.n_tokens = n_tokens;
    p.vecs = (int64_t)d * size / 16;
    p.status = view.status;
    device = view.device;
    return MLORA_OK;
}

// A row-major operand: 16-byte aligned, rows d elements or more apart; its stride in bytes.
bool row_operand(const void *ptr, int64_t ld, int32_t d, int32_t dtype, int64_t &bytes)
{
    const int size = dtype_size(dtype);
    bytes = ld * size;
    return ptr != nullptr && aligned16(ptr) && ld >= d && bytes % 16 == 0;
}

}  // namespace

cudaError_t prepare_row_kernels()
{
    return cudaFuncSetAttribute(group_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kGroupSmem);
}

}  // namespace mlora

using namespace mlora;

extern "C" {

mlora_status mlora_group_rows(mlora_pool *pool, const int32_t *row_slots, int32_t n_rows, int32_t top_k,
                              const mlora_row_groups *out, void *stream)
{
    mlora_pool_view view;
    if (!mlora_pool_get_view(pool, &view) || out == nullptr || n_rows < 0 || top_k < 1) return MLORA_ERR_INVALID_ARG;
    const int64_t n = (int64_t)n_rows * top_k;
    if (n > kMaxEntries) return MLORA_ERR_INVALID_ARG;
    if (out->offsets == nullptr) return MLORA_ERR_INVALID_ARG;
    if (n > 0 && (row_slots == nullptr || out->slots == nullptr || out->order == nullptr || out->positions == nullptr))
        return MLORA_ERR_INVALID_ARG;
    const int64_t bins = (int64_t)view.n_slots + 2;
    // the tables beside one ranking warp's have to fit
    if (bins * 4 * kGroupTables > kGroupSmem) return MLORA_ERR_UNSUPPORTED;
    mlora_device_guard guard(view.device);
    if (!guard.ok) return MLORA_ERR_CUDA;
    mlora_status st = mlora_prepare_device(view.device);
    if (st != MLORA_OK) return st;
    GroupParams p{};
    p.row_slots = row_slots;
    p.n = (int32_t)n;
    p.n_slots = view.n_slots;
    p.n_segments = (int32_t)std::min<int64_t>((int64_t)view.n_slots + 1, n);
    p.slot_rank = view.slot_rank;
    p.offsets = out->offsets;
    p.slots = out->slots;
    p.ranks = out->ranks;
    p.order = out->order;
    p.positions = out->positions;
    p.status = view.status;
    const unsigned cluster = (unsigned)std::clamp<int64_t>((n + 1023) / 1024, 1, kGroupMaxCluster);
    // as many ranking warps as have 32 entries each and whose tables fit
    int warps = kGroupMaxWarps;
    while (warps > 1 && (bins * 4 * (warps + kGroupTables - 1) > kGroupSmem || (int64_t)cluster * 16 * warps >= n))
        warps /= 2;
    p.warps = warps;
    p.range = (int32_t)((((n + cluster * warps - 1) / (cluster * warps)) + 31) / 32 * 32);
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3(cluster, 1, 1);
    cfg.blockDim = dim3((unsigned)std::max({32 * warps, 128, (int)std::min<int64_t>(1024, (bins + 31) / 32 * 32)}), 1, 1);
    cfg.dynamicSmemBytes = (size_t)bins * 4 * (warps + kGroupTables - 1);
    cfg.stream = static_cast<cudaStream_t>(stream);
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, group_kernel, p) == cudaSuccess ? MLORA_OK : MLORA_ERR_CUDA;
}

mlora_status mlora_gather_rows(mlora_pool *pool, const int32_t *positions, int32_t n_rows, int32_t top_k, const void *X,
                               int64_t ldx, int32_t dtype, int32_t d, int32_t n_tokens, void *Xs, int64_t ldxs,
                               void *stream)
{
    RowParams p{};
    int device = 0;
    mlora_status st = row_common(pool, positions, n_rows, top_k, n_tokens, d, dtype, p, device);
    if (st != MLORA_OK) return st;
    if (n_rows == 0 || n_tokens == 0) return MLORA_OK;
    if (!row_operand(X, ldx, d, dtype, p.ld_in) || !row_operand(Xs, ldxs, d, dtype, p.ld_grouped_out))
        return MLORA_ERR_INVALID_ARG;
    p.in = static_cast<const uint8_t *>(X);
    p.grouped_out = static_cast<uint8_t *>(Xs);
    mlora_device_guard guard(device);
    if (!guard.ok) return MLORA_ERR_CUDA;
    return launch_rows(ROW_GATHER, dtype, p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? MLORA_OK
                                                                                               : MLORA_ERR_CUDA;
}

mlora_status mlora_combine_rows(mlora_pool *pool, const int32_t *positions, const float *weights, int32_t n_rows,
                                int32_t top_k, const void *Ys, int64_t ldys, int32_t dtype, int32_t d,
                                int32_t n_tokens, void *Y, int64_t ldy, void *stream)
{
    RowParams p{};
    int device = 0;
    mlora_status st = row_common(pool, positions, n_rows, top_k, n_tokens, d, dtype, p, device);
    if (st != MLORA_OK) return st;
    if (n_rows == 0) return MLORA_OK;
    if (!row_operand(Y, ldy, d, dtype, p.ld_out)) return MLORA_ERR_INVALID_ARG;
    if (n_tokens > 0 && !row_operand(Ys, ldys, d, dtype, p.ld_grouped_in)) return MLORA_ERR_INVALID_ARG;
    p.weights = weights;
    p.grouped_in = static_cast<const uint8_t *>(Ys);
    p.out = static_cast<uint8_t *>(Y);
    mlora_device_guard guard(device);
    if (!guard.ok) return MLORA_ERR_CUDA;
    return launch_rows(ROW_COMBINE, dtype, p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? MLORA_OK
                                                                                                : MLORA_ERR_CUDA;
}

mlora_status mlora_combine_rows_backward(mlora_pool *pool, const int32_t *positions, const float *weights,
                                         int32_t n_rows, int32_t top_k, const void *dY, int64_t lddy, const void *Ys,
                                         int64_t ldys, int32_t dtype, int32_t d, int32_t n_tokens, void *dYs,
                                         int64_t lddys, float *dweights, void *stream)
{
    RowParams p{};
    int device = 0;
    mlora_status st = row_common(pool, positions, n_rows, top_k, n_tokens, d, dtype, p, device);
    if (st != MLORA_OK) return st;
    if (n_rows == 0) return MLORA_OK;
    if (dYs == nullptr && dweights == nullptr) return MLORA_ERR_INVALID_ARG;
    if (!row_operand(dY, lddy, d, dtype, p.ld_in)) return MLORA_ERR_INVALID_ARG;
    if (n_tokens > 0) {
        if (dYs != nullptr && !row_operand(dYs, lddys, d, dtype, p.ld_grouped_out)) return MLORA_ERR_INVALID_ARG;
        if (dweights != nullptr && !row_operand(Ys, ldys, d, dtype, p.ld_grouped_in)) return MLORA_ERR_INVALID_ARG;
    }
    p.weights = weights;
    p.in = static_cast<const uint8_t *>(dY);
    p.grouped_in = static_cast<const uint8_t *>(Ys);
    p.grouped_out = static_cast<uint8_t *>(dYs);
    p.dweights = dweights;
    mlora_device_guard guard(device);
    if (!guard.ok) return MLORA_ERR_CUDA;
    return launch_rows(ROW_BACKWARD, dtype, p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? MLORA_OK
                                                                                                 : MLORA_ERR_CUDA;
}

}  // extern "C"
