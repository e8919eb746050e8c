// slot_operand.cuh -- the low-rank A operand of the GEMMs that add LoRA products in the
// tensor core (base_gemm.cu, mx_gemm.cu).
#pragma once

#include "kernels.cuh"
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

// One row's s * H as the bf16 hi + lo parts that stage_operand writes, zeros past its rank, for
// kernels that stage every row's own once.  PARTS threads share a row, each RK / PARTS of the ranks.
template <int RK, int PARTS>
struct RowOperand {
    static constexpr int N = RK / PARTS;   // a multiple of 8
    uint32_t hi[N / 2], lo[N / 2];

    __device__ __forceinline__ void load(const float *hsrc, int rank, float sc, int part)
    {
        const int c0 = part * N;
        float h[N];
        if (rank == RK) {
#pragma unroll
            for (int i = 0; i < N / 4; ++i) {
                const float4 v = reinterpret_cast<const float4 *>(hsrc + c0)[i];
                h[4 * i] = v.x, h[4 * i + 1] = v.y, h[4 * i + 2] = v.z, h[4 * i + 3] = v.w;
            }
        } else {
#pragma unroll
            for (int c = 0; c < N; ++c) h[c] = c0 + c < rank ? hsrc[c0 + c] : 0.f;
        }
#pragma unroll
        for (int c = 0; c < N / 2; ++c) {
            float h0, l0, h1, l1;
            split_bf16(sc * h[2 * c], h0, l0);
            split_bf16(sc * h[2 * c + 1], h1, l1);
            hi[c] = pack_bf16x2(h0, h1);
            lo[c] = pack_bf16x2(l0, l1);
        }
    }

    // Row r of the operand (hi, then lo).
    __device__ __forceinline__ void store(uint8_t *buf, int r, int part) const
    {
        constexpr int HOP = kOperandRows * RK * 2;
#pragma unroll
        for (int cg = 0; cg < N / 8; ++cg) {
            const int off = ((part * (N / 8) + cg) * (kOperandRows / 8) + r / 8) * 128 + (r % 8) * 16;
            *reinterpret_cast<uint4 *>(buf + off) =
                make_uint4(hi[4 * cg], hi[4 * cg + 1], hi[4 * cg + 2], hi[4 * cg + 3]);
            *reinterpret_cast<uint4 *>(buf + HOP + off) =
                make_uint4(lo[4 * cg], lo[4 * cg + 1], lo[4 * cg + 2], lo[4 * cg + 3]);
        }
    }
};

// The problems of segment g (status bits as the other kernels report them), 0 if it
// is a valid adapter segment; *rank and *scale are set for a valid one.
__device__ __forceinline__ unsigned segment_problem(const TileParams &p, int g, int a, int p0, int p1, int &rank,
                                                    float &scale)
{
    if (a < -1 || a >= p.n_slots) return kFlagBadSlot;
    if (p0 < 0 || p1 < p0 || p1 > p.n_tokens) return kFlagBadOffsets;
    if (a < 0) return 0;
    rank = p.slot_rank[a];
    scale = p.scales ? p.scales[g] : p.slot_scale[a];
    if (p.generations && p.slot_gen[a] != p.generations[g]) return kFlagStaleSlot;
    if (rank <= 0) return kFlagSlotEmpty;
    if ((p.ranks && p.ranks[g] != rank) || rank_bucket(rank) == 0) return kFlagBadRank;
    return 0;
}

// The segment that may hold grouped position q: the last g with offsets[g] <= q.
__device__ __forceinline__ int segment_of_position(const TileParams &p, int q)
{
    int lo = 0, hi = p.n_segments - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (p.offsets[mid] <= q) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// A block's copy of the segments in shared memory, {first position, slot (-1: base or invalid), scale,
// rank} each: a search through L2 is a chain of dependent loads of 0.4 us each (256 rows of 64
// slots took 5 us to find so).  An end record closes it.
struct SegmentTable {
    int4 *records;   // null: too many segments, they are read where they are
    int n;
};

// All `threads` of the caller take part; it synchronises them afterwards.  `reporter` flags the
// segments' problems.
__device__ __forceinline__ SegmentTable copy_segments(const TileParams &p, int4 *records, int capacity, int tid,
                                                      int threads, bool reporter)
{
    SegmentTable t{p.n_segments < capacity ? records : nullptr, p.n_segments};
    if (t.records == nullptr && !reporter) return t;
    for (int g = tid; g < p.n_segments; g += threads) {
        // two rounds of loads, each all at once (segment_problem's come one after the other)
        const int p0 = p.offsets[g], p1 = p.offsets[g + 1], a = p.slots[g];
        const int want_rank = p.ranks ? p.ranks[g] : 0;
        const float seg_scale = p.scales ? p.scales[g] : 0.f;
        const uint32_t want_gen = p.generations ? p.generations[g] : 0u;
        const int at = a >= 0 && a < p.n_slots ? a : 0;
        const int rank = p.slot_rank[at];
        const float scale = p.scales ? seg_scale : p.slot_scale[at];
        const uint32_t gen = p.generations ? p.slot_gen[at] : 0u;
        unsigned f = 0;
        if (a < -1 || a >= p.n_slots) f = kFlagBadSlot;
        else if (p0 < 0 || p1 < p0 || p1 > p.n_tokens) f = kFlagBadOffsets;
        else if (a >= 0) {
            if (gen != want_gen) f = kFlagStaleSlot;
            else if (rank <= 0) f = kFlagSlotEmpty;
            else if ((p.ranks && want_rank != rank) || rank_bucket(rank) == 0) f = kFlagBadRank;
        }
        if (f && reporter) atomicOr(p.status, f);
        // (an end that differs from the next segment's beginning is no valid segment's)
        if (t.records) records[g] = make_int4(p0, f || a < 0 ? -1 : a, __float_as_int(scale), rank);
    }
    if (t.records && tid == 0) records[p.n_segments] = make_int4(p.offsets[p.n_segments], -1, 0, 0);
    return t;
}

// {q, slot, scale, rank} of grouped position q if it lies in a valid adapter segment, else {-1, ...}.
__device__ __forceinline__ int4 row_of_position(const TileParams &p, const SegmentTable &t, int q)
{
    const int4 none = make_int4(-1, -1, 0, 0);
    if (t.records) {
        int lo = 0, hi = t.n - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (t.records[mid].x <= q) lo = mid;
            else hi = mid - 1;
        }
        const int4 v = t.records[lo];
        if (v.y < 0 || q < v.x || q >= t.records[lo + 1].x) return none;
        return make_int4(q, v.y, v.z, v.w);
    }
    const int g = segment_of_position(p, q);
    const int a = p.slots[g], p0 = p.offsets[g], p1 = p.offsets[g + 1];
    int rank = 0;
    float scale = 0.f;
    if (a < 0 || q < p0 || q >= p1 || segment_problem(p, g, a, p0, p1, rank, scale)) return none;
    return make_int4(q, a, __float_as_int(scale), rank);
}

// A row that nothing has claimed (as unsigned, so that every grouped position is below it).
constexpr unsigned kUnclaimed = 0xffffffffu;

// Finds the rows of a block [row0, row0 + n): claims[r] (preset to -1, that is kUnclaimed) gets the lowest
// grouped position that names row r and lies in a valid adapter segment, whatever the order of the
// claims, so that all CTAs that look the same rows up agree.  A row claimed twice is flagged;
// `reporter` flags rows that do not exist.
__device__ __forceinline__ void claim_rows(const TileParams &p, const SegmentTable &t, int row0, int n, int *claims,
                                           int tid, int threads, bool reporter)
{
    for (int64_t q0 = tid; q0 < p.n_tokens; q0 += 4 * threads) {
        int row[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int64_t q = q0 + u * threads;
            row[u] = q < p.n_tokens && p.token_indices ? p.token_indices[q] : (int)q;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int64_t q = q0 + u * threads;
            if (q >= p.n_tokens) continue;
            const bool exists = row[u] >= 0 && row[u] < p.n_rows;
            const bool in = exists && row[u] >= row0 && row[u] < row0 + n;
            if (!in && !(reporter && !exists)) continue;
            if (row_of_position(p, t, (int)q).x < 0) continue;
            if (!in || atomicMin(reinterpret_cast<unsigned *>(&claims[row[u] - row0]), (unsigned)q) != kUnclaimed)
                atomicOr(p.status, kFlagBadRow);
        }
    }
}

// Whether row r is the first of its block with this slot (>= 0); slots[] in shared memory,
// 16-byte aligned, and the whole warp takes part.
__device__ __forceinline__ bool first_with_slot(const int *slots, int r, int slot)
{
    const unsigned same = __match_any_sync(0xffffffffu, slot);
    if (slot < 0 || (r & 31) != __ffs(same) - 1) return false;
    const int4 *v = reinterpret_cast<const int4 *>(slots);
    bool found = false;
    for (int i = 0; i < (r & ~31) / 4; i += 8) {   // a warp's 32 rows at a time
        int4 s[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) s[u] = v[i + u];
#pragma unroll
        for (int u = 0; u < 8; ++u) found |= s[u].x == slot || s[u].y == slot || s[u].z == slot || s[u].w == slot;
    }
    return !found;
}

// Index of a slot in a list of `count` distinct slots that holds it (in shared memory, 16-byte
// aligned, with room for a multiple of 16).
__device__ __forceinline__ int slot_index(const int *list, int count, int slot)
{
    const int4 *v = reinterpret_cast<const int4 *>(list);
    for (int i = 0; 4 * i < count; i += 4) {
        int4 s[4];
        int at = -1;
#pragma unroll
        for (int u = 0; u < 4; ++u) s[u] = v[i + u];
#pragma unroll
        for (int u = 3; u >= 0; --u) {   // the first match wins (entries past the count may be anything)
            if (s[u].w == slot) at = 4 * u + 3;
            if (s[u].z == slot) at = 4 * u + 2;
            if (s[u].y == slot) at = 4 * u + 1;
            if (s[u].x == slot) at = 4 * u;
        }
        if (at >= 0) return 4 * i + at;
    }
    return 0;
}

}  // namespace mlora
