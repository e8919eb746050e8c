// mx_quant.cu -- rows to 4-bit microscaled floating point and back.
//
// Format (OCP microscaling formats, MXFP4): a block of 32 consecutive elements of a row has
// the scale 2^e, e = floor(log2(max |x|)) - 2 clamped to [-127, 127], kept as the byte
// e + 127; each element is x / 2^e rounded to the nearest e2m1 value (0, .5, 1, 1.5, 2, 3, 4,
// 6 with a sign; ties to the even code, beyond 6 to 6).  The byte is the fp32 exponent field of
// the block's maximum less two (not below zero), and x / 2^e is an exact product, so the
// conversion's rounding is the only one.  A block that holds an infinity or a NaN gets the scale
// byte 255 (NaN) and zero codes: all its values read back as NaN.
//
// Layout: two codes per byte, the first in the low half, rows padded with zero codes to whole
// blocks; scale bytes in tiles of 128 rows x 4 blocks (512 bytes) as the tensor core wants them
// in tensor memory: row r of the tile and block b at 16 (r % 32) + 4 (r / 32) + b.  A warp
// takes 256 columns of rows r, r + 32, r + 64, r + 96 of a tile: eight elements per lane and
// row, all loads issued before the first is used; the 4 x 4 scale bytes of one r are transposed
// between the lanes and stored together.  HBM bound: n d (size + 17/32) bytes.  14336 x 4096 bf16:
// quantise 26.3 us (0.87 of the measured copy rate; 28.6 with each row's maximum compared as fp32),
// dequantise 25.2 (0.91); 7168 x 4096 fp32: 21.4 and 26.2 (0.96 and 0.78).
#include "mlora.h"

#include <algorithm>
#include <cstdint>

#include <cuda_fp16.h>

#include "internal.h"
#include "kernels.cuh"
#include "ptx.cuh"

namespace mlora {

namespace {

constexpr int kQuantThreads = 256;
constexpr int kTileRowsMx = 128;

// Eight elements of type T at `p` as fp32.
template <typename T>
struct Eight;
template <>
struct Eight<__nv_bfloat16> {
    uint4 v;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { v = __ldg(reinterpret_cast<const uint4 *>(p)); }
    __device__ __forceinline__ void zero() { v = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void get(float (&f)[8]) const
    {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ void store(__nv_bfloat16 *p, const float (&f)[8])
    {
        *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                                   pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
    }
};
template <>
struct Eight<__half> {
    uint4 v;
    __device__ __forceinline__ void load(const __half *p) { v = __ldg(reinterpret_cast<const uint4 *>(p)); }
    __device__ __forceinline__ void zero() { v = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void get(float (&f)[8]) const
    {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 two = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
            f[2 * i] = two.x;
            f[2 * i + 1] = two.y;
        }
    }
    static __device__ __forceinline__ void store(__half *p, const float (&f)[8])
    {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <>
struct Eight<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *p)
    {
        a = __ldg(reinterpret_cast<const float4 *>(p));
        b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
    }
    __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void get(float (&f)[8]) const
    {
        f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
    }
};

struct MxRows {
    uint8_t *codes;
    int64_t ld;        // bytes
    uint8_t *scales;
    int32_t n_rows, n_cols;
    int32_t chunks;    // 256-column chunks of a row
};

// Warp -> (128-row tile, r of 0..31, 256-column chunk).
__device__ __forceinline__ bool my_unit(const MxRows &q, int64_t w, int &row0, int &chunk)
{
    const int64_t tiles = ((int64_t)q.n_rows + kTileRowsMx - 1) / kTileRowsMx;
    if (w >= tiles * 32 * q.chunks) return false;
    chunk = (int)(w % q.chunks);
    const int64_t r = w / q.chunks;
    row0 = (int)(r / 32 * kTileRowsMx + r % 32);
    return true;
}

// The 16 scale bytes of (row0's r, tile `half` of the chunk).
__device__ __forceinline__ uint8_t *scale_vec(const MxRows &q, int row0, int chunk, int half)
{
    return q.scales + ((int64_t)(row0 / kTileRowsMx) * 2 * q.chunks + 2 * chunk + half) * 512 + (row0 % 32) * 16;
}

// A magnitude's own 16 bits as those of the fp32 it converts to.
__device__ __forceinline__ uint32_t magnitude_bits(__nv_bfloat16, uint32_t m) { return m << 16; }
__device__ __forceinline__ uint32_t magnitude_bits(__half, uint32_t m)
{
    return __float_as_uint(__half2float(__ushort_as_half((unsigned short)m)));
}

// The largest magnitude of each row's block of 32 (four lanes), as fp32 bits: NaN above infinity
// above the rest.  16-bit types compare their own bits, two elements or two rows at a time.
template <typename T>
__device__ __forceinline__ void block_maxima(const Eight<T> (&x)[4], uint32_t (&big)[4])
{
    if constexpr (sizeof(T) == 2) {
        uint32_t m[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const uint4 v = x[u].v;
            m[u] = __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu), __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
        }
#pragma unroll
        for (int u = 0; u < 4; u += 2) {
            uint32_t p = __vmaxu2(__byte_perm(m[u], m[u + 1], 0x5410), __byte_perm(m[u], m[u + 1], 0x7632));
            p = __vmaxu2(p, __shfl_xor_sync(0xffffffffu, p, 1));
            p = __vmaxu2(p, __shfl_xor_sync(0xffffffffu, p, 2));
            big[u] = magnitude_bits(T(), p & 0xffffu);
            big[u + 1] = magnitude_bits(T(), p >> 16);
        }
    } else {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            float f[8];
            x[u].get(f);
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(f[i]) & 0x7fffffffu);
            m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
            big[u] = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
        }
    }
}

// (16-bit types: the 32 registers that let whole SMs of threads reside)
template <typename T>
__global__ void __launch_bounds__(kQuantThreads, sizeof(T) == 2 ? 8 : 5) mx_quantize_kernel(const T *X, int64_t ldx, const MxRows q)
{
    griddep_launch_dependents();   // a product of Q may set itself up meanwhile; it waits for this grid
    const int lane = threadIdx.x & 31;
    int row0, chunk;
    if (!my_unit(q, ((int64_t)blockIdx.x * kQuantThreads + threadIdx.x) >> 5, row0, chunk)) return;
    const int col = chunk * 256 + lane * 8;
    Eight<T> x[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const int row = row0 + 32 * u;
        if (row < q.n_rows && col < q.n_cols) x[u].load(X + row * ldx + col);
        else x[u].zero();
    }
    uint32_t big[4];
    block_maxima(x, big);
    uint32_t bytes = 0;   // this block's scale bytes, one per row
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const bool finite = big[u] < 0x7f800000u;
        const int field = (int)(big[u] >> 23);
        const uint32_t s = finite ? (uint32_t)max(field - 2, 0) : 255u;
        bytes |= s << (8 * u);
        float f[8];
        x[u].get(f);
        // 2^-e; a block that is not finite gets zero codes
        const float inv = finite ? __uint_as_float((254u - s) << 23) : 0.f;
        uint32_t c = 0;
        if (finite) {
            c = e2m1x8(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv, f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv);
        }
        const int row = row0 + 32 * u;
        if (row < q.n_rows && col / 32 <= (q.n_cols - 1) / 32)   // the padding of the last block too
            *reinterpret_cast<uint32_t *>(q.codes + row * q.ld + col / 2) = c;
    }
    // 4 x 4 bytes, blocks x rows -> rows x blocks: lane u of each half stores row u's word
    uint32_t b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] = __shfl_sync(0xffffffffu, bytes, (lane & 16) + 4 * i);
    const int u = lane & 3;
    const uint32_t sel = u | (u + 4) << 4;
    const uint32_t word = __byte_perm(__byte_perm(b[0], b[1], sel), __byte_perm(b[2], b[3], sel), 0x5410);
    if ((lane & 15) < 4) *reinterpret_cast<uint32_t *>(scale_vec(q, row0, chunk, lane >> 4) + 4 * u) = word;
}

template <typename T>
__global__ void __launch_bounds__(kQuantThreads, 8) mx_dequantize_kernel(const MxRows q, T *X, int64_t ldx)
{
    const int lane = threadIdx.x & 31;
    int row0, chunk;
    if (!my_unit(q, ((int64_t)blockIdx.x * kQuantThreads + threadIdx.x) >> 5, row0, chunk)) return;
    // A lane's eight elements: eight columns in a row; in fp32 four, and four 128 columns on, so that a
    // store instruction writes 512 consecutive bytes (16 of every 32 at a time: 7168 x 4096 took 37 us).
    constexpr bool kSplit = sizeof(T) == 4;
    constexpr int kNext = kSplit ? 128 : 4;
    const int col = chunk * 256 + lane * (kSplit ? 4 : 8);
    const bool in[2] = {col < q.n_cols, col + kNext < q.n_cols};   // n_cols is a multiple of 8
    const uint4 sv = *reinterpret_cast<const uint4 *>(scale_vec(q, row0, chunk, kSplit ? 0 : lane >> 4));
    uint4 tv = sv;
    if (kSplit) tv = *reinterpret_cast<const uint4 *>(scale_vec(q, row0, chunk, 1));
    const uint32_t words[2][4] = {{sv.x, sv.y, sv.z, sv.w}, {tv.x, tv.y, tv.z, tv.w}};
    const int byte = kSplit ? lane >> 3 : (lane >> 2) & 3;
    uint32_t c[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const int row = row0 + 32 * u;
        const uint8_t *src = q.codes + row * q.ld + col / 2;
        c[u] = 0;
        if (row >= q.n_rows) continue;
        if constexpr (kSplit) {
            if (in[0]) c[u] = *reinterpret_cast<const uint16_t *>(src);
            if (in[1]) c[u] |= (uint32_t)*reinterpret_cast<const uint16_t *>(src + kNext / 2) << 16;
        } else {
            if (in[0]) c[u] = *reinterpret_cast<const uint32_t *>(src);
        }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const int row = row0 + 32 * u;
        if (row >= q.n_rows) continue;
        float f[8], scale[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t s = (words[h][u] >> (8 * byte)) & 0xffu;
            // 2^(s - 127): subnormal for s = 0, NaN for 255
            scale[h] = __uint_as_float(s == 255u ? 0x7fc00000u : s == 0u ? 0x00400000u : s << 23);
        }
        e2m1x8_to_float(c[u], f);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] *= scale[i / 4];
        T *y = X + row * ldx + col;
        if constexpr (kSplit) {
            if (in[0]) *reinterpret_cast<float4 *>(y) = make_float4(f[0], f[1], f[2], f[3]);
            if (in[1]) *reinterpret_cast<float4 *>(y + kNext) = make_float4(f[4], f[5], f[6], f[7]);
        } else {
            if (in[0]) Eight<T>::store(y, f);
        }
    }
}

unsigned quant_blocks(const MxRows &q)
{
    const int64_t warps = ((int64_t)q.n_rows + kTileRowsMx - 1) / kTileRowsMx * 32 * q.chunks;
    return (unsigned)((warps * 32 + kQuantThreads - 1) / kQuantThreads);
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

mlora_status check_operand(const void *X, int32_t dtype, int64_t ldx, const mlora_mx_matrix *Q, bool &empty)
{
    if (Q == nullptr) return MLORA_ERR_INVALID_ARG;
    if (dtype != MLORA_DTYPE_BF16 && dtype != MLORA_DTYPE_FP16 && dtype != MLORA_DTYPE_FP32) return MLORA_ERR_INVALID_ARG;
    mlora_status st = mlora_mx_check_matrix(Q);
    if (st != MLORA_OK) return st;
    empty = Q->n_rows == 0;
    if (empty) return MLORA_OK;
    if (X == nullptr || !aligned16(X) || ldx < Q->n_cols || ldx % (dtype == MLORA_DTYPE_FP32 ? 4 : 8) != 0)
        return MLORA_ERR_INVALID_ARG;
    return MLORA_OK;
}

MxRows rows_of(const mlora_mx_matrix *Q)
{
    MxRows q;
    q.codes = static_cast<uint8_t *>(Q->codes);
    q.ld = Q->ld;
    q.scales = static_cast<uint8_t *>(Q->scales);
    q.n_rows = Q->n_rows;
    q.n_cols = Q->n_cols;
    q.chunks = (int32_t)(((int64_t)Q->n_cols + 255) / 256);
    return q;
}

}  // namespace

}  // namespace mlora

using namespace mlora;

// Sizes, strides and pointers of a quantised matrix (an empty one needs no memory).
mlora_status mlora_mx_check_matrix(const mlora_mx_matrix *Q)
{
    if (Q->n_rows < 0 || Q->n_cols <= 0) return MLORA_ERR_INVALID_ARG;
    if (Q->n_cols % 8 != 0) return MLORA_ERR_UNSUPPORTED;
    if (Q->ld % 16 != 0 || Q->ld < ((int64_t)Q->n_cols + 31) / 32 * 16) return MLORA_ERR_INVALID_ARG;
    if (Q->n_rows > 0 && (Q->codes == nullptr || Q->scales == nullptr || !aligned16(Q->codes) || !aligned16(Q->scales)))
        return MLORA_ERR_INVALID_ARG;
    return MLORA_OK;
}

extern "C" {

int64_t mlora_mx_scale_bytes(int32_t n_rows, int32_t n_cols)
{
    if (n_rows < 0 || n_cols < 0) return -1;
    return ((int64_t)n_rows + 127) / 128 * (((int64_t)n_cols + 255) / 256) * 1024;
}

mlora_status mlora_mx_quantize(const void *X, int32_t x_dtype, int64_t ldx, const mlora_mx_matrix *Q, void *stream)
{
    bool empty = false;
    mlora_status st = check_operand(X, x_dtype, ldx, Q, empty);
    if (st != MLORA_OK || empty) return st;
    const MxRows q = rows_of(Q);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const unsigned b = quant_blocks(q);
    if (x_dtype == MLORA_DTYPE_BF16)
        mx_quantize_kernel<<<b, kQuantThreads, 0, s>>>(static_cast<const __nv_bfloat16 *>(X), ldx, q);
    else if (x_dtype == MLORA_DTYPE_FP16)
        mx_quantize_kernel<<<b, kQuantThreads, 0, s>>>(static_cast<const __half *>(X), ldx, q);
    else
        mx_quantize_kernel<<<b, kQuantThreads, 0, s>>>(static_cast<const float *>(X), ldx, q);
    return cudaGetLastError() == cudaSuccess ? MLORA_OK : MLORA_ERR_CUDA;
}

mlora_status mlora_mx_dequantize(const mlora_mx_matrix *Q, void *X, int32_t x_dtype, int64_t ldx, void *stream)
{
    bool empty = false;
    mlora_status st = check_operand(X, x_dtype, ldx, Q, empty);
    if (st != MLORA_OK || empty) return st;
    const MxRows q = rows_of(Q);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const unsigned b = quant_blocks(q);
    if (x_dtype == MLORA_DTYPE_BF16)
        mx_dequantize_kernel<<<b, kQuantThreads, 0, s>>>(q, static_cast<__nv_bfloat16 *>(X), ldx);
    else if (x_dtype == MLORA_DTYPE_FP16)
        mx_dequantize_kernel<<<b, kQuantThreads, 0, s>>>(q, static_cast<__half *>(X), ldx);
    else
        mx_dequantize_kernel<<<b, kQuantThreads, 0, s>>>(q, static_cast<float *>(X), ldx);
    return cudaGetLastError() == cudaSuccess ? MLORA_OK : MLORA_ERR_CUDA;
}

}  // extern "C"
