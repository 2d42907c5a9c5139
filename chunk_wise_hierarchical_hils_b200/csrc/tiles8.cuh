// tiles8.cuh -- tiles of the 8-bit cache in shared memory and their mma.sync products (sm_100a).
//
// A tile is 16 rows (keys) of D bytes.  Rows lie one after the other, a row's 16-byte pieces permuted so that both ways
// of reading a tile touch every bank once: as keys (eight rows of one half of the tile, one piece) and as values
// (eight rows in a row, one piece).  Straight from global memory to registers, without shared memory, the same reads
// hit banks two and four at a time (rows are 128 bytes apart), and L1 was what bound the kernels (84% busy at 238 us
// for the landmarks of 1M tokens).
//
// Index orders inside a product are free: with lane (r, t) = (lane / 4, lane % 4)
//   keys    ldmatrix, four 8 x 16-byte matrices: 4 bytes of d = 16 c + 4 t .. of a row, the A fragments of k-step c.  Row
//           r of the tile's first half is key 4 (r / 2) + r % 2, of its second half the key two further
//   values  ldmatrix on bytes, transposed: keys 4 t .. 4 t + 3 of column d = 16 c + r (and + 8): the A fragments of a
//           product over the keys, whose first half of k is keys 4 t, 4 t + 1, as movmatrix hands out the
//           probabilities of the key order above
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "e4m3.cuh"

namespace hils {
namespace t8 {

// Where 16-byte piece ch of row `row` lies in a tile.
template <int D>
__device__ __forceinline__ uint32_t piece_at(int row, int ch)
{
    const int b = ((row >> 1) ^ (row >> 3)) & 1;
    if constexpr (D == 128) return (uint32_t)(row * 128 + ((ch ^ ((row & 1) | ((row >> 1) & 2) | (b << 2))) << 4));
    else return (uint32_t)(row * 64 + ((ch ^ (((row >> 2) & 1) | (b << 1))) << 4));
}

// Row of a tile that row r of half h stands for when the tile is read as keys.
__device__ __forceinline__ int key_row(int r, int h) { return 4 * (r >> 1) + (r & 1) + 2 * h; }

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// One warp asks for ROWS rows (a multiple of 16) from src to dst (shared).  PART: rows behind row `top` (below 0 where all
// of them are) may not be read, and row `top` stands in for them.
template <int D, int ROWS, bool PART>
__device__ __forceinline__ void load_rows(uint32_t dst, const uint8_t *src, int top)
{
    constexpr int CH = D / 16, STEP = 32 / CH;   // pieces a row, rows a step
    const int lane = threadIdx.x & 31, row0 = lane / CH, ch = lane % CH;
#pragma unroll
    for (int i = 0; i < ROWS / STEP; ++i) {
        const int row = row0 + i * STEP;
        // 16 rows make a period of piece_at
        const uint32_t at = piece_at<D>(row & 15, ch) + (uint32_t)(row & ~15) * D;
        cp_async16(dst + at, src + (PART ? min(row, top) : row) * D + 16 * ch);
    }
}

// The tile at `tile`, as keys: w[c][h] = bytes d = 16 c + 4 t .. of the row that row r of half h stands for.
template <int D>
__device__ __forceinline__ void read_keys(uint32_t tile, uint32_t (&w)[D / 16][2])
{
    const int lane = threadIdx.x & 31, row = key_row(lane & 7, (lane >> 3) & 1), c0 = lane >> 4;
#pragma unroll
    for (int c = 0; c < D / 16; c += 2)
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[c][0]), "=r"(w[c][1]), "=r"(w[c + 1][0]), "=r"(w[c + 1][1])
                     : "r"(tile + piece_at<D>(row, c + c0))
                     : "memory");
}

// The tile as values, columns d = 16 c .. 16 c + 31: w[x][h] = keys 4 t .. 4 t + 3 of d = 16 (c + x) + r + 8 h.
template <int D>
__device__ __forceinline__ void read_values(uint32_t tile, int c, uint32_t (&w)[2][2])
{
    const int lane = threadIdx.x & 31;
    asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w[0][0]), "=r"(w[0][1]), "=r"(w[1][0]), "=r"(w[1][1])
                 : "r"(tile + piece_at<D>(lane & 15, c + (lane >> 4)))
                 : "memory");
}

// D (16 x 8, f32) += A (16 x 16, f16) B (16 x 8)
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same with A as bytes: w0 of rows 0..7, w1 of rows 8..15, the low two bytes in the first half of k.
__device__ __forceinline__ void mma_bytes(float (&d)[4], uint32_t w0, uint32_t w1, uint32_t b0, uint32_t b1)
{
    mma_f16(d, e4m3x2_to_f16x2(w0), e4m3x2_to_f16x2(w1), e4m3x2_to_f16x2(w0 >> 16), e4m3x2_to_f16x2(w1 >> 16), b0, b1);
}

__device__ __forceinline__ void add4(float (&a)[4], const float (&x)[4])
{
#pragma unroll
    for (int e = 0; e < 4; ++e) a[e] += x[e];
}

// 8 x 8 matrix of 16-bit elements, transposed across the warp
__device__ __forceinline__ uint32_t movmatrix_t(uint32_t x)
{
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi)
{
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ float2 unpack_f16(uint32_t v) { return __half22float2(*reinterpret_cast<const __half2 *>(&v)); }

// Four consecutive elements, widened; four results, rounded.
__device__ __forceinline__ void load4(const float *p, float *o)
{
    const float4 v = __ldg(reinterpret_cast<const float4 *>(p));
    o[0] = v.x; o[1] = v.y; o[2] = v.z; o[3] = v.w;
}
__device__ __forceinline__ void load4(const __nv_bfloat16 *p, float *o)
{
    const uint2 v = __ldg(reinterpret_cast<const uint2 *>(p));
    o[0] = __uint_as_float(v.x << 16); o[1] = __uint_as_float(v.x & 0xFFFF0000u);
    o[2] = __uint_as_float(v.y << 16); o[3] = __uint_as_float(v.y & 0xFFFF0000u);
}
__device__ __forceinline__ void store4(float *p, float4 v) { *reinterpret_cast<float4 *>(p) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16 *p, float4 v)
{
    const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
    *reinterpret_cast<uint2 *>(p) = make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
}

}  // namespace t8
}  // namespace hils
