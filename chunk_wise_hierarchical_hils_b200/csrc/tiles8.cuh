// tiles8.cuh -- register tiles of the 8-bit cache and their mma.sync products (sm_100a).
//
// A warp takes tiles of 16 rows (keys) straight from global memory into registers.  The index orders inside an mma product
// are free, so rows and columns are permuted until what a lane's 16-byte loads bring is what its fragments hold; lane
// (r, t) = (lane / 4, lane % 4):
//   K tile   rows r and r + 8, bytes d = 64 s + 16 t + 0..15 (s < d / 64): the A fragments of a product over d
//   V tile   rows 2t, 2t+1, 2t+8, 2t+9, bytes d = (d / 8) r + ..: after a byte transpose (four rows x four columns) the
//            A fragments of a product over the rows
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "e4m3.cuh"

namespace hils {
namespace t8 {

// volatile: the loads stay where a kernel's pipeline issues them
__device__ __forceinline__ void ldg16(uint32_t *w, const uint8_t *p)
{
    asm volatile("ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "l"(p));
}

__device__ __forceinline__ void ldg8(uint32_t *w, const uint8_t *p)
{
    asm volatile("ld.global.nc.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "l"(p));
}

// One tile, D / 8 words a lane.  Keys: [2 rows][D / 64 segments][4 words]; values: [4 rows][D / 32 words].
// p: the tile's first row + this lane's column (16 t, or (D / 8) r).  PART: rows behind row `top` (counted from the
// tile's first; below 0 where the tile holds none) may not be read, and row `top` stands in for them.
template <int D, bool PART = false>
__device__ __forceinline__ void load_k(uint32_t *w, const uint8_t *p, int r, int top = 0)
{
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int s = 0; s < D / 64; ++s)
            ldg16(w + (h * (D / 64) + s) * 4, p + (PART ? min(8 * h + r, top) : 8 * h + r) * D + 64 * s);
}

template <int D, bool PART = false>
__device__ __forceinline__ void load_v(uint32_t *w, const uint8_t *p, int t, int top = 0)
{
    constexpr int W = D / 32;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const int key = 2 * t + (q & 1) + 8 * (q >> 1);
        const uint8_t *src = p + (PART ? min(key, top) : key) * D;
        if constexpr (W == 4) ldg16(w + q * W, src);
        else ldg8(w + q * W, src);
    }
}

// D (16 x 8, f32) += A (16 x 16, f16) B (16 x 8)
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
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

// Stores N consecutive results (N = 8 or 16), 16-byte aligned.
template <int N>
__device__ __forceinline__ void store_n(float *p, const float *v)
{
#pragma unroll
    for (int i = 0; i < N; i += 4) *reinterpret_cast<float4 *>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
}
template <int N>
__device__ __forceinline__ void store_n(__nv_bfloat16 *p, const float *v)
{
#pragma unroll
    for (int i = 0; i < N; i += 8) {
        uint4 u;
        uint32_t *w = reinterpret_cast<uint32_t *>(&u);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const __nv_bfloat162 x = __floats2bfloat162_rn(v[i + 2 * j], v[i + 2 * j + 1]);
            w[j] = *reinterpret_cast<const uint32_t *>(&x);
        }
        *reinterpret_cast<uint4 *>(p + i) = u;
    }
}

}  // namespace t8
}  // namespace hils
