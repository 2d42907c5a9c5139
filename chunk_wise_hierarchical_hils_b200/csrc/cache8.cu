// cache8.cu -- writing keys and values into the 8-bit cache, and reading them back.
//
// One scale serves the C rows of a chunk on one side (keys or values) of one kv-head: attention and landmark
// generation take whole chunks, so a chunk's scale is one number per tile for them.  The scale is a power of two,
// the smallest with which the chunk's largest magnitude stays within e4m3's 448: dividing by it is exact, the one
// rounding is the conversion to e4m3, and when a later row raises a chunk's scale the rows already there move to
// the new scale by a shift of their exponents (exact but for values that become subnormal).
#include <float.h>

#include "cache8.h"
#include "common.cuh"
#include "e4m3.cuh"

namespace hils {
namespace {

// Sixteen consecutive elements as floats.
__device__ __forceinline__ void load16(const float *p, float *o) { load8(p, o); load8(p + 8, o + 8); }
__device__ __forceinline__ void load16(const __nv_bfloat16 *p, float *o) { load8(p, o); load8(p + 8, o + 8); }

// Append.  One block per (b, kv-head, chunk touched, side), 64 elements a thread: the new rows are read once and
// held in registers between the maximum and the conversion, so the pass moves each byte once and is bound by HBM
// (or, for a decode step's single rows, by its latency).
template <typename Tin, int D>
__global__ void append_kernel(const Tin *__restrict__ K, const Tin *__restrict__ V, uint8_t *__restrict__ K8,
                              uint8_t *__restrict__ V8, float *__restrict__ ks, float *__restrict__ vs, Cache8 p, int t0,
                              int t1, int c0, int nb)
{
    constexpr int UNITS = 4;   // units of 16 elements per thread: blockDim.x = C * D / 64
    __shared__ float s_max[8];
    const int tid = threadIdx.x, nt = blockDim.x;
    const int side = blockIdx.x & 1;
    const long long u = blockIdx.x >> 1;
    const long long bg = u / nb;
    const int c = c0 + (int)(u - bg * nb);
    const Tin *src = (side ? V : K) + (size_t)bg * (size_t)(t1 - t0) * D;
    uint8_t *dst = (side ? V8 : K8) + ((size_t)bg * p.T + (size_t)c * p.C) * D;
    float *scale = (side ? vs : ks) + (size_t)bg * p.nL + c;
    const int r0 = max(t0 - c * p.C, 0);                               // the chunk's rows [r0, r1) are new
    const int r1 = (int)min((long long)t1 - (long long)c * p.C, (long long)p.C);
    const float old = r0 > 0 ? *scale : 0.f;

    float x[UNITS][16];
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < UNITS; ++i) {
        const int e = (i * nt + tid) * 16, row = e / D;
        if (row >= r0 && row < r1) {
            load16(src + (size_t)((long long)c * p.C + row - t0) * D + e % D, x[i]);
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const float a = fabsf(x[i][j]);
                m = fmaxf(m, a <= FLT_MAX ? a : 0.f);                  // infinities and NaN have no say in the scale
            }
        }
    }
    m = warp_max(m);
    if ((tid & 31) == 0) s_max[tid >> 5] = m;
    __syncthreads();
    for (int w = 0; w < nt / 32; ++w) m = fmaxf(m, s_max[w]);
    const float inv_new = exp2_int(-scale_exponent(m));
    float s = exp2_int(scale_exponent(m)), inv = inv_new;
    if (r0 > 0) {
        if (s > old) {
            // the scale grows: the rows already in the chunk go over to it
            const float f = old * inv;
#pragma unroll
            for (int i = 0; i < UNITS; ++i) {
                const int e = (i * nt + tid) * 16;
                if (e / D < r0) {
                    uint4 v = *reinterpret_cast<const uint4 *>(dst + e);
                    uint32_t *w = reinterpret_cast<uint32_t *>(&v);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float a[4];
                        e4m3x4_to_float(w[j], a);
                        w[j] = to_e4m3x4(a[0] * f, a[1] * f, a[2] * f, a[3] * f);
                    }
                    *reinterpret_cast<uint4 *>(dst + e) = v;
                }
            }
        } else {
            s = old;
            inv = 1.0f / old;
        }
    }
#pragma unroll
    for (int i = 0; i < UNITS; ++i) {
        const int e = (i * nt + tid) * 16, row = e / D;
        if (row >= r0 && row < r1) {
            uint4 v;
            uint32_t *w = reinterpret_cast<uint32_t *>(&v);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                w[j] = to_e4m3x4(x[i][4 * j] * inv, x[i][4 * j + 1] * inv, x[i][4 * j + 2] * inv, x[i][4 * j + 3] * inv);
            *reinterpret_cast<uint4 *>(dst + e) = v;
        }
    }
    if (tid == 0) *scale = s;
}

__device__ __forceinline__ void store16(float *p, const float *v)
{
#pragma unroll
    for (int i = 0; i < 4; ++i)
        reinterpret_cast<float4 *>(p)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
}

__device__ __forceinline__ void store16(__nv_bfloat16 *p, const float *v)
{
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        uint4 u;
        uint32_t *w = reinterpret_cast<uint32_t *>(&u);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            __nv_bfloat162 t = __floats2bfloat162_rn(v[8 * i + 2 * j], v[8 * i + 2 * j + 1]);
            w[j] = *reinterpret_cast<uint32_t *>(&t);
        }
        reinterpret_cast<uint4 *>(p)[i] = u;
    }
}

// Read back.  Units of 16 elements; one pass, bound by HBM.
template <typename Tout, int D>
__global__ void __launch_bounds__(256)
    read_kernel(const uint8_t *__restrict__ K8, const uint8_t *__restrict__ V8, const float *__restrict__ ks,
                const float *__restrict__ vs, Tout *__restrict__ K, Tout *__restrict__ V, Cache8 p, int t0, long long units)
{
    const int side = blockIdx.z;
    const size_t bg = blockIdx.y;
    const uint8_t *src = (side ? V8 : K8) + (bg * p.T + (size_t)t0) * D;
    const float *scale = (side ? vs : ks) + bg * p.nL;
    Tout *dst = (side ? V : K) + bg * (size_t)units * 16;
    const long long u = (long long)blockIdx.x * 256 + threadIdx.x;
    if (u >= units) return;
    const float s = __ldg(scale + (t0 + (int)(u / (D / 16))) / p.C);
    const uint4 v = __ldg(reinterpret_cast<const uint4 *>(src) + u);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    float o[16];
#pragma unroll
    for (int j = 0; j < 4; ++j) e4m3x4_to_float(w[j], o + 4 * j);
#pragma unroll
    for (int j = 0; j < 16; ++j) o[j] *= s;
    store16(dst + (size_t)u * 16, o);
}

}  // namespace

cudaError_t launch_cache_append(const Cache8 &c, hils_dtype in, const void *K, const void *V, uint8_t *K8, uint8_t *V8,
                                float *ks, float *vs, int t0, int t1, cudaStream_t s)
{
    const int c0 = t0 / c.C, nb = (t1 - 1) / c.C - c0 + 1;
    const unsigned grid = (unsigned)(2ll * c.B * c.Hkv * nb);
    const int threads = c.C * c.d / 64;
    auto run = [&](auto kern, auto *k, auto *v) {
        kern<<<grid, threads, 0, s>>>(k, v, K8, V8, ks, vs, c, t0, t1, c0, nb);
        return cudaGetLastError();
    };
    if (in == HILS_BF16) {
        auto *k = static_cast<const __nv_bfloat16 *>(K), *v = static_cast<const __nv_bfloat16 *>(V);
        return c.d == 128 ? run(append_kernel<__nv_bfloat16, 128>, k, v) : run(append_kernel<__nv_bfloat16, 64>, k, v);
    }
    auto *k = static_cast<const float *>(K), *v = static_cast<const float *>(V);
    return c.d == 128 ? run(append_kernel<float, 128>, k, v) : run(append_kernel<float, 64>, k, v);
}

cudaError_t launch_cache_read(const Cache8 &c, hils_dtype out, const uint8_t *K8, const uint8_t *V8, const float *ks,
                              const float *vs, void *K, void *V, int t0, int t1, cudaStream_t s)
{
    const long long units = (long long)(t1 - t0) * (c.d / 16);
    const dim3 grid((unsigned)((units + 255) / 256), (unsigned)(c.B * c.Hkv), 2);
    auto run = [&](auto kern, auto *k, auto *v) {
        kern<<<grid, 256, 0, s>>>(K8, V8, ks, vs, k, v, c, t0, units);
        return cudaGetLastError();
    };
    if (out == HILS_BF16) {
        auto *k = static_cast<__nv_bfloat16 *>(K), *v = static_cast<__nv_bfloat16 *>(V);
        return c.d == 128 ? run(read_kernel<__nv_bfloat16, 128>, k, v) : run(read_kernel<__nv_bfloat16, 64>, k, v);
    }
    auto *k = static_cast<float *>(K), *v = static_cast<float *>(V);
    return c.d == 128 ? run(read_kernel<float, 128>, k, v) : run(read_kernel<float, 64>, k, v);
}

}  // namespace hils
