// landmarks8.cu -- landmark generation from the keys of the 8-bit cache.
//
// "Hierarchical Sparse Attention Done Right" (arXiv 2607.02980v1), Sec. 3, "Linear surrogate for chunk mass": the
// landmark query u attends over its chunk's keys; with keys k_t = s_c e_t (e_t the e4m3 rows, s_c the chunk's
// scale) the logits are scale s_c <u, e_t>, the landmark is s_c sum_t p_t e_t, and the entropy of p is the chunk's
// bias.  One warp per chunk, one pass over its rows with a running maximum and sums, a lane holding d / 32 columns.
#include "cache8.h"
#include "common.cuh"
#include "e4m3.cuh"

namespace hils {
namespace {

constexpr int kWarps = 4;

template <typename Tin, int D>
__global__ void __launch_bounds__(32 * kWarps)
    landmarks8_kernel(const uint8_t *__restrict__ K8, const float *__restrict__ ks, const Tin *__restrict__ U,
                      Tin *__restrict__ L, float *__restrict__ beta, Cache8 p, float scale, int c0, int span, int t_end)
{
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const long long unit = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (unit >= (long long)p.B * p.Hkv * span) return;
    const long long bg = unit / span;
    const int c = c0 + (int)(unit - bg * span);
    const int rows = min(p.C, t_end - c * p.C);
    const uint8_t *kc = K8 + ((size_t)bg * p.T + (size_t)c * p.C) * D + lane * E;
    const size_t lrow = ((size_t)bg * p.nL + c) * D + lane * E;
    const float sc = ks[(size_t)bg * p.nL + c];
    float u[E], acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        u[e] = to_float(U[lrow + e]) * (scale * sc);
        acc[e] = 0.f;
    }
    float m = -INFINITY, z = 0.f, y = 0.f;
    for (int t = 0; t < rows; ++t) {
        float k[4];
        if constexpr (E == 4) e4m3x4_to_float(*reinterpret_cast<const uint32_t *>(kc + (size_t)t * D), k);
        else e4m3x4_to_float(*reinterpret_cast<const uint16_t *>(kc + (size_t)t * D), k);
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) s = fmaf(u[e], k[e], s);
        s = warp_sum(s);
        const float mn = fmaxf(m, s), r = expf(m - mn), w = expf(s - mn);
        // y = sum of w (x - m): moves with the maximum like z, less the shift it brings
        y = (m == -INFINITY) ? 0.f : r * (y + (m - mn) * z);
        z = z * r + w;
        y = fmaf(w, s - mn, y);
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = fmaf(w, k[e], acc[e] * r);
        m = mn;
    }
    const float inv = 1.0f / z;
#pragma unroll
    for (int e = 0; e < E; ++e) store_out(L + lrow + e, acc[e] * (inv * sc));
    if (beta && lane == 0) beta[(size_t)bg * p.nL + c] = logf(z) - y * inv;
}

}  // namespace

cudaError_t launch_landmarks8(const Cache8 &c, hils_dtype in, float scale, const uint8_t *K8, const float *ks,
                              const void *U, void *L, float *beta, int c0, int c1, int t_end, cudaStream_t s)
{
    const int span = c1 - c0;
    const unsigned grid = (unsigned)(((long long)c.B * c.Hkv * span + kWarps - 1) / kWarps);
    auto run = [&](auto kern, auto *u, auto *l) {
        kern<<<grid, 32 * kWarps, 0, s>>>(K8, ks, u, l, beta, c, scale, c0, span, t_end);
        return cudaGetLastError();
    };
    if (in == HILS_BF16) {
        auto *u = static_cast<const __nv_bfloat16 *>(U);
        auto *l = static_cast<__nv_bfloat16 *>(L);
        return c.d == 128 ? run(landmarks8_kernel<__nv_bfloat16, 128>, u, l)
                          : run(landmarks8_kernel<__nv_bfloat16, 64>, u, l);
    }
    auto *u = static_cast<const float *>(U);
    auto *l = static_cast<float *>(L);
    return c.d == 128 ? run(landmarks8_kernel<float, 128>, u, l) : run(landmarks8_kernel<float, 64>, u, l);
}

}  // namespace hils
