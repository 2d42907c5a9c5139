// attend8.cu -- chunk attention and fusion over the 8-bit cache (CUDA cores, every shape).
//
// "Hierarchical Sparse Attention Done Right" (arXiv 2607.02980v1), Abstract and Sec. 3 "Hierarchical softmax", with
// keys ks_c e and values vs_c e' (e4m3 rows e, e', one scale per chunk and side): the chunk's logits carry
// scale * ks_c, its output carries the fusion weight times vs_c.
//
// One block per query group (b, g, i), one warp per head; a chunk's visible rows are widened to float32 in shared
// memory once for the group's heads.
#include "attend_simt.cuh"
#include "cache8.h"
#include "e4m3.cuh"

namespace hils {
namespace {

template <int D>
__device__ __forceinline__ void stage8(float *dst, const uint8_t *src, int rows, float scale)
{
    for (int e = threadIdx.x; e < rows * D / 4; e += blockDim.x) {
        float v[4];
        e4m3x4_to_float(__ldg(reinterpret_cast<const uint32_t *>(src) + e), v);
        reinterpret_cast<float4 *>(dst)[e] = make_float4(v[0] * scale, v[1] * scale, v[2] * scale, v[3] * scale);
    }
}

template <typename Tin, typename Tout, int D>
__global__ void attend8_kernel(Dims p, const Tin *__restrict__ Q, const uint8_t *__restrict__ K8,
                               const uint8_t *__restrict__ V8, const float *__restrict__ ks, const float *__restrict__ vs,
                               const int32_t *__restrict__ sel_idx, const float *__restrict__ sel_score,
                               Tout *__restrict__ O)
{
    extern __shared__ __align__(16) unsigned char smem_raw[];
    float *Ks = reinterpret_cast<float *>(smem_raw);
    float *Vs = Ks + (size_t)p.C * D;
    float *qsm = Vs + (size_t)p.C * D;                                       // [G][D]
    float *wsm = qsm + (size_t)p.G * D;                                      // [G][k+1]
    int *chunk = reinterpret_cast<int *>(wsm + (size_t)p.G * (p.k + 1));     // [k+1]

    const int i = blockIdx.x;
    const size_t bg = blockIdx.y;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long pos = (long long)p.q_offset + i;
    const int ns = p.k + 1;
    const size_t row = (bg * p.G + warp) * p.N + i;
    const int32_t *si = sel_idx + (bg * p.N + i) * p.k;
    for (int x = lane; x < D; x += 32) qsm[warp * D + x] = to_float(Q[row * D + x]) * p.scale;
    for (int j = threadIdx.x; j < ns; j += blockDim.x) chunk[j] = (j < p.k) ? si[j] : (int)(pos / p.C);
    __syncthreads();
    // fusion weights; a slot without a chunk has no weight, whatever its score
    float mx = -INFINITY, z = 0.f;
    for (int j = lane; j < ns; j += 32) mx = fmaxf(mx, chunk[j] < 0 ? -INFINITY : sel_score[row * ns + j]);
    mx = warp_max(mx);
    for (int j = lane; j < ns; j += 32) {
        const float s = chunk[j] < 0 ? -INFINITY : sel_score[row * ns + j];
        const float e = (s == -INFINITY) ? 0.f : expf(s - mx);
        wsm[warp * ns + j] = e;
        z += e;
    }
    z = warp_sum(z);
    const float inv = z > 0.f ? 1.0f / z : (z == 0.f ? 0.f : z);             // no weight at all: a zero row; NaN stays
    float acc[D / 32];
#pragma unroll
    for (int x = 0; x < D / 32; ++x) acc[x] = 0.f;
    for (int j = 0; j < ns; ++j) {
        const int c = chunk[j];
        if (c < 0) continue;
        const int n_vis = (int)min((long long)p.C, pos - (long long)c * p.C + 1);
        const size_t at = (bg * p.T + (size_t)c * p.C) * D;
        __syncthreads();
        stage8<D>(Ks, K8 + at, n_vis, ks[bg * p.nL + c]);
        stage8<D>(Vs, V8 + at, n_vis, vs[bg * p.nL + c]);
        __syncthreads();
        warp_attend_chunk<float, D>(qsm + warp * D, Ks, Vs, n_vis, wsm[warp * ns + j] * inv, acc);
    }
#pragma unroll
    for (int x = 0; x < D / 32; ++x) store_out(O + row * D + lane * (D / 32) + x, acc[x]);
}

template <typename Tin, typename Tout, int D>
cudaError_t launch_t(const Dims &p, const void *Q, const uint8_t *K8, const uint8_t *V8, const float *ks, const float *vs,
                     const int32_t *sel_idx, const float *sel_score, void *O, cudaStream_t s)
{
    const int ns = p.k + 1;
    const size_t smem = (2 * (size_t)p.C * D + (size_t)p.G * D + (size_t)p.G * ns + ns) * 4;
    auto kern = attend8_kernel<Tin, Tout, D>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    kern<<<dim3(p.N, p.B * p.Hkv), 32 * p.G, smem, s>>>(p, static_cast<const Tin *>(Q), K8, V8, ks, vs, sel_idx, sel_score,
                                                        static_cast<Tout *>(O));
    return cudaGetLastError();
}

}  // namespace

size_t attend8_ws_bytes(const Dims &, hils_dtype, hils_dtype) { return 0; }

cudaError_t launch_attend8(const Dims &p, hils_dtype in, hils_dtype out, const void *Q, const uint8_t *K8,
                           const uint8_t *V8, const float *ks, const float *vs, const int32_t *sel_idx,
                           const float *sel_score, void *O, void *, const DeviceCtl &, cudaStream_t s)
{
    auto run = [&](auto f64, auto f128) {
        return p.d == 64 ? f64(p, Q, K8, V8, ks, vs, sel_idx, sel_score, O, s)
                         : f128(p, Q, K8, V8, ks, vs, sel_idx, sel_score, O, s);
    };
    if (in == HILS_F32)
        return out == HILS_F32 ? run(launch_t<float, float, 64>, launch_t<float, float, 128>)
                               : run(launch_t<float, __nv_bfloat16, 64>, launch_t<float, __nv_bfloat16, 128>);
    return out == HILS_F32 ? run(launch_t<__nv_bfloat16, float, 64>, launch_t<__nv_bfloat16, float, 128>)
                           : run(launch_t<__nv_bfloat16, __nv_bfloat16, 64>, launch_t<__nv_bfloat16, __nv_bfloat16, 128>);
}

}  // namespace hils
