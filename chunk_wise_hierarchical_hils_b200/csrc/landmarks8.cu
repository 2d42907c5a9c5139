// landmarks8.cu -- landmark generation from the keys of the 8-bit cache.
//
// "Hierarchical Sparse Attention Done Right" (arXiv 2607.02980v1), Sec. 3, "Linear surrogate for chunk mass": the
// landmark query u attends over its chunk's keys; with keys k_t = s_c e_t (e_t the e4m3 rows, s_c the chunk's
// scale) the logits are scale s_c <u, e_t>, the landmark is s_c sum_t p_t e_t, and the entropy of p is the chunk's
// bias.
//
// Every key byte is read once from HBM and used in two products, so the kernel is bound by HBM as long as the
// products stay cheap: both run on e4m3 mma.sync tiles, in which the keys are operands as they are.  One warp per
// chunk, with the pipeline of the attention kernel: a chunk is a stream of tiles, as keys (for the logits) and again as
// values (for the sum; these loads hit L1), through four register buffers, running on into the warp's next chunk.
//
// Numbers.  The other operand, one row of u or p, is float32: it is split into pieces of e4m3's four bits, each 2^4 finer
// than the one before, in the columns the product has anyway (column c holds piece c): six pieces hold 24 bits (u
// relative to the row's largest, p relative to the chunk's largest).  The columns' sums meet in float32.
#include "cache8.h"
#include "common.cuh"
#include "tiles8.cuh"

namespace hils {
namespace {

using namespace t8;

constexpr int kWarps = 4;
constexpr int kBlocksPerSm = 3;

// Piece r (the lane's column) of the values a, b, both below 256 in magnitude, as two e4m3 bytes: 16^r times what
// pieces 0..r-1 leave of them; no piece beyond the sixth.
__device__ __forceinline__ uint32_t piece_pair(float a, float b, int r)
{
    uint32_t h = pack_f16(a, b);
    if (r >= 3) {
        const float2 y = unpack_f16(h);
        h = pack_f16((a - y.x) * 4096.0f, (b - y.y) * 4096.0f);
    }
    const int q = r >= 3 ? r - 3 : r;
    const uint32_t p0 = f16x2_to_e4m3x2(h), h1 = e4m3_rest<16>(h, p0);
    const uint32_t p1 = f16x2_to_e4m3x2(h1), p2 = f16x2_to_e4m3x2(e4m3_rest<16>(h1, p1));
    return r >= 6 ? 0u : q == 0 ? p0 : q == 1 ? p1 : p2;
}

__device__ __forceinline__ float sum_t(float x)   // over the four lanes of a row
{
    x += __shfl_xor_sync(0xFFFFFFFFu, x, 1);
    return x + __shfl_xor_sync(0xFFFFFFFFu, x, 2);
}

template <typename T>
__device__ __forceinline__ void store4(T *p, float a, float b, float c, float d)
{
    store_out(p, a); store_out(p + 1, b); store_out(p + 2, c); store_out(p + 3, d);
}
template <>
__device__ __forceinline__ void store4(float *p, float a, float b, float c, float d)
{
    *reinterpret_cast<float4 *>(p) = make_float4(a, b, c, d);
}
template <>
__device__ __forceinline__ void store4(__nv_bfloat16 *p, float a, float b, float c, float d)
{
    const __nv_bfloat162 x = __floats2bfloat162_rn(a, b), y = __floats2bfloat162_rn(c, d);
    *reinterpret_cast<uint2 *>(p) = make_uint2(*reinterpret_cast<const uint32_t *>(&x), *reinterpret_cast<const uint32_t *>(&y));
}

template <typename Tin, int D, int C>
__global__ void __launch_bounds__(32 * kWarps, kBlocksPerSm)
    landmarks8_kernel(const uint8_t *__restrict__ K8, const float *__restrict__ ks, const Tin *__restrict__ U,
                      Tin *__restrict__ L, float *__restrict__ beta, Cache8 p, float scale, int c0, int span, int t_end)
{
    constexpr int MT = C / 16, KS = D / 32, DT = D / 16, WORDS = D / 8, W = D / 32;
    const int lane = threadIdx.x & 31, r = lane >> 2, t = lane & 3;
    const long long units = (long long)p.B * p.Hkv * span, step = (long long)gridDim.x * kWarps;
    const float f0 = exp2_int(-8 * t), f1 = exp2_int(-8 * t - 4);   // worth of pieces 2t and 2t + 1

    struct At {
        long long bg;
        int c, rows;
        const uint8_t *row0;
    };
    auto at = [&](long long u) {
        At a;
        a.bg = u / span;
        a.c = c0 + (int)(u - a.bg * span);
        a.rows = (int)min((long long)C, (long long)t_end - (long long)a.c * C);
        a.row0 = K8 + ((size_t)a.bg * p.T + (size_t)a.c * C) * D;
        return a;
    };
    uint32_t buf[4][WORDS];
    auto load_tile = [&](int n, const At &a) {
        if (n < MT) load_k<D>(buf[n & 3], a.row0 + 16 * n * D + 16 * t, r, a.rows - 16 * n);
        else load_v<D>(buf[n & 3], a.row0 + 16 * (n - MT) * D + (D / 8) * r, t, a.rows - 16 * (n - MT));
    };

    long long unit = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (unit >= units) return;   // whole warps leave; no block barrier follows
    At a = at(unit);
#pragma unroll
    for (int n = 0; n < 4; ++n) load_tile(n, a);
    for (;;) {
        const long long next = unit + step;
        const bool more = next < units;
        At an = a;
        if (more) an = at(next);
        const size_t crow = (size_t)a.bg * p.nL + a.c;
        const float sc = __ldg(ks + crow);

        // the landmark query's pieces: lane (r, t) holds piece r at d = 64 s + 16 t .. + 15
        uint32_t ub[KS][2];
        float fu;
        {
            float x[D / 64][16], m = 0.f;
            const Tin *ur = U + crow * D + 16 * t;
#pragma unroll
            for (int s = 0; s < D / 64; ++s) {
                load8(ur + 64 * s, x[s]);
                load8(ur + 64 * s + 8, x[s] + 8);
#pragma unroll
                for (int e = 0; e < 16; ++e) m = fmaxf(m, fabsf(x[s][e]));
            }
            m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
            m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
            const int sh = min(7 - ((int)(__float_as_uint(m) >> 23) - 127), 120);
            const float f = exp2_int(sh);
            fu = scale * exp2_int(-sh) * sc;
#pragma unroll
            for (int s = 0; s < D / 64; ++s)
#pragma unroll
                for (int w = 0; w < 4; ++w)
                    ub[2 * s + w / 2][w & 1] = piece_pair(x[s][4 * w] * f, x[s][4 * w + 1] * f, r) |
                                               (piece_pair(x[s][4 * w + 2] * f, x[s][4 * w + 3] * f, r) << 16);
        }

        // logits of rows r and r + 8 of each tile
        float x[MT][2];
#pragma unroll
        for (int m = 0; m < MT; m += 2) {
            float d[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
            for (int kk = 0; kk < KS; ++kk)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const uint32_t *w = buf[(m + u) & 3];
                    mma_e4m3(d[u], w[2 * kk], w[2 * KS + 2 * kk], w[2 * kk + 1], w[2 * KS + 2 * kk + 1], ub[kk][0], ub[kk][1]);
                }
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int n = m + u + 4;
                if (n < 2 * MT) load_tile(n, a);
                else if (more) load_tile(n - 2 * MT, an);
                x[m + u][0] = sum_t(fmaf(d[u][1], f1, d[u][0] * f0)) * fu;
                x[m + u][1] = sum_t(fmaf(d[u][3], f1, d[u][2] * f0)) * fu;
            }
        }

        // p (unnormalised, at most 1), its sum z, and y = sum p ln p
        float mx = -INFINITY, z = 0.f, y = 0.f;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                if (16 * m + 8 * h + r < a.rows) mx = fmaxf(mx, x[m][h]);
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float d = x[m][h] - mx;
                const float w = 16 * m + 8 * h + r < a.rows ? expf(d) : 0.f;
                z += w;
                y += w == 0.f ? 0.f : w * d;
                x[m][h] = w;
            }
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
            z += __shfl_xor_sync(0xFFFFFFFFu, z, o);
            y += __shfl_xor_sync(0xFFFFFFFFu, y, o);
        }

        // sum of p k: tile (w, hw) rows r / r + 8 are d = (D / 8) r + 4 w + 2 hw (+ 1)
        float o[DT][4];
#pragma unroll
        for (int i = 0; i < DT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
#pragma unroll
        for (int m = 0; m < MT; m += 2) {
            uint32_t pb[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                // keys 2t, 2t + 1 of the tile's first and second eight rows
                float v[4];
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    v[q] = __shfl_sync(0xFFFFFFFFu, x[m + u][q >> 1], 4 * (2 * t + (q & 1))) * 255.0f;
                pb[u] = piece_pair(v[0], v[1], r) | (piece_pair(v[2], v[3], r) << 16);
            }
            const uint32_t *v0 = buf[(MT + m) & 3], *v1 = buf[(MT + m + 1) & 3];
#pragma unroll
            for (int w = 0; w < W; ++w) {
                uint32_t ta[4], tb[4];
                transpose4(v0[w], v0[W + w], v0[2 * W + w], v0[3 * W + w], ta);
                transpose4(v1[w], v1[W + w], v1[2 * W + w], v1[3 * W + w], tb);
                mma_e4m3(o[2 * w], ta[0], ta[1], tb[0], tb[1], pb[0], pb[1]);
                mma_e4m3(o[2 * w + 1], ta[2], ta[3], tb[2], tb[3], pb[0], pb[1]);
            }
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int n = MT + m + u + 4;
                if (n < 2 * MT) load_tile(n, a);
                else if (more) load_tile(n - 2 * MT, an);
            }
        }
        const float inv = 1.0f / z, g = inv * sc * (1.0f / 255.0f);
#pragma unroll
        for (int w = 0; w < W; ++w) {
            float v[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float(&e)[4] = o[2 * w + (q >> 1)];
                v[q] = sum_t(fmaf(e[2 * (q & 1) + 1], f1, e[2 * (q & 1)] * f0)) * g;
            }
            if ((w & 3) == t) store4(L + crow * D + (D / 8) * r + 4 * w, v[0], v[1], v[2], v[3]);
        }
        if (beta && lane == 0) beta[crow] = logf(z) - y * inv;
        if (!more) return;
        unit = next;
        a = an;
    }
}

template <typename Tin, int D, int C>
cudaError_t launch_t(const Cache8 &c, float scale, const uint8_t *K8, const float *ks, const void *U, void *L, float *beta,
                     int c0, int c1, int t_end, cudaStream_t s)
{
    const long long units = (long long)c.B * c.Hkv * (c1 - c0), blocks = (units + kWarps - 1) / kWarps;
    const unsigned grid = (unsigned)(blocks < 148 * kBlocksPerSm ? blocks : 148 * kBlocksPerSm);
    landmarks8_kernel<Tin, D, C><<<grid, 32 * kWarps, 0, s>>>(K8, ks, static_cast<const Tin *>(U), static_cast<Tin *>(L), beta,
                                                              c, scale, c0, c1 - c0, t_end);
    return cudaGetLastError();
}

template <typename Tin, int D>
cudaError_t launch_c(const Cache8 &c, float scale, const uint8_t *K8, const float *ks, const void *U, void *L, float *beta,
                     int c0, int c1, int t_end, cudaStream_t s)
{
    auto *f = c.C == 32 ? launch_t<Tin, D, 32> : c.C == 64 ? launch_t<Tin, D, 64> : launch_t<Tin, D, 128>;
    return f(c, scale, K8, ks, U, L, beta, c0, c1, t_end, s);
}

}  // namespace

cudaError_t launch_landmarks8(const Cache8 &c, hils_dtype in, float scale, const uint8_t *K8, const float *ks,
                              const void *U, void *L, float *beta, int c0, int c1, int t_end, cudaStream_t s)
{
    auto *f = in == HILS_BF16 ? (c.d == 128 ? launch_c<__nv_bfloat16, 128> : launch_c<__nv_bfloat16, 64>)
                              : (c.d == 128 ? launch_c<float, 128> : launch_c<float, 64>);
    return f(c, scale, K8, ks, U, L, beta, c0, c1, t_end, s);
}

}  // namespace hils
