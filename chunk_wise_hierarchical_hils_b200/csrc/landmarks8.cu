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
// than the one before, in the columns the product has anyway (column c holds piece c).  For float32 results six pieces
// hold 24 bits (u relative to the row's largest, p to the chunk's largest); for bf16 ones two pieces hold a bf16 u
// and three the 11 bits of p (2^-12 of its value, where the result's own rounding is 2^-9).  The columns' sums meet in
// float32.  A lane splits the values it holds and the pieces change places in shared memory: splitting the row in
// every lane that needs one piece of it took three times the instructions (2129 a chunk against 750).
#include "cache8.h"
#include "common.cuh"
#include "tiles8.cuh"

namespace hils {
namespace {

using namespace t8;

constexpr int kWarps = 4;
constexpr int kBlocksPerSm = 3;

// The pieces of two values below 256 in magnitude: o[c] holds the e4m3 bytes of 16^c times what pieces 0 .. c - 1 leave.
template <int N>
__device__ __forceinline__ void pieces(float a, float b, uint32_t (&o)[N])
{
    static_assert(N == 2 || N == 3 || N == 6, "pieces of one or two f16 values");
    uint32_t h = pack_f16(a, b);
    const float2 y = unpack_f16(h);
#pragma unroll
    for (int c = 0; c < (N < 3 ? N : 3); ++c) {
        o[c] = f16x2_to_e4m3x2(h);
        h = e4m3_rest<16>(h, o[c]);
    }
    if constexpr (N == 6) {
        h = pack_f16((a - y.x) * 4096.0f, (b - y.y) * 4096.0f);
#pragma unroll
        for (int c = 3; c < 6; ++c) {
            o[c] = f16x2_to_e4m3x2(h);
            h = e4m3_rest<16>(h, o[c]);
        }
    }
}

// Four consecutive elements, raw until they are used.
__device__ __forceinline__ void widen4(float4 v, float *o) { o[0] = v.x; o[1] = v.y; o[2] = v.z; o[3] = v.w; }
__device__ __forceinline__ void widen4(uint2 v, float *o)
{
    o[0] = __uint_as_float(v.x << 16); o[1] = __uint_as_float(v.x & 0xFFFF0000u);
    o[2] = __uint_as_float(v.y << 16); o[3] = __uint_as_float(v.y & 0xFFFF0000u);
}
template <typename T>
struct Raw4 { typedef uint2 type; };
template <>
struct Raw4<float> { typedef float4 type; };

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

// PART: the one chunk that t_end ends inside; otherwise whole chunks.
template <typename Tin, int D, int C, bool PART>
__global__ void __launch_bounds__(32 * kWarps, kBlocksPerSm)
    landmarks8_kernel(const uint8_t *__restrict__ K8, const float *__restrict__ ks, const Tin *__restrict__ U,
                      Tin *__restrict__ L, float *__restrict__ beta, Cache8 p, float scale, int c0, int span, int t_end)
{
    constexpr int MT = C / 16, KS = D / 32, DT = D / 16, WORDS = D / 8, W = D / 32;
    constexpr bool F32 = sizeof(Tin) == 4;
    constexpr int NU = F32 ? 6 : 2, NP = F32 ? 6 : 3;   // pieces of u and of p
    typedef typename Raw4<Tin>::type Raw;
    // pieces on their way between lanes: u's as [word of the row][piece] (a word: four values), p's as [tile][piece][lane t]
    __shared__ __align__(16) uint32_t s_u[kWarps][D / 4][8];
    __shared__ uint32_t s_p[kWarps][MT][8][4];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, t = lane & 3;
    const unsigned units = (unsigned)(p.B * p.Hkv) * (unsigned)span, step = gridDim.x * kWarps;
    const float f0 = exp2_int(-8 * t), f1 = exp2_int(-8 * t - 4);   // worth of pieces 2t and 2t + 1

    unsigned unit = blockIdx.x * kWarps + warp;
    if (unit >= units) return;   // whole warps leave; no block barrier follows
    for (int i = lane; i < D / 4 * 8; i += 32) (&s_u[warp][0][0])[i] = 0u;   // columns without a piece stay zero
    for (int i = lane; i < MT * 32; i += 32) (&s_p[warp][0][0][0])[i] = 0u;

    struct At {
        size_t crow;
        int rows;
        const uint8_t *row0;
    };
    auto at = [&](unsigned u) {
        At a;
        const unsigned bg = u / (unsigned)span;
        const int c = c0 + (int)(u - bg * (unsigned)span);
        a.crow = (size_t)bg * p.nL + c;
        a.rows = PART ? t_end - c * C : C;
        a.row0 = K8 + ((size_t)bg * p.T + (size_t)c * C) * D;
        return a;
    };
    uint32_t buf[4][WORDS];
    auto load_tile = [&](int n, const At &a) {
        if (n < MT) load_k<D, PART>(buf[n & 3], a.row0 + 16 * n * D + 16 * t, r, a.rows - 1 - 16 * n);
        else load_v<D, PART>(buf[n & 3], a.row0 + 16 * (n - MT) * D + (D / 8) * r, t, a.rows - 1 - 16 * (n - MT));
    };
    // the landmark query: lane (r, t) takes its word r of column block t (d = 64 (r / 4) + 16 t + 4 (r % 4))
    const int ud = (64 * (r >> 2) + 16 * t + 4 * (r & 3)) % D;   // d = 64: lanes of r >= 4 repeat the others
    auto load_u = [&](const At &a) { return *reinterpret_cast<const Raw *>(U + a.crow * D + ud); };

    At a = at(unit);
#pragma unroll
    for (int n = 0; n < 4; ++n) load_tile(n, a);
    Raw ur = load_u(a);
    float sc = __ldg(ks + a.crow);
    for (;;) {
        const bool more = units - unit > step;
        const At an = at(more ? unit + step : unit);   // behind the last chunk its own tiles again: no branch around a load

        // the landmark query's pieces: lane (r, t) holds piece r at d = 64 s + 16 t .. + 15
        uint32_t ub[KS][2];
        float fu;
        {
            float u[4];
            widen4(ur, u);
            const float m = warp_max(fmaxf(fmaxf(fabsf(u[0]), fabsf(u[1])), fmaxf(fabsf(u[2]), fabsf(u[3]))));
            const int sh = min(7 - ((int)(__float_as_uint(m) >> 23) - 127), 120);
            const float f = exp2_int(sh);
            fu = scale * exp2_int(-sh) * sc;
            uint32_t pa[NU], pb[NU];
            pieces(u[0] * f, u[1] * f, pa);
            pieces(u[2] * f, u[3] * f, pb);
            __syncwarp();
            if (4 * r < D / 4)
#pragma unroll
                for (int c = 0; c < NU; ++c) s_u[warp][4 * r + t][c] = pa[c] | (pb[c] << 16);
            __syncwarp();
#pragma unroll
            for (int w = 0; w < 2 * KS; ++w) ub[w >> 1][w & 1] = s_u[warp][4 * w + t][r];
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
                else load_tile(n - 2 * MT, an);
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
                if (!PART || 16 * m + 8 * h + r < a.rows) mx = fmaxf(mx, x[m][h]);
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float d = x[m][h] - mx;
                const float w = !PART || 16 * m + 8 * h + r < a.rows ? expf(d) : 0.f;
                z += w;
                y += w == 0.f ? 0.f : w * d;
                x[m][h] = w;
            }
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
            z += __shfl_xor_sync(0xFFFFFFFFu, z, o);
            y += __shfl_xor_sync(0xFFFFFFFFu, y, o);
        }

        // p's pieces: the four lanes of a row hold the same values, lane t splits those of tiles t, t + 4 (rows r, r + 8).
        // The word of lane t holds rows 2t, 2t + 1, 2t + 8, 2t + 9, as a V tile's columns do.
#pragma unroll
        for (int m0 = 0; m0 < MT; m0 += 4) {
            float v0 = x[m0][0], v1 = x[m0][1];
#pragma unroll
            for (int q = 1; q < 4; ++q)
                if (m0 + q < MT && t == q) {
                    v0 = x[m0 + q][0];
                    v1 = x[m0 + q][1];
                }
            uint32_t pc[NP];
            pieces(v0 * 255.0f, v1 * 255.0f, pc);
            if (m0 + t < MT) {
                uint8_t *b = reinterpret_cast<uint8_t *>(&s_p[warp][m0 + t][0][r >> 1]) + (r & 1);
#pragma unroll
                for (int c = 0; c < NP; ++c) {
                    b[16 * c] = (uint8_t)pc[c];
                    b[16 * c + 2] = (uint8_t)(pc[c] >> 8);
                }
            }
        }
        __syncwarp();

        // sum of p k: tile (w, hw) rows r / r + 8 are d = (D / 8) r + 4 w + 2 hw (+ 1)
        float o[DT][4];
#pragma unroll
        for (int i = 0; i < DT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
#pragma unroll
        for (int m = 0; m < MT; m += 2) {
            const uint32_t b0 = s_p[warp][m][r][t], b1 = s_p[warp][m + 1][r][t];
            const uint32_t *v0 = buf[(MT + m) & 3], *v1 = buf[(MT + m + 1) & 3];
#pragma unroll
            for (int w = 0; w < W; ++w) {
                uint32_t ta[4], tb[4];
                transpose4(v0[w], v0[W + w], v0[2 * W + w], v0[3 * W + w], ta);
                transpose4(v1[w], v1[W + w], v1[2 * W + w], v1[3 * W + w], tb);
                mma_e4m3(o[2 * w], ta[0], ta[1], tb[0], tb[1], b0, b1);
                mma_e4m3(o[2 * w + 1], ta[2], ta[3], tb[2], tb[3], b0, b1);
            }
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int n = MT + m + u + 4;
                if (n < 2 * MT) load_tile(n, a);
                else load_tile(n - 2 * MT, an);
            }
            if (m == 0) ur = load_u(an);
        }
        const float inv = 1.0f / z, g = inv * sc * (1.0f / 255.0f);
        sc = __ldg(ks + an.crow);

        // the columns' sums: v[4 w + q] is this lane's share of d = (D / 8) r + 4 w + q; lane t keeps the sums of w = t
        float v[4 * W];
#pragma unroll
        for (int i = 0; i < 4 * W; ++i) {
            const float(&e)[4] = o[i >> 1];
            v[i] = fmaf(e[2 * (i & 1) + 1], f1, e[2 * (i & 1)] * f0);
        }
        if constexpr (W == 4) {
            float h[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {   // w = t mod 2 stay
                const int w = (i >> 2) * 2, q = i & 3;
                const float keep = (t & 1) ? v[4 * (w + 1) + q] : v[4 * w + q];
                const float give = (t & 1) ? v[4 * w + q] : v[4 * (w + 1) + q];
                h[i] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, 1);
            }
            float k4[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float keep = (t & 2) ? h[4 + q] : h[q], give = (t & 2) ? h[q] : h[4 + q];
                k4[q] = (keep + __shfl_xor_sync(0xFFFFFFFFu, give, 2)) * g;
            }
            store4(L + a.crow * D + (D / 8) * r + 4 * t, k4[0], k4[1], k4[2], k4[3]);
        } else {
#pragma unroll
            for (int i = 0; i < 4 * W; ++i) v[i] = sum_t(v[i]) * g;
#pragma unroll
            for (int w = 0; w < W; ++w)
                if (t == w) store4(L + a.crow * D + (D / 8) * r + 4 * w, v[4 * w], v[4 * w + 1], v[4 * w + 2], v[4 * w + 3]);
        }
        if (beta && lane == 0) beta[a.crow] = logf(z) - y * inv;
        if (!more) return;
        unit += step;
        a = an;
    }
}

template <typename Tin, int D, int C>
cudaError_t launch_t(const Cache8 &c, float scale, const uint8_t *K8, const float *ks, const void *U, void *L, float *beta,
                     int c0, int c1, int t_end, cudaStream_t s)
{
    auto run = [&](auto kern, int first, int span) {
        const long long units = (long long)c.B * c.Hkv * span, blocks = (units + kWarps - 1) / kWarps;
        const unsigned grid = (unsigned)(blocks < 148 * kBlocksPerSm ? blocks : 148 * kBlocksPerSm);
        kern<<<grid, 32 * kWarps, 0, s>>>(K8, ks, static_cast<const Tin *>(U), static_cast<Tin *>(L), beta, c, scale, first,
                                          span, t_end);
        return cudaGetLastError();
    };
    const int whole = t_end / C;   // chunks before the one that t_end ends inside
    cudaError_t e = cudaSuccess;
    if (c0 < whole) e = run(landmarks8_kernel<Tin, D, C, false>, c0, (c1 < whole ? c1 : whole) - c0);
    if (e == cudaSuccess && c1 > whole) e = run(landmarks8_kernel<Tin, D, C, true>, whole, 1);
    return e;
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
