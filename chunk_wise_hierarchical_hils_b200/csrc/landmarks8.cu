// landmarks8.cu -- landmark generation from the keys of the 8-bit cache.
//
// "Hierarchical Sparse Attention Done Right" (arXiv 2607.02980v1), Sec. 3, "Linear surrogate for chunk mass": the
// landmark query u attends over its chunk's keys; with keys k_t = s_c e_t (e_t the e4m3 rows, s_c the chunk's
// scale) the logits are scale s_c <u, e_t>, the landmark is s_c sum_t p_t e_t, and the entropy of p is the chunk's
// bias.
//
// Every key byte is read once from HBM and used in two products (logits, sum), so the kernel is bound by HBM as long as
// the products stay cheap: one warp per chunk, mma.sync tiles of f16 (e4m3 is exact in it) read from two chunk buffers
// in shared memory, one in use and one being filled.  (mma.sync has an e4m3 form, but on this GPU it runs as
// conversions and two f16 products: 1134 instructions a chunk against 735 in the f16 form.)
//
// Numbers.  The other operand, one row of u or p, is float32, scaled by a power of two (u so that its largest lies in
// [2^14, 2^15), p by 2^15): its f16 value is column 0 of the product and, for float32 results, what that leaves is column
// 1 (2^-22 of the value together).  bf16 landmark queries are exact in column 0 down to 2^-31 of their largest, and p's half
// step there, 2^-11, is below that of the bf16 result (2^-8).  Sums are float32.
#include "cache8.h"
#include "common.cuh"
#include "sm100.cuh"
#include "tiles8.cuh"

namespace hils {
namespace {

using namespace t8;

// Warps a block has, and blocks an SM: two chunks a warp, of 227 KB.
constexpr int warps_of(int chunk_bytes) { return chunk_bytes == 16384 ? 6 : 4; }
constexpr int blocks_of(int chunk_bytes) { return chunk_bytes == 16384 ? 1 : chunk_bytes == 8192 ? 3 : 4; }

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

// What f16 leaves of two values.
__device__ __forceinline__ uint32_t rest_f16(float a, float b, uint32_t h)
{
    const float2 y = unpack_f16(h);
    return pack_f16(a - y.x, b - y.y);
}

// PART: the one chunk that t_end ends inside; otherwise whole chunks.
template <typename Tin, int D, int C, bool PART>
__global__ void __launch_bounds__(32 * warps_of(C * D), blocks_of(C * D))
    landmarks8_kernel(const uint8_t *__restrict__ K8, const float *__restrict__ ks, const Tin *__restrict__ U,
                      Tin *__restrict__ L, float *__restrict__ beta, Cache8 p, float scale, int c0, int span, int t_end)
{
    constexpr int MT = C / 16, KS = D / 16, W = warps_of(C * D);
    constexpr bool F32 = sizeof(Tin) == 4;
    constexpr float PTOP = 32768.0f;
    typedef typename Raw4<Tin>::type Raw;
    extern __shared__ __align__(128) unsigned char s_chunks[];   // [warp][2][C][D]
    // the landmark query's columns 0, 1 (and 2: zeros, for all the others): [column][t][word: two values]
    __shared__ __align__(16) uint32_t s_u[W][3][4][2 * KS + 4];
    __shared__ __align__(16) float s_out[W][D];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, t = lane & 3;
    const unsigned units = (unsigned)(p.B * p.Hkv) * (unsigned)span, step = gridDim.x * W;
    const uint32_t ring = sm100::smem_addr(s_chunks) + (uint32_t)warp * (2 * C * D);

    unsigned unit = blockIdx.x * W + warp;
    if (unit >= units) return;   // whole warps leave; no block barrier follows
    if (r < 2 * KS / 4)   // columns without a value stay zero
#pragma unroll
        for (int c = 1; c < 3; ++c) *reinterpret_cast<uint4 *>(&s_u[warp][c][t][4 * r]) = make_uint4(0u, 0u, 0u, 0u);

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
    auto load_chunk = [&](uint32_t slot, const At &a) { load_rows<D, C, PART>(ring + slot * (C * D), a.row0, a.rows - 1); };
    // the landmark query: lane (r, t) takes d = 16 r + 4 t .. (d = 64: lanes of r >= 4 repeat the others)
    const int ud = (16 * r + 4 * t) % D;
    auto load_u = [&](const At &a) { return *reinterpret_cast<const Raw *>(U + a.crow * D + ud); };

    At a = at(unit);
    uint32_t slot = 0;
    load_chunk(0, a);
    cp_commit();
    Raw ur = load_u(a);
    float sc = __ldg(ks + a.crow);
    for (;;) {
        const bool more = units - unit > step;
        const At an = at(more ? unit + step : unit);
        if (more) load_chunk(slot ^ 1u, an);
        cp_commit();

        // the landmark query: lane (r, t) holds column r at d = 16 c + 4 t .. + 3
        uint32_t ub[KS][2];
        float fu;
        {
            float u[4];
            widen4(ur, u);
            const float m = __uint_as_float(__reduce_max_sync(
                0xFFFFFFFFu, __float_as_uint(fmaxf(fmaxf(fabsf(u[0]), fabsf(u[1])), fmaxf(fabsf(u[2]), fabsf(u[3]))))));
            const int sh = min(14 - ((int)(__float_as_uint(m) >> 23) - 127), 120);
            const float f = exp2_int(sh);
            fu = scale * 1.4426950408889634f * exp2_int(-sh) * sc;   // logits in powers of two
            const uint32_t h0 = pack_f16(u[0] * f, u[1] * f), h1 = pack_f16(u[2] * f, u[3] * f);
            __syncwarp();
            if (r < KS) {
                *reinterpret_cast<uint2 *>(&s_u[warp][0][t][2 * r]) = make_uint2(h0, h1);
                if constexpr (F32)
                    *reinterpret_cast<uint2 *>(&s_u[warp][1][t][2 * r]) =
                        make_uint2(rest_f16(u[0] * f, u[1] * f, h0), rest_f16(u[2] * f, u[3] * f, h1));
            }
            __syncwarp();
#pragma unroll
            for (int k = 0; k < KS; k += 2) {
                const uint4 v = *reinterpret_cast<const uint4 *>(&s_u[warp][min(r, 2)][t][2 * k]);
                ub[k][0] = v.x; ub[k][1] = v.y; ub[k + 1][0] = v.z; ub[k + 1][1] = v.w;
            }
        }

        cp_wait<1>();
        __syncwarp();
        const uint32_t tile0 = ring + slot * (C * D);

        // logits of the keys that rows r of both halves of a tile stand for: columns 0 and 1 are lane t = 0's (the others'
        // are zeros and stay unused)
        float x[MT][2];
#pragma unroll
        for (int m = 0; m < MT; m += 2) {
            float d[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
            uint32_t w[2][KS][2];
            read_keys<D>(tile0 + m * (16 * D), w[0]);
            read_keys<D>(tile0 + (m + 1) * (16 * D), w[1]);
#pragma unroll
            for (int c = 0; c < KS; ++c)
#pragma unroll
                for (int u = 0; u < 2; ++u) mma_bytes(d[u], w[u][c][0], w[u][c][1], ub[c][0], ub[c][1]);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                x[m + u][0] = (d[u][0] + d[u][1]) * fu;
                x[m + u][1] = (d[u][2] + d[u][3]) * fu;
            }
        }

        // p (unnormalised, at most 1), its sum z, and y = sum p log2 p
        float mx = -INFINITY, z = 0.f, y = 0.f;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                if (!PART || 16 * m + key_row(r, h) < a.rows) mx = fmaxf(mx, x[m][h]);
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float d = x[m][h] - mx;
                const float w = !PART || 16 * m + key_row(r, h) < a.rows ? sm100::ex2_approx(d) : 0.f;
                z += w;
                y = fmaf(w, fmaxf(d, -200.0f), y);   // w is 0 there
                x[m][h] = w;
            }
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
            z += __shfl_xor_sync(0xFFFFFFFFu, z, o);
            y += __shfl_xor_sync(0xFFFFFFFFu, y, o);
        }

        // sum of p k: tile c, rows r and r + 8 are d = 16 c + r (+ 8)
        float o[KS][4];
#pragma unroll
        for (int i = 0; i < KS; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            // column r of p for keys 4t, 4t + 1 and 4t + 2, 4t + 3 of the tile
            uint32_t b[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float v = x[m][h] * PTOP;
                uint32_t c = pack_f16(v, 0.f);
                if constexpr (F32) c = pack_f16(v, v - unpack_f16(c).x);
                b[h] = movmatrix_t(t == 0 ? c : 0u);
            }
#pragma unroll
            for (int c = 0; c < KS; c += 2) {
                uint32_t w[2][2];
                read_values<D>(tile0 + m * (16 * D), c, w);
                mma_bytes(o[c], w[0][0], w[0][1], b[0], b[1]);
                mma_bytes(o[c + 1], w[1][0], w[1][1], b[0], b[1]);
            }
        }
        ur = load_u(an);
        const float inv = 1.0f / z, g = inv * sc * (1.0f / PTOP);
        sc = __ldg(ks + an.crow);
        if (t == 0) {
#pragma unroll
            for (int c = 0; c < KS; ++c) {
                s_out[warp][16 * c + r] = (o[c][0] + o[c][1]) * g;
                s_out[warp][16 * c + r + 8] = (o[c][2] + o[c][3]) * g;
            }
        }
        __syncwarp();   // also: every lane has read the chunk, its buffer may be filled again
        if (4 * lane < D) {
            const float4 v = *reinterpret_cast<const float4 *>(&s_out[warp][4 * lane]);
            store4(L + a.crow * D + 4 * lane, v);
        }
        if (beta && lane == 0) beta[a.crow] = logf(z) - y * inv * 0.6931471805599453f;
        if (!more) return;
        unit += step;
        a = an;
        slot ^= 1u;
    }
}

template <typename Tin, int D, int C>
cudaError_t launch_t(const Cache8 &c, float scale, const uint8_t *K8, const float *ks, const void *U, void *L, float *beta,
                     int c0, int c1, int t_end, cudaStream_t s)
{
    auto run = [&](auto kern, int first, int span) {
        constexpr int W = warps_of(C * D), smem = W * 2 * C * D;
        const long long units = (long long)c.B * c.Hkv * span, blocks = (units + W - 1) / W, most = 148 * blocks_of(C * D);
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        kern<<<(unsigned)(blocks < most ? blocks : most), 32 * W, smem, s>>>(
            K8, ks, static_cast<const Tin *>(U), static_cast<Tin *>(L), beta, c, scale, first, span, t_end);
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
