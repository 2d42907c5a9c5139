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

// 16 bytes of rows as they are loaded (eight bf16 or four float32 elements), with what append asks of them: the largest
// magnitude so far as an ordered integer (infinities and NaN above every number), the same without those, the values.
struct Rows8 {
    static constexpr int N = 8;
    typedef uint2 Bytes;
    uint4 v;
    __device__ __forceinline__ const uint32_t *w() const { return reinterpret_cast<const uint32_t *>(&v); }
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { v = __ldg(reinterpret_cast<const uint4 *>(p)); }
    __device__ __forceinline__ uint32_t top(uint32_t m) const   // two running maxima of 16 bits
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) m = __vmaxu2(m, w()[i] & 0x7FFF7FFFu);
        return m;
    }
    static __device__ __forceinline__ uint32_t bits(uint32_t m) { return max(m << 16, m & 0xFFFF0000u); }   // as float32 bits
    __device__ __forceinline__ void values(float *x) const { unpack_bf16x8(v, x); }
    static __device__ __forceinline__ Bytes bytes(const float *x)
    {
        return make_uint2(to_e4m3x4(x[0], x[1], x[2], x[3]), to_e4m3x4(x[4], x[5], x[6], x[7]));
    }
};

struct Rows4 {
    static constexpr int N = 4;
    typedef uint32_t Bytes;
    float4 v;
    __device__ __forceinline__ void load(const float *p) { v = __ldg(reinterpret_cast<const float4 *>(p)); }
    __device__ __forceinline__ uint32_t top(uint32_t m) const
    {
        const uint32_t a = max(__float_as_uint(v.x) & 0x7FFFFFFFu, __float_as_uint(v.y) & 0x7FFFFFFFu);
        return max(m, max(a, max(__float_as_uint(v.z) & 0x7FFFFFFFu, __float_as_uint(v.w) & 0x7FFFFFFFu)));
    }
    static __device__ __forceinline__ uint32_t bits(uint32_t m) { return m; }
    __device__ __forceinline__ void values(float *x) const { x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w; }
    static __device__ __forceinline__ Bytes bytes(const float *x) { return to_e4m3x4(x[0], x[1], x[2], x[3]); }
};

template <typename T> struct RowsOf { typedef Rows8 type; };
template <> struct RowsOf<float> { typedef Rows4 type; };

// Append.  One block per (b, kv-head, chunk touched, side), eight pieces of 16 bytes a thread: the new rows are
// read once and stay in registers, as loaded, between the maximum and the conversion, so the pass moves each byte once
// and is bound by HBM (or, for a decode step's single rows, by its latency).  The maximum is taken on the numbers' bits,
// two bf16 at a time: with float comparisons that leave infinities and NaN out of every element the pass took 48.6 us on
// four 8K prompts; now 30.7 us (201 MB at the measured copy rate).  They are left out by a second look at the chunks
// that hold one.
template <typename Tin, int D>
__global__ void append_kernel(const Tin *__restrict__ K, const Tin *__restrict__ V, uint8_t *__restrict__ K8,
                              uint8_t *__restrict__ V8, float *__restrict__ ks, float *__restrict__ vs, Cache8 p, int t0,
                              int t1, int c0, int nb)
{
    typedef typename RowsOf<Tin>::type Rows;
    constexpr int N = Rows::N, UNITS = 8;   // blockDim.x = C * D / (8 N)
    __shared__ uint32_t s_max[16], s_fin[16];
    const int tid = threadIdx.x, nt = blockDim.x;
    const int side = blockIdx.x & 1;
    const unsigned u = blockIdx.x >> 1, bg = u / (unsigned)nb;
    const int c = c0 + (int)(u - bg * (unsigned)nb);
    const int r0 = max(t0 - c * p.C, 0);                               // the chunk's rows [r0, r1) are new
    const int r1 = (int)min((long long)t1 - (long long)c * p.C, (long long)p.C);
    // rows of the chunk, in the source and in the cache
    const Tin *src = (side ? V : K) + (size_t)bg * (size_t)(t1 - t0) * D + ((long long)c * p.C - t0) * D;
    uint8_t *dst = (side ? V8 : K8) + ((size_t)bg * p.T + (size_t)c * p.C) * D;
    float *scale = (side ? vs : ks) + (size_t)bg * p.nL + c;
    const float old = r0 > 0 ? *scale : 0.f;

    Rows x[UNITS];
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < UNITS; ++i) {
        const int e = (i * nt + tid) * N, row = e / D;
        if (row >= r0 && row < r1) x[i].load(src + e);
    }
#pragma unroll
    for (int i = 0; i < UNITS; ++i) {
        const int row = (i * nt + tid) * N / D;
        if (row >= r0 && row < r1) m = x[i].top(m);
    }
    uint32_t top = __reduce_max_sync(0xFFFFFFFFu, Rows::bits(m));
    if ((tid & 31) == 0) s_max[tid >> 5] = top;
    __syncthreads();
    for (int w = 0; w < nt / 32; ++w) top = max(top, s_max[w]);
    if (top >= 0x7F800000u) {
        // an infinity or NaN among the rows (the same for the whole block): the largest of the others
        float f = 0.f;
#pragma unroll
        for (int i = 0; i < UNITS; ++i) {
            const int row = (i * nt + tid) * N / D;
            if (row >= r0 && row < r1) {
                float v[N];
                x[i].values(v);
#pragma unroll
                for (int j = 0; j < N; ++j) f = fmaxf(f, fabsf(v[j]) <= FLT_MAX ? fabsf(v[j]) : 0.f);
            }
        }
        top = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(f));
        if ((tid & 31) == 0) s_fin[tid >> 5] = top;
        __syncthreads();
        for (int w = 0; w < nt / 32; ++w) top = max(top, s_fin[w]);
    }
    const int e2 = scale_exponent(__uint_as_float(top));
    float s = exp2_int(e2), inv = exp2_int(-e2);
    if (r0 > 0) {
        if (s > old) {
            // the scale grows: the rows already in the chunk go over to it
            const float f = old * inv;
#pragma unroll
            for (int i = 0; i < UNITS * N / 16; ++i) {
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
        const int e = (i * nt + tid) * N, row = e / D;
        if (row >= r0 && row < r1) {
            float v[N];
            x[i].values(v);
#pragma unroll
            for (int j = 0; j < N; ++j) v[j] *= inv;
            *reinterpret_cast<typename Rows::Bytes *>(dst + e) = Rows::bytes(v);
        }
    }
    if (tid == 0) *scale = s;
}

// Read back.  A thread takes kPieces pieces of what makes 16 bytes of the result (eight bf16 or four float32 elements),
// a block's threads in a row, so that loads and stores are whole sectors; one pass, bound by HBM (128K tokens of eight
// kv-heads, 805 MB: 120 us, the copy rate).
constexpr int kPieces = 4;

__device__ __forceinline__ void store_values(float *out, uint32_t b, float s)
{
    float v[4];
    e4m3x4_to_float(b, v);
    *reinterpret_cast<float4 *>(out) = make_float4(v[0] * s, v[1] * s, v[2] * s, v[3] * s);
}

// A product has up to 28 bits (4 of the value) and bf16 keeps 8: it is rounded once where float32 holds it exactly, which
// is so for scales whose last four bits are zero (what an append writes has none set), down to 2^-117 (2^-9 of which is
// float32's smallest normal number).  With any other scale it is taken in 64 bits, behind a branch: chosen element by
// element both were computed (128K tokens 169 us against 120).
__device__ __forceinline__ bool exact_products(float s)
{
    const uint32_t u = __float_as_uint(s);
    return (u & 15u) == 0u && ((u >> 23) & 255u) >= 127u - 117u;
}

__device__ __forceinline__ void store_values(__nv_bfloat16 *out, uint2 b, float s)
{
    float v[8];
    e4m3x4_to_float(b.x, v);
    e4m3x4_to_float(b.y, v + 4);
    uint4 u;
    uint32_t *w = reinterpret_cast<uint32_t *>(&u);
    if (exact_products(s)) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const __nv_bfloat162 t = __floats2bfloat162_rn(v[2 * j] * s, v[2 * j + 1] * s);
            w[j] = *reinterpret_cast<const uint32_t *>(&t);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const __nv_bfloat162 t = __halves2bfloat162(__double2bfloat16((double)v[2 * j] * s),
                                                        __double2bfloat16((double)v[2 * j + 1] * s));
            w[j] = *reinterpret_cast<const uint32_t *>(&t);
        }
    }
    *reinterpret_cast<uint4 *>(out) = u;
}

template <typename Tout, int D>
__global__ void __launch_bounds__(256)
    read_kernel(const uint8_t *__restrict__ K8, const uint8_t *__restrict__ V8, const float *__restrict__ ks,
                const float *__restrict__ vs, Tout *__restrict__ K, Tout *__restrict__ V, Cache8 p, int t0, long long units)
{
    constexpr int N = 16 / sizeof(Tout);
    typedef typename RowsOf<Tout>::type::Bytes Bytes;
    const int side = blockIdx.z;
    const size_t bg = blockIdx.y;
    const uint8_t *src = (side ? V8 : K8) + (bg * p.T + (size_t)t0) * D;
    const float *scale = (side ? vs : ks) + bg * p.nL;
    Tout *dst = (side ? V : K) + bg * (size_t)units * N;
    const long long u0 = (long long)blockIdx.x * (256 * kPieces) + threadIdx.x;
    Bytes b[kPieces];
    float s[kPieces];
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
        const long long u = u0 + 256 * i;
        if (u < units) {
            b[i] = __ldg(reinterpret_cast<const Bytes *>(src) + u);
            s[i] = __ldg(scale + (t0 + (int)(u / (D / N))) / p.C);
        }
    }
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
        const long long u = u0 + 256 * i;
        if (u < units) store_values(dst + (size_t)u * N, b[i], s[i]);
    }
}

}  // namespace

cudaError_t launch_cache_append(const Cache8 &c, hils_dtype in, const void *K, const void *V, uint8_t *K8, uint8_t *V8,
                                float *ks, float *vs, int t0, int t1, cudaStream_t s)
{
    const int c0 = t0 / c.C, nb = (t1 - 1) / c.C - c0 + 1;
    const unsigned grid = (unsigned)(2ll * c.B * c.Hkv * nb);
    const int threads = c.C * c.d / (in == HILS_BF16 ? 64 : 32);
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
    const long long units = (long long)(t1 - t0) * c.d / (out == HILS_BF16 ? 8 : 4);   // pieces of a kv-head's side
    const dim3 grid((unsigned)((units + 256 * kPieces - 1) / (256 * kPieces)), (unsigned)(c.B * c.Hkv), 2);
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
