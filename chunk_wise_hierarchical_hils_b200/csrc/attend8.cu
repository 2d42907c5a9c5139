// attend8.cu -- chunk attention and fusion over the 8-bit cache, a row of work per query group: single-token decode,
// few queries, and every shape and type.
//
// "Hierarchical Sparse Attention Done Right" (arXiv 2607.02980v1), Abstract and Sec. 3 "Hierarchical softmax", with
// keys ks_c e and values vs_c e' (e4m3 rows e, e', one scale per chunk and side):
//   x_j = (scale ks_c) <q, e_j>,  p = softmax_j(x) over the keys seen,  o = sum_c (w_c vs_c) sum_j p_j e'_j.
// Every selected chunk is 2 C d bytes that one query group uses once, so the kernel's job is to keep loads in
// flight; the products run on mma.sync tiles (4 heads x 64 keys x 128 columns is far below a tcgen05 tile).
//
// One warp takes a whole chunk at a time, straight from global memory into registers: no shared-memory tiles,
// because e4m3 bytes have to pass through registers anyway to become f16 (exact), and because the index orders of an
// mma product are free: the d index of Q K^T and the d rows of V^T P are permuted so that what a lane's 16-byte loads
// bring is what its fragments hold.
//   S^T = K Q^T     A = 16 keys x 16 of d, B = 8 heads: lane (r, t) = (lane / 4, lane % 4) loads 16 bytes of keys r
//                   and r + 8 at d = 64 s + 16 t, whose words are its A fragments of four k-steps
//   O^T = V^T P^T   A = 16 of d x 16 keys: the lane loads 16 bytes at d = 16 r of keys 2t, 2t+1, 2t+8, 2t+9; byte
//                   permutes pair the keys; P^T comes from S^T's accumulators by movmatrix
// The eight columns are heads: a group of more than eight is two rows of work.  While a chunk's probabilities are
// made the next chunk's keys are on their way, and its values during the next chunk's scores, so a warp
// keeps 8 to 16 KB in flight.
//
// Numbers.  A query row is scaled by a power of two to just below 2^15 and taken in f16: bf16 queries keep their 8 bits down
// to 2^-29 of the row's largest, and below that an error of 2^-39 of it; float32 queries are two f16 pieces (22 bits).
// P carries w_c vs_c / max_c'(w vs) and a factor 2^14 into f16 (2^-12 of the value down to 2^-28 of the row's
// largest weight); for float32 results it is two f16 pieces.  All sums are float32.
//
// A row's slots are split over the warps of one block or of a cluster of blocks, and the partial rows meet in shared
// memory (distributed shared memory for a cluster): no workspace, no atomics, a fixed order.
#include <math.h>
#include <stdlib.h>
#include <string.h>
#include <type_traits>

#include "attend_simt.cuh"
#include "cache8.h"
#include "sm100.cuh"
#include "tiles8.cuh"

namespace hils {
namespace {

using namespace t8;

constexpr int kWarps = 4;
constexpr int kHeads = 8;      // heads a row of work covers
constexpr int kMaxSlots = HILS_MAX_K + 1;

__device__ __forceinline__ uint32_t cluster_rank() { uint32_t r; asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r)); return r; }
__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
__device__ __forceinline__ float ld_cluster(uint32_t addr, uint32_t rank)
{
    uint32_t a;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}

// Blocks an SM holds, by the registers a thread needs.
constexpr int blocks_per_sm(int D, int C, bool wide_q) { return D == 64 ? 4 : (C == 128 || wide_q) ? 2 : 3; }

// SOLO: every warp has a row of work to itself; otherwise the warps of a block, or of a cluster of cs blocks, share one.
template <typename Tin, typename Tout, int D, int C, bool SOLO>
__global__ void __launch_bounds__(32 * kWarps, blocks_per_sm(D, C, sizeof(Tin) == 4))
    attend8_kernel(Dims p, int cs, int hgs, const Tin *__restrict__ Q, const uint8_t *__restrict__ K8,
                   const uint8_t *__restrict__ V8, const float *__restrict__ ks, const float *__restrict__ vs,
                   const int32_t *__restrict__ sel_idx, const float *__restrict__ sel_score, Tout *__restrict__ O)
{
    constexpr bool QHL = sizeof(Tin) == 4, PHL = sizeof(Tout) == 4;
    constexpr int MT = C / 16, KS = D / 16, DT = D / 16, WORDS = D / 8;
    constexpr int ROWS = SOLO ? kWarps : 1;           // rows of work a block has
    __shared__ float s_part[SOLO ? 1 : kWarps][kHeads][D + 4];   // + 4: a fragment's eight head rows on distinct banks
    __shared__ float s_weights[ROWS][kHeads][kMaxSlots];
    __shared__ float s_tops[ROWS][kHeads];
    __shared__ int s_chunks[ROWS][kMaxSlots];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, r = lane >> 2, t = lane & 3;
    const int rank = !SOLO && cs > 1 ? (int)cluster_rank() : 0;
    const int unit = SOLO ? blockIdx.x * kWarps + warp : blockIdx.x / cs, i = unit / hgs;
    if (SOLO && i >= p.N) return;                     // whole warps leave; a block of lone warps has no barrier
    float (&s_w)[kHeads][kMaxSlots] = s_weights[SOLO ? warp : 0];
    float (&s_top)[kHeads] = s_tops[SOLO ? warp : 0];
    int (&s_chunk)[kMaxSlots] = s_chunks[SOLO ? warp : 0];
    const size_t bg = blockIdx.y;
    const int h0 = (unit % hgs) * kHeads, nh = min(p.G - h0, kHeads);
    const long long pos = (long long)p.q_offset + i;
    const int ci = (int)(pos / C), ns = p.k + 1, nw = SOLO ? 1 : kWarps * cs, me = SOLO ? 0 : rank * kWarps + warp;
    const int32_t *si = sel_idx + (bg * p.N + i) * p.k;
    const uint8_t *Kb = K8 + bg * (size_t)p.T * D + 16 * t;
    const uint8_t *Vb = V8 + bg * (size_t)p.T * D + (D / 8) * r;

    // A chunk is a stream of 2 MT tiles, its keys' and then its values', through four register buffers: once tile n
    // is used, its buffer is loaded with tile n + 4 of the stream, which runs on into the warp's next chunk.
    uint32_t buf[4][WORDS];
    auto load_tile = [&](auto part, int n, int c, int top) {   // tile n of chunk c, whose last row seen is `top`
        constexpr bool PART = decltype(part)::value;
        if (n < MT) load_k<D, PART>(buf[n & 3], Kb + ((size_t)c * C + 16 * n) * D, r, top - 16 * n);
        else load_v<D, PART>(buf[n & 3], Vb + ((size_t)c * C + 16 * (n - MT)) * D, t, top - 16 * (n - MT));
    };

    // The own chunk, whose rows behind the query are not seen, is the first in the order of work and past chunks (whole
    // ones) follow: turn 0 is slot k, turn x > 0 slot x - 1.  This warp's turns are me, me + nw, ..
    auto chunk_of = [&](int j) { return j < p.k ? __ldg(si + j) : j == p.k ? ci : -1; };
    int turn = me, c = turn == 0 ? ci : chunk_of(turn <= p.k ? turn - 1 : ns);
    while (c < 0 && turn + nw < ns) { turn += nw; c = chunk_of(turn - 1); }
    const int own_top = (int)(pos - (long long)ci * C);
    if (turn == 0) {
#pragma unroll
        for (int n = 0; n < 4; ++n) load_tile(std::true_type(), n, c, own_top);
    } else if (c >= 0) {
#pragma unroll
        for (int n = 0; n < 4; ++n) load_tile(std::false_type(), n, c, C - 1);
    }

    // the query rows: lane (r, t) holds head h0 + r at d = 64 s + 16 t .. + 15
    uint32_t qh[KS][2], ql[QHL ? KS : 1][2];
    float fq;   // scale log2(e) / the row's power of two, for head r
    {
        float x[D / 64][16], m = 0.f;
        const Tin *qr = Q + ((bg * p.G + h0 + min(r, nh - 1)) * p.N + i) * D + 16 * t;
#pragma unroll
        for (int s = 0; s < D / 64; ++s) {
            load8(qr + 64 * s, x[s]);
            load8(qr + 64 * s + 8, x[s] + 8);
#pragma unroll
            for (int e = 0; e < 16; ++e) m = fmaxf(m, fabsf(x[s][e]));
        }
        m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
        m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
        const int sh = min(14 - ((int)(__float_as_uint(m) >> 23) - 127), 120);
        const float f = exp2_int(sh);
        fq = p.scale * 1.4426950408889634f * exp2_int(-sh);
#pragma unroll
        for (int s = 0; s < D / 64; ++s)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float a = x[s][2 * e] * f, b = x[s][2 * e + 1] * f;
                const uint32_t v = pack_f16(a, b);
                qh[4 * s + e / 2][e & 1] = v;
                if constexpr (QHL) {
                    const float2 y = unpack_f16(v);
                    ql[4 * s + e / 2][e & 1] = pack_f16(a - y.x, b - y.y);
                }
            }
    }
    // this lane's columns of the products are heads 2t and 2t + 1
    const float fq0 = __shfl_sync(0xFFFFFFFFu, fq, 8 * t), fq1 = __shfl_sync(0xFFFFFFFFu, fq, 8 * t + 4);

    // slot factors w_c vs_c over the row's largest, times 2^14; a slot without a chunk has no weight, whatever its score
    for (int h = SOLO ? 0 : warp; h < kHeads; h += SOLO ? 1 : kWarps) {
        if (h >= nh) {   // columns without a head: no weight
            for (int jj = lane; jj < ns; jj += 32) s_w[h][jj] = 0.f;
            continue;
        }
        float s[3], v[3], mx = -INFINITY, z = 0.f, top = 0.f;
#pragma unroll
        for (int u = 0; u < 3; ++u) {
            const int jj = lane + 32 * u;
            const int cc = chunk_of(jj);
            s[u] = cc >= 0 ? __ldg(sel_score + ((bg * p.G + h0 + h) * p.N + i) * ns + jj) : -INFINITY;
            v[u] = cc >= 0 ? __ldg(vs + bg * p.nL + cc) : 0.f;
            if (h == 0 && jj < ns) s_chunk[jj] = cc;
            mx = fmaxf(mx, s[u]);
        }
        mx = warp_max(mx);
#pragma unroll
        for (int u = 0; u < 3; ++u) {
            s[u] = (s[u] == -INFINITY) ? 0.f : expf(s[u] - mx);
            z += s[u];
        }
        z = warp_sum(z);
        const float iz = z == 0.f ? 0.f : 1.0f / z;
#pragma unroll
        for (int u = 0; u < 3; ++u) {
            s[u] = s[u] == 0.f ? 0.f : s[u] * iz * v[u];
            top = fmaxf(top, fabsf(s[u]));
        }
        top = warp_max(top);
        const float f = top > 0.f ? 16384.0f / top : 1.0f;
#pragma unroll
        for (int u = 0; u < 3; ++u)
            if (lane + 32 * u < ns) s_w[h][lane + 32 * u] = s[u] * f;
        if (lane == 0) s_top[h] = top > 0.f ? top * (1.0f / 16384.0f) : 0.f;
    }
    if constexpr (SOLO) __syncwarp();
    else __syncthreads();

    float oacc[DT][4];
#pragma unroll
    for (int a = 0; a < DT; ++a)
#pragma unroll
        for (int e = 0; e < 4; ++e) oacc[a][e] = 0.f;

    auto attend_chunk = [&](auto own_chunk) {   // the chunk of this turn, whose first four tiles are loaded or on their way
        constexpr bool OWN = decltype(own_chunk)::value;
        // the next turn of this warp that holds a chunk
        int tn = turn, cn = -1;
        while (cn < 0 && tn + nw < ns) { tn += nw; cn = s_chunk[tn - 1]; }
        auto load_next = [&](int n) {
            if (n < 2 * MT) load_tile(own_chunk, n, c, OWN ? own_top : C - 1);
            else if (cn >= 0) load_tile(std::false_type(), n - 2 * MT, cn, C - 1);
        };
        const float kc = __ldg(ks + bg * p.nL + c);
        const float f0 = fq0 * kc, f1 = fq1 * kc;

        // scores, two tiles of keys at a time: their products are independent of one another
        float sacc[MT][4];
#pragma unroll
        for (int m = 0; m < MT; m += 2) {
#pragma unroll
            for (int e = 0; e < 4; ++e) sacc[m][e] = sacc[m + 1][e] = 0.f;
#pragma unroll
            for (int kk = 0; kk < KS; ++kk) {
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const uint32_t *w = buf[(m + u) & 3];
                    const uint32_t w0 = w[kk], w1 = w[KS + kk];
                    const uint32_t a0 = e4m3x2_to_f16x2(w0), a1 = e4m3x2_to_f16x2(w1);
                    const uint32_t a2 = e4m3x2_to_f16x2(w0 >> 16), a3 = e4m3x2_to_f16x2(w1 >> 16);
                    mma_f16(sacc[m + u], a0, a1, a2, a3, qh[kk][0], qh[kk][1]);
                    if constexpr (QHL) mma_f16(sacc[m + u], a0, a1, a2, a3, ql[kk][0], ql[kk][1]);
                }
            }
#pragma unroll
            for (int u = 0; u < 2; ++u) load_next(m + u + 4);
        }

        // softmax over the keys seen (rows r, r + 8 of each tile, then across the lanes of a column).  Rows of the own
        // chunk that the query does not see hold its last row again: they do not change the maximum and weigh nothing.
        // The factors are not negative: the largest product is the largest logit.
        float m0 = fmaxf(sacc[0][0], sacc[0][2]), m1 = fmaxf(sacc[0][1], sacc[0][3]);
#pragma unroll
        for (int m = 1; m < MT; ++m) {
            m0 = sm100::fmax3(m0, sacc[m][0], sacc[m][2]);
            m1 = sm100::fmax3(m1, sacc[m][1], sacc[m][3]);
        }
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
            m0 = fmaxf(m0, __shfl_xor_sync(0xFFFFFFFFu, m0, o));
            m1 = fmaxf(m1, __shfl_xor_sync(0xFFFFFFFFu, m1, o));
        }
        m0 *= f0;
        m1 *= f1;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int e = 0; e < 4; ++e) sacc[m][e] = sm100::ex2_approx(fmaf(sacc[m][e], (e & 1) ? f1 : f0, (e & 1) ? -m1 : -m0));
        if constexpr (OWN) {
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (16 * m + 8 * (e >> 1) + r > own_top) sacc[m][e] = 0.f;
        }
        float l0 = 0.f, l1 = 0.f;
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            l0 += sacc[m][0] + sacc[m][2];
            l1 += sacc[m][1] + sacc[m][3];
        }
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
            l0 += __shfl_xor_sync(0xFFFFFFFFu, l0, o);
            l1 += __shfl_xor_sync(0xFFFFFFFFu, l1, o);
        }
        const int slot = OWN ? p.k : turn - 1;
        const float g0 = __fdividef(s_w[2 * t][slot], l0), g1 = __fdividef(s_w[2 * t + 1][slot], l1);   // 1 <= l <= C

        // values
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const float(&e)[4] = sacc[m];
            const uint32_t *vw = buf[(MT + m) & 3];
            const float x0 = e[0] * g0, x1 = e[1] * g1, x2 = e[2] * g0, x3 = e[3] * g1;
            const uint32_t pa = pack_f16(x0, x1), pb = pack_f16(x2, x3);
            const uint32_t b0 = movmatrix_t(pa), b1 = movmatrix_t(pb);
            uint32_t c0 = 0u, c1 = 0u;
            if constexpr (PHL) {
                const float2 ya = unpack_f16(pa), yb = unpack_f16(pb);
                c0 = movmatrix_t(pack_f16(x0 - ya.x, x1 - ya.y));
                c1 = movmatrix_t(pack_f16(x2 - yb.x, x3 - yb.y));
            }
#pragma unroll
            for (int w = 0; w < D / 32; ++w) {
                const uint32_t k0 = vw[w], k1 = vw[D / 32 + w], k8 = vw[2 * (D / 32) + w], k9 = vw[3 * (D / 32) + w];
#pragma unroll
                for (int hw = 0; hw < 2; ++hw) {
                    const uint32_t lo = __byte_perm(k0, k1, hw ? 0x7362 : 0x5140);
                    const uint32_t hi = __byte_perm(k8, k9, hw ? 0x7362 : 0x5140);
                    const uint32_t a0 = e4m3x2_to_f16x2(lo), a1 = e4m3x2_to_f16x2(lo >> 16);
                    const uint32_t a2 = e4m3x2_to_f16x2(hi), a3 = e4m3x2_to_f16x2(hi >> 16);
                    mma_f16(oacc[2 * w + hw], a0, a1, a2, a3, b0, b1);
                    if constexpr (PHL) mma_f16(oacc[2 * w + hw], a0, a1, a2, a3, c0, c1);
                }
            }
            load_next(MT + m + 4);
        }
        turn = tn;
        c = cn;
    };
    if (turn == 0) attend_chunk(std::true_type());
    while (c >= 0) attend_chunk(std::false_type());

    if constexpr (SOLO) {
        // tile a, row r is d = (D / 8) r + 2 a, row r + 8 the next one; columns are heads 2t, 2t + 1
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int h = 2 * t + q;
            if (h < nh) {
                const float f = s_top[h];
                float v[2 * DT];
#pragma unroll
                for (int a = 0; a < DT; ++a) {
                    v[2 * a] = oacc[a][q] * f;
                    v[2 * a + 1] = oacc[a][2 + q] * f;
                }
                store_n<2 * DT>(O + ((bg * p.G + h0 + h) * p.N + i) * D + (D / 8) * r, v);
            }
        }
    } else {
        // the warps' rows meet: tile a, row r is d = (D / 8) r + 2 a, row r + 8 the next one; columns are heads 2t, 2t + 1
#pragma unroll
        for (int a = 0; a < DT; ++a) {
            const int x = (D / 8) * r + 2 * a;
            *reinterpret_cast<float2 *>(&s_part[warp][2 * t][x]) = make_float2(oacc[a][0], oacc[a][2]);
            *reinterpret_cast<float2 *>(&s_part[warp][2 * t + 1][x]) = make_float2(oacc[a][1], oacc[a][3]);
        }
        __syncthreads();
        if (cs > 1) {
            for (int e = tid; e < nh * D; e += 32 * kWarps) {
                const int h = e / D, x = e % D;
                float a = s_part[0][h][x];
#pragma unroll
                for (int w = 1; w < kWarps; ++w) a += s_part[w][h][x];
                s_part[0][h][x] = a;
            }
            cluster_sync();
            for (int e = rank * 32 * kWarps + tid; e < nh * D; e += cs * 32 * kWarps) {
                const int h = e / D, x = e % D;
                const uint32_t addr = sm100::smem_addr(&s_part[0][h][x]);
                float a = 0.f;
                for (int k = 0; k < cs; ++k) a += ld_cluster(addr, (uint32_t)k);
                store_out(O + ((bg * p.G + h0 + h) * p.N + i) * D + x, a * s_top[h]);
            }
            cluster_sync();   // the others' reads of this block's rows
            return;
        }
        for (int e = tid; e < nh * D; e += 32 * kWarps) {
            const int h = e / D, x = e % D;
            float a = s_part[0][h][x];
#pragma unroll
            for (int w = 1; w < kWarps; ++w) a += s_part[w][h][x];
            store_out(O + ((bg * p.G + h0 + h) * p.N + i) * D + x, a * s_top[h]);
        }
    }
}

// How the rows are shared out: cs = 0: a warp a row (SOLO), else teams of cs blocks; and the time it is expected to
// take, in the time of a warp's chunk (2.9 us with every SM full).  Weighed: a warp's turns of its row (the longest
// list and the mean), the start and end of a row (3 chunks for a lone warp, 1.5 for a team, its merge included), and how
// often the resident warps start over.  8 rows of 65 slots go to teams of eight blocks (11.3 us; six 12.3, four 15.7),
// 128 rows of 33 slots to teams of three (20.5 us; two 23.8, four, which queue, 31), 4072 rows of 33 slots to single
// blocks (303 us; lone warps 347), 65536 rows of 17 slots and 2006 rows of 5 to lone warps (2.18 ms and 12.8 us; blocks
// 2.54 ms and 20.1 us).
struct Share {
    int cs;
    double time;
};

Share share_of(const Dims &p, int per_sm)
{
    const double rows = (double)p.B * p.Hkv * ((p.G + kHeads - 1) / kHeads) * p.N, blocks = 148.0 * per_sm;
    const int ns = p.k + 1;
    auto rounds = [](double x) { return x <= 1.0 ? 1.0 : x <= 4.0 ? ceil(x) + 0.25 : x + 0.5; };
    Share best = {0, rounds(rows / (blocks * kWarps)) * (ns + 3.0)};
    for (int cs = 1; cs <= 8; ++cs) {
        const int w = kWarps * cs;
        const double turns = 0.5 * ((ns + w - 1) / w + (double)ns / w);
        const double t = rounds(rows * cs / blocks) * (turns + 1.5);
        if (t < best.time) best = {cs, t};
    }
    return best;
}

int per_sm_of(const Dims &p, hils_dtype in) { return blocks_per_sm(p.d, p.C, in == HILS_F32); }

template <typename Tin, typename Tout, int D, int C>
cudaError_t launch_t(const Dims &p, const void *Q, const uint8_t *K8, const uint8_t *V8, const float *ks, const float *vs,
                     const int32_t *sel_idx, const float *sel_score, void *O, cudaStream_t s)
{
    const int hgs = (p.G + kHeads - 1) / kHeads;
    const int cs = share_of(p, blocks_per_sm(D, C, sizeof(Tin) == 4)).cs;
    const long long units = (long long)p.N * hgs;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(cs ? units * cs : (units + kWarps - 1) / kWarps), (unsigned)(p.B * p.Hkv));
    cfg.blockDim = dim3(32 * kWarps);
    cfg.stream = s;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = (unsigned)cs;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = cs > 1 ? 1 : 0;
    auto *kern = cs ? attend8_kernel<Tin, Tout, D, C, false> : attend8_kernel<Tin, Tout, D, C, true>;
    return cudaLaunchKernelEx(&cfg, kern, p, cs, hgs, static_cast<const Tin *>(Q), K8, V8, ks, vs, sel_idx, sel_score,
                              static_cast<Tout *>(O));
}

template <typename Tin, typename Tout>
cudaError_t launch_d(const Dims &p, const void *Q, const uint8_t *K8, const uint8_t *V8, const float *ks, const float *vs,
                     const int32_t *sel_idx, const float *sel_score, void *O, cudaStream_t s)
{
    auto go = [&](auto f32, auto f64, auto f128) {
        return (p.C == 32 ? f32 : p.C == 64 ? f64 : f128)(p, Q, K8, V8, ks, vs, sel_idx, sel_score, O, s);
    };
    return p.d == 64 ? go(launch_t<Tin, Tout, 64, 32>, launch_t<Tin, Tout, 64, 64>, launch_t<Tin, Tout, 64, 128>)
                     : go(launch_t<Tin, Tout, 128, 32>, launch_t<Tin, Tout, 128, 64>, launch_t<Tin, Tout, 128, 128>);
}

}  // namespace

size_t attend8_ws_bytes(const Dims &, hils_dtype, hils_dtype) { return 0; }

// Test control: HILS_Q8_KERNEL=rows or =union forces the kernel (the latter where it covers the shape).
static bool use_union(const Dims &p, hils_dtype in, hils_dtype out)
{
    if (!attend8_tc_supported(p, in, out)) return false;
    const char *force = getenv("HILS_Q8_KERNEL");
    if (force && strcmp(force, "rows") == 0) return false;
    if (force && strcmp(force, "union") == 0) return true;
    // The union's cost is known only for selections that have nothing to do with one another, its worst case: of V
    // visible chunks a block's BQ queries then want V (1 - (1 - k / V)^BQ).  A chunk of it takes 0.8 us and a
    // block's set-up 5 us (8K prefill, 62 chunks on average: 835 us against 2.18 ms by rows; 509 queries at 130K, 810 chunks
    // a block of which a query wants 33: 474 us against 303).
    const double BQ = 128 / p.G, V = (p.q_offset + 0.5 * p.N) / p.C + 1.0;
    const double U = V * (1.0 - pow(1.0 - fmin(1.0, p.k / V), BQ)) + BQ / p.C + 1.0;
    const double blocks = (double)p.B * p.Hkv * ((p.N + BQ - 1) / BQ) / 148.0;
    const double t_union = (blocks <= 1.0 ? 1.0 : blocks + 0.5) * (5.0 + 0.8 * fmin(U, V + 1.0));
    return t_union < 2.9 * share_of(p, per_sm_of(p, in)).time;
}

cudaError_t launch_attend8(const Dims &p, hils_dtype in, hils_dtype out, const void *Q, const uint8_t *K8,
                           const uint8_t *V8, const float *ks, const float *vs, const int32_t *sel_idx,
                           const float *sel_score, void *O, void *, const DeviceCtl &ctl, cudaStream_t s)
{
    if (use_union(p, in, out)) return launch_attend8_tc(p, Q, K8, V8, ks, vs, sel_idx, sel_score, O, ctl, s);
    if (in == HILS_F32)
        return out == HILS_F32 ? launch_d<float, float>(p, Q, K8, V8, ks, vs, sel_idx, sel_score, O, s)
                               : launch_d<float, __nv_bfloat16>(p, Q, K8, V8, ks, vs, sel_idx, sel_score, O, s);
    return out == HILS_F32 ? launch_d<__nv_bfloat16, float>(p, Q, K8, V8, ks, vs, sel_idx, sel_score, O, s)
                           : launch_d<__nv_bfloat16, __nv_bfloat16>(p, Q, K8, V8, ks, vs, sel_idx, sel_score, O, s);
}

}  // namespace hils
