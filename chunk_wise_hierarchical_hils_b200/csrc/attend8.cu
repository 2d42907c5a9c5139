// attend8.cu -- chunk attention and fusion over the 8-bit cache, a row of work per query group: single-token decode,
// few queries, and every shape and type.
//
// "Hierarchical Sparse Attention Done Right" (arXiv 2607.02980v1), Abstract and Sec. 3 "Hierarchical softmax", with
// keys ks_c e and values vs_c e' (e4m3 rows e, e', one scale per chunk and side):
//   x_j = (scale ks_c) <q, e_j>,  p = softmax_j(x) over the keys seen,  o = sum_c (w_c vs_c) sum_j p_j e'_j.
// Every selected chunk is 2 C d bytes that one query group uses once, so the kernel's job is to keep loads in
// flight; the products run on mma.sync tiles (4 heads x 64 keys x 128 columns is far below a tcgen05 tile).
//
// One warp takes a whole chunk at a time, on tiles of 16 keys in shared memory that it fills itself (tiles8.cuh):
//   S^T = K Q^T     A = 16 keys x 16 of d, B = 8 heads
//   O^T = V^T P^T   A = 16 of d x 16 keys (bytes transposed as they are read); P^T comes from S^T's accumulators by
//                   movmatrix
// e4m3 becomes f16 (exact) in registers.  The eight columns are heads (float32 queries or results: four heads and their
// second pieces); a group of more is two or more rows of work.  A
// chunk is a stream of pairs of tiles, its keys' and then its values', through a ring of up to four pairs: once a pair is
// used its place is filled with the pair four further on, which runs on into the warp's next chunk, so a warp has
// 8 to 16 KB in flight or in use.
//
// Numbers.  A query row is scaled by a power of two so that its largest element lies in [2^14, 2^15), and taken in f16, whose
// normal numbers end at 2^-14 and whose steps at 2^-24: bf16 queries keep their 8 bits down to 2^-31 of the row's largest,
// and below that an error of 2^-39 of it; float32 queries are two f16 pieces (2^-22 of an element, or 2^-39 of the largest).
// P carries w_c vs_c / max_c'(w vs) and a factor 2^14 into f16 (half a step, 2^-11 of the value, down to 2^-28 of the row's
// largest weight); for float32 results it is two f16 pieces (2^-22).  All sums are float32; the tensor cores cut what they add to an
// accumulator off instead of rounding it, so for float32 results every product starts from zero and is added by the
// float32 units (a chain of 264 products lost 1.6e-6 of the result and one of 516 9e-6, started afresh the error is 2e-7 and
// 4e-7, root mean square).
//
// A row's slots are split over the warps of one block or of a cluster of blocks, and the partial rows meet in shared
// memory (distributed shared memory for a cluster): no workspace, no atomics, a fixed order.
#include <math.h>
#include <stdlib.h>
#include <string.h>
#include <type_traits>

#include "common.cuh"
#include "cache8.h"
#include "sm100.cuh"
#include "tiles8.cuh"

namespace hils {
namespace {

using namespace t8;

constexpr int kWarps = 4;
constexpr int kMaxTeam = 8;    // blocks of a cluster that share a row (the portable limit)
constexpr int kCols = 8;       // columns of a product
// Heads a row of work covers: one a column; with float32 queries or results four, whose second pieces take the others.
constexpr int heads_of(bool wide) { return wide ? 4 : 8; }
constexpr int kMaxSlots = HILS_MAX_K + 1;

__device__ __forceinline__ uint32_t cluster_rank() { uint32_t r; asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r)); return r; }
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.aligned;" ::: "memory"); }
// v to `addr` (an address of this block's shared memory) of the cluster's block `rank`
__device__ __forceinline__ void st_cluster(uint32_t addr, uint32_t rank, float4 v)
{
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(a), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w) : "memory");
}

// Largest of the warp's values in one integer reduction; the first for any values, the second for values that are not
// negative.
__device__ __forceinline__ float redux_max(float x)
{
    const uint32_t u = __float_as_uint(x);
    const uint32_t k = __reduce_max_sync(0xFFFFFFFFu, (u & 0x80000000u) ? ~u : u | 0x80000000u);
    return __uint_as_float((k & 0x80000000u) ? k & 0x7FFFFFFFu : ~k);
}
__device__ __forceinline__ float redux_max_pos(float x)
{
    return __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(x)));
}

// Blocks an SM holds: by registers, and for d = 128 by 16 KB of ring a warp.
constexpr int blocks_per_sm(int D, int C, bool wide_out) { return (D == 64 ? 4 : 3) - (C == 128 && wide_out ? 1 : 0); }

constexpr int ring_space(int D, int C)   // a warp's shared memory: its ring, later its partial rows
{
    const int ring = (C / 16 < 4 ? C / 16 : 4) * 32 * D, rows = (kCols * (D + 4) * 4 + 127) / 128 * 128;
    return ring > rows ? ring : rows;
}

// SOLO: every warp has a row of work to itself; otherwise the warps of a block, or of a cluster of cs blocks, share one.
template <typename Tin, typename Tout, int D, int C, bool SOLO>
__global__ void __launch_bounds__(32 * kWarps, blocks_per_sm(D, C, sizeof(Tout) == 4))
    attend8_kernel(Dims p, int cs, int hgs, const Tin *__restrict__ Q, const uint8_t *__restrict__ K8,
                   const uint8_t *__restrict__ V8, const float *__restrict__ ks, const float *__restrict__ vs,
                   const int32_t *__restrict__ sel_idx, const float *__restrict__ sel_score, Tout *__restrict__ O)
{
    constexpr bool QHL = sizeof(Tin) == 4, PHL = sizeof(Tout) == 4;
    constexpr bool WIDE = QHL || PHL;                 // columns 4 .. 7: the second pieces of columns 0 .. 3
    constexpr int HEADS = heads_of(WIDE), MT = C / 16, KS = D / 16;
    constexpr int NP = MT, RP = NP < 4 ? NP : 4;      // pairs of tiles a chunk is (half of them keys), pairs in a ring
    constexpr int PAIR = 32 * D;
    constexpr int ROWS = SOLO ? kWarps : 1;           // rows of work a block has
    constexpr int PITCH = D + 4;                      // of a row of partial results: lanes of a fragment on distinct banks
    constexpr int SPACE = ring_space(D, C);
    extern __shared__ __align__(128) unsigned char s_ring[];   // [warp][SPACE]: its ring, then its partial rows
    __shared__ float s_weights[ROWS][HEADS][kMaxSlots];
    __shared__ float s_tops[ROWS][HEADS];
    __shared__ int s_chunks[ROWS][kMaxSlots];
    __shared__ __align__(16) float s_shares[SOLO ? 4 : HEADS * D + 4 * kMaxTeam];   // [block of the cluster][slice]

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, r = lane >> 2, t = lane & 3;
    const int rank = !SOLO && cs > 1 ? (int)cluster_rank() : 0;
    const int unit = SOLO ? blockIdx.x * kWarps + warp : blockIdx.x / cs, i = unit / hgs;
    if (SOLO && i >= p.N) return;                     // whole warps leave; a block of lone warps has no barrier
    if (!SOLO && cs > 1) cluster_arrive();            // waited for before the first access to another block
    float (&s_w)[HEADS][kMaxSlots] = s_weights[SOLO ? warp : 0];
    float (&s_top)[HEADS] = s_tops[SOLO ? warp : 0];
    int (&s_chunk)[kMaxSlots] = s_chunks[SOLO ? warp : 0];
    const size_t bg = blockIdx.y;
    const int h0 = (unit % hgs) * HEADS, nh = min(p.G - h0, HEADS);
    const long long pos = (long long)p.q_offset + i;
    const int ci = (int)(pos / C), ns = p.k + 1, nw = SOLO ? 1 : kWarps * cs, me = SOLO ? 0 : rank * kWarps + warp;
    const int32_t *si = sel_idx + (bg * p.N + i) * p.k;
    const uint8_t *Kb = K8 + bg * (size_t)p.T * D, *Vb = V8 + bg * (size_t)p.T * D;
    const uint32_t ring = sm100::smem_addr(s_ring) + (uint32_t)warp * SPACE;
    float *part = reinterpret_cast<float *>(s_ring + warp * SPACE);   // [head][PITCH]

    auto load_pair = [&](auto part_chunk, int n, int c, int top) {   // pair n of chunk c, whose last row seen is `top`
        constexpr bool PART = decltype(part_chunk)::value;
        const int row = 32 * (n < NP / 2 ? n : n - NP / 2);
        load_rows<D, 32, PART>(ring + (uint32_t)(n % RP) * PAIR, (n < NP / 2 ? Kb : Vb) + ((size_t)c * C + row) * D, top - row);
        cp_commit();
    };

    // Everything the start needs and knows the place of is asked for first: the row's slots and its heads' scores (lane l
    // holds slots l, l + 32, l + 64), the query rows.
    constexpr int HW = SOLO ? HEADS : HEADS / kWarps;   // heads whose weights this warp works out
    int cc[3];
    float s[HW][3], x[KS][4];
#pragma unroll
    for (int u = 0; u < 3; ++u) cc[u] = lane + 32 * u < p.k ? __ldg(si + lane + 32 * u) : -1;
#pragma unroll
    for (int u = 0; u < 3; ++u)
#pragma unroll
        for (int q = 0; q < HW; ++q) {
            const int h = SOLO ? q : warp + q * kWarps;
            s[q][u] = lane + 32 * u < ns && h < nh
                          ? __ldg(sel_score + ((bg * p.G + h0 + h) * p.N + i) * ns + lane + 32 * u) : -INFINITY;
        }
    {
        const Tin *qr = Q + ((bg * p.G + h0 + min(r % HEADS, nh - 1)) * p.N + i) * D + 4 * t;
#pragma unroll
        for (int c16 = 0; c16 < KS; ++c16) load4(qr + 16 * c16, x[c16]);
    }
    // An entry that is no past chunk of the query is an empty slot: nothing outside the cache is read for it.
#pragma unroll
    for (int u = 0; u < 3; ++u) {
        const int jj = lane + 32 * u;
        cc[u] = jj == p.k ? ci : (unsigned)cc[u] < (unsigned)ci ? cc[u] : -1;
        if ((SOLO || warp == 0) && jj < ns) s_chunk[jj] = cc[u];
    }
    auto chunk_of = [&](int j) { return __shfl_sync(0xFFFFFFFFu, j < 32 ? cc[0] : j < 64 ? cc[1] : cc[2], j & 31); };

    // The own chunk, whose rows behind the query are not seen, is the first in the order of work and past chunks (whole
    // ones) follow: turn 0 is slot k, turn x > 0 slot x - 1.  This warp's turns are me, me + nw, ..
    int turn = me, c = turn == 0 ? ci : turn <= p.k ? chunk_of(turn - 1) : -1;
    while (c < 0 && turn + nw < ns) { turn += nw; c = chunk_of(turn - 1); }
    const int own_top = (int)(pos - (long long)ci * C);
    if (turn == 0) {
#pragma unroll
        for (int n = 0; n < RP; ++n) load_pair(std::true_type(), n, c, own_top);
    } else if (c >= 0) {
#pragma unroll
        for (int n = 0; n < RP; ++n) load_pair(std::false_type(), n, c, C - 1);
    }
    float v[3];
#pragma unroll
    for (int u = 0; u < 3; ++u) v[u] = cc[u] >= 0 ? __ldg(vs + bg * p.nL + cc[u]) : 0.f;

    // the query rows: lane (r, t) holds column r, which is head h0 + r (or its second piece), at d = 16 c + 4 t .. + 3
    uint32_t qf[KS][2];
    float fq;   // scale log2(e) / the row's power of two, for the head of column r
    {
        float m = 0.f;
#pragma unroll
        for (int c16 = 0; c16 < KS; ++c16)
            m = fmaxf(m, fmaxf(fmaxf(fabsf(x[c16][0]), fabsf(x[c16][1])), fmaxf(fabsf(x[c16][2]), fabsf(x[c16][3]))));
        m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
        m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
        const int sh = min(14 - ((int)(__float_as_uint(m) >> 23) - 127), 120);
        const float f = exp2_int(sh);
        fq = p.scale * 1.4426950408889634f * exp2_int(-sh);
#pragma unroll
        for (int c16 = 0; c16 < KS; ++c16)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float a = x[c16][2 * e] * f, b = x[c16][2 * e + 1] * f;
                qf[c16][e] = pack_f16(a, b);
                if constexpr (QHL) {
                    const float2 y = unpack_f16(qf[c16][e]);
                    if (r >= HEADS) qf[c16][e] = pack_f16(a - y.x, b - y.y);
                }
            }
    }
    // this lane's columns of the products are heads hd and hd + 1
    const int hd = 2 * t % HEADS;
    const float fq0 = __shfl_sync(0xFFFFFFFFu, fq, 4 * hd), fq1 = __shfl_sync(0xFFFFFFFFu, fq, 4 * hd + 4);

    // slot factors w_c vs_c over the row's largest, times 2^14; a slot without a chunk has no weight, whatever its score
    {
#pragma unroll
        for (int q = 0; q < HW; ++q) {
            const int h = SOLO ? q : warp + q * kWarps;
            if (h >= nh) {   // columns without a head: no weight
                for (int jj = lane; jj < ns; jj += 32) s_w[h][jj] = 0.f;
                continue;
            }
#pragma unroll
            for (int u = 0; u < 3; ++u) s[q][u] = cc[u] >= 0 ? s[q][u] : -INFINITY;
            const float mx = redux_max(fmaxf(fmaxf(s[q][0], s[q][1]), s[q][2]));
            float z = 0.f, top = 0.f;
#pragma unroll
            for (int u = 0; u < 3; ++u) {
                s[q][u] = (s[q][u] == -INFINITY) ? 0.f : expf(s[q][u] - mx);
                z += s[q][u];
            }
            z = warp_sum(z);
            const float iz = z == 0.f ? 0.f : 1.0f / z;
#pragma unroll
            for (int u = 0; u < 3; ++u) {
                s[q][u] = s[q][u] == 0.f ? 0.f : s[q][u] * iz * v[u];
                top = fmaxf(top, s[q][u]);
            }
            top = redux_max_pos(top);
            if (top > 0.f) top = fmaxf(top, 1e-34f);   // its inverse stays finite
            const float f = top > 0.f ? 16384.0f / top : 1.0f;
#pragma unroll
            for (int u = 0; u < 3; ++u)
                if (lane + 32 * u < ns) s_w[h][lane + 32 * u] = s[q][u] * f;
            if (lane == 0) s_top[h] = top > 0.f ? top * (1.0f / 16384.0f) : 0.f;
        }
    }
    if constexpr (SOLO) __syncwarp();
    else __syncthreads();

    float oacc[KS][4];   // tile c, rows r and r + 8: d = 16 c + r (+ 8); columns are heads 2t, 2t + 1
#pragma unroll
    for (int a = 0; a < KS; ++a)
#pragma unroll
        for (int e = 0; e < 4; ++e) oacc[a][e] = 0.f;

    auto attend_chunk = [&](auto own_chunk) {   // the chunk of this turn, whose first pairs of tiles are on their way
        constexpr bool OWN = decltype(own_chunk)::value;
        // the next turn of this warp that holds a chunk
        int tn = turn, cn = -1;
        while (cn < 0 && tn + nw < ns) { tn += nw; cn = s_chunk[tn - 1]; }
        // use(n, f): f on pair n of the stream once it is there; then its place is filled with the pair RP further on
        auto use = [&](int n, auto f) {
            cp_wait<RP - 1>();
            __syncwarp();
            f(ring + (uint32_t)(n % RP) * PAIR);
            __syncwarp();
            if (n + RP < NP) load_pair(own_chunk, n + RP, c, OWN ? own_top : C - 1);
            else if (cn >= 0) load_pair(std::false_type(), n + RP - NP, cn, C - 1);
            else cp_commit();   // groups are counted
        };
        const float kc = __ldg(ks + bg * p.nL + c);
        const int slot = OWN ? p.k : turn - 1;
        // a head that gives the slot no weight takes its logits as zeros: their factor may be beyond float32, and a NaN would
        // reach the head's row through the weight of zero
        const float w0 = s_w[hd][slot], w1 = s_w[hd + 1][slot];
        const float f0 = w0 == 0.f ? 0.f : fq0 * kc, f1 = w1 == 0.f ? 0.f : fq1 * kc;

        // scores, two tiles of keys at a time: their products are independent of one another
        float sacc[MT][4];
#pragma unroll
        for (int m = 0; m < MT; m += 2)
            use(m / 2, [&](uint32_t tile) {
                uint32_t w[2][KS][2];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    read_keys<D>(tile + u * 16 * D, w[u]);
                    sacc[m + u][0] = sacc[m + u][1] = sacc[m + u][2] = sacc[m + u][3] = 0.f;
                }
#pragma unroll
                for (int k = 0; k < KS; ++k)
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        if constexpr (PHL) {
                            float x[4] = {0.f, 0.f, 0.f, 0.f};
                            mma_bytes(x, w[u][k][0], w[u][k][1], qf[k][0], qf[k][1]);
                            add4(sacc[m + u], x);
                        } else {
                            mma_bytes(sacc[m + u], w[u][k][0], w[u][k][1], qf[k][0], qf[k][1]);
                        }
                    }
            });
        if constexpr (QHL) {   // the pieces meet: both lanes of a head go on with the sum
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int e = 0; e < 4; ++e) sacc[m][e] += __shfl_xor_sync(0xFFFFFFFFu, sacc[m][e], 2);
        }

        // softmax over the keys seen (those of rows r, r + 8 of each tile, then across the lanes of a column).  Rows of the own
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
                    if (16 * m + key_row(r, e >> 1) > own_top) sacc[m][e] = 0.f;
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
        const float g0 = __fdividef(w0, l0), g1 = __fdividef(w1, l1);   // 1 <= l <= C

        // values
#pragma unroll
        for (int m = 0; m < MT; m += 2)
            use(NP / 2 + m / 2, [&](uint32_t tile) {
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const float(&e)[4] = sacc[m + u];
                    const float x0 = e[0] * g0, x1 = e[1] * g1, x2 = e[2] * g0, x3 = e[3] * g1;
                    uint32_t pa = pack_f16(x0, x1), pb = pack_f16(x2, x3);
                    if constexpr (WIDE) {   // the second columns: what f16 leaves, or nothing
                        const float2 ya = unpack_f16(pa), yb = unpack_f16(pb);
                        const uint32_t ra = PHL ? pack_f16(x0 - ya.x, x1 - ya.y) : 0u, rb = PHL ? pack_f16(x2 - yb.x, x3 - yb.y) : 0u;
                        pa = t < 2 ? pa : ra;
                        pb = t < 2 ? pb : rb;
                    }
                    const uint32_t b0 = movmatrix_t(pa), b1 = movmatrix_t(pb);
#pragma unroll
                    for (int k = 0; k < KS; k += 2) {
                        uint32_t w[2][2];
                        read_values<D>(tile + u * 16 * D, k, w);
#pragma unroll
                        for (int v = 0; v < 2; ++v) {
                            if constexpr (PHL) {
                                float x[4] = {0.f, 0.f, 0.f, 0.f};
                                mma_bytes(x, w[v][0], w[v][1], b0, b1);
                                add4(oacc[k + v], x);
                            } else {
                                mma_bytes(oacc[k + v], w[v][0], w[v][1], b0, b1);
                            }
                        }
                    }
                }
            });
        turn = tn;
        c = cn;
    };
    if (turn == 0) attend_chunk(std::true_type());
    while (c >= 0) attend_chunk(std::false_type());

    // the rows of partial results take the ring's place (nothing is on its way into it any more)
    __syncwarp();
#pragma unroll
    for (int a = 0; a < KS; ++a)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if constexpr (PHL) oacc[a][e] += __shfl_xor_sync(0xFFFFFFFFu, oacc[a][e], 2);   // both pieces
            if (!WIDE || t < 2) part[(2 * t + (e & 1)) * PITCH + 16 * a + r + 8 * (e >> 1)] = oacc[a][e];
        }
    if constexpr (SOLO) {
        __syncwarp();
        for (int e = lane; e < nh * D / 4; e += 32) {
            const int h = e / (D / 4), x = e % (D / 4) * 4;
            const float4 v = *reinterpret_cast<const float4 *>(part + h * PITCH + x);
            const float f = s_top[h];
            store4(O + ((bg * p.G + h0 + h) * p.N + i) * D + x, make_float4(v.x * f, v.y * f, v.z * f, v.w * f));
        }
    } else {
        // the warps' rows, and a cluster's, are added in order
        __syncthreads();
        float *sum = reinterpret_cast<float *>(s_ring);
        auto block_sum = [&](int e) {   // elements 4 e .. 4 e + 3 of the rows
            const float *at = sum + e / (D / 4) * PITCH + e % (D / 4) * 4;
            float4 a = *reinterpret_cast<const float4 *>(at);
#pragma unroll
            for (int w = 1; w < kWarps; ++w) {
                const float4 y = *reinterpret_cast<const float4 *>(at + w * (SPACE / 4));
                a = make_float4(a.x + y.x, a.y + y.y, a.z + y.z, a.w + y.w);
            }
            return a;
        };
        auto store = [&](int e, float4 a) {
            const int h = e / (D / 4), y = e % (D / 4) * 4;
            const float f = s_top[h];
            store4(O + ((bg * p.G + h0 + h) * p.N + i) * D + y, make_float4(a.x * f, a.y * f, a.z * f, a.w * f));
        };
        const int n4 = nh * D / 4;
        if (cs > 1) {
            // Every block of the cluster finishes a slice of the rows: the others send it their sums of that slice.  One
            // barrier: nothing of a block is accessed by others behind it.
            const int slice = (n4 + cs - 1) / cs;
            cluster_wait();   // all blocks have started
            for (int e = tid; e < n4; e += 32 * kWarps) {
                const int to = e / slice;
                st_cluster(sm100::smem_addr(&s_shares[4 * (rank * slice + e - to * slice)]), (uint32_t)to, block_sum(e));
            }
            __syncwarp();
            cluster_arrive();
            cluster_wait();
            for (int e = tid; e < slice && rank * slice + e < n4; e += 32 * kWarps) {
                float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int k = 0; k < kMaxTeam; ++k)
                    if (k < cs) {
                        const float4 y = *reinterpret_cast<const float4 *>(&s_shares[4 * (k * slice + e)]);
                        a = make_float4(a.x + y.x, a.y + y.y, a.z + y.z, a.w + y.w);
                    }
                store(rank * slice + e, a);
            }
            return;
        }
        for (int e = tid; e < n4; e += 32 * kWarps) store(e, block_sum(e));
    }
}

// How the rows are shared out: cs = 0: a warp a row (SOLO), else teams of cs blocks; and the time it is expected to
// take, in the time of a warp's chunk (1.9 us with every SM full).  Weighed: a warp's turns of its row (the longest
// list and the mean), the start and end of a row (3 chunks for a lone warp, 1.5 for a team, its merge included), and how
// often the resident warps start over.  Measured side by side: 8 rows of 65 slots, teams of eight blocks 8.5 us, six 8.8,
// four 10.6; 128 rows of 33 slots, teams of three 17.1 us, two 17.9, four, which queue, 24; 4072 rows of 33 slots, single
// blocks 188 us, lone warps 190, pairs 263; 65536 rows of 17 slots and 2006 rows of 5, lone warps 1.35 ms and 11 us, blocks
// 1.65 ms and 16 us.  Those are d = 128, C = 64 but for the last.  Against every other share, forced, on 288 problems (all six
// (d, C), bf16 and float32, four heads a group, 8 to 8192 rows of 5 to 65 slots) the rule's choice takes 1.02 times the
// fastest's time in the median of each form, 1.03 to 1.11 on average, at most 1.5 (128 rows of 5 slots, d = 64, C = 32: 6.0 us
// against 4.0 with one block a row; 512 rows of 17, d = 128, C = 32: 19.1 against 13.3): few or short chunks on rows that
// just fill the card, where a start weighs more chunks than assumed and a second block more than it saves.
struct Share {
    int cs;
    double time;
};

Share share_of(const Dims &p, int per_sm, int heads)
{
    const double rows = (double)p.B * p.Hkv * ((p.G + heads - 1) / heads) * p.N, blocks = 148.0 * per_sm;
    // slots that can hold a chunk: no more than the last query has chunks before its own
    const int ns = (int)fmin(p.k, ((double)p.q_offset + p.N - 1) / p.C) + 1;
    auto rounds = [](double x) { return x <= 1.0 ? 1.0 : x <= 4.0 ? ceil(x) + 0.25 : x + 0.5; };
    Share best = {0, rounds(rows / (blocks * kWarps)) * (ns + 3.0)};
    for (int cs = 1; cs <= kMaxTeam; ++cs) {
        const int w = kWarps * cs;
        const double turns = 0.5 * ((ns + w - 1) / w + (double)ns / w);
        const double t = rounds(rows * cs / blocks) * (turns + 1.5);
        if (t < best.time) best = {cs, t};
    }
    return best;
}

// Test control: HILS_Q8_SHARE=0 .. 8 gives every row a lone warp (0) or that many blocks; -1: the rule decides.
int forced_share()
{
    const char *v = getenv("HILS_Q8_SHARE");
    return v && v[0] >= '0' && v[0] <= '0' + kMaxTeam && !v[1] ? v[0] - '0' : -1;
}

template <typename Tin, typename Tout, int D, int C>
cudaError_t launch_t(const Dims &p, const void *Q, const uint8_t *K8, const uint8_t *V8, const float *ks, const float *vs,
                     const int32_t *sel_idx, const float *sel_score, void *O, cudaStream_t s)
{
    constexpr int heads = heads_of(sizeof(Tin) == 4 || sizeof(Tout) == 4);
    const int hgs = (p.G + heads - 1) / heads;
    const int forced = forced_share();
    const int cs = forced >= 0 ? forced : share_of(p, blocks_per_sm(D, C, sizeof(Tout) == 4), heads).cs;
    const long long units = (long long)p.N * hgs;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(cs ? units * cs : (units + kWarps - 1) / kWarps), (unsigned)(p.B * p.Hkv));
    cfg.blockDim = dim3(32 * kWarps);
    cfg.dynamicSmemBytes = kWarps * ring_space(D, C);
    cfg.stream = s;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = (unsigned)cs;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = cs > 1 ? 1 : 0;
    auto *kern = cs ? attend8_kernel<Tin, Tout, D, C, false> : attend8_kernel<Tin, Tout, D, C, true>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)cfg.dynamicSmemBytes);
    if (e != cudaSuccess) return e;
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

// Test control: HILS_Q8_KERNEL=rows or =union forces the kernel (the latter where it covers the shape).
static bool use_union(const Dims &p, hils_dtype in, hils_dtype out)
{
    if (!attend8_tc_supported(p, in, out)) return false;
    const char *force = getenv("HILS_Q8_KERNEL");
    if (force && strcmp(force, "rows") == 0) return false;
    if (force && strcmp(force, "union") == 0) return true;
    if (!attend8_tc_fits(p)) return false;
    // The host does not know the selection: the union is priced for selections that have nothing to do with one another, its
    // worst case (509 queries at 130K that keep the same 32 past chunks run by rows in 183 us, where the union takes 42).  Of V
    // visible chunks a block's BQ queries then want V (1 - (1 - k / V)^BQ).  A chunk of it takes 0.8 us and a
    // block's set-up 5 us (8K prefill, 62 chunks on average: 810 us against 1.32 ms by rows; 509 queries at 130K, 810 chunks
    // a block of which a query wants 33: 474 us against 184).
    const double BQ = 128 / p.G, V = (p.q_offset + 0.5 * p.N) / p.C + 1.0;
    const double U = V * (1.0 - pow(1.0 - fmin(1.0, p.k / V), BQ)) + BQ / p.C + 1.0;
    const double blocks = (double)p.B * p.Hkv * ((p.N + BQ - 1) / BQ) / 148.0;
    const double t_union = (blocks <= 1.0 ? 1.0 : blocks + 0.5) * (5.0 + 0.8 * fmin(U, V + 1.0));
    return t_union < 1.9 * share_of(p, blocks_per_sm(p.d, p.C, false), heads_of(false)).time;
}

cudaError_t launch_attend8(const Dims &p, hils_dtype in, hils_dtype out, const void *Q, const uint8_t *K8,
                           const uint8_t *V8, const float *ks, const float *vs, const int32_t *sel_idx,
                           const float *sel_score, void *O, const DeviceCtl &ctl, cudaStream_t s)
{
    if (use_union(p, in, out)) return launch_attend8_tc(p, Q, K8, V8, ks, vs, sel_idx, sel_score, O, ctl, s);
    if (in == HILS_F32)
        return out == HILS_F32 ? launch_d<float, float>(p, Q, K8, V8, ks, vs, sel_idx, sel_score, O, s)
                               : launch_d<float, __nv_bfloat16>(p, Q, K8, V8, ks, vs, sel_idx, sel_score, O, s);
    return out == HILS_F32 ? launch_d<__nv_bfloat16, float>(p, Q, K8, V8, ks, vs, sel_idx, sel_score, O, s)
                           : launch_d<__nv_bfloat16, __nv_bfloat16>(p, Q, K8, V8, ks, vs, sel_idx, sel_score, O, s);
}

}  // namespace hils
