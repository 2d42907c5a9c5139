// attend8_tc.cu -- prefill attention over the 8-bit cache on the sm_100a tensor cores (bf16 in and out, d = 128, C = 64).
//
// "Hierarchical Sparse Attention Done Right" (arXiv 2607.02980v1), Sec. 4 "Kernel design": adjacent queries share chunks,
// so a block of queries is processed over the union of their chunks; Abstract / Sec. 3 "Hierarchical softmax": softmax
// inside every chunk, chunk outputs fused by the softmax of the retrieval scores.  With keys ks_c e and values vs_c e':
//   P = (w_c vs_c / l) exp(x - max x),  x = (scale ks_c) <q, e>,  O = sum_c P e'.
//
// One CTA owns 128 rows = (128 / G) consecutive queries x the G heads of a kv-group and walks the union of their chunks,
// two at a time.  The cache's bytes are tensor-core operands where they can be:
//   S = Q K^T   kind::f8f6f4: key tiles as TMA brings them.  A bf16 query row is scaled by a power of two so that its
//               largest element lies in [2^7, 2^8), and is the sum of two e4m3 values (8 bits in two times 4).  The
//               second's step is 2^-9: elements below 2^-9 of the row's largest lose up to 2^-17 of it (2^-10 on 2^7), all
//               others nothing.  So two products replace a conversion of every key tile.
//   O += P V    kind::f16: the probabilities keep f16's 11 bits (three e4m3 products would be needed for
//               that), so value tiles are widened to f16 (exact) in shared memory by four warps of their own.
//               (By the softmax warps, between their other work, the 8K prefill took 946 us.)
// What a row's weights w_c vs_c are divided by is the row's own largest, times 2^-14: f16 rounds a weight by 2^-11 of
// itself down to 2^-28 of the largest, and the row is multiplied back in float32 at the end.
//
// Roles, meeting on mbarriers (pair p = chunks 2p, 2p + 1 of the union; buffers go by p % 2):
//   warp 0  TMA of key pairs    (K_LAND; a slot frees with the key product, QK_DONE)
//   warp 1  TMA of value pairs  (V8_LAND; a slot frees when four warps have widened it, V8_FREE); TMEM
//   warp 2  key products        (after K_LAND and S_FREE, the eight warps' reads of pair p - 2; announces QK_DONE)
//   warp 3  value products      (after PV_READY, eight warps, and V16_READY, four; announces PV_DONE)
//   warps 4..7   widen value pairs (after V8_LAND, and PV_DONE of pair p - 2, which frees the f16 slot)
//   warps 8..19  three softmax groups of four, group t % 3 takes chunk t, a thread a row: reads S from TMEM, writes P to it
//           (after PV_DONE of pair p - 2)
// A parity wait must not run two phases ahead: a softmax warp skips pairs, but one that waits for PV_DONE of pair p - 2 has
// seen that of p - 4 or of a later pair, and products complete in order.  Every wait is bounded; on expiry the CTA
// records HILS_ERR_TIMEOUT, drains its copies and products, frees its TMEM and exits.
//
// Registers: 640 threads start with 96 each; the first four warps keep 40, the widening ones 56 and the softmax
// warps take 128 (the sum of the shares is what the block was launched with, which the host checks).
#include <cuda.h>
#include <cuda_fp16.h>
#include <stdlib.h>
#include <string.h>

#include <atomic>

#include "cache8.h"
#include "chunk_softmax.cuh"
#include "common.cuh"
#include "e4m3.cuh"
#include "sm100.cuh"

namespace hils {
namespace {

using namespace sm100;

constexpr int kGroups = 3;
constexpr int kSoft = 8;                              // first softmax warp
constexpr int kThreads = 32 * kSoft + 128 * kGroups;
constexpr int kLaunchRegs = 96;                       // registers a thread is launched with
constexpr int kRegsIssue = 40, kRegsWiden = 56, kRegsSoft = 128;
static_assert(kRegsIssue + kRegsWiden + kGroups * kRegsSoft == kThreads / 128 * kLaunchRegs, "register shares");
constexpr int kRows = 128;
constexpr int kChunk = 64;
constexpr int kD = 128;
constexpr uint32_t kTmemCols = 512;                  // two S pairs (128 columns each), O (128), two P pairs (64 each)
constexpr uint32_t kColO = 256, kColP = 384;
constexpr uint32_t kQTile = kRows * kD;              // bytes of one of the query's two e4m3 tiles
constexpr uint32_t kPair8 = 2 * kChunk * kD;         // a pair of e4m3 tiles
constexpr uint32_t kPair16 = 2 * kPair8;             // f16 values: [c0 d0-63 | c1 d0-63 | c0 d64-127 | c1 d64-127]
constexpr unsigned long long kDrainNs = 2000000000ull;
constexpr int kPolyPairEvery = 0;   // every exponential on the special-function unit (8K prompt: 810 us; one pair in eight by
                                      // polynomial 823, in four 833, in two 940)
constexpr float kTopW = 16384.0f;

constexpr uint32_t IDESC_QK2 = idesc_f16_f32(128, 128, false, false);   // kind::f8f6f4 reads the same fields: 0 is e4m3
constexpr uint32_t IDESC_QK1 = idesc_f16_f32(128, 64, false, false);
constexpr uint32_t IDESC_PV = idesc_f16_f32(128, 128, false, true);

// D[tmem] (+)= A[smem] * B[smem], kind::f8f6f4 (e4m3 in, f32 accumulate), one CTA
__device__ __forceinline__ void mma_f8_ss(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

struct Layout {
    uint32_t q, k, v8, v16, bar, misc, bitmap, uni, selbuf, wts, qlist, qslot, qvs, qcnt, fq, top, total;
};

__host__ __device__ inline uint32_t al16(uint32_t x) { return (x + 15u) & ~15u; }

enum : int { K_LAND = 0, S_FREE = 2, QK_DONE = 4, V8_LAND = 6, V8_FREE = 8, V16_READY = 10, PV_READY = 12, PV_DONE = 14, MMA_DONE = 16, O_FULL = 18, N_BARS = 19 };

__host__ __device__ inline Layout make_layout(int k, int nwords, int BQ)
{
    Layout L;
    const uint32_t ns = (uint32_t)(k + 1);
    L.q = 0;
    L.k = 2 * kQTile;
    L.v8 = L.k + 2 * kPair8;
    L.v16 = L.v8 + 2 * kPair8;
    L.bar = L.v16 + 2 * kPair16;
    L.misc = L.bar + al16(N_BARS * 8);
    L.bitmap = L.misc + 16;
    L.uni = al16(L.bitmap + 4u * (uint32_t)nwords);
    L.selbuf = al16(L.uni + 4u * ns * (uint32_t)BQ);
    L.wts = al16(L.selbuf + 4u * (uint32_t)k * (uint32_t)BQ);     // scores, then weights, by slot: [row][slot]
    L.qlist = al16(L.wts + 4u * ns * (uint32_t)kRows);            // a query's chunks, ascending
    L.qslot = al16(L.qlist + 4u * ns * (uint32_t)BQ);             // and their slots
    L.qvs = al16(L.qslot + 4u * ns * (uint32_t)BQ);               // value scales by slot
    L.qcnt = al16(L.qvs + 4u * ns * (uint32_t)BQ);
    L.fq = al16(L.qcnt + 4u * (uint32_t)BQ);                      // a row's logit factor
    L.top = L.fq + 4u * kRows;                                    // a row's largest weight * 2^-14
    L.total = L.top + 4u * kRows;
    return L;
}

// lane 0 waits, the result is broadcast so the warp decides uniformly
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, unsigned long long lim, volatile int *abort_flag,
                                          unsigned int *status)
{
    int ok = 0;
    if ((threadIdx.x & 31) == 0) ok = mbar_wait(bar, parity, lim, abort_flag, status) ? 1 : 0;
    return __shfl_sync(0xFFFFFFFFu, ok, 0) != 0;
}

template <int G>
__global__ void __launch_bounds__(kThreads, 1)
    attend8_tc_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, Dims p,
                      const __nv_bfloat16 *__restrict__ Q, const float *__restrict__ ks, const float *__restrict__ vs,
                      const int32_t *__restrict__ sel_idx, const float *__restrict__ sel_score,
                      __nv_bfloat16 *__restrict__ O, unsigned int *status, unsigned long long limit_ns, int nwords,
                      int inject_stall)
{
    constexpr int BQ = kRows / G;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *base = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    const Layout Ly = make_layout(p.k, nwords, BQ);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // later query tiles see more chunks and take longer: they are dispatched first
    const int q0 = (int)(gridDim.x - 1 - blockIdx.x) * BQ, g = blockIdx.y, b = blockIdx.z;
    const int nq = min(BQ, p.N - q0);
    const int ns = p.k + 1;
    const int t_end = (int)min((long long)p.T, (long long)p.q_offset + q0 + nq);   // no query of the block sees a later token

    const uint32_t sQ = smem_addr(base + Ly.q), sK = smem_addr(base + Ly.k), sV8 = smem_addr(base + Ly.v8);
    const uint32_t sV16 = smem_addr(base + Ly.v16), bar0 = smem_addr(base + Ly.bar);
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(base + Ly.misc);
    int *n_union_p = reinterpret_cast<int *>(base + Ly.misc + 4);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(base + Ly.misc + 8);
    uint32_t *bitmap = reinterpret_cast<uint32_t *>(base + Ly.bitmap);
    int *uni = reinterpret_cast<int *>(base + Ly.uni);
    int *selbuf = reinterpret_cast<int *>(base + Ly.selbuf);
    float *wts = reinterpret_cast<float *>(base + Ly.wts);
    int *qlist = reinterpret_cast<int *>(base + Ly.qlist);
    int *qslot = reinterpret_cast<int *>(base + Ly.qslot);
    float *qvs = reinterpret_cast<float *>(base + Ly.qvs);
    int *qcnt = reinterpret_cast<int *>(base + Ly.qcnt);
    float *fqs = reinterpret_cast<float *>(base + Ly.fq);
    float *tops = reinterpret_cast<float *>(base + Ly.top);
    auto BAR = [&](int i) { return bar0 + 8u * (uint32_t)i; };
    const size_t bg = (size_t)b * p.Hkv + g;
    const float *ksb = ks + bg * p.nL, *vsb = vs + bg * p.nL;

    // ---- set-up --------------------------------------------------------------
    if (tid == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(BAR(K_LAND + s), 1);
            mbar_init(BAR(S_FREE + s), 8);
            mbar_init(BAR(QK_DONE + s), 1);
            mbar_init(BAR(V8_LAND + s), 1);
            mbar_init(BAR(V8_FREE + s), 4);
            mbar_init(BAR(V16_READY + s), 4);
            mbar_init(BAR(PV_READY + s), 8);
            mbar_init(BAR(PV_DONE + s), 1);
            mbar_init(BAR(MMA_DONE + s), 1);
        }
        mbar_init(BAR(O_FULL), 1);
        fence_mbar_init();
        *abort_flag = 0;
        prefetch_tensormap(&tmK);
        prefetch_tensormap(&tmV);
    }
    if (warp == 1) {
        tmem_alloc(smem_addr(tmem_holder), kTmemCols);
        tmem_relinquish();
    }
    // every global load of the set-up is in flight before the first is used: the block's query rows (eight a warp, four
    // elements a lane), its selection and its scores
    uint2 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = 8 * warp + i, qi = r / G, h = r % G;
        v[i] = make_uint2(0u, 0u);
        if (r < kRows && qi < nq) v[i] = __ldg(reinterpret_cast<const uint2 *>(Q + ((bg * G + h) * p.N + q0 + qi) * kD) + lane);
    }
    for (int i = tid; i < nwords; i += kThreads) bitmap[i] = 0u;
    const int32_t *sel_base = sel_idx + (bg * p.N + q0) * p.k;
#pragma unroll 4
    for (int e = tid; e < nq * p.k; e += kThreads) {
        // an entry that is no past chunk of its query is an empty slot: nothing outside the cache is read for it
        const int c = __ldg(sel_base + e), own_c = (int)(((long long)p.q_offset + q0 + e / p.k) / kChunk);
        selbuf[e] = (unsigned)c < (unsigned)own_c ? c : -1;
    }
#pragma unroll 4
    for (int e = tid; e < G * nq * ns; e += kThreads) {
        const int h = e / (nq * ns), rem = e - h * (nq * ns), qi = rem / ns;
        wts[(qi * G + h) * ns + rem - qi * ns] = __ldg(sel_score + (bg * G + h) * p.N * ns + (size_t)q0 * ns + rem);
    }
    // the query rows as two e4m3 tiles with the 128-byte swizzle
    if (warp < kRows / 8) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = 8 * warp + i;
            float x[4] = {__uint_as_float(v[i].x << 16), __uint_as_float(v[i].x & 0xFFFF0000u),
                          __uint_as_float(v[i].y << 16), __uint_as_float(v[i].y & 0xFFFF0000u)};
            // the largest magnitude's bits: one integer reduction over the warp
            const float m = __uint_as_float(__reduce_max_sync(
                0xFFFFFFFFu, __float_as_uint(fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3]))))));
            const int sh = min(7 - ((int)(__float_as_uint(m) >> 23) - 127), 120);
            const float f = exp2_int(sh);
            float rest[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] *= f;
            const uint32_t hi = to_e4m3x4(x[0], x[1], x[2], x[3]);
            e4m3x4_to_float(hi, rest);
            const uint32_t lo = to_e4m3x4(x[0] - rest[0], x[1] - rest[1], x[2] - rest[2], x[3] - rest[3]);
            const uint32_t at = (uint32_t)r * 128u + ((uint32_t)((lane >> 2) ^ (r & 7)) << 4) + (uint32_t)(lane & 3) * 4u;
            *reinterpret_cast<uint32_t *>(base + Ly.q + at) = hi;
            *reinterpret_cast<uint32_t *>(base + Ly.q + kQTile + at) = lo;
            if (lane == 0) fqs[r] = p.scale * 1.4426950408889634f * exp2_int(-sh);
        }
    }
    fence_proxy_async_smem();
    __syncthreads();

    // mark the selected and own chunks; with few bitmap words the bits are OR-reduced across the warp first, so that
    // the shared-memory atomics do not all land on the same words
    const int n_marks = nq * p.k + nq;
    for (int e0 = warp * 32; e0 < n_marks; e0 += kThreads) {
        const int e = e0 + lane;
        int c = -1;
        if (e < nq * p.k) c = selbuf[e];
        else if (e < n_marks) c = (int)(((long long)p.q_offset + q0 + (e - nq * p.k)) / kChunk);
        if (nwords <= 8) {
            for (int wd = 0; wd < nwords; ++wd) {
                const unsigned int bits = __reduce_or_sync(0xFFFFFFFFu, (c >= 0 && (c >> 5) == wd) ? (1u << (c & 31)) : 0u);
                if (lane == 0 && bits) atomicOr(&bitmap[wd], bits);
            }
        } else if (c >= 0) {
            atomicOr(&bitmap[c >> 5], 1u << (c & 31));
        }
    }
    __syncthreads();

    if (warp == 0) {
        // ascending list of the union's chunks
        int running = 0;
        for (int w0 = 0; w0 < nwords; w0 += 32) {
            uint32_t word = (w0 + lane < nwords) ? bitmap[w0 + lane] : 0u;
            const int cnt = __popc(word);
            int incl = cnt;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xFFFFFFFFu, incl, o);
                if (lane >= o) incl += y;
            }
            int off = running + incl - cnt;
            while (word) {
                const int bit = __ffs(word) - 1;
                uni[off++] = (w0 + lane) * 32 + bit;
                word &= word - 1;
            }
            running += __shfl_sync(0xFFFFFFFFu, incl, 31);
        }
        if (lane == 0) *n_union_p = running;
    }
    // each query's chunks in ascending order with the slot each came from: one thread per (query, slot) counts the
    // query's smaller chunks (chunks are distinct; of one named twice, against the rule, the first slot counts)
    for (int e = tid - 32; e >= 0 && e < nq * ns; e += kThreads - 32) {
        const int qi = e / ns, j = e % ns;
        const int own_c = (int)(((long long)p.q_offset + q0 + qi) / kChunk);
        const int *sl = selbuf + qi * p.k;
        const int c = (j < p.k) ? sl[j] : own_c;
        qvs[qi * ns + j] = c < 0 ? 0.f : __ldg(vsb + c);
        if (c < 0) continue;
        int rank = 0;
        for (int j2 = 0; j2 < p.k; ++j2)   // -1 never counts
            rank += (unsigned)sl[j2] < (unsigned)c + (unsigned)(j2 < j);
        rank += own_c < c;
        qlist[qi * ns + rank] = c;
        qslot[qi * ns + rank] = j;
        if (j == p.k) qcnt[qi] = rank + 1;   // the own chunk is the largest
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_holder;
    const int n_union = *n_union_p, n_pairs = (n_union + 1) >> 1;

    // the roles' register shares (whole warpgroups: warps 0..3, 4..7 and the softmax groups)
    if (warp < 4) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssue));
    else if (warp < kSoft) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsWiden));
    else asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoft));

    if (warp < 2) {
        // ---------------- key (warp 0) and value (warp 1) tiles, two chunks per slot
        if (lane == 0) {
            const CUtensorMap *tm = warp == 0 ? &tmK : &tmV;
            const uint32_t land = BAR(warp == 0 ? K_LAND : V8_LAND), freed = BAR(warp == 0 ? QK_DONE : V8_FREE);
            const uint32_t dst0 = warp == 0 ? sK : sV8;
            const int row0 = (int)(bg * p.T);
            int pr = 0;
            for (; pr < n_pairs; ++pr) {
                const uint32_t st = (uint32_t)(pr & 1);
                if (pr >= 2 && !mbar_wait(freed + 8u * st, (uint32_t)(((pr >> 1) - 1) & 1), limit_ns, abort_flag, status)) break;
                const bool two = 2 * pr + 1 < n_union;
                mbar_arrive_expect_tx(land + 8u * st, two ? kPair8 : kPair8 / 2);
                tma_load_2d(dst0 + st * kPair8, tm, land + 8u * st, 0, row0 + uni[2 * pr] * kChunk);
                if (two) tma_load_2d(dst0 + st * kPair8 + kPair8 / 2, tm, land + 8u * st, 0, row0 + uni[2 * pr + 1] * kChunk);
            }
            // the copies land before the CTA exits
            for (int v = pr > 2 ? pr - 2 : 0; v < pr; ++v)
                mbar_drain(land + 8u * (uint32_t)(v & 1), (uint32_t)((v >> 1) & 1), kDrainNs);
        }
        __syncwarp();
    } else if (warp < 4) {
        // ---------------- MMA issue: warp 2 the key products, warp 3 the value products
        if (lane == 0) {
            const bool keys = warp == 2;
            bool ok = true;
            // test control: wait once on a barrier nothing signals, so the bounded wait expires
            if (keys && inject_stall) ok = mbar_wait(BAR(MMA_DONE), 0, limit_ns, abort_flag, status);
            const uint64_t dq = smem_desc_sw128(sQ, 16, 1024);
            for (int i = 0; ok && i < n_pairs; ++i) {
                const int sl = i & 1;
                const uint32_t ph = (uint32_t)((i >> 1) & 1);
                if (keys) {
                    ok = mbar_wait(BAR(K_LAND + sl), ph, limit_ns, abort_flag, status) &&
                         (i < 2 || mbar_wait(BAR(S_FREE + sl), ph ^ 1u, limit_ns, abort_flag, status));
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t dk = smem_desc_sw128(sK + (uint32_t)sl * kPair8, 16, 1024);
                    const uint32_t idesc = (2 * i + 1 < n_union) ? IDESC_QK2 : IDESC_QK1;
#pragma unroll
                    for (int s = 0; s < 8; ++s)   // both pieces of the query, four steps of 32 each
                        mma_f8_ss(tmem + (uint32_t)sl * 128u, dq + (uint64_t)(((s >> 2) * kQTile + (s & 3) * 32u) >> 4),
                                  dk + (uint64_t)(((s & 3) * 32u) >> 4), idesc, s > 0 ? 1u : 0u);
                    mma_commit(BAR(QK_DONE + sl));
                } else {
                    ok = mbar_wait(BAR(V16_READY + sl), ph, limit_ns, abort_flag, status) &&
                         mbar_wait(BAR(PV_READY + sl), ph, limit_ns, abort_flag, status);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t pa = tmem + kColP + (uint32_t)sl * 64u;
                    const uint64_t dv = smem_desc_sw128(sV16 + (uint32_t)sl * kPair16, 16384, 1024);
                    const int steps = (2 * i + 1 < n_union) ? 8 : 4;
#pragma unroll
                    for (int s = 0; s < 8; ++s)
                        if (s < steps)
                            mma_f16_ts(tmem + kColO, pa + 8u * s, dv + (uint64_t)((2048u * s) >> 4), IDESC_PV,
                                       (i > 0 || s > 0) ? 1u : 0u);
                    mma_commit(BAR(PV_DONE + sl));
                }
            }
            if (ok && !keys) mma_commit(BAR(O_FULL));
            // drain: every MMA this thread issued completes before TMEM is released
            const uint32_t done = BAR(MMA_DONE + (keys ? 0 : 1));
            mma_commit(done);
            mbar_drain(done, 0, kDrainNs);
        }
        __syncwarp();
    } else if (warp < kSoft) {
        // ---------------- value pairs to f16: 16 bytes (key row, d = 16 j ..) a step
        const int th = tid - 128, j = th & 7;
        for (int pr = 0; pr < n_pairs; ++pr) {
            const int sl = pr & 1;
            const uint32_t ph = (uint32_t)((pr >> 1) & 1);
            if (!warp_wait(BAR(V8_LAND + sl), ph, limit_ns, abort_flag, status) ||
                (pr >= 2 && !warp_wait(BAR(PV_DONE + sl), ph ^ 1u, limit_ns, abort_flag, status)))
                break;
            const int n_ch = (2 * pr + 1 < n_union) ? 2 : 1;
            for (int x = 0; x < n_ch; ++x) {
                const int left = t_end - uni[2 * pr + x] * kChunk;   // rows behind the last query become zeros
                const unsigned char *src = base + Ly.v8 + sl * kPair8 + x * (kPair8 / 2);
                unsigned char *dst = base + Ly.v16 + sl * kPair16 + x * 8192u + (j >> 2) * 16384u;
                uint4 v[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int row = (th + 128 * u) >> 3;
                    v[u] = reinterpret_cast<const uint4 *>(src)[row * 8 + (j ^ (row & 7))];
                }
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int row = (th + 128 * u) >> 3;
                    if (row >= left) v[u] = make_uint4(0u, 0u, 0u, 0u);
                    const uint4 a = make_uint4(e4m3x2_to_f16x2(v[u].x), e4m3x2_to_f16x2(v[u].x >> 16),
                                               e4m3x2_to_f16x2(v[u].y), e4m3x2_to_f16x2(v[u].y >> 16));
                    const uint4 z = make_uint4(e4m3x2_to_f16x2(v[u].z), e4m3x2_to_f16x2(v[u].z >> 16),
                                               e4m3x2_to_f16x2(v[u].w), e4m3x2_to_f16x2(v[u].w >> 16));
                    // the second half's odd pieces go first: eight lanes, eight bank groups
                    const int e = (2 * j) & 7, odd = j >> 2;
                    *reinterpret_cast<uint4 *>(dst + row * 128u + (((e + odd) ^ (row & 7)) << 4)) = odd ? z : a;
                    *reinterpret_cast<uint4 *>(dst + row * 128u + (((e + 1 - odd) ^ (row & 7)) << 4)) = odd ? a : z;
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(BAR(V8_FREE + sl));
                mbar_arrive(BAR(V16_READY + sl));
            }
        }
    } else {
        // ---------------- softmax groups (chunks round-robin) and epilogue
        {
            // weights of each row by slot, eight lanes a row: w vs over the row's largest, times 2^14
            const int l8 = lane & 7;
            constexpr int S8 = (HILS_MAX_K + 8) / 8;   // slots a lane holds at most
            auto max8 = [](float x) {
#pragma unroll
                for (int o = 4; o; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, o));
                return x;
            };
            for (int r = 4 * (warp - kSoft) + (lane >> 3); r < kRows; r += 16 * kGroups) {   // the same count for every warp's lanes
                const int qi = min(r / G, nq - 1);
                float *sc = wts + r * ns;
                const int *sl = selbuf + qi * p.k;
                const float *sv = qvs + qi * ns;
                const bool live = r / G < nq;
                float x[S8], M = -INFINITY, Z = 0.f, top = 0.f;
#pragma unroll
                for (int u = 0; u < S8; ++u) {
                    const int j = l8 + 8 * u;
                    x[u] = -INFINITY;
                    if (8 * u < ns) {   // a slot without a chunk has no weight, whatever its score
                        if (live && j < ns && (j == p.k || sl[j] >= 0)) x[u] = sc[j];
                        M = fmaxf(M, x[u]);
                    }
                }
                M = max8(M);
#pragma unroll
                for (int u = 0; u < S8; ++u)
                    if (8 * u < ns) {
                        x[u] = (x[u] == -INFINITY) ? 0.f : __expf(x[u] - M);
                        Z += x[u];
                    }
#pragma unroll
                for (int o = 4; o; o >>= 1) Z += __shfl_xor_sync(0xFFFFFFFFu, Z, o);
                const float iz = Z == 0.f ? 0.f : 1.0f / Z;
#pragma unroll
                for (int u = 0; u < S8; ++u)
                    if (8 * u < ns) {
                        const int j = l8 + 8 * u;
                        x[u] = (x[u] == 0.f || j >= ns) ? 0.f : x[u] * iz * sv[j];
                        top = fmaxf(top, x[u]);
                    }
                top = max8(top);
                if (top > 0.f) top = fmaxf(top, 1e-34f);   // its inverse stays finite
                const float f = top > 0.f ? kTopW / top : 1.0f;
#pragma unroll
                for (int u = 0; u < S8; ++u)
                    if (l8 + 8 * u < ns) sc[l8 + 8 * u] = x[u] * f;
                if (l8 == 0) tops[r] = top > 0.f ? top * (1.0f / kTopW) : 0.f;
            }
        }
        // the softmax warps wait for the weights (named barrier 1: theirs only)
        asm volatile("bar.sync 1, %0;" ::"r"(32 * 4 * kGroups) : "memory");
        const int grp = (warp - kSoft) >> 2;
        const int qq = warp & 3;
        const int r = 32 * qq + lane, h = r % G, qi = r / G;
        const bool valid = qi < nq;
        const long long pos = (long long)p.q_offset + q0 + qi;
        const int own = (int)(pos / kChunk);
        const int cnt = valid ? qcnt[qi] : 0;
        const int *lst = qlist + qi * ns, *slt = qslot + qi * ns;
        const float *wr = wts + r * ns;
        const float fq = fqs[r];
        const uint32_t lane_off = (uint32_t)(32 * qq) << 16;
        int ptr = 0;
        bool ok = true;
        for (int t = grp; t < n_union; t += kGroups) {
            const int pr = t >> 1, sl = pr & 1;
            const uint32_t ph = (uint32_t)((pr >> 1) & 1);
            const int c = uni[t];
            const float kc = __ldg(ksb + c);
            const int left = min(kChunk, t_end - c * kChunk);   // tokens of the chunk that any query of the block sees
            if (!warp_wait(BAR(QK_DONE + sl), ph, limit_ns, abort_flag, status)) { ok = false; break; }
            tc_fence_after();
            uint32_t sv[64];
            const uint32_t tS = tmem + lane_off + (uint32_t)sl * 128u + (uint32_t)(t & 1) * 64u;
            tmem_ld32(tS, sv);
            tmem_ld32(tS + 32u, sv + 32);
            tmem_wait_ld();
            // the scores are in registers: the S buffer may take the pair after next
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(BAR(S_FREE + sl));

            while (ptr < cnt && lst[ptr] < c) ++ptr;
            const float w = (ptr < cnt && lst[ptr] == c) ? wr[slt[ptr]] : 0.f;
            uint32_t pk[32];
            if (__any_sync(0xFFFFFFFFu, w != 0.f)) {   // rows with w = 0 get P = 0 from the scaling
                const int n_vis = (c == own && valid) ? (int)(pos - (long long)c * kChunk + 1) : left;
                // a factor too small for float32 makes every logit the same number: the smallest normal one does that too.
                // A row without weight takes that one: its own may be beyond float32, and a NaN would outlive w = 0
                const float f = w == 0.f ? 0.f : fq * kc;
                chunk_softmax_row<kPolyPairEvery>(sv, n_vis, w, fmaxf(f, 1.2e-38f), pk);
            } else {
#pragma unroll
                for (int j = 0; j < 32; ++j) pk[j] = 0u;
            }
            if (pr >= 2 && !warp_wait(BAR(PV_DONE + sl), ph ^ 1u, limit_ns, abort_flag, status)) { ok = false; break; }
            tmem_st32(tmem + lane_off + kColP + (uint32_t)sl * 64u + (uint32_t)(t & 1) * 32u, pk);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(BAR(PV_READY + sl));
                // a lone last chunk has no second group: this one stands in for it
                if (t == n_union - 1 && !(t & 1)) mbar_arrive(BAR(PV_READY + sl));
            }
        }
        if (ok && warp_wait(BAR(O_FULL), 0, limit_ns, abort_flag, status)) {
            tc_fence_after();
            const float f = valid ? tops[r] : 0.f;
            __nv_bfloat16 *orow = O + ((bg * G + h) * p.N + q0 + qi) * kD;
            for (int cb = grp; cb < kD / 32; cb += kGroups) {
                uint32_t v[32];
                tmem_ld32(tmem + lane_off + kColO + (uint32_t)(cb * 32), v);
                tmem_wait_ld();
                if (valid) {
#pragma unroll
                    for (int i = 0; i < 32; i += 8) {
                        uint32_t w4[4];
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            const __nv_bfloat162 a = __floats2bfloat162_rn(__uint_as_float(v[i + 2 * x]) * f,
                                                                           __uint_as_float(v[i + 2 * x + 1]) * f);
                            w4[x] = *reinterpret_cast<const uint32_t *>(&a);
                        }
                        *reinterpret_cast<uint4 *>(orow + cb * 32 + i) = make_uint4(w4[0], w4[1], w4[2], w4[3]);
                    }
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

constexpr uint32_t kSmemLimit = 227 * 1024;

uint32_t smem_bytes(const Dims &p)
{
    const int c_max = (int)(((long long)p.q_offset + p.N - 1) / kChunk);
    return make_layout(p.k, c_max / 32 + 1, kRows / p.G).total + 1024;
}

// The warps' register shares are drawn from what the block is launched with: a build whose kernel has another number of
// registers would wait for them forever, and does not run it.  A query of the number that fails is made again by the next
// call.  Test control: HILS_Q8_UNION_UNFIT=1 takes this build for such a one.
template <int G>
bool fits_g()
{
    static std::atomic<int> known{0};
    int regs = known.load(std::memory_order_relaxed);
    if (regs == 0) {
        cudaFuncAttributes a;
        if (cudaFuncGetAttributes(&a, attend8_tc_kernel<G>) != cudaSuccess) {
            (void)cudaGetLastError();
            return false;
        }
        regs = a.numRegs;
        known.store(regs, std::memory_order_relaxed);
    }
    const char *unfit = getenv("HILS_Q8_UNION_UNFIT");
    return regs == kLaunchRegs && !(unfit && strcmp(unfit, "1") == 0);
}

template <int G>
cudaError_t launch_g(const Dims &p, const void *Q, const uint8_t *K8, const uint8_t *V8, const float *ks, const float *vs,
                     const int32_t *sel_idx, const float *sel_score, void *O, const DeviceCtl &ctl, cudaStream_t s)
{
    constexpr int BQ = kRows / G;
    CUtensorMap tk, tv;
    const cuuint64_t dims[2] = {(cuuint64_t)kD, (cuuint64_t)p.B * p.Hkv * p.T};
    const cuuint64_t strides[1] = {(cuuint64_t)kD};
    const cuuint32_t box[2] = {(cuuint32_t)kD, (cuuint32_t)kChunk};
    if (!encode_tensor_map_sw128(&tk, CU_TENSOR_MAP_DATA_TYPE_UINT8, K8, 2, dims, strides, box) ||
        !encode_tensor_map_sw128(&tv, CU_TENSOR_MAP_DATA_TYPE_UINT8, V8, 2, dims, strides, box))
        return cudaErrorInvalidValue;
    const int c_max = (int)(((long long)p.q_offset + p.N - 1) / kChunk);
    const uint32_t smem = smem_bytes(p);
    auto kern = attend8_tc_kernel<G>;
    if (!fits_g<G>()) return cudaErrorInvalidConfiguration;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    kern<<<dim3((p.N + BQ - 1) / BQ, p.Hkv, p.B), kThreads, smem, s>>>(
        tk, tv, p, static_cast<const __nv_bfloat16 *>(Q), ks, vs, sel_idx, sel_score, static_cast<__nv_bfloat16 *>(O),
        ctl.status, (unsigned long long)ctl.wait_limit, c_max / 32 + 1, ctl.inject_stall);
    return cudaGetLastError();
}

}  // namespace

bool attend8_tc_supported(const Dims &p, hils_dtype in, hils_dtype out)
{
    if (in != HILS_BF16 || out != HILS_BF16 || p.d != kD || p.C != kChunk || p.N < 2) return false;
    if (p.G != 1 && p.G != 2 && p.G != 4 && p.G != 8 && p.G != 16) return false;
    if ((long long)p.B * p.Hkv * p.T > 0x7FFFFFFFll) return false;   // a tile's row is a 32-bit coordinate
    return smem_bytes(p) <= kSmemLimit;
}

bool attend8_tc_fits(const Dims &p)
{
    return p.G == 1 ? fits_g<1>() : p.G == 2 ? fits_g<2>() : p.G == 4 ? fits_g<4>() : p.G == 8 ? fits_g<8>() : fits_g<16>();
}

cudaError_t launch_attend8_tc(const Dims &p, const void *Q, const uint8_t *K8, const uint8_t *V8, const float *ks,
                              const float *vs, const int32_t *sel_idx, const float *sel_score, void *O,
                              const DeviceCtl &ctl, cudaStream_t s)
{
    auto *f = p.G == 1 ? launch_g<1> : p.G == 2 ? launch_g<2> : p.G == 4 ? launch_g<4> : p.G == 8 ? launch_g<8> : launch_g<16>;
    return f(p, Q, K8, V8, ks, vs, sel_idx, sel_score, O, ctl, s);
}

}  // namespace hils
