// cache8.h -- launchers of the 8-bit key/value cache (not part of the ABI): writing and reading it, landmark
// generation from its keys, and chunk attention over it.  K8 / V8 are e4m3 bytes [B][Hkv][T][d]; ks / vs hold one
// float32 scale per (b, kv-head, chunk).
#pragma once

#include "internal.h"

namespace hils {

// The part of a problem that the cache's own calls use.
struct Cache8 {
    int B, Hkv, T, d, C, nL;
};

cudaError_t launch_cache_append(const Cache8 &c, hils_dtype in, const void *K, const void *V, uint8_t *K8, uint8_t *V8,
                                float *ks, float *vs, int t0, int t1, cudaStream_t s);
cudaError_t launch_cache_read(const Cache8 &c, hils_dtype out, const uint8_t *K8, const uint8_t *V8, const float *ks,
                              const float *vs, void *K, void *V, int t0, int t1, cudaStream_t s);
// Landmarks of chunks [c0, c1) from key rows below t_end.
cudaError_t launch_landmarks8(const Cache8 &c, hils_dtype in, float scale, const uint8_t *K8, const float *ks,
                              const void *U, void *L, float *beta, int c0, int c1, int t_end, cudaStream_t s);

// Chunk attention over the 8-bit cache: rows of work (every shape and type), or the union of a query block's chunks on
// the tensor cores (bf16 in and out, d = 128, C = 64).
bool attend8_tc_supported(const Dims &p, hils_dtype in, hils_dtype out);
bool attend8_tc_fits(const Dims &p);   // this build's kernel has the registers that its warps share out
cudaError_t launch_attend8_tc(const Dims &p, const void *Q, const uint8_t *K8, const uint8_t *V8, const float *ks,
                              const float *vs, const int32_t *sel_idx, const float *sel_score, void *O,
                              const DeviceCtl &ctl, cudaStream_t s);
cudaError_t launch_attend8(const Dims &p, hils_dtype in, hils_dtype out, const void *Q, const uint8_t *K8,
                           const uint8_t *V8, const float *ks, const float *vs, const int32_t *sel_idx,
                           const float *sel_score, void *O, const DeviceCtl &ctl, cudaStream_t s);

}  // namespace hils
