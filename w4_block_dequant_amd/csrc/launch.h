// Kernel launchers (one per entry point).  Arguments are already validated;
// each launcher only enqueues work on `stream` and returns hipGetLastError().
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "plan.h"
#include "splitk.h"

namespace w4 {

// scales are fp32, or binary16 bit patterns when f16 is set
hipError_t launch_quantize_pack(const float *W, int64_t K, int64_t N, uint8_t *Wq, void *scales,
                                bool f16, uint8_t *zeros, int *d_status, hipStream_t stream);
hipError_t launch_unpack(const uint8_t *Wq, const uint8_t *zeros, int64_t K, int64_t N,
                         uint8_t *q, uint8_t *z, hipStream_t stream);
hipError_t launch_dequantize(const uint8_t *Wq, const void *scales, bool f16,
                             const uint8_t *zeros, int64_t K, int64_t N, float *out,
                             hipStream_t stream);

hipError_t launch_gemv(const GemvPlan &plan, const float *x, int64_t K, const uint8_t *Wq,
                       const float *scales, const uint8_t *zeros, int64_t N, const float *bias,
                       float *y, void *workspace, hipStream_t stream);

hipError_t launch_small_m(const SmallMPlan &plan, const float *x, int64_t M, int64_t K,
                          const uint8_t *Wq, const float *scales, const uint8_t *zeros,
                          int64_t N, const float *bias, float *y, void *workspace,
                          hipStream_t stream);

hipError_t launch_prepack_kmajor(const uint8_t *Wq, const void *scales, bool f16,
                                 const uint8_t *zeros, int64_t K, int64_t N, uint8_t *Pq, void *Ps,
                                 uint8_t *Pz, hipStream_t stream);
hipError_t launch_gemv_kmajor(const KmajorPlan &plan, const float *x, int64_t M, int64_t K,
                              const uint8_t *Pq, const void *Ps, bool f16, const void *Pz,
                              int64_t N, const float *bias, const float *residual, int act,
                              float *y, hipStream_t stream, bool affine = false);
// Group-64 affine variant: quantize + pack, dequantize, K-major copy.
hipError_t launch_g64_quantize_pack(const float *W, int64_t K, int64_t N, uint8_t *Wq,
                                    float *scales, float *mins, int *d_status, hipStream_t stream);
hipError_t launch_g64_dequantize(const uint8_t *Wq, const float *scales, const float *mins,
                                 int64_t K, int64_t N, float *W_hat, hipStream_t stream);
hipError_t launch_prepack_g64(const uint8_t *Wq, const float *scales, const float *mins,
                              int64_t K, int64_t N, uint8_t *Pq, float *Ps, float *Pm,
                              hipStream_t stream);
// The fused epilogue alone (K = 0: the pre-activation values are the bias).
hipError_t launch_epilogue_only(const float *bias, int64_t M, int64_t N, const float *residual,
                                int act, float *y, hipStream_t stream);

hipError_t launch_bias_fill(const float *bias, int64_t M, int64_t N, float *y,
                            hipStream_t stream);

hipError_t launch_head_quantize(const float *E, int64_t K, int64_t N, int64_t ldq, int8_t *Q,
                                float *hs, int *d_status, hipStream_t stream);
hipError_t launch_head_logits(const HeadPlan &plan, const float *x, int64_t K, const int8_t *Q,
                              int64_t ldq, const float *hs, int64_t N, float *logits,
                              void *workspace, hipStream_t stream);
hipError_t launch_embed(const int64_t *tokens, int64_t T, const int8_t *Q, int64_t ldq,
                        const float *hs, int64_t K, int64_t N, float *out, int *d_status,
                        hipStream_t stream);
hipError_t launch_mm_x3(const X3Plan &p, const float *x, int64_t M, int64_t K, const uint8_t *Pq,
                        const void *Ps, bool f16, const uint8_t *Pz, int64_t N, const float *bias,
                        const float *residual, int act, float *y, void *workspace,
                        hipStream_t stream);
hipError_t launch_head_prepack(const int8_t *Q, int64_t K, int64_t N, int64_t ldq, int8_t *Qt,
                               int64_t ldt, hipStream_t stream);
hipError_t launch_head_logits_kmajor(const float *x, int64_t K, const int8_t *Qt, int64_t ldt,
                                     const float *hs, int64_t N, float *logits,
                                     hipStream_t stream);
size_t head_rows_workspace(int64_t M, int64_t K);
hipError_t launch_head_rows_kmajor(const float *x, int64_t M, int64_t K, const int8_t *Qt,
                                  int64_t ldt, const float *hs, int64_t N, float *logits,
                                  void *workspace, hipStream_t stream);
hipError_t launch_embed_kmajor(const int64_t *tokens, int64_t T, const int8_t *Qt, int64_t ldt,
                               const float *hs, int64_t K, int64_t N, float *out, int *d_status,
                               hipStream_t stream);

// Paged key-value cache (kv.h): append, attention of one new token in each
// sequence, eviction.  max_len is already the effective bound on lens.
struct KvPool;
hipError_t launch_kv_append(const KvPool &c, int dtype, const float *k, int64_t k_stride,
                            const float *v, int64_t v_stride, int64_t rows, const int32_t *table,
                            int64_t seqs, int64_t cols, const int32_t *seq, const int32_t *at,
                            int *d_status, hipStream_t stream);
size_t kv_attend_workspace(const KvPool &c, int64_t seqs, int64_t q_heads, int64_t max_len);
hipError_t launch_kv_attend(const KvPool &c, int dtype, const float *q, int64_t q_stride,
                            int64_t q_heads, const int32_t *table, int64_t seqs, int64_t cols,
                            const int32_t *lens, const int32_t *starts, int64_t max_len,
                            float scale, float *out, void *workspace, int *d_status,
                            hipStream_t stream);
hipError_t launch_kv_evict(const KvPool &c, int row_bytes, const int32_t *table, int64_t seqs,
                           int64_t cols, const int32_t *lens, int64_t max_len, int64_t keep,
                           int64_t recent, const int32_t *table_out, int64_t cols_out,
                           int32_t *kept, int32_t *lens_out, int *d_status, hipStream_t stream);

// Log probabilities of given tokens, entropy and the largest entries.
size_t logprobs_workspace(int64_t M, int64_t N, int64_t top);
hipError_t launch_logprobs(const float *logits, int64_t M, int64_t N, int64_t ld,
                           const int64_t *tokens, int64_t top, float *logprob, float *entropy,
                           int64_t *top_ids, float *top_logprob, void *workspace, int *d_status,
                           hipStream_t stream);

// Streaming-read reference: `loads` 16-byte loads per lane, 256 lanes per
// workgroup, one XOR word per wave into out[read_bytes_words(...)].
int64_t read_bytes_groups(int64_t bytes, int loads);
int64_t read_bytes_words(int64_t bytes, int loads);
hipError_t launch_read_bytes(const void *src, int64_t bytes, int loads, uint32_t *out,
                             hipStream_t stream);

}  // namespace w4
