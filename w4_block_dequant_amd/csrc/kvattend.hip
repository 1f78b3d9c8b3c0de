// Attention of one new token in each sequence over the paged cache (see kv.h
// and include/w4.h): s = scale q.k, p = softmax(s), out = sum p v, and the
// optional growth of each position's weight by its p summed over the query
// heads that share its key head.
//
// One workgroup takes one (sequence, query head) and passes over its positions
// in tiles of 256 with a running maximum and sum: a lane forms one score, then
// the lanes take head_dim columns of the values.  A second kernel forms the
// weights once the maxima and sums are final.
#include <math.h>

#include "kv.h"
#include "launch.h"

namespace w4 {
namespace {

template <int DT>
__device__ __forceinline__ float kv_score(const KvPool &c, const float *q, int64_t row) {
    const auto *k = (const typename KvType<DT>::T *)c.k + row * c.dim;
    float s = 0.0f;
    for (int d = 0; d < c.dim; ++d) s = fmaf(q[d], KvType<DT>::get(k[d]), s);
    return DT == KV_I8 ? s * c.k_scale[row] : s;
}

__device__ __forceinline__ int64_t kv_find(const KvPool &c, const int32_t *table, int h, int t,
                                           int *d_status) {
    const int page = table[t >> c.shift];
    if (!kv_page_ok(c, page)) {
        set_status(d_status, W4_ERR_BAD_SHAPE);
        return -1;
    }
    return kv_row(c, page, h, t & ((1 << c.shift) - 1));
}

template <int DT>
__global__ __launch_bounds__(256) void k_kv_attend(KvPool c, const float *q, int64_t q_stride,
                                                   int q_heads, const int32_t *table,
                                                   int64_t cols, const int32_t *lens,
                                                   const int32_t *starts, int most, float scale,
                                                   float *out, float *stats, int *d_status) {
    __shared__ float sq[256], sp[256], red[256];
    __shared__ int64_t srow[256];
    const int64_t b = blockIdx.x / q_heads;
    const int hq = (int)(blockIdx.x % q_heads), h = hq / (q_heads / c.heads);
    const int n = kv_length(lens, b, most, d_status);
    const int lo = starts ? max(starts[b], 0) : 0;
    const int x = threadIdx.x;
    if (x < c.dim) sq[x] = q[b * q_stride + (int64_t)hq * c.dim + x];
    __syncthreads();
    float m = -INFINITY, l = 0.0f, acc = 0.0f;
    for (int t0 = lo; t0 < n; t0 += 256) {
        const int t = t0 + x;
        const int64_t row = t < n ? kv_find(c, table + b * cols, h, t, d_status) : -1;
        const float s = row >= 0 ? scale * kv_score<DT>(c, sq, row) : -INFINITY;
        red[x] = s;
        __syncthreads();
        for (int o = 128; o > 0; o >>= 1) {
            if (x < o) red[x] = fmaxf(red[x], red[x + o]);
            __syncthreads();
        }
        const float top = fmaxf(m, red[0]);
        __syncthreads();
        const float p = row >= 0 ? expf(s - top) : 0.0f;
        sp[x] = DT == KV_I8 && row >= 0 ? p * c.v_scale[row] : p;
        srow[x] = row;
        red[x] = p;
        __syncthreads();
        for (int o = 128; o > 0; o >>= 1) {
            if (x < o) red[x] += red[x + o];
            __syncthreads();
        }
        const float fade = top == -INFINITY ? 1.0f : expf(m - top);
        l = l * fade + red[0];
        acc *= fade;
        m = top;
        if (x < c.dim)
            for (int i = 0; i < 256; ++i)
                if (srow[i] >= 0)
                    acc = fmaf(sp[i],
                               KvType<DT>::get(((const typename KvType<DT>::T *)
                                                    c.v)[srow[i] * c.dim + x]),
                               acc);
        __syncthreads();
    }
    if (x < c.dim)
        out[(b * q_heads + hq) * c.dim + x] = m == -INFINITY ? 0.0f : acc / l;
    if (stats && x == 0) {
        stats[2 * (b * q_heads + hq)] = m;
        stats[2 * (b * q_heads + hq) + 1] = l;
    }
}

template <int DT>
__global__ __launch_bounds__(256) void k_kv_weigh(KvPool c, const float *q, int64_t q_stride,
                                                  int q_heads, const int32_t *table, int64_t cols,
                                                  const int32_t *lens, const int32_t *starts,
                                                  int most, float scale, const float *stats) {
    const int64_t b = blockIdx.x / c.heads;
    const int h = (int)(blockIdx.x % c.heads), G = q_heads / c.heads;
    const int n = kv_length(lens, b, most, nullptr);
    const int lo = starts ? max(starts[b], 0) : 0;
    for (int t = lo + (int)threadIdx.x; t < n; t += 256) {
        const int64_t row = kv_find(c, table + b * cols, h, t, nullptr);
        if (row < 0) continue;
        float p = 0.0f;
        for (int g = 0; g < G; ++g) {
            const int64_t hq = b * q_heads + h * G + g;
            const float s =
                scale * kv_score<DT>(c, q + b * q_stride + (int64_t)(h * G + g) * c.dim, row);
            p += expf(s - stats[2 * hq]) / stats[2 * hq + 1];
        }
        c.weight[row] += p;
    }
}

}  // namespace

size_t kv_attend_workspace(const KvPool &c, int64_t seqs, int64_t q_heads, int64_t max_len) {
    (void)max_len;
    return c.weight ? align_up((size_t)(seqs * q_heads) * 8, 256) : 0;
}

hipError_t launch_kv_attend(const KvPool &c, int dtype, const float *q, int64_t q_stride,
                            int64_t q_heads, const int32_t *table, int64_t seqs, int64_t cols,
                            const int32_t *lens, const int32_t *starts, int64_t max_len,
                            float scale, float *out, void *workspace, int *d_status,
                            hipStream_t stream) {
    auto go = [&](auto attend, auto weigh) {
        float *stats = c.weight ? (float *)workspace : nullptr;
        hipLaunchKernelGGL(attend, dim3((unsigned)(seqs * q_heads)), dim3(256), 0, stream, c, q,
                           q_stride, (int)q_heads, table, cols, lens, starts, (int)max_len, scale,
                           out, stats, d_status);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess || !stats) return e;
        hipLaunchKernelGGL(weigh, dim3((unsigned)(seqs * c.heads)), dim3(256), 0, stream, c, q,
                           q_stride, (int)q_heads, table, cols, lens, starts, (int)max_len, scale,
                           stats);
        return hipGetLastError();
    };
    switch (dtype) {
    case KV_F32: return go(k_kv_attend<KV_F32>, k_kv_weigh<KV_F32>);
    case KV_F16: return go(k_kv_attend<KV_F16>, k_kv_weigh<KV_F16>);
    case KV_BF16: return go(k_kv_attend<KV_BF16>, k_kv_weigh<KV_BF16>);
    default: return go(k_kv_attend<KV_I8>, k_kv_weigh<KV_I8>);
    }
}

}  // namespace w4
