// Append of new keys and values to the paged cache, with the conversion to the
// cache's type (see kv.h and include/w4.h).
//
// One workgroup takes one (row, head): its two rows of head_dim fp32 values
// are read once and stored converted.  KV_I8 needs the row's largest magnitude
// before the first code.
#include "kv.h"
#include "launch.h"

namespace w4 {
namespace {

template <int DT>
__global__ __launch_bounds__(64) void k_kv_append(KvPool c, const float *k, int64_t k_stride,
                                                  const float *v, int64_t v_stride,
                                                  const int32_t *table, int64_t seqs,
                                                  int64_t cols, const int32_t *seq,
                                                  const int32_t *at, int *d_status) {
    const int64_t r = blockIdx.x / c.heads;
    const int h = (int)(blockIdx.x % c.heads);
    const int lane = threadIdx.x;
    const int s = seq[r], t = at[r];
    if (s < 0) return;
    if (s >= seqs || t < 0 || (t >> c.shift) >= cols) {
        set_status(d_status, W4_ERR_BAD_SHAPE);
        return;
    }
    const int page = table[s * cols + (t >> c.shift)];
    if (!kv_page_ok(c, page)) {
        set_status(d_status, W4_ERR_BAD_SHAPE);
        return;
    }
    const int64_t row = kv_row(c, page, h, t & ((1 << c.shift) - 1));
    if (c.weight && lane == 0) c.weight[row] = 0.0f;
    for (int w = 0; w < 2; ++w) {
        const float *x = (w ? v + r * v_stride : k + r * k_stride) + (int64_t)h * c.dim;
        void *pool = w ? c.v : c.k;
        if constexpr (DT == KV_I8) {
            float m = 0.0f;
            bool bad = false;
            for (int d = lane; d < c.dim; d += 64) {
                m = fmaxf(m, fabsf(x[d]));
                bad |= !isfinite(x[d]);
            }
            for (int o = 32; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
            if (bad) set_status(d_status, W4_ERR_NONFINITE);
            const float scale = m / 127.0f;
            for (int d = lane; d < c.dim; d += 64) {
                const float q = scale == 0.0f ? 0.0f : rintf(x[d] / scale);
                ((int8_t *)pool)[row * c.dim + d] = (int8_t)fminf(fmaxf(q, -127.0f), 127.0f);
            }
            if (lane == 0) (w ? c.v_scale : c.k_scale)[row] = scale;
        } else {
            for (int d = lane; d < c.dim; d += 64)
                ((typename KvType<DT>::T *)pool)[row * c.dim + d] = KvType<DT>::put(x[d]);
        }
    }
}

}  // namespace

hipError_t launch_kv_append(const KvPool &c, int dtype, const float *k, int64_t k_stride,
                            const float *v, int64_t v_stride, int64_t rows, const int32_t *table,
                            int64_t seqs, int64_t cols, const int32_t *seq, const int32_t *at,
                            int *d_status, hipStream_t stream) {
    const dim3 grid((unsigned)(rows * c.heads));
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, grid, dim3(64), 0, stream, c, k, k_stride, v, v_stride, table,
                           seqs, cols, seq, at, d_status);
        return hipGetLastError();
    };
    switch (dtype) {
    case KV_F32: return go(k_kv_append<KV_F32>);
    case KV_F16: return go(k_kv_append<KV_F16>);
    case KV_BF16: return go(k_kv_append<KV_BF16>);
    default: return go(k_kv_append<KV_I8>);
    }
}

}  // namespace w4
