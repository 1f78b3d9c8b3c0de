// Eviction from the paged cache by accumulated attention weight (see kv.h and
// include/w4.h).
//
// Two launches.  k_kv_select, one workgroup for each (sequence, head), finds
// the key of the last row that stays, bit by bit from the top (the largest
// threshold that at least the wanted number of rows reach), takes the lowest
// positions among the rows that tie with it, and writes the positions that
// stay in ascending order.  k_kv_move copies those rows to their new pages.
#include "kv.h"
#include "launch.h"

namespace w4 {
namespace {

__device__ __forceinline__ uint32_t evict_key(float w) {
    return __builtin_isnan(w) ? 0u : order_key(w);
}

__device__ __forceinline__ int block_sum(int v, int *s) {
    __syncthreads();
    s[threadIdx.x] = v;
    __syncthreads();
    for (int o = 128; o > 0; o >>= 1) {
        if (threadIdx.x < (unsigned)o) s[threadIdx.x] += s[threadIdx.x + o];
        __syncthreads();
    }
    return s[0];
}

__global__ __launch_bounds__(256) void k_kv_select(KvPool c, const int32_t *table, int64_t cols,
                                                   const int32_t *lens, int most, int keep,
                                                   int recent, int32_t *kept, int32_t *lens_out,
                                                   int *d_status) {
    __shared__ int s[256];
    const int64_t b = blockIdx.x / c.heads;
    const int h = (int)(blockIdx.x % c.heads);
    const int L = kv_length(lens, b, most, d_status);
    const int n = min(L, keep);
    int32_t *to = kept + ((int64_t)b * c.heads + h) * keep;
    if (h == 0 && threadIdx.x == 0) lens_out[b] = n;
    for (int i = n + (int)threadIdx.x; i < keep; i += 256) to[i] = -1;
    if (L <= keep) {
        for (int i = threadIdx.x; i < n; i += 256) to[i] = i;
        return;
    }
    const int r = min(recent, keep), want = keep - r, m = L - r;
    auto key = [&](int t) {
        const int page = table[b * cols + (t >> c.shift)];
        if (!kv_page_ok(c, page)) return 0u;
        return evict_key(c.weight[kv_row(c, page, h, t & ((1 << c.shift) - 1))]);
    };
    uint32_t least = 0;  // the largest threshold that `want` rows reach
    for (int bit = 31; bit >= 0; --bit) {
        const uint32_t trial = least | (1u << bit);
        int above = 0;
        for (int t = threadIdx.x; t < m; t += 256) above += key(t) >= trial;
        if (block_sum(above, s) >= want) least = trial;
    }
    int above = 0;
    for (int t = threadIdx.x; t < m; t += 256) above += key(t) > least;
    const int ties = want - block_sum(above, s);
    int base = 0, tied = 0;  // rows written and ties taken before this tile
    for (int t0 = 0; t0 < L; t0 += 256) {
        const int t = t0 + (int)threadIdx.x;
        const uint32_t u = t < m ? key(t) : 0;
        const bool tie = t < m && u == least;
        __syncthreads();
        s[threadIdx.x] = tie;
        __syncthreads();
        int before = 0, all = 0;
        for (int i = 0; i < 256; ++i) {
            before += i < (int)threadIdx.x ? s[i] : 0;
            all += s[i];
        }
        const bool stay = t < L && (t >= m || u > least || (tie && tied + before < ties));
        tied += all;
        __syncthreads();
        s[threadIdx.x] = stay;
        __syncthreads();
        before = all = 0;
        for (int i = 0; i < 256; ++i) {
            before += i < (int)threadIdx.x ? s[i] : 0;
            all += s[i];
        }
        if (stay) to[base + before] = t;
        base += all;
    }
}

// One wave copies one row of (sequence, head, new position) in 8-byte pieces.
__global__ __launch_bounds__(64) void k_kv_move(KvPool c, int row_bytes, const int32_t *table,
                                                int64_t cols, const int32_t *table_out,
                                                int64_t cols_out, int keep, const int32_t *kept,
                                                int *d_status) {
    const int64_t bh = blockIdx.y;
    const int64_t b = bh / c.heads;
    const int h = (int)(bh % c.heads), mask = (1 << c.shift) - 1;
    for (int i = blockIdx.x; i < keep; i += gridDim.x) {
        const int t = kept[bh * keep + i];
        if (t < 0) continue;
        const int from = table[b * cols + (t >> c.shift)];
        const int into = table_out[b * cols_out + (i >> c.shift)];
        if (!kv_page_ok(c, from) || !kv_page_ok(c, into)) {
            set_status(d_status, W4_ERR_BAD_SHAPE);
            continue;
        }
        const int64_t src = kv_row(c, from, h, t & mask), dst = kv_row(c, into, h, i & mask);
        for (int x = threadIdx.x * 8; x < row_bytes; x += 64 * 8) {
            *(u32x2_t *)((char *)c.k + dst * row_bytes + x) =
                *(const u32x2_t *)((const char *)c.k + src * row_bytes + x);
            *(u32x2_t *)((char *)c.v + dst * row_bytes + x) =
                *(const u32x2_t *)((const char *)c.v + src * row_bytes + x);
        }
        if (threadIdx.x == 0) {
            c.weight[dst] = c.weight[src];
            if (c.k_scale) {
                c.k_scale[dst] = c.k_scale[src];
                c.v_scale[dst] = c.v_scale[src];
            }
        }
    }
}

}  // namespace

hipError_t launch_kv_evict(const KvPool &c, int row_bytes, const int32_t *table, int64_t seqs,
                           int64_t cols, const int32_t *lens, int64_t max_len, int64_t keep,
                           int64_t recent, const int32_t *table_out, int64_t cols_out,
                           int32_t *kept, int32_t *lens_out, int *d_status, hipStream_t stream) {
    const unsigned bh = (unsigned)(seqs * c.heads);
    hipLaunchKernelGGL(k_kv_select, dim3(bh), dim3(256), 0, stream, c, table, cols, lens,
                       (int)max_len, (int)keep, (int)recent, kept, lens_out, d_status);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t rows = keep < max_len ? keep : max_len;
    if (rows == 0) return hipSuccess;
    hipLaunchKernelGGL(k_kv_move, dim3((unsigned)(rows < 4096 ? rows : 4096), bh), dim3(64), 0,
                       stream, c, row_bytes, table, cols, table_out, cols_out, (int)keep, kept,
                       d_status);
    return hipGetLastError();
}

}  // namespace w4
