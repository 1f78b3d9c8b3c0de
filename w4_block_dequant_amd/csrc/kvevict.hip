// Eviction from the paged cache by accumulated attention weight (see kv.h and
// include/w4.h).
//
// Two launches.  k_kv_select, one workgroup of 16 waves for each (sequence,
// head), finds the key of the last row that stays and writes the positions that
// stay in ascending order; k_kv_move copies those rows to their new pages, bound
// by the bytes it reads and writes.
//
// Selection.  A weight's key is its value in an order that unsigned integers
// have.  The keys are kept in registers (up to 32 in a lane; sequences past
// 32768 are read again) and narrowed down by histograms of 256 bins: first over the
// range from the smallest to the largest key, then over the bin in which the
// wanted count is reached, until that bin is wanted whole or is one key.  Of a
// few thousand keys with distinct weights that takes two or three histograms;
// equal ones at most four.  Rows that tie with the last one stay in order of
// position: wave w owns the w-th stretch of positions, so counts of the waves
// before it place its rows.
#include "kv.h"
#include "launch.h"

namespace w4 {
namespace {

constexpr int kSelWaves = 16;

__device__ __forceinline__ uint32_t evict_key(float w) {
    return __builtin_isnan(w) ? 0u : order_key(w);
}

// R: keys of a lane held in registers (0: read again each time).
template <int R>
__global__ __launch_bounds__(64 * kSelWaves) void k_kv_select(
    const int32_t *__restrict__ table, const int32_t *__restrict__ lens, int64_t cols, int most,
    int keep, int recent, KvPool c, int32_t *kept, int32_t *lens_out, int *d_status) {
    __shared__ uint32_t s_hist[256];
    __shared__ uint32_t s_low[kSelWaves], s_high[kSelWaves], s_pick[4];
    const int64_t b = blockIdx.x / c.heads;
    const int h = (int)(blockIdx.x % c.heads);
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int L = kv_length(lens, b, most, d_status);
    const int n = min(L, keep);
    int32_t *to = kept + (int64_t)blockIdx.x * keep;
    if (h == 0 && threadIdx.x == 0) lens_out[b] = n;
    for (int i = n + (int)threadIdx.x; i < keep; i += 64 * kSelWaves) to[i] = -1;
    if (L <= keep) {
        for (int i = threadIdx.x; i < n; i += 64 * kSelWaves) to[i] = i;
        return;
    }
    // of the first m positions `want` stay; the newest r all do
    const int r = min(recent, keep), want = keep - r, m = L - r;
    for (int i = threadIdx.x; i < r; i += 64 * kSelWaves) to[want + i] = m + i;
    if (want == 0) return;

    const int32_t *tab = table + b * cols;
    const int rounds = (m + 64 * kSelWaves - 1) / (64 * kSelWaves);  // at most R, if R > 0
    const int first = wave * rounds * 64 + lane;
    auto read = [&](int t) {
        const int page = tab[t >> c.shift];
        return kv_page_ok(c, page)
                   ? evict_key(c.weight[kv_row(c, page, h, t & ((1 << c.shift) - 1))])
                   : 0u;
    };
    uint32_t held[R ? R : 1];
    if constexpr (R > 0) {
#pragma unroll
        for (int i = 0; i < R; ++i)
            held[i] = i < rounds && first + 64 * i < m ? read(first + 64 * i) : 0u;
    }
    // f(key, position) for every position of the lane
    auto each = [&](auto f) {
        if constexpr (R > 0) {
#pragma unroll
            for (int i = 0; i < R; ++i) {
                if (i >= rounds) break;
                f(held[i], first + 64 * i, first + 64 * i < m);
            }
        } else {
            for (int i = 0; i < rounds; ++i) {
                const int t = first + 64 * i;
                f(t < m ? read(t) : 0u, t, t < m);
            }
        }
    };

    uint32_t low = 0xFFFFFFFFu, high = 0;
    each([&](uint32_t key, int, bool in) {
        low = in ? min(low, key) : low;
        high = in ? max(high, key) : high;
    });
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
        low = min(low, (uint32_t)__shfl_xor((int)low, o));
        high = max(high, (uint32_t)__shfl_xor((int)high, o));
    }
    if (lane == 0) s_low[wave] = low, s_high[wave] = high;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kSelWaves; ++w) low = min(low, s_low[w]), high = max(high, s_high[w]);

    // keys [low, low + span] hold the last row that stays; `left` of them stay
    uint32_t span = high - low, left = (uint32_t)want;
    int shift = max(0, 24 - __builtin_clz(span | 1u));
    uint32_t least, ties;  // rows above `least` stay, and the first `ties` rows equal to it
    for (;;) {
        if (threadIdx.x < 256) s_hist[threadIdx.x] = 0;
        __syncthreads();
        each([&](uint32_t key, int, bool in) {
            if (in && key >= low && key - low <= span) atomicAdd(&s_hist[(key - low) >> shift], 1u);
        });
        __syncthreads();
        if (wave == 0) {
            // lane: bins 255 - 4 lane .. 252 - 4 lane, counted from the top
            uint32_t n4[4], sum = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) n4[i] = s_hist[255 - 4 * lane - i], sum += n4[i];
            uint32_t upto = sum;
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) {
                const uint32_t v = (uint32_t)__shfl_up((int)upto, o);
                if (lane >= o) upto += v;
            }
            uint32_t above = upto - sum;
            if (above < left && upto >= left) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (above < left && above + n4[i] >= left) {
                        s_pick[0] = 255 - 4 * lane - i;
                        s_pick[1] = above;
                        s_pick[2] = n4[i];
                    }
                    above += n4[i];
                }
            }
        }
        __syncthreads();
        low += s_pick[0] << shift;
        left -= s_pick[1];
        if (s_pick[2] == left) {  // the bin stays whole
            least = low - 1;      // low > 0: the smallest key of all does not stay
            ties = 0;
            break;
        }
        if (shift == 0) {
            least = low;
            ties = left;
            break;
        }
        span = (1u << shift) - 1;
        shift = max(0, shift - 8);
    }

    uint32_t over = 0, same = 0;
    each([&](uint32_t key, int, bool in) {
        over += (uint32_t)__popcll(__ballot(in && key > least));
        same += (uint32_t)__popcll(__ballot(in && key == least));
    });
    __syncthreads();
    if (lane == 0) s_low[wave] = over, s_high[wave] = same;
    __syncthreads();
    uint32_t base = 0, tied = 0;  // rows of the waves before: above, and equal
    for (int w = 0; w < wave; ++w) base += s_low[w], tied += s_high[w];
    const uint64_t below = (1ull << lane) - 1;
    each([&](uint32_t key, int t, bool in) {
        const uint64_t up = __ballot(in && key > least), eq = __ballot(in && key == least);
        const uint32_t rank = tied + (uint32_t)__popcll(eq & below);  // among the equal ones
        const uint32_t place =
            base + (uint32_t)__popcll(up & below) + min(rank, ties);
        if (in && (key > least || (key == least && rank < ties))) to[place] = t;
        base += (uint32_t)__popcll(up);
        tied += (uint32_t)__popcll(eq);
    });
}

// A workgroup copies kMoveRows rows of one (sequence, head), keys and values, in
// pieces of 16 bytes (8 where a row is no multiple of 16), four pieces of a
// thread in flight.  A row's pages are looked up once.
constexpr int kMoveRows = 64;

template <class T>
__global__ __launch_bounds__(256) void k_kv_move(const int32_t *__restrict__ table,
                                                 const int32_t *__restrict__ table_out,
                                                 const int32_t *__restrict__ kept, int64_t cols,
                                                 int64_t cols_out, int keep, int pieces,
                                                 int tiles, KvPool c, int *d_status) {
    __shared__ int64_t s_from[kMoveRows], s_into[kMoveRows];
    const int64_t bh = blockIdx.x / tiles;
    const int i0 = (int)(blockIdx.x % tiles) * kMoveRows;
    const int64_t b = bh / c.heads;
    const int h = (int)(bh % c.heads), mask = (1 << c.shift) - 1;
    if (threadIdx.x < kMoveRows) {
        const int i = i0 + (int)threadIdx.x;
        const int t = i < keep ? kept[bh * keep + i] : -1;
        int64_t src = -1, dst = -1;
        if (t >= 0) {
            const int from = table[b * cols + (t >> c.shift)];
            const int into = table_out[b * cols_out + (i >> c.shift)];
            if (kv_page_ok(c, from) && kv_page_ok(c, into)) {
                src = kv_row(c, from, h, t & mask), dst = kv_row(c, into, h, i & mask);
                c.weight[dst] = c.weight[src];
                if (c.k_scale) {
                    c.k_scale[dst] = c.k_scale[src];
                    c.v_scale[dst] = c.v_scale[src];
                }
            } else {
                set_status(d_status, W4_ERR_BAD_SHAPE);
            }
        }
        s_from[threadIdx.x] = src;
        s_into[threadIdx.x] = dst;
    }
    __syncthreads();
    const T *kf = (const T *)c.k, *vf = (const T *)c.v;
    T *kt = (T *)c.k, *vt = (T *)c.v;
    const int all = kMoveRows * pieces;
    for (int x0 = threadIdx.x; x0 < all; x0 += 2 * 256) {
        T kv[2], vv[2];
        int64_t at[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int x = x0 + 256 * j;
            const int row = x < all ? x / pieces : 0, piece = x - row * pieces;
            const int64_t src = x < all ? s_from[row] : -1;
            at[j] = src < 0 ? -1 : s_into[row] * pieces + piece;
            if (at[j] >= 0) {
                kv[j] = __builtin_nontemporal_load(kf + src * pieces + piece);
                vv[j] = __builtin_nontemporal_load(vf + src * pieces + piece);
            }
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
            if (at[j] >= 0) {
                kt[at[j]] = kv[j];
                vt[at[j]] = vv[j];
            }
    }
}

}  // namespace

hipError_t launch_kv_evict(const KvPool &c, int row_bytes, const int32_t *table, int64_t seqs,
                           int64_t cols, const int32_t *lens, int64_t max_len, int64_t keep,
                           int64_t recent, const int32_t *table_out, int64_t cols_out,
                           int32_t *kept, int32_t *lens_out, int *d_status, hipStream_t stream) {
    const int64_t bh = seqs * c.heads;
    auto select = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3((unsigned)bh), dim3(64 * kSelWaves), 0, stream, table,
                           lens, cols, (int)max_len, (int)keep, (int)recent, c, kept, lens_out,
                           d_status);
        return hipGetLastError();
    };
    const int64_t rounds = (max_len + 64 * kSelWaves - 1) / (64 * kSelWaves);
    hipError_t e = rounds <= 4    ? select(k_kv_select<4>)
                   : rounds <= 16 ? select(k_kv_select<16>)
                   : rounds <= 32 ? select(k_kv_select<32>)
                                  : select(k_kv_select<0>);
    if (e != hipSuccess) return e;
    const int64_t rows = keep < max_len ? keep : max_len;
    const int64_t tiles = (rows + kMoveRows - 1) / kMoveRows;
    if (tiles == 0) return hipSuccess;
    if (tiles * bh > 0x7FFFFFFF) return hipErrorInvalidValue;
    auto move = [&](auto kernel, int piece) {
        hipLaunchKernelGGL(kernel, dim3((unsigned)(tiles * bh)), dim3(256), 0, stream, table,
                           table_out, kept, cols, cols_out, (int)keep, row_bytes / piece,
                           (int)tiles, c, d_status);
        return hipGetLastError();
    };
    return row_bytes % 16 == 0 ? move(k_kv_move<u32x4_t>, 16) : move(k_kv_move<u32x2_t>, 8);
}

}  // namespace w4
