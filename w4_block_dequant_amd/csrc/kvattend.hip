// Attention of one new token in each sequence over the paged cache (see kv.h
// and include/w4.h):
//   s[h, t] = scale q[h].k[t],  p = softmax over t,  out[h] = sum_t p[h, t] v[t],
// and the optional growth of each position's weight by its p summed over the
// query heads that share its key head.
//
// Bound: the cache's bytes, read once.  All G query heads of a key head are
// taken together, on the matrix cores, whatever G is: a key or value element
// costs a fixed few instructions, where the vector ALUs would spend one or
// more per query head on it (at 8 heads and 16-bit elements that alone passes
// the time of the reads).
//
// Work split.  One workgroup of 4 waves takes one (sequence, key head, block of
// up to 16 query heads, stretch of split_len positions); its waves take tiles
// of 32 positions in turn, each with a running maximum m and sum l for every
// head, and add up at the end in wave order.  Where the plan makes several
// stretches, each leaves (m, l, sum p v) in the workspace and a second kernel
// joins them in stretch order; so results are deterministic.  No LDS and no
// barrier in the loop over positions.
//
// Tile.  Lane (c, x) = (lane / 16, lane % 16).
//   Scores: the keys are the MFMA's A operand (row x = position t0 + 16 u + x,
//   dims 32 b + 8 c .. + 7 of block b, u = 0, 1), the queries its B operand
//   (column x = head x); the result leaves lane (c, x) with positions
//   t0 + 16 u + 4 c + i (i = 0..3) of head x.
//   Output: those eight p are, in place, the A operand (row x = head x) of the
//   product with the values if its k index 8 c + j stands for position
//   4 c + j (j < 4) or 16 + 4 c + j - 4: nothing moves between lanes.  The lane
//   reads the DL dims DL x .. of those eight positions' values, and the B
//   operand of dim e is the e-th element of each (a 16-bit transpose within the
//   lane, one v_perm for two elements); acc[e] leaves head 4 c + i, dim DL x + e.
//
// Operands are exact or as good as fp32, sums are fp32 (the matrix cores'):
//   bf16 cache: q and p are split exactly into three bf16 terms.
//   int8 cache: codes are exact in bf16; the scales multiply s and p in fp32.
//   fp16 cache: q (scaled by a power of two to [2^14, 2^15)) and p (in units of
//     2^-15) are split into two fp16 terms, h = fp16(a) and fp16(a - h): 2^-24
//     relative, 2^-40 of the row's largest absolute.
//   fp32 cache: v_mfma_f32_16x16x4_f32, one k step for each of a lane's 8 dims.
// Scores are in units of log2(e): p = exp2(s - m).  Positions outside the
// range get s = -infinity by selection and values of zero, whatever their
// slots hold; an address is never formed from a table entry that the range
// does not need or whose page the pool does not have.
#include <math.h>

#include "kv.h"
#include "launch.h"

namespace w4 {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));

typedef float f32x4u_t __attribute__((ext_vector_type(4), aligned(4)));

constexpr int kWaves = 4;

__device__ __forceinline__ uint32_t hi16_pair(uint32_t lo, uint32_t hi) {
    return __builtin_amdgcn_perm(hi, lo, 0x07060302u);
}
__device__ __forceinline__ uint32_t lo16_pair(uint32_t lo, uint32_t hi) {
    return __builtin_amdgcn_perm(hi, lo, 0x05040100u);
}
__device__ __forceinline__ uint32_t fbits(float v) { return __builtin_bit_cast(uint32_t, v); }
// What truncation to bf16 leaves (exact).
__device__ __forceinline__ float bf16_rest(float v) {
    return v - __builtin_bit_cast(float, fbits(v) & 0xFFFF0000u);
}
__device__ __forceinline__ uint32_t f16_pair(float a, float b) {
    return (uint32_t)f32_to_f16_bits(a) | (uint32_t)f32_to_f16_bits(b) << 16;
}
// Element i (0..3) of four signed codes, as fp32.
__device__ __forceinline__ float code_at(uint32_t w, int i) {
    return (float)(int)(int8_t)(w >> (8 * i));
}

// PARTS: terms that q and p are split into; operand words (of 8 elements).
template <int DT>
struct Parts {
    static constexpr int n = DT == KV_F16 ? 2 : 3;
};
template <>
struct Parts<KV_F32> {
    static constexpr int n = 1;
};

// Eight fp32 values as matrix operands: 4 words for each term (fp32: as they are).
template <int DT>
struct Split {
    static constexpr int words = DT == KV_F32 ? 8 : 4;
    uint32_t w[Parts<DT>::n][words];
    __device__ __forceinline__ void set(const float *f) {
        if constexpr (DT == KV_F32) {
#pragma unroll
            for (int i = 0; i < 8; ++i) w[0][i] = fbits(f[i]);
        } else if constexpr (DT == KV_F16) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float a = f[2 * i], b = f[2 * i + 1];
                const float ha = (float)(_Float16)a, hb = (float)(_Float16)b;
                w[0][i] = f16_pair(ha, hb);
                w[1][i] = f16_pair(a - ha, b - hb);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float a = f[2 * i], b = f[2 * i + 1];
                const float a1 = bf16_rest(a), b1 = bf16_rest(b);
                w[0][i] = hi16_pair(fbits(a), fbits(b));
                w[1][i] = hi16_pair(fbits(a1), fbits(b1));
                w[2][i] = hi16_pair(fbits(bf16_rest(a1)), fbits(bf16_rest(b1)));
            }
        }
    }
};

template <int DT>
__device__ __forceinline__ f32x4_t mfma8(const uint32_t *a, const uint32_t *b, f32x4_t c) {
    if constexpr (DT == KV_F32) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            c = __builtin_amdgcn_mfma_f32_16x16x4f32(__builtin_bit_cast(float, a[e]),
                                                     __builtin_bit_cast(float, b[e]), c, 0, 0, 0);
        return c;
    } else {
        const u32x4_t av = {a[0], a[1], a[2], a[3]}, bv = {b[0], b[1], b[2], b[3]};
        if constexpr (DT == KV_F16)
            return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, av),
                                                          __builtin_bit_cast(f16x8_t, bv), c, 0, 0,
                                                          0);
        else
            return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, av),
                                                           __builtin_bit_cast(bf16x8_t, bv), c, 0,
                                                           0, 0);
    }
}

template <int DT>
constexpr int kElem = DT == KV_F32 ? 4 : DT == KV_I8 ? 1 : 2;

// N consecutive elements from p (N * size bytes, aligned to their number of
// bytes or 16), as words.
template <int BYTES>
__device__ __forceinline__ void load_words(const char *p, uint32_t *w) {
    if constexpr (BYTES == 4) {
        w[0] = load_stream<uint32_t>(p);
    } else if constexpr (BYTES == 8) {
        const u32x2_t v = load_stream<u32x2_t>(p);
        w[0] = v.x;
        w[1] = v.y;
    } else {
#pragma unroll
        for (int i = 0; i < BYTES / 16; ++i) {
            const u32x4_t v = load_stream<u32x4_t>(p + 16 * i);
#pragma unroll
            for (int j = 0; j < 4; ++j) w[4 * i + j] = v[j];
        }
    }
}

// Where the two 16-position halves of a tile lie.
struct TilePages {
    int64_t row[2];  // pool row of the half's first position
    bool ok[2];
};

// NB: blocks of 32 dims of a query; DL: dims of the values that a lane owns.
template <int DT, int NB, int DL>
__global__ __launch_bounds__(64 * kWaves) void k_kv_attend(
    KvPool c, const float *__restrict__ q, const int32_t *__restrict__ table,
    const int32_t *__restrict__ lens, const int32_t *__restrict__ starts, float *out, float *stats,
    float *part, float *scores, int64_t q_stride, int64_t cols, int64_t score_stride,
    int64_t units, int q_heads, int splits, int split_len, int most, float scale, bool vecq,
    int *d_status) {
    constexpr int ES = kElem<DT>;
    constexpr int KW = 8 * ES / 4;           // words of a lane's 8 key dims
    constexpr int DC = DL < 8 ? DL : 8;      // dims of one chunk of a lane's values
    constexpr int NC = DL / DC;              // chunks
    constexpr int VW = DC * ES / 4;          // words of a chunk
    constexpr int P = Parts<DT>::n;
    __shared__ float s_m[kWaves][16], s_l[kWaves][16];
    __shared__ float s_acc[kWaves][16][NC * 16 * DC + 4];

    const int G = q_heads / c.heads;
    const int blocks = (G + 15) / 16;  // of query heads
    // unit = (sequence, key head, stretch); blocks of query heads that read the
    // same keys are 8 workgroups apart, on the same XCD
    const int per = 8 * blocks;
    const int64_t unit = (int64_t)(blockIdx.x / per) * 8 + blockIdx.x % 8;
    const int gb = (int)(blockIdx.x % per) / 8;
    const int split = (int)(unit % splits);
    const int64_t bh = unit / splits;
    const int64_t b = bh / c.heads;
    const int h = (int)(bh % c.heads);
    if (unit >= units) return;  // the last eight, padded
    const int g0 = gb * 16, gn = min(16, G - g0);
    const int hq0 = h * G + g0;

    const int lane = threadIdx.x & 63, x = lane & 15, cg = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = kv_length(lens, b, most, d_status);
    const int lo = starts ? max(starts[b], 0) : 0;
    const int first = max(split * split_len, lo & ~31);
    const int last = min((split + 1) * split_len, n);
    const int mask = (1 << c.shift) - 1;
    const int32_t *tab = table + b * cols;

    // queries: column x of the B operands, all blocks
    Split<DT> qs[NB];
    float sc = scale * 1.4426950408889634f;
    {
        float f[NB][8];
        const float *qp = q + b * q_stride + (int64_t)(hq0 + x) * c.dim;
#pragma unroll
        for (int k = 0; k < NB; ++k) {
            const int d0 = 32 * k + 8 * cg;
            const bool in = x < gn && d0 < c.dim;
            if (vecq) {
                const f32x4_t z = {0.0f, 0.0f, 0.0f, 0.0f};
                const f32x4_t v0 = in ? *(const f32x4_t *)(qp + d0) : z;
                const f32x4_t v1 = in ? *(const f32x4_t *)(qp + d0 + 4) : z;
#pragma unroll
                for (int e = 0; e < 4; ++e) f[k][e] = v0[e], f[k][4 + e] = v1[e];
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) f[k][e] = in ? qp[d0 + e] : 0.0f;
            }
        }
        if constexpr (DT == KV_F16) {
            float top = 0.0f;
#pragma unroll
            for (int k = 0; k < NB; ++k)
#pragma unroll
                for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(f[k][e]));
            top = fmaxf(top, __shfl_xor(top, 16));
            top = fmaxf(top, __shfl_xor(top, 32));
            // top in [2^(e-1), 2^e): to [2^14, 2^15); the shift undone in sc
            const int up = top > 0.0f ? min(15 - ilogbf(top) - 1, 100) : 0;
#pragma unroll
            for (int k = 0; k < NB; ++k)
#pragma unroll
                for (int e = 0; e < 8; ++e) f[k][e] = ldexpf(f[k][e], up);
            sc = ldexpf(sc, -up);
        }
#pragma unroll
        for (int k = 0; k < NB; ++k) qs[k].set(f[k]);
    }

    auto find = [&](int t0) {
        TilePages p;
        const int e0 = t0 >> c.shift, e1 = (t0 + 16) >> c.shift;
        const int p0 = tab[e0];
        const int p1 = e1 == e0 || t0 + 16 >= last ? p0 : tab[e1];
        p.ok[0] = kv_page_ok(c, p0);
        p.ok[1] = kv_page_ok(c, p1);
        if (!p.ok[0] || !p.ok[1]) set_status(d_status, W4_ERR_BAD_SHAPE);
        p.row[0] = kv_row(c, p.ok[0] ? p0 : 0, h, t0 & mask);
        p.row[1] = kv_row(c, p.ok[1] ? p1 : 0, h, (t0 + 16) & mask);
        return p;
    };

    const int row_bytes = c.dim * ES;
    // dims past head_dim read the row's start: their q is zero, their outputs
    // are not stored
    int koff[NB];
#pragma unroll
    for (int k = 0; k < NB; ++k)
        koff[k] = x * row_bytes + (32 * k + 8 * cg < c.dim ? (32 * k + 8 * cg) * ES : 0);
    int voff[NC];
#pragma unroll
    for (int k = 0; k < NC; ++k)
        voff[k] = 4 * cg * row_bytes + (x * DL + k * DC < c.dim ? (x * DL + k * DC) * ES : 0);

    uint32_t kw[2][NB][KW];
    uint32_t vw[8][NC][VW];
    f32x4_t ksc[2], vsc[2];
    auto load_keys = [&](const TilePages &p) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const char *base = (const char *)c.k + p.row[u] * row_bytes;
#pragma unroll
            for (int k = 0; k < NB; ++k) load_words<8 * ES>(base + koff[k], kw[u][k]);
            if constexpr (DT == KV_I8) {
                ksc[u] = *(const f32x4u_t *)(c.k_scale + p.row[u] + 4 * cg);
            }
        }
    };
    auto load_values = [&](const TilePages &p) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const char *base = (const char *)c.v + p.row[u] * row_bytes;
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int k = 0; k < NC; ++k)
                    load_words<DC * ES>(base + voff[k] + j * row_bytes, vw[4 * u + j][k]);
            if constexpr (DT == KV_I8) {
                vsc[u] = *(const f32x4u_t *)(c.v_scale + p.row[u] + 4 * cg);
            }
        }
    };

    float m = -INFINITY, l = 0.0f;
    f32x4_t acc[NC * DC];
    const f32x4_t zero4 = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int e = 0; e < NC * DC; ++e) acc[e] = zero4;

    int t0 = first + 32 * wave;
    if (t0 < last) {
        TilePages pg = find(t0);
        load_keys(pg);
        load_values(pg);
        for (; t0 < last; t0 += 32 * kWaves) {
            // the next tile's loads go out as soon as this tile has used its own
            // (past the end: this tile's again, so that nothing depends on a branch)
            const TilePages next = t0 + 32 * kWaves < last ? find(t0 + 32 * kWaves) : pg;
            f32x4_t s[2] = {zero4, zero4};
#pragma unroll
            for (int k = 0; k < NB; ++k)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    uint32_t a[8];
                    if constexpr (DT == KV_I8) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            a[i] = hi16_pair(fbits(code_at(kw[u][k][i / 2], 2 * (i & 1))),
                                             fbits(code_at(kw[u][k][i / 2], 2 * (i & 1) + 1)));
                    } else {
#pragma unroll
                        for (int i = 0; i < KW; ++i) a[i] = kw[u][k][i];
                    }
#pragma unroll
                    for (int r = P - 1; r >= 0; --r) s[u] = mfma8<DT>(a, qs[k].w[r], s[u]);
                }
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    s[u][i] *= sc;
                    if constexpr (DT == KV_I8) s[u][i] *= ksc[u][i];
                }
            load_keys(next);
            const bool whole = t0 >= lo && t0 + 32 <= last && pg.ok[0] && pg.ok[1];
            bool in[2][4];
            if (!whole) {
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int t = t0 + 16 * u + 4 * cg + i;
                        in[u][i] = t >= lo && t < last && pg.ok[u];
                        if (!in[u][i]) s[u][i] = -INFINITY;
                    }
            }
            if (scores && x < gn) {
                float *to = scores + (b * q_heads + hq0 + x) * score_stride + t0 + 4 * cg;
                *(f32x4_t *)to = s[0];
                *(f32x4_t *)(to + 16) = s[1];
            }
            float top = s[0][0];
#pragma unroll
            for (int i = 1; i < 8; ++i) top = fmaxf(top, s[i / 4][i % 4]);
            if (__any(top > m)) {
                top = fmaxf(top, __shfl_xor(top, 16));
                top = fmaxf(top, __shfl_xor(top, 32));
                top = fmaxf(top, m);
                const float fade = top == -INFINITY ? 1.0f : exp2f(m - top);
                m = top;
                l *= fade;
                f32x4_t fr;
#pragma unroll
                for (int i = 0; i < 4; ++i) fr[i] = __shfl(fade, 4 * cg + i);
#pragma unroll
                for (int e = 0; e < NC * DC; ++e)
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[e][i] *= fr[i];
            }
            // nothing seen yet: every s is -infinity, and p is 0
            const float ref = (m == -INFINITY ? 0.0f : m) - (DT == KV_F16 ? 15.0f : 0.0f);
            float p[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                p[i] = exp2f(s[i / 4][i % 4] - ref);
                l += p[i];
            }
            if constexpr (DT == KV_I8) {
#pragma unroll
                for (int i = 0; i < 8; ++i) p[i] *= vsc[i / 4][i % 4];
                if (!whole) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (!in[i / 4][i % 4]) p[i] = 0.0f;
                }
            } else if (!whole) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
#pragma unroll
                    for (int k = 0; k < NC; ++k)
#pragma unroll
                        for (int i = 0; i < VW; ++i)
                            if (!in[j / 4][j % 4]) vw[j][k][i] = 0;
            }
            Split<DT> ps;
            ps.set(p);
#pragma unroll
            for (int k = 0; k < NC; ++k)
#pragma unroll
                for (int e = 0; e < DC; ++e) {
                    uint32_t v[8];
                    if constexpr (DT == KV_F32) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) v[j] = vw[j][k][e];
                    } else if constexpr (DT == KV_I8) {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            v[j] = hi16_pair(fbits(code_at(vw[2 * j][k][e / 4], e % 4)),
                                             fbits(code_at(vw[2 * j + 1][k][e / 4], e % 4)));
                    } else {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            v[j] = e % 2 ? hi16_pair(vw[2 * j][k][e / 2], vw[2 * j + 1][k][e / 2])
                                         : lo16_pair(vw[2 * j][k][e / 2], vw[2 * j + 1][k][e / 2]);
                    }
#pragma unroll
                    for (int r = P - 1; r >= 0; --r)
                        acc[k * DC + e] = mfma8<DT>(ps.w[r], v, acc[k * DC + e]);
                }
            load_values(next);
            pg = next;
        }
    }

    // the four waves' parts, added in wave order
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);
    if (cg == 0) s_m[wave][x] = m, s_l[wave][x] = l;
#pragma unroll
    for (int e = 0; e < NC * DC; ++e)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            s_acc[wave][4 * cg + i][DL * x + e] = acc[e][i];
    __syncthreads();
    const int64_t rows = (b * q_heads + hq0) * splits + split;  // + g * splits
    for (int i = threadIdx.x; i < gn * c.dim; i += 64 * kWaves) {
        const int g = i / c.dim, d = i % c.dim;
        float M = s_m[0][g];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) M = fmaxf(M, s_m[w][g]);
        float L = 0.0f, o = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            const float f = s_m[w][g] == -INFINITY ? 0.0f : exp2f(s_m[w][g] - M);
            L += f * s_l[w][g];
            o += f * s_acc[w][g][d];
        }
        if (part)
            part[(rows + (int64_t)g * splits) * c.dim + d] = o;
        else
            out[(b * q_heads + hq0 + g) * c.dim + d] = L == 0.0f ? 0.0f : o / L;
        if (stats && d == 0) {
            stats[2 * (rows + (int64_t)g * splits)] = M;
            stats[2 * (rows + (int64_t)g * splits) + 1] = L;
        }
    }
}

// Maximum and sum of one head over its stretches (sum 0: the stretch held nothing).
__device__ __forceinline__ void joined(const float *stats, int splits, float &M, float &L) {
    M = -INFINITY;
    for (int s = 0; s < splits; ++s) M = fmaxf(M, stats[2 * s]);
    L = 0.0f;
    for (int s = 0; s < splits; ++s)
        if (stats[2 * s + 1] != 0.0f) L += exp2f(stats[2 * s] - M) * stats[2 * s + 1];
}

constexpr int kWeighTile = 1024;

// Workgroups below `joins` join the stretches of one (sequence, query head);
// the others grow the weights of kWeighTile positions of one (sequence, key
// head) from the scores that the first kernel left.
__global__ __launch_bounds__(256) void k_kv_join(KvPool c, const int32_t *table,
                                                 const int32_t *lens, const int32_t *starts,
                                                 float *out, const float *stats,
                                                 const float *part, const float *scores,
                                                 int64_t cols, int64_t score_stride, int64_t joins,
                                                 int64_t tiles, int q_heads, int splits, int most,
                                                 float unit) {
    __shared__ float s_m[256], s_l[256];
    if ((int64_t)blockIdx.x < joins) {
        const int64_t row = blockIdx.x;
        float M, L;
        joined(stats + 2 * row * splits, splits, M, L);
        for (int d = threadIdx.x; d < c.dim; d += 256) {
            float o = 0.0f;
            for (int s = 0; s < splits; ++s) {
                const float *st = stats + 2 * (row * splits + s);
                if (st[1] != 0.0f)
                    o += exp2f(st[0] - M) * part[(row * splits + s) * c.dim + d];
            }
            out[row * c.dim + d] = L == 0.0f ? 0.0f : o / L;
        }
        return;
    }
    const int64_t w = blockIdx.x - joins;
    const int64_t bh = w / tiles, b = bh / c.heads;
    const int h = (int)(bh % c.heads), G = q_heads / c.heads;
    const int n = kv_length(lens, b, most, nullptr);
    const int lo = max((int)(w % tiles) * kWeighTile, starts ? max(starts[b], 0) : 0);
    const int hi = min((int)(w % tiles + 1) * kWeighTile, n);
    if (lo >= hi) return;
    float p[kWeighTile / 256] = {};
    for (int g0 = 0; g0 < G; g0 += 256) {
        const int gn = min(256, G - g0);
        __syncthreads();
        if ((int)threadIdx.x < gn) {
            const int64_t row = b * q_heads + h * G + g0 + threadIdx.x;
            joined(stats + 2 * row * splits, splits, s_m[threadIdx.x], s_l[threadIdx.x]);
        }
        __syncthreads();
        for (int g = 0; g < gn; ++g) {
            const float M = s_m[g], L = s_l[g];
            const float *from = scores + (b * q_heads + h * G + g0 + g) * score_stride;
#pragma unroll
            for (int i = 0; i < kWeighTile / 256; ++i) {
                const int t = lo + (int)threadIdx.x + 256 * i;
                if (t < hi && L != 0.0f) p[i] += exp2f(from[t] - M) * unit / L;
            }
        }
    }
    const int32_t *tab = table + b * cols;
#pragma unroll
    for (int i = 0; i < kWeighTile / 256; ++i) {
        const int t = lo + (int)threadIdx.x + 256 * i;
        if (t >= hi) continue;
        const int page = tab[t >> c.shift];
        if (kv_page_ok(c, page)) c.weight[kv_row(c, page, h, t & ((1 << c.shift) - 1))] += p[i];
    }
}

}  // namespace

size_t kv_attend_workspace(const KvPool &c, int64_t seqs, int64_t q_heads, int64_t max_len) {
    return plan_kv_attend(seqs, q_heads, c.heads, c.dim, max_len, c.weight != nullptr).workspace;
}

hipError_t launch_kv_attend(const KvPool &c, int dtype, const float *q, int64_t q_stride,
                            int64_t q_heads, const int32_t *table, int64_t seqs, int64_t cols,
                            const int32_t *lens, const int32_t *starts, int64_t max_len,
                            float scale, float *out, void *workspace, int *d_status,
                            hipStream_t stream) {
    const bool weigh = c.weight != nullptr;
    const KvAttendPlan p = plan_kv_attend(seqs, q_heads, c.heads, c.dim, max_len, weigh);
    const int64_t units = seqs * c.heads * p.splits;
    const int64_t groups = (units + 7) / 8 * 8 * ((q_heads / c.heads + 15) / 16);
    const int64_t joins = p.splits > 1 ? seqs * q_heads : 0;
    const int64_t tiles = weigh ? (max_len + kWeighTile - 1) / kWeighTile : 0;
    const int64_t second = joins + tiles * seqs * c.heads;
    if (groups > 0x7FFFFFFF || second > 0x7FFFFFFF) return hipErrorInvalidValue;
    char *ws = (char *)workspace;
    float *stats = second > 0 ? (float *)(ws + p.stats) : nullptr;
    float *part = p.splits > 1 ? (float *)(ws + p.part) : nullptr;
    float *scores = weigh ? (float *)(ws + p.scores) : nullptr;
    const bool vecq = q_stride % 4 == 0 && (uintptr_t)q % 16 == 0;
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3((unsigned)groups), dim3(64 * kWaves), 0, stream, c, q,
                           table, lens, starts, out, stats, part, scores, q_stride, cols,
                           p.score_stride, units, (int)q_heads, (int)p.splits, (int)p.split_len,
                           (int)max_len, scale, vecq, d_status);
        return hipGetLastError();
    };
#define KV_BY_DIM(DT)                                          \
    (c.dim <= 64    ? go(k_kv_attend<DT, 2, 4>)                \
     : c.dim <= 96  ? go(k_kv_attend<DT, 3, 8>)                \
     : c.dim <= 128 ? go(k_kv_attend<DT, 4, 8>)                \
                    : go(k_kv_attend<DT, 8, 16>))
    hipError_t e = dtype == KV_F32    ? KV_BY_DIM(KV_F32)
                   : dtype == KV_F16  ? KV_BY_DIM(KV_F16)
                   : dtype == KV_BF16 ? KV_BY_DIM(KV_BF16)
                                      : KV_BY_DIM(KV_I8);
#undef KV_BY_DIM
    if (e != hipSuccess || second == 0) return e;
    hipLaunchKernelGGL(k_kv_join, dim3((unsigned)second), dim3(256), 0, stream, c, table, lens,
                       starts, out, stats, part, scores, cols, p.score_stride, joins, tiles,
                       (int)q_heads, (int)p.splits, (int)max_len,
                       dtype == KV_F16 ? 32768.0f : 1.0f);
    return hipGetLastError();
}

}  // namespace w4
