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
// Work split.  The work is one list: for every sequence, for every row block
// (a key head and up to 16 of its query heads), kOpen units for the block's start
// and end and then one for each step of 128 positions.  Each of the W workgroups
// takes the same number of consecutive units, whatever the lengths are (the
// host does not know them; a split by a bound on the length left half of the
// workgroups idle on a ragged batch and paid 4 us for each start of a
// workgroup).  The four waves of a workgroup take the 32-position tiles of a
// step in turn, each with a running maximum m and sum l for every head, and add
// up at a block's end in wave order.  A block that one workgroup has whole goes
// straight to the output; the parts of one that crosses workgroups (at most two
// for each workgroup) go to the workspace as (m, l, sum p v), and a second
// kernel joins them in order.  So results are deterministic.  No LDS and no
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
// 2^v; below 2^-126 it is 0, which no sum of p notices.
__device__ __forceinline__ float pow2(float v) { return __builtin_amdgcn_exp2f(v); }
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

// Where the two 16-position halves of a tile lie.  No padding: the compiler
// copies padding through memory, puts that into LDS, and then reads the
// workgroup's size from the dispatch packet in host memory, 15 us for a grid
// of 2000 waves.
struct TilePages {
    int64_t row0, row1;  // pool row of the half's first position
    int ok0, ok1;
};

// Sums over a wave in six additions: every lane's sum of itself and the lanes
// below, and the whole wave's.
template <int CTRL, int ROWS>
__device__ __forceinline__ int scan_step(int v) {
    return v + __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xF, false);
}
__device__ __forceinline__ int wave_scan(int v) {
    v = scan_step<0x111, 0xF>(v);  // from 1, 2, 4, 8 lanes below, within 16
    v = scan_step<0x112, 0xF>(v);
    v = scan_step<0x114, 0xF>(v);
    v = scan_step<0x118, 0xF>(v);
    v = scan_step<0x142, 0xA>(v);  // lanes 15 and 47 to the 16 above
    return scan_step<0x143, 0xC>(v);  // lane 31 to the upper half
}
__device__ __forceinline__ int wave_sum(int v) {
    return __builtin_amdgcn_readlane(wave_scan(v), 63);
}

// Steps of one sequence: 128 positions each, from the tile that holds lo on.
constexpr int kStep = 128;
__device__ __forceinline__ int kv_steps(int lo, int n) {
    return n > lo ? (n - (lo & ~31) + kStep - 1) / kStep : 0;
}
// Units that a block counts beside its steps, before them: what its start and
// end cost a workgroup.
constexpr int kOpen = kKvOpenUnits;
constexpr int kPart = kKvPartSteps;  // the least steps of a part
__device__ __forceinline__ int kv_units(int steps, int part) {
    return part ? max(1, (steps + part - 1) / part) : steps + kOpen;
}

// What the first kernel leaves for the second, in the workspace.
struct KvParts {
    float2 *stat;    // [2 W, 16] (m, l) of a workgroup's two unfinished blocks
    float *sum;      // [2 W, 16, head_dim] their sum p v
    int2 *owner;     // [seqs * row blocks] first and last workgroup of the block
    float2 *whole;   // [seqs * q_heads] (m, l) of blocks that one workgroup had
    float *scores;   // [seqs * q_heads, score_stride], in units of log2(e)
    int64_t score_stride;
};

// NB: blocks of 32 dims of a query; DL: dims of the values that a lane owns.
template <int DT, int NB, int DL>
__global__ __launch_bounds__(64 * kWaves) void k_kv_attend(
    const float *__restrict__ q, const int32_t *__restrict__ table,
    const int32_t *__restrict__ lens, const int32_t *__restrict__ starts, int seqs, int q_heads,
    int most, float scale, int64_t q_stride, int64_t cols, KvPool c, float *out, KvParts parts,
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
    const int gblocks = (G + 15) / 16;
    const int blocks = c.heads * gblocks;  // row blocks of a sequence
    const int lane = threadIdx.x & 63, x = lane & 15, cg = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int mask = (1 << c.shift) - 1;
    auto first_of = [&](int b) { return starts ? max(starts[b], 0) : 0; };

    // This workgroup's units [u0, u1) of the list, and the sequence b that holds
    // u0 (`base`: its first unit).  Where every block can be cut into parts of at
    // most `part` steps with one part to a workgroup, and that is no longer than
    // an even share and the crossing it saves, the units are those parts.
    int b = 0, u0, u1, base = 0, part = 0;
    uint32_t total, groups;  // units; workgroups that have any
    {
        auto steps_of = [&](int i) {
            return i < seqs ? kv_steps(first_of(i), min(max(lens[i], 0), most)) : 0;
        };
        const int mine = steps_of(lane);
        int sum = mine;
        for (int i = lane + 64; i < seqs; i += 64) sum += steps_of(i);
        const uint32_t steps = (uint32_t)wave_sum(sum) * blocks;
        total = steps + (uint32_t)seqs * blocks * kOpen;
        if ((uint32_t)seqs * blocks <= gridDim.x) {
            const uint32_t even = steps / gridDim.x;
            for (uint32_t s = max(even, (uint32_t)kPart); s <= max(even, (uint32_t)kPart) + 2; ++s) {
                int count = lane < seqs ? max(1, (mine + (int)s - 1) / (int)s) : 0;
                for (int i = lane + 64; i < seqs; i += 64)
                    count += max(1, (steps_of(i) + (int)s - 1) / (int)s);
                const uint32_t all = (uint32_t)wave_sum(count) * blocks;
                if (all <= gridDim.x) {
                    part = (int)s;
                    total = all;
                    break;
                }
            }
        }
        groups = min(gridDim.x, total);
        if (blockIdx.x >= groups) return;
        const uint32_t each = total / groups, rest = total % groups;
        u0 = (int)(blockIdx.x * each + blockIdx.x * rest / groups);
        u1 = (int)((blockIdx.x + 1) * each + (blockIdx.x + 1) * rest / groups);
        for (int i0 = 0;; i0 += 64) {
            const int st = i0 == 0 ? mine : steps_of(i0 + lane);
            const int have = i0 + lane < seqs ? kv_units(st, part) * blocks : 0;
            const int upto = wave_scan(have);
            const uint64_t past = __ballot(base + upto > u0);
            if (past) {
                const int at = __builtin_ctzll(past);
                b = i0 + at;
                base += __builtin_amdgcn_readlane(upto - have, at);
                break;
            }
            base += __builtin_amdgcn_readlane(upto, 63);
        }
    }

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

    int n = kv_length(lens, b, most, d_status), lo = first_of(b), steps = kv_steps(lo, n);
    for (int u = u0; u < u1;) {
    // block vb of sequence b, its steps [from, to)
    const int units = kv_units(steps, part);
    const int vb = (u - base) / units, start = base + vb * units;
    const int stop = min(u1, start + units);
    const int even = part ? (steps + units - 1) / units : 0;
    const int from = part ? (u - start) * even : max(u - start - kOpen, 0);
    const int to = part ? min((u - start + 1) * even, steps) : stop - start - kOpen;
    const int h = vb / gblocks, g0 = vb % gblocks * 16, gn = min(16, G - g0);
    const int hq0 = h * G + g0;
    const int first = (lo & ~31) + from * kStep, last = min((lo & ~31) + to * kStep, n);
    const int32_t *tab = table + (int64_t)b * cols;
    const bool whole_block = from == 0 && to == steps;
    if (parts.owner && u == start && threadIdx.x == 0) {
        // the workgroup of unit v is ((v + 1) groups - 1) / total
        const int lead = part ? 0 : kOpen;
        const int at = (int)(((uint64_t)(start + lead + 1) * groups - 1) / total);
        const int end = (int)(((uint64_t)(start + units) * groups - 1) / total);
        parts.owner[(int64_t)b * blocks + vb] = steps ? make_int2(at, end) : make_int2(0, 0);
    }
    if (to > from) {

    auto find = [&](int t0) {
        TilePages p;
        const int e0 = t0 >> c.shift, e1 = (t0 + 16) >> c.shift;
        const int p0 = tab[e0];
        const int p1 = e1 == e0 || t0 + 16 >= last ? p0 : tab[e1];
        p.ok0 = kv_page_ok(c, p0);
        p.ok1 = kv_page_ok(c, p1);
        if (!p.ok0 || !p.ok1) set_status(d_status, W4_ERR_BAD_SHAPE);
        p.row0 = kv_row(c, p.ok0 ? p0 : 0, h, t0 & mask);
        p.row1 = kv_row(c, p.ok1 ? p1 : 0, h, (t0 + 16) & mask);
        return p;
    };

    uint32_t kw[2][NB][KW];
    uint32_t vw[8][NC][VW];
    f32x4_t ksc[2], vsc[2];
    auto load_keys = [&](const TilePages &p) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int64_t row = u ? p.row1 : p.row0;
            const char *base = (const char *)c.k + row * row_bytes;
#pragma unroll
            for (int k = 0; k < NB; ++k) load_words<8 * ES>(base + koff[k], kw[u][k]);
            if constexpr (DT == KV_I8) {
                ksc[u] = *(const f32x4u_t *)(c.k_scale + row + 4 * cg);
            }
        }
    };
    auto load_values = [&](const TilePages &p) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int64_t row = u ? p.row1 : p.row0;
            const char *base = (const char *)c.v + row * row_bytes;
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int k = 0; k < NC; ++k)
                    load_words<DC * ES>(base + voff[k] + j * row_bytes, vw[4 * u + j][k]);
            if constexpr (DT == KV_I8) {
                vsc[u] = *(const f32x4u_t *)(c.v_scale + row + 4 * cg);
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
        // queries: column x of the B operands, all blocks
        Split<DT> qs[NB];
        float sc = scale * 1.4426950408889634f;
        {
            float f[NB][8];
            // heads past the block and dims past head_dim read others' and count as zero
            const float *qp = q + (int64_t)b * q_stride + (int64_t)(hq0 + min(x, gn - 1)) * c.dim;
#pragma unroll
            for (int k = 0; k < NB; ++k) {
                const int d0 = 32 * k + 8 * cg;
                const bool in = x < gn && d0 < c.dim;
                const f32x4u_t *at = (const f32x4u_t *)(qp + (d0 < c.dim ? d0 : 0));
                const f32x4_t v0 = at[0], v1 = at[1];
#pragma unroll
                for (int e = 0; e < 4; ++e) f[k][e] = in ? v0[e] : 0.0f, f[k][4 + e] = in ? v1[e] : 0.0f;
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
            const bool whole = t0 >= lo && t0 + 32 <= last && pg.ok0 && pg.ok1;
            // bit 4 u + i: this lane's position takes part
            uint32_t in = 0xFFu;
            if (!whole) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int t = t0 + 16 * (i / 4) + 4 * cg + i % 4;
                    if (t < lo || t >= last || !(i < 4 ? pg.ok0 : pg.ok1)) {
                        in &= ~(1u << i);
                        s[i / 4][i % 4] = -INFINITY;
                    }
                }
            }
            if (parts.scores && x < gn) {
                float *at = parts.scores +
                            ((int64_t)b * q_heads + hq0 + x) * parts.score_stride + t0 + 4 * cg;
                *(f32x4_t *)at = s[0];
                *(f32x4_t *)(at + 16) = s[1];
            }
            float top = s[0][0];
#pragma unroll
            for (int i = 1; i < 8; ++i) top = fmaxf(top, s[i / 4][i % 4]);
            if (__any(top > m)) {
                top = fmaxf(top, __shfl_xor(top, 16));
                top = fmaxf(top, __shfl_xor(top, 32));
                top = fmaxf(top, m);
                const float fade = top == -INFINITY ? 1.0f : pow2(m - top);
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
                p[i] = pow2(s[i / 4][i % 4] - ref);
                l += p[i];
            }
            if constexpr (DT == KV_I8) {
#pragma unroll
                for (int i = 0; i < 8; ++i) p[i] *= vsc[i / 4][i % 4];
                if (!whole) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (!(in >> i & 1u)) p[i] = 0.0f;
                }
            } else if (!whole) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
#pragma unroll
                    for (int k = 0; k < NC; ++k)
#pragma unroll
                        for (int i = 0; i < VW; ++i)
                            if (!(in >> j & 1u)) vw[j][k][i] = 0;
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
    const int64_t row = (int64_t)b * q_heads + hq0;
    const int64_t slot = (2 * (int64_t)blockIdx.x + (from == 0)) * 16;
    for (int i = threadIdx.x; i < gn * c.dim; i += 64 * kWaves) {
        const int g = i / c.dim, d = i % c.dim;
        float M = s_m[0][g];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) M = fmaxf(M, s_m[w][g]);
        float L = 0.0f, o = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            const float f = s_m[w][g] == -INFINITY ? 0.0f : pow2(s_m[w][g] - M);
            L += f * s_l[w][g];
            o += f * s_acc[w][g][d];
        }
        if (whole_block) {
            out[(row + g) * c.dim + d] = L == 0.0f ? 0.0f : o / L;
            if (parts.whole && d == 0) parts.whole[row + g] = make_float2(M, L);
        } else {
            parts.sum[(slot + g) * c.dim + d] = o;
            if (d == 0) parts.stat[slot + g] = make_float2(M, L);
        }
    }
    __syncthreads();
    } else if (steps == 0 && u == start) {
        // nothing to attend to
        for (int i = threadIdx.x; i < gn * c.dim; i += 64 * kWaves)
            out[((int64_t)b * q_heads + hq0) * c.dim + i] = 0.0f;
    }
    u = stop;
    if (u < u1 && vb + 1 == blocks) {
        base = u;
        ++b;
        n = kv_length(lens, b, most, d_status), lo = first_of(b), steps = kv_steps(lo, n);
    }
    }
}

// Maximum and sum of one head over the parts of its block, by one wave; every
// lane gets both.  Part 0 is the second part of workgroup w0, part i > 0 the
// first of w0 + i.
__device__ __forceinline__ int64_t part_slot(int w0, int i) {
    return (2 * (int64_t)(w0 + i) + (i == 0)) * 16;
}
__device__ __forceinline__ void joined(const float2 *stat, int w0, int count, int g, float &M,
                                       float &L) {
    const int lane = threadIdx.x & 63;
    M = -INFINITY;
    for (int i = lane; i < count; i += 64) M = fmaxf(M, stat[part_slot(w0, i) + g].x);
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor(M, o));
    L = 0.0f;
    for (int i = lane; i < count; i += 64) {
        const float2 v = stat[part_slot(w0, i) + g];
        if (v.y != 0.0f) L += pow2(v.x - M) * v.y;
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) L += __shfl_xor(L, o);
}

constexpr int kWeighTile = 1024;

// Workgroups below `joins` join the parts of one (sequence, query head):
// 1 << quad_bits threads take four dims each, the workgroup's 256 >> quad_bits
// groups of them every so many-th part, and the groups' sums are added in
// group order.  The others grow the weights of kWeighTile positions of one
// (sequence, key head) from the scores that the first kernel left.
__global__ __launch_bounds__(256) void k_kv_join(const int32_t *__restrict__ table,
                                                 const int32_t *__restrict__ lens,
                                                 const int32_t *__restrict__ starts,
                                                 float *__restrict__ out, KvParts parts,
                                                 int64_t cols, int64_t joins, int64_t tiles,
                                                 int q_heads, int most, float unit, int quad_bits,
                                                 KvPool c) {
    __shared__ float s_m[256], s_l[256];
    __shared__ f32x4_t s_o[256];
    const int G = q_heads / c.heads, gblocks = (G + 15) / 16;
    if ((int64_t)blockIdx.x < joins) {
        const int64_t row = blockIdx.x, b = row / q_heads;
        const int hq = (int)(row % q_heads), h = hq / G, g = hq % G;
        const int2 own = parts.owner[(b * c.heads + h) * gblocks + g / 16];
        if (own.x == own.y) return;  // one workgroup had it whole (or it is empty)
        const int count = own.y - own.x + 1;
        float M, L;
        joined(parts.stat, own.x, count, g % 16, M, L);
        const int quad = threadIdx.x & ((1 << quad_bits) - 1), group = threadIdx.x >> quad_bits;
        const int groups = 256 >> quad_bits, d = min(4 * quad, c.dim - 4);
        f32x4_t o = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int i = group; i < count; i += groups) {
            const int64_t slot = part_slot(own.x, i) + g % 16;
            const f32x4_t v = *(const f32x4_t *)(parts.sum + slot * c.dim + d);
            const float2 st = parts.stat[slot];
            const float f = st.y != 0.0f ? pow2(st.x - M) : 0.0f;
#pragma unroll
            for (int j = 0; j < 4; ++j) o[j] = fmaf(f, v[j], o[j]);
        }
        s_o[threadIdx.x] = o;
        __syncthreads();
        if (group == 0 && 4 * quad < c.dim) {
            for (int i = 1; i < groups; ++i) o += s_o[(i << quad_bits) + quad];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                out[row * c.dim + 4 * quad + j] = L == 0.0f ? 0.0f : o[j] / L;
        }
        return;
    }
    const int64_t w = blockIdx.x - joins;
    const int64_t bh = w / tiles, b = bh / c.heads;
    const int h = (int)(bh % c.heads);
    const int n = kv_length(lens, b, most, nullptr);
    const int lo = max((int)(w % tiles) * kWeighTile, starts ? max(starts[b], 0) : 0);
    const int hi = min((int)(w % tiles + 1) * kWeighTile, n);
    if (lo >= hi) return;
    float p[kWeighTile / 256] = {};
    for (int g0 = 0; g0 < G; g0 += 256) {
        const int gn = min(256, G - g0);
        __syncthreads();
        for (int g = threadIdx.x >> 6; g < gn; g += 4) {
            const int2 own = parts.owner[(b * c.heads + h) * gblocks + (g0 + g) / 16];
            float M, L;
            if (own.x == own.y) {
                const float2 v = parts.whole[b * q_heads + h * G + g0 + g];
                M = v.x, L = v.y;
            } else {
                joined(parts.stat, own.x, own.y - own.x + 1, (g0 + g) % 16, M, L);
            }
            if ((threadIdx.x & 63) == 0) s_m[g] = M, s_l[g] = L == 0.0f ? 0.0f : unit / L;
        }
        __syncthreads();
        for (int g = 0; g < gn; ++g) {
            const float M = s_m[g], f = s_l[g];
            const float *from =
                parts.scores + (b * q_heads + h * G + g0 + g) * parts.score_stride;
#pragma unroll
            for (int i = 0; i < kWeighTile / 256; ++i) {
                const int t = lo + (int)threadIdx.x + 256 * i;
                if (t < hi && f != 0.0f) p[i] += pow2(from[t] - M) * f;
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
    const int64_t joins = p.split ? seqs * q_heads : 0;
    const int64_t tiles = weigh ? (max_len + kWeighTile - 1) / kWeighTile : 0;
    const int64_t second = joins + tiles * seqs * c.heads;
    if (second > 0x7FFFFFFF) return hipErrorInvalidValue;
    char *ws = (char *)workspace;
    KvParts parts = {};
    if (p.split) {
        parts.stat = (float2 *)(ws + p.stat);
        parts.sum = (float *)(ws + p.sum);
    }
    if (second > 0) parts.owner = (int2 *)(ws + p.owner);
    if (weigh) {
        parts.whole = (float2 *)(ws + p.whole);
        parts.scores = (float *)(ws + p.scores);
    }
    parts.score_stride = p.score_stride;
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3((unsigned)p.groups), dim3(64 * kWaves), 0, stream, q,
                           table, lens, starts, (int)seqs, (int)q_heads, (int)max_len, scale,
                           q_stride, cols, c, out, parts, d_status);
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
    int quad_bits = 1;
    while (4 << quad_bits < c.dim) ++quad_bits;
    hipLaunchKernelGGL(k_kv_join, dim3((unsigned)second), dim3(256), 0, stream, table, lens,
                       starts, out, parts, cols, joins, tiles, (int)q_heads, (int)max_len,
                       dtype == KV_F16 ? 32768.0f : 1.0f, quad_bits, c);
    return hipGetLastError();
}

}  // namespace w4
