// What the paged cache's kernels share: the cache as a kernel argument, its
// element types and the checks of what the host cannot see (lengths, positions
// and page ids on the device).
#pragma once

#include "common.h"

namespace w4 {

// The cache of include/w4.h with the page size as a shift; passed by value.
struct KvPool {
    void *k, *v;
    float *k_scale, *v_scale;  // KV_I8 only
    float *weight;             // may be null
    int pages, heads, shift, dim;
};

__device__ __forceinline__ bool kv_page_ok(const KvPool &c, int page) {
    return (unsigned)page < (unsigned)c.pages;
}

// Row index (position's row of head_dim elements) within a pool; also the
// index into the scales and weights.  64-bit: pools may pass 2^31 elements.
__device__ __forceinline__ int64_t kv_row(const KvPool &c, int page, int head, int slot) {
    return (((int64_t)page * c.heads + head) << c.shift) + slot;
}

// A length from the device, cut to [0, most]; says so in *d_status.
__device__ __forceinline__ int kv_length(const int32_t *lens, int64_t b, int most,
                                         int *d_status) {
    const int n = lens[b];
    if (n < 0 || n > most) {
        set_status(d_status, W4_ERR_BAD_SHAPE);
        return n < 0 ? 0 : most;
    }
    return n;
}

// Element types: KV_F32, KV_F16, KV_BF16, KV_I8 (codes; the caller scales).
template <int DT>
struct KvType;
template <>
struct KvType<KV_F32> {
    using T = float;
    static __device__ __forceinline__ float get(T v) { return v; }
    static __device__ __forceinline__ T put(float v) { return v; }
};
template <>
struct KvType<KV_F16> {
    using T = uint16_t;
    static __device__ __forceinline__ float get(T v) { return f16_bits_to_f32(v); }
    static __device__ __forceinline__ T put(float v) { return f32_to_f16_bits(v); }
};
template <>
struct KvType<KV_BF16> {
    using T = uint16_t;
    static __device__ __forceinline__ float get(T v) {
        return __builtin_bit_cast(float, (uint32_t)v << 16);
    }
    // to nearest, ties to even; a NaN keeps its sign and stays a NaN
    static __device__ __forceinline__ T put(float v) {
        const uint32_t u = __builtin_bit_cast(uint32_t, v);
        if ((u & 0x7FFFFFFFu) > 0x7F800000u) return (uint16_t)((u >> 16) | 0x40u);
        return (uint16_t)((u + 0x7FFFu + ((u >> 16) & 1u)) >> 16);
    }
};
template <>
struct KvType<KV_I8> {
    using T = int8_t;
    static __device__ __forceinline__ float get(T v) { return (float)v; }
};

// fp32 values in an order that unsigned integers have: larger value, larger
// key.  -0 counts as +0; the caller decides about NaN.
__device__ __forceinline__ uint32_t order_key(float v) {
    const uint32_t u = __builtin_bit_cast(uint32_t, v == 0.0f ? 0.0f : v);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float order_value(uint32_t key) {
    return __builtin_bit_cast(float, key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}

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

}  // namespace w4
