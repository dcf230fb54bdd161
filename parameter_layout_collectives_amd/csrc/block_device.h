// Device code that the kernels of the 8-bit blocks share: 8 elements of any
// input type as fp32, and 8 fp32 values as e4m3 codes with their block's scale.
#pragma once

#include "block.h"

namespace tide {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// Vectors of a row of any width and start: aligned as one element is.
typedef uint32_t half_u32x4 __attribute__((ext_vector_type(4), aligned(2)));
typedef float row_f32x4 __attribute__((ext_vector_type(4), aligned(4)));

// 8 consecutive elements as fp32.  `vec`: all `n` asked for are whole vectors
// (n is 0 or 8 then).
template <int ET>
__device__ __forceinline__ void load8(const char *p, int n, bool vec, float *v) {
#pragma unroll
    for (int i = 0; i < 8; i++) v[i] = 0.0f;
    if (n <= 0) return;
    if (ET == kElemF32) {
        const float *f = reinterpret_cast<const float *>(p);
        if (vec || n >= 8) {
            const f32x4 a = __builtin_nontemporal_load(reinterpret_cast<const row_f32x4 *>(f));
            const f32x4 b = __builtin_nontemporal_load(reinterpret_cast<const row_f32x4 *>(f + 4));
#pragma unroll
            for (int i = 0; i < 4; i++) v[i] = a[i], v[4 + i] = b[i];
        } else {
            for (int i = 0; i < 8; i++)
                if (i < n) v[i] = f[i];
        }
        return;
    }
    uint32_t w[4] = {0, 0, 0, 0};
    if (vec || n >= 8) {
        const u32x4 a = __builtin_nontemporal_load(reinterpret_cast<const half_u32x4 *>(p));
#pragma unroll
        for (int i = 0; i < 4; i++) w[i] = a[i];
    } else {
        const uint16_t *h = reinterpret_cast<const uint16_t *>(p);
#pragma unroll
        for (int i = 0; i < 8; i++) {
            // no branch, as each would wait for its load (60000 x 999: 73 -> 59 us);
            // in fp32 it is the other way round (10^6 x 41: 66 us, so 76)
            const uint32_t x = h[min(i, n - 1)];
            w[i / 2] |= i < n ? x << (16 * (i & 1)) : 0;
        }
    }
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const uint32_t h = (w[i / 2] >> (16 * (i & 1))) & 0xffffu;
        v[i] = ET == kElemBf16
                   ? __uint_as_float(h << 16)
                   : static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(h)));
    }
}

// The largest value over the 16 lanes of a row (DPP rotations by 8, 4, 2, 1).
__device__ __forceinline__ uint32_t max16(uint32_t u) {
    u = max(u, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(u), 0x128, 0xf, 0xf, false)));
    u = max(u, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(u), 0x124, 0xf, 0xf, false)));
    u = max(u, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(u), 0x122, 0xf, 0xf, false)));
    u = max(u, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(u), 0x121, 0xf, 0xf, false)));
    return u;
}

// The block exponent of a largest finite magnitude, given as its pattern:
// a = m * 2^k with 1 <= m < 2 is at most 448 * 2^e = 1.75 * 2^(8+e) from e = k - 8
// on if m <= 1.75, else from k - 7 on.
__device__ __forceinline__ int exponent_of(uint32_t top) {
    const int e = static_cast<int>(top >> 23) - 127 - 8 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0);
    return top == 0 ? 0 : min(119, max(-117, e));
}

// One lane's 8 values -> 8 codes; the block's scale byte is the same in all
// 16 lanes.  Patterns of |x| order like the values, so the maximum is taken on
// them as integers.  A block with an infinity or a NaN, or with a value that has
// to be cut at 448 * 2^119, shows as a maximum above that number's pattern and
// takes the long way.
__device__ __forceinline__ u32x2 encode8(const float *v, uint32_t *scale) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; i++) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
    top = max16(top);
    float y[8];
    bool odd = false;                     // an inf or a NaN among this lane's 8
    int e;
    if (top <= 0x7f600000u) {
        e = exponent_of(top);
        const float s = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
        for (int i = 0; i < 8; i++) y[i] = v[i] * s;
    } else {                              // the same for all 16 lanes
        top = 0;
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const uint32_t u = __float_as_uint(v[i]) & 0x7fffffffu;
            const bool finite = u < 0x7f800000u;
            odd |= !finite;
            top = max(top, finite ? u : 0u);
        }
        e = exponent_of(max16(top));
        const float s = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
        for (int i = 0; i < 8; i++) y[i] = __builtin_amdgcn_fmed3f(v[i] * s, -448.0f, 448.0f);
    }
    *scale = static_cast<uint32_t>(e + 127);
    int lo = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], lo, true);
    int hi = __builtin_amdgcn_cvt_pk_fp8_f32(y[4], y[5], 0, false);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(y[6], y[7], hi, true);
    u32x2 c = {static_cast<uint32_t>(lo), static_cast<uint32_t>(hi)};
    if (odd) {
#pragma unroll
        for (int i = 0; i < 8; i++)
            if ((__float_as_uint(v[i]) & 0x7f800000u) == 0x7f800000u) {
                const uint32_t m = 0xffu << (8 * (i & 3)), nan = 0x7fu << (8 * (i & 3));
                if (i < 4)
                    c.x = (c.x & ~m) | nan;
                else
                    c.y = (c.y & ~m) | nan;
            }
    }
    return c;
}

}  // namespace
}  // namespace tide
