// fp8_quant.cuh -- rounding to e4m3 with a scale for a group of 128 (internal).
//
// A group whose largest magnitude is a (at least 2^-100) has the scale
// RN(a / 448) and the codes nearest_e4m3(448 x / a), ties to even: 448 is the
// largest e4m3 value. Quotients of 16-bit inputs lie on the border between two
// codes now and then (448 x / a has few bits), so the quotient is rounded
// correctly to binary32 before the conversion: an exact tie stays one. A
// product with 448 / a or with the scale's reciprocal would break such ties at
// random.
#pragma once

#include "common.cuh"

namespace gai4 {
namespace fp8 {

constexpr int kGroup = 128;
constexpr float kLeastMax = 7.888609052210118e-31f;   // 2^-100

// |v| as an integer that grows with it; infinities above every number, NaN
// above infinities (a maximum of these does not lose a NaN)
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

struct Scale {
    float amax;   // at least 2^-100; infinite or NaN if the group holds such a value
    float rcp;
};
__device__ __forceinline__ Scale scale_of(uint32_t amax_bits) {
    const uint32_t least = __float_as_uint(kLeastMax);
    Scale s;
    s.amax = __uint_as_float(amax_bits < least ? least : amax_bits);
    s.rcp = __frcp_rn(s.amax);
    return s;
}
__device__ __forceinline__ float scale_value(const Scale& s) { return __fdiv_rn(s.amax, 448.0f); }

// 448 x / amax, rounded to nearest: c = 448 x 2^-9 (exact for 16-bit x, no
// overflow), a first quotient from the correctly rounded reciprocal, and one
// correction by its exact residual. If amax is infinite or NaN the residual is
// NaN, and with it every code of the group.
__device__ __forceinline__ float quotient(float x, const Scale& s) {
    const float c = x * 0.875f;
    const float t = c * s.rcp;
    return fmaf(fmaf(-t, s.amax, c), s.rcp, t) * 512.0f;
}

// two codes, `lo` in the low byte
__device__ __forceinline__ uint32_t codes2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// 8 values -> 8 codes
__device__ __forceinline__ uint2 codes8(const float (&v)[8], const Scale& s) {
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = codes2(quotient(v[2 * i], s), quotient(v[2 * i + 1], s));
    return make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
}

// ---------------------------------------------------------------------------
// 8 consecutive elements of a row: 16-byte accesses, or one by one with the
// row's end at `left` elements (VEC false)
// ---------------------------------------------------------------------------
template <typename T, bool VEC>
__device__ __forceinline__ void load8(const typename T::storage* p, int64_t left, float (&v)[8]) {
    if constexpr (VEC) {
        if constexpr (T::kBytes == 4) {
            const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
            v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
            v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
        } else {
            const uint4 a = *reinterpret_cast<const uint4*>(p);
            const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[2 * i] = T::to_f32((uint16_t)(w[i] & 0xffffu));
                v[2 * i + 1] = T::to_f32((uint16_t)(w[i] >> 16));
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < left ? T::to_f32(p[i]) : 0.f;
    }
}

template <typename T, bool VEC>
__device__ __forceinline__ void store8(typename T::storage* p, int64_t left, const float (&v)[8]) {
    if constexpr (VEC) {
        if constexpr (T::kBytes == 4) {
            reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
            reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i] = (uint32_t)T::from_f32(v[2 * i]) | (uint32_t)T::from_f32(v[2 * i + 1]) << 16;
            *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < left) p[i] = T::from_f32(v[i]);
    }
}

template <bool VEC>
__device__ __forceinline__ void store_codes8(uint8_t* p, int64_t left, uint2 c) {
    if constexpr (VEC) {
        *reinterpret_cast<uint2*>(p) = c;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < left) p[i] = (uint8_t)((i < 4 ? c.x : c.y) >> (8 * (i & 3)));
    }
}

__device__ __forceinline__ uint32_t amax8(const float (&v)[8]) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, abs_bits(v[i]));
    return m;
}
// over the 16 lanes that hold a group
__device__ __forceinline__ uint32_t group_max(uint32_t m) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    return m;
}

}  // namespace fp8
}  // namespace gai4
