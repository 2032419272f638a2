// fp8_quant.cuh -- rounding to e4m3 with a scale for a group of 128 (internal).
//
// A group whose largest magnitude is a (at least 2^-100) has the scale
// RN(a / 448) and the codes nearest_e4m3(448 x / a), ties to even: 448 is the
// largest e4m3 value. Quotients of 16-bit inputs lie on the border between two
// codes now and then (448 x / a has few bits), so the quotient is rounded
// correctly to binary32 before the conversion: an exact tie stays one. A
// product with 448 / a as one number, or with the scale's reciprocal, would break
// such ties at random.
#pragma once

#include "common.cuh"

namespace gai4 {
namespace fp8 {

constexpr int kGroup = 128;
constexpr float kLeastMax = 7.888609052210118e-31f;   // 2^-100

// the larger magnitude; a NaN stays one
__device__ __forceinline__ float max_abs(float a, float b) {
    float r;
    asm("{\n .reg .f32 x, y;\n abs.f32 x, %1;\n abs.f32 y, %2;\n max.NaN.f32 %0, x, y;\n}" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

struct Scale {
    float amax;      // at least 2^-100 (infinite or NaN if the group holds such a value)
    float f, rest;   // 448 / amax as a sum of two
};
__device__ __forceinline__ Scale scale_of(float amax) {
    Scale s;
    s.amax = max_abs(amax, kLeastMax);
    s.f = __fdiv_rn(448.0f, s.amax);
    s.rest = fmaf(-s.f, s.amax, 448.0f) * (s.f * (1.0f / 448.0f));   // the residual is exact
    return s;
}
__device__ __forceinline__ float scale_value(const Scale& s) { return __fdiv_rn(s.amax, 448.0f); }

// 448 x / amax, good to 2^-46 before its one rounding, so that what is exact in
// binary32 stays exact. If amax is infinite or NaN the residual is NaN, and with it
// every code of the group.
__device__ __forceinline__ float quotient(float x, const Scale& s) { return fmaf(x, s.f, x * s.rest); }

// two codes, `lo` in the low byte
__device__ __forceinline__ uint32_t codes2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// 8 quotients -> 8 codes
__device__ __forceinline__ uint2 codes8(const float (&q)[8]) {
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = codes2(q[2 * i], q[2 * i + 1]);
    return make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
}
__device__ __forceinline__ uint2 codes8(const float (&v)[8], const Scale& s) {
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = quotient(v[i], s);
    return codes8(q);
}

// ---------------------------------------------------------------------------
// A thread's eight elements of a group of 128 that 16 threads hold. VEC: eight
// neighbours, in 16-byte accesses. Otherwise every 16th, so that the single
// accesses of the threads lie side by side. `left`: from the first of them to the
// row's end.
// ---------------------------------------------------------------------------
template <bool VEC>
__device__ __forceinline__ int column_of(int thread) {   // thread of the row
    return VEC ? thread * 8 : (thread >> 4) * kGroup + (thread & 15);
}
constexpr int kApart = 16;

template <typename T, bool VEC>
struct Eight {
    // as loaded: 16 bytes of 16-bit elements, or values
    static constexpr bool kPacked = VEC && T::kBytes == 2;
    uint4 w;
    float v[kPacked ? 1 : 8];

    __device__ __forceinline__ void load(const typename T::storage* p, int64_t left) {
        if constexpr (kPacked) {
            w = *reinterpret_cast<const uint4*>(p);
        } else if constexpr (VEC) {
            const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
            v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
            v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                typename T::storage raw = 0;
                if (kApart * i < left) raw = p[kApart * i];
                // (the zero is not converted apart, behind a branch: the loads are issued together)
                if constexpr (T::kBytes == 2) asm("" : "+h"(raw));
                v[i] = T::to_f32(raw);
            }
        }
    }
    __device__ __forceinline__ void zero() {
        if constexpr (kPacked) {
            w = make_uint4(0, 0, 0, 0);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = 0.f;
        }
    }
    // from here on the values are made anew (not kept as binary32 from before)
    __device__ __forceinline__ void keep() {
        if constexpr (kPacked) asm("" : "+r"(w.x), "+r"(w.y), "+r"(w.z), "+r"(w.w));
    }
    __device__ __forceinline__ void values(float (&to)[8]) const {
        if constexpr (kPacked) {
            const uint32_t h[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                to[2 * i] = T::to_f32((uint16_t)(h[i] & 0xffffu));
                to[2 * i + 1] = T::to_f32((uint16_t)(h[i] >> 16));
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) to[i] = v[i];
        }
    }
};

template <typename T, bool VEC>
__device__ __forceinline__ void store8(typename T::storage* p, int64_t left, const float (&v)[8]) {
    if constexpr (VEC) {
        if constexpr (T::kBytes == 4) {
            reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
            reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = pack16<T>(v[2 * i], v[2 * i + 1]);
            *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (kApart * i < left) p[kApart * i] = T::from_f32(v[i]);
    }
}

template <bool VEC>
__device__ __forceinline__ void store_codes8(uint8_t* p, int64_t left, uint2 c) {
    if constexpr (VEC) {
        *reinterpret_cast<uint2*>(p) = c;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (kApart * i < left) p[kApart * i] = (uint8_t)((i < 4 ? c.x : c.y) >> (8 * (i & 3)));
    }
}

__device__ __forceinline__ float amax8(const float (&v)[8]) {
    float m = max_abs(v[0], v[1]);
#pragma unroll
    for (int i = 2; i < 8; ++i) m = max_abs(m, v[i]);
    return m;
}
// over the 16 lanes that hold a group
__device__ __forceinline__ float group_max(float m) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m = max_abs(m, __shfl_xor_sync(0xffffffffu, m, o));
    return m;
}

}  // namespace fp8
}  // namespace gai4
