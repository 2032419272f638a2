// rope.cu -- rotary positions (internal): pairs (a, b) of a head's first
// `rot` channels turn by the angle positions[token] * inv_freq[pair],
//   a' = (a cos - b sin) * mscale      b' = (b cos + a sin) * mscale
// with the pair (i, i + rot / 2) or, interleaved, (2i, 2i + 1).
//
// Every row is read and written once: bound by HBM, for a few tokens by the
// launch. A block computes the sines of its tokens' angles once, in shared
// memory, and turns all heads with them; no table over positions is kept or
// read.
//
// An angle of a far position does not fit binary32. inv_freq (a double, in
// radians) is turned into a 64-bit fraction of a turn by integer arithmetic;
// position * fraction modulo 2^64 is then the exact rest of the turns, good to
// 2^-33 of a turn at any 32-bit position, and its top bits are the argument of
// a sine in half turns.
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace gai4 {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxPairs = 2048;   // (token, pair) sines in a block's shared memory

struct RopeArgs {
    const void* in[2];   // query and key rows
    void* out[2];
    int64_t in_stride[2], out_stride[2];
    int heads[2];
    const int32_t* positions;
    const double* inv_freq;
    float mscale;
    int64_t tokens;
    int d, half;         // channels of a head; pairs
    int per_block;       // tokens of a block
    int head_split;      // blocks of a token's heads
    int pass;            // 1: channels from 2 * half on are copied (outputs elsewhere)
};

// radians -> turns modulo 1, in units of 2^-64. 1 / (2 pi) = C 2^-66; the
// product of the 53-bit significand with C is shifted to the binary point.
// Infinite and NaN frequencies are left to the caller.
__device__ __forceinline__ uint64_t turn_fraction(double f) {
    const uint64_t b = (uint64_t)__double_as_longlong(f);
    const int be = (int)(b >> 52) & 0x7ff;
    const uint64_t m = (b & 0xfffffffffffffull) | (be ? 1ull << 52 : 0ull);
    constexpr uint64_t C = 0xa2f9836e4e441529ull;
    const uint64_t lo = m * C, hi = __umul64hi(m, C);
    // f = m 2^(e - 52), e = be - 1023: turns 2^64 = (hi : lo) 2^(e - 54)
    const int shift = 54 + 1023 - (be ? be : 1);
    uint64_t t;
    if (shift <= 0)
        t = -shift < 64 ? lo << -shift : 0;
    else if (shift < 64)
        t = (hi << (64 - shift)) | (lo >> shift);
    else
        t = shift < 128 ? hi >> (shift - 64) : 0;
    return (int64_t)b < 0 ? 0 - t : t;
}

// W consecutive elements as one access
template <typename T, int W>
struct Vec;
template <> struct Vec<BF16, 8> { using type = uint4; };
template <> struct Vec<BF16, 4> { using type = uint2; };
template <> struct Vec<BF16, 2> { using type = uint32_t; };
template <> struct Vec<BF16, 1> { using type = uint16_t; };
template <int W> struct Vec<F16, W> : Vec<BF16, W> {};
template <> struct Vec<F32, 4> { using type = uint4; };
template <> struct Vec<F32, 2> { using type = uint2; };
template <> struct Vec<F32, 1> { using type = float; };

template <typename T, int W>
union Pack {
    typename Vec<T, W>::type v;
    typename T::storage e[W];
};

// Items of a block: (token, head, chunk). A chunk is W pairs (two accesses of
// W elements each way) or, past them, W channels that are copied.
template <typename T, int W, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeArgs a) {
    using S = typename T::storage;
    using V = typename Vec<T, W>::type;
    pdl_launch_dependents();
    pdl_wait();   // the kernels before this one are complete: global memory may be read
    __shared__ __align__(16) float cs[2][kMaxPairs];
    const int64_t t0 = (int64_t)(blockIdx.x / (unsigned)a.head_split) * a.per_block;
    const int part = (int)(blockIdx.x % (unsigned)a.head_split);
    const int tokens = (int)min((int64_t)a.per_block, a.tokens - t0);
    for (int i = threadIdx.x; i < tokens * a.half; i += kThreads) {
        const int t = i / a.half;
        const double f = a.inv_freq[i - t * a.half];
        const uint64_t turns = (uint64_t)(int64_t)a.positions[t0 + t] * turn_fraction(f);
        float s, c;
        sincospif((float)(int64_t)turns * 0x1p-63f, &s, &c);
        const float m = isfinite(f) ? a.mscale : __uint_as_float(0x7fffffffu);
        cs[0][i] = c * m;
        cs[1][i] = s * m;
    }
    __syncthreads();
    const int heads = a.heads[0] + a.heads[1];
    const int h0 = heads * part / a.head_split, h1 = heads * (part + 1) / a.head_split;
    const int turned = a.half / W, chunks = turned + (a.pass ? (a.d - 2 * a.half) / W : 0);
    const int items = tokens * (h1 - h0) * chunks;
    for (int i = threadIdx.x; i < items; i += kThreads) {
        const int r = i / chunks, chunk = i - r * chunks;
        const int t = r / (h1 - h0);
        int head = h0 + r - t * (h1 - h0);
        const int which = head >= a.heads[0];
        if (which) head -= a.heads[0];
        const S* src = static_cast<const S*>(a.in[which]) + (t0 + t) * a.in_stride[which] + (int64_t)head * a.d;
        S* dst = static_cast<S*>(a.out[which]) + (t0 + t) * a.out_stride[which] + (int64_t)head * a.d;
        if (chunk >= turned) {
            const int at = 2 * a.half + (chunk - turned) * W;
            *reinterpret_cast<V*>(dst + at) = *reinterpret_cast<const V*>(src + at);
            continue;
        }
        const int at = INTERLEAVED ? 2 * chunk * W : chunk * W, next = INTERLEAVED ? W : a.half;
        Pack<T, W> p, q;
        p.v = *reinterpret_cast<const V*>(src + at);
        q.v = *reinterpret_cast<const V*>(src + at + next);
        const float* c = cs[0] + t * a.half + chunk * W;
        const float* s = cs[1] + t * a.half + chunk * W;
        if constexpr (!INTERLEAVED) {
#pragma unroll
            for (int j = 0; j < W; ++j) {
                const float u = T::to_f32(p.e[j]), v = T::to_f32(q.e[j]);
                p.e[j] = T::from_f32(u * c[j] - v * s[j]);
                q.e[j] = T::from_f32(v * c[j] + u * s[j]);
            }
        } else {
            S e[2 * W];
#pragma unroll
            for (int j = 0; j < W; ++j) {
                e[j] = p.e[j];
                e[W + j] = q.e[j];
            }
#pragma unroll
            for (int j = 0; j < W; ++j) {
                const float u = T::to_f32(e[2 * j]), v = T::to_f32(e[2 * j + 1]);
                e[2 * j] = T::from_f32(u * c[j] - v * s[j]);
                e[2 * j + 1] = T::from_f32(v * c[j] + u * s[j]);
            }
#pragma unroll
            for (int j = 0; j < W; ++j) {
                p.e[j] = e[j];
                q.e[j] = e[W + j];
            }
        }
        *reinterpret_cast<V*>(dst + at) = p.v;
        *reinterpret_cast<V*>(dst + at + next) = q.v;
    }
}

// elements of an access that every row and half of a head starts on
template <typename T>
int width(const RopeArgs& a) {
    for (int w = 16 / T::kBytes; w > 1; w /= 2) {
        bool ok = a.half % w == 0 && a.d % w == 0;
        for (int i = 0; i < 2; ++i)
            if (a.heads[i] > 0)
                ok = ok && (uintptr_t)a.in[i] % (w * T::kBytes) == 0 && (uintptr_t)a.out[i] % (w * T::kBytes) == 0 &&
                     a.in_stride[i] % w == 0 && a.out_stride[i] % w == 0;
        if (ok) return w;
    }
    return 1;
}

template <typename T>
cudaError_t rope_typed(RopeArgs a, bool interleaved, cudaStream_t s) {
    const int w = width<T>(a);
    const int64_t heads = a.heads[0] + a.heads[1];
    const int64_t per_token = heads * (a.half / w);   // items
    // About four items a thread; while that leaves SMs idle, fewer tokens a
    // block, then a token's heads on several blocks (which compute the same sines)
    const int64_t sms = num_sms();
    int64_t per = std::max<int64_t>(1, std::min<int64_t>(4 * kThreads / std::max<int64_t>(1, per_token), kMaxPairs / a.half));
    per = std::max<int64_t>(1, std::min(per, a.tokens / (4 * sms)));
    int64_t split = 1;
    while (per == 1 && a.tokens * split < 2 * sms && per_token / split > kThreads && split * 2 <= heads) split *= 2;
    a.per_block = (int)per;
    a.head_split = (int)split;
    const int64_t blocks = (a.tokens + per - 1) / per * split;
    if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
    const dim3 grid((unsigned)blocks), block(kThreads);
    if constexpr (T::kBytes == 2)
        if (w == 8)
            return launch_pdl(interleaved ? rope_kernel<T, 8, true> : rope_kernel<T, 8, false>, grid, block, 0, s, a);
    switch (w) {
    case 4: return launch_pdl(interleaved ? rope_kernel<T, 4, true> : rope_kernel<T, 4, false>, grid, block, 0, s, a);
    case 2: return launch_pdl(interleaved ? rope_kernel<T, 2, true> : rope_kernel<T, 2, false>, grid, block, 0, s, a);
    default: return launch_pdl(interleaved ? rope_kernel<T, 1, true> : rope_kernel<T, 1, false>, grid, block, 0, s, a);
    }
}

}  // namespace

cudaError_t launch_rope(const RopeLaunch& L, cudaStream_t s) {
    RopeArgs a{};
    for (int i = 0; i < 2; ++i) {
        a.in[i] = L.in[i];
        a.out[i] = L.out[i];
        a.in_stride[i] = L.in_stride[i];
        a.out_stride[i] = L.out_stride[i];
        a.heads[i] = L.heads[i];
        if (L.heads[i] > 0 && L.in[i] != L.out[i]) a.pass = 1;
    }
    a.positions = L.positions;
    a.inv_freq = L.inv_freq;
    a.mscale = L.mscale;
    a.tokens = L.tokens;
    a.d = L.head_dim;
    a.half = L.rot_dim / 2;
    switch (L.dtype) {
    case GAI4_F16: return rope_typed<F16>(a, L.interleaved, s);
    case GAI4_F32: return rope_typed<F32>(a, L.interleaved, s);
    default: return rope_typed<BF16>(a, L.interleaved, s);
    }
}

}  // namespace gai4
