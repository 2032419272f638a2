// rope.cu -- rotary positions (internal): pairs (a, b) of a head's first
// `rot` channels turn by the angle positions[token] * inv_freq[pair],
//   a' = (a cos - b sin) * mscale      b' = (b cos + a sin) * mscale
// with the pair (i, i + rot / 2) or, interleaved, (2i, 2i + 1).
//
// Every row is read and written once: bound by HBM, for a few tokens by the
// launch. A block computes the sines of its tokens' angles once, in shared
// memory, and turns all heads with them; no table over positions is kept or
// read. 20011 tokens of 40 heads of 128, 16 bits: 62 to 65 us (93 to 97% of the
// measured HBM rate); 64 tokens: 2.3 us.
//
// An angle of a far position does not fit binary32. inv_freq (a double, in
// radians) is turned into a 64-bit fraction of a turn by integer arithmetic;
// position * fraction modulo 2^64 is then the exact rest of the turns, good to
// 2^-32 of a turn at any 32-bit position; it is the argument of a sine in half
// turns, as the sum of two binary32 numbers.
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

// radians -> turns modulo 1, in units of 2^-64. 1 / (2 pi) = C 2^-130 with 128 bits;
// the product of the 53-bit significand with C, but for its last 64 bits, is shifted
// to the binary point. Frequencies of 2^53 and more, whose neighbours are 2 radians
// apart, and those that are no numbers are left to the caller.
__device__ __forceinline__ uint64_t turn_fraction(double f) {
    const uint64_t b = (uint64_t)__double_as_longlong(f);
    const int be = (int)(b >> 52) & 0x7ff;
    const uint64_t m = (b & 0xfffffffffffffull) | (be ? 1ull << 52 : 0ull);
    constexpr uint64_t C1 = 0xa2f9836e4e441529ull, C0 = 0xfc2757d1f534ddc0ull;
    const uint64_t low = m * C1, lo = low + __umul64hi(m, C0), hi = __umul64hi(m, C1) + (lo < low);
    // f = m 2^(e - 52), e = be - 1023: turns 2^64 = (hi : lo) 2^(e - 54)
    const int shift = 54 + 1023 - (be ? be : 1);   // (2 or more)
    const uint64_t l = shift < 64 ? lo : hi, h = shift < 64 ? hi : 0;
    const uint64_t t = shift < 128 ? l >> (shift & 63) | h << 1 << (~shift & 63) : 0;
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

// cos or sin of N neighbouring pairs
template <int N>
__device__ __forceinline__ void load_pairs(const float* p, float* v) {
    if constexpr (N >= 4) {
#pragma unroll
        for (int j = 0; j < N; j += 4) {
            const float4 f = *reinterpret_cast<const float4*>(p + j);
            v[j] = f.x; v[j + 1] = f.y; v[j + 2] = f.z; v[j + 3] = f.w;
        }
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = p[j];
    }
}

// One pair; written out, so that the widths of access round alike.
__device__ __forceinline__ float first(float x, float y, float c, float s) { return fmaf(x, c, -(y * s)); }
__device__ __forceinline__ float second(float x, float y, float c, float s) { return fmaf(x, s, y * c); }

// Turns W pairs: halves (p[j], q[j]), or neighbours along p and then q. 16-bit
// elements are taken and rounded two at a time.
template <typename T, int W, bool INTERLEAVED>
__device__ __forceinline__ void turn(Pack<T, W>& p, Pack<T, W>& q, const float (&c)[W], const float (&s)[W]) {
    if constexpr (T::kBytes == 2 && W >= 2) {
        constexpr int kWords = W / 2;
        uint32_t* a = reinterpret_cast<uint32_t*>(&p);
        uint32_t* b = reinterpret_cast<uint32_t*>(&q);
        const auto low = [](uint32_t w) { return T::to_f32((uint16_t)(w & 0xffffu)); };
        const auto high = [](uint32_t w) { return T::to_f32((uint16_t)(w >> 16)); };
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            if constexpr (INTERLEAVED) {
                const float x = low(a[i]), y = high(a[i]), u = low(b[i]), v = high(b[i]);
                const int j = kWords + i;
                a[i] = pack16<T>(first(x, y, c[i], s[i]), second(x, y, c[i], s[i]));
                b[i] = pack16<T>(first(u, v, c[j], s[j]), second(u, v, c[j], s[j]));
            } else {
                const float x = low(a[i]), u = high(a[i]), y = low(b[i]), v = high(b[i]);
                const int j = 2 * i;
                a[i] = pack16<T>(first(x, y, c[j], s[j]), first(u, v, c[j + 1], s[j + 1]));
                b[i] = pack16<T>(second(x, y, c[j], s[j]), second(u, v, c[j + 1], s[j + 1]));
            }
        }
    } else if constexpr (INTERLEAVED) {
        typename T::storage e[2 * W];
#pragma unroll
        for (int j = 0; j < W; ++j) {
            e[j] = p.e[j];
            e[W + j] = q.e[j];
        }
#pragma unroll
        for (int j = 0; j < W; ++j) {
            const float x = T::to_f32(e[2 * j]), y = T::to_f32(e[2 * j + 1]);
            e[2 * j] = T::from_f32(first(x, y, c[j], s[j]));
            e[2 * j + 1] = T::from_f32(second(x, y, c[j], s[j]));
        }
#pragma unroll
        for (int j = 0; j < W; ++j) {
            p.e[j] = e[j];
            q.e[j] = e[W + j];
        }
    } else {
#pragma unroll
        for (int j = 0; j < W; ++j) {
            const float x = T::to_f32(p.e[j]), y = T::to_f32(q.e[j]);
            p.e[j] = T::from_f32(first(x, y, c[j], s[j]));
            q.e[j] = T::from_f32(second(x, y, c[j], s[j]));
        }
    }
}

// A chunk is W pairs of a head (two accesses of W elements each way, half of the
// turned channels apart, so that neighbouring threads' lie side by side) or, past
// them, two accesses that are copied. A thread has one chunk of its block's rows
// (token, head), kBatch rows at a time: their loads are under way while the
// sines are computed.
template <typename T, int W, bool INTERLEAVED, bool PASS, int kBatch>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeArgs a) {
    using S = typename T::storage;
    using V = typename Vec<T, W>::type;
    pdl_launch_dependents();
    pdl_wait();   // the kernels before this one are complete: global memory may be read
    __shared__ __align__(16) float cs[2][kMaxPairs];
    const int64_t t0 = (int64_t)(blockIdx.x / (unsigned)a.head_split) * a.per_block;
    const int part = (int)(blockIdx.x % (unsigned)a.head_split);
    const int tokens = (int)min((int64_t)a.per_block, a.tokens - t0);
    const int all = a.heads[0] + a.heads[1];
    const int h0 = (int)((int64_t)all * part / a.head_split), heads = (int)((int64_t)all * (part + 1) / a.head_split) - h0;
    const int rows = tokens * heads;
    const float per_head = 1.0f / (float)heads;   // rows are below 2^21: (r + 1/2) / heads is never taken across a whole number
    // (copied accesses: the second of a chunk half of them apart, none for the last if they are odd)
    const int turned = a.half / W, copied = PASS ? (a.d - 2 * a.half) / W : 0, apart = (copied + 1) / 2;
    const int chunks = turned + apart;
    const int wide = chunks < kThreads ? kThreads / chunks : 1;   // rows that the block's threads take at a time
    const int tid = threadIdx.x;
    int chunk = chunks < kThreads ? tid % chunks : tid, r = chunks < kThreads ? tid / chunks : 0;
    if (r >= wide) chunk = chunks;   // (threads left over)

    S* to[kBatch];
    int pairs[kBatch];   // first pair's place among the sines
    Pack<T, W> p[kBatch], q[kBatch];
    // (single elements of a neighbouring pair are next to each other)
    constexpr bool kSingle = INTERLEAVED && W == 1;
    int next = kSingle ? 1 : a.half;   // from the first access to the second
    bool two = true;
    const auto load = [&]() {
        int at = (kSingle ? 2 : W) * chunk;
        if constexpr (PASS) {
            const bool turn = chunk < turned;
            next = turn ? (kSingle ? 1 : a.half) : apart * W;
            two = turn || chunk - turned + apart < copied;
            if (!turn) at = 2 * a.half + (chunk - turned) * W;
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int row = r + u * wide;
            if (chunk >= chunks || row >= rows) continue;
            const int t = (int)(((float)row + 0.5f) * per_head);
            int head = h0 + row - t * heads;
            const int which = head >= a.heads[0];
            if (which) head -= a.heads[0];
            const int64_t token = t0 + t;
            const S* src = static_cast<const S*>(a.in[which]) + token * a.in_stride[which] + (int64_t)head * a.d + at;
            to[u] = static_cast<S*>(a.out[which]) + token * a.out_stride[which] + (int64_t)head * a.d + at;
            pairs[u] = t * a.half + chunk * (INTERLEAVED && W > 1 ? W / 2 : W);
            p[u].v = *reinterpret_cast<const V*>(src);
            if (two) q[u].v = *reinterpret_cast<const V*>(src + next);
        }
    };
    load();
    for (int i = tid; i < tokens * a.half; i += kThreads) {
        const int t = i / a.half;
        const double f = a.inv_freq[i - t * a.half];
        const int64_t turns = (int64_t)((uint64_t)(int64_t)a.positions[t0 + t] * turn_fraction(f));
        // the angle in half turns as a sum of two: sine and cosine of the first, turned by the second
        const float hi = (float)turns, lo = (float)(turns - (int64_t)hi) * (3.14159265f * 0x1p-63f);
        float s, c;
        sincospif(hi * 0x1p-63f, &s, &c);
        const float m = fabs(f) < 0x1p53 ? a.mscale : __uint_as_float(0x7fffffffu);
        cs[0][i] = fmaf(-s, lo, c) * m;
        cs[1][i] = fmaf(c, lo, s) * m;
    }
    __syncthreads();
    while (chunk < chunks) {
        for (int first = r;;) {
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                if (first + u * wide >= rows) continue;
                if (!PASS || chunk < turned) {
                    float c[W], s[W];
                    if constexpr (INTERLEAVED && W > 1) {
                        // half of the pairs in each access
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            load_pairs<W / 2>(cs[0] + pairs[u] + h * (a.half / 2), c + h * (W / 2));
                            load_pairs<W / 2>(cs[1] + pairs[u] + h * (a.half / 2), s + h * (W / 2));
                        }
                    } else {
                        load_pairs<W>(cs[0] + pairs[u], c);
                        load_pairs<W>(cs[1] + pairs[u], s);
                    }
                    turn<T, W, INTERLEAVED>(p[u], q[u], c, s);
                }
                *reinterpret_cast<V*>(to[u]) = p[u].v;
                if (two) *reinterpret_cast<V*>(to[u] + next) = q[u].v;
            }
            r += kBatch * wide;
            first = r;
            if (r >= rows) break;
            load();
        }
        if (chunks <= kThreads) break;
        chunk += kThreads;   // (heads of more chunks than a block has threads)
        r = 0;
        if (chunk < chunks) load();
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

template <typename T, int W, bool INTERLEAVED>
cudaError_t rope_launch(RopeArgs a, cudaStream_t s) {
    // Many tokens, 16 bits: two rows a thread at a time, twice a block; f32: one, four
    // times; but enough blocks to go round. In us, (rows, times) (2, 2), (1, 2), (1, 4):
    // 20011 tokens of 40 heads of 128, bf16, 62, 80, 65; 3000 of them 13.1, 15.3, 14.1;
    // f32: 4099 of 40 of 128 31, 29, 29, 4099 of 32 of 80, 32 channels turned, 17.8, 21.8,
    // 16.8.
    constexpr int kMany = T::kBytes == 2 ? 2 : 1, kTimes = T::kBytes == 2 ? 2 : 4;
    const int64_t heads = a.heads[0] + a.heads[1];
    const bool pass = a.pass && a.d > 2 * a.half;
    const int64_t per_token = heads * (a.half / W + (pass ? ((a.d - 2 * a.half) / W + 1) / 2 : 0));   // chunks
    const int64_t sms = num_sms();
    int64_t per = 1, split = 1;
    const bool many = a.tokens * per_token > 4 * sms * kThreads;
    if (many)
        per = std::max<int64_t>(1, std::min<int64_t>({kTimes * kMany * kThreads / per_token, kMaxPairs / a.half, a.tokens / (6 * sms)}));
    else   // while SMs are idle, a token's heads go to several blocks, which compute the same sines
        while (a.tokens * split < 2 * sms && per_token / split > kThreads && split * 2 <= heads) split *= 2;
    a.per_block = (int)per;
    a.head_split = (int)split;
    const int64_t blocks = (a.tokens + per - 1) / per * split;
    if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
    const dim3 grid((unsigned)blocks), block(kThreads);
    if (pass)
        return launch_pdl(many ? rope_kernel<T, W, INTERLEAVED, true, kMany> : rope_kernel<T, W, INTERLEAVED, true, 1>, grid,
                          block, 0, s, a);
    return launch_pdl(many ? rope_kernel<T, W, INTERLEAVED, false, kMany> : rope_kernel<T, W, INTERLEAVED, false, 1>, grid, block,
                      0, s, a);
}

template <typename T>
cudaError_t rope_typed(const RopeArgs& a, bool interleaved, cudaStream_t s) {
    switch (width<T>(a)) {
    case 8:
        if constexpr (T::kBytes == 2) return interleaved ? rope_launch<T, 8, true>(a, s) : rope_launch<T, 8, false>(a, s);
        return cudaErrorInvalidValue;
    case 4: return interleaved ? rope_launch<T, 4, true>(a, s) : rope_launch<T, 4, false>(a, s);
    case 2: return interleaved ? rope_launch<T, 2, true>(a, s) : rope_launch<T, 2, false>(a, s);
    default: return interleaved ? rope_launch<T, 1, true>(a, s) : rope_launch<T, 1, false>(a, s);
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
