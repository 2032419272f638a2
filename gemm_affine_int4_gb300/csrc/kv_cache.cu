// kv_cache.cu -- bookkeeping and rows of the paged 4-bit key/value cache
// (gai4_kv_plan, gai4_kv_append, gai4_kv_read).
#include "common.cuh"
#include "internal.h"

namespace gai4 {
namespace {

// ---------------------------------------------------------------------------
// plan: with old length l, n new tokens and page size P, request r needs
// ceil((l + n) / P) - ceil(l / P) new pages; exclusive prefix sums over the
// requests of n, of the pages taken and of the pages given back say where its
// rows, its pops and its pushes are. Every block computes the sums over all
// requests for itself (8 bytes a request, from L2) and then does its share of
// the tokens, so no block waits for another. Reads and writes do not meet:
// pushed pages are written at or above free_count and read only below it (a
// popped page that was pushed in this step is taken from the finished
// request's row), and table columns are written only from ceil(l / P) on.
// Bound by latency, a chain of dependent reads, scans and barriers: 64 requests
// of one token 3.2 us; 1000 requests with up to 133 new tokens each (0.9 MB)
// 7.7 us.
// ---------------------------------------------------------------------------
constexpr int kPlanThreads = 1024;

struct Sum3 {
    long long q, took, gave;
};

__device__ __forceinline__ Sum3 add3(Sum3 a, Sum3 b) { return {a.q + b.q, a.took + b.took, a.gave + b.gave}; }

__device__ __forceinline__ Sum3 shfl_up3(Sum3 v, int o) {
    return {__shfl_up_sync(0xffffffffu, v.q, o), __shfl_up_sync(0xffffffffu, v.took, o),
            __shfl_up_sync(0xffffffffu, v.gave, o)};
}

// largest i in [0, n) with a[i] <= x, for ascending a with a[0] <= x
__device__ __forceinline__ int last_not_above(const int* a, int n, int x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(kPlanThreads) kv_plan_kernel(const KvPlanLaunch p) {
    extern __shared__ int plan_smem[];
    __shared__ Sum3 warp_sums[32];
    __shared__ int bad_rows, bad_len;
    pdl_launch_dependents();
    pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, B = p.batch, pl = p.page_log2;
    const long long pm = (1ll << pl) - 1;
    int* cu = plan_smem;           // [B + 1] first row of each request
    int* tk = cu + B + 1;          // [B + 1] pages popped before it
    int* gv = tk + B + 1;          // [B + 1] pages pushed before it
    if (tid == 0) bad_rows = bad_len = 0;
    __syncthreads();

    // each thread takes `per` consecutive requests
    const int per = (B + kPlanThreads - 1) / kPlanThreads;
    const int r0 = min(tid * per, B), r1 = min(r0 + per, B);
    auto one = [&](int r, int& rows_bad, int& len_bad) {
        const long long l = p.kv_lens[r], n = p.q_lens[r];
        const long long had = (l + pm) >> pl, need = n < 0 ? had : (l + n + pm) >> pl;
        len_bad |= l < 0;
        rows_bad += need > p.max_blocks;
        return n < 0 ? Sum3{0, 0, had} : Sum3{n, need - had, 0};
    };
    Sum3 mine{0, 0, 0};
    int rows_bad = 0, len_bad = 0;
    for (int r = r0; r < r1; ++r) mine = add3(mine, one(r, rows_bad, len_bad));
    if (rows_bad) atomicAdd(&bad_rows, rows_bad);
    if (len_bad) bad_len = 1;
    Sum3 inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Sum3 u = shfl_up3(inc, o);
        if (lane >= o) inc = add3(inc, u);
    }
    if (lane == 31) warp_sums[warp] = inc;
    __syncthreads();
    if (warp == 0) {
        Sum3 w = warp_sums[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const Sum3 u = shfl_up3(w, o);
            if (lane >= o) w = add3(w, u);
        }
        warp_sums[lane] = w;
    }
    __syncthreads();
    const Sum3 total = warp_sums[31];
    Sum3 at = {inc.q - mine.q, inc.took - mine.took, inc.gave - mine.gave};
    if (warp > 0) at = add3(at, warp_sums[warp - 1]);

    const long long count = p.free_count[0];
    const long long missing = total.took - (count + total.gave);
    const long long over = total.q - p.num_tokens;
    const bool wrong = bad_len || count < 0 || count + total.gave > p.free_capacity;
    const bool refused = missing > 0 || bad_rows > 0 || over > 0 || wrong;
    const long long top = refused ? count : count + total.gave;
    if (blockIdx.x == 0 && tid == 0) {
        const long long most = 0x7fffffff;
        p.info[0] = wrong ? 0 : (int)min(max(missing, 0ll), most);
        p.info[1] = bad_rows;
        p.info[2] = (int)min(max(over, 0ll), most);
        p.info[3] = wrong;
        p.free_count_out[0] = (int)(refused ? count : top - total.took);
        p.cu_q[B] = refused ? 0 : (int)total.q;
    }
    if (tid == 0) {
        cu[B] = (int)total.q;
        tk[B] = (int)total.took;
        gv[B] = (int)total.gave;
    }
    int unused = 0;
    for (int r = r0; r < r1; ++r) {
        cu[r] = (int)at.q;
        tk[r] = (int)at.took;
        gv[r] = (int)at.gave;
        at = add3(at, one(r, unused, unused));
        if (blockIdx.x == 0) {
            const int l = p.kv_lens[r], n = p.q_lens[r];
            p.cu_q[r] = refused ? 0 : cu[r];
            p.kv_lens_out[r] = refused ? l : (n < 0 ? 0 : l + n);
        }
    }
    __syncthreads();

    const long long stride = (long long)gridDim.x * kPlanThreads, first = (long long)blockIdx.x * kPlanThreads + tid;
    if (refused) {
        for (long long t = first; t < p.num_tokens; t += stride) {
            p.slots[t] = -1;
            p.positions[t] = 0;
        }
        return;
    }
    // page number `i` from the bottom of the stack after the pushes
    auto stack = [&](int i) {
        if (i < count) return p.free_blocks[i];
        const int j = i - (int)count;
        const int r = last_not_above(gv, B, j);
        return p.table[(long long)r * p.max_blocks + (j - gv[r])];
    };
    // tokens
    for (long long t = first; t < p.num_tokens; t += stride) {
        long long slot = -1;
        int pos = 0;
        if (t < total.q) {
            const int r = last_not_above(cu, B, (int)t);
            const int l = p.kv_lens[r];
            const int had = (int)((l + pm) >> pl);
            pos = l + ((int)t - cu[r]);
            const int blk = pos >> pl;
            const int page = blk < had ? p.table[(long long)r * p.max_blocks + blk]
                                       : stack((int)top - 1 - (tk[r] + blk - had));
            slot = ((long long)page << pl) + (pos & pm);
        }
        p.slots[t] = slot;
        p.positions[t] = pos;
    }
    // pushes and new table entries, one request per warp
    const int nwarps = gridDim.x * (kPlanThreads / 32);
    for (int r = blockIdx.x * (kPlanThreads / 32) + warp; r < B; r += nwarps) {
        const int gave = gv[r + 1] - gv[r], took = tk[r + 1] - tk[r];
        int* row = p.table + (long long)r * p.max_blocks;
        for (int j = lane; j < gave; j += 32) p.free_blocks[count + gv[r] + j] = row[j];
        if (took > 0) {
            const int had = (int)((p.kv_lens[r] + pm) >> pl);
            for (int j = lane; j < took; j += 32) row[had + j] = stack((int)top - 1 - (tk[r] + j));
        }
    }
}

// ---------------------------------------------------------------------------
// rows: lane-sized pieces of 8 elements = one word of codes
// ---------------------------------------------------------------------------
// slot -> first row index of (page, head, offset), or -1 outside the pool
__device__ __forceinline__ long long cache_row(long long slot, int h, const KvShape& sh) {
    if (slot < 0 || slot >= (sh.num_blocks << sh.page_log2)) return -1;
    const long long page = slot >> sh.page_log2;
    return (((page * sh.hkv + h) << sh.page_log2) + (slot & ((1ll << sh.page_log2) - 1)));
}

template <typename T, bool VEC>
__device__ __forceinline__ void load8(const void* p, long long at, float (&x)[8]) {
    const typename T::storage* s = static_cast<const typename T::storage*>(p) + at;
    if constexpr (!VEC) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = T::to_f32(s[i]);
    } else if constexpr (T::kBytes == 4) {
        const float4 a = *reinterpret_cast<const float4*>(s), b = *reinterpret_cast<const float4*>(s + 4);
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    } else {
        const uint4 a = *reinterpret_cast<const uint4*>(s);
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = T::to_f32((uint16_t)w[i]);
            x[2 * i + 1] = T::to_f32((uint16_t)(w[i] >> 16));
        }
    }
}

// two binary32 operations at once
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n add.rn.f32x2 d, a, b;\n"
        " mov.b64 {%0, %1}, d;\n}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n .reg .b64 a, b, c, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mov.b64 c, {%6, %7};\n"
        " fma.rn.f32x2 d, a, b, c;\n mov.b64 {%0, %1}, d;\n}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float mul_sat(float a, float b) {
    float d;
    asm("mul.rn.sat.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

// Codes of eight elements: clamp(rint((x - b) / s), 0, 15), the quotient an
// IEEE division. A fifteenth of the reciprocal, clamped to [0, 1] and taken
// fifteenfold, is within 1e-5 of the quotient clamped to [0, 15], so its
// rounding is the code unless it lies next to a half; only then (and where the
// reciprocal is not finite) the divisions are done. Adding 3 * 2^22 rounds to
// an integer, in the sum's low bits.
__device__ __forceinline__ uint32_t codes8(const float (&x)[8], float s, float b) {
    if (s == 0.0f) return 0u;
    float inv;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
    const float k = inv * (1.0f / 15.0f), magic = 12582912.0f;
    const float2 nb = make_float2(-b, -b), up = make_float2(magic, magic), down = make_float2(-magic, -magic);
    const float2 c15 = make_float2(15.0f, 15.0f), m15 = make_float2(-15.0f, -15.0f);
    uint32_t word = 0;
    float far = 0.0f;   // largest distance from an integer
#pragma unroll
    for (int i = 6; i >= 0; i -= 2) {
        float2 u = add2(make_float2(x[i], x[i + 1]), nb);
        u.x = mul_sat(u.x, k);
        u.y = mul_sat(u.y, k);
        const float2 y = fma2(u, c15, up);
        const float2 d = fma2(u, m15, add2(y, down));
        far = fmaxf(far, fmaxf(fabsf(d.x), fabsf(d.y)));
        word = word * 16u + (__float_as_uint(y.y) & 15u);
        word = word * 16u + (__float_as_uint(y.x) & 15u);
    }
    if (far >= 0.4999f || !(inv < 1e38f)) {
        word = 0;
        for (int i = 0; i < 8; ++i) {
            const float r = rintf(__fdiv_rn(__fsub_rn(x[i], b), s));
            const uint32_t q = r <= 0.0f ? 0u : (r >= 15.0f ? 15u : (uint32_t)r);
            word |= q << (4 * i);
        }
    }
    return word;
}

// One group is GS / 8 neighbouring lanes; its extremes come from a butterfly
// over them. Scale, bias and codes are those of gai4_quantize: the same
// binary32 steps, each rounded once. A warp has SETS sets of rows in flight:
// four where they still give every SM work, else one (64 tokens of 2 x 8 rows
// and two reads: 5.5 us with one, 8.9 with four). Bound by instructions: 20011
// tokens of 2 x 8 rows of 128 f16 values in groups of 32 (113 MB), 36 us; with
// a division for every code it took 82.
// No signal of programmatic launch here: what is written is in the form of
// packed weights, which gai4_qmv and gai4_qmm_t read before the kernels ahead of
// them have ended.
template <typename T, int D, int GS, bool VEC, int SETS>
__global__ void __launch_bounds__(256) kv_append_kernel(const void* k, long long ks, const void* v, long long vs,
                                                        const int64_t* __restrict__ slots, KvCache kc, KvCache vc,
                                                        KvShape sh, int tokens) {
    constexpr int LPR = D / 8, LPG = GS / 8;   // lanes per row and per group
    constexpr int RPW = 32 / LPR;              // rows of a warp's set
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int sub = lane / LPR, li = lane % LPR;
    // a block's rows: consecutive tokens of one head of k or v (whose slots
    // are neighbours as a rule)
    const int tb = blockIdx.x / (2 * sh.hkv), unit = blockIdx.x - tb * (2 * sh.hkv);
    const bool is_v = unit >= sh.hkv;
    const int h = is_v ? unit - sh.hkv : unit;
    const void* in = is_v ? v : k;
    const long long stride = is_v ? vs : ks;
    const KvCache c = is_v ? vc : kc;
    const int token0 = (tb * 8 + (threadIdx.x >> 5)) * RPW * SETS + sub;
    float x[SETS][8];
    long long dst[SETS];
#pragma unroll
    for (int u = 0; u < SETS; ++u) {
        const int token = token0 + u * RPW;
        const bool live = token < tokens;
        load8<T, VEC>(in, (live ? token : 0) * stride + (long long)h * D + li * 8, x[u]);
        dst[u] = live ? cache_row(slots[token], h, sh) : -1;
    }
#pragma unroll
    for (int u = 0; u < SETS; ++u) {
        float mn = x[u][0], mx = x[u][0];
#pragma unroll
        for (int i = 1; i < 8; ++i) {
            mn = fminf(mn, x[u][i]);
            mx = fmaxf(mx, x[u][i]);
        }
#pragma unroll
        for (int o = 1; o < LPG; o <<= 1) {
            mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        }
        const typename T::storage s_h = T::from_f32(__fdiv_rn(__fsub_rn(mx, mn), 15.0f)), b_h = T::from_f32(mn);
        const uint32_t word = codes8(x[u], T::to_f32(s_h), T::to_f32(b_h));
        if (dst[u] >= 0) {
            const_cast<uint32_t*>(c.packed)[dst[u] * LPR + li] = word;
            if (li % LPG == 0) {
                const long long g = dst[u] * (D / GS) + li / LPG;
                static_cast<typename T::storage*>(const_cast<void*>(c.scales))[g] = s_h;
                static_cast<typename T::storage*>(const_cast<void*>(c.biases))[g] = b_h;
            }
        }
    }
}

// A thread expands one word (eight values, two stores); neighbouring threads
// write on. Bound by the writes: 20011 tokens of 8 rows of 128 values (82 MB
// out, 15 in), 22 us, where a fill of 82 MB takes 15; with four values a thread
// it took 24, with the tokens of one head a block 25.
template <typename T, int D, int GS>
__global__ void __launch_bounds__(256) kv_read_kernel(KvCache c, const int64_t* __restrict__ slots, float* out,
                                                      KvShape sh, long long rows) {
    constexpr int LPR = D / 8, RPB = 256 / LPR;   // threads of a row, rows of a block
    pdl_launch_dependents();
    pdl_wait();
    const int li = threadIdx.x % LPR;
    const long long row = (long long)blockIdx.x * RPB + threadIdx.x / LPR;   // (token, head)
    if (row >= rows) return;
    const long long token = row / sh.hkv;
    const long long src = cache_row(slots[token], (int)(row - token * sh.hkv), sh);
    uint32_t w = 0u;
    float s = 0.0f, b = 0.0f;
    if (src >= 0) {
        w = c.packed[src * LPR + li];
        const long long g = src * (D / GS) + li / (GS / 8);
        s = T::to_f32(static_cast<const typename T::storage*>(c.scales)[g]);
        b = T::to_f32(static_cast<const typename T::storage*>(c.biases)[g]);
    }
    float4* o = reinterpret_cast<float4*>(out) + (row * LPR + li) * 2;
#pragma unroll
    for (int i = 0; i < 2; ++i)
        o[i] = make_float4(fmaf(s, (float)((w >> (16 * i)) & 15u), b), fmaf(s, (float)((w >> (16 * i + 4)) & 15u), b),
                           fmaf(s, (float)((w >> (16 * i + 8)) & 15u), b), fmaf(s, (float)((w >> (16 * i + 12)) & 15u), b));
}

// calls f<T, D, GS>() for the runtime type, head size and group size
template <typename F>
cudaError_t by_type(int dtype, F&& f) {
    switch (dtype) {
    case GAI4_F32: return f(F32{});
    case GAI4_F16: return f(F16{});
    default: return f(BF16{});
    }
}

template <int D_, int GS_>
struct Sizes {
    static constexpr int D = D_, GS = GS_;
};
template <typename F>
cudaError_t by_sizes(int d, int gs, F&& f) {
    if (d == 64) return gs == 32 ? f(Sizes<64, 32>{}) : f(Sizes<64, 64>{});
    return gs == 32 ? f(Sizes<128, 32>{}) : gs == 64 ? f(Sizes<128, 64>{}) : f(Sizes<128, 128>{});
}

}  // namespace

cudaError_t launch_kv_plan(const KvPlanLaunch& L, cudaStream_t s) {
    const size_t smem = 3 * sizeof(int) * (size_t)(L.batch + 1);
    if (smem > 48 * 1024) {
        static bool allowed[64];
        const cudaError_t e = allow_smem_once(kv_plan_kernel, 3 * sizeof(int) * (kKvPlanMaxBatch + 1), allowed);
        if (e != cudaSuccess) return e;
    }
    int64_t blocks = (L.num_tokens + 2 * kPlanThreads - 1) / (2 * kPlanThreads);
    const int64_t by_rows = (L.batch + 255) / 256;
    if (blocks < by_rows) blocks = by_rows;
    if (blocks > num_sms()) blocks = num_sms();
    return launch_pdl(kv_plan_kernel, dim3((unsigned)blocks), dim3(kPlanThreads), smem, s, L);
}

cudaError_t launch_kv_append(const void* k, int64_t ks, const void* v, int64_t vs, const int64_t* slots, KvCache kc,
                             KvCache vc, const KvShape& sh, int64_t num_tokens, cudaStream_t s) {
    return by_type(sh.dtype, [&](auto t) {
        using T = decltype(t);
        return by_sizes(sh.d, sh.gs, [&](auto z) {
            using Z = decltype(z);
            const bool vec = ((uintptr_t)k & 15) == 0 && ((uintptr_t)v & 15) == 0 && ks * T::kBytes % 16 == 0 &&
                             vs * T::kBytes % 16 == 0;
            // block numbers of one launch stay below 2^31
            constexpr int per_set = 8 * (32 / (Z::D / 8));   // tokens of a block with one set of rows a warp
            const int64_t chunk = ((1ll << 30) / (2 * sh.hkv)) * per_set;
            for (int64_t t0 = 0; t0 < num_tokens; t0 += chunk) {
                const int64_t n = num_tokens - t0 < chunk ? num_tokens - t0 : chunk;
                const int sets = n * 2 * sh.hkv >= 4ll * 8 * per_set * num_sms() ? 4 : 1, per_block = per_set * sets;
                const dim3 grid((unsigned)((n + per_block - 1) / per_block * (2 * sh.hkv)));
                const void* kp = static_cast<const char*>(k) + t0 * ks * T::kBytes;
                const void* vp = static_cast<const char*>(v) + t0 * vs * T::kBytes;
                const auto kernel = vec ? (sets == 4 ? kv_append_kernel<T, Z::D, Z::GS, true, 4> : kv_append_kernel<T, Z::D, Z::GS, true, 1>)
                                        : (sets == 4 ? kv_append_kernel<T, Z::D, Z::GS, false, 4> : kv_append_kernel<T, Z::D, Z::GS, false, 1>);
                const cudaError_t e = launch_pdl(kernel, grid, dim3(256), 0, s, kp, (long long)ks, vp, (long long)vs,
                                                 slots + t0, kc, vc, sh, (int)n);
                if (e != cudaSuccess) return e;
            }
            return cudaSuccess;
        });
    });
}

cudaError_t launch_kv_read(KvCache c, const int64_t* slots, float* out, const KvShape& sh, int64_t num_tokens,
                           cudaStream_t s) {
    return by_type(sh.dtype, [&](auto t) {
        using T = decltype(t);
        return by_sizes(sh.d, sh.gs, [&](auto z) {
            using Z = decltype(z);
            constexpr int per_block = 256 / (Z::D / 8);
            const long long rows = num_tokens * sh.hkv, blocks = (rows + per_block - 1) / per_block;
            if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
            return launch_pdl(kv_read_kernel<T, Z::D, Z::GS>, dim3((unsigned)blocks), dim3(256), 0, s, c, slots, out, sh, rows);
        });
    });
}

}  // namespace gai4
