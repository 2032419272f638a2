// kv_attention.cu -- causal attention over the paged 4-bit key/value cache.
//
// Simple form: one block per (query row, query head). Each of its warps walks
// every fourth key with the running maximum and sum of a softmax, a lane
// holding D / 32 neighbouring elements; the four partial results are joined in
// shared memory. Everything in binary32.
#include <math.h>

#include "common.cuh"
#include "internal.h"

namespace gai4 {
namespace {

template <typename T, int D, int GS>
__global__ void __launch_bounds__(128) kv_attention_simple(const KvAttnLaunch p) {
    constexpr int E = D / 32;   // elements per lane
    __shared__ float sm_m[4], sm_l[4], sm_o[4][D];
    pdl_launch_dependents();
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long t = blockIdx.x;
    const int head = blockIdx.y, h = head / p.group;
    const int hq = p.sh.hkv * p.group;
    // request of this row: the last with cu_q[r] <= t
    int lo = 0, hi = p.batch;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.cu_q[mid] <= t) lo = mid;
        else hi = mid;
    }
    const int r = lo, q0 = p.cu_q[r], q1 = p.cu_q[r + 1];
    const bool mine = t >= q0 && t < q1;
    const long long cap = p.max_blocks << p.sh.page_log2;
    const long long kv = min((long long)p.kv_lens[r], cap);
    const long long pos = kv - (q1 - q0) + (t - q0);
    const long long end = mine ? pos + 1 : 0;
    const long long begin = p.window > 0 && end > p.window ? end - p.window : 0;

    float q[E], o[E];
    using St = typename T::storage;
    const St* qp = static_cast<const St*>(p.q) + t * p.q_stride + (long long)head * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        q[e] = T::to_f32(qp[e]);
        o[e] = 0.f;
    }
    float m = -INFINITY, l = 0.f;
    const int word = lane * E / 8, shift = (lane * E % 8) * 4, grp = lane * E / GS;
    for (long long j = begin + warp; j < end; j += 4) {
        const int page = p.table[(long long)r * p.max_blocks + (j >> p.sh.page_log2)];
        if (page < 0 || page >= p.sh.num_blocks) continue;
        const long long row = (((long long)page * p.sh.hkv + h) << p.sh.page_log2) + (j & ((1 << p.sh.page_log2) - 1));
        const uint32_t kw = p.k.packed[row * (D / 8) + word] >> shift, vw = p.v.packed[row * (D / 8) + word] >> shift;
        const long long g = row * (D / GS) + grp;
        const float ks = T::to_f32(static_cast<const St*>(p.k.scales)[g]);
        const float kb = T::to_f32(static_cast<const St*>(p.k.biases)[g]);
        const float vs = T::to_f32(static_cast<const St*>(p.v.scales)[g]);
        const float vb = T::to_f32(static_cast<const St*>(p.v.biases)[g]);
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) s = fmaf(q[e], fmaf(ks, (float)((kw >> (4 * e)) & 15u), kb), s);
        s = warp_sum(s) * p.scale;
        const float mn = fmaxf(m, s);
        const float c = mn == -INFINITY ? 0.f : expf(m - mn), w = mn == -INFINITY ? 0.f : expf(s - mn);
        m = mn;
        l = l * c + w;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = o[e] * c + w * fmaf(vs, (float)((vw >> (4 * e)) & 15u), vb);
    }
    if (lane == 0) {
        sm_m[warp] = m;
        sm_l[warp] = l;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) sm_o[warp][lane * E + e] = o[e];
    __syncthreads();
    float M = fmaxf(fmaxf(sm_m[0], sm_m[1]), fmaxf(sm_m[2], sm_m[3])), L = 0.f, acc = 0.f;
    const int d = threadIdx.x;
    for (int w = 0; w < 4; ++w) {
        const float c = sm_m[w] == -INFINITY ? 0.f : expf(sm_m[w] - M);
        L += sm_l[w] * c;
        if (d < D) acc += sm_o[w][d] * c;
    }
    if (d < D)
        static_cast<St*>(p.out)[t * p.out_stride + (long long)head * D + d] = T::from_f32(L == 0.f ? 0.f : acc / L);
    if (p.lse && d == 0) p.lse[t * hq + head] = L == 0.f ? -INFINITY : M + logf(L);
}

template <typename T>
cudaError_t launch_simple(const KvAttnLaunch& L, cudaStream_t s) {
    const dim3 grid((unsigned)L.num_tokens, (unsigned)(L.sh.hkv * L.group));
    const dim3 block(128);
    if (L.sh.d == 64)
        return L.sh.gs == 32 ? launch_pdl(kv_attention_simple<T, 64, 32>, grid, block, 0, s, L)
                             : launch_pdl(kv_attention_simple<T, 64, 64>, grid, block, 0, s, L);
    return L.sh.gs == 32   ? launch_pdl(kv_attention_simple<T, 128, 32>, grid, block, 0, s, L)
           : L.sh.gs == 64 ? launch_pdl(kv_attention_simple<T, 128, 64>, grid, block, 0, s, L)
                           : launch_pdl(kv_attention_simple<T, 128, 128>, grid, block, 0, s, L);
}

}  // namespace

size_t kv_attention_workspace(int group, int d) { return 0; }

cudaError_t launch_kv_attention(const KvAttnLaunch& L, cudaStream_t s) {
    switch (L.sh.dtype) {
    case GAI4_F32: return launch_simple<F32>(L, s);
    case GAI4_F16: return launch_simple<F16>(L, s);
    default: return launch_simple<BF16>(L, s);
    }
}

}  // namespace gai4
