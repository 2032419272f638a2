// kv_attention_tc.cu -- causal attention over the paged 4-bit key/value cache
// for many query rows per key/value head (prompts and chunks of them), bf16
// and f16, on the tensor cores (tcgen05, accumulators in tensor memory).
//
// One CTA (one per SM) takes 256 query rows of one key/value head, as two M
// tiles of 128 (a row is one query head of one token: the heads that share
// the key head lie side by side), and walks the keys in tiles of 128 tokens:
//   S_i = Q_i K^T          tcgen05, Q and K from shared memory
//   P_i = exp2(f S_i - m)  four warps per M tile, one thread per row
//   O_i += P_i V           tcgen05, P from tensor memory, V from shared memory
// The products of one M tile run while the other's softmax does. Keys and
// values are expanded once per CTA for both M tiles by four warps of their
// own, rounded once to T (fma of code, scale and bias), as gai4_qmm_t rounds
// its weights.
//
// Tensor memory: S_0, S_1, O_0, O_1, 128 columns each; P_i overwrites the
// first 64 columns of S_i. Products are issued in the order PV_0 QK_0 PV_1
// QK_1, so the commit of QK_i of a tile also says that PV_i of the tile
// before it has finished: a softmax warp may then rescale O_i, which it does
// only when a row's maximum has grown by more than 2^8 (P and the sum are
// merely larger until then).
//
// Codes of a word come out of it as pairs (0, 4), (1, 5), (2, 6), (3, 7); that
// order of the channels is kept in shared memory (queries are stored in it,
// outputs put back from it), which saves a permutation per pair.
// bf16: a code masked out of its word is the subnormal c 2^-133 (or c 2^-129),
// and fma(c 2^-133, s 2^93, b 2^-40) is the value times 2^-40, rounded once;
// the power leaves through f and through the last division. Keys and values
// from 2^-86 to 2^37 keep all their bits.
// f16: codes by the offset of 1024, then fma(c, s, b).
//
// Every barrier is waited on by the same role phase after phase.
#include <math.h>

#include "common.cuh"
#include "internal.h"
#include "pipeline.cuh"

namespace gai4 {
namespace kvt {

using namespace pipe;

constexpr int kKeys = 128;            // tokens of a key tile
constexpr int kRows = 256;            // query rows of a CTA
constexpr int kThreads = 32 * 14;     // 8 softmax warps, 4 expanding, 1 product issuer, 1 producer
constexpr int kRing = 3;              // packed stages (keys and values in turn)

__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// 128-byte swizzled operand descriptors: low word start address and leading
// byte offset, high word stride byte offset (1024: from 8 rows to the next),
// version 1, layout SWIZZLE_128B
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << (46 - 32)) | (2u << (61 - 32));
__device__ __forceinline__ uint32_t desc_k(uint32_t a) { return ((a >> 4) & 0x3FFFu) | (1u << 16); }
// N-major operand (rows are the contraction): leading offset from 64 columns to the next 64
__device__ __forceinline__ uint32_t desc_n(uint32_t a) { return ((a >> 4) & 0x3FFFu) | ((kKeys * 128u >> 4) << 16); }

// instruction descriptor, kind::f16, fp32 accumulate, M = 128; bit 16: B is N-major
constexpr uint32_t idesc(bool bf, int n, bool b_n_major) {
    return (1u << 4) | ((bf ? 1u : 0u) << 7) | ((bf ? 1u : 0u) << 10) | ((b_n_major ? 1u : 0u) << 16) |
           ((uint32_t)(n >> 3) << 17) | ((128u >> 4) << 24);
}

// issued by a converged warp: one elected lane
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t id, uint32_t acc) {
    asm volatile(
        "{\n .reg .pred p, e;\n .reg .b32 r;\n .reg .b64 x, y;\n elect.sync r|e, 0xffffffff;\n setp.ne.b32 p, %4, 0;\n"
        " mov.b64 x, {%1, %5};\n mov.b64 y, {%2, %5};\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n}" ::"r"(d),
        "r"(a_lo), "r"(b_lo), "r"(id), "r"(acc), "r"(kDescHi)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t id, uint32_t acc) {
    asm volatile(
        "{\n .reg .pred p, e;\n .reg .b32 r;\n .reg .b64 y;\n elect.sync r|e, 0xffffffff;\n setp.ne.b32 p, %4, 0;\n"
        " mov.b64 y, {%2, %5};\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n}" ::"r"(d),
        "r"(a), "r"(b_lo), "r"(id), "r"(acc), "r"(kDescHi)
        : "memory");
}
__device__ __forceinline__ void commit(uint64_t* bar) {
    asm volatile(
        "{\n .reg .pred e;\n .reg .b32 r;\n elect.sync r|e, 0xffffffff;\n"
        " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}" ::"r"(smem_u32(bar))
        : "memory");
}

__device__ __forceinline__ void tmem_ld32(uint32_t a, uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
          "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
          "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(a)
        : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t a, const uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(a),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
        "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
        "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
        : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t a, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16};" ::"r"(a),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}
__device__ __forceinline__ void tmem_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
template <bool BF>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t d;
    if constexpr (BF) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}
template <bool BF>
__device__ __forceinline__ uint32_t fma2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    if constexpr (BF) asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    else asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
__device__ __forceinline__ uint32_t mul_bf2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t sub_f16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// power of two that values and keys carry (see above)
template <bool BF>
constexpr float kUndo = BF ? 1099511627776.f : 1.f;   // 2^40

// scale and bias of a group, in the forms that the codes need
template <bool BF>
struct Group {
    uint32_t s0, s1, b;
    __device__ __forceinline__ Group(uint32_t s, uint32_t bias) {
        s |= s << 16;
        bias |= bias << 16;
        if constexpr (BF) {
            s0 = mul_bf2(s, 0x6E006E00u);      // s 2^93 (for codes at bits 0..3)
            s1 = mul_bf2(s, 0x6C006C00u);      // s 2^89 (bits 4..7)
            b = mul_bf2(bias, 0x2B802B80u);    // b 2^-40
        } else {
            s0 = s1 = s;
            b = bias;
        }
    }
};

// one word of codes -> values (0, 4), (1, 5), (2, 6), (3, 7)
template <bool BF>
__device__ __forceinline__ uint4 expand(uint32_t w, const Group<BF>& g) {
    uint4 o;
    const uint32_t h = w >> 8;
    if constexpr (BF) {
        o.x = fma2<true>(w & 0x000F000Fu, g.s0, g.b);
        o.y = fma2<true>(w & 0x00F000F0u, g.s1, g.b);
        o.z = fma2<true>(h & 0x000F000Fu, g.s0, g.b);
        o.w = fma2<true>(h & 0x00F000F0u, g.s1, g.b);
    } else {
        // 1024 + c, and 64 (1024 + 16 c) / 1024 - 64 = c
        o.x = fma2<false>(sub_f16x2((w & 0x000F000Fu) | 0x64006400u, 0x64006400u), g.s0, g.b);
        o.y = fma2<false>(fma2<false>((w & 0x00F000F0u) | 0x64006400u, 0x2C002C00u, 0xD400D400u), g.s0, g.b);
        o.z = fma2<false>(sub_f16x2((h & 0x000F000Fu) | 0x64006400u, 0x64006400u), g.s0, g.b);
        o.w = fma2<false>(fma2<false>((h & 0x00F000F0u) | 0x64006400u, 0x2C002C00u, 0xD400D400u), g.s0, g.b);
    }
    return o;
}

template <int D>
struct Smem {
    static constexpr uint32_t kAtom = 128 * 128;                        // 128 rows x 64 channels
    static constexpr uint32_t kTile = (D / 64) * kAtom;                 // one Q, K or V tile
    static constexpr uint32_t kMaxNG = D / 32;
    static constexpr uint32_t kStage = kKeys * (D / 2 + 4 * kMaxNG);    // codes, scales, biases
    static constexpr uint32_t q = 0, k = 2 * kTile, v = k + 2 * kTile, ring = v + 2 * kTile,
                              masks = ring + kRing * kStage, bars = masks + kRing * 16, total = bars + 256;
};

struct Req {
    int q0, qn, kv;
};
__device__ __forceinline__ Req request(const KvAttnLaunch& p, int r) {
    Req q;
    const int n = (int)p.num_tokens;
    q.q0 = min(max(p.cu_q[r], 0), n);
    q.qn = max(min(p.cu_q[r + 1], n) - q.q0, 0);
    q.kv = (int)min((long long)max(p.kv_lens[r], 0), (long long)p.max_blocks << p.sh.page_log2);
    return q;
}

template <bool BF, int D>
__global__ void __launch_bounds__(kThreads, 1)
    kv_attention_tc_kernel(const __grid_constant__ KvAttnLaunch p, const int gs_log2, const int min_rows, const int vec_q,
                           const int vec_out) {
    using T = typename std::conditional<BF, BF16, F16>::type;
    using M = Smem<D>;
    extern __shared__ uint8_t raw[];
    __shared__ long long warp_units[kThreads / 32];
    __shared__ int unit_r, unit_i, abort_flag;
    __shared__ uint32_t tmem_slot;
    uint8_t* smem = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + M::bars);
    uint64_t *ring_full = bars, *ring_empty = bars + kRing, *k_full = bars + 2 * kRing, *k_empty = k_full + 2,
             *v_full = k_full + 4, *v_empty = k_full + 6, *s_full = k_full + 8, *p_full = k_full + 10,
             *q_full = k_full + 12, *o_full = k_full + 13;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    pdl_launch_dependents();
    if (tid == 0) {
        for (int i = 0; i < kRing; ++i) {
            mbar_init(&ring_full[i], 1);
            mbar_init(&ring_empty[i], 4);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&k_full[i], 4);
            mbar_init(&k_empty[i], 1);
            mbar_init(&v_full[i], 4);
            mbar_init(&v_empty[i], 1);
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 4);
        }
        mbar_init(q_full, 8);
        mbar_init(o_full, 1);
        abort_flag = 0;
        unit_r = -1;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_async();
    }
    pdl_wait();

    // unit of this CTA: (request, block of 256 rows, key/value head), the
    // blocks of a request from the last (longest) to the first
    auto blocks_of = [&](const Req& q) {
        const long long rows = (long long)q.qn * p.group;
        return rows >= min_rows ? (rows + kRows - 1) / kRows : 0ll;
    };
    const int per = (p.batch + kThreads - 1) / kThreads;
    const int r0 = min(tid * per, p.batch), r1 = min(r0 + per, p.batch);
    long long mine = 0;
    for (int r = r0; r < r1; ++r) mine += blocks_of(request(p, r)) * p.sh.hkv;
    long long inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += u;
    }
    if (lane == 31) warp_units[warp] = inc;
    __syncthreads();
    long long before = inc - mine;
    for (int i = 0; i < warp; ++i) before += warp_units[i];
    if (before <= blockIdx.x && blockIdx.x < before + mine) {
        long long at = before;
        int r = r0;
        for (long long n; at + (n = blocks_of(request(p, r)) * p.sh.hkv) <= blockIdx.x; ++r) at += n;
        unit_r = r;
        unit_i = (int)(blockIdx.x - at);
    }
    // rows that belong to no request
    {
        const int hq = p.sh.hkv * p.group;
        const long long first = max(min((long long)p.cu_q[p.batch], (long long)p.num_tokens), 0ll);
        for (long long row = first + blockIdx.x; row < p.num_tokens; row += gridDim.x) {
            uint16_t* o = static_cast<uint16_t*>(p.out) + row * p.out_stride;
            for (int i = tid; i < hq * D; i += kThreads) o[i] = 0;
            if (p.lse)
                for (int i = tid; i < hq; i += kThreads) p.lse[row * hq + i] = -INFINITY;
        }
    }
    __syncthreads();
    if (unit_r < 0) return;
    if (warp == 12) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_slot)), "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = tmem_slot;

    const Req rq = request(p, unit_r);
    const int rows = (int)min((long long)rq.qn * p.group, 0x7fffffffll);
    const int nblk = (rows + kRows - 1) / kRows;
    const int blk = nblk - 1 - unit_i / p.sh.hkv, h = unit_i % p.sh.hkv;
    const int row0 = blk * kRows;
    const int nm = rows - row0 > 128 ? 2 : 1;               // M tiles with rows
    // key tiles that some row sees
    const int tok_a = row0 / p.group, tok_b = min(row0 + kRows, rows) - 1;
    const long long pos_a = (long long)rq.kv - rq.qn + tok_a, pos_b = (long long)rq.kv - rq.qn + tok_b / p.group;
    const long long lo = p.window > 0 ? max(pos_a - p.window + 1, 0ll) : 0;
    const int t_first = (int)(lo / kKeys);
    const int t_end = (int)((max(pos_b + 1, 0ll) + kKeys - 1) / kKeys);
    const int n = max(t_end - t_first, 0);
    const Ctl ctl{p.status, p.spin_limit, &abort_flag};

    if (warp == 13) {
        // ---------------- producer: packed keys and values of each tile in turn ----------------
        const int pl = p.sh.page_log2;
        const int pieces = pl >= 7 ? 1 : kKeys >> pl, tokens = pl >= 7 ? kKeys : 1 << pl;
        const int piece = lane / 3, which = lane - 3 * piece;
        const bool active = piece < pieces;
        const int ng = D >> gs_log2;
        const uint32_t row_bytes = which == 0 ? D / 2 : 2 * ng;
        const uint32_t bytes = tokens * row_bytes;
        const uint32_t dst0 = smem_u32(smem + M::ring) +
                              (which == 0 ? 0u : kKeys * (D / 2) + (which - 1) * kKeys * 2 * ng) + piece * bytes;
        const uint8_t* src[2];
        src[0] = static_cast<const uint8_t*>(which == 0   ? static_cast<const void*>(p.k.packed)
                                             : which == 1 ? p.k.scales
                                                          : p.k.biases);
        src[1] = static_cast<const uint8_t*>(which == 0   ? static_cast<const void*>(p.v.packed)
                                             : which == 1 ? p.v.scales
                                                          : p.v.biases);
        const int* table = p.table + (long long)unit_r * p.max_blocks;
        const int npages = (rq.kv + (1 << pl) - 1) >> pl;
        uint32_t* masks = reinterpret_cast<uint32_t*>(smem + M::masks);
        int issued = 0, tok = t_first * kKeys + piece * tokens;
        int page = n > 0 && active && (tok >> pl) < npages ? table[tok >> pl] : -1;
        bool ok = true;
        for (int t = 0; t < n && ok; ++t) {
            const bool there = active && page >= 0 && page < p.sh.num_blocks;
            const uint32_t votes = __ballot_sync(0xffffffffu, there && which == 0);
            const long long line = there ? (((long long)page * p.sh.hkv + h) << pl) + (tok & ((1 << pl) - 1)) : 0;
            const int left = rq.kv - (t_first + t) * kKeys;
            tok += kKeys;
            page = active && (tok >> pl) < npages ? table[tok >> pl] : -1;   // of the next tile
            // token bits of this tile, 32 per lane for lanes 0..3
            uint32_t m = 0;
            for (int b = 0; b < 32; b += 16) {
                const int o = (lane & 3) * 32 + b;
                const int pc = o / tokens;
                if ((votes >> (3 * pc)) & 1u) m |= 0xffffu << b;
            }
            const int l = left - (lane & 3) * 32;
            if (l < 32) m &= l <= 0 ? 0u : (1u << l) - 1u;
            for (int kv = 0; kv < 2; ++kv, ++issued) {
                const int s = issued % kRing;
                if (!warp_wait(&ring_empty[s], ((issued / kRing) & 1) ^ 1, ctl)) {
                    ok = false;
                    break;
                }
                if (lane < 4) masks[s * 4 + lane] = m;
                __syncwarp();
                if (lane == 0)
                    mbar_arrive_expect_tx(&ring_full[s], (uint32_t)__popc(votes) * tokens * (D / 2 + 4 * ng));
                __syncwarp();
                if (there)
                    asm volatile(
                        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                            dst0 + s * M::kStage),
                        "l"(src[kv] + line * row_bytes), "r"(bytes), "r"(smem_u32(&ring_full[s]))
                        : "memory");
            }
        }
        for (int i = issued > kRing ? issued - kRing : 0; i < issued; ++i)
            mbar_wait_drain(&ring_full[i % kRing], (i / kRing) & 1, ctl.limit, ctl.status);
    } else if (warp == 12) {
        // ---------------- products ----------------
        constexpr uint32_t id_s = idesc(BF, kKeys, false), id_o = idesc(BF, D, true);
        const uint32_t qb = smem_u32(smem + M::q), kb = smem_u32(smem + M::k), vb = smem_u32(smem + M::v);
        auto qk = [&](int i, int j) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t o = (kk >> 2) * M::kAtom + (kk & 3) * 32;
                mma_ss(tmem + 128 * i, desc_k(qb + i * M::kTile + o), desc_k(kb + (j & 1) * M::kTile + o), id_s, kk > 0);
            }
            commit(&s_full[i]);
        };
        auto pv = [&](int i, int j) {
#pragma unroll
            for (int kk = 0; kk < kKeys / 16; ++kk)
                mma_ts(tmem + 256 + 128 * i, tmem + 128 * i + 8 * kk, desc_n(vb + (j & 1) * M::kTile + kk * 2048), id_o,
                       j > 0 || kk > 0);
        };
        bool ok = n > 0 && warp_wait(q_full, 0, ctl) && warp_wait(&k_full[0], 0, ctl);
        if (ok) {
            fence_after();
            for (int i = 0; i < nm; ++i) qk(i, 0);
            commit(&k_empty[0]);
        }
        for (int j = 0; ok && j < n; ++j) {
            ok = warp_wait(&v_full[j & 1], (j >> 1) & 1, ctl);
            for (int i = 0; ok && i < nm; ++i) {
                ok = warp_wait(&p_full[i], j & 1, ctl);
                if (!ok) break;
                fence_after();
                pv(i, j);
                if (i == nm - 1) commit(&v_empty[j & 1]);
                if (j + 1 < n) {
                    if (i == 0) ok = warp_wait(&k_full[(j + 1) & 1], ((j + 1) >> 1) & 1, ctl);
                    if (!ok) break;
                    fence_after();
                    qk(i, j + 1);
                    if (i == nm - 1) commit(&k_empty[(j + 1) & 1]);
                }
            }
        }
        commit(o_full);
        if (lane == 0) mbar_wait_drain(o_full, 0, ctl.limit, ctl.status);   // no product may outlive the tensor memory
        __syncwarp();
    } else if (warp >= 8) {
        // ---------------- expanding keys and values: one token per thread ----------------
        const int r = (warp - 8) * 32 + lane;
        const int ng = D >> gs_log2;
        const uint32_t row = (uint32_t)r * 128u;
        const uint32_t* masks = reinterpret_cast<const uint32_t*>(smem + M::masks);
        for (int i = 0; i < 2 * n; ++i) {
            const int s = i % kRing, j = i >> 1;
            uint64_t *full = i & 1 ? &v_full[j & 1] : &k_full[j & 1], *empty = i & 1 ? &v_empty[j & 1] : &k_empty[j & 1];
            uint8_t* dst = smem + (i & 1 ? M::v : M::k) + (j & 1) * M::kTile + row;
            (void)warp_wait(&ring_full[s], (i / kRing) & 1, ctl);
            (void)warp_wait(empty, ((j >> 1) & 1) ^ 1, ctl);
            const uint8_t* st = smem + M::ring + s * M::kStage;
            const uint16_t* sc = reinterpret_cast<const uint16_t*>(st + kKeys * (D / 2)) + r * ng;
            const uint16_t* bi = sc + kKeys * ng;
            const bool valid = (masks[s * 4 + (r >> 5)] >> (r & 31)) & 1u;   // else zeros: the slot may hold anything
#pragma unroll
            for (int x = 0; x < D / 32; ++x) {
                // 32 channels; neighbouring rows take them in another order (banks)
                const int c = (x + (r >> (D == 128 ? 1 : 2))) & (D / 32 - 1);
                const uint4 w = *reinterpret_cast<const uint4*>(st + r * (D / 2) + c * 16);
                const int g = (32 * c) >> gs_log2;
                const Group<BF> gr(valid ? sc[g] : 0u, valid ? bi[g] : 0u);
                const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int ch = 4 * c + k;   // 16-byte chunk of the row
                    *reinterpret_cast<uint4*>(dst + (ch >> 3) * M::kAtom + (((ch & 7) ^ (r & 7)) << 4)) =
                        expand<BF>(ww[k], gr);
                }
            }
            fence_async();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(full);
                mbar_arrive(&ring_empty[s]);
            }
        }
    } else {
        // ---------------- softmax: M tile i, one row per thread ----------------
        const int i = warp >> 2, r = (warp & 3) * 32 + lane;
        const int row = row0 + i * 128 + r;
        const bool live = row < rows;
        const int tok = live ? row / p.group : 0;
        const int head = h * p.group + (live ? row - tok * p.group : 0);
        // query row into shared memory; a negative scale turns its sign
        {
            const uint16_t* src = static_cast<const uint16_t*>(p.q) + (long long)(rq.q0 + tok) * p.q_stride + (long long)head * D;
            const uint32_t flip = p.scale < 0.f ? 0x80008000u : 0u;
            uint8_t* dst = smem + M::q + i * M::kTile + r * 128;
#pragma unroll 4
            for (int ch = 0; ch < D / 8; ++ch) {
                uint32_t w[4] = {0u, 0u, 0u, 0u};
                if (live) {
                    if (vec_q) {
                        const uint4 x = *reinterpret_cast<const uint4*>(src + 8 * ch);
                        w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
                    } else {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            w[k] = (uint32_t)src[8 * ch + 2 * k] | ((uint32_t)src[8 * ch + 2 * k + 1] << 16);
                    }
                }
                uint4 o;
                o.x = __byte_perm(w[0], w[2], 0x5410) ^ flip;
                o.y = __byte_perm(w[0], w[2], 0x7632) ^ flip;
                o.z = __byte_perm(w[1], w[3], 0x5410) ^ flip;
                o.w = __byte_perm(w[1], w[3], 0x7632) ^ flip;
                *reinterpret_cast<uint4*>(dst + (ch >> 3) * M::kAtom + (((ch & 7) ^ (r & 7)) << 4)) = o;
            }
            fence_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(q_full);
        }
        if (i < nm) {
            const long long pos = (long long)rq.kv - rq.qn + tok;
            // keys [lo_key, hi_key) of this row
            const int hi_key = live ? (int)max(pos + 1, 0ll) : 0;
            const int lo_key = p.window > 0 && live ? (int)max(pos - p.window + 1, 0ll) : 0;
            int hi_min = live ? hi_key : 0x7fffffff, lo_max = lo_key;
            hi_min = __reduce_min_sync(0xffffffffu, hi_min);
            lo_max = __reduce_max_sync(0xffffffffu, lo_max);
            // scores to powers of two; a tiny factor in the place of 0 keeps masked scores at -inf
            const float f = fmaxf(fabsf(p.scale) * 1.4426950408889634f, 1e-30f) * kUndo<BF>;
            const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
            const uint32_t s_tm = tmem + 128 * i + lanes, o_tm = tmem + 256 + 128 * i + lanes;
            const int pl = p.sh.page_log2;
            const int* table = p.table + (long long)unit_r * p.max_blocks;
            const int npages = (rq.kv + (1 << pl) - 1) >> pl;
            float m = -INFINITY, l = 0.f;
            for (int j = 0; j < n; ++j) {
                const int key0 = (t_first + j) * kKeys;
                // 16-token pieces without a page
                bool gone = false;
                if (lane < 8 && ((key0 + 16 * lane) >> pl) < npages) {
                    const int page = table[(key0 + 16 * lane) >> pl];
                    gone = page < 0 || page >= p.sh.num_blocks;
                }
                const uint32_t holes = __ballot_sync(0xffffffffu, gone);
                const bool masked = holes != 0 || key0 + kKeys > hi_min || key0 < lo_max;
                const int hi = hi_key - key0, lo_ = lo_key - key0;
                auto hide = [&](int c, float s) {
                    return c >= hi || c < lo_ || ((holes >> (c >> 4)) & 1u) ? -INFINITY : s;
                };
                (void)warp_wait(&s_full[i], j & 1, ctl);
                fence_after();
                float mx = -INFINITY;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t v[32];
                    tmem_ld32(s_tm + 32 * c, v);
                    tmem_ld_wait();
                    if (masked) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(hide(32 * c + e, __uint_as_float(v[e])));
                    }
#pragma unroll
                    for (int e = 0; e < 32; e += 2)
                        mx = fmaxf(mx, fmaxf(__uint_as_float(v[e]), __uint_as_float(v[e + 1])));
                }
                mx *= f;
                if (__any_sync(0xffffffffu, mx > m + 8.f || (m == -INFINITY && mx > m))) {
                    const float mn = fmaxf(m, mx);
                    const float a = m == -INFINITY ? 0.f : ex2(m - mn);
                    if (j > 0) {
#pragma unroll
                        for (int c = 0; c < D / 32; ++c) {
                            uint32_t v[32];
                            tmem_ld32(o_tm + 32 * c, v);
                            tmem_ld_wait();
#pragma unroll
                            for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * a);
                            tmem_st32(o_tm + 32 * c, v);
                        }
                    }
                    l *= a;
                    m = mn;
                }
                const float shift = m == -INFINITY ? 0.f : -m;
                float l0 = 0.f, l1 = 0.f;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t v[32], o[16];
                    tmem_ld32(s_tm + 32 * c, v);
                    tmem_ld_wait();
                    if (masked) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(hide(32 * c + e, __uint_as_float(v[e])));
                    }
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        const float a = ex2(fmaf(__uint_as_float(v[e]), f, shift));
                        const float b = ex2(fmaf(__uint_as_float(v[e + 1]), f, shift));
                        l0 += a;
                        l1 += b;
                        o[e / 2] = pack2<BF>(a, b);
                    }
                    tmem_st16(s_tm + 16 * c, o);
                }
                l += l0 + l1;
                tmem_st_wait();
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[i]);
            }
            // ---- output
            (void)warp_wait(o_full, 0, ctl);
            fence_after();
            const float inv = l > 0.f ? kUndo<BF> / l : 0.f;
            uint16_t* dst = static_cast<uint16_t*>(p.out) + (long long)(rq.q0 + tok) * p.out_stride + (long long)head * D;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                uint32_t v[32];
                if (n > 0) {
                    tmem_ld32(o_tm + 32 * c, v);
                    tmem_ld_wait();
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    uint16_t y[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        // channels lie in the order 0 4 1 5 2 6 3 7
                        const float x = l == 0.f ? 0.f : __uint_as_float(v[8 * k + e]) * inv;
                        y[(e >> 1) + 4 * (e & 1)] = T::from_f32(x);
                    }
                    if (live) {
                        uint16_t* d = dst + 32 * c + 8 * k;
                        if (vec_out)
                            *reinterpret_cast<uint4*>(d) =
                                make_uint4(y[0] | ((uint32_t)y[1] << 16), y[2] | ((uint32_t)y[3] << 16),
                                           y[4] | ((uint32_t)y[5] << 16), y[6] | ((uint32_t)y[7] << 16));
                        else
#pragma unroll
                            for (int e = 0; e < 8; ++e) d[e] = y[e];
                    }
                }
            }
            if (live && p.lse)
                p.lse[(long long)(rq.q0 + tok) * (p.sh.hkv * p.group) + head] =
                    l == 0.f ? -INFINITY : fmaf(m, 0.6931471805599453f, logf(l));
        }
    }
    fence_before();
    __syncthreads();
    fence_after();
    if (warp == 12)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
}

template <bool BF, int D>
cudaError_t launch(const KvAttnLaunch& L, int min_rows, cudaStream_t s) {
    const int vec_q = ((uintptr_t)L.q & 15) == 0 && L.q_stride % 8 == 0;
    const int vec_out = ((uintptr_t)L.out & 15) == 0 && L.out_stride % 8 == 0;
    const size_t smem = Smem<D>::total + 1024;
    static bool allowed[64];
    const cudaError_t e = allow_smem_once(kv_attention_tc_kernel<BF, D>, smem, allowed);
    if (e != cudaSuccess) return e;
    // at most: every request leaves a partly filled block
    const int64_t rows = L.num_tokens * L.group;
    const int64_t partly = L.batch < rows / min_rows + 1 ? L.batch : rows / min_rows + 1;
    const int64_t units = (rows / kRows + partly) * L.sh.hkv;
    if (units > 0x7fffffff) return cudaErrorInvalidValue;
    int lg = 5;
    while ((1 << lg) < L.sh.gs) ++lg;
    return launch_pdl(kv_attention_tc_kernel<BF, D>, dim3((unsigned)units), dim3(kThreads), smem, s, L, lg, min_rows,
                      vec_q, vec_out);
}

}  // namespace kvt

cudaError_t launch_kv_attention_tc(const KvAttnLaunch& L, int min_rows, cudaStream_t s) {
    const bool bf = L.sh.dtype == GAI4_BF16;
    if (L.sh.d == 64) return bf ? kvt::launch<true, 64>(L, min_rows, s) : kvt::launch<false, 64>(L, min_rows, s);
    return bf ? kvt::launch<true, 128>(L, min_rows, s) : kvt::launch<false, 128>(L, min_rows, s);
}

}  // namespace gai4
