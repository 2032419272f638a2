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
// Work split: a unit is (request, block of 256 rows, key/value head); all
// units lie on one line, each with places in proportion to its key tiles (and
// kStart more for its queries and output), and the line is cut evenly over
// one CTA per SM. So prompts of any shape, causal blocks of any length and
// one row over a long cache alike keep every SM busy to the end. A unit that
// is cut leaves (m, l, O) records in the workspace, which a second kernel
// joins in order.
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
// 8 softmax warps, 4 expanding, 1 product issuer, 1 producer, 2 idle (warpgroups
// share a register count)
constexpr int kThreads = 32 * 16;
// registers of a thread: launched with 128 (512 x 128 = 65536); softmax, which
// holds a row's 128 scores, then takes what the others leave:
// 256 x 184 + 128 x 96 + 128 x 40 = 64512
constexpr int kSoftmaxRegs = 184, kExpandRegs = 96, kIssueRegs = 40;
constexpr int kRing = 3;              // packed stages (keys and values in turn)
constexpr int kStart = 8;             // what the start and end of a unit cost, in key tiles
constexpr int kPart = 16;             // places of a key tile

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
__device__ __forceinline__ void tmem_st16(uint32_t a, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16};" ::"r"(a),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t a, uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
        "[%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(a)
        : "memory");
}
// bits 0..n - 1
__device__ __forceinline__ uint32_t below(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; }
__device__ __forceinline__ void tmem_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float y;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}
// two binary32 operations at once
__device__ __forceinline__ float2 fma2f(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n .reg .b64 a, b, c, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mov.b64 c, {%6, %7};\n"
        " fma.rn.f32x2 d, a, b, c;\n mov.b64 {%0, %1}, d;\n}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 add2f(float2 a, float2 b) {
    float2 d;
    asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n add.rn.f32x2 d, a, b;\n"
        " mov.b64 {%0, %1}, d;\n}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
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

// records of cut units: per CTA two of (O [D / 4][256] float4, m [256],
// l [256]), number 0 for the end (or a middle) of a unit, 1 for its beginning,
// and two int4: {request or -1, unit, last CTA, 0} of record 1, {request or
// -1, unit, 0, 0} of record 0
__host__ __device__ constexpr size_t rec_floats(int d) { return (size_t)kRows * (d + 2); }
__host__ __device__ constexpr size_t meta_bytes(int ctas) { return ((size_t)ctas * 32 + 255) / 256 * 256; }

struct Req {
    int q0, qn, kv;
    int nblk;               // blocks of 256 rows
    int places, more;       // places of the units of block 0, and how many more each later block's have
};
__device__ __forceinline__ Req request(const KvAttnLaunch& p, int r) {
    Req q;
    const int n = (int)p.num_tokens;
    q.q0 = min(max(p.cu_q[r], 0), n);
    q.qn = max(min(p.cu_q[r + 1], n) - q.q0, 0);
    q.kv = (int)min((long long)max(p.kv_lens[r], 0), (long long)p.max_blocks << p.sh.page_log2);
    q.nblk = (int)(((long long)q.qn * p.group + kRows - 1) / kRows);
    const int toks = min(kRows / p.group + 1, q.qn);
    const long long keys = p.window > 0 ? min((long long)q.kv, (long long)p.window) + toks : max(q.kv - q.qn, 0) + toks;
    q.places = kPart * (kStart + (int)((keys + kKeys - 1) / kKeys));
    q.more = p.window > 0 ? 0 : kPart * kRows / kKeys / p.group;
    return q;
}
// places of the units of blocks 0..b - 1 for one head
__device__ __forceinline__ long long places_before(const Req& q, long long b) { return b * q.places + q.more * (b * (b - 1) / 2); }

// A warp's walk along the line, kept in shared memory (every lane writes the
// same): it is needed between segments only, and the softmax warps have no
// registers to spare for it.
struct Walk {
    long long c, c1;
    int r, blk, h;
    long long place, places;      // within the unit, of the unit
    Req q;
    int row0, rows, t_first, n;   // first row, the request's rows, first key tile, key tiles (at least 1)

    __device__ void init(const KvAttnLaunch& p, int r0, long long off, long long c0, long long c1_) {
        c = c0;
        c1 = c1_;
        r = r0;
        q = request(p, r);
        int lo = 0, hi = q.nblk;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (places_before(q, mid) * p.sh.hkv <= off) lo = mid;
            else hi = mid;
        }
        blk = lo;
        off -= places_before(q, blk) * p.sh.hkv;
        places = q.places + (long long)q.more * blk;
        h = (int)(off / places);
        place = off - h * places;
        unit(p);
    }
    __device__ void unit(const KvAttnLaunch& p) {
        places = q.places + (long long)q.more * blk;
        rows = (int)min((long long)q.qn * p.group, 0x7fffffffll);
        row0 = blk * kRows;
        const long long pos0 = (long long)q.kv - q.qn;
        const long long pos_a = pos0 + row0 / p.group, pos_b = pos0 + (min(row0 + (kRows - 1), rows - 1)) / p.group;
        const long long lo = p.window > 0 ? max(pos_a - p.window + 1, 0ll) : 0;
        t_first = (int)(lo / kKeys);
        n = max((int)((max(pos_b + 1, 0ll) + kKeys - 1) / kKeys) - t_first, 1);
    }
    __device__ bool more() const { return c < c1; }
    __device__ long long here() const { return min(places - place, c1 - c); }
    // tiles of this segment
    __device__ int first() const { return (int)(place * n / places); }
    __device__ int last() const { return (int)((place + here()) * n / places); }
    __device__ void advance(const KvAttnLaunch& p) {
        __syncwarp();   // every lane has read what it needs
        Walk w = *this;
        w.step(p);
        __syncwarp();
        *this = w;
        __syncwarp();
    }
    __device__ void step(const KvAttnLaunch& p) {
        const long long k = here();
        c += k;
        place += k;
        if (place < places || c >= c1) return;
        place = 0;
        if (++h == p.sh.hkv) {
            h = 0;
            if (++blk == q.nblk) {
                blk = 0;
                do q = request(p, ++r);
                while (q.nblk == 0);
            }
        }
        unit(p);
    }
    // number of M tiles with rows
    __device__ int tiles_m() const { return rows - row0 > 128 ? 2 : 1; }
};

// eight channels of an output row, in the order 0 4 1 5 2 6 3 7, rounded once
template <typename T>
__device__ __forceinline__ void store8(uint16_t* d, const float (&y)[8], int vec) {
    uint16_t z[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) z[(e >> 1) + 4 * (e & 1)] = T::from_f32(y[e]);
    if (vec) {
        *reinterpret_cast<uint4*>(d) = make_uint4(z[0] | ((uint32_t)z[1] << 16), z[2] | ((uint32_t)z[3] << 16),
                                                  z[4] | ((uint32_t)z[5] << 16), z[6] | ((uint32_t)z[7] << 16));
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) d[e] = z[e];
    }
}

template <bool BF, int D>
__global__ void __launch_bounds__(kThreads, 1)
    kv_attention_tc_kernel(const __grid_constant__ KvAttnLaunch p, const int gs_log2, const int vec_q, const int vec_out) {
    using T = typename std::conditional<BF, BF16, F16>::type;
    using M = Smem<D>;
    extern __shared__ uint8_t raw[];
    __shared__ long long warp_cost[kThreads / 32], start_off;
    __shared__ int start_r, abort_flag;
    __shared__ uint32_t tmem_slot;
    uint8_t* smem = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + M::bars);
    uint64_t *ring_full = bars, *ring_empty = bars + kRing, *k_full = bars + 2 * kRing, *k_empty = k_full + 2,
             *v_full = k_full + 4, *v_empty = k_full + 6, *s_full = k_full + 8, *p_full = k_full + 10,
             *q_full = k_full + 14, *o_full = k_full + 15, *fin = k_full + 16;
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
            mbar_init(&p_full[2 * i], 4);       // probabilities of the first 64 keys
            mbar_init(&p_full[2 * i + 1], 4);   // and of the others
        }
        mbar_init(q_full, 8);
        mbar_init(o_full, 1);
        mbar_init(fin, 1);
        abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_async();
    }
    pdl_wait();

    // the line: its length, and where this CTA's part begins. Each thread sums
    // a strip of requests.
    const int per_thread = (p.batch + kThreads - 1) / kThreads;
    const int r0 = min(tid * per_thread, p.batch), r1 = min(r0 + per_thread, p.batch);
    auto cost = [&](int r) {
        const Req q = request(p, r);
        return places_before(q, q.nblk) * p.sh.hkv;
    };
    long long mine = 0;
    for (int r = r0; r < r1; ++r) mine += cost(r);
    long long inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += u;
    }
    if (lane == 31) warp_cost[warp] = inc;
    __syncthreads();
    long long total = 0, before = inc - mine;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) {
        if (i < warp) before += warp_cost[i];
        total += warp_cost[i];
    }
    const long long per = max((total + gridDim.x - 1) / gridDim.x, (long long)kPart);
    const long long c0 = min((long long)blockIdx.x * per, total), c1 = min(c0 + per, total);
    if (c0 < c1 && before <= c0 && c0 < before + mine) {
        int r = r0;
        long long at = before;
        for (long long n; at + (n = cost(r)) <= c0; ++r) at += n;
        start_r = r;
        start_off = c0 - at;
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
    uint8_t* ws = static_cast<uint8_t*>(p.workspace);
    int4* meta = reinterpret_cast<int4*>(ws) + 2 * blockIdx.x;
    float* recs = reinterpret_cast<float*>(ws + meta_bytes(gridDim.x)) + blockIdx.x * 2 * rec_floats(D);
    if (tid < 2 && c0 >= c1) meta[tid] = make_int4(-1, 0, 0, 0);
    if (c0 >= c1) return;
    if (warp == 12) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_slot)), "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = tmem_slot;

    __shared__ Walk walks[kThreads / 32];
    Walk& w = walks[warp];
    {
        Walk first;
        first.init(p, start_r, start_off, c0, c1);
        w = first;
        __syncwarp();
    }
    const Ctl ctl{p.status, p.spin_limit, &abort_flag};

    if (warp >= 12) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssueRegs));
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
        uint32_t* masks = reinterpret_cast<uint32_t*>(smem + M::masks);
        int issued = 0;
        bool ok = true;
        for (; w.more() && ok; w.advance(p)) {
        const int t_a = w.first(), t_b = w.last(), h = w.h;
        const int* table = p.table + (long long)w.r * p.max_blocks;
        const int npages = (w.q.kv + (1 << pl) - 1) >> pl;
        int tok = (w.t_first + t_a) * kKeys + piece * tokens;
        int page = t_a < t_b && active && (tok >> pl) < npages ? table[tok >> pl] : -1;
        for (int t = t_a; t < t_b && ok; ++t) {
            const bool there = active && page >= 0 && page < p.sh.num_blocks;
            const uint32_t votes = __ballot_sync(0xffffffffu, there && which == 0);
            const long long line = there ? (((long long)page * p.sh.hkv + h) << pl) + (tok & ((1 << pl) - 1)) : 0;
            const int left = w.q.kv - (w.t_first + t) * kKeys;
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
        auto pv = [&](int i, int j, int half, bool add) {
#pragma unroll
            for (int k = 0; k < kKeys / 32; ++k) {
                const int kk = k + (kKeys / 32) * half;
                mma_ts(tmem + 256 + 128 * i, tmem + 128 * i + 8 * kk, desc_n(vb + (j & 1) * M::kTile + kk * 2048), id_o,
                       add || k > 0);
            }
        };
        bool ok = true;
        int units = 0, jj = 0;          // segments and tiles so far
        uint32_t np = 0;                // parity of the probabilities of each M tile, one bit each
        for (; w.more() && ok; w.advance(p)) {
            const int n = w.last() - w.first(), nm = w.tiles_m();
            if (n == 0) continue;
            ok = warp_wait(q_full, units & 1, ctl) && warp_wait(&k_full[jj & 1], (jj >> 1) & 1, ctl);
            if (!ok) break;
            fence_after();
            for (int i = 0; i < nm; ++i) qk(i, jj);
            commit(&k_empty[jj & 1]);
            for (int j = 0; ok && j < n; ++j, ++jj) {
                ok = warp_wait(&v_full[jj & 1], (jj >> 1) & 1, ctl);
                for (int i = 0; ok && i < nm; ++i) {
                    for (int half = 0; ok && half < 2; ++half) {
                        ok = warp_wait(&p_full[2 * i + half], (np >> i) & 1u, ctl);
                        if (!ok) break;
                        fence_after();
                        pv(i, jj, half, j > 0 || half > 0);
                    }
                    if (!ok) break;
                    np ^= 1u << i;
                    if (i == nm - 1) commit(&v_empty[jj & 1]);
                    if (j + 1 < n) {
                        if (i == 0) ok = warp_wait(&k_full[(jj + 1) & 1], ((jj + 1) >> 1) & 1, ctl);
                        if (!ok) break;
                        fence_after();
                        qk(i, jj + 1);
                        if (i == nm - 1) commit(&k_empty[(jj + 1) & 1]);
                    }
                }
            }
            commit(o_full);
            ++units;
        }
        // no product may outlive the tensor memory
        commit(fin);
        if (lane == 0) mbar_wait_drain(fin, 0, ctl.limit, ctl.status);
        __syncwarp();
    } else if (warp >= 14) {
    } else if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kExpandRegs));
        // ---------------- expanding keys and values: one token per thread ----------------
        const int r = (warp - 8) * 32 + lane;
        const int ng = D >> gs_log2;
        // 32 channels at a time; neighbouring rows take them in another order
        // (banks). Offsets of the packed words, of the row's scales and of the
        // swizzled 16-byte chunks:
        uint32_t from[D / 32], group[D / 32], to[D / 32], chunk[4];
#pragma unroll
        for (int x = 0; x < D / 32; ++x) {
            const int c = (x + (r >> (D == 128 ? 1 : 2))) & (D / 32 - 1);
            from[x] = r * (D / 2) + c * 16;
            group[x] = kKeys * (D / 2) + 2 * (r * ng + ((32 * c) >> gs_log2));
            to[x] = r * 128 + (c >> 1) * M::kAtom + ((((c & 1) << 2) ^ (r & 4)) << 4);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) chunk[k] = (k ^ (r & 3)) << 4;
        const uint32_t* masks = reinterpret_cast<const uint32_t*>(smem + M::masks);
        int i = 0;                     // keys and values of all tiles in turn
        for (; w.more(); w.advance(p)) {
        for (const int end = i + 2 * (w.last() - w.first()); i < end; ++i) {
            const int s = i % kRing, j = i >> 1;
            uint64_t *full = i & 1 ? &v_full[j & 1] : &k_full[j & 1], *empty = i & 1 ? &v_empty[j & 1] : &k_empty[j & 1];
            uint8_t* dst = smem + (i & 1 ? M::v : M::k) + (j & 1) * M::kTile;
            (void)warp_wait(&ring_full[s], (i / kRing) & 1, ctl);
            (void)warp_wait(empty, ((j >> 1) & 1) ^ 1, ctl);
            const uint8_t* st = smem + M::ring + s * M::kStage;
            const bool valid = (masks[s * 4 + (r >> 5)] >> (r & 31)) & 1u;   // else zeros: the slot may hold anything
#pragma unroll
            for (int x = 0; x < D / 32; ++x) {
                const uint4 w = *reinterpret_cast<const uint4*>(st + from[x]);
                const uint8_t* sc = st + group[x];
                const Group<BF> gr(valid ? *reinterpret_cast<const uint16_t*>(sc) : 0u,
                                   valid ? *reinterpret_cast<const uint16_t*>(sc + kKeys * 2 * ng) : 0u);
                const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) *reinterpret_cast<uint4*>(dst + to[x] + chunk[k]) = expand<BF>(ww[k], gr);
            }
            fence_async();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(full);
                mbar_arrive(&ring_empty[s]);
            }
        }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
        // ---------------- softmax: M tile i, one row per thread ----------------
        const int i = warp >> 2, r = (warp & 3) * 32 + lane;
        int units = 0, ns = 0;         // segments and score tiles so far
        bool has0 = false, has1 = false;
        for (; w.more(); w.advance(p)) {
        const int t_a = w.first(), t_b = w.last();
        if (t_a == t_b) continue;
        const int rq_q0 = w.q.q0, rq_kv = w.q.kv, pos0 = rq_kv - w.q.qn, h = w.h, nm = w.tiles_m();
        const int row = w.row0 + i * 128 + r;
        const bool live = row < w.rows;
        const int tok = live ? row / p.group : 0;
        const int head = h * p.group + (live ? row - tok * p.group : 0);
        // query row into shared memory; a negative scale turns its sign
        {
            const uint16_t* src = static_cast<const uint16_t*>(p.q) + (long long)(rq_q0 + tok) * p.q_stride + (long long)head * D;
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
            const long long pos = (long long)pos0 + tok;
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
            const int* table = p.table + (long long)w.r * p.max_blocks;
            const int npages = (rq_kv + (1 << pl) - 1) >> pl;
            const int t_first = w.t_first;
            float m = -INFINITY, l = 0.f;
            for (int j = t_a; j < t_b; ++j) {
                const int key0 = (t_first + j) * kKeys;
                // 16-token pieces without a page
                bool gone = false;
                if (lane < 8 && ((key0 + 16 * lane) >> pl) < npages) {
                    const int page = table[(key0 + 16 * lane) >> pl];
                    gone = page < 0 || page >= p.sh.num_blocks;
                }
                const uint32_t holes = __ballot_sync(0xffffffffu, gone);
                const bool masked = holes != 0 || key0 + kKeys > hi_min || key0 < lo_max;
                (void)warp_wait(&s_full[i], ns & 1, ctl);
                ++ns;
                fence_after();
                uint32_t v[4][32];
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_ld32(s_tm + 32 * c, v[c]);
                tmem_ld_wait();
                if (masked) {
                    const int hi = hi_key - key0, lo_ = lo_key - key0;
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        // bits of the keys that the row sees
                        uint32_t see = below(hi - 32 * c) & ~below(lo_ - 32 * c);
                        if ((holes >> (2 * c)) & 1u) see &= 0xffff0000u;
                        if ((holes >> (2 * c + 1)) & 1u) see &= 0x0000ffffu;
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (!(see & (1u << e))) v[c][e] = 0xff800000u;   // -inf
                    }
                }
                float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int e = 0; e < 32; e += 2)
                        mx4[(e >> 1) & 3] = max3(mx4[(e >> 1) & 3], __uint_as_float(v[c][e]), __uint_as_float(v[c][e + 1]));
                float mx = max3(mx4[0], mx4[1], fmaxf(mx4[2], mx4[3]));
                mx *= f;
                if (__any_sync(0xffffffffu, mx > m + 8.f || (m == -INFINITY && mx > m))) {
                    const float mn = fmaxf(m, mx);
                    const float a = m == -INFINITY ? 0.f : ex2(m - mn);
                    if (j > t_a) {
#pragma unroll 1
                        for (int c = 0; c < D / 16; ++c) {   // (16 columns: the scores stay in registers)
                            uint32_t y[16];
                            tmem_ld16(o_tm + 16 * c, y);
                            tmem_ld_wait();
#pragma unroll
                            for (int e = 0; e < 16; ++e) y[e] = __float_as_uint(__uint_as_float(y[e]) * a);
                            tmem_st16(o_tm + 16 * c, y);
                        }
                    }
                    l *= a;
                    m = mn;
                }
                const float shift = m == -INFINITY ? 0.f : -m;
                float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                const float2 f2 = make_float2(f, f), shift2 = make_float2(shift, shift);
#pragma unroll
                for (int half = 0; half < 2; ++half) {
#pragma unroll
                    for (int c = 2 * half; c < 2 * half + 2; ++c) {
                        uint32_t o[16];
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            float2 x = fma2f(make_float2(__uint_as_float(v[c][e]), __uint_as_float(v[c][e + 1])), f2, shift2);
                            x.x = ex2(x.x);
                            x.y = ex2(x.y);
                            sum[(e >> 1) & 1] = add2f(sum[(e >> 1) & 1], x);
                            o[e / 2] = pack2<BF>(x.x, x.y);
                        }
                        tmem_st16(s_tm + 16 * c, o);
                    }
                    tmem_st_wait();
                    fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&p_full[2 * i + half]);
                }
                l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
            }
            // ---- output, or a record of it
            (void)warp_wait(o_full, units & 1, ctl);
            fence_after();
            const bool begins = t_a == 0, whole = begins && t_b == w.n;
            const float inv = l > 0.f ? kUndo<BF> / l : 0.f;
            uint16_t* dst = static_cast<uint16_t*>(p.out) + (long long)(rq_q0 + tok) * p.out_stride + (long long)head * D;
            float* rec = recs + (begins ? rec_floats(D) : 0);
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
                uint32_t v[32];
                tmem_ld32(o_tm + 32 * c, v);
                tmem_ld_wait();
                if (whole) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        float y[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) y[e] = l == 0.f ? 0.f : __uint_as_float(v[8 * k + e]) * inv;
                        if (live) store8<T>(dst + 32 * c + 8 * k, y, vec_out);
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        reinterpret_cast<uint4*>(rec)[(8 * c + k) * kRows + i * 128 + r] =
                            make_uint4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
                }
            }
            if (whole) {
                if (live && p.lse)
                    p.lse[(long long)(rq_q0 + tok) * (p.sh.hkv * p.group) + head] =
                        l == 0.f ? -INFINITY : fmaf(m, 0.6931471805599453f, logf(l));
            } else {
                rec[kRows * D + i * 128 + r] = m;
                rec[kRows * (D + 1) + i * 128 + r] = l;
                if (tid == 0) {
                    const int unit = w.blk * p.sh.hkv + h;
                    // record 1 begins a unit that goes on: its last CTA holds the unit's last place
                    meta[begins ? 0 : 1] = make_int4(w.r, unit, (int)((w.c - w.place + w.places - 1) / per), 0);
                }
                (begins ? has1 : has0) = true;
            }
            fence_before();
        } else {
            (void)warp_wait(o_full, units & 1, ctl);
        }
        ++units;
        }
        if (tid == 0) {
            if (!has1) meta[0] = make_int4(-1, 0, 0, 0);
            if (!has0) meta[1] = make_int4(-1, 0, 0, 0);
        }
    }
    fence_before();
    __syncthreads();
    fence_after();
    if (warp == 12)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
}

// joins the records of a cut unit, in the order of the CTAs: block (i, c) 32
// channels of the unit that begins in CTA i and goes on, one row per thread
template <bool BF, int D>
__global__ void __launch_bounds__(kRows)
    kv_combine_tc_kernel(const __grid_constant__ KvAttnLaunch p, const int ctas, const int vec_out) {
    using T = typename std::conditional<BF, BF16, F16>::type;
    pdl_launch_dependents();
    pdl_wait();
    const uint8_t* ws = static_cast<const uint8_t*>(p.workspace);
    const int4* metas = reinterpret_cast<const int4*>(ws);
    const int4 meta = metas[2 * blockIdx.x];
    if (meta.x < 0) return;
    const Req rq = request(p, meta.x);
    const int blk = meta.y / p.sh.hkv, h = meta.y % p.sh.hkv, c = blockIdx.y;
    const long long row = (long long)blk * kRows + threadIdx.x;
    if (row >= (long long)rq.qn * p.group) return;
    const float* recs = reinterpret_cast<const float*>(ws + meta_bytes(ctas));
    float m = -INFINITY, l = 0.f, y[32];
#pragma unroll
    for (int e = 0; e < 32; ++e) y[e] = 0.f;
    for (int i = blockIdx.x; i <= meta.z; ++i) {
        if (i > (int)blockIdx.x) {   // a CTA may hold places of the unit and no tile
            const int4 other = metas[2 * i + 1];
            if (other.x != meta.x || other.y != meta.y) continue;
        }
        const float* rec = recs + ((size_t)i * 2 + (i == (int)blockIdx.x ? 1 : 0)) * rec_floats(D);
        const float mi = rec[kRows * D + threadIdx.x], li = rec[kRows * (D + 1) + threadIdx.x];
        float4 v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = reinterpret_cast<const float4*>(rec)[(8 * c + k) * kRows + threadIdx.x];
        if (mi == -INFINITY) continue;
        const float mn = fmaxf(m, mi);
        const float a = m == -INFINITY ? 0.f : ex2(m - mn), b = ex2(mi - mn);
        m = mn;
        l = l * a + li * b;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            y[4 * k] = y[4 * k] * a + v[k].x * b;
            y[4 * k + 1] = y[4 * k + 1] * a + v[k].y * b;
            y[4 * k + 2] = y[4 * k + 2] * a + v[k].z * b;
            y[4 * k + 3] = y[4 * k + 3] * a + v[k].w * b;
        }
    }
    const int tok = (int)(row / p.group), head = h * p.group + (int)(row - (long long)tok * p.group);
    uint16_t* dst = static_cast<uint16_t*>(p.out) + (long long)(rq.q0 + tok) * p.out_stride + (long long)head * D + 32 * c;
    const float inv = l > 0.f ? kUndo<BF> / l : 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        float z[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) z[e] = l == 0.f ? 0.f : y[8 * k + e] * inv;
        store8<T>(dst + 8 * k, z, vec_out);
    }
    if (p.lse && c == 0)
        p.lse[(long long)(rq.q0 + tok) * (p.sh.hkv * p.group) + head] =
            l == 0.f ? -INFINITY : fmaf(m, 0.6931471805599453f, logf(l));
}

template <bool BF, int D>
cudaError_t launch(const KvAttnLaunch& L, cudaStream_t s) {
    const int vec_q = ((uintptr_t)L.q & 15) == 0 && L.q_stride % 8 == 0;
    const int vec_out = ((uintptr_t)L.out & 15) == 0 && L.out_stride % 8 == 0;
    const size_t smem = Smem<D>::total + 1024;
    static bool allowed[64];
    cudaError_t e = allow_smem_once(kv_attention_tc_kernel<BF, D>, smem, allowed);
    if (e != cudaSuccess) return e;
    int lg = 5;
    while ((1 << lg) < L.sh.gs) ++lg;
    const int ctas = num_sms();
    e = launch_pdl(kv_attention_tc_kernel<BF, D>, dim3(ctas), dim3(kThreads), smem, s, L, lg, vec_q, vec_out);
    if (e != cudaSuccess) return e;
    return launch_pdl(kv_combine_tc_kernel<BF, D>, dim3(ctas, D / 32), dim3(kRows), 0, s, L, ctas, vec_out);
}

}  // namespace kvt

size_t kv_attention_tc_workspace(int d) {
    return kvt::meta_bytes(num_sms()) + (size_t)num_sms() * 2 * kvt::rec_floats(d) * sizeof(float);
}

cudaError_t launch_kv_attention_tc(const KvAttnLaunch& L, cudaStream_t s) {
    const bool bf = L.sh.dtype == GAI4_BF16;
    if (L.sh.d == 64) return bf ? kvt::launch<true, 64>(L, s) : kvt::launch<false, 64>(L, s);
    return bf ? kvt::launch<true, 128>(L, s) : kvt::launch<false, 128>(L, s);
}

}  // namespace gai4
