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
// its weights; probabilities are rounded to T as well, the tensor cores' input.
// These roundings double the error of the output's own (bf16: 0.0033 of the
// outputs' size against 0.0016, f16: 4.4e-4 against 2.1e-4); scores, maxima,
// sums and O are binary32.
//
// Tensor memory: S_0, S_1, O_0, O_1, 128 columns each; P_i overwrites the
// first 64 columns of S_i. Products are issued in the order PV_0 QK_0 PV_1
// QK_1, so the commit of QK_i of a tile also says that PV_i of the tile
// before it has finished: a softmax warp may then rescale O_i, which it does
// only when a row's maximum has grown by more than 2^8 (P and the sum are
// merely larger until then; f16 has room for it, see kAbove).
//
// Codes of a word come out of it as pairs (0, 4), (1, 5), (2, 6), (3, 7); that
// order of the channels is kept in shared memory (queries are stored in it,
// outputs put back from it), which saves a permutation per pair.
// bf16: a code masked out of its word is the subnormal c 2^-133 (or c 2^-129),
// and fma(c 2^-133, s 2^93, b 2^-40) is the value times 2^-40, rounded once;
// the power leaves through f and through the last division. Keys and values
// from 2^-86 to 2^37 keep all their bits.
// f16: codes by the offset of 1024, then fma(c, s, b); keys up to 65504. Value
// groups that reach beyond it are multiplied apart, in binary32.
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
//
// What bounds it: the chain scores - softmax - products of each M tile, of
// which two hide each other only in part (of 3770 cycles a key tile, the
// products take at least 2050, a row's softmax 2500 beside its neighbours), and
// shared memory: Q K^T alone reads its full 128 bytes a cycle. A prompt of 8192 bf16 tokens, 8
// key/value heads of 128, 4 query heads each (550 GFLOP below the diagonal):
// 465 us, 1.2 PFLOP/s (f16 497); when it took 460, without the exponentials 446,
// without the expansion 439, without both 405. Six prompts' chunks of 333 to
// 1500 rows behind up to 7000 tokens: 331 us (f16 355). Tensor pipe 53 % of the
// cycles.
// Slower, and not kept: two warps that issue products (641 us at the time, with
// one 456), eight warps that expand (532), 64-key tiles with the queries in
// tensor memory (536), any further unrolling (the instruction cache), two
// threads a row (579; the expanding warps then wait for issue slots), the first
// probabilities under the last tile's maximum beside the search for the new one
// (468).
#include <math.h>

#include "common.cuh"
#include "internal.h"
#include "pipeline.cuh"

namespace gai4 {
namespace kvt {

using namespace pipe;

constexpr int kKeys = 128;            // tokens of a key tile and of a packed stage
constexpr int kRows = 256;            // query rows of a CTA
// warp 0 issues the products, 1 loads, 2-3 are idle (the four warps of a
// warpgroup share a register count), 4-11 softmax, 12-15 expand.
constexpr int kThreads = 32 * 16;
constexpr int kLoader = 1, kSoftmax = 4, kExpand = 12;
// registers of a thread: launched with 128 (512 x 128 = 65536); softmax, which
// holds a row's 128 scores, then takes what the others leave:
// 256 x 184 + 128 x 88 + 128 x 48 = 64512
constexpr int kSoftmaxRegs = 184, kExpandRegs = 88, kIssueRegs = 48;
constexpr int kRing = 3;              // packed stages, keys and values in turn
constexpr int kBufs = 2;              // expanded key tiles, and value tiles
// What the start and end of a unit cost, in key tiles. With 3, 6 and 9 a prompt
// of 8192 tokens took 537, 458 and 471 us, six chunks 368, 333 and 337.
constexpr int kStart = 6;
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

// Products of one tile, issued by a converged warp: one lane is elected for
// all of them, as the issuing warp's instructions are on the critical path.
// Operands step through shared memory by offsets (in 16 bytes) of their
// descriptors, P through tensor memory 8 columns (16 elements) at a time.
#define KVT_OPEN                                                                                                  \
    "{\n .reg .pred e, z, o;\n .reg .b32 r, t, u;\n .reg .b64 x, y;\n elect.sync r|e, 0xffffffff;\n"              \
    " setp.ne.b32 z, %5, 0;\n setp.eq.b32 o, 0, 0;\n"
#define KVT_SS(k, acc)                                                                                            \
    " add.u32 u, %1, " #k ";\n mov.b64 x, {u, %4};\n add.u32 t, %2, " #k ";\n mov.b64 y, {t, %4};\n"             \
    " @e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, " #acc ";\n"
#define KVT_TS(a, b, acc)                                                                                         \
    " add.u32 u, %1, " #a ";\n add.u32 t, %2, " #b ";\n mov.b64 y, {t, %4};\n"                                   \
    " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [u], y, %3, " #acc ";\n"
#define KVT_COMMIT " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%6];\n"
// S = Q K^T: both K-major, 64 or 128 channels (4 or 8 steps); then the commit
template <int D>
__device__ __forceinline__ void products_qk(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t id, uint64_t* bar) {
    if constexpr (D == 64)
        asm volatile(KVT_OPEN KVT_SS(0, z) KVT_SS(2, o) KVT_SS(4, o) KVT_SS(6, o) KVT_COMMIT "}" ::"r"(d), "r"(a_lo),
                     "r"(b_lo), "r"(id), "r"(kDescHi), "r"(0), "r"(smem_u32(bar))
                     : "memory");
    else
        asm volatile(KVT_OPEN KVT_SS(0, z) KVT_SS(2, o) KVT_SS(4, o) KVT_SS(6, o) KVT_SS(1024, o) KVT_SS(1026, o)
                         KVT_SS(1028, o) KVT_SS(1030, o) KVT_COMMIT "}" ::"r"(d),
                     "r"(a_lo), "r"(b_lo), "r"(id), "r"(kDescHi), "r"(0), "r"(smem_u32(bar))
                     : "memory");
}
// O += P V over 64 keys (4 steps); V is N-major
__device__ __forceinline__ void products_pv(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t id, uint32_t acc) {
    asm volatile(KVT_OPEN KVT_TS(0, 0, z) KVT_TS(8, 128, o) KVT_TS(16, 256, o) KVT_TS(24, 384, o) "}" ::"r"(d), "r"(a),
                 "r"(b_lo), "r"(id), "r"(kDescHi), "r"(acc)
                 : "memory");
}
#undef KVT_OPEN
#undef KVT_SS
#undef KVT_TS
#undef KVT_COMMIT
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
__device__ __forceinline__ void tmem_ld8(uint32_t a, uint32_t (&v)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                 : "r"(a)
                 : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t a, const uint32_t (&v)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(a), "r"(v[0]),
                 "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
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

// Probabilities are taken relative to 2^-kAbove of a row's largest, so that
// binary16 holds them from 2^15 (the maximum may lag by 2^8) down: all 11 bits to
// 2^-21 of the largest, and multiples of 2^-31 of it below. Without it, many keys
// beside one that takes nearly all were a sixth off at 1.4e-7 each.
template <bool BF>
constexpr float kAbove = BF ? 0.f : 7.f;

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

// Values of a group that cannot be expanded: scale or bias is not finite (bf16:
// or the scale is 2^35 or more). A sign bit of one of the result's halves says
// so, the scale's in the lower one.
template <bool BF>
__device__ __forceinline__ uint32_t too_wide(uint32_t s, uint32_t b) {
    return ((s | b << 16) & 0x7fff7fffu) + (BF ? 0x00802F00u : 0x04000400u);
}
// f16: groups whose values cannot all be expanded, two of them, a sign bit for
// each in its half: those, and finite ones whose last code, 15 s + b, is rounded
// to infinity (the others lie between that and b).
__device__ __forceinline__ uint32_t too_large(uint32_t s0, uint32_t b0, uint32_t s1, uint32_t b1) {
    return (fma2<false>(s0 | s1 << 16, 0x4B804B80u, b0 | b1 << 16) & 0x7fff7fffu) + 0x04000400u;
}

// columns of tensor memory (128 for each M tile)
constexpr uint32_t kS = 0, kO = 256;

template <int D>
struct Smem {
    static constexpr uint32_t kAtom = 128 * 128;                        // 128 rows x 64 channels
    static constexpr uint32_t kTile = (D / 64) * kAtom;                 // one tile of queries, keys or values
    static constexpr uint32_t kMaxNG = D / 32;
    static constexpr uint32_t kStage = kKeys * (D / 2 + 4 * kMaxNG);    // codes, scales, biases
    static constexpr uint32_t q = 0, k = 2 * kTile, v = k + kBufs * kTile, ring = v + kBufs * kTile,
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
    int places, more;       // places of the units of block 0, and how many more each later block's have (rounded
                            // down: 0 above 32 query heads, where later blocks count too little)
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
    // tiles of this segment: kStart tiles' places come before the first
    // tile's (places are only an estimate: the last place ends the last tile)
    __device__ int tile_at(long long x) const {
        return x >= places ? n : min(max((int)(x / kPart) - kStart, 0), n);
    }
    __device__ int first() const { return tile_at(place); }
    __device__ int last() const { return tile_at(place + here()); }
    __device__ void advance(const KvAttnLaunch& p) { advance_to(p, *this); }
    __device__ void advance_to(const KvAttnLaunch& p, Walk& to) const {
        __syncwarp();   // every lane has read what it needs
        Walk w = *this;
        w.step(p);
        __syncwarp();
        to = w;
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

// 16-token pieces of keys [a, b) (a multiple of 128) that have no page: bit n
// of the result for piece n, n modulo 32; called by a whole warp
__device__ __forceinline__ uint32_t holes(const KvAttnLaunch& p, const Walk& w, int a, int b, int lane) {
    const int pl = p.sh.page_log2;
    const int* table = p.table + (long long)w.r * p.max_blocks;
    const int end = min(b, w.q.kv);
    bool gone = false;
    for (int key = a + 16 * lane; key < end; key += 512) {
        const int page = table[key >> pl];
        gone |= page < 0 || page >= p.sh.num_blocks;
    }
    return __ballot_sync(0xffffffffu, gone);
}

// eight channels of an output row, given in the order 0 4 1 5 2 6 3 7, rounded once
template <typename T>
__device__ __forceinline__ uint4 round8(const float (&y)[8]) {
    uint32_t z[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) z[(e >> 1) + 4 * (e & 1)] = T::from_f32(y[e]);
    return make_uint4(z[0] | (z[1] << 16), z[2] | (z[3] << 16), z[4] | (z[5] << 16), z[6] | (z[7] << 16));
}
__device__ __forceinline__ void put8(uint16_t* d, uint4 y, int vec) {
    if (vec) {
        *reinterpret_cast<uint4*>(d) = y;
    } else {
        const uint32_t w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) d[e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
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
    __shared__ volatile int wide_values;   // some value tile had groups that were set apart (see below)
    __shared__ uint32_t tmem_slot;
    uint8_t* smem = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + M::bars);
    // (two of most: keys / values, M tiles, buffers)
    // (done[t % kBufs]: the products QK of tile t have finished, and with them PV of tile t - 1; v_free[t % kBufs]: PV of
    // tile t, which comes before QK of the second M tile's next scores)
    uint64_t *ring_full = bars, *ring_empty = bars + kRing, *k_full = bars + 2 * kRing, *v_full = k_full + kBufs,
             *done = v_full + kBufs, *s_full = done + kBufs, *p_full = s_full + 2, *q_full = s_full + 6, *o_full = s_full + 7,
             *fin = s_full + 8, *v_free = s_full + 9;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    pdl_launch_dependents();
    if (tid == 0) {
        for (int i = 0; i < kRing; ++i) {
            mbar_init(&ring_full[i], 1);
            mbar_init(&ring_empty[i], 4);
        }
        for (int i = 0; i < kBufs; ++i) {
            mbar_init(&k_full[i], 4);
            mbar_init(&v_full[i], 4);
            mbar_init(&done[i], 1);
            mbar_init(&v_free[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[2 * i], 4);       // probabilities of the first 64 keys
            mbar_init(&p_full[2 * i + 1], 4);   // and of the others
        }
        mbar_init(q_full, 8);
        mbar_init(o_full, 1);
        mbar_init(fin, 1);
        abort_flag = 0;
        wide_values = 0;
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
    if (warp == 0 && c0 < c1) {
        __syncwarp();
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_slot)), "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
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
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = tmem_slot;

    __shared__ Walk walks[kThreads / 32 + 8];   // (two for each softmax warp)
    Walk& w = walks[warp];
    {
        Walk first;
        first.init(p, start_r, start_off, c0, c1);
        w = first;
        __syncwarp();
    }
    const Ctl ctl{p.status, p.spin_limit, &abort_flag};

    if (warp < kSoftmax) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssueRegs));
    if (warp == kLoader) {
        // ---------------- loader: packed keys and values of each tile in turn ----------------
        // lane: page of the tile, and one of three arrays
        const int pl = p.sh.page_log2;
        const int pieces = pl >= 7 ? 1 : kKeys >> pl, tokens = pl >= 7 ? kKeys : 1 << pl;
        const int piece = lane / 3, array = lane - 3 * piece;    // codes, scales, biases
        const bool active = piece < pieces;
        const int ng = D >> gs_log2;
        const uint32_t row_bytes = array == 0 ? D / 2 : 2 * ng;
        const uint32_t bytes = tokens * row_bytes;
        const uint32_t dst0 = smem_u32(smem + M::ring) +
                              (array == 0 ? 0u : kKeys * (D / 2) + (array - 1) * kKeys * 2 * ng) + piece * bytes;
        auto source = [&](const KvCache& c) {
            return static_cast<const uint8_t*>(array == 0 ? static_cast<const void*>(c.packed) : array == 1 ? c.scales : c.biases);
        };
        const uint8_t* const src_k = source(p.k);
        const uint8_t* const src_v = source(p.v);
        uint32_t* masks = reinterpret_cast<uint32_t*>(smem + M::masks);
        int issued = 0, s = 0;
        uint32_t parity = 1;
        bool ok = true;
        for (; w.more() && ok; w.advance(p)) {
            const int h = w.h, kv_len = w.q.kv;
            const int* table = p.table + (long long)w.r * p.max_blocks;
            const int npages = (kv_len + (1 << pl) - 1) >> pl;
            int key = (w.t_first + w.first()) * kKeys;           // first token of the tile
            const int end = (w.t_first + w.last()) * kKeys;
            int at = (key + piece * tokens) >> pl;
            int page = key < end && active && at < npages ? table[at] : -1;
            for (; key < end && ok; key += kKeys) {
                const bool there = active && page >= 0 && page < p.sh.num_blocks;
                const uint32_t votes = __ballot_sync(0xffffffffu, there && array == 0);
                const long long line =
                    there ? (((long long)page * p.sh.hkv + h) << pl) + ((key + piece * tokens) & ((1 << pl) - 1)) : 0;
                at = (key + kKeys + piece * tokens) >> pl;
                page = active && at < npages ? table[at] : -1;   // of the next tile
                // bits of the tokens that are there, 32 for each of lanes 0 to 3
                uint32_t m = 0;
#pragma unroll
                for (int b = 0; b < 32; b += 16)
                    if ((votes >> (3 * (((lane & 3) * 32 + b) / tokens))) & 1u) m |= 0xffffu << b;
                m &= below(kv_len - key - (lane & 3) * 32);
#pragma unroll
                for (int side = 0; side < 2; ++side) {
                    ok = warp_wait(&ring_empty[s], parity, ctl);
                    if (!ok) break;
                    if (lane < 4) masks[s * 4 + lane] = m;
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive_expect_tx(&ring_full[s], (uint32_t)__popc(votes) * tokens * (D / 2 + 4 * ng));
                    __syncwarp();
                    if (there)
                        asm volatile(
                            "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                                dst0 + s * M::kStage),
                            "l"((side ? src_v : src_k) + line * row_bytes), "r"(bytes), "r"(smem_u32(&ring_full[s]))
                            : "memory");
                    ++issued;
                    if (++s == kRing) {
                        s = 0;
                        parity ^= 1u;
                    }
                }
            }
        }
        for (int i = issued > kRing ? issued - kRing : 0; i < issued; ++i)
            mbar_wait_drain(&ring_full[i % kRing], (i / kRing) & 1, ctl.limit, ctl.status);
    } else if (warp == 0) {
        // ---------------- products ----------------
        constexpr uint32_t id_s = idesc(BF, kKeys, false), id_o = idesc(BF, D, true);
        // (addresses below 2^18: offsets do not carry out of their field)
        const uint32_t q0 = desc_k(smem_u32(smem + M::q)), k0 = desc_k(smem_u32(smem + M::k)),
                       v0 = desc_n(smem_u32(smem + M::v));
        // key tile j and value tile j are in buffer j % kBufs
        auto qk = [&](int i, int buf) {
            products_qk<D>(tmem + kS + 128 * i, q0 + i * (M::kTile >> 4), k0 + buf * (M::kTile >> 4), id_s, &s_full[i]);
        };
        auto pv = [&](int i, int buf, int half, bool add) {
            products_pv(tmem + kO + 128 * i, tmem + kS + 128 * i + 32 * half, v0 + buf * (M::kTile >> 4) + 512 * half, id_o, add);
        };
        // a wait without the vote of warp_wait: the lanes leave the loop
        // together as a rule, and meet again before the next product
        bool ok = true;
        auto wait = [&](uint64_t* bar, uint32_t parity) {
            if (!mbar_try_wait(bar, parity) && !mbar_wait(bar, parity, ctl)) ok = false;
            __syncwarp();
        };
        int units = 0, buf = 0;         // segments so far, buffer of the tile in work
        uint32_t parity = 0;            // of that buffer's barriers
        uint32_t np0 = 0, np1 = 0;      // of the probabilities of each M tile
        for (; w.more(); w.advance(p)) {
            const int n = w.last() - w.first();
            const bool both = w.tiles_m() == 2;
            if (n == 0) continue;
            wait(q_full, units & 1);
            wait(&k_full[buf], parity);
            fence_after();
            qk(0, buf);
            if (both) qk(1, buf);
            commit(&done[buf]);
            for (int j = 0; j < n; ++j) {
                const bool more = j + 1 < n;
                const int next = buf + 1 == kBufs ? 0 : buf + 1;
                const uint32_t next_parity = next == 0 ? parity ^ 1u : parity;
                // (keys and values are there before the probabilities as a rule)
                wait(&v_full[buf], parity);
                if (more) wait(&k_full[next], next_parity);
                wait(&p_full[0], np0);
                if (__any_sync(0xffffffffu, !ok)) break;   // a wait timed out
                fence_after();
                pv(0, buf, 0, j > 0);
                wait(&p_full[1], np0);
                np0 ^= 1u;
                fence_after();
                pv(0, buf, 1, true);
                if (!both) commit(&v_free[buf]);
                if (more) qk(0, next);
                if (both) {
                    wait(&p_full[2], np1);
                    fence_after();
                    pv(1, buf, 0, j > 0);
                    wait(&p_full[3], np1);
                    np1 ^= 1u;
                    fence_after();
                    pv(1, buf, 1, true);
                    commit(&v_free[buf]);
                    if (more) qk(1, next);
                }
                if (more) commit(&done[next]);
                buf = next;
                parity = next_parity;
            }
            commit(o_full);
            if (__any_sync(0xffffffffu, !ok)) break;
            ++units;
        }
        // no product may outlive the tensor memory
        commit(fin);
        if (lane == 0) mbar_wait_drain(fin, 0, ctl.limit, ctl.status);
        __syncwarp();
    } else if (warp < kSoftmax) {
    } else if (warp >= kExpand) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kExpandRegs));
        // ---------------- expanding keys and values: one token per thread ----------------
        const int r = (warp - kExpand) * 32 + lane;
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
        const uint32_t* masks = reinterpret_cast<const uint32_t*>(smem + M::masks) + (r >> 5);
        int j = 0, s = 0;              // tiles so far, packed stage
        uint32_t parity = 0;           // of that stage
        for (; w.more(); w.advance(p)) {
            for (const int end = j + (w.last() - w.first()); j < end; ++j) {
                const int buf = j & 1;
#pragma unroll 1
                for (int side = 0; side < 2; ++side) {      // keys, values
                    uint8_t* dst = smem + (side ? M::v : M::k) + buf * M::kTile;
                    (void)warp_wait(&ring_full[s], parity, ctl);
                    const uint8_t* st = smem + M::ring + s * M::kStage;
                    const bool valid = (masks[4 * s] >> (r & 31)) & 1u;   // else zeros: the slot may hold anything
                    uint4 y[D / 32];
                    uint32_t scale[D / 32], bias[D / 32];
#pragma unroll
                    for (int x = 0; x < D / 32; ++x) {   // (all loads before the first store: they may not pass one)
                        y[x] = *reinterpret_cast<const uint4*>(st + from[x]);
                        const uint8_t* sc = st + group[x];
                        scale[x] = valid ? *reinterpret_cast<const uint16_t*>(sc) : 0u;
                        bias[x] = valid ? *reinterpret_cast<const uint16_t*>(sc + kKeys * 2 * ng) : 0u;
                    }
                    // Values that are not finite once expanded would reach the rows that do not see their token, as
                    // 0 x NaN: zeros in their place, and the softmax warps add to the outputs that need it what was
                    // left out. (f16: the exact test for values only, 497 us for the prompt; for keys as well 504, with
                    // the values saturated here instead 516.)
                    uint32_t wide = 0;
                    if constexpr (BF) {
#pragma unroll
                        for (int x = 0; x < D / 32; ++x) wide |= too_wide<BF>(scale[x], bias[x]);
                        if (side && (wide & 0x80008000u)) {
#pragma unroll
                            for (int x = 0; x < D / 32; ++x)
                                if (too_wide<BF>(scale[x], bias[x]) & 0x80008000u) scale[x] = bias[x] = 0;
                            wide_values = 1;
                        }
                    } else {
                        if (side) {
#pragma unroll
                            for (int x = 0; x < D / 32; x += 2) wide |= too_large(scale[x], bias[x], scale[x + 1], bias[x + 1]);
                            if (wide & 0x80008000u) {
#pragma unroll
                                for (int x = 0; x < D / 32; ++x)
                                    if (too_large(scale[x], bias[x], 0u, 0u) & 0x8000u) scale[x] = bias[x] = 0;
                                wide_values = 1;
                            }
                        }
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&ring_empty[s]);
                    // the buffer's last tile
                    const int t = j - kBufs;
                    if (t >= 0) (void)warp_wait(side ? &v_free[buf] : &done[buf], (t >> 1) & 1, ctl);
#pragma unroll
                    for (int x = 0; x < D / 32; ++x) {
                        const Group<BF> gr(scale[x], bias[x]);
                        const uint32_t ww[4] = {y[x].x, y[x].y, y[x].z, y[x].w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) *reinterpret_cast<uint4*>(dst + to[x] + chunk[e]) = expand<BF>(ww[e], gr);
                    }
                    fence_async();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(side ? &v_full[buf] : &k_full[buf]);
                    if (++s == kRing) {
                        s = 0;
                        parity ^= 1u;
                    }
                }
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
        // ---------------- softmax: M tile i, one row per thread ----------------
        const int i = (warp - kSoftmax) >> 2, r = (warp & 3) * 32 + lane;
        // Queries come and outputs go a warp at a time, D / 8 lanes to a row
        // (row by thread would touch 32 lines an instruction), the outputs by
        // way of the query tile, which is free by then.
        constexpr int L = D / 8, R = 32 / L;        // lanes of a row, rows at a time
        const int lr = lane / L, lc = lane % L;     // this lane's row and 16-byte chunk
        uint8_t* const qtile = smem + M::q + i * M::kTile;
        auto chunk_at = [&](int row, int ch) { return qtile + (ch >> 3) * M::kAtom + row * 128 + (((ch & 7) ^ (row & 7)) << 4); };
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t s_tm = tmem + kS + 128 * i + lanes, o_tm = tmem + kO + 128 * i + lanes;
        const uint32_t flip = p.scale < 0.f ? 0x80008000u : 0u;   // a negative scale turns the queries' sign
        // f(k, address or null) for this lane's chunk of its row number k, of
        // `rows` [.., heads, D] with a token stride
        auto each_row = [&](const Walk& w, auto* base, long long stride, auto&& f) {
            const int first = w.row0 + i * 128 + (warp & 3) * 32 + lr;
            const int tok = first / p.group;
            int hd = first - tok * p.group, left = w.rows - first;
            auto* at = base + (w.q.q0 + tok) * stride + (w.h * p.group + hd) * D + lc * 8;
            const long long wrap = stride - p.group * D;
#pragma unroll
            for (int k = 0; k < 32 / R; ++k) {
                f(k, left > k * R ? at : nullptr);
                at += R * D;
                hd += R;
#pragma unroll
                for (int e = 0; e < R; ++e)
                    if (hd >= p.group) {
                        hd -= p.group;
                        at += wrap;
                    }
            }
        };
        // this lane's chunk of its row number k in the query tile
        uint8_t* const my_chunk = qtile + (lc >> 3) * M::kAtom + ((warp & 3) * 32 + lr) * 128;
        const uint32_t my_swizzle = ((lc & 7) ^ lr) << 4;
        auto tile_at = [&](int k) {
            return reinterpret_cast<uint4*>(my_chunk + k * R * 128 + (my_swizzle ^ (((k * R) & 7) << 4)));
        };
        auto prefetch_q = [&](const Walk& w) {
            each_row(w, static_cast<const uint16_t*>(p.q), p.q_stride, [&](int, const uint16_t* src) {
                if (src) asm volatile("prefetch.global.L2 [%0];" ::"l"(src));
            });
        };
        auto load_q = [&](const Walk& w) {
            uint4 y[32 / R];
            each_row(w, static_cast<const uint16_t*>(p.q), p.q_stride, [&](int k, const uint16_t* src) {
                y[k] = make_uint4(0u, 0u, 0u, 0u);
                if (src) {
                    if (vec_q) {
                        y[k] = *reinterpret_cast<const uint4*>(src);
                    } else {
                        uint32_t x[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) x[e] = (uint32_t)src[2 * e] | ((uint32_t)src[2 * e + 1] << 16);
                        y[k] = make_uint4(x[0], x[1], x[2], x[3]);
                    }
                }
            });
#pragma unroll
            for (int k = 0; k < 32 / R; ++k) {
                uint4 o;
                o.x = __byte_perm(y[k].x, y[k].z, 0x5410) ^ flip;
                o.y = __byte_perm(y[k].x, y[k].z, 0x7632) ^ flip;
                o.z = __byte_perm(y[k].y, y[k].w, 0x5410) ^ flip;
                o.w = __byte_perm(y[k].y, y[k].w, 0x7632) ^ flip;
                *tile_at(k) = o;
            }
            fence_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(q_full);
        };
        // the segment in work and the next one that has a tile: what is not
        // needed in the loop over the keys stays in shared memory
        Walk* cur = &w;
        Walk* next = &walks[kThreads / 32 + warp - kSoftmax];
        uint32_t s_parity = 0, o_parity = 0;   // of the score tiles and segments so far
        if (tid == 32 * kSoftmax) meta[0] = meta[1] = make_int4(-1, 0, 0, 0);
        while (cur->more() && cur->first() == cur->last()) cur->advance(p);
        bool more = cur->more();
        if (more) load_q(*cur);
        while (more) {
        float m = -INFINITY, l = 0.f;
        if (i < cur->tiles_m()) {
            const int row = cur->row0 + i * 128 + r;
            const bool live = row < cur->rows;
            const long long pos = (long long)cur->q.kv - cur->q.qn + (live ? row / p.group : 0);
            // keys [lo_key, hi_key) of this row
            const int hi_key = live ? (int)max(pos + 1, 0ll) : 0;
            const int lo_key = p.window > 0 && live ? (int)max(pos - p.window + 1, 0ll) : 0;
            int hi_min = live ? hi_key : 0x7fffffff, lo_max = lo_key;
            hi_min = __reduce_min_sync(0xffffffffu, hi_min);
            lo_max = __reduce_max_sync(0xffffffffu, lo_max);
            // scores to powers of two; the least factor in the place of 0 keeps masked scores at -inf
            const float f = fmaxf(fabsf(p.scale) * 1.4426950408889634f * kUndo<BF>, 1.4e-45f);
            const int first_key = (cur->t_first + cur->first()) * kKeys, end_key = (cur->t_first + cur->last()) * kKeys;
            const bool holes_here = holes(p, *cur, first_key, end_key, lane) != 0;
            for (int key0 = first_key; key0 < end_key; key0 += kKeys) {
                const bool masked = holes_here || key0 + kKeys > hi_min || key0 < lo_max;
                (void)warp_wait(&s_full[i], s_parity, ctl);
                s_parity ^= 1u;
                fence_after();
                uint32_t v[kKeys / 32][32];
#pragma unroll
                for (int c = 0; c < kKeys / 32; ++c) tmem_ld32(s_tm + 32 * c, v[c]);
                tmem_ld_wait();
                if (masked) {
                    const int hi = hi_key - key0, lo_ = lo_key - key0;
                    const uint32_t gone = holes_here ? holes(p, *cur, key0, key0 + kKeys, lane) : 0u;
#pragma unroll
                    for (int c = 0; c < kKeys / 32; ++c) {
                        // bits of the keys that the row sees
                        uint32_t see = below(hi - 32 * c) & ~below(lo_ - 32 * c);
                        if ((gone >> (2 * c)) & 1u) see &= 0xffff0000u;
                        if ((gone >> (2 * c + 1)) & 1u) see &= 0x0000ffffu;
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (!(see & (1u << e))) v[c][e] = 0xff800000u;   // -inf
                    }
                }
                float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int c = 0; c < kKeys / 32; ++c)
#pragma unroll
                    for (int e = 0; e < 32; e += 2)
                        mx4[(e >> 1) & 3] = max3(mx4[(e >> 1) & 3], __uint_as_float(v[c][e]), __uint_as_float(v[c][e + 1]));
                float mx = max3(mx4[0], mx4[1], fmaxf(mx4[2], mx4[3]));
                mx *= f;
                if (__any_sync(0xffffffffu, mx > m + (8.f + kAbove<BF>) || (m == -INFINITY && mx > m))) {
                    const float mn = fmaxf(m, mx - kAbove<BF>);
                    const float a = m == -INFINITY ? 0.f : ex2(m - mn);
                    if (key0 > first_key) {
#pragma unroll 1
                        for (int c = 0; c < D / 8; ++c) {   // (8 columns: the scores stay in registers)
                            uint32_t y[8];
                            tmem_ld8(o_tm + 8 * c, y);
                            tmem_ld_wait();
#pragma unroll
                            for (int e = 0; e < 8; ++e) y[e] = __float_as_uint(__uint_as_float(y[e]) * a);
                            tmem_st8(o_tm + 8 * c, y);
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
        }
        cur->advance_to(p, *next);
        while (next->more() && next->first() == next->last()) next->advance(p);
        more = next->more();
        if (more) prefetch_q(*next);   // (held in registers during the output they spill)
        // ---- output, or a record of it
        (void)warp_wait(o_full, o_parity, ctl);
        o_parity ^= 1u;
        fence_after();
        const bool begins = cur->first() == 0, whole = begins && cur->last() == cur->n, mine = i < cur->tiles_m();
        const int row0 = cur->row0, rows = cur->rows, rq_q0 = cur->q.q0, h = cur->h;
        // Values that were set apart (a flag of the CTA, which stays), a token at a time: groups whose channels are NaN
        // in this row, and f16 products that are added to O in binary32, with the score taken once more, as the
        // probability is gone. Rare: only the result counts.
        uint32_t nan_groups = 0;
        if (mine && wide_values) {
            const int row = row0 + i * 128 + r, pl = p.sh.page_log2, ng = D >> gs_log2;
            const bool live = row < rows;
            const int tok = live ? row / p.group : 0;
            const long long pos = live ? (long long)cur->q.kv - cur->q.qn + tok : -1;
            const long long lo = p.window > 0 ? pos - p.window + 1 : 0;
            const int end = min((cur->t_first + cur->last()) * kKeys, cur->q.kv);
            const int* table = p.table + (long long)cur->r * p.max_blocks;
            const uint16_t *vs = static_cast<const uint16_t*>(p.v.scales), *vb = static_cast<const uint16_t*>(p.v.biases);
#pragma unroll 1
            for (int key0 = (cur->t_first + cur->first()) * kKeys; key0 < end; key0 += 32) {
                const int key = key0 + lane, page = key < end ? table[key >> pl] : -1;
                uint32_t groups = 0, large = 0;
                long long line = 0;                 // cache row
                if (page >= 0 && page < p.sh.num_blocks) {
                    line = (((long long)page * p.sh.hkv + h) << pl) + (key & ((1 << pl) - 1));
#pragma unroll 1
                    for (int g = 0; g < ng; ++g) {
                        const uint32_t s = vs[line * ng + g], b = vb[line * ng + g];
                        if (too_wide<BF>(s, b) & 0x80008000u) groups |= 1u << g;
                        else if (!BF && (too_large(s, b, 0u, 0u) & 0x8000u)) large |= 1u << g;
                    }
                }
#pragma unroll 1
                for (uint32_t some = __ballot_sync(0xffffffffu, (groups | large) != 0); some != 0; some &= some - 1) {
                    const int o = __ffs(some) - 1;
                    const uint32_t of = __shfl_sync(0xffffffffu, groups, o);
                    const bool sees = key0 + o >= lo && key0 + o <= pos;
                    if (sees) nan_groups |= of;
                    if constexpr (!BF) {
                        const uint32_t add = __shfl_sync(0xffffffffu, large, o);
                        if (add == 0) continue;
                        const long long at = __shfl_sync(0xffffffffu, line, o);
                        float prob = 0.f;
                        if (sees) {
                            float dot = 0.f;                // (the queries are still in their tile)
#pragma unroll 4
                            for (int c = 0; c < D / 8; ++c) {
                                const long long g = at * ng + ((8 * c) >> gs_log2);
                                const uint4 k = expand<BF>(p.k.packed[at * (D / 8) + c],
                                                           Group<BF>(static_cast<const uint16_t*>(p.k.scales)[g],
                                                                     static_cast<const uint16_t*>(p.k.biases)[g]));
                                const uint4 q = *reinterpret_cast<const uint4*>(chunk_at(r, c));
                                const uint32_t kw[4] = {k.x, k.y, k.z, k.w}, qw[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    dot = fmaf(T::to_f32((uint16_t)qw[e]), T::to_f32((uint16_t)kw[e]), dot);
                                    dot = fmaf(T::to_f32((uint16_t)(qw[e] >> 16)), T::to_f32((uint16_t)(kw[e] >> 16)), dot);
                                }
                            }
                            prob = ex2(fmaf(dot, fabsf(p.scale) * 1.4426950408889634f, m == -INFINITY ? 0.f : -m));
                        }
#pragma unroll 1
                        for (int c = 0; c < D / 8; ++c) {
                            const int g = (8 * c) >> gs_log2;
                            if (!((add >> g) & 1u)) continue;
                            const float s = F16::to_f32(vs[at * ng + g]), b = F16::to_f32(vb[at * ng + g]);
                            const uint32_t w = p.v.packed[at * (D / 8) + c];
                            uint32_t y[8];
                            tmem_ld8(o_tm + 8 * c, y);
                            tmem_ld_wait();
#pragma unroll
                            for (int e = 0; e < 8; ++e) {   // (channels in the order 0 4 1 5 2 6 3 7)
                                const float v = fmaf(s, (float)((w >> (4 * ((e >> 1) + 4 * (e & 1)))) & 15u), b);
                                if (sees) y[e] = __float_as_uint(fmaf(prob, v, __uint_as_float(y[e])));
                            }
                            tmem_st8(o_tm + 8 * c, y);
                            tmem_st_wait();
                        }
                    }
                }
            }
        }
        auto is_nan = [&](int c) { return ((nan_groups >> ((32 * c) >> gs_log2)) & 1u) != 0; };   // channels 32 c on
        if (mine && whole) {
            const float inv = l > 0.f ? kUndo<BF> / l : 0.f;
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
                uint32_t v[32];
                tmem_ld32(o_tm + 32 * c, v);
                tmem_ld_wait();
                if (is_nan(c)) {
#pragma unroll
                    for (int e = 0; e < 32; ++e) v[e] = 0x7fffffffu;
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float y[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[e] = l == 0.f ? 0.f : __uint_as_float(v[8 * k + e]) * inv;
                    *reinterpret_cast<uint4*>(chunk_at(r, 4 * c + k)) = round8<T>(y);
                }
            }
            __syncwarp();
            each_row(*cur, static_cast<uint16_t*>(p.out), p.out_stride, [&](int k, uint16_t* dst) {
                if (dst) put8(dst, *tile_at(k), vec_out);
            });
            __syncwarp();
            const int row = row0 + i * 128 + r;
            if (p.lse && row < rows) {
                const int tok = row / p.group;
                p.lse[(long long)(rq_q0 + tok) * (p.sh.hkv * p.group) + h * p.group + (row - tok * p.group)] =
                    l == 0.f ? -INFINITY : fmaf(m, 0.6931471805599453f, logf(l));
            }
        } else if (!whole) {
            float* rec = recs + (begins ? rec_floats(D) : 0);
            if (mine) {
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t v[32];
                    tmem_ld32(o_tm + 32 * c, v);
                    tmem_ld_wait();
                    if (is_nan(c)) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) v[e] = 0x7fffffffu;
                    }
                    if (row0 + i * 128 + r < rows) {
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            reinterpret_cast<uint4*>(rec)[(8 * c + k) * kRows + i * 128 + r] =
                                make_uint4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
                    }
                }
                rec[kRows * D + i * 128 + r] = m;
                rec[kRows * (D + 1) + i * 128 + r] = l;
            }
            // record 1 begins a unit that goes on
            if (tid == 32 * kSoftmax)
                meta[begins ? 0 : 1] = make_int4(cur->r, cur->blk * p.sh.hkv + h,
                                                 (int)((cur->c - cur->place + cur->places - 1) / per), 0);
        }
        fence_before();
        if (more) load_q(*next);
        Walk* const done = cur;
        cur = next;
        next = done;
        }
    }
    fence_before();
    __syncthreads();
    fence_after();
    if (warp == 0)
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
        if (saw_nothing(mi, li)) continue;
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
        put8(dst + 8 * k, round8<T>(z), vec_out);
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
