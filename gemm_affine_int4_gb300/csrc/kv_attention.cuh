// kv_attention.cuh -- causal attention over the paged 4-bit key/value cache
// for few query rows per key/value head (one token or a few per request), and
// for f32 activations at any length.
//
// Mathematics. With k_j = s q_j + b per group of a key row, q . k_j =
// sum_g s_g (q_g . c_g) + b_g (sum of q_g): the 4-bit codes go into the matrix
// unit as they are (exact in binary16) and scale and bias are applied to the
// products in binary32. For values, p_j s_j is rounded to binary16 and
// multiplied with the codes less 8, and sum_j p_j (b_j + 8 s_j) is kept in
// binary32. So no key or value is ever rounded; softmax maximum and sum run
// over the keys once.
//
//  * A code masked out of its word is a binary16 subnormal, c * 2^-24 (bits
//    0..3 of a half) or c * 2^-20 (bits 4..7): no conversion at all. The query
//    operand is scaled by a power of two per row so that its largest element
//    is near 2^13 (queries keep all their bits; 2^-4 more for the elements
//    that meet bits 4..7); the powers of two leave in the score's factor.
//  * The value side's p s is scaled by a power of two R, one for each query row,
//    that follows the largest |s| that the row sees (its accumulators are
//    rescaled when it grows), so any range of scales works and binary16 has 38
//    bits of room. Rounding p s to 11 bits is the path's one rounding below 32
//    bits: its errors are independent from key to key, and bf16 / f16 outputs
//    are rounded to 8 / 11 bits after it (4 requests of 131072 f16 tokens:
//    3.1e-4 of the outputs' size, against 2.1e-4 for the output's rounding
//    alone).
//  * f32 queries and f32 p s are split in two binary16 parts (22 bits).
//
// Shape of the products (mma m16n8k16, tokens or value channels along M, query
// rows along N): S^T = K Q^T and O^T = V^T P^T. One N tile is 8 query rows
// (tokens x query heads of one key/value head), so the usual 4 to 8 query
// heads per key head waste little. The matrix unit is no limit here (24 % busy);
// tcgen05 would need the codes expanded through shared memory first, which
// costs more than all the rest of this kernel.
//
// Work split. Tokens are cut into 64-token tiles; a unit is (request,
// key/value head, block of 8 NT query rows), and all units' tiles form one
// line that is cut evenly over the CTAs: ragged lengths and few long requests
// alike fill the GPU. In a CTA a producer warp streams tiles through a ring of
// shared-memory stages (one bulk copy per page and side for the codes, 16-byte
// asynchronous copies for scales and biases), consumer warps take half a tile
// in turn with accumulators of their own, and take turns at joining them at
// the end of a unit, while the others go on. A unit that is cut leaves (m, l,
// O) records in the workspace, which a second kernel joins in order; its
// launch overlaps the first. No sum depends on timing: results repeat.
//
// What bounds it: dependent instructions. The two or three consumer warps of an
// SMSP issue in 59 % of its cycles, and each mostly waits for its own last
// result. 4 requests of 90001 to 131072 tokens, 8 key/value heads of 128 f16
// values, 8 query heads each (494 MB): 113 us, 4.4 TB/s; with the loads alone 83
// us, with the products alone 111 (of 114 at the time). 48 requests of up to
// 4500 tokens (126 MB): 43 us.
#pragma once

#include <math.h>

#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "pipeline.cuh"

namespace gai4 {
namespace kvs {

using namespace pipe;

constexpr int kTile = 64;                       // tokens of a stage of the ring, loaded at once
constexpr int kSub = 32;                        // tokens that a consumer warp works on: half a stage
constexpr int kBlocks = kSub / 16;              // 16-token blocks of a sub-tile
// Units of up to so many tokens, by the width of the block table or the
// window: they are not cut, and the joining kernel is not launched. Measured
// not cut / cut, in us, at 8 key/value heads of 128 and 4 query heads each: one request of 60 tokens 6.4/9.0, of 300
// 8.3/8.9, of 500 9.7/9.3, of 1000 12.6/10.4; 16 requests of 500 11.6/13.1, of
// 1000 15.6/14.5; 64 of 500 20.8/24.1, of 1000 30.2/32.1, of 2000 46.9/42.5.
// The host's part of a call falls by 2.5 us as well. (The width stands for the
// requests' lengths, which the host does not know: under a wide table short
// requests are cut.)
constexpr int kWholeTokens = 512;
// What the start and join of a unit cost, in tiles (see Walk). Measured with 2,
// 4, 6 and 9: 48 ragged requests of up to 4500 tokens 52.7, 45.8, 42.2, 42.3
// us; 96 of up to 2000 in a step 65, 57, 54, 54; 30 in f32 36.6, 34.0, 35.2, 36.1.
constexpr int kStart = 6;

template <typename T_, int D_, int GS_, int NT_>
struct Cfg {
    using T = T_;
    static constexpr int D = D_, GS = GS_, NT = NT_;
    static constexpr int NG = D / GS;                       // groups of a row
    static constexpr int NC = 8 * NT;                       // query rows (columns of the products)
    static constexpr int E = T::kBytes;
    static constexpr bool kSplit = E == 4;                  // two binary16 parts
    static constexpr uint32_t kCodes = kTile * D / 2, kSb = kTile * NG * E;
    static constexpr uint32_t kStage = 2 * kCodes + 4 * kSb;
    static constexpr int DP = D + 4;                        // padded row of the join buffer
    // Consumer warps, and one producer: 8 warps divide the registers well (two
    // CTAs of 128 registers a thread, or one of 255); 12 where 168 are enough.
    static constexpr int kCtas = NT == 1 && !kSplit ? 2 : 1;   // resident CTAs per SM
    static constexpr int kWarps = kSplit && NT == 1 && D == 64 ? 11 : 7;
    static constexpr int kThreads = 32 * (kWarps + 1);
    static constexpr uint32_t kJoin = kWarps * NC * DP * 4 + 2 * kWarps * NC * 4;
    static constexpr uint32_t kBudget = (kCtas == 2 ? 112 : 225) * 1024 - kJoin - 1024;
    // A multiple of kWarps (odd), so that half a slot is always waited on by the
    // same warp, fill after fill: try_wait.parity takes a fill two behind for
    // done, and with other depths a warp could wait for a slot's next fill while
    // the one before, another warp's, is still on its way.
    static constexpr int kStages = (kBudget / (kStage + 24) < 2 * kWarps ? kBudget / (kStage + 24) : 2 * kWarps) / kWarps * kWarps;
    static constexpr uint32_t kSmem = kStages * kStage + kJoin + kStages * 24 + 256;
    static_assert(kStages >= kWarps && kStages % kWarps == 0 && kWarps % 2 == 1, "ring too short");
};

// records of cut units in the workspace: per CTA two of (O [NC][D], m [NC],
// l [NC]), number 0 for the end (or a middle) of a unit, 1 for its beginning,
// and one int4 about the latter: {last CTA of the unit or -1, query row of its
// row 0, head and place of row 0 among the head's query heads, rows}
__host__ __device__ constexpr size_t rec_floats(int nc, int d) { return (size_t)nc * (d + 2); }
__host__ __device__ constexpr size_t meta_bytes(int ctas) { return ((size_t)ctas * 16 + 255) / 256 * 256; }

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}
__device__ __forceinline__ uint32_t transpose8(uint32_t a) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}
// d = A B + c
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1, const float* c) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %11, %12, %13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}
// two binary32 operations at once, on neighbouring registers
__device__ __forceinline__ void add2(float& x, float& y, float a, float b) {
    asm("{\n .reg .b64 u, v;\n mov.b64 u, {%0, %1};\n mov.b64 v, {%2, %3};\n add.rn.f32x2 u, u, v;\n mov.b64 {%0, %1}, u;\n}"
        : "+f"(x), "+f"(y)
        : "f"(a), "f"(b));
}
__device__ __forceinline__ void mul2(float& x, float& y, float a, float b) {
    asm("{\n .reg .b64 u, v;\n mov.b64 u, {%0, %1};\n mov.b64 v, {%2, %3};\n mul.rn.f32x2 u, u, v;\n mov.b64 {%0, %1}, u;\n}"
        : "+f"(x), "+f"(y)
        : "f"(a), "f"(b));
}
__device__ __forceinline__ void fma2(float& x, float& y, float a, float b, float c, float d) {   // x = x a + c, y = y b + d
    asm("{\n .reg .b64 u, v, w;\n mov.b64 u, {%0, %1};\n mov.b64 v, {%2, %3};\n mov.b64 w, {%4, %5};\n"
        " fma.rn.f32x2 u, u, v, w;\n mov.b64 {%0, %1}, u;\n}"
        : "+f"(x), "+f"(y)
        : "f"(a), "f"(b), "f"(c), "f"(d));
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}
// token of row r (0..7) of a product's 8-row block: the P operand's rows 2t
// and 2t + 1 are tokens t and t + 4, so that neighbouring lanes of the value
// loads read neighbouring tokens
__device__ __forceinline__ int row_token(int r) { return (r >> 1) + 4 * (r & 1); }

// NG neighbouring scales or biases
template <typename T, int NG>
__device__ __forceinline__ void load_groups(const uint8_t* p, float (&v)[NG]) {
    if constexpr (T::kBytes == 4) {
        if constexpr (NG == 1) v[0] = *reinterpret_cast<const float*>(p);
        else
#pragma unroll
            for (int i = 0; i < NG; i += 2) {
                const float2 f = *reinterpret_cast<const float2*>(p + 4 * i);
                v[i] = f.x;
                v[i + 1] = f.y;
            }
    } else if constexpr (NG == 1) {
        v[0] = T::to_f32(*reinterpret_cast<const uint16_t*>(p));
    } else {
#pragma unroll
        for (int i = 0; i < NG; i += 2) {
            const uint32_t w = *reinterpret_cast<const uint32_t*>(p + 2 * i);
            v[i] = T::to_f32((uint16_t)w);
            v[i + 1] = T::to_f32((uint16_t)(w >> 16));
        }
    }
}

struct Req {
    int q0, qn, kv, tile0, ntile;   // first query row, rows, cached tokens, first tile, tiles of each unit
};

// units of request r: all rows of a request share the range of tiles that any
// of them sees (at least one tile, so that every unit writes its output)
__device__ __forceinline__ Req request(const KvAttnLaunch& p, int r) {
    Req q;
    const int n = (int)p.num_tokens;
    q.q0 = min(max(p.cu_q[r], 0), n);
    q.qn = max(min(p.cu_q[r + 1], n) - q.q0, 0);
    const long long cap = p.max_blocks << p.sh.page_log2;
    q.kv = (int)min((long long)max(p.kv_lens[r], 0), cap);
    const long long lo = p.window > 0 ? max((long long)q.kv - q.qn - p.window + 1, 0ll) : 0;
    q.tile0 = (int)(min(lo, (long long)q.kv) / kTile);
    q.ntile = max((q.kv + kTile - 1) / kTile - q.tile0, 1);
    return q;
}
__device__ __forceinline__ int row_blocks(const KvAttnLaunch& p, const Req& q, int nc) {
    return (q.qn * p.group + nc - 1) / nc;   // (num_tokens * group is below 2^31)
}

// what the rows of a unit may see
struct Limits {
    int rows;             // rows of the unit, at most NC
    int first;            // index of row 0 among the request's tokens x heads, modulo the heads
    int i0;               // token of row 0
    int lo_max, hi_min;   // keys in [lo_max, hi_min) are seen by every row of the unit
};

__device__ __forceinline__ int lowest_key(const KvAttnLaunch& p, long long pos) {
    return p.window > 0 ? (int)max(pos - p.window + 1, 0ll) : 0;
}

// A warp's walk along the line of tiles. Each unit begins with kStart places
// without work, which stand for its query load and join, so that CTAs with
// many short units get fewer tiles; a unit belongs to the CTA that has its
// first tile's place. Without CUT that CTA has all of it, and no other kernel
// has to join anything. Kept in shared memory (every lane writes the same): it
// is needed between segments, and the consumers have no registers to spare.
template <int NC, bool CUT>
struct Walk {
    long long c, c1;
    int r, h, rb, nrb, place;   // request, head, row block (of nrb), place within the unit (tile + kStart)
    Req q;
    int a, b;                   // tiles of the segment that some row of the unit can see
    Limits L;

    __device__ void init(const KvAttnLaunch& p, int r0, long long off, long long c0, long long c1_) {
        c = c0;
        c1 = c1_;
        r = r0;
        q = request(p, r);
        nrb = row_blocks(p, q, NC);
        const int unit = (int)(off / (q.ntile + kStart));
        place = (int)(off - (long long)unit * (q.ntile + kStart));
        h = unit / nrb;
        rb = unit - h * nrb;
        settle(p);
    }
    __device__ bool more() const { return c < c1; }
    // places of this segment
    __device__ int here() const {
        const int rest = q.ntile + kStart - place;
        return CUT ? (int)min((long long)rest, c1 - c) : rest;
    }
    // it has no tile (without CUT: none of this CTA's)
    __device__ bool idle() const { return CUT ? place + here() <= kStart : place > kStart || c + (kStart - place) >= c1; }
    __device__ bool begins() const { return place <= kStart; }
    __device__ bool ends() const { return place + here() == q.ntile + kStart; }
    __device__ void step(const KvAttnLaunch& p) {
        const int n = here();
        c += n;
        place += n;
        if (place < q.ntile + kStart) return;
        place = 0;
        if (++rb < nrb) return;
        rb = 0;
        if (++h < p.sh.hkv || c >= c1) return;
        h = 0;
        do {
            q = request(p, ++r);
            nrb = row_blocks(p, q, NC);
        } while (nrb == 0);   // (c < c1: there is another unit)
    }
    // on to a segment with a tile's place (or the end), and its limits
    __device__ void settle(const KvAttnLaunch& p) {
        while (more() && idle()) step(p);
        if (!more()) return;
        const int rr0 = rb * NC;
        L.rows = min(NC, q.qn * p.group - rr0);
        L.i0 = rr0 / p.group;
        L.first = rr0 - L.i0 * p.group;
        const long long pos0 = (long long)q.kv - q.qn + L.i0, pos1 = pos0 + (L.first + L.rows - 1) / p.group;
        L.hi_min = (int)max(pos0 + 1, 0ll);
        L.lo_max = lowest_key(p, pos1);
        a = max(max(place - kStart, 0), lowest_key(p, pos0) / kTile - q.tile0);
        b = max(a, min(place - kStart + here(), (int)((max(pos1 + 1, 0ll) + kTile - 1) / kTile) - q.tile0));
    }
    __device__ void advance(const KvAttnLaunch& p) {
        __syncwarp();   // every lane has read what it needs
        Walk w = *this;
        w.step(p);
        w.settle(p);
        __syncwarp();
        *this = w;
        __syncwarp();
    }
};

// The producer, two stages at a time (its chain of waits and votes costs about
// a thousand cycles beside busy consumers: with one stage at a time it set the
// pace). Of each stage the codes come by bulk copies, one for each page and
// side, issued by one lane each; scales and biases, a ninth of the bytes, by
// 16-byte asynchronous copies of the whole warp: bulk copies take a lane's
// issue each, and with small pages there would be up to 24 of them.
template <class C, bool CUT>
__device__ __forceinline__ void producer(const KvAttnLaunch& p, Walk<C::NC, CUT>& w, uint8_t* ring, uint64_t* full,
                                         uint64_t* empty, uint32_t* masks, const Ctl& ctl) {
    constexpr int S = C::kStages;
    constexpr int kRow = C::NG * C::E;                      // bytes of a token's scales (or biases)
    constexpr int kPer = C::kSb / 16;                       // 16-byte chunks of each of the four arrays
    constexpr int kCopies = 4 * kPer / 32;                  // of them for each lane
    const int lane = threadIdx.x & 31;
    const int pl = p.sh.page_log2, in_page = (1 << pl) - 1;
    const int pp = pl >= 6 ? 0 : 6 - pl;                    // log2 of the pages of a stage
    const int tokens = kTile >> pp;                         // tokens of a page in it
    const int pieces = 1 << pp;
    // bulk copies: lane = page + pieces * (side + 2 * stage of the two)
    const int piece = lane & (pieces - 1), side = (lane >> pp) & 1, j = lane >> (pp + 1);
    const bool leader = (lane & (2 * pieces - 1)) == 0;
    const uint32_t code_bytes = (uint32_t)tokens * (C::D / 2);
    const uint8_t* codes = reinterpret_cast<const uint8_t*>(side == 0 ? p.k.packed : p.v.packed);
    const uint32_t ring_s = smem_u32(ring);
    const uint32_t code_dst = ring_s + side * C::kCodes + piece * code_bytes;
    // 16-byte copies: chunk lane + 32 i of the arrays laid end to end
    const uint8_t* sb_src[kCopies];
#pragma unroll
    for (int i = 0; i < kCopies; ++i) {
        const int idx = lane + 32 * i, array = idx / kPer, chunk = idx % kPer, pc = chunk * 16 / kRow / tokens;
        const void* base = array == 0 ? p.k.scales : array == 1 ? p.k.biases : array == 2 ? p.v.scales : p.v.biases;
        sb_src[i] = static_cast<const uint8_t*>(base) + (chunk * 16 - pc * tokens * kRow);
    }
    const uint32_t sb_dst = ring_s + 2 * C::kCodes + lane * 16;
    int slot = 0, issued = 0;       // next stage's slot, stages issued
    uint32_t phase = 1;             // parity of the slot's "empty" wait
    bool ok = true;
    for (; w.more() && ok; w.advance(p)) {
        const int a = w.a, b = w.b, h = w.h, kv_len = w.q.kv;
        const int* row = p.table + (long long)w.r * p.max_blocks;
        const int nblk = (kv_len + in_page) >> pl;
        int tok0 = (w.q.tile0 + a + j) * kTile;             // first token of this lane's stage
        int at = (tok0 + piece * tokens) >> pl;
        int page = j < 2 && a + j < b && at < nblk ? row[at] : -1;
        for (int t = a; t < b; t += 2, tok0 += 2 * kTile) {
            const int n = min(2, b - t);
            const bool live = j < n;
            const bool there = live && page >= 0 && page < p.sh.num_blocks;
            const uint32_t votes = __ballot_sync(0xffffffffu, there);
            const int off = (tok0 + piece * tokens) & in_page;
            const long long line = there ? (((long long)page * p.sh.hkv + h) << pl) + off : 0;   // first row
            at = (tok0 + 2 * kTile + piece * tokens) >> pl;
            page = j < 2 && t + 2 + j < b && at < nblk ? row[at] : -1;   // for the next turn
            int my_slot = slot + j;
            const bool wrapped = my_slot >= S;
            if (wrapped) my_slot -= S;
            bool mine = true;
            if (live) mine = mbar_wait(&empty[my_slot], wrapped ? phase ^ 1u : phase, ctl);
            if (!__all_sync(0xffffffffu, mine)) {
                ok = false;
                break;
            }
            if (live && leader) {
                const uint32_t got = (votes >> lane) & ((1u << pieces) - 1u);
                unsigned long long m = 0;
                for (int i = 0; i < pieces; ++i)
                    if ((got >> i) & 1u) m |= (pp == 0 ? ~0ull : (1ull << tokens) - 1) << (i * tokens);
                const int left = kv_len - tok0;
                if (left < 64) m &= left <= 0 ? 0ull : (1ull << left) - 1;
                masks[2 * my_slot] = (uint32_t)m;
                masks[2 * my_slot + 1] = (uint32_t)(m >> 32);
                mbar_arrive_expect_tx(&full[my_slot], __popc(got) * 2u * code_bytes);
            }
            __syncwarp();
            if (there) bulk_load(code_dst + (uint32_t)my_slot * C::kStage, codes + line * (C::D / 2), code_bytes, &full[my_slot]);
            __syncwarp();
            for (int k = 0; k < n; ++k) {
                const uint32_t dst = sb_dst + (uint32_t)slot * C::kStage;
                const int first = k * 2 * pieces;           // lane of the stage's first page
#pragma unroll
                for (int i = 0; i < kCopies; ++i) {
                    const int pc = (lane + 32 * i) % kPer * 16 / kRow / tokens;
                    const long long ln = __shfl_sync(0xffffffffu, line, first + pc);
                    if ((votes >> (first + pc)) & 1u)
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + 512 * i), "l"(sb_src[i] + ln * kRow)
                                     : "memory");
                }
                // this lane's copies count as its arrival once they have landed
                asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(&full[slot])) : "memory");
                if (++slot == S) {
                    slot = 0;
                    phase ^= 1u;
                }
            }
            issued += n;
        }
    }
    // no copy may land after the CTA has gone
    for (int i = issued > S ? issued - S : 0; i < issued; ++i) mbar_wait_drain(&full[i % S], (i / S) & 1, ctl.limit, ctl.status);
}

// Scales and biases (their bits) from which a group's middle, 8 s + b, may be
// beyond binary32
constexpr uint32_t kFarScale = 250u << 23, kFarBias = 253u << 23;   // 2^123, 2^126

// per-warp running state of a unit
template <class C>
struct Acc {
    float o[C::D / 16][C::NT][4];   // O^T less sum p (b + 8 s): [value channel block][rows][..], in units of R 2^-14 and of 2^-24, 2^-20 (f32: 1)
    float ab[C::NG][C::NT][2];      // sum p (b + 8 s)
    float m[C::NT][2], l[C::NT][2];
    float inv[C::NT][2];            // 2^14 / R
    uint32_t limit;                 // the least R of all columns, at most kFarScale (bits): scales up to it need no attention
};

// exponent field of R, a power of two of at least 2^-100
__device__ __forceinline__ int r_exponent(float inv) { return 268 - (int)(__float_as_uint(inv) >> 23); }
__device__ __forceinline__ float r_inverse(int e) { return __uint_as_float((uint32_t)(268 - e) << 23); }

template <class C>
__device__ __forceinline__ void clear(Acc<C>& a) {
#pragma unroll
    for (int i = 0; i < C::D / 16; ++i)
#pragma unroll
        for (int n = 0; n < C::NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) a.o[i][n][e] = 0.f;
#pragma unroll
    for (int n = 0; n < C::NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            a.m[n][e] = -INFINITY;
            a.l[n][e] = 0.f;
#pragma unroll
            for (int g = 0; g < C::NG; ++g) a.ab[g][n][e] = 0.f;
        }
#pragma unroll
    for (int n = 0; n < C::NT; ++n) a.inv[n][0] = a.inv[n][1] = r_inverse(27);
    a.limit = 0;
}

// query operand of one unit
template <class C>
struct Query {
    uint32_t b[C::kSplit ? 2 : 1][C::D / 16][C::NT][2];
    float f[C::NT][2];            // score factor of columns 2t, 2t + 1: log2(e) scale, powers of two undone
    float sq[C::NG][C::NT][2];    // log2(e) scale * sum of the group's elements
};

// A unit's query elements as they come: word k (GS / 32) + j of the lane holds
// channels 8 (k (GS / 8) + t (GS / 32) + j) on
template <class C>
struct RawQuery {
    uint4 w[C::NT][C::D / 32][C::E / 2];
};

template <class C>
__device__ __forceinline__ void fetch_query(const KvAttnLaunch& p, const Req& rq, int h, int rb, bool vec, RawQuery<C>& R) {
    using St = typename C::T::storage;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int n = 0; n < C::NT; ++n) {
        const int rr = rb * C::NC + n * 8 + g;
        const bool valid = rr < rq.qn * p.group;
        const int i = valid ? rr / p.group : 0;
        const int head = h * p.group + (valid ? rr - i * p.group : 0);
        const St* src = static_cast<const St*>(p.q) + (rq.q0 + i) * p.q_stride + (long long)head * C::D;
#pragma unroll
        for (int k = 0; k < C::NG; ++k)
#pragma unroll
            for (int j = 0; j < C::GS / 32; ++j) {
                uint4(&y)[C::E / 2] = R.w[n][k * (C::GS / 32) + j];
                const St* s = src + 8 * (k * (C::GS / 8) + t * (C::GS / 32) + j);
#pragma unroll
                for (int e = 0; e < C::E / 2; ++e) {
                    y[e] = make_uint4(0u, 0u, 0u, 0u);
                    if (valid && vec) {
                        y[e] = reinterpret_cast<const uint4*>(s)[e];
                    } else if (valid) {
                        uint32_t z[4];
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            if constexpr (C::E == 4) z[x] = __float_as_uint(s[4 * e + x]);
                            else z[x] = (uint32_t)s[2 * x] | ((uint32_t)s[2 * x + 1] << 16);
                        y[e] = make_uint4(z[0], z[1], z[2], z[3]);
                    }
                }
            }
    }
}

template <class C>
__device__ __forceinline__ void make_query(const KvAttnLaunch& p, const RawQuery<C>& R, Query<C>& Q) {
    using T = typename C::T;
    const int lane = threadIdx.x & 31, t = lane & 3;
    const float sl = p.scale * 1.4426950408889634f;
#pragma unroll
    for (int n = 0; n < C::NT; ++n) {
        float x[C::D / 32][8];
        float amax = 0.f, sum[C::NG];
#pragma unroll
        for (int k = 0; k < C::NG; ++k) {
            sum[k] = 0.f;
#pragma unroll
            for (int j = 0; j < C::GS / 32; ++j) {
                const int wi = k * (C::GS / 32) + j;
                float(&y)[8] = x[wi];
#pragma unroll
                for (int e = 0; e < C::E / 2; ++e) {
                    const uint4 r = R.w[n][wi][e];
                    const uint32_t z[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if constexpr (C::E == 4) {
                            y[4 * e + i] = __uint_as_float(z[i]);
                        } else {
                            y[2 * i] = T::to_f32((uint16_t)z[i]);
                            y[2 * i + 1] = T::to_f32((uint16_t)(z[i] >> 16));
                        }
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    amax = fmaxf(amax, fabsf(y[e]));
                    sum[k] += y[e];
                }
            }
        }
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        // largest element to [2^13, 2^14); exponents kept where both powers are normal
        const int e = min(max((int)(__float_as_uint(amax) >> 23), 20), 254);
        const float up = __uint_as_float((uint32_t)(267 - e) << 23), down = __uint_as_float((uint32_t)(e - 13) << 23);
#pragma unroll
        for (int k = 0; k < C::NG; ++k) {
            sum[k] += __shfl_xor_sync(0xffffffffu, sum[k], 1);
            sum[k] += __shfl_xor_sync(0xffffffffu, sum[k], 2);
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const int from = (2 * t + c) * 4;
            // 2^24 in two steps: down may be as large as 2^114
            Q.f[n][c] = __shfl_sync(0xffffffffu, down * sl, from) * 16777216.f;
#pragma unroll
            for (int k = 0; k < C::NG; ++k) Q.sq[k][n][c] = __shfl_sync(0xffffffffu, sum[k], from) * sl;
        }
#pragma unroll
        for (int wi = 0; wi < C::D / 32; ++wi) {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                // elements (2 half, 2 half + 4) meet bits 0..3, the next ones bits 4..7
                float y[4] = {x[wi][2 * half] * up, x[wi][2 * half + 4] * up, x[wi][2 * half + 1] * up * 0.0625f,
                              x[wi][2 * half + 5] * up * 0.0625f};
#pragma unroll
                for (int part = 0; part < (C::kSplit ? 2 : 1); ++part) {
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const uint32_t w = pack_f16(y[2 * k], y[2 * k + 1]);
                        Q.b[part][2 * wi + half][n][k] = w;
                        if constexpr (C::kSplit) {
                            const float2 back = __half22float2(*reinterpret_cast<const __half2*>(&w));
                            y[2 * k] -= back.x;
                            y[2 * k + 1] -= back.y;
                        }
                    }
                }
            }
        }
    }
}

// two codes as binary16: c 2^-24 (bits 0..3 of the halves) or c 2^-20 (bits
// 4..7) as they stand, or c - 8 (exact)
template <bool CENTRED, int HIGH>
__device__ __forceinline__ uint32_t value_codes(uint32_t w) {
    const uint32_t c = w & (HIGH ? 0x00F000F0u : 0x000F000Fu);
    if constexpr (!CENTRED) return c;
    uint32_t d;
    if constexpr (HIGH)   // (1024 + 16 c) / 16 - 72
        asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(c | 0x64006400u), "r"(0x2C002C00u), "r"(0xD480D480u));
    else                  // (1024 + c) - 1032
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(c | 0x64006400u), "r"(0x64086408u));
    return d;
}

// whether a value group has to be set apart: it, or its middle, is not finite
__device__ __forceinline__ bool far_group(float s, float b) { return !(fabsf(fmaf(8.f, s, b)) < INFINITY); }

// Tokens (bits of `bad`) with such groups: the rows that see one get NaN in the
// group's channels, and the group is zeroed in the stage, so that 0 x NaN does
// not reach the rows that do not see it.
template <class C, bool CUT>
__device__ __forceinline__ void set_apart(const uint8_t* stage, int sub, uint32_t bad, int tok0, const Walk<C::NC, CUT>& w,
                                          const KvAttnLaunch& p, Acc<C>& A) {
    using St = typename C::T::storage;
    const int lane = threadIdx.x & 31, t = lane & 3;
    St* vsc = reinterpret_cast<St*>(const_cast<uint8_t*>(stage) + 2 * C::kCodes + 2 * C::kSb) + (sub * kSub + lane) * C::NG;
    St* vbi = vsc + kTile * C::NG;
    uint32_t groups = 0;
#pragma unroll
    for (int k = 0; k < C::NG; ++k) {
        const float s = C::T::to_f32(vsc[k]), b = C::T::to_f32(vbi[k]);
        if (!far_group(s, b)) continue;
        groups |= 1u << k;
        vsc[k] = vbi[k] = St(0);
    }
    for (; bad != 0; bad &= bad - 1) {
        const int o = __ffs(bad) - 1, j = tok0 + o;
        const uint32_t of = __shfl_sync(0xffffffffu, groups, o);
#pragma unroll
        for (int n = 0; n < C::NT; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int col = n * 8 + 2 * t + c;
                const long long pos = (long long)w.q.kv - w.q.qn + w.L.i0 + (w.L.first + col) / p.group;
                if (col >= w.L.rows || j > pos || j < lowest_key(p, pos)) continue;
#pragma unroll
                for (int k = 0; k < C::NG; ++k)
                    if ((of >> k) & 1u) A.ab[k][n][c] = __uint_as_float(0x7fffffffu);
            }
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // before the next fill
    __syncwarp();
}

template <class C, bool CUT>
__device__ __forceinline__ void tile(const uint8_t* stage, int sub, uint32_t mask, int tok0, const Query<C>& Q,
                                     const KvAttnLaunch& p, const Walk<C::NC, CUT>& w, int lo_max, int hi_min, Acc<C>& A) {
    using T = typename C::T;
    constexpr int NT = C::NT, NG = C::NG, D = C::D, GS = C::GS;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const uint8_t* st = stage + sub * (kSub * D / 2);                       // this half's key codes; value codes kCodes on
    const uint8_t* ksc = stage + 2 * C::kCodes + sub * (kSub * NG * C::E);
    const uint8_t* kbi = ksc + C::kSb;
    const uint8_t* vsc = kbi + C::kSb;
    const uint8_t* vbi = vsc + C::kSb;
    const int tg = row_token(g);

    // ---- scores, in units of log2: x[16-token block][8-column block][row g | g + 8, column 2t | 2t + 1].
    // The products of both blocks and of a pair of groups are interleaved:
    // each depends on its own last one only.
    float x[kBlocks][NT][4];
    {
        constexpr int W = GS / 32;            // words per lane, row and group
        constexpr int KP = NG == 1 ? 1 : 2;   // groups at a time
        float u[kBlocks][NT][4], v[kBlocks][NT][4];
#pragma unroll
        for (int k0 = 0; k0 < NG; k0 += KP) {
            uint32_t wd[kBlocks][2][KP][W];   // [block][row g | g + 8][group][word]
            float acc[kBlocks][KP][NT][4];
#pragma unroll
            for (int mb = 0; mb < kBlocks; ++mb)
#pragma unroll
                for (int k = 0; k < KP; ++k) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint32_t* w = reinterpret_cast<const uint32_t*>(st + (16 * mb + 8 * e + tg) * (D / 2) +
                                                                              (k0 + k) * (GS / 2)) + t * W;
                        if constexpr (W == 1) {
                            wd[mb][e][k][0] = *w;
                        } else if constexpr (W == 2) {
                            const uint2 y = *reinterpret_cast<const uint2*>(w);
                            wd[mb][e][k][0] = y.x;
                            wd[mb][e][k][1] = y.y;
                        } else {
                            const uint4 y = *reinterpret_cast<const uint4*>(w);
                            wd[mb][e][k][0] = y.x;
                            wd[mb][e][k][1] = y.y;
                            wd[mb][e][k][2] = y.z;
                            wd[mb][e][k][3] = y.w;
                        }
                    }
                }
            const float zero[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < W; ++j)
#pragma unroll
                for (int half = 0; half < 2; ++half)
#pragma unroll
                    for (int part = 0; part < (C::kSplit ? 2 : 1); ++part)
#pragma unroll
                        for (int k = 0; k < KP; ++k)
#pragma unroll
                            for (int mb = 0; mb < kBlocks; ++mb) {
                                const uint32_t a = half ? wd[mb][0][k][j] >> 8 : wd[mb][0][k][j];
                                const uint32_t b = half ? wd[mb][1][k][j] >> 8 : wd[mb][1][k][j];
                                const int ks = 2 * ((k0 + k) * W + j) + half;
#pragma unroll
                                for (int n = 0; n < NT; ++n)
                                    mma16816(acc[mb][k][n], a & 0x000F000Fu, b & 0x000F000Fu, a & 0x00F000F0u,
                                             b & 0x00F000F0u, Q.b[part][ks][n][0], Q.b[part][ks][n][1],
                                             j + half + part == 0 ? zero : acc[mb][k][n]);
                            }
#pragma unroll
            for (int mb = 0; mb < kBlocks; ++mb) {
                float sc[2][NG], bi[2][NG];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    load_groups<T, NG>(ksc + (16 * mb + 8 * e + tg) * NG * C::E, sc[e]);
                    load_groups<T, NG>(kbi + (16 * mb + 8 * e + tg) * NG * C::E, bi[e]);
                }
#pragma unroll
                for (int k = 0; k < KP; ++k)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float s = sc[e >> 1][k0 + k], b = bi[e >> 1][k0 + k], q = Q.sq[k0 + k][n][e & 1];
                            u[mb][n][e] = k0 + k == 0 ? acc[mb][k][n][e] * s : fmaf(acc[mb][k][n][e], s, u[mb][n][e]);
                            v[mb][n][e] = k0 + k == 0 ? b * q : fmaf(b, q, v[mb][n][e]);
                        }
            }
        }
#pragma unroll
        for (int mb = 0; mb < kBlocks; ++mb)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; e += 2) {
                    x[mb][n][e] = u[mb][n][e];
                    x[mb][n][e + 1] = u[mb][n][e + 1];
                    fma2(x[mb][n][e], x[mb][n][e + 1], Q.f[n][0], Q.f[n][1], v[mb][n][e], v[mb][n][e + 1]);
                }
    }
    // ---- masks: only on tiles that some row does not see in full
    if (mask != ~0u || tok0 + kSub > hi_min || tok0 < lo_max) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int col = n * 8 + 2 * t + c;
                const long long pos = (long long)w.q.kv - w.q.qn + w.L.i0 + (w.L.first + col) / p.group;
                const int hi = col < w.L.rows ? (int)max(pos + 1, 0ll) : 0, lo = lowest_key(p, pos);
#pragma unroll
                for (int mb = 0; mb < kBlocks; ++mb)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int o = 16 * mb + tg + 8 * e, j = tok0 + o;
                        if (!((mask >> o) & 1) || j >= hi || j < lo) x[mb][n][2 * e + c] = -INFINITY;
                    }
            }
    }
    // ---- running maximum of every column
    float mx[NT][2];
    bool grew = false;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            float m = fmaxf(x[0][n][c], x[0][n][c + 2]);
#pragma unroll
            for (int mb = 1; mb < kBlocks; ++mb) m = fmaxf(m, fmaxf(x[mb][n][c], x[mb][n][c + 2]));
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
            mx[n][c] = m;
            grew |= m > A.m[n][c];
        }
    // whether some R has to grow: the largest value scale of the tile
    // (non-negative numbers, infinity and NaN are ordered as integers)
    uint32_t smax = 0, bmax = 0;
    static_assert(kSub == 32, "a lane per token");
    {
        float s[NG], b[NG];
        load_groups<T, NG>(vsc + lane * NG * C::E, s);
        load_groups<T, NG>(vbi + lane * NG * C::E, b);
#pragma unroll
        for (int k = 0; k < NG; ++k) {
            smax = max(smax, __float_as_uint(s[k]) & 0x7fffffffu);
            bmax = max(bmax, __float_as_uint(b[k]) & 0x7fffffffu);
        }
    }
    if (__any_sync(0xffffffffu, grew || smax > A.limit || bmax >= kFarBias)) {
        bool far = false;
        if (smax >= kFarScale || bmax >= kFarBias) {
            float s[NG], b[NG];
            load_groups<T, NG>(vsc + lane * NG * C::E, s);
            load_groups<T, NG>(vbi + lane * NG * C::E, b);
#pragma unroll
            for (int k = 0; k < NG; ++k) far |= far_group(s[k], b[k]);
        }
        const uint32_t bad = __ballot_sync(0xffffffffu, far);
        if (bad != 0) {
            set_apart<C, CUT>(stage, sub, bad, tok0, w, p, A);
            float s[NG];
            load_groups<T, NG>(vsc + lane * NG * C::E, s);
            smax = 0;
#pragma unroll
            for (int k = 0; k < NG; ++k) smax = max(smax, __float_as_uint(s[k]) & 0x7fffffffu);
        }
        float down[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) down[n][0] = down[n][1] = 1.f;
        const uint32_t sb = __reduce_max_sync(0xffffffffu, smax);
        if (sb > A.limit) {
            // a column's R follows the scales of the tokens that it sees: in sub-tiles that not every row sees in full
            // (up to the last cached token; scales are zero from there on), column by column
            uint32_t big[NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n) big[n][0] = big[n][1] = sb;
            if (tok0 < lo_max || min(tok0 + kSub, w.q.kv) > hi_min) {
#pragma unroll 1
                for (int col = 0; col < w.L.rows; ++col) {
                    const long long pos = (long long)w.q.kv - w.q.qn + w.L.i0 + (w.L.first + col) / p.group;
                    const int j = tok0 + lane;
                    const uint32_t of = __reduce_max_sync(0xffffffffu, j <= pos && j >= lowest_key(p, pos) ? smax : 0u);
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int c = 0; c < 2; ++c)
                            if (col == n * 8 + 2 * t + c) big[n][c] = of;
                }
            }
            int least = kFarScale >> 23;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int re = r_exponent(A.inv[n][c]);
                    const int ne = max(re, (int)(big[n][c] >> 23) + ((big[n][c] & 0x7fffffu) != 0));
                    down[n][c] = ex2((float)(re - ne));
                    A.inv[n][c] = r_inverse(ne);
                    least = min(least, ne);
                }
            A.limit = (uint32_t)__reduce_min_sync(0xffffffffu, least) << 23;
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const float m = fmaxf(A.m[n][c], mx[n][c]);
                const float f = A.m[n][c] == -INFINITY ? 0.f : ex2(A.m[n][c] - m);
                A.m[n][c] = m;
                A.l[n][c] *= f;
#pragma unroll
                for (int k = 0; k < NG; ++k) A.ab[k][n][c] *= f;
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    A.o[i][n][c] *= f * down[n][c];
                    A.o[i][n][c + 2] *= f * down[n][c];
                }
            }
    }
    // ---- probabilities
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const float m0 = A.m[n][0] == -INFINITY ? 0.f : -A.m[n][0], m1 = A.m[n][1] == -INFINITY ? 0.f : -A.m[n][1];
#pragma unroll
        for (int mb = 0; mb < kBlocks; ++mb)
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
                add2(x[mb][n][e], x[mb][n][e + 1], m0, m1);
                x[mb][n][e] = ex2(x[mb][n][e]);
                x[mb][n][e + 1] = ex2(x[mb][n][e + 1]);
                add2(A.l[n][0], A.l[n][1], x[mb][n][e], x[mb][n][e + 1]);
            }
    }
    // ---- values. What the matrix unit sums are p s (c - 8), the mean of the
    // codes taken off, and only over this sub-tile; sum p (b + 8 s) and the sums
    // over the sub-tiles are binary32 additions. (The unit truncates its sums:
    // over a whole unit, with uncentred codes, 30 f32 requests were 2e-5 off.)
    // bf16 / f16: the sums of the codes as they are start at -8 sum p s, which
    // leaves a few 2^-24 of it. f32: the codes themselves are centred.
    constexpr int kParts = C::kSplit ? 2 : 1;
    uint32_t P[kBlocks][kParts][NG][NT][2];
#pragma unroll
    for (int mb = 0; mb < kBlocks; ++mb) {
        float sc[2][NG], bi[2][NG], z[NT][4];   // z: p 2^14 / R (0 where s / R may be anything)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            load_groups<T, NG>(vsc + (16 * mb + tg + 8 * e) * NG * C::E, sc[e]);
            load_groups<T, NG>(vbi + (16 * mb + tg + 8 * e) * NG * C::E, bi[e]);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                z[n][2 * e] = x[mb][n][2 * e];
                z[n][2 * e + 1] = x[mb][n][2 * e + 1];
                mul2(z[n][2 * e], z[n][2 * e + 1], A.inv[n][0], A.inv[n][1]);
            }
        }
#pragma unroll
        for (int k = 0; k < NG; ++k) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float f = sc[e][k], mid = fmaf(8.f, f, bi[e][k]);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
#pragma unroll
                    for (int c = 0; c < 2; ++c) A.ab[k][n][c] = fmaf(x[mb][n][2 * e + c], mid, A.ab[k][n][c]);
                    float y0 = z[n][2 * e], y1 = z[n][2 * e + 1];
                    mul2(y0, y1, f, f);
                    const uint32_t w = pack_f16(y0, y1);
                    P[mb][0][k][n][e] = transpose8(w);
                    if constexpr (C::kSplit) {
                        const float2 back = __half22float2(*reinterpret_cast<const __half2*>(&w));
                        P[mb][1][k][n][e] = transpose8(pack_f16(y0 - back.x, y1 - back.y));
                    }
                }
            }
        }
    }
    // -8 sum p s, in the units of rows g (2^-24) and g + 8 (2^-20): where the sums start (f32: at 0)
    float start[NG][NT][4];
#pragma unroll
    for (int k = 0; k < NG; ++k)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int e = 0; e < 4; ++e) start[k][n][e] = 0.f;
            if constexpr (!C::kSplit) {
                const float zero[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int mb = 0; mb < kBlocks; ++mb)
                    mma16816(start[k][n], 0x80088008u, 0x80808080u, 0x80088008u, 0x80808080u, P[mb][0][k][n][0],
                             P[mb][0][k][n][1], mb == 0 ? zero : start[k][n]);
            }
        }
    // rows g / g + 8 of a value block: codes 2i / 2i + 1 of this lane's word
    const uint8_t* vc = st + C::kCodes + t * (D / 2);   // tokens t, t + 4, t + 8, t + 12 of each 16-token block
    constexpr int kChunks = GS == 32 ? NG : D / 64;
#pragma unroll
    for (int j = 0; j < kChunks; ++j) {
        const int word = GS == 32 ? 4 * j + (g >> 1) : 8 * j + g;
        uint32_t w[kBlocks][4];
#pragma unroll
        for (int mb = 0; mb < kBlocks; ++mb)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[mb][i] = *reinterpret_cast<const uint32_t*>(vc + (16 * mb + 4 * i) * (D / 2) + word * 4);
        constexpr int kHalves = GS == 32 ? 1 : 2;
#pragma unroll
        for (int hh = 0; hh < kHalves; ++hh) {
            const uint32_t sel = GS == 32 ? ((g & 1) ? 0x7632u : 0x5410u) : (hh ? 0x7632u : 0x5410u);
            const int k = GS == 32 ? j : (j * 64) / GS;
            uint32_t a[kBlocks], b[kBlocks];
#pragma unroll
            for (int mb = 0; mb < kBlocks; ++mb) {
                a[mb] = __byte_perm(w[mb][0], w[mb][1], sel);
                b[mb] = __byte_perm(w[mb][2], w[mb][3], sel);
            }
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int blk = GS == 32 ? 2 * j + q : 4 * j + 2 * hh + q;
                float acc[NT][4];
#pragma unroll
                for (int mb = 0; mb < kBlocks; ++mb) {
                    const uint32_t aa = q ? a[mb] >> 8 : a[mb], bb = q ? b[mb] >> 8 : b[mb];
                    const uint32_t a0 = value_codes<C::kSplit, 0>(aa), a1 = value_codes<C::kSplit, 1>(aa);
                    const uint32_t a2 = value_codes<C::kSplit, 0>(bb), a3 = value_codes<C::kSplit, 1>(bb);
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int part = 0; part < kParts; ++part)
                            mma16816(acc[n], a0, a1, a2, a3, P[mb][part][k][n][0], P[mb][part][k][n][1],
                                     mb + part == 0 ? start[k][n] : acc[n]);
                }
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; e += 2) add2(A.o[blk][n][e], A.o[blk][n][e + 1], acc[n][e], acc[n][e + 1]);
            }
        }
    }
}

// a warp's results of a segment into its place of the join buffer
template <class C>
__device__ __forceinline__ void deposit(Acc<C>& A, uint8_t* buf) {
    constexpr int NT = C::NT, NC = C::NC, D = C::D, DP = C::DP;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    float* o = reinterpret_cast<float*>(buf);
    float* sm = o + C::kWarps * NC * DP;
    float* sl = sm + C::kWarps * NC;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
#pragma unroll
            for (int s = 4; s < 32; s <<= 1) {
                A.l[n][c] += __shfl_xor_sync(0xffffffffu, A.l[n][c], s);
#pragma unroll
                for (int k = 0; k < C::NG; ++k) A.ab[k][n][c] += __shfl_xor_sync(0xffffffffu, A.ab[k][n][c], s);
            }
        }
    constexpr float kLow = C::kSplit ? 1.f / 16384.f : 1024.f, kHigh = C::kSplit ? 1.f / 16384.f : 64.f;   // 2^-14 / the codes' unit
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const int col = n * 8 + 2 * t + c;
            if (g == 0) {
                sm[warp * NC + col] = A.m[n][c];
                sl[warp * NC + col] = A.l[n][c];
            }
            float* dst = o + (warp * NC + col) * DP;
            const float R = __uint_as_float((uint32_t)r_exponent(A.inv[n][c]) << 23);
            if constexpr (C::GS == 32) {
#pragma unroll
                for (int k = 0; k < C::NG; ++k) {   // channels 32 k + 8 (g >> 1) + 4 (g & 1) + 0..3
                    float4 f;
                    f.x = fmaf(A.o[2 * k][n][c] * kLow, R, A.ab[k][n][c]);
                    f.y = fmaf(A.o[2 * k][n][c + 2] * kHigh, R, A.ab[k][n][c]);
                    f.z = fmaf(A.o[2 * k + 1][n][c] * kLow, R, A.ab[k][n][c]);
                    f.w = fmaf(A.o[2 * k + 1][n][c + 2] * kHigh, R, A.ab[k][n][c]);
                    *reinterpret_cast<float4*>(dst + 32 * k + 4 * g) = f;
                }
            } else {
#pragma unroll
                for (int j = 0; j < D / 64; ++j)
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh) {   // channels 64 j + 8 g + 4 hh + 0..3
                        const int k = (j * 64) / C::GS, b = 4 * j + 2 * hh;
                        float4 f;
                        f.x = fmaf(A.o[b][n][c] * kLow, R, A.ab[k][n][c]);
                        f.y = fmaf(A.o[b][n][c + 2] * kHigh, R, A.ab[k][n][c]);
                        f.z = fmaf(A.o[b + 1][n][c] * kLow, R, A.ab[k][n][c]);
                        f.w = fmaf(A.o[b + 1][n][c + 2] * kHigh, R, A.ab[k][n][c]);
                        *reinterpret_cast<float4*>(dst + 64 * j + 8 * g + 4 * hh) = f;
                    }
            }
        }
}
// one that had no sub-tile of the segment
template <class C>
__device__ __forceinline__ void deposit_nothing(uint8_t* buf) {
    float* sm = reinterpret_cast<float*>(buf) + C::kWarps * C::NC * C::DP;
    float* sl = sm + C::kWarps * C::NC;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane < C::NC) {
        sm[warp * C::NC + lane] = -INFINITY;
        sl[warp * C::NC + lane] = 0.f;
    }
}

// joins what the warps have deposited, by one warp: each lane four channels of
// a column, write(column, channel, float4 O, m, l) with O not yet divided by l
template <class C, typename F>
__device__ __forceinline__ void join(const uint8_t* buf, int columns, F&& write) {
    constexpr int NC = C::NC, D = C::D, DP = C::DP;
    const float* o = reinterpret_cast<const float*>(buf);
    const float* sm = o + C::kWarps * NC * DP;
    const float* sl = sm + C::kWarps * NC;
    for (int i = threadIdx.x & 31; i < columns * (D / 4); i += 32) {
        const int col = i / (D / 4), d = (i % (D / 4)) * 4;
        float m = -INFINITY;
#pragma unroll
        for (int w = 0; w < C::kWarps; ++w) m = fmaxf(m, sm[w * NC + col]);
        float l = 0.f;
        float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < C::kWarps; ++w) {
            const float mw = sm[w * NC + col], lw = sl[w * NC + col];
            if (!saw_nothing(mw, lw)) {
                const float e = ex2(mw - m);
                const float4 v = *reinterpret_cast<const float4*>(o + (w * NC + col) * DP + d);
                l = fmaf(lw, e, l);
                f.x = fmaf(v.x, e, f.x);
                f.y = fmaf(v.y, e, f.y);
                f.z = fmaf(v.z, e, f.z);
                f.w = fmaf(v.w, e, f.w);
            }
        }
        write(col, d, f, m, l);
    }
}

// one query row's four channels, divided by the softmax sum and rounded once
template <typename T>
__device__ __forceinline__ void store_out(const KvAttnLaunch& p, bool vec, long long row, int head, int D, int d, float4 f,
                                          float m, float l) {
    using St = typename T::storage;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    if (l == 0.f) f = make_float4(0.f, 0.f, 0.f, 0.f);
    St* o = static_cast<St*>(p.out) + row * p.out_stride + (long long)head * D + d;
    const St v[4] = {T::from_f32(f.x * inv), T::from_f32(f.y * inv), T::from_f32(f.z * inv), T::from_f32(f.w * inv)};
    if (vec) {
        if constexpr (T::kBytes == 4)
            *reinterpret_cast<float4*>(o) = make_float4(v[0], v[1], v[2], v[3]);
        else
            *reinterpret_cast<uint2*>(o) =
                make_uint2((uint32_t)v[0] | ((uint32_t)v[1] << 16), (uint32_t)v[2] | ((uint32_t)v[3] << 16));
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = v[i];
    }
    if (p.lse && d == 0)
        p.lse[row * ((long long)p.sh.hkv * p.group) + head] =
            l == 0.f ? -INFINITY : fmaf(m, 0.6931471805599453f, logf(l));
}

template <class C, bool CUT>
__global__ void __launch_bounds__(C::kThreads, C::kCtas)
    kv_attention_kernel(const __grid_constant__ KvAttnLaunch p, const int vec_q, const int vec_out) {
    using T = typename C::T;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ long long warp_cost[C::kWarps + 1];
    __shared__ long long start_off;
    __shared__ int start_r, abort_flag;
    constexpr int S = C::kStages;
    uint8_t* ring = smem;
    uint8_t* buf = ring + S * C::kStage;
    uint64_t* full = reinterpret_cast<uint64_t*>(buf + C::kJoin);
    uint64_t* empty = full + S;
    uint32_t* masks = reinterpret_cast<uint32_t*>(empty + S);
    uint64_t *deposited = reinterpret_cast<uint64_t*>(masks + 2 * S), *joined = deposited + 1;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    pdl_launch_dependents();
    if (tid == 0) {
        mbar_init(deposited, C::kWarps);
        mbar_init(joined, 1);
        for (int i = 0; i < S; ++i) {
            mbar_init(&full[i], 33);   // the codes' copies, and each lane's of scales and biases
            mbar_init(&empty[i], 2);   // one warp for each half
        }
        abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    pdl_wait();

    // the line of tiles: its length, and where this CTA's part begins. Each
    // thread sums a strip of requests.
    const int per_thread = (p.batch + C::kThreads - 1) / C::kThreads;
    const int r0 = min(tid * per_thread, p.batch), r1 = min(r0 + per_thread, p.batch);
    auto cost = [&](int r) {
        const Req q = request(p, r);
        return (long long)row_blocks(p, q, C::NC) * p.sh.hkv * (q.ntile + kStart);
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
    for (int i = 0; i <= C::kWarps; ++i) {
        if (i < warp) before += warp_cost[i];
        total += warp_cost[i];
    }
    const long long per = max((total + gridDim.x - 1) / gridDim.x, 1ll);
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
            auto* o = static_cast<typename T::storage*>(p.out) + row * p.out_stride;
            for (int i = tid; i < hq * C::D; i += C::kThreads) o[i] = T::from_f32(0.f);
            if (p.lse)
                for (int i = tid; i < hq; i += C::kThreads) p.lse[row * hq + i] = -INFINITY;
        }
    }
    uint8_t* ws = static_cast<uint8_t*>(p.workspace);
    int4* meta = reinterpret_cast<int4*>(ws) + blockIdx.x;
    float* recs = reinterpret_cast<float*>(ws + meta_bytes(gridDim.x)) + blockIdx.x * 2 * rec_floats(C::NC, C::D);
    __syncthreads();
    if (c0 >= c1) {
        if (CUT && tid == 0) *meta = make_int4(-1, 0, 0, 0);
        return;
    }

    __shared__ Walk<C::NC, CUT> walks[C::kWarps + 1];
    Walk<C::NC, CUT>& w = walks[warp];
    {
        Walk<C::NC, CUT> first;
        first.init(p, start_r, start_off, c0, c1);
        w = first;
        __syncwarp();
    }
    const Ctl ctl{p.status, p.spin_limit, &abort_flag};
    if (warp == C::kWarps) {
        producer<C, CUT>(p, w, ring, full, empty, masks, ctl);
        return;
    }
    // ---- consumers. Each warp deposits its part of a segment and goes on; the
    // warps take turns at joining. (With a barrier of all warps instead, every
    // segment cost the time that the slowest warp was behind.)
    int seq = 0;                                   // first sub-tile of the current segment (two to a stage)
    int my = warp, slot = warp >> 1, phase = 0;    // this warp's next sub-tile: every kWarps-th, and its stage's slot
    int turn = 0;                                  // the warp that joins the current segment
    uint32_t parity = 0;                           // of the segments' number
    if (CUT && tid == 0) *meta = make_int4(-1, 0, 0, 0);  // until this CTA holds the beginning of a unit that goes on
    RawQuery<C> raw;                               // (fetched by every warp, with a part in the segment or not: by
    bool more = w.more();                          // some, it would live in registers all along)
    if (more) fetch_query<C>(p, w.q, w.h, w.rb, vec_q != 0, raw);
    while (more) {
        const int end = seq + 2 * (w.b - w.a);     // sub-tiles up to this segment's last
        const bool part = my < end;
        if (part) {
            Query<C> Q;
            make_query<C>(p, raw, Q);
            Acc<C> A;
            clear<C>(A);
            const int lo_max = w.L.lo_max, hi_min = w.L.hi_min, key0 = (w.q.tile0 + w.a) * kTile - seq * kSub;
            for (; my < end; my += C::kWarps) {
                const int sub = my & 1, tok0 = key0 + my * kSub;
                // after a time-out the outputs are undefined, but every role still ends
                (void)warp_wait(&full[slot], (uint32_t)phase, ctl);
                uint8_t* st = ring + (size_t)slot * C::kStage;
                const uint32_t mask = masks[2 * slot + sub];
                if (mask != 0) {
                    if (mask != ~0u) {
                        // scales and biases of slots without a token may hold anything
                        if (!((mask >> lane) & 1))
                            for (int k = 0; k < 4; ++k)
                                for (int i = 0; i < C::NG * C::E / 2; ++i)
                                    reinterpret_cast<uint16_t*>(st + 2 * C::kCodes +
                                                                k * C::kSb)[(sub * kSub + lane) * (C::NG * C::E / 2) + i] = 0;
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // before the next fill
                        __syncwarp();
                    }
                    tile<C, CUT>(st, sub, mask, tok0, Q, p, w, lo_max, hi_min, A);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&empty[slot]);
                slot += ((my + C::kWarps) >> 1) - (my >> 1);
                if (slot >= S) {
                    slot -= S;
                    phase ^= 1;
                }
            }
            (void)warp_wait(joined, parity ^ 1u, ctl);   // the buffer is free
            deposit<C>(A, buf);
        } else {
            (void)warp_wait(joined, parity ^ 1u, ctl);
            deposit_nothing<C>(buf);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(deposited);
        seq = end;
        const bool begins = w.begins(), whole = begins && w.ends();
        const int q0 = w.q.q0 + w.L.i0, h = w.h, first = w.L.first, rows = w.L.rows;
        if (CUT && begins && !whole && tid == 0) {
            const long long end_of_unit = w.c - w.place + w.q.ntile + kStart;   // on the line
            *meta = make_int4((int)((end_of_unit - 1) / per), q0, h << 16 | first, rows);
        }
        w.advance(p);
        more = w.more();
        if (more) fetch_query<C>(p, w.q, w.h, w.rb, vec_q != 0, raw);
        if (turn == warp) {
            (void)warp_wait(deposited, parity, ctl);
            float* rec = recs + (begins ? rec_floats(C::NC, C::D) : 0);
            join<C>(buf, rows, [&](int col, int d, float4 f, float m, float l) {
                if (!CUT || whole) {
                    const int i = (first + col) / p.group;
                    store_out<T>(p, vec_out != 0, q0 + i, h * p.group + (first + col - i * p.group), C::D, d, f, m, l);
                } else {
                    *reinterpret_cast<float4*>(rec + col * C::D + d) = f;
                    if (d == 0) {
                        rec[C::NC * C::D + col] = m;
                        rec[C::NC * C::D + C::NC + col] = l;
                    }
                }
            });
            __syncwarp();
            if (lane == 0) mbar_arrive(joined);
        }
        parity ^= 1u;
        if (++turn == C::kWarps) turn = 0;
    }
}

// joins the records of a cut unit, in the order of the CTAs: block (i, c) the
// column c of the unit that begins in CTA i and goes on
template <class C>
__global__ void __launch_bounds__(128) kv_combine_kernel(const __grid_constant__ KvAttnLaunch p, const int ctas,
                                                         const int vec_out) {
    constexpr int D = C::D, NC = C::NC, G = 128 / (D / 4);   // groups of threads that share the records
    __shared__ float sm[G], sl[G];
    __shared__ float4 so[128];
    pdl_launch_dependents();
    pdl_wait();
    const uint8_t* ws = static_cast<const uint8_t*>(p.workspace);
    const int4 meta = reinterpret_cast<const int4*>(ws)[blockIdx.x];
    const int col = blockIdx.y;
    if (meta.x < 0 || col >= meta.w) return;
    const float* recs = reinterpret_cast<const float*>(ws + meta_bytes(ctas));
    const int gi = threadIdx.x / (D / 4), d = (threadIdx.x % (D / 4)) * 4;
    const int n = meta.x - (int)blockIdx.x + 1;
    float m = -INFINITY, l = 0.f;
    float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int i = gi; i < n; i += G) {
        const float* rec = recs + ((size_t)(blockIdx.x + i) * 2 + (i == 0 ? 1 : 0)) * rec_floats(NC, D);
        const float mi = rec[NC * D + col], li = rec[NC * D + NC + col];
        const float4 v = *reinterpret_cast<const float4*>(rec + col * D + d);
        if (saw_nothing(mi, li)) continue;
        const float mn = fmaxf(m, mi);
        const float c = m == -INFINITY ? 0.f : ex2(m - mn), e = ex2(mi - mn);
        m = mn;
        l = l * c + li * e;
        f.x = f.x * c + v.x * e;
        f.y = f.y * c + v.y * e;
        f.z = f.z * c + v.z * e;
        f.w = f.w * c + v.w * e;
    }
    so[threadIdx.x] = f;
    if (d == 0) {
        sm[gi] = m;
        sl[gi] = l;
    }
    __syncthreads();
    if (gi != 0) return;
    float M = sm[0];
#pragma unroll
    for (int i = 1; i < G; ++i) M = fmaxf(M, sm[i]);
    float Ls = 0.f;
    float4 F = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < G; ++i) {
        if (saw_nothing(sm[i], sl[i])) continue;
        const float e = ex2(sm[i] - M);
        const float4 v = so[i * (D / 4) + threadIdx.x];
        Ls = fmaf(sl[i], e, Ls);
        F.x = fmaf(v.x, e, F.x);
        F.y = fmaf(v.y, e, F.y);
        F.z = fmaf(v.z, e, F.z);
        F.w = fmaf(v.w, e, F.w);
    }
    const int h = (uint32_t)meta.z >> 16, rr = (meta.z & 0xffff) + col, i = rr / p.group;
    store_out<typename C::T>(p, vec_out != 0, meta.y + i, h * p.group + (rr - i * p.group), D, d, F, M, Ls);
}

template <class C>
cudaError_t launch(const KvAttnLaunch& L, cudaStream_t s) {
    const int e = C::E;
    const int vec_q = ((uintptr_t)L.q & 15) == 0 && L.q_stride * e % 16 == 0;
    const int vec_out = ((uintptr_t)L.out & 15) == 0 && L.out_stride * e % 16 == 0;
    const int ctas = num_sms() * C::kCtas;
    static bool allowed[2][64];
    long long tokens = L.max_blocks << L.sh.page_log2;   // of the longest unit
    if (L.window > 0 && L.window <= kWholeTokens) tokens = std::min(tokens, (long long)(L.window + L.max_q_len));
    if (tokens <= kWholeTokens) {
        const cudaError_t err = allow_smem_once(kv_attention_kernel<C, false>, C::kSmem, allowed[0]);
        if (err != cudaSuccess) return err;
        return launch_pdl(kv_attention_kernel<C, false>, dim3(ctas), dim3(C::kThreads), C::kSmem, s, L, vec_q, vec_out);
    }
    cudaError_t err = allow_smem_once(kv_attention_kernel<C, true>, C::kSmem, allowed[1]);
    if (err != cudaSuccess) return err;
    err = launch_pdl(kv_attention_kernel<C, true>, dim3(ctas), dim3(C::kThreads), C::kSmem, s, L, vec_q, vec_out);
    if (err != cudaSuccess) return err;
    return launch_pdl(kv_combine_kernel<C>, dim3(ctas, C::NC), dim3(128), 0, s, L, ctas, vec_out);
}

// 8 columns when the rows of a request and head fit them, else 16 (fewer
// passes over the keys, but half the warps per SM). With 16 rows, 8 / 16
// columns, bf16, 8 key/value heads of 128: 20 requests of 16000 tokens 167/138
// us, 16 of 4000 48.4/45.3, 64 of 1000 66/78, one of 4000 14.8/17.1; with 8
// rows: 92/128, 30.9/39.1, -, -. Long contexts decide, where a call takes long.
template <typename T>
cudaError_t launch_type(const KvAttnLaunch& L, cudaStream_t s) {
    const bool one = L.max_q_len * L.group <= 8;
    if (L.sh.d == 64) {
        if (L.sh.gs == 32) return one ? launch<Cfg<T, 64, 32, 1>>(L, s) : launch<Cfg<T, 64, 32, 2>>(L, s);
        return one ? launch<Cfg<T, 64, 64, 1>>(L, s) : launch<Cfg<T, 64, 64, 2>>(L, s);
    }
    if (L.sh.gs == 32) return one ? launch<Cfg<T, 128, 32, 1>>(L, s) : launch<Cfg<T, 128, 32, 2>>(L, s);
    if (L.sh.gs == 64) return one ? launch<Cfg<T, 128, 64, 1>>(L, s) : launch<Cfg<T, 128, 64, 2>>(L, s);
    return one ? launch<Cfg<T, 128, 128, 1>>(L, s) : launch<Cfg<T, 128, 128, 2>>(L, s);
}

}  // namespace kvs
}  // namespace gai4
