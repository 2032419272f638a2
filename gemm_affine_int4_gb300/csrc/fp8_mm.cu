// fp8_mm.cu -- product of e4m3 activations and e4m3 weights with a scale for
// each block of 128 (internal; sm_103a: TMA, mbarrier, tcgen05 / TMEM, clusters):
//   out[m, n] = sum_b sx[m, b] sw[n / 128, b] sum_{k in block b} x[m, k] w[n, k]
//
// The inner sums run on the tensor cores, 128 columns at a time, into tensor
// memory; warps read them back, multiply by the block's scales and add them up
// in registers, in binary32.
#include <cuda.h>

#include <algorithm>
#include <cstring>

#include "common.cuh"
#include "internal.h"
#include "pipeline.cuh"

namespace gai4 {

namespace fp8mm {

using namespace pipe;

constexpr int kBlock = 128;   // columns of a scale; bytes of a row of a swizzled tile

__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// K-major operand of 128-byte rows, 128-byte swizzle: low word start address
// and leading byte offset, high word stride byte offset (8 rows), version 1,
// layout SWIZZLE_128B
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << (46 - 32)) | (2u << (61 - 32));
__device__ __forceinline__ uint32_t desc_lo(uint32_t a) { return ((a >> 4) & 0x3FFFu) | (1u << 16); }

// instruction descriptor, kind::f8f6f4: binary32 accumulators, both operands
// e4m3 and K-major
constexpr uint32_t idesc(int m, int n) { return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24); }

// the products of one block of 128 columns (4 steps of 32), by one lane of a
// converged warp; then the commits to two barriers
__device__ __forceinline__ void block_products(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t id, uint64_t* slot_free,
                                               uint64_t* done) {
    asm volatile(
        "{\n .reg .pred e, z, o;\n .reg .b32 r, t, u;\n .reg .b64 x, y;\n elect.sync r|e, 0xffffffff;\n"
        " setp.ne.b32 z, 0, 0;\n setp.eq.b32 o, 0, 0;\n"
        " mov.b64 x, {%1, %4};\n mov.b64 y, {%2, %4};\n"
        " @e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, %3, z;\n"
        " add.u32 u, %1, 2;\n mov.b64 x, {u, %4};\n add.u32 t, %2, 2;\n mov.b64 y, {t, %4};\n"
        " @e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, %3, o;\n"
        " add.u32 u, %1, 4;\n mov.b64 x, {u, %4};\n add.u32 t, %2, 4;\n mov.b64 y, {t, %4};\n"
        " @e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, %3, o;\n"
        " add.u32 u, %1, 6;\n mov.b64 x, {u, %4};\n add.u32 t, %2, 6;\n mov.b64 y, {t, %4};\n"
        " @e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, %3, o;\n"
        " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%5];\n"
        " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%6];\n}" ::"r"(d),
        "r"(a_lo), "r"(b_lo), "r"(id), "r"(kDescHi), "r"(smem_u32(slot_free)), "r"(smem_u32(done))
        : "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t a, uint32_t* v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(a)
        : "memory");
}

__device__ __forceinline__ float lds1(uint32_t a) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}

__device__ __forceinline__ float as_f32(uint32_t v) { return __uint_as_float(v); }
__device__ __forceinline__ float4 lds4(const float* p) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(smem_u32(p))
                 : "memory");
    return v;
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
__device__ __forceinline__ uint32_t mapa(uint32_t a, uint32_t rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
    return r;
}

__device__ __forceinline__ void store_at(uint32_t cluster_addr, int v) {
    asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(cluster_addr), "r"(v) : "memory");
}
__device__ __forceinline__ int load_at(uint32_t cluster_addr) {
    int v;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(cluster_addr) : "memory");
    return v;
}

// How often the i-th of `of` places has been used by `count` uses in turn, and
// the parity of the last use (of one at least)
__device__ __forceinline__ int rounds(int count, int of, int i) { return count > i ? (count - 1 - i) / of + 1 : 0; }
__device__ __forceinline__ uint32_t last_phase(int count, int of, int i) { return (uint32_t)(rounds(count, of, i) - 1) & 1u; }
// bytes that were announced and will not come
__device__ __forceinline__ void mbar_complete_tx(uint64_t* bar, uint32_t bytes) {
    asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}

// Issued by a converged warp, one lane of which is elected: a barrier's bytes
// to come, and a load that reports to it.
__device__ __forceinline__ void expect_warp(uint32_t bar, uint32_t bytes) {
    asm volatile(
        "{\n .reg .pred e;\n .reg .b32 r;\n elect.sync r|e, 0xffffffff;\n"
        " @e mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n}" ::"r"(bar),
        "r"(bytes)
        : "memory");
}

__device__ __forceinline__ void load_warp(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y) {
    asm volatile(
        "{\n .reg .pred e;\n .reg .b32 r;\n elect.sync r|e, 0xffffffff;\n"
        " @e cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];\n}" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

// Whether both barriers' phases are over, asked for together: an answer takes
// some 100 cycles. (It may wait a while for them.)
__device__ __forceinline__ bool both_ready(uint32_t bar, uint32_t phase, uint32_t bar2, uint32_t phase2) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p, q;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
        " mbarrier.try_wait.parity.shared::cta.b64 q, [%3], %4;\n and.pred p, p, q;\n selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(bar), "r"(phase), "r"(bar2), "r"(phase2)
        : "memory");
    return ok != 0;
}
// at once
__device__ __forceinline__ bool is_ready(uint32_t bar, uint32_t phase) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(bar), "r"(phase)
        : "memory");
    return ok != 0;
}

// four bytes from global memory, or zeros
__device__ __forceinline__ void copy4(float* to, const float* from, bool in) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(to)), "l"(from), "r"(in ? 4 : 0) : "memory");
}
// four values into shared memory of the cluster; 16 bytes are counted at `bar`
__device__ __forceinline__ void send4(uint32_t to, uint32_t bar, float x, float y, float z, float w) {
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(to),
                 "f"(x), "f"(y), "f"(z), "f"(w), "r"(bar)
                 : "memory");
}

// ---------------------------------------------------------------------------
// Few tokens. The 128 weight rows of a tile are the M dimension of the product
// and MT tokens its N dimension; a cluster of up to 8 CTAs shares a tile, each
// CTA with a part of the blocks of K. No workspace, no second launch: the CTAs
// send their sums to the cluster's shared memory (four tokens of a row at a
// time, to the CTA that joins them), where a barrier counts the bytes, and a
// CTA that has sent its own and joins none is done.
//
//   warp 0     TMA producer: a block of weights [128 x 128] and of tokens [MT x 128] a stage
//   warp 1     issues the products, into tensor memory buffers of MT columns in turn
//   warp 2     sx[m, b] * sw[b] of the tile's tokens into shared memory, four blocks at a time
//   warp 3     takes and frees tensor memory, lets the next kernel start
//   warps 4-7  thread = weight row: sum[m] += D[m] * scale[m]; join
//
// Bound by HBM where the weights are many, by the start, a block's chain and the
// join where they are few: 56 x 5120 x 17408 takes 20.2 to 20.5 us (4.5 TB/s, 66% of the
// measured rate: 240 CTAs on 152 SMs, so 88 of them have two), 1 x 4096 x 4096 4.6 us
// (8 blocks a CTA), of which 2.5 are the weights' time. A block takes 230 ns (16 tokens) to 460 (128),
// and rings of 7 to 11 stages, a second producer and scales read earlier change that
// by 3% at most: an SM takes in 63 to 80 bytes a ns, whatever the tokens.
// ---------------------------------------------------------------------------
constexpr int kTile = 128;
constexpr int kFewBatch = 4, kFewBatches = 3;
constexpr int kThreads = 256;
constexpr int kMostSplit = 8;

// the CTAs that may share a tile
constexpr int kSplits[] = {1, 2, 3, 4, 6, 8};
// groups of four tokens that a CTA of `split` joins at most
constexpr int groups_of(int mt, int split) { return (mt / 4 + split - 1) / split; }
constexpr int most_groups(int mt) {
    int most = 0;
    for (int s : kSplits) most = s > 1 && s * groups_of(mt, s) > most ? s * groups_of(mt, s) : most;
    return most;
}

template <int MT>
struct Few {
    static constexpr int kStage = kTile * kBlock + MT * kBlock;
    // two CTAs an SM (113 KB each), of the widest one
    static constexpr int kPerSm = MT == 128 ? 1 : 2;
    static constexpr int kStages = MT == 16 ? 5 : MT == 32 ? 4 : MT == 64 ? 3 : 4;
    static constexpr int kBufs = MT == 128 ? 2 : 4;
    static constexpr int kCols = kBufs * MT;   // 64, 128, 256, 256
    static constexpr int kPitch = MT + 4;      // floats of a block's scales
    static constexpr int kJoin = most_groups(MT) * kTile * 16;   // bytes
    static constexpr size_t kSmem = (size_t)kStages * kStage + kJoin + 1024;
    static_assert(kCols <= 256, "two CTAs share an SM's 512 columns");
};

struct FewArgs {
    const float* w_scales;
    const float* x_scales;
    void* out;
    int64_t M, N;
    int blocks;      // of K
    int m_chunks;
    int split;       // cluster size
    int until[2];    // loads of CTAs of even and odd rank end before this block
    int* status;
    long long spin_limit;
};

// A share of the registers of warps 0-3 goes to warps 4-7: 128 x 56 + 128 x 200 = 256 x 128.
// The four warps of a warpgroup execute this one instruction, ahead of their roles.
template <int MT>
__device__ __forceinline__ void give_registers() {
    if constexpr (MT == 128) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
}

template <typename T, int MT>
__global__ void __launch_bounds__(kThreads, 2) few_kernel(const __grid_constant__ CUtensorMap w_map,
                                                          const __grid_constant__ CUtensorMap x_map,
                                                          const __grid_constant__ FewArgs a) {
    using C = Few<MT>;
    extern __shared__ uint8_t dyn[];
    __shared__ __align__(8) uint64_t full[C::kStages], empty[C::kStages], d_full[C::kBufs], d_empty[C::kBufs];
    __shared__ __align__(8) uint64_t s_full[kFewBatches], s_empty[kFewBatches];
    __shared__ __align__(8) uint64_t tmem_ready, tmem_done, joined;
    __shared__ __align__(16) float scales[kFewBatches][kFewBatch][C::kPitch];
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;
    __shared__ int loads, products;   // issued
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn) + 1023) & ~(uintptr_t)1023);
    uint8_t* join = ring + C::kStages * C::kStage;   // [sender][group][row] of four sums

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)(blockIdx.x % (unsigned)a.split);
    const unsigned pair = blockIdx.x / (unsigned)a.split;
    const int64_t m0 = (int64_t)(pair % (unsigned)a.m_chunks) * MT;
    const int tile = (int)(pair / (unsigned)a.m_chunks);
    const int64_t n0 = (int64_t)tile * kTile;
    const int b0 = (int)((int64_t)a.blocks * rank / a.split), b1 = (int)((int64_t)a.blocks * (rank + 1) / a.split);
    const int count = b1 - b0;
    const int live = (int)min((int64_t)MT, a.M - m0);   // tokens of this chunk
    const int groups = (live + 3) / 4;
    const int own = groups > rank ? (groups - rank + a.split - 1) / a.split : 0;   // groups rank, rank + split, ...
    const Ctl ctl{a.status, a.spin_limit, &abort_flag};

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < C::kBufs; ++i) {
            mbar_init(&d_full[i], 1);
            mbar_init(&d_empty[i], 4);
        }
        for (int i = 0; i < kFewBatches; ++i) {
            mbar_init(&s_full[i], 32);
            mbar_init(&s_empty[i], 4);
        }
        mbar_init(&tmem_ready, 1);
        mbar_init(&tmem_done, 4);
        mbar_init(&joined, 1);
        abort_flag = loads = products = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        if (a.split > 1 && own > 0) mbar_arrive_expect_tx(&joined, (uint32_t)(a.split * own * kTile * 16));
    }
    __syncthreads();
    if (a.split > 1) cluster_arrive();   // (waited for before the first sum is sent)

    using S = typename T::storage;
    S* out = static_cast<S*>(a.out);
    bool freed = false;   // (of warp 3)

    if (warp < 4) {
        give_registers<MT>();
        if (warp == 0) {
            // the first stages' weights before the kernels ahead of this one have finished
            const uint32_t to = smem_u32(ring);
            const int bring = min(count, a.until[rank & 1]), first = min(bring, C::kStages);
            for (int i = 0; i < first; ++i) {
                expect_warp(smem_u32(&full[i]), C::kStage);
                load_warp(to + i * C::kStage, &w_map, smem_u32(&full[i]), (b0 + i) * kBlock, (int)n0);
            }
            pdl_wait();
            for (int i = 0; i < first; ++i)
                load_warp(to + i * C::kStage + kTile * kBlock, &x_map, smem_u32(&full[i]), (b0 + i) * kBlock, (int)m0);
            int slot = 0, i = first;
            uint32_t phase = 0;
            for (; i < bring; ++i) {
                if (!warp_wait(&empty[slot], phase, ctl)) break;
                const uint32_t st = to + slot * C::kStage;
                expect_warp(smem_u32(&full[slot]), C::kStage);
                load_warp(st, &w_map, smem_u32(&full[slot]), (b0 + i) * kBlock, (int)n0);
                load_warp(st + kTile * kBlock, &x_map, smem_u32(&full[slot]), (b0 + i) * kBlock, (int)m0);
                if (++slot == C::kStages) {
                    slot = 0;
                    phase ^= 1u;
                }
            }
            if (lane == 0) loads = i;
        } else if (warp == 1) {
            pdl_wait();   // (before every first wait with a limit: a kernel ahead may run for long)
            const bool ready = warp_wait(&tmem_ready, 0, ctl);
            fence_after();
            const uint32_t tmem = tmem_slot, from = smem_u32(ring);
            int slot = 0, buf = 0, i = 0;
            uint32_t phase = 0, d_phase = 1;   // (the first round finds every buffer free)
            for (; ready && i < count; ++i) {
                if (!__all_sync(0xffffffffu, both_ready(smem_u32(&full[slot]), phase, smem_u32(&d_empty[buf]), d_phase)) &&
                    !(warp_wait(&full[slot], phase, ctl) && warp_wait(&d_empty[buf], d_phase, ctl)))
                    break;
                fence_after();
                const uint32_t st = desc_lo(from + slot * C::kStage);
                block_products(tmem + buf * MT, st, st + (kTile * kBlock >> 4), idesc(kTile, MT), &empty[slot], &d_full[buf]);
                if (++slot == C::kStages) {
                    slot = 0;
                    phase ^= 1u;
                }
                if (++buf == C::kBufs) {
                    buf = 0;
                    d_phase ^= 1u;
                }
            }
            if (lane == 0) products = i;
        } else if (warp == 2) {
            pdl_wait();
            // Lanes: 4 blocks of K by 8 tokens. A batch is copied while the one before
            // it lands and is multiplied in place.
            const int k = lane & 3, i0 = lane >> 2;
            const int batches = (count + kFewBatch - 1) / kFewBatch;
            const float* sw = a.w_scales + (int64_t)tile * a.blocks + b0 + k;
            const float* sx = a.x_scales + (m0 + i0) * a.blocks + b0 + k;
            const auto start = [&](int j) {
                const bool in = j * kFewBatch + k < count;
                float* to = &scales[j % kFewBatches][k][i0];
#pragma unroll 4
                for (int t = 0; t < MT; t += 8) {
                    const bool there = in && t + i0 < live;
                    copy4(to + t, there ? sx + (int64_t)t * a.blocks + j * kFewBatch : a.x_scales, there);
                }
                asm volatile("cp.async.commit_group;" ::: "memory");
                return in ? sw[j * kFewBatch] : 0.f;
            };
            float w = start(0);
            for (int j = 0; j < batches; ++j) {
                float next = 0.f;
                if (j + 1 < batches) {
                    const int n = j + 1;
                    if (n >= kFewBatches &&
                        !warp_wait(&s_empty[n % kFewBatches], (uint32_t)(n / kFewBatches - 1) & 1u, ctl))
                        break;
                    next = start(n);
                    asm volatile("cp.async.wait_group 1;" ::: "memory");
                } else {
                    asm volatile("cp.async.wait_group 0;" ::: "memory");
                }
                float* mine = &scales[j % kFewBatches][k][i0];
#pragma unroll 4
                for (int t = 0; t < MT; t += 8) mine[t] *= w;
                mbar_arrive(&s_full[j % kFewBatches]);
                w = next;
            }
            asm volatile("cp.async.wait_all;" ::: "memory");   // (after a time-out, the next batch's)
        } else if (warp == 3) {
            // Tensor memory is taken after the kernels before this one have finished,
            // and the next one may start after it is taken; and it is free again
            // before the cluster's CTAs wait for each other's sums. So no CTA holds
            // columns while it waits for one that may need them.
            pdl_wait();
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_slot)),
                         "r"(C::kCols)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
            fence_before();
            pdl_launch_dependents();
            if (lane == 0) mbar_arrive(&tmem_ready);
            if (warp_wait(&tmem_done, 0, ctl)) {
                fence_after();
                asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_slot), "r"(C::kCols) : "memory");
                freed = true;
                // The other commits of the last products arrive before the CTA leaves.
                if (lane < min(count, C::kStages)) mbar_wait(&empty[lane], last_phase(count, C::kStages, lane), ctl);
                __syncwarp();
            }
        }
    } else {
        if constexpr (MT == 128) asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
        const int row = threadIdx.x & 127;
        const int64_t n = n0 + row;
        pdl_wait();
        bool ok = warp_wait(&tmem_ready, 0, ctl);
        fence_after();
        const uint32_t lanes = tmem_slot + ((uint32_t)(warp & 3) << 21);
        float sum[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m) sum[m] = 0.f;
        int buf = 0, batch = 0;
        uint32_t d_phase = 0, s_phase = 0;
        for (int i = 0; ok && i < count; ++i) {
            const int k = i % kFewBatch;
            if (k == 0 && !(ok = warp_wait(&s_full[batch], s_phase, ctl))) break;
            if (!(ok = warp_wait(&d_full[buf], d_phase, ctl))) break;
            fence_after();
            const float* sc = scales[batch][k];
            uint32_t d[2][16];
            tmem_ld16(lanes + buf * MT, d[0]);
#pragma unroll
            for (int c = 0; c < MT / 16; ++c) {
                float4 f[4];   // (asked for while the products are on their way)
#pragma unroll
                for (int t = 0; t < 4; ++t) f[t] = lds4(sc + 16 * c + 4 * t);
                tmem_ld_wait();
                if (c + 1 < MT / 16) {
                    tmem_ld16(lanes + buf * MT + 16 * (c + 1), d[(c + 1) & 1]);
                } else {
                    fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&d_empty[buf]);
                }
#pragma unroll
                for (int t = 0; t < 16; t += 4) {
                    const float4 s = f[t / 4];
                    sum[16 * c + t] = fmaf(as_f32(d[c & 1][t]), s.x, sum[16 * c + t]);
                    sum[16 * c + t + 1] = fmaf(as_f32(d[c & 1][t + 1]), s.y, sum[16 * c + t + 1]);
                    sum[16 * c + t + 2] = fmaf(as_f32(d[c & 1][t + 2]), s.z, sum[16 * c + t + 2]);
                    sum[16 * c + t + 3] = fmaf(as_f32(d[c & 1][t + 3]), s.w, sum[16 * c + t + 3]);
                }
            }
            if (++buf == C::kBufs) {
                buf = 0;
                d_phase ^= 1u;
            }
            if (k == kFewBatch - 1) {
                __syncwarp();
                if (lane == 0) mbar_arrive(&s_empty[batch]);
                if (++batch == kFewBatches) {
                    batch = 0;
                    s_phase ^= 1u;
                }
            }
        }
        fence_before();
        __syncwarp();
        if (ok && lane == 0) mbar_arrive(&tmem_done);
        if (a.split == 1) {
            if (n < a.N) {
#pragma unroll
                for (int m = 0; m < MT; ++m)
                    if (m < live) out[(m0 + m) * a.N + n] = T::from_f32(sum[m]);
            }
        } else {
            cluster_wait();   // every CTA's barriers are there
            const int slots = groups_of(MT, a.split);
            const uint32_t at = smem_u32(join) + (uint32_t)(rank * slots * kTile + row) * 16;
            int to = 0;
            uint32_t place = at;
#pragma unroll
            for (int q = 0; q < MT / 4; ++q) {
                if (4 * q < live)
                    send4(mapa(place, to), mapa(smem_u32(&joined), to), sum[4 * q], sum[4 * q + 1], sum[4 * q + 2], sum[4 * q + 3]);
                if (++to == a.split) {
                    to = 0;
                    place += kTile * 16;
                }
            }
            // what this CTA joins, in the order of the ranks
            if (own > 0 && warp_wait(&joined, 0, ctl)) {
                for (int q = 0; q < own; ++q) {
                    const float* from = reinterpret_cast<const float*>(join) + (q * kTile + row) * 4;
                    float4 s = lds4(from);
                    for (int r = 1; r < a.split; ++r) {
                        const float4 v = lds4(from + r * slots * kTile * 4);
                        s.x += v.x;
                        s.y += v.y;
                        s.z += v.z;
                        s.w += v.w;
                    }
                    const int m = 4 * (q * a.split + rank);
                    if (n < a.N) {
                        S* o = out + (m0 + m) * a.N + n;
                        o[0] = T::from_f32(s.x);
                        if (m + 1 < live) o[a.N] = T::from_f32(s.y);
                        if (m + 2 < live) o[2 * a.N] = T::from_f32(s.z);
                        if (m + 3 < live) o[3 * a.N] = T::from_f32(s.w);
                    }
                }
            }
        }
    }

    // What was issued lands before the CTA leaves; without a time-out it has: both
    // commits of the last products were waited for above, and so were the sums sent
    // to this CTA.
    __syncthreads();
    if (!abort_flag) return;
    if (threadIdx.x == 0) {
        for (int i = 0; i < min(loads, C::kStages); ++i)
            mbar_wait_drain(&full[i], last_phase(loads, C::kStages, i), a.spin_limit, a.status);
        for (int i = 0; i < min(products, C::kStages); ++i)
            mbar_wait_drain(&empty[i], last_phase(products, C::kStages, i), a.spin_limit, a.status);
        for (int i = 0; i < min(products, C::kBufs); ++i)
            mbar_wait_drain(&d_full[i], last_phase(products, C::kBufs, i), a.spin_limit, a.status);
    }
    fence_before();
    __syncthreads();
    fence_after();
    if (warp == 3 && !freed)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_slot), "r"(C::kCols) : "memory");
    if (a.split > 1) {
        // Every CTA sends its sums, whether they are whole or not. Those for this one may
        // still be on their way: after the others have sent theirs, or left, the barrier
        // that counts their bytes is waited for.
        if (warp < 4) cluster_wait();
        cluster_arrive();
        cluster_wait();
        if (threadIdx.x == 0 && own > 0) mbar_wait_drain(&joined, 0, a.spin_limit, a.status);
    }
}

template <typename... KArgs, typename... Args>
static cudaError_t launch_cluster(void (*kernel)(KArgs...), unsigned grid, unsigned block, size_t smem, unsigned cluster,
                                  cudaStream_t stream, const Args&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

static bool encode(CUtensorMap* map, CUtensorMapDataType type, const void* p, int64_t rows, int64_t cols, int64_t pitch,
                   int box_rows, int box_cols, CUtensorMapSwizzle swizzle) {
    auto fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)pitch};
    const cuuint32_t box[2] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows};
    const cuuint32_t one[2] = {1, 1};
    return fn(map, type, 2, const_cast<void*>(p), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// e4m3 rows as an operand: boxes of 128 columns
static bool make_map(CUtensorMap* map, const void* p, int64_t rows, int64_t cols, int box_rows) {
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, p, rows, cols, cols, box_rows, kBlock, CU_TENSOR_MAP_SWIZZLE_128B);
}
// outputs: boxes of 32 rows of `bytes`
template <typename T>
static bool make_out_map(CUtensorMap* map, const void* p, int64_t rows, int64_t cols, int bytes) {
    const CUtensorMapDataType type = T::kBytes == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_UINT16;
    return encode(map, type, p, rows, cols, cols * T::kBytes, 32, bytes / T::kBytes,
                  bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE);
}

// Shared memory of a kernel that hands registers over, on the current device.
// setmaxnreg.inc waits until it finds what it asks for, so the kernel must have
// been launched with `regs` registers a thread (the shares add up to that).
template <typename Kernel>
static cudaError_t prepare(Kernel kernel, size_t smem, bool (&done)[64], int dev, int regs, int carveout = -1) {
    if (done[dev]) return cudaSuccess;
    if (regs > 0) {
        cudaFuncAttributes f;
        const cudaError_t e = cudaFuncGetAttributes(&f, kernel);
        if (e != cudaSuccess) return e;
        if ((f.numRegs + 7) / 8 * 8 != regs) return cudaErrorInvalidDeviceFunction;
    }
    return allow_smem_once(kernel, smem, done, carveout);
}

template <typename T, int MT>
static cudaError_t few_prepare(int dev) {
    static bool done[64];
    return prepare(few_kernel<T, MT>, Few<MT>::kSmem, done, dev, MT == 128 ? 128 : 0, cudaSharedmemCarveoutMaxShared);
}

// How many clusters of a size find SMs of their own (a cluster lies within a part
// of the GPU, so not every SM takes part in large ones).
template <typename T, int MT>
static int clusters_at_once(int dev, int split) {
    static int known[64][kMostSplit + 1];
    if (known[dev][split] > 0) return known[dev][split];
    if (few_prepare<T, MT>(dev) != cudaSuccess) return std::max(1, num_sms() / split);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)split);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Few<MT>::kSmem;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)split;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, few_kernel<T, MT>, &cfg) != cudaSuccess || n < 1) {
        cudaGetLastError();
        n = std::max(1, num_sms() / split);
    }
    return known[dev][split] = n;
}

// The split that should end first, and when, in ns: a start and an end, which
// grow with the tokens; a block of K of a CTA that has an SM to itself, 1.4 times
// that where two share one, and 1.3 us more since the next call's CTAs then find
// no room to load their weights early; or HBM at 6.2 TB/s. Measured in us, split
// 1, 2, 3, 4, 6, 8 (16, 64, 16, 64, 64, 16 tokens at once):
//   1 x 4096 x 4096     10.1   7.0   5.5   4.6   6.2   6.7
//   64 x 2048 x 2048     9.2   7.0   6.1   5.2   4.7   6.3
//   16 x 14336 x 5120   16.6  16.6  17.3  16.9  18.1  20.5
//   33 x 5120 x 14336   43.0  24.6  19.1  20.4  17.3  21.3
//   56 x 5120 x 17408   52.0  29.8  23.1  23.7  20.5  25.3
//   16 x 256 x 16384    33.3  18.1  13.0  10.3   7.9   6.4
// and 16, 32, 64, 128 tokens at once, each with its best split:
//   128 x 361 x 256      2.3   2.8   3.9   6.3
//   64 x 1024 x 1024     2.7   3.1   3.7   4.2
//   40 x 4096 x 4096    10.0   8.1   6.9   7.9
//   2000 x 300 x 512     6.7   5.2   4.8   7.2
template <typename T, int MT>
static int64_t few_plan(const Fp8MmLaunch& L, int* split) {
    using C = Few<MT>;
    constexpr int64_t kBlockNs = MT == 16 ? 250 : MT == 32 ? 300 : MT == 64 ? 390 : 460;
    const int64_t clusters = (L.N + kTile - 1) / kTile * ((L.M + MT - 1) / MT);
    const int64_t blocks = (L.K + kBlock - 1) / kBlock, hbm = L.N * L.K / 6200;
    const int64_t ends = 2300 + 25 * std::min<int64_t>(L.M, MT);
    int64_t best = -1;
    for (int n : kSplits) {
        if (n > blocks) break;
        const int64_t alone = clusters_at_once<T, MT>(L.device, n), each = (blocks + n - 1) / n;
        const int64_t at_once = alone * C::kPerSm, rounds = (clusters + at_once - 1) / at_once;
        const int64_t cost = clusters <= alone
                                 ? ends + std::max(kBlockNs * each, hbm)
                                 : (ends + 1300) * rounds + std::max(kBlockNs * (C::kPerSm > 1 ? 14 : 10) / 10 * each * rounds, hbm);
        if (best < 0 || cost < best) {
            best = cost;
            *split = n;
        }
    }
    return best;
}

template <typename T, int MT>
static cudaError_t few_launch(const Fp8MmLaunch& L, int split, cudaStream_t s) {
    using C = Few<MT>;
    CUtensorMap w_map, x_map;
    if (!make_map(&w_map, L.w, L.N, L.K, kTile) || !make_map(&x_map, L.x, L.M, L.K, MT)) return cudaErrorInvalidValue;
    const cudaError_t e = few_prepare<T, MT>(L.device);
    if (e != cudaSuccess) return e;
    const int64_t tiles = (L.N + kTile - 1) / kTile, chunks = (L.M + MT - 1) / MT;
    if (tiles * chunks * split > 0x7fffffff) return cudaErrorInvalidConfiguration;
    const FewArgs a{L.w_scales, L.x_scales, L.out, L.M, L.N, (int)((L.K + kBlock - 1) / kBlock), (int)chunks, split,
                    {std::min(L.until[0][0], L.until[0][1]), std::min(L.until[1][0], L.until[1][1])}, L.status, L.spin_limit};
    return launch_cluster(few_kernel<T, MT>, (unsigned)(tiles * chunks * split), kThreads, C::kSmem, (unsigned)split, s,
                          w_map, x_map, a);
}

// ---------------------------------------------------------------------------
// Many tokens. Two CTAs on neighbouring SMs share a tile of 256 tokens x NT
// weight rows (cta_group::2): each brings 128 tokens and half of the weight
// rows into its shared memory, and the products read both halves, so a block of
// K costs an SM (128 + NT / 2) x 128 bytes of loads for 128 x NT x 128 products.
// The pairs walk over the tiles, with the ring and the tensor memory buffers
// running on from tile to tile.
//
//   warp 0      TMA producer of the CTA's weight rows
//   warp 2      TMA producer of its tokens; copies the scales of the tokens and of
//               the tile's weight blocks, kBatch blocks of K at a time
//   warps 1, 3  (first CTA) issue the products for the pair, each with half of the
//               weight rows (warp 3 also allocates tensor memory and lets the next
//               kernel start)
//   warps 4-11  thread = token, half of the tile's columns (one product's):
//               sum[n] += D[n] * (sx sw), one factor for all of them
// Two producers and two issuers, since a block of K is 512 cycles of products,
// and waits, a load and an issue take a warp some 150 to 250 cycles each.
//
// 8192 x 14336 x 5120 takes 437 us at full clocks (2.75 PFLOP/s; 471 to 498 where the
// power limit lowers them): 850 cycles a block of K. Without the multiplications
// they are 730, so most of the rest is a tensor memory buffer's round trip (commit,
// wait, read, arrivals from both CTAs, wait): with two of each half the 512 columns
// are full. Measured no faster: whole products of 256 rows with issuers in turn
// (439), packed pairs of multiplications (447), 32 or 64 columns at a time (438 to
// 443), polling instead of waiting issuers (465), 16 scaling warps (525).
// ---------------------------------------------------------------------------
constexpr int kSumWarps = 8;
constexpr int kPairThreads = 32 * (4 + kSumWarps);
constexpr int kPairRows = 256;
constexpr int kBatch = 8;
// 384 threads x 168 registers = 128 x 72 + 256 x 216
constexpr int kLaunchRegs = 168, kControlRegs = 72, kSumRegs = 216;
static_assert(kPairThreads * kLaunchRegs == 128 * kControlRegs + 32 * kSumWarps * kSumRegs, "");

constexpr int kOutBox = 32 * 128;   // bytes of a warp: 32 rows of 128

template <int NT>
struct Many {
    static constexpr int kStage = kTile * kBlock + NT / 2 * kBlock;   // of one CTA
    static constexpr int kStages = NT == 256 ? 5 : 6;
    static constexpr int kCols = NT / 2;        // columns of a product, and of a thread
    static constexpr int kPart = NT / 4;        // of them from one CTA's weight rows
    static constexpr int kBufs = 2;             // of each half
    static constexpr int kOutBytes = NT == 256 ? 128 : 96;   // of a row in a stored box
    static constexpr size_t kSmem = (size_t)kStages * kStage + kSumWarps * kOutBox + 1024;
    static_assert(2 * kBufs * kCols <= 512 && kPart * kBlock % 1024 == 0 && kPart % 16 == 0, "");
};

struct ManyArgs {
    const float* w_scales;
    const float* x_scales;
    void* out;
    int64_t M, N;
    int blocks;                 // of K
    int tiles_m, tiles_n;
    int pairs;
    int aligned;                // rows of out start on 16-byte boundaries: out_map is there
    int until[2][2];            // loads of a CTA's weights and tokens end before this block
    int* status;
    long long spin_limit;
};

// tiles in strips of 8 tiles of tokens: the pairs' operands of a moment stay in L2
constexpr int kStrip = 8;
__device__ __forceinline__ void tile_at(const ManyArgs& a, int t, int& tm, int& tn) {
    const int strip = t / (kStrip * a.tiles_n), first = strip * kStrip;
    const int height = min(kStrip, a.tiles_m - first), r = t - first * a.tiles_n;
    tm = first + r % height;
    tn = r / height;
}

// Both CTAs' loads report to the first CTA's barrier. Issued by a converged
// warp, one lane of which is elected.
__device__ __forceinline__ void pair_load(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y) {
    asm volatile(
        "{\n .reg .pred e;\n .reg .b32 r;\n elect.sync r|e, 0xffffffff;\n"
        " @e cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3}], "
        "[%4];\n}" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
// as block_products, for both CTAs of the pair; the commits reach both
__device__ __forceinline__ void pair_products(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t id, uint64_t* slot_free,
                                              uint64_t* done) {
    asm volatile(
        "{\n .reg .pred e, z, o;\n .reg .b32 r, t, u;\n .reg .b64 x, y;\n .reg .b16 m;\n elect.sync r|e, 0xffffffff;\n"
        " setp.ne.b32 z, 0, 0;\n setp.eq.b32 o, 0, 0;\n mov.b16 m, 3;\n"
        " mov.b64 x, {%1, %4};\n mov.b64 y, {%2, %4};\n"
        " @e tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], x, y, %3, z;\n"
        " add.u32 u, %1, 2;\n mov.b64 x, {u, %4};\n add.u32 t, %2, 2;\n mov.b64 y, {t, %4};\n"
        " @e tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], x, y, %3, o;\n"
        " add.u32 u, %1, 4;\n mov.b64 x, {u, %4};\n add.u32 t, %2, 4;\n mov.b64 y, {t, %4};\n"
        " @e tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], x, y, %3, o;\n"
        " add.u32 u, %1, 6;\n mov.b64 x, {u, %4};\n add.u32 t, %2, 6;\n mov.b64 y, {t, %4};\n"
        " @e tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], x, y, %3, o;\n"
        " @e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%5], m;\n"
        " @e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%6], m;\n}" ::"r"(d),
        "r"(a_lo), "r"(b_lo), "r"(id), "r"(kDescHi), "r"(smem_u32(slot_free)), "r"(smem_u32(done))
        : "memory");
}

__device__ __forceinline__ void arrive_at(uint32_t cluster_bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}

// column within the tile of column c of a product: NT / 4 columns are weight
// rows of the first CTA, the others of the second, NT / 2 further
template <int NT>
__device__ __forceinline__ int column(int half, int c) {
    return c / (NT / 4) * (NT / 2) + half * (NT / 4) + c % (NT / 4);
}

// place of byte `b` of row r in a box of stored rows
template <int kBytes>
__device__ __forceinline__ uint32_t boxed(int r, int b) {
    return r * kBytes + (kBytes == 128 ? ((b >> 4 ^ (r & 7)) << 4 | (b & 15)) : b);
}

__device__ __forceinline__ void store_box(const CUtensorMap* map, uint32_t src, int x, int y) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];\n"
                 "cp.async.bulk.commit_group;" ::"l"(map),
                 "r"(x), "r"(y), "r"(src)
                 : "memory");
}

// Scales of kBatch blocks of K, from kb on, by a warp: rows m on of the
// activations, block rows wr and wr + 1 of the weights; zeros outside. The
// copies' completion arrives at `bar` (32 arrivals).
__device__ __forceinline__ void copy_scales(const ManyArgs& a, int m, int wr, int w_rows, int kb, float (*sx)[kTile + 4],
                                            float (*sw)[2], uint64_t* bar) {
    const int lane = threadIdx.x & 31, k = lane & 7, i = lane >> 3;   // 8 blocks by 4 rows
    const bool in = kb + k < a.blocks;
    const int rows = in ? (int)min((int64_t)kTile, a.M - m) - i : 0;
    const float* from = in ? a.x_scales + (int64_t)(m + i) * a.blocks + kb + k : a.x_scales;
#pragma unroll 4
    for (int r = 0; r < kTile; r += 4) copy4(&sx[k][r + i], r < rows ? from + (int64_t)r * a.blocks : a.x_scales, r < rows);
    const bool w_in = in && i < 2 && wr + i < w_rows;
    if (i < 2) copy4(&sw[k][i], w_in ? a.w_scales + (int64_t)(wr + i) * a.blocks + kb + k : a.w_scales, w_in);
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// what a CTA has issued, blocks of K or batches of scales
struct Issued {
    int loads[2];      // of weights, of tokens
    int products[2];   // of the halves
    int batches;
};

template <typename T, int NT>
__global__ void __launch_bounds__(kPairThreads, 1) many_kernel(const __grid_constant__ CUtensorMap w_map,
                                                               const __grid_constant__ CUtensorMap x_map,
                                                               const __grid_constant__ CUtensorMap out_map,
                                                               const __grid_constant__ ManyArgs a) {
    using C = Many<NT>;
    extern __shared__ uint8_t dyn[];
    __shared__ __align__(8) uint64_t full[C::kStages], empty[C::kStages], d_full[2][C::kBufs], d_empty[2][C::kBufs];
    __shared__ __align__(8) uint64_t s_full[2], s_empty[2];
    __shared__ __align__(8) uint64_t tmem_ready;
    __shared__ float sx[2][kBatch][kTile + 4], sw[2][kBatch][2];
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;
    __shared__ Issued issued;
    __shared__ int gave_up;   // one of the two CTAs
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn) + 1023) & ~(uintptr_t)1023);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)(blockIdx.x & 1u), pair = (int)(blockIdx.x >> 1);
    const int tiles = a.tiles_m * a.tiles_n;
    const Ctl ctl{a.status, a.spin_limit, &abort_flag};

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 2);   // both halves' products
        }
        for (int i = 0; i < 2 * C::kBufs; ++i) {
            mbar_init(&d_full[0][i], 1);
            mbar_init(&d_empty[0][i], kSumWarps);   // half of each CTA's
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 32);
            mbar_init(&s_empty[i], kSumWarps);
        }
        mbar_init(&tmem_ready, 2);
        abort_flag = gave_up = 0;
        issued = Issued{};
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    cluster_arrive();   // the other CTA reports to these barriers
    cluster_wait();

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kControlRegs));
        const uint32_t lead = mapa(smem_u32(full), 0);   // the first CTA's barriers
        if (warp == 0) {
            const uint32_t to = smem_u32(ring) + kTile * kBlock;
            const int until = a.until[rank][0];
            int slot = 0, g = 0;
            uint32_t phase = 1;   // (the first round finds every slot free)
            bool ok = true;
            for (int t = pair; ok && t < tiles; t += a.pairs) {
                int tm, tn;
                tile_at(a, t, tm, tn);
                const int n = tn * NT + rank * (NT / 2);
                const int end = min(a.blocks, until - g);
                for (int kb = 0; kb < end; ++kb, ++g) {
                    if (g == C::kStages) pdl_wait();   // (as in few_kernel)
                    if (g >= C::kStages && !(ok = warp_wait(&empty[slot], phase, ctl))) break;
                    if (rank == 0) expect_warp(smem_u32(&full[slot]), 2 * C::kStage);
                    pair_load(to + slot * C::kStage, &w_map, lead + 8 * slot, kb * kBlock, n);
                    if (++slot == C::kStages) {
                        slot = 0;
                        phase ^= 1u;
                    }
                }
                if (end < a.blocks) break;
            }
            if (lane == 0) issued.loads[0] = g;
        } else if (warp == 2) {
            pdl_wait();
            const uint32_t to = smem_u32(ring);
            const int until = a.until[rank][1];
            const int w_rows = (int)((a.N + kBlock - 1) / kBlock);
            int slot = 0, g = 0, j = 0;
            uint32_t phase = 1;
            bool ok = true;
            for (int t = pair; ok && t < tiles; t += a.pairs) {
                int tm, tn;
                tile_at(a, t, tm, tn);
                const int m = tm * kPairRows + rank * kTile;
                const int end = min(a.blocks, until - g);
                for (int kb = 0; kb < end; ++kb, ++g) {
                    if (kb % kBatch == 0) {
                        if (j >= 2 && !(ok = warp_wait(&s_empty[j & 1], (uint32_t)(j / 2 - 1) & 1u, ctl))) break;
                        copy_scales(a, m, (int)((int64_t)tn * NT / kBlock), w_rows, kb, sx[j & 1], sw[j & 1], &s_full[j & 1]);
                        ++j;
                    }
                    if (g >= C::kStages && !(ok = warp_wait(&empty[slot], phase, ctl))) break;
                    pair_load(to + slot * C::kStage, &x_map, lead + 8 * slot, kb * kBlock, m);
                    if (++slot == C::kStages) {
                        slot = 0;
                        phase ^= 1u;
                    }
                }
                if (end < a.blocks) break;
            }
            if (lane == 0) {
                issued.loads[1] = g;
                issued.batches = j;
            }
        } else {
            if (warp == 3) {
                // (the order of these: see few_kernel)
                pdl_wait();
                asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&tmem_slot))
                             : "memory");
                asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
                fence_before();
                pdl_launch_dependents();
                // both CTAs' columns are there before the first product
                if (lane < 2) arrive_at(mapa(smem_u32(&tmem_ready), lane));
                __syncwarp();
            }
            if (rank == 0) {
                pdl_wait();
                bool ok = warp_wait(&tmem_ready, 0, ctl);
                fence_after();
                const uint32_t tmem = tmem_slot, from = smem_u32(ring);
                // warp 1 takes the first half of both CTAs' weight rows, warp 3 the second
                const int half = warp >> 1;
                const int total = (tiles - pair + a.pairs - 1) / a.pairs * a.blocks;
                int slot = 0, buf = 0, g = 0;
                uint32_t phase = 0, d_phase = 1;
                for (; ok && g < total; ++g) {
                    // (the first round finds every buffer free: a barrier's phase before its first is over)
                    if (!__all_sync(0xffffffffu, both_ready(smem_u32(&full[slot]), phase, smem_u32(&d_empty[half][buf]), d_phase)) &&
                        !(ok = warp_wait(&full[slot], phase, ctl) && warp_wait(&d_empty[half][buf], d_phase, ctl)))
                        break;
                    fence_after();
                    const uint32_t st = desc_lo(from + slot * C::kStage);
                    pair_products(tmem + (2 * buf + half) * C::kCols, st, st + (kTile * kBlock + half * C::kPart * kBlock >> 4),
                                  idesc(kPairRows, C::kCols), &empty[slot], &d_full[half][buf]);
                    if (++slot == C::kStages) {
                        slot = 0;
                        phase ^= 1u;
                    }
                    if (++buf == C::kBufs) {
                        buf = 0;
                        d_phase ^= 1u;
                    }
                }
                if (lane == 0) issued.products[half] = g;
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSumRegs));
        using S = typename T::storage;
        constexpr int kPart = C::kPart, kChunk = 16;
        const int half = (warp - 4) >> 2;
        const int row = (warp & 3) * 32 + lane;
        pdl_wait();
        bool ok = warp_wait(&tmem_ready, 0, ctl);
        fence_after();
        const uint32_t mine = tmem_slot + ((uint32_t)(warp & 3) << 21) + half * C::kCols;
        const uint32_t sx_at = smem_u32(&sx[0][0][row]), sw_at = smem_u32(&sw[0][0][0]);
        const uint32_t filled = smem_u32(&d_full[half][0]), released = mapa(smem_u32(&d_empty[half][0]), 0);
        const uint32_t box = smem_u32(ring) + C::kStages * C::kStage + (warp - 4) * kOutBox;
        int buf = 0, batch = 0;
        uint32_t d_phase = 0, s_phase = 0;
        bool ready = false;   // the next buffer is known to be filled
        for (int t = pair; ok && t < tiles; t += a.pairs) {
            float sum[C::kCols];
#pragma unroll
            for (int i = 0; i < C::kCols; ++i) sum[i] = 0.f;
            int tm, tn;
            tile_at(a, t, tm, tn);
            uint32_t second = 0;   // chunks in the second weight block that the tile touches
            if constexpr (NT != 256) {
#pragma unroll
                for (int c = 0; c < C::kCols / kChunk; ++c)
                    second |= (tn * NT % kBlock + column<NT>(half, kChunk * c)) / kBlock << c;
            }
            for (int k0 = 0; ok && k0 < a.blocks; k0 += kBatch) {
                if (!(ok = warp_wait(&s_full[batch], s_phase, ctl))) break;
                const int n = min(kBatch, a.blocks - k0);
                uint32_t xs = sx_at + batch * (kBatch * (kTile + 4) * 4), ws = sw_at + batch * (kBatch * 8);
                float x = lds1(xs), w0 = lds1(ws), w1 = lds1(ws + 4);
                for (int k = 0; k < n; ++k) {
                    if (!ready && !(ok = warp_wait(&d_full[half][buf], d_phase, ctl))) break;
                    fence_after();
                    const uint32_t at = mine + buf * NT;
                    const float s0 = x * w0, s1 = x * w1;
                    uint32_t d[2][kChunk];
                    tmem_ld16(at, d[0]);
#pragma unroll
                    for (int c = 0; c < C::kCols / kChunk; ++c) {
                        tmem_ld_wait();
                        if (c + 1 < C::kCols / kChunk) {
                            tmem_ld16(at + kChunk * (c + 1), d[(c + 1) & 1]);
                        } else {
                            // the buffer goes back, and what the next block needs is
                            // asked for, before the last products
                            fence_before();
                            __syncwarp();
                            if (lane == 0) arrive_at(released + 8 * buf);
                            if (++buf == C::kBufs) {
                                buf = 0;
                                d_phase ^= 1u;
                            }
                            ready = is_ready(filled + 8 * buf, d_phase);
                            if (k + 1 < n) {
                                xs += (kTile + 4) * 4;
                                ws += 8;
                            }
                            x = lds1(xs);
                            w0 = lds1(ws);
                            w1 = lds1(ws + 4);
                        }
                        // the weight block of 16 columns: that of their CTA's rows, or by place
                        const float f = NT == 256 ? (kChunk * c < kPart ? s0 : s1) : (second >> c & 1) ? s1 : s0;
#pragma unroll
                        for (int i = 0; i < kChunk; ++i)
                            sum[kChunk * c + i] = fmaf(as_f32(d[c & 1][i]), f, sum[kChunk * c + i]);
                    }
                    ready = __all_sync(0xffffffffu, ready);
                }
                if (lane == 0) mbar_arrive(&s_empty[batch]);   // (what was read last has arrived: the vote)
                batch ^= 1;
                if (batch == 0) s_phase ^= 1u;
            }
            if (!ok) break;
            const int64_t m0 = (int64_t)tm * kPairRows + rank * kTile + (warp & 3) * 32;
            if (m0 >= a.M) continue;
            // 128 (96) bytes of the warp's rows at a time through shared memory: by
            // a TMA store, which cuts off what lies beyond the matrix, or where rows
            // are not aligned for that, row after row. Rows of 128 bytes are
            // swizzled, those of 96 spread over the banks as they are.
            constexpr int kEach = C::kOutBytes / T::kBytes;
            const int rows = (int)min((int64_t)32, a.M - m0);
#pragma unroll
            for (int c = 0; c < C::kCols; c += kEach) {
                const int64_t n = (int64_t)tn * NT + column<NT>(half, c);
                if (n >= a.N) continue;
                if (a.aligned && lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                __syncwarp();
#pragma unroll
                for (int i = 0; i < C::kOutBytes / 16; ++i) {
                    uint32_t w[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if constexpr (T::kBytes == 4)
                            w[j] = __float_as_uint(sum[c + 4 * i + j]);
                        else
                            w[j] = pack16<T>(sum[c + 8 * i + 2 * j], sum[c + 8 * i + 2 * j + 1]);
                    }
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(box + boxed<C::kOutBytes>(lane, 16 * i)),
                                 "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                                 : "memory");
                }
                if (a.aligned) {
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) store_box(&out_map, box, (int)n, (int)m0);
                    continue;
                }
                __syncwarp();
                const uint8_t* from = ring + C::kStages * C::kStage + (warp - 4) * kOutBox;
                const int cols = (int)min((int64_t)kEach, a.N - n);
                S* out = static_cast<S*>(a.out) + m0 * a.N + n;
#pragma unroll 4
                for (int r = 0; r < rows; ++r, out += a.N)
#pragma unroll
                    for (int e = 0; e < kEach; e += 32)
                        if (e + lane < cols)
                            out[e + lane] = *reinterpret_cast<const S*>(from + boxed<C::kOutBytes>(r, (e + lane) * T::kBytes));
            }
        }
        __syncwarp();
        if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        __syncwarp();
    }

    // What was issued lands before the CTAs leave. Without a time-out it has but for
    // the other commits of the last products, which a thread each waits for. After one,
    // both CTAs learn of it, and of how much each of them has issued.
    __syncthreads();
    if (abort_flag) {
        if (threadIdx.x < 2) store_at(mapa(smem_u32(&gave_up), threadIdx.x), 1);
    } else {
        const int fills = (tiles - pair + a.pairs - 1) / a.pairs * a.blocks;
        if (threadIdx.x < min(fills, C::kStages))
            mbar_wait_drain(&empty[threadIdx.x], last_phase(fills, C::kStages, threadIdx.x), a.spin_limit, a.status);
    }
    fence_before();
    __syncthreads();
    cluster_arrive();
    cluster_wait();
    if (gave_up) {
        if (threadIdx.x == 0) {
            int loads[2][2], products[2];
            for (int i = 0; i < 2; ++i) {
                for (int r = 0; r < 2; ++r) loads[r][i] = load_at(mapa(smem_u32(&issued.loads[i]), r));
                products[i] = load_at(mapa(smem_u32(&issued.products[i]), 0));
            }
            for (int i = 0; rank == 0 && i < C::kStages; ++i) {
                // Of the stage's last round, the loads that were not issued are counted as
                // having landed; or, if it was the weights' load that announces the bytes, the
                // others are announced.
                constexpr int kBytes[2] = {NT / 2 * kBlock, kTile * kBlock};
                int round = 0, bytes = 0;
                for (int l = 0; l < 4; ++l) round = max(round, rounds(loads[l >> 1][l & 1], C::kStages, i));
                if (round == 0) continue;
                for (int l = 0; l < 4; ++l)
                    bytes += rounds(loads[l >> 1][l & 1], C::kStages, i) == round ? kBytes[l & 1] : 0;
                if (rounds(loads[0][0], C::kStages, i) < round)
                    mbar_arrive_expect_tx(&full[i], (uint32_t)bytes);
                else if (bytes < 2 * C::kStage)
                    mbar_complete_tx(&full[i], (uint32_t)(2 * C::kStage - bytes));
                mbar_wait_drain(&full[i], (uint32_t)(round - 1) & 1u, a.spin_limit, a.status);
            }
            for (int i = 0; i < C::kStages; ++i) {   // (the same for the two halves' products)
                const int r0 = rounds(products[0], C::kStages, i), r1 = rounds(products[1], C::kStages, i);
                if (max(r0, r1) == 0) continue;
                if (r0 != r1) mbar_arrive(&empty[i]);
                mbar_wait_drain(&empty[i], (uint32_t)(max(r0, r1) - 1) & 1u, a.spin_limit, a.status);
            }
            for (int i = 0; i < 2 * C::kBufs; ++i) {
                const int n = products[i / C::kBufs], b = i % C::kBufs;
                if (n > b) mbar_wait_drain(&d_full[i / C::kBufs][b], last_phase(n, C::kBufs, b), a.spin_limit, a.status);
            }
            for (int i = 0; i < min(issued.batches, 2); ++i)
                mbar_wait_drain(&s_full[i], last_phase(issued.batches, 2, i), a.spin_limit, a.status);
        }
        __syncthreads();
        cluster_arrive();
        cluster_wait();
    }
    fence_after();
    if (warp == 3)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem_slot) : "memory");
    cluster_arrive();
    cluster_wait();
}

template <typename T, int NT>
static cudaError_t many_launch(const Fp8MmLaunch& L, cudaStream_t s) {
    using C = Many<NT>;
    const int aligned = (L.N * T::kBytes) % 16 == 0 && (uintptr_t)L.out % 16 == 0;
    CUtensorMap w_map, x_map, out_map = {};
    if (!make_map(&w_map, L.w, L.N, L.K, NT / 2) || !make_map(&x_map, L.x, L.M, L.K, kTile) ||
        (aligned && !make_out_map<T>(&out_map, L.out, L.M, L.N, C::kOutBytes)))
        return cudaErrorInvalidValue;
    static bool done[64];
    const cudaError_t e = prepare(many_kernel<T, NT>, C::kSmem, done, L.device, kLaunchRegs);
    if (e != cudaSuccess) return e;
    const int64_t tm = (L.M + kPairRows - 1) / kPairRows, tn = (L.N + NT - 1) / NT;
    const int pairs = (int)std::min<int64_t>(tm * tn, num_sms() / 2);
    // (a pair counts its blocks of K in 32 bits)
    if (tm * tn > 0x7fffffff - 4096 || (tm * tn + pairs - 1) / pairs * ((L.K + kBlock - 1) / kBlock) > 0x7fffffff)
        return cudaErrorInvalidConfiguration;
    const ManyArgs a{L.w_scales, L.x_scales, L.out, L.M, L.N, (int)((L.K + kBlock - 1) / kBlock), (int)tm, (int)tn, pairs,
                     aligned, {{L.until[0][0], L.until[0][1]}, {L.until[1][0], L.until[1][1]}}, L.status, L.spin_limit};
    return launch_cluster(many_kernel<T, NT>, 2 * (unsigned)pairs, kPairThreads, C::kSmem, 2, s, w_map, x_map, out_map, a);
}

// The pairs are taken to need 5.5 us and 0.455 us a block of K and round of tiles
// with 256 weight rows, 0.42 us with 192 (8192 x 14336 x 5120: 24 rounds in 471 us,
// 32 in 510; 1111 x 5000 x 14416: 2 rounds in 110, 2 in 94, so that 192 rows need 0.39
// to 0.40). Whatever should end first is taken; few / many in us: 128 x 4096 x 4096
// 10.3 / 16.5, 256 x 4096 x 4096 13.9 / 16.7, 512 x 4096 x 4096 20.3 / 17.0, 256 x 14336
// x 5120 41 / 24, 512 x 1024 x 8192 13.4 / 28.
struct Form {
    int which;   // of kTiles
    int ctas;    // that share a tile
};
constexpr int kTiles[][2] = {{16, 128}, {32, 128}, {64, 128}, {128, 128}, {256, 192}, {256, 256}};   // tokens, weight rows

template <typename T>
static Form choose(const Fp8MmLaunch& L) {
    int split[] = {1, 1, 1, 1, 2, 2};
    int64_t least = few_plan<T, 16>(L, &split[0]);
    int choice = 0;
    const auto offer = [&](int c, int64_t cost) {
        if (cost < least) {
            least = cost;
            choice = c;
        }
    };
    if (L.M > 16) offer(1, few_plan<T, 32>(L, &split[1]));
    if (L.M > 32) offer(2, few_plan<T, 64>(L, &split[2]));
    if (L.M > 64) {
        offer(3, few_plan<T, 128>(L, &split[3]));
        const int64_t tm = (L.M + kPairRows - 1) / kPairRows, pairs = num_sms() / 2, blocks = (L.K + kBlock - 1) / kBlock;
        const auto rounds = [&](int nt) { return (tm * ((L.N + nt - 1) / nt) + pairs - 1) / pairs; };
        offer(4, 5500 + 420 * blocks * rounds(192));
        offer(5, 5500 + 455 * blocks * rounds(256));
    }
    return {choice, split[choice]};
}

template <typename T>
static cudaError_t typed(const Fp8MmLaunch& L, cudaStream_t s) {
    const Form f = choose<T>(L);
    switch (f.which) {
    case 0: return few_launch<T, 16>(L, f.ctas, s);
    case 1: return few_launch<T, 32>(L, f.ctas, s);
    case 2: return few_launch<T, 64>(L, f.ctas, s);
    case 3: return few_launch<T, 128>(L, f.ctas, s);
    case 4: return many_launch<T, 192>(L, s);
    default: return many_launch<T, 256>(L, s);
    }
}

}  // namespace fp8mm

cudaError_t launch_fp8_mm(const Fp8MmLaunch& L, int dtype, cudaStream_t s) {
    switch (dtype) {
    case GAI4_F16: return fp8mm::typed<F16>(L, s);
    case GAI4_F32: return fp8mm::typed<F32>(L, s);
    default: return fp8mm::typed<BF16>(L, s);
    }
}

void plan_fp8_mm(const Fp8MmLaunch& L, int dtype, int* tokens, int* weight_rows, int* ctas) {
    const fp8mm::Form f = dtype == GAI4_F16   ? fp8mm::choose<F16>(L)
                          : dtype == GAI4_F32 ? fp8mm::choose<F32>(L)
                                              : fp8mm::choose<BF16>(L);
    *tokens = fp8mm::kTiles[f.which][0];
    *weight_rows = fp8mm::kTiles[f.which][1];
    *ctas = f.ctas;
}

}  // namespace gai4
