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

// (a, b) += (x * s, y * t): one packed instruction
__device__ __forceinline__ void fma2(float& a, float& b, uint32_t x, uint32_t y, float s, float t) {
    asm("{\n .reg .b64 u, v, w;\n mov.b64 u, {%2, %3};\n mov.b64 v, {%4, %5};\n mov.b64 w, {%0, %1};\n"
        " fma.rn.f32x2 w, u, v, w;\n mov.b64 {%0, %1}, w;\n}"
        : "+f"(a), "+f"(b)
        : "r"(x), "r"(y), "f"(s), "f"(t));
}

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
__device__ __forceinline__ float ld_cluster(uint32_t a) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}

// ---------------------------------------------------------------------------
// Few tokens. The 128 weight rows of a tile are the M dimension of the product
// and MT tokens its N dimension; a cluster of up to 8 CTAs shares a tile, each
// CTA with a part of the blocks of K, and joins its sums through distributed
// shared memory in a fixed order: no workspace, no second launch.
//
//   warp 0     TMA producer: a block of weights [128 x 128] and of tokens [MT x 128] a stage
//   warp 1     issues the products, into tensor memory buffers of MT columns in turn
//   warp 2     sx[m, b] * sw[b] of the tile's tokens into shared memory, kBatch blocks at a time
//   warp 3     allocates tensor memory, lets the next kernel start
//   warps 4-7  thread = weight row: sum[m] += D[m] * scale[m]
// ---------------------------------------------------------------------------
constexpr int kTile = 128;
constexpr int kBatch = 8;
constexpr int kThreads = 256;

template <int MT>
struct Few {
    static constexpr int kStage = kTile * kBlock + MT * kBlock;
    // two CTAs an SM
    static constexpr int kStages = MT == 16 ? 6 : MT == 32 ? 5 : MT == 64 ? 4 : 3;
    static constexpr int kBufs = MT == 128 ? 2 : 4;
    static constexpr int kCols = kBufs * MT;   // 64, 128, 256, 256
    static constexpr int kPitch = MT + 4;      // floats of a block's scales
    static constexpr size_t kSmem = (size_t)kStages * kStage + 1024;
    static_assert(kCols <= 256, "two CTAs share an SM's 512 columns");
    static_assert(kStages * kStage >= kTile * MT * 4, "the ring takes the sums at the end");
};

struct FewArgs {
    const float* w_scales;
    const float* x_scales;
    void* out;
    int64_t M, N;
    int blocks;      // of K
    int m_chunks;
    int split;       // cluster size
    int* status;
    long long spin_limit;
};

// a share of warps 0-3 goes to warps 4-7: 128 x 56 + 128 x 200 = 256 x 128
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
    __shared__ __align__(8) uint64_t s_full[2], s_empty[2];
    __shared__ __align__(16) float scales[2][kBatch][C::kPitch];
    __shared__ __align__(8) uint64_t tmem_ready;
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;
    __shared__ int loads, products;   // issued
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn) + 1023) & ~(uintptr_t)1023);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)(blockIdx.x % (unsigned)a.split);
    const unsigned pair = blockIdx.x / (unsigned)a.split;
    const int64_t m0 = (int64_t)(pair % (unsigned)a.m_chunks) * MT;
    const int tile = (int)(pair / (unsigned)a.m_chunks);
    const int64_t n0 = (int64_t)tile * kTile;
    const int b0 = (int)((int64_t)a.blocks * rank / a.split), b1 = (int)((int64_t)a.blocks * (rank + 1) / a.split);
    const int count = b1 - b0;
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
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 32);
            mbar_init(&s_empty[i], 4);
        }
        mbar_init(&tmem_ready, 1);
        abort_flag = loads = products = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();

    using S = typename T::storage;
    S* out = static_cast<S*>(a.out);
    const int row = threadIdx.x & 127;
    const int64_t n = n0 + row;
    const int live = (int)min((int64_t)MT, a.M - m0);   // tokens of this chunk
    float* mine = reinterpret_cast<float*>(ring);       // the CTA's sums in the end, [token][row]

    // 128 sums a thread: the registers go to the warps that hold them
    if (warp == 0) {
        give_registers<MT>();
        if (lane == 0) {
            // the first stages' weights before the kernels ahead of this one have finished
            const int first = min(count, C::kStages);
            for (int i = 0; i < first; ++i) {
                mbar_arrive_expect_tx(&full[i], C::kStage);
                tma_load_2d(ring + i * C::kStage, &w_map, &full[i], (b0 + i) * kBlock, (int)n0);
            }
            pdl_wait();
            loads = first;
            for (int i = 0; i < first; ++i)
                tma_load_2d(ring + i * C::kStage + kTile * kBlock, &x_map, &full[i], (b0 + i) * kBlock, (int)m0);
            for (int i = first; i < count; ++i) {
                const int slot = i % C::kStages;
                if (!mbar_wait(&empty[slot], (uint32_t)(i / C::kStages - 1) & 1u, ctl)) break;
                uint8_t* st = ring + slot * C::kStage;
                mbar_arrive_expect_tx(&full[slot], C::kStage);
                tma_load_2d(st, &w_map, &full[slot], (b0 + i) * kBlock, (int)n0);
                tma_load_2d(st + kTile * kBlock, &x_map, &full[slot], (b0 + i) * kBlock, (int)m0);
                loads = i + 1;
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        give_registers<MT>();
        const bool ready = warp_wait(&tmem_ready, 0, ctl);
        fence_after();
        const uint32_t tmem = tmem_slot;
        for (int i = 0; ready && i < count; ++i) {
            const int slot = i % C::kStages, buf = i % C::kBufs;
            if (i >= C::kBufs && !warp_wait(&d_empty[buf], (uint32_t)(i / C::kBufs - 1) & 1u, ctl)) break;
            if (!warp_wait(&full[slot], (uint32_t)(i / C::kStages) & 1u, ctl)) break;
            fence_after();
            const uint32_t st = smem_u32(ring + slot * C::kStage);
            block_products(tmem + buf * MT, desc_lo(st), desc_lo(st + kTile * kBlock), idesc(kTile, MT), &empty[slot],
                           &d_full[buf]);
            if (lane == 0) products = i + 1;
        }
    } else if (warp == 2) {
        give_registers<MT>();
        pdl_wait();
        const float* sw = a.w_scales + (int64_t)tile * a.blocks;
        for (int j = 0; j * kBatch < count; ++j) {
            // lanes: 8 blocks of K by 4 tokens
            const int kb = b0 + j * kBatch + (lane & 7);
            const bool in = kb < b1;
            const float w = in ? sw[kb] : 0.f;
            if (j >= 2 && !warp_wait(&s_empty[j & 1], (uint32_t)(j / 2 - 1) & 1u, ctl)) break;
            const float* sx = a.x_scales + (m0 + (lane >> 3)) * a.blocks + kb;
            float* to = &scales[j & 1][lane & 7][lane >> 3];
#pragma unroll 4
            for (int t = 0; t < MT / 4; ++t)
                to[4 * t] = in && 4 * t + (lane >> 3) < live ? sx[(int64_t)(4 * t) * a.blocks] * w : 0.f;
            mbar_arrive(&s_full[j & 1]);
        }
    } else if (warp == 3) {
        give_registers<MT>();
        // Tensor memory is taken after the kernels before this one have
        // finished, and the next one may start after it is taken: of two
        // kernels on an SM, none holds columns that the other needs to end.
        pdl_wait();
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_slot)),
                     "r"(C::kCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        fence_before();
        pdl_launch_dependents();
        if (lane == 0) mbar_arrive(&tmem_ready);
    } else {
        if constexpr (MT == 128) asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
        const bool ready = warp_wait(&tmem_ready, 0, ctl);
        fence_after();
        const uint32_t tmem = tmem_slot;
        const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21);
        float sum[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m) sum[m] = 0.f;
        for (int i = 0; ready && i < count; ++i) {
            const int buf = i % C::kBufs, j = i / kBatch;
            if (i % kBatch == 0 && !warp_wait(&s_full[j & 1], (uint32_t)(j / 2) & 1u, ctl)) break;
            if (!warp_wait(&d_full[buf], (uint32_t)(i / C::kBufs) & 1u, ctl)) break;
            fence_after();
            const float* sc = scales[j & 1][i % kBatch];
            uint32_t d[2][16];
            tmem_ld16(lanes + buf * MT, d[0]);
#pragma unroll
            for (int c = 0; c < MT / 16; ++c) {
                tmem_ld_wait();
                if (c + 1 < MT / 16) tmem_ld16(lanes + buf * MT + 16 * (c + 1), d[(c + 1) & 1]);
#pragma unroll
                for (int t = 0; t < 16; t += 4) {
                    const float4 s = lds4(sc + 16 * c + t);
                    fma2(sum[16 * c + t], sum[16 * c + t + 1], d[c & 1][t], d[c & 1][t + 1], s.x, s.y);
                    fma2(sum[16 * c + t + 2], sum[16 * c + t + 3], d[c & 1][t + 2], d[c & 1][t + 3], s.z, s.w);
                }
            }
            fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&d_empty[buf]);
                if (i % kBatch == kBatch - 1) mbar_arrive(&s_empty[j & 1]);
            }
        }
        pdl_wait();   // (every thread that writes outputs)
        if (a.split == 1) {
            if (n < a.N) {
#pragma unroll
                for (int m = 0; m < MT; ++m)
                    if (m < live) out[(m0 + m) * a.N + n] = T::from_f32(sum[m]);
            }
        } else {
            // (the last products have been waited for: the ring is free)
#pragma unroll
            for (int m = 0; m < MT; ++m) mine[m * kTile + row] = sum[m];
        }
    }

    // What was issued lands before the CTA leaves. Without a time-out it has:
    // the commit of the last products was waited for above.
    __syncthreads();
    if (abort_flag && threadIdx.x == 0) {
        for (int i = 0; i < min(loads, C::kStages); ++i)
            mbar_wait_drain(&full[i], (uint32_t)((loads - 1 - i) / C::kStages) & 1u, a.spin_limit, a.status);
        for (int i = 0; i < min(products, C::kBufs); ++i)
            mbar_wait_drain(&d_full[i], (uint32_t)((products - 1 - i) / C::kBufs) & 1u, a.spin_limit, a.status);
    }
    fence_before();
    __syncthreads();
    fence_after();
    // (before the cluster's CTAs wait for each other: a CTA that holds tensor
    // memory waits for none of them)
    if (warp == 3)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_slot), "r"(C::kCols) : "memory");

    if (a.split == 1) return;
    pdl_wait();
    // token m is joined by rank m % split, in the order of the ranks
    cluster_arrive();
    cluster_wait();
    for (int m = rank + a.split * (int)(threadIdx.x >> 7); m < live; m += 2 * a.split) {
        float s = 0.f;
        for (int r = 0; r < a.split; ++r) s += ld_cluster(mapa(smem_u32(mine + m * kTile + row), r));
        if (n < a.N) out[(m0 + m) * a.N + n] = T::from_f32(s);
    }
    cluster_arrive();   // no CTA leaves while another reads its sums
    cluster_wait();
}

static bool make_map(CUtensorMap* map, const void* p, int64_t rows, int64_t cols, int box_rows) {
    auto fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)cols};
    const cuuint32_t box[2] = {(cuuint32_t)kBlock, (cuuint32_t)box_rows};
    const cuuint32_t one[2] = {1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(p), dims, strides, box, one,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int MT>
static cudaError_t few_launch(const Fp8MmLaunch& L, cudaStream_t s) {
    using C = Few<MT>;
    CUtensorMap w_map, x_map;
    if (!make_map(&w_map, L.w, L.N, L.K, kTile) || !make_map(&x_map, L.x, L.M, L.K, MT)) return cudaErrorInvalidValue;
    static bool done[64];
    cudaError_t e = allow_smem_once(few_kernel<T, MT>, C::kSmem, done);
    if (e != cudaSuccess) return e;
    const int64_t tiles = (L.N + kTile - 1) / kTile, chunks = (L.M + MT - 1) / MT;
    const int blocks = (int)((L.K + kBlock - 1) / kBlock);
    // as many CTAs as two an SM hold
    int split = (int)std::min<int64_t>({8, blocks, std::max<int64_t>(1, 2 * (int64_t)num_sms() / (tiles * chunks))});
    if (tiles * chunks * split > 0x7fffffff) return cudaErrorInvalidConfiguration;
    const FewArgs a{L.w_scales, L.x_scales, L.out, L.M, L.N, blocks, (int)chunks, split, L.status, L.spin_limit};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tiles * chunks * split));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)split;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, few_kernel<T, MT>, w_map, x_map, a);
}

template <typename T>
static cudaError_t typed(const Fp8MmLaunch& L, cudaStream_t s) {
    if (L.M <= 16) return few_launch<T, 16>(L, s);
    if (L.M <= 32) return few_launch<T, 32>(L, s);
    if (L.M <= 64) return few_launch<T, 64>(L, s);
    return few_launch<T, 128>(L, s);
}

}  // namespace fp8mm

cudaError_t launch_fp8_mm(const Fp8MmLaunch& L, int dtype, cudaStream_t s) {
    switch (dtype) {
    case GAI4_F16: return fp8mm::typed<F16>(L, s);
    case GAI4_F32: return fp8mm::typed<F32>(L, s);
    default: return fp8mm::typed<BF16>(L, s);
    }
}

}  // namespace gai4
