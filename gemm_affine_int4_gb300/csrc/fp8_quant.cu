// fp8_quant.cu -- activations and weights into e4m3 (internal).
//
// Activations: a scale for each 128 consecutive elements of a row. Weights: a
// scale for each block of 128 rows x 128 columns. Both read every value once
// and write a byte for it: bound by HBM (16-bit inputs 3 bytes a value, binary32
// 5), for a few rows by the launch. 5000 x 5001, whose elements are read and written
// singly, in us: weights bf16 34, f32 26; activations 25, 25 (floors 11, 18).
#include <algorithm>

#include "fp8_quant.cuh"
#include "internal.h"

namespace gai4 {

namespace {

using namespace fp8;

constexpr int kThreads = 256;

// A block takes blockDim.x eights of kRows * blockDim.y rows, a thread one eight
// of kRows of them, all loaded before the first is used; `across` blocks take a
// row.
template <typename T, bool VEC, int kRows>
__global__ void __launch_bounds__(kThreads) quantize_x_fp8_kernel(const typename T::storage* __restrict__ x,
                                                                  int64_t x_stride, uint8_t* __restrict__ codes,
                                                                  float* __restrict__ scales, int64_t rows,
                                                                  int64_t cols, unsigned across) {
    pdl_launch_dependents();
    pdl_wait();   // the kernels before this one are complete: global memory may be read
    const unsigned down = blockIdx.x / across;
    const int64_t col = (int64_t)(blockIdx.x - down * across) * blockDim.x * 8 + column_of<VEC>(threadIdx.x);
    const int64_t row = (int64_t)down * blockDim.y * kRows + threadIdx.y;
    Eight<T, VEC> in[kRows];
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
        const int64_t r = row + j * blockDim.y;
        if (r < rows && col < cols)
            in[j].load(x + r * x_stride + col, cols - col);
        else
            in[j].zero();
    }
    const int64_t blocks = (cols + kGroup - 1) / kGroup;
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
        const int64_t r = row + j * blockDim.y;
        float v[8];
        in[j].values(v);
        const Scale s = scale_of(group_max(amax8(v)));
        if (r >= rows || col >= cols) continue;
        store_codes8<VEC>(codes + r * cols + col, cols - col, codes8(v, s));
        if ((threadIdx.x & 15) == 0) scales[r * blocks + col / kGroup] = scale_value(s);
    }
}

// One block of 128 x 128 a CTA: thread t holds eights t % 16 of the rows
// t / 16 + 16 j, in registers from the maximum to the codes: as loaded, so that 16-bit
// inputs leave room for five CTAs an SM (14336 x 5120: bf16 34 us; 46 with the values
// kept in binary32 and three CTAs; f32 55 us, 98% of the measured HBM rate).
template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads, VEC && T::kBytes == 2 ? 5 : 3) quantize_fp8_kernel(const typename T::storage* __restrict__ w,
                                                                uint8_t* __restrict__ codes,
                                                                float* __restrict__ scales, int64_t N, int64_t K) {
    // no programmatic launch: what this kernel writes may be read as weights
    pdl_wait();
    __shared__ float part[kThreads / 32];
    const int64_t k = (int64_t)blockIdx.x * kGroup + column_of<VEC>(threadIdx.x & 15);
    const int64_t n0 = (int64_t)blockIdx.y * kGroup + (threadIdx.x >> 4);
    Eight<T, VEC> in[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        if (n0 + 16 * j < N && k < K)
            in[j].load(w + (n0 + 16 * j) * K + k, K - k);
        else
            in[j].zero();
    }
    float m = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        float v[8];
        in[j].values(v);
        m = max_abs(m, amax8(v));
    }
    m = group_max(m);
    m = max_abs(m, __shfl_xor_sync(0xffffffffu, m, 16));
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) m = max_abs(m, part[i]);
    const Scale s = scale_of(m);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        in[j].keep();
        float v[8];
        in[j].values(v);
        if (n0 + 16 * j < N && k < K) store_codes8<VEC>(codes + (n0 + 16 * j) * K + k, K - k, codes8(v, s));
    }
    if (threadIdx.x == 0) scales[blockIdx.y * (int64_t)gridDim.x + blockIdx.x] = scale_value(s);
}

bool vec_ok(const void* p, int64_t stride, int64_t cols, int elem, const void* codes) {
    return cols % 8 == 0 && (uintptr_t)p % 16 == 0 && (stride * elem) % 16 == 0 && (uintptr_t)codes % 8 == 0;
}

template <typename T>
cudaError_t x_launch(const void* x, int64_t x_stride, uint8_t* codes, float* scales, int64_t rows, int64_t cols,
                     cudaStream_t s) {
    const auto* p = static_cast<const typename T::storage*>(x);
    const int64_t eights = (cols + kGroup - 1) / kGroup * 16;
    const bool vec = vec_ok(x, x_stride, cols, T::kBytes, codes);
    // few values: one eight a thread, on as many SMs as there are. Single elements too:
    // an eight of those is eight loads (5000 x 5001, bf16: 25 us, 32 with four rows a
    // thread; 14336 x 5120 in 16-byte accesses: 55, and 42).
    const bool few = !vec || rows * eights <= (int64_t)num_sms() * 4 * kThreads;
    const int tx = (int)std::min<int64_t>(eights, 128), ty = tx % 32 ? kThreads / tx & ~1 : kThreads / tx;   // whole warps
    const int64_t across = (eights + tx - 1) / tx, down = (rows + ty * (few ? 1 : 4) - 1) / (ty * (few ? 1 : 4));
    if (across * down > 0x7fffffff) return cudaErrorInvalidConfiguration;
    auto* k = !vec ? quantize_x_fp8_kernel<T, false, 1> : few ? quantize_x_fp8_kernel<T, true, 1> : quantize_x_fp8_kernel<T, true, 4>;
    return launch_pdl(k, dim3((unsigned)(across * down)), dim3(tx, ty), 0, s, p, x_stride, codes, scales, rows, cols,
                      (unsigned)across);
}

template <typename T>
cudaError_t w_launch(const void* w, uint8_t* codes, float* scales, int64_t N, int64_t K, cudaStream_t s) {
    const auto* p = static_cast<const typename T::storage*>(w);
    const dim3 grid((unsigned)((K + kGroup - 1) / kGroup), (unsigned)((N + kGroup - 1) / kGroup));
    return launch_pdl(vec_ok(w, K, K, T::kBytes, codes) ? quantize_fp8_kernel<T, true> : quantize_fp8_kernel<T, false>,
                      grid, dim3(kThreads), 0, s, p, codes, scales, N, K);
}

}  // namespace

cudaError_t launch_quantize_x_fp8(const void* x, int64_t x_stride, uint8_t* codes, float* scales, int dtype,
                                  int64_t rows, int64_t cols, cudaStream_t s) {
    switch (dtype) {
    case GAI4_F16: return x_launch<F16>(x, x_stride, codes, scales, rows, cols, s);
    case GAI4_F32: return x_launch<F32>(x, x_stride, codes, scales, rows, cols, s);
    default: return x_launch<BF16>(x, x_stride, codes, scales, rows, cols, s);
    }
}

cudaError_t launch_quantize_fp8(const void* w, uint8_t* codes, float* scales, int dtype, int64_t N, int64_t K,
                                cudaStream_t s) {
    switch (dtype) {
    case GAI4_F16: return w_launch<F16>(w, codes, scales, N, K, s);
    case GAI4_F32: return w_launch<F32>(w, codes, scales, N, K, s);
    default: return w_launch<BF16>(w, codes, scales, N, K, s);
    }
}

}  // namespace gai4
