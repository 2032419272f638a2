// norm.cu -- root-mean-square norm of rows (internal):
//   h = x + residual        y = h / sqrt(mean(h^2) + eps) * gain
// with h rounded to T as the new residual, and y rounded to T or to e4m3 with a
// scale for each 128 elements (fp8_quant.cuh). Sums, h and y are binary32; y is
// rounded once.
//
// Each value is read once and written once, so a long input is bound by HBM and
// a few rows by the latency of a load, the sum across the row and a store. A
// row is held in registers between the sum and the outputs: `warps` warps take
// a row, a thread kUnits eights of it, a row's width of threads apart (16 lanes
// hold a group of 128). Rows too long for that are read a second time.
#include "fp8_quant.cuh"
#include "internal.h"

namespace gai4 {

namespace {

using namespace fp8;

constexpr int kMaxWarps = 32;

struct NormArgs {
    const void* x;
    int64_t x_stride;
    const void* residual;   // NULL: none
    int64_t r_stride;
    const void* gain;       // NULL: ones
    void* out;              // each of the outputs may be NULL
    void* residual_out;
    uint8_t* codes;
    float* scales;
    int64_t rows, cols;
    float eps;
};

// 8 values of h, zeros past the row's end
template <typename T, bool VEC>
__device__ __forceinline__ void load_h(const NormArgs& a, int64_t row, int64_t col, float (&h)[8]) {
    using S = typename T::storage;
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = 0.f;
    if (col >= a.cols) return;
    load8<T, VEC>(static_cast<const S*>(a.x) + row * a.x_stride + col, a.cols - col, h);
    if (a.residual) {
        float r[8];
        load8<T, VEC>(static_cast<const S*>(a.residual) + row * a.r_stride + col, a.cols - col, r);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] += r[i];
    }
}

// writes the row's 8 values; every lane of the warp calls it
template <typename T, bool VEC>
__device__ __forceinline__ void finish8(const NormArgs& a, int64_t row, int64_t col, float inv, float (&h)[8]) {
    using S = typename T::storage;
    const bool in = row < a.rows && col < a.cols;
    const int64_t left = a.cols - col, at = row * a.cols + col;
    if (in && a.residual_out) store8<T, VEC>(static_cast<S*>(a.residual_out) + at, left, h);
    float g[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] = 1.f;
    if (in && a.gain) load8<T, VEC>(static_cast<const S*>(a.gain) + col, left, g);
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = h[i] * inv * g[i];
    if (in && a.out) store8<T, VEC>(static_cast<S*>(a.out) + at, left, h);
    if (a.codes) {   // (uniform)
        const Scale s = scale_of(group_max(amax8(h)));
        if (in) store_codes8<VEC>(a.codes + at, left, codes8(h, s));
        if (in && (threadIdx.x & 15) == 0)
            a.scales[row * ((a.cols + kGroup - 1) / kGroup) + col / kGroup] = scale_value(s);
    }
}

__device__ __forceinline__ float sum_squares(const float (&h)[8]) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s = fmaf(h[i], h[i], s);
    return s;
}

// sum over the `warps` warps of a row (threadIdx.y: the row of the block)
__device__ __forceinline__ float row_sum(float s, int warps, float (*part)[kMaxWarps]) {
    s = warp_sum(s);
    if (warps == 1) return s;
    if ((threadIdx.x & 31) == 0) part[threadIdx.y][threadIdx.x >> 5] = s;
    __syncthreads();
    const int lane = threadIdx.x & 31;
    return warp_sum(lane < warps ? part[threadIdx.y][lane] : 0.f);
}

// 1 / sqrt(mean + eps)
__device__ __forceinline__ float inverse_root(float sum, const NormArgs& a) {
    return __frsqrt_rn(__fdiv_rn(sum, (float)a.cols) + a.eps);
}

// blockDim = (32 * warps, rows a block); kUnits eights a thread cover the row
template <typename T, bool VEC, int kUnits>
__global__ void __launch_bounds__(1024) rms_norm_kernel(const __grid_constant__ NormArgs a) {
    pdl_launch_dependents();
    pdl_wait();   // the kernels before this one are complete: global memory may be read
    __shared__ float part[32][kMaxWarps];
    const int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    float h[kUnits][8];
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < kUnits; ++j) {
        const int64_t col = ((int64_t)j * blockDim.x + threadIdx.x) * 8;
        load_h<T, VEC>(a, row, row < a.rows ? col : a.cols, h[j]);
    }
#pragma unroll
    for (int j = 0; j < kUnits; ++j) s += sum_squares(h[j]);
    const float inv = inverse_root(row_sum(s, blockDim.x / 32, part), a);
#pragma unroll
    for (int j = 0; j < kUnits; ++j)
        finish8<T, VEC>(a, row, ((int64_t)j * blockDim.x + threadIdx.x) * 8, inv, h[j]);
}

// rows of any length, one a block, read twice (the outputs may lie on the
// inputs: an eight is read again by the thread that writes it, before it does)
template <typename T, bool VEC>
__global__ void __launch_bounds__(1024) rms_norm_long_kernel(const __grid_constant__ NormArgs a) {
    pdl_launch_dependents();
    pdl_wait();
    __shared__ float part[1][kMaxWarps];
    const int64_t row = blockIdx.x;
    float s = 0.f;
    for (int64_t col = (int64_t)threadIdx.x * 8; col < a.cols; col += (int64_t)blockDim.x * 8) {
        float h[8];
        load_h<T, VEC>(a, row, col, h);
        s += sum_squares(h);
    }
    const float inv = inverse_root(row_sum(s, blockDim.x / 32, part), a);
    for (int64_t at = 0; at < a.cols; at += (int64_t)blockDim.x * 8) {
        const int64_t col = at + (int64_t)threadIdx.x * 8;
        float h[8];
        load_h<T, VEC>(a, row, col, h);
        finish8<T, VEC>(a, row, col, inv, h);
    }
}

template <typename T, bool VEC>
cudaError_t norm_launch(const NormArgs& a, cudaStream_t s) {
    const int64_t eights = (a.cols + 7) / 8;
    const int64_t wide = (eights + 31) / 32;   // warps that take the row at one eight a thread
    if (wide > kMaxWarps * 4) {
        return launch_pdl(rms_norm_long_kernel<T, VEC>, dim3((unsigned)a.rows), dim3(1024), 0, s, a);
    }
    // Few rows: as many threads a row as it has eights. Many rows: fewer
    // threads with more eights each, so that more rows are under way.
    const bool few = a.rows <= 2 * num_sms();
    int units = few ? 1 : wide > 4 ? 4 : wide > 1 ? 2 : 1;
    while ((wide + units - 1) / units > kMaxWarps) units *= 2;
    const int warps = (int)((wide + units - 1) / units);
    const int per = few ? 1 : warps >= 8 ? 1 : 8 / warps;
    const dim3 block(32 * warps, per);
    const dim3 grid((unsigned)((a.rows + per - 1) / per));
    auto* k = units == 1 ? rms_norm_kernel<T, VEC, 1> : units == 2 ? rms_norm_kernel<T, VEC, 2> : rms_norm_kernel<T, VEC, 4>;
    return launch_pdl(k, grid, block, 0, s, a);
}

template <typename T>
cudaError_t norm_typed(const NormArgs& a, cudaStream_t s) {
    const auto rows16 = [&](const void* p, int64_t stride) {
        return (uintptr_t)p % 16 == 0 && (stride * T::kBytes) % 16 == 0;   // (NULL is)
    };
    const bool vec = a.cols % 8 == 0 && rows16(a.x, a.x_stride) && rows16(a.residual, a.residual ? a.r_stride : 0) &&
                     rows16(a.gain, 0) && rows16(a.out, a.cols) && rows16(a.residual_out, a.cols) &&
                     (uintptr_t)a.codes % 8 == 0;
    return vec ? norm_launch<T, true>(a, s) : norm_launch<T, false>(a, s);
}

}  // namespace

cudaError_t launch_rms_norm(const void* x, int64_t x_stride, const void* residual, int64_t r_stride, const void* gain,
                            void* out, void* residual_out, uint8_t* codes, float* scales, int dtype, int64_t rows,
                            int64_t cols, float eps, cudaStream_t s) {
    const NormArgs a{x, x_stride, residual, r_stride, gain, out, residual_out, codes, scales, rows, cols, eps};
    switch (dtype) {
    case GAI4_F16: return norm_typed<F16>(a, s);
    case GAI4_F32: return norm_typed<F32>(a, s);
    default: return norm_typed<BF16>(a, s);
    }
}

}  // namespace gai4
