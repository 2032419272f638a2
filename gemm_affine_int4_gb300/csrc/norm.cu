// norm.cu -- root-mean-square norm of rows (internal):
//   h = x + residual        y = h / sqrt(mean(h^2) + eps) * gain
// with h rounded to T as the new residual, and y rounded to T or to e4m3 with a
// scale for each 128 elements (fp8_quant.cuh). Sums, h and y are binary32; y is
// rounded once.
//
// A group's codes are those of p = h * gain: y / max |y| = p / max |p|, the root
// of the row divides out, and only the scales wait for it. So codes and the new
// residual are written while the row's sum is still being taken, and the codes
// do not carry its rounding.
//
// Each value is read once and written once, so a long input is bound by HBM and
// a few rows by the latency of a load, the sum across the row and a store. A
// row belongs to some warps; a thread takes kUnits eights of it, a row's width of
// threads apart (16 lanes hold a group of 128), and keeps p for y in T. Rows too
// long for that are read a second time. Many rows into e4m3 alone are a warp's each.
// 20011 x 5120, bf16, residual: codes 114 us (93% of the measured HBM rate), y 136 to 140
// (86 to 89%); without one: codes 72 to 74 (62 to 64%), y 69 (88%); 64 x 4096, codes: 2.1 us.
#include <algorithm>

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

// an eight of a row's inputs, and of the gain, as loaded
template <typename T, bool VEC>
struct Inputs {
    Eight<T, VEC> x, r;
    __device__ __forceinline__ void load(const NormArgs& a, int64_t row, int64_t col) {
        using S = typename T::storage;
        if (row < a.rows && col < a.cols) {
            x.load(static_cast<const S*>(a.x) + row * a.x_stride + col, a.cols - col);
            if (a.residual) r.load(static_cast<const S*>(a.residual) + row * a.r_stride + col, a.cols - col);
        } else {
            x.zero();
            r.zero();
        }
    }
};
template <typename T, bool VEC>
__device__ __forceinline__ void load_gain(const NormArgs& a, int64_t col, Eight<T, VEC>& g) {
    if (a.gain && col < a.cols)
        g.load(static_cast<const typename T::storage*>(a.gain) + col, a.cols - col);
    else
        g.zero();
}

// What can be done with an eight of the row before its root is known: p, and
// the largest |p| of the group (with codes). Returns the sum of squares of h.
// Every lane of the warp calls it.
template <typename T, bool VEC>
__device__ __forceinline__ float begin8(const NormArgs& a, const Inputs<T, VEC>& from, const Eight<T, VEC>& gain,
                                        int64_t row, int64_t col, bool write, float (&p)[8], float& amax) {
    using S = typename T::storage;
    const bool in = row < a.rows && col < a.cols;
    const int64_t left = a.cols - col, at = row * a.cols + col;
    float sum = 0.f;
    from.x.values(p);
    if (a.residual) {
        float r[8];
        from.r.values(r);
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] += r[i];
    }
    if (write && in && a.residual_out) store8<T, VEC>(static_cast<S*>(a.residual_out) + at, left, p);
#pragma unroll
    for (int i = 0; i < 8; ++i) sum = fmaf(p[i], p[i], sum);
    if (a.gain) {
        float g[8];
        gain.values(g);
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] *= g[i];
    }
    if (write && a.codes) {   // (uniform)
        const Scale scale = scale_of(group_max(amax8(p)));
        amax = scale.amax;
        if (in) store_codes8<VEC>(a.codes + at, left, codes8(p, scale));
    }
    return sum;
}

// and after it is: y in T, scales
template <typename T, bool VEC>
__device__ __forceinline__ void end8(const NormArgs& a, int64_t row, int64_t col, float inv, const float (&p)[8], float amax) {
    using S = typename T::storage;
    if (row >= a.rows || col >= a.cols) return;
    if (a.out) {
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = p[i] * inv;
        store8<T, VEC>(static_cast<S*>(a.out) + row * a.cols + col, a.cols - col, y);
    }
    if (a.codes && (threadIdx.x & 15) == 0)
        a.scales[row * ((a.cols + kGroup - 1) / kGroup) + col / kGroup] = __fdiv_rn(inv * amax, 448.0f);
}

// sum over a row's threads: blockDim.x of them, 16 or whole warps (threadIdx.y:
// the row of the block)
__device__ __forceinline__ float row_sum(float s, float (*part)[kMaxWarps]) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (blockDim.x == 16) return s;
    s += __shfl_xor_sync(0xffffffffu, s, 16);
    if (blockDim.x == 32) return s;
    const int lane = threadIdx.x & 31;
    if (lane == 0) part[threadIdx.y][threadIdx.x >> 5] = s;
    __syncthreads();
    return warp_sum(lane < blockDim.x / 32 ? part[threadIdx.y][lane] : 0.f);
}

// 1 / sqrt(mean + eps)
__device__ __forceinline__ float inverse_root(float sum, const NormArgs& a) {
    return __frsqrt_rn(__fdiv_rn(sum, (float)a.cols) + a.eps);
}

// blockDim = (threads a row, rows a block); kUnits eights a thread cover the
// row. With LOOP a block takes rows gridDim.x * blockDim.y apart: the gain is
// read once, and a row is read while the one before it is summed and written.
// An output in the place of an input: an eight is written by the thread that has
// read it.
template <typename T, bool VEC, int kUnits, bool LOOP>
__global__ void __launch_bounds__(kUnits == 4 ? 512 : 1024) rms_norm_kernel(const __grid_constant__ NormArgs a) {
    pdl_launch_dependents();
    pdl_wait();   // the kernels before this one are complete: global memory may be read
    __shared__ float part[2][16][kMaxWarps];
    Inputs<T, VEC> in[kUnits];
    Eight<T, VEC> gain[kUnits];
    const int col0 = column_of<VEC>(threadIdx.x), step = blockDim.x * 8;
    int64_t first = (int64_t)blockIdx.x * blockDim.y;   // row of the block's first threads
#pragma unroll
    for (int j = 0; j < kUnits; ++j) in[j].load(a, first + threadIdx.y, col0 + j * step);
#pragma unroll
    for (int j = 0; j < kUnits; ++j) load_gain<T, VEC>(a, col0 + j * step, gain[j]);
    int turn = 0;
    do {
        const int64_t row = first + threadIdx.y;
        first += (int64_t)gridDim.x * blockDim.y;
        float p[kUnits][8], amax[kUnits], s = 0.f;
#pragma unroll
        for (int j = 0; j < kUnits; ++j) {
            amax[j] = 0.f;
            s += begin8<T, VEC>(a, in[j], gain[j], row, col0 + j * step, true, p[j], amax[j]);
        }
        if constexpr (LOOP) {
#pragma unroll
            for (int j = 0; j < kUnits; ++j) in[j].load(a, first + threadIdx.y, col0 + j * step);
        }
        const float inv = inverse_root(row_sum(s, part[turn]), a);
#pragma unroll
        for (int j = 0; j < kUnits; ++j) end8<T, VEC>(a, row, col0 + j * step, inv, p[j], amax[j]);
        turn ^= 1;
    } while (LOOP && first < a.rows);
}

// y in T alone, without a residual, many 16-bit rows: as the kernel above with LOOP,
// but a row stays as it was loaded until its root is known, half of the registers
// of its values.
template <typename T, int kUnits>
__global__ void __launch_bounds__(512, 2) rms_norm_plain_kernel(const __grid_constant__ NormArgs a) {
    using S = typename T::storage;
    pdl_launch_dependents();
    pdl_wait();   // the kernels before this one are complete: global memory may be read
    __shared__ float part[2][16][kMaxWarps];
    Eight<T, true> x[kUnits], next[kUnits], gain[kUnits];
    const int col0 = threadIdx.x * 8, step = blockDim.x * 8;
    int64_t first = (int64_t)blockIdx.x * blockDim.y;   // row of the block's first threads
    const auto load = [&](int64_t row) {
#pragma unroll
        for (int j = 0; j < kUnits; ++j) {
            const int col = col0 + j * step;
            if (row < a.rows && col < a.cols)
                next[j].load(static_cast<const S*>(a.x) + row * a.x_stride + col, 8);
            else
                next[j].zero();
        }
    };
    load(first + threadIdx.y);
#pragma unroll
    for (int j = 0; j < kUnits; ++j) load_gain<T, true>(a, col0 + j * step, gain[j]);
    int turn = 0;
    do {
        const int64_t row = first + threadIdx.y;
        first += (int64_t)gridDim.x * blockDim.y;
        float s = 0.f;
#pragma unroll
        for (int j = 0; j < kUnits; ++j) {
            float v[8];
            next[j].values(v);
#pragma unroll
            for (int i = 0; i < 8; ++i) s = fmaf(v[i], v[i], s);
            x[j] = next[j];
        }
        load(first + threadIdx.y);
        const float inv = inverse_root(row_sum(s, part[turn]), a);
#pragma unroll
        for (int j = 0; j < kUnits; ++j) {
            const int col = col0 + j * step;
            if (row >= a.rows || col >= a.cols) continue;
            x[j].keep();
            float v[8], g[8];
            x[j].values(v);
            if (a.gain) {
                gain[j].keep();
                gain[j].values(g);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] *= g[i];
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] *= inv;
            store8<T, true>(static_cast<S*>(a.out) + row * a.cols + col, 8, v);
        }
        turn ^= 1;
    } while (first < a.rows);
}

// rows of any length, one a block, read twice (nothing is written in between:
// outputs may lie on inputs): 700 x 40000, bf16, residual 56 to 59 us, at 59% of HBM once
template <typename T, bool VEC>
__global__ void __launch_bounds__(1024) rms_norm_long_kernel(const __grid_constant__ NormArgs a) {
    pdl_launch_dependents();
    pdl_wait();
    __shared__ float part[1][kMaxWarps];
    const int64_t row = blockIdx.x;
    Inputs<T, VEC> in;
    Eight<T, VEC> gain;
    float p[8], amax = 0.f, s = 0.f;
    for (int64_t col = column_of<VEC>(threadIdx.x); col < a.cols; col += (int64_t)blockDim.x * 8) {
        in.load(a, row, col);
        load_gain<T, VEC>(a, col, gain);
        s += begin8<T, VEC>(a, in, gain, row, col, false, p, amax);
    }
    const float inv = inverse_root(row_sum(s, part), a);
    for (int64_t at = 0; at < a.cols; at += (int64_t)blockDim.x * 8) {
        const int64_t col = at + column_of<VEC>(threadIdx.x);
        in.load(a, row, col);
        load_gain<T, VEC>(a, col, gain);
        begin8<T, VEC>(a, in, gain, row, col, true, p, amax);
        end8<T, VEC>(a, row, col, inv, p, amax);
    }
}

// Many rows into e4m3 alone: a warp goes through its row, a step of 256 behind its
// loads, without a barrier. Codes and the new residual are written on the way, and
// of the row no more is kept than its groups' maxima (in shared memory), for the
// scales. One step ahead and 36 warps an SM; two steps and 24 take 141 us instead of
// 114 (20011 x 5120, bf16, residual). Without a residual half as much is on its way, 18 KB
// an SM, and bounds it: 72 to 74 us for 46 of HBM; and so it is for fewer rows than those 36
// warps an SM (3000 x 28672 with a residual 118, for 89). y in T would be written in a second
// pass: 107 us, rms_norm_kernel 80.
constexpr int kRowWarps = 4;
template <typename T, bool VEC>
__global__ void __launch_bounds__(32 * kRowWarps, 6) rms_norm_codes_kernel(const __grid_constant__ NormArgs a) {
    using S = typename T::storage;
    pdl_launch_dependents();
    pdl_wait();   // the kernels before this one are complete: global memory may be read
    extern __shared__ float maxima[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t row = (int64_t)blockIdx.x * kRowWarps + warp;
    if (row >= a.rows) return;
    const int cols = (int)a.cols, groups = (cols + kGroup - 1) / kGroup;
    float* maximum = maxima + warp * groups;
    const int col0 = column_of<VEC>(lane);
    const S* x = static_cast<const S*>(a.x) + row * a.x_stride + col0;
    const S* r = a.residual ? static_cast<const S*>(a.residual) + row * a.r_stride + col0 : nullptr;
    const S* g = a.gain ? static_cast<const S*>(a.gain) + col0 : nullptr;
    S* h = a.residual_out ? static_cast<S*>(a.residual_out) + row * a.cols + col0 : nullptr;
    uint8_t* codes = a.codes + row * a.cols + col0;
    Eight<T, VEC> in, res, gain;
    const auto load = [&](int left) {
        if (left > 0) {
            in.load(x, left);
            if (r) res.load(r, left);
            if (g) gain.load(g, left);
        } else {
            in.zero();
            res.zero();
            gain.zero();
        }
    };
    load(cols - col0);
    float sum = 0.f;
    for (int at = 0, left = cols - col0; at < cols; at += 256, left -= 256) {
        float p[8], q[8];
        in.values(p);
        if (r) {
            res.values(q);
#pragma unroll
            for (int i = 0; i < 8; ++i) p[i] += q[i];
        }
        if (h && left > 0) store8<T, VEC>(h + at, left, p);
        float squares = 0.f;   // (of the step: so the row's sum has few roundings)
#pragma unroll
        for (int i = 0; i < 8; ++i) squares = fmaf(p[i], p[i], squares);
        sum += squares;
        if (g) {
            gain.values(q);
#pragma unroll
            for (int i = 0; i < 8; ++i) p[i] *= q[i];
        }
        x += 256;
        if (r) r += 256;
        if (g) g += 256;
        load(left - 256);
        const Scale scale = scale_of(group_max(amax8(p)));
        if (left > 0) {
            store_codes8<VEC>(codes + at, left, codes8(p, scale));
            if ((lane & 15) == 0) maximum[at / kGroup + (lane >> 4)] = scale.amax;
        }
    }
    const float inv = inverse_root(warp_sum(sum), a);
    __syncwarp();
    for (int i = lane; i < groups; i += 32) a.scales[row * groups + i] = __fdiv_rn(inv * maximum[i], 448.0f);
}

template <typename T, bool VEC>
cudaError_t norm_launch(const NormArgs& a, cudaStream_t s) {
    const int64_t eights = (a.cols + 7) / 8;
    const int64_t wide = (eights + 31) / 32;   // warps that take the row at one eight a thread
    // Into e4m3 alone, a warp a row: in us, and with the kernels below, bf16 with a
    // residual 20011 x 5120 114, 125; 20011 x 1000 27, 28; 3000 x 28672 118, 175; without
    // one 20011 x 5120 72, 104; f32 without one 10000 x 5120 53, 59. Not for rows that do
    // not go round among 36 warps an SM (6000 x 2048 20, 18; 700 x 40000 112, 57), short
    // ones (30000 x 512 21, 20), and f32 with a residual (10000 x 5120 101, 95).
    const bool long_rows = wide > kMaxWarps * 2;
    if (a.codes && !a.out && a.cols > 512 && a.cols <= 262144 && a.rows >= (long_rows ? 8 : 64) * num_sms() &&
        (long_rows || T::kBytes == 2 || !a.residual))
        return launch_pdl(rms_norm_codes_kernel<T, VEC>, dim3((unsigned)((a.rows + kRowWarps - 1) / kRowWarps)),
                          dim3(32 * kRowWarps), (size_t)((a.cols + kGroup - 1) / kGroup * 4 * kRowWarps), s, a);
    if (long_rows)
        return launch_pdl(rms_norm_long_kernel<T, VEC>, dim3((unsigned)a.rows), dim3(1024), 0, s, a);
    // Few rows: as many threads a row as it has eights. Many rows: two eights a
    // thread, so that more is on its way (20011 x 5120, bf16, residual and codes:
    // 158 us with one, 130 with two), and blocks that take row after row (125 us).
    // Those pay off for 16-bit rows only: 10000 x 5120 in f32 takes 96 us without,
    // 134 with, as registers run out. Without a residual half as much is read at a
    // time: four eights (y alone, before it had a kernel of its own: 80 us, two 87).
    const bool few = a.rows <= 2 * num_sms();
    const bool loop = !few && T::kBytes == 2 && VEC && wide > 1;
    int units = few || wide == 1 ? 1 : loop && !a.residual && wide > 4 ? 4 : 2;
    if (units == 1 && wide > kMaxWarps) units = 2;
    const int threads = eights <= 16 ? 16 : 32 * (int)((wide + units - 1) / units);
    const int per = few ? 1 : std::max(1, 256 / threads);
    // (a block of at least a warp)
    const dim3 block(threads, threads == 16 ? std::max(per, 2) : per);
    const int64_t blocks = (a.rows + block.y - 1) / block.y;
    if (loop && a.out && !a.codes && !a.residual && !a.residual_out) {
        // In us, and with the kernel above: bf16 20011 x 5120 69, 80; 10000 x 4096 28, 34;
        // 30000 x 1024 21, 27; 4000 x 14336 39, 51.
        if constexpr (T::kBytes == 2 && VEC) {
            units = wide >= 4 ? 4 : 2;
            const int tx = 32 * (int)((wide + units - 1) / units), ty = std::max(1, 256 / tx);
            const dim3 grid((unsigned)std::min<int64_t>((a.rows + ty - 1) / ty, (int64_t)num_sms() * (1024 / (tx * ty))));
            return launch_pdl(units == 4 ? rms_norm_plain_kernel<T, 4> : rms_norm_plain_kernel<T, 2>, grid, dim3(tx, ty), 0, s, a);
        }
    }
    if (loop) {
        const dim3 grid((unsigned)std::min<int64_t>(blocks, (int64_t)num_sms() * std::max(1, 1024 / (threads * per))));
        if constexpr (T::kBytes == 2 && VEC)
            return launch_pdl(units == 4 ? rms_norm_kernel<T, VEC, 4, true> : rms_norm_kernel<T, VEC, 2, true>, grid, block, 0,
                              s, a);
    }
    return launch_pdl(units == 1 ? rms_norm_kernel<T, VEC, 1, false> : rms_norm_kernel<T, VEC, 2, false>,
                      dim3((unsigned)blocks), block, 0, s, a);
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
