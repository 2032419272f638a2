// layer_api.cu -- C ABI of the operators around the attention: rotary
// positions, norm, e4m3 quantization and product (declared in include/gai4.h):
// argument validation and launch. No allocation.
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "common.cuh"
#include "internal.h"

using namespace gai4;

namespace {

bool aligned_to(const void* p, uintptr_t n) { return ((uintptr_t)p % n) == 0; }
bool known(int dtype) { return dtype == GAI4_F32 || dtype == GAI4_F16 || dtype == GAI4_BF16; }
uintptr_t elem_bytes(int dtype) { return dtype == GAI4_F32 ? 4 : 2; }
gai4_status done(cudaError_t e) { return e == cudaSuccess ? GAI4_OK : GAI4_ERR_CUDA; }

constexpr int64_t kMost = 0x7fffffff;

// rows of `row` elements, `stride` apart: byte offsets stay in 64 bits
bool strided(int64_t stride, int64_t row, int64_t rows) { return stride >= row && stride <= (1ll << 60) / rows; }

// Whether rows that are written lie apart from rows that are read (or, for
// rows of one width, in their very place).
bool apart(const void* in, int64_t in_stride, int64_t in_row, const void* out, int64_t out_stride, int64_t out_row,
           int64_t rows, int64_t e) {
    if (in == out && in_stride == out_stride && in_row == out_row) return true;
    const uintptr_t a0 = (uintptr_t)in, a1 = a0 + (uintptr_t)(((rows - 1) * in_stride + in_row) * e);
    const uintptr_t b0 = (uintptr_t)out, b1 = b0 + (uintptr_t)(((rows - 1) * out_stride + out_row) * e);
    if (a1 <= b0 || b1 <= a0) return true;
    // slices of the same rows (the heads of one projection): apart within a row
    if (in_stride != out_stride) return false;
    const uintptr_t pitch = (uintptr_t)(in_stride * e);
    const uintptr_t off = b0 >= a0 ? (b0 - a0) % pitch : pitch - 1 - (a0 - b0 - 1) % pitch;
    return off >= (uintptr_t)(in_row * e) && off + (uintptr_t)(out_row * e) <= pitch;
}

gai4_status fp8_mm_sizes(gai4_dtype dtype, int64_t M, int64_t N, int64_t K) {
    if (!known(dtype)) return GAI4_ERR_UNSUPPORTED;
    if (M < 0 || M > kMost - 512 || N < 1 || N > kMost - 512 || K < 1 || K > kMost - 512) return GAI4_ERR_INVALID_ARG;
    return K % 16 != 0 ? GAI4_ERR_UNSUPPORTED : GAI4_OK;
}

// L.status NULL: the library's own
gai4_status fp8_mm(Fp8MmLaunch& L, gai4_dtype dtype, void* stream) {
    const gai4_status sizes = fp8_mm_sizes(dtype, L.M, L.N, L.K);
    if (sizes != GAI4_OK) return sizes;
    if (L.M == 0) return GAI4_OK;
    if (!L.w || !L.w_scales || !L.x || !L.x_scales || !L.out) return GAI4_ERR_INVALID_ARG;
    if (!aligned_to(L.w, 16) || !aligned_to(L.x, 16) || !aligned_to(L.w_scales, 4) || !aligned_to(L.x_scales, 4) ||
        !aligned_to(L.out, elem_bytes(dtype)))
        return GAI4_ERR_MISALIGNED;
    if (!L.status) L.status = status_ptr();
    if (!L.status || cudaGetDevice(&L.device) != cudaSuccess || L.device >= 64) return GAI4_ERR_CUDA;
    return done(launch_fp8_mm(L, dtype, (cudaStream_t)stream));
}

}  // namespace

extern "C" {

gai4_status gai4_rope_inv_freq(double* inv_freq, float* mscale, int rot_dim, double base, int scaling, double factor,
                               double original_len, double low, double high) {
    if (!inv_freq || !mscale || rot_dim < 2 || rot_dim % 2 != 0 || !(base > 1.0) || !isfinite(base))
        return GAI4_ERR_INVALID_ARG;
    if (scaling < GAI4_ROPE_NONE || scaling > GAI4_ROPE_SMOOTH) return GAI4_ERR_UNSUPPORTED;
    const bool ramp = scaling == GAI4_ROPE_YARN || scaling == GAI4_ROPE_SMOOTH;
    if (scaling != GAI4_ROPE_NONE && (!(factor >= 1.0) || !isfinite(factor))) return GAI4_ERR_INVALID_ARG;
    if (ramp && (!(original_len > 0.0) || !isfinite(original_len) || !(low > 0.0) || !(high > low) || !isfinite(high)))
        return GAI4_ERR_INVALID_ARG;
    constexpr double two_pi = 6.283185307179586476925286766559;
    if (scaling == GAI4_ROPE_NTK && rot_dim > 2) base *= pow(factor, (double)rot_dim / (rot_dim - 2));
    double first = 0.0, last = 0.0;
    if (scaling == GAI4_ROPE_YARN) {
        // the pairs that make `high` and `low` turns over the original length
        const auto pair = [&](double turns) { return rot_dim * log(original_len / (turns * two_pi)) / (2.0 * log(base)); };
        first = std::max(floor(pair(high)), 0.0);
        last = std::min(ceil(pair(low)), rot_dim - 1.0);
    }
    for (int i = 0; i < rot_dim / 2; ++i) {
        const double f = pow(base, -2.0 * i / rot_dim);
        double divided = 0.0;   // share of the divided frequency
        if (scaling == GAI4_ROPE_LINEAR) divided = 1.0;
        if (scaling == GAI4_ROPE_YARN) divided = (i - first) / std::max(last - first, 0.001);
        if (scaling == GAI4_ROPE_SMOOTH) divided = 1.0 - (original_len * f / two_pi - low) / (high - low);
        divided = std::min(std::max(divided, 0.0), 1.0);
        inv_freq[i] = f / factor * divided + f * (1.0 - divided);
        if (scaling == GAI4_ROPE_NONE || scaling == GAI4_ROPE_NTK) inv_freq[i] = f;
    }
    *mscale = scaling == GAI4_ROPE_YARN ? (float)(0.1 * log(factor) + 1.0) : 1.0f;
    return GAI4_OK;
}

gai4_status gai4_rope(const void* q, int64_t q_token_stride, void* q_out, int64_t q_out_token_stride, const void* k,
                      int64_t k_token_stride, void* k_out, int64_t k_out_token_stride, const int32_t* positions,
                      const double* inv_freq, float mscale, gai4_dtype dtype, int64_t num_tokens, int64_t q_heads,
                      int64_t kv_heads, int head_dim, int rot_dim, int interleaved, void* stream) {
    if (!known(dtype) || head_dim > 1024) return GAI4_ERR_UNSUPPORTED;
    if (head_dim < 1 || rot_dim < 2 || rot_dim % 2 != 0 || rot_dim > head_dim || num_tokens < 0 || num_tokens > kMost ||
        q_heads < 0 || kv_heads < 0 || q_heads + kv_heads < 1 || q_heads > 65535 || kv_heads > 65535)
        return GAI4_ERR_INVALID_ARG;
    if (num_tokens == 0) return GAI4_OK;
    if (!positions || !inv_freq) return GAI4_ERR_INVALID_ARG;
    if (!aligned_to(positions, 4) || !aligned_to(inv_freq, 8)) return GAI4_ERR_MISALIGNED;
    RopeLaunch L{{q, k}, {q_out, k_out}, {q_token_stride, k_token_stride}, {q_out_token_stride, k_out_token_stride},
                 {(int)q_heads, (int)kv_heads}, positions, inv_freq, mscale, num_tokens, head_dim, rot_dim, interleaved != 0,
                 dtype};
    const int64_t e = (int64_t)elem_bytes(dtype);
    for (int i = 0; i < 2; ++i) {
        if (L.heads[i] == 0) continue;
        const int64_t row = (int64_t)L.heads[i] * head_dim;
        if (!L.in[i] || !L.out[i] || !strided(L.in_stride[i], row, num_tokens) || !strided(L.out_stride[i], row, num_tokens))
            return GAI4_ERR_INVALID_ARG;
        if (!aligned_to(L.in[i], e) || !aligned_to(L.out[i], e)) return GAI4_ERR_MISALIGNED;
    }
    for (int i = 0; i < 2; ++i)
        for (int o = 0; o < 2; ++o)
            if (L.heads[i] > 0 && L.heads[o] > 0 &&
                (!apart(L.in[i], L.in_stride[i], (int64_t)L.heads[i] * head_dim, L.out[o], L.out_stride[o],
                        (int64_t)L.heads[o] * head_dim, num_tokens, e) ||
                 (i != o && L.in[i] == L.out[o])))
                return GAI4_ERR_INVALID_ARG;
    if (q_heads > 0 && kv_heads > 0 &&
        (q_out == k_out || !apart(q_out, q_out_token_stride, q_heads * head_dim, k_out, k_out_token_stride,
                                  kv_heads * head_dim, num_tokens, e)))
        return GAI4_ERR_INVALID_ARG;
    return done(launch_rope(L, (cudaStream_t)stream));
}

gai4_status gai4_rms_norm(const void* x, int64_t x_row_stride, const void* residual, int64_t residual_row_stride,
                          const void* gain, void* out, void* residual_out, uint8_t* codes, float* scales,
                          gai4_dtype dtype, int64_t rows, int64_t cols, float eps, void* stream) {
    if (!known(dtype)) return GAI4_ERR_UNSUPPORTED;
    if (rows < 0 || rows > kMost || cols < 1 || cols > kMost || !(eps >= 0.f) || !isfinite(eps))
        return GAI4_ERR_INVALID_ARG;
    if (rows == 0) return GAI4_OK;
    if (!x || (!out && !residual_out && !codes) || (codes == nullptr) != (scales == nullptr)) return GAI4_ERR_INVALID_ARG;
    if (!strided(x_row_stride, cols, rows) || (residual && !strided(residual_row_stride, cols, rows)))
        return GAI4_ERR_INVALID_ARG;
    const uintptr_t e = elem_bytes(dtype);
    for (const void* p : {x, residual, gain, (const void*)out, (const void*)residual_out})
        if (!aligned_to(p, e)) return GAI4_ERR_MISALIGNED;
    if (!aligned_to(scales, 4)) return GAI4_ERR_MISALIGNED;
    if (out && out == residual_out) return GAI4_ERR_INVALID_ARG;
    for (const void* o : {(const void*)out, (const void*)residual_out})
        if (o && (!apart(x, x_row_stride, cols, o, cols, cols, rows, (int64_t)e) ||
                  (residual && !apart(residual, residual_row_stride, cols, o, cols, cols, rows, (int64_t)e))))
            return GAI4_ERR_INVALID_ARG;
    return done(launch_rms_norm(x, x_row_stride, residual, residual_row_stride, gain, out, residual_out, codes, scales,
                                dtype, rows, cols, eps, (cudaStream_t)stream));
}

gai4_status gai4_quantize_x_fp8(const void* x, int64_t x_row_stride, uint8_t* codes, float* scales, gai4_dtype dtype,
                                int64_t M, int64_t K, void* stream) {
    if (!known(dtype)) return GAI4_ERR_UNSUPPORTED;
    if (M < 0 || M > kMost || K < 1 || K > kMost) return GAI4_ERR_INVALID_ARG;
    if (M == 0) return GAI4_OK;
    if (!strided(x_row_stride, K, M)) return GAI4_ERR_INVALID_ARG;
    if (!x || !codes || !scales) return GAI4_ERR_INVALID_ARG;
    if (!aligned_to(x, elem_bytes(dtype)) || !aligned_to(scales, 4)) return GAI4_ERR_MISALIGNED;
    return done(launch_quantize_x_fp8(x, x_row_stride, codes, scales, dtype, M, K, (cudaStream_t)stream));
}

gai4_status gai4_quantize_fp8(const void* w, uint8_t* codes, float* scales, gai4_dtype dtype, int64_t N, int64_t K,
                              void* stream) {
    if (!known(dtype)) return GAI4_ERR_UNSUPPORTED;
    if (N < 1 || N > 65535 * 128 || K < 1 || K > kMost) return GAI4_ERR_INVALID_ARG;   // (grid y: 65535)
    if (!w || !codes || !scales) return GAI4_ERR_INVALID_ARG;
    if (!aligned_to(w, elem_bytes(dtype)) || !aligned_to(scales, 4)) return GAI4_ERR_MISALIGNED;
    return done(launch_quantize_fp8(w, codes, scales, dtype, N, K, (cudaStream_t)stream));
}

gai4_status gai4_fp8_mm_t(const uint8_t* w_codes, const float* w_scales, const uint8_t* x_codes, const float* x_scales,
                          void* out, gai4_dtype dtype, int64_t M, int64_t N, int64_t K, void* stream) {
    Fp8MmLaunch L{w_codes, w_scales, x_codes, x_scales, out, M, N, K, nullptr, 2000000000LL, 0};   // ~1 s a wait
    return fp8_mm(L, dtype, stream);
}

gai4_status gai4_fp8_mm_t_plan(int64_t M, int64_t N, int64_t K, gai4_dtype dtype, int* tokens, int* weight_rows, int* ctas) {
    if (!tokens || !weight_rows || !ctas) return GAI4_ERR_INVALID_ARG;
    const gai4_status sizes = fp8_mm_sizes(dtype, M, N, K);
    if (sizes != GAI4_OK) return sizes;
    if (M == 0) return GAI4_ERR_INVALID_ARG;
    Fp8MmLaunch L{nullptr, nullptr, nullptr, nullptr, nullptr, M, N, K, nullptr, 0, 0};
    if (cudaGetDevice(&L.device) != cudaSuccess || L.device >= 64) return GAI4_ERR_CUDA;
    plan_fp8_mm(L, dtype, tokens, weight_rows, ctas);
    return GAI4_OK;
}

gai4_status gai4_check_fp8_mm_wait(const uint8_t* w_codes, const float* w_scales, const uint8_t* x_codes,
                                   const float* x_scales, void* out, gai4_dtype dtype, int64_t M, int64_t N, int64_t K,
                                   int withheld, int blocks, int64_t limit_cycles, int* status, void* stream) {
    if (!status || withheld < 0 || withheld > 15 || blocks < 0 || limit_cycles <= 0 || limit_cycles > 4000000000LL)
        return GAI4_ERR_INVALID_ARG;
    if (!aligned_to(status, 4)) return GAI4_ERR_MISALIGNED;
    Fp8MmLaunch L{w_codes, w_scales, x_codes, x_scales, out, M, N, K, status, limit_cycles, 0};
    for (int i = 0; i < 4; ++i)
        if (withheld >> i & 1) L.until[i >> 1][i & 1] = blocks;
    return fp8_mm(L, dtype, stream);
}

}  // extern "C"
