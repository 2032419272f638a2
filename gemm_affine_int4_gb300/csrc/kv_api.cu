// kv_api.cu -- C ABI of the paged 4-bit key/value cache (declared in
// include/gai4.h): argument validation and launch. No allocation.
#include <stdint.h>

#include <algorithm>

#include "common.cuh"
#include "internal.h"

using namespace gai4;

namespace {

bool aligned_to(const void* p, uintptr_t n) { return ((uintptr_t)p % n) == 0; }

int log2_page(int page_size) {
    for (int l = 4; l <= 8; ++l)
        if (page_size == 1 << l) return l;
    return -1;
}

int elem_bytes(int dtype) { return dtype == GAI4_F32 ? 4 : 2; }

// the cache's own sizes; fills `sh`
gai4_status check_shape(int dtype, int gs, int64_t hkv, int d, int64_t num_blocks, int page_size, KvShape* sh) {
    if (dtype != GAI4_F32 && dtype != GAI4_F16 && dtype != GAI4_BF16) return GAI4_ERR_UNSUPPORTED;
    if ((d != 64 && d != 128) || (gs != 32 && gs != 64 && gs != 128) || gs > d) return GAI4_ERR_UNSUPPORTED;
    const int pl = log2_page(page_size);
    if (pl < 0) return GAI4_ERR_UNSUPPORTED;
    if (hkv < 1 || hkv > 65535 || num_blocks < 1 || num_blocks > 0x7fffffff) return GAI4_ERR_INVALID_ARG;
    *sh = KvShape{dtype, gs, (int)hkv, d, pl, num_blocks};
    return GAI4_OK;
}

gai4_status check_cache(const KvCache& c) {
    if (!c.packed || !c.scales || !c.biases) return GAI4_ERR_INVALID_ARG;
    if (!aligned_to(c.packed, 16) || !aligned_to(c.scales, 16) || !aligned_to(c.biases, 16))
        return GAI4_ERR_MISALIGNED;
    return GAI4_OK;
}

// Query rows per key/value head up to which the split kernel (8 or 16 rows a
// pass over the keys) is taken; above, the tensor-core kernel (256 rows a
// pass). Split / tensor-core kernel in us, bf16, 8 key/value heads of 128, at
// 16, 24, 32 and 40 rows: 16 requests of 4000 tokens 45/67, 70/67, 76/68,
// 102/68; 20 of 16000 138/215, -, 257/217, 369/217; 64 of 1000 78/110, -,
// 133/112, -; one of 4000 17/-, 18/-, 18/-, 21/37. The two meet between 24 and
// 32 rows, and up to there the split kernel also rounds less.
constexpr int kManyRows = 32;

// the split kernel: two records of 16 query rows (32-bit O, m, l) for each of
// two CTAs per SM, and a line of 16 bytes per CTA; the tensor-core kernel's
// records are longer
size_t attention_workspace(int d, int dtype) {
    const size_t ctas = 2 * (size_t)num_sms();
    const size_t split = (ctas * 16 + 255) / 256 * 256 + ctas * 2 * 16 * (size_t)(d + 2) * 4;
    return dtype == GAI4_F32 ? split : std::max(split, kv_attention_tc_workspace(d));
}

gai4_status done(cudaError_t e) { return e == cudaSuccess ? GAI4_OK : GAI4_ERR_CUDA; }

}  // namespace

extern "C" {

gai4_status gai4_kv_plan(const int32_t* kv_lens, const int32_t* q_lens, int32_t* block_table, int64_t max_blocks,
                         int32_t* free_blocks, int64_t free_capacity, const int32_t* free_count, int64_t* slots,
                         int32_t* positions, int64_t num_tokens, int32_t* cu_q, int32_t* kv_lens_out,
                         int32_t* free_count_out, int32_t* info, int64_t batch, int page_size, void* stream) {
    const int pl = log2_page(page_size);
    if (pl < 0 || batch > kKvPlanMaxBatch) return GAI4_ERR_UNSUPPORTED;
    if (batch < 1 || max_blocks < 1 || max_blocks > (0x7fffffff >> pl) || free_capacity < 1 ||
        free_capacity > 0x7fffffff || num_tokens < 0 || num_tokens > 0x7fffffff)
        return GAI4_ERR_INVALID_ARG;
    if (!kv_lens || !q_lens || !block_table || !free_blocks || !free_count || !cu_q || !kv_lens_out ||
        !free_count_out || !info || (num_tokens > 0 && (!slots || !positions)))
        return GAI4_ERR_INVALID_ARG;
    if (kv_lens_out == kv_lens || free_count_out == free_count) return GAI4_ERR_INVALID_ARG;
    const void* words[] = {kv_lens, q_lens, block_table, free_blocks, free_count, positions, cu_q, kv_lens_out,
                           free_count_out, info};
    for (const void* p : words)
        if (!aligned_to(p, 4)) return GAI4_ERR_MISALIGNED;
    if (!aligned_to(slots, 8)) return GAI4_ERR_MISALIGNED;
    const KvPlanLaunch L{kv_lens, q_lens, block_table, max_blocks, free_blocks, free_capacity, free_count, slots,
                         positions, num_tokens, cu_q, kv_lens_out, free_count_out, info, (int)batch, pl};
    return done(launch_kv_plan(L, (cudaStream_t)stream));
}

gai4_status gai4_kv_append(const void* k, int64_t k_token_stride, const void* v, int64_t v_token_stride,
                           const int64_t* slots, uint32_t* k_packed, void* k_scales, void* k_biases,
                           uint32_t* v_packed, void* v_scales, void* v_biases, gai4_dtype dtype, int group_size,
                           int64_t num_tokens, int64_t kv_heads, int head_dim, int64_t num_blocks, int page_size,
                           void* stream) {
    KvShape sh;
    gai4_status st = check_shape(dtype, group_size, kv_heads, head_dim, num_blocks, page_size, &sh);
    if (st != GAI4_OK) return st;
    if (num_tokens < 0 || num_tokens > 0x7fffffff) return GAI4_ERR_INVALID_ARG;
    const KvCache kc{k_packed, k_scales, k_biases}, vc{v_packed, v_scales, v_biases};
    if ((st = check_cache(kc)) != GAI4_OK || (st = check_cache(vc)) != GAI4_OK) return st;
    if (num_tokens == 0) return GAI4_OK;
    if (!k || !v || !slots) return GAI4_ERR_INVALID_ARG;
    if (k_token_stride < kv_heads * head_dim || v_token_stride < kv_heads * head_dim) return GAI4_ERR_INVALID_ARG;
    const uintptr_t e = (uintptr_t)elem_bytes(dtype);
    if (!aligned_to(k, e) || !aligned_to(v, e) || !aligned_to(slots, 8)) return GAI4_ERR_MISALIGNED;
    return done(launch_kv_append(k, k_token_stride, v, v_token_stride, slots, kc, vc, sh, num_tokens,
                                 (cudaStream_t)stream));
}

gai4_status gai4_kv_read(const uint32_t* packed, const void* scales, const void* biases, const int64_t* slots,
                         float* out, gai4_dtype dtype, int group_size, int64_t num_tokens, int64_t kv_heads,
                         int head_dim, int64_t num_blocks, int page_size, void* stream) {
    KvShape sh;
    gai4_status st = check_shape(dtype, group_size, kv_heads, head_dim, num_blocks, page_size, &sh);
    if (st != GAI4_OK) return st;
    if (num_tokens < 0 || num_tokens > 0x7fffffff) return GAI4_ERR_INVALID_ARG;
    const KvCache c{packed, scales, biases};
    if ((st = check_cache(c)) != GAI4_OK) return st;
    if (num_tokens == 0) return GAI4_OK;
    if (!slots || !out) return GAI4_ERR_INVALID_ARG;
    if (!aligned_to(out, 16) || !aligned_to(slots, 8)) return GAI4_ERR_MISALIGNED;
    return done(launch_kv_read(c, slots, out, sh, num_tokens, (cudaStream_t)stream));
}

size_t gai4_kv_attention_workspace_bytes(int64_t q_heads, int64_t kv_heads, int head_dim, gai4_dtype dtype) {
    KvShape sh;
    if (check_shape(dtype, 32, kv_heads, head_dim, 1, 16, &sh) != GAI4_OK) return 0;
    if (q_heads < 1 || q_heads % kv_heads != 0 || q_heads / kv_heads > 65535) return 0;
    return attention_workspace(head_dim, dtype);
}

gai4_status gai4_kv_attention(const void* q, int64_t q_token_stride, const uint32_t* k_packed, const void* k_scales,
                              const void* k_biases, const uint32_t* v_packed, const void* v_scales,
                              const void* v_biases, const int32_t* block_table, int64_t max_blocks,
                              const int32_t* kv_lens, const int32_t* cu_q, void* out, int64_t out_token_stride,
                              float* lse, gai4_dtype dtype, int group_size, int64_t batch, int64_t num_tokens,
                              int64_t max_q_len, int64_t q_heads, int64_t kv_heads, int head_dim, int64_t num_blocks,
                              int page_size, float scale, int64_t window, void* workspace, size_t workspace_bytes,
                              void* stream) {
    KvAttnLaunch L;
    gai4_status st = check_shape(dtype, group_size, kv_heads, head_dim, num_blocks, page_size, &L.sh);
    if (st != GAI4_OK) return st;
    if (q_heads < 1 || q_heads % kv_heads != 0 || q_heads / kv_heads > 65535) return GAI4_ERR_INVALID_ARG;
    // the kernels step through a request's tokens in 32 bits, up to 1200 past its last tile
    constexpr int64_t most_tokens = 0x80000000ll - 4096;
    if (batch < 1 || batch > 0x7ffffff || num_tokens < 0 || num_tokens > 0x7fffffff || max_q_len < 0 || max_blocks < 1 ||
        max_blocks > (most_tokens >> L.sh.page_log2) || window < 0)
        return GAI4_ERR_INVALID_ARG;
    L.k = KvCache{k_packed, k_scales, k_biases};
    L.v = KvCache{v_packed, v_scales, v_biases};
    if ((st = check_cache(L.k)) != GAI4_OK || (st = check_cache(L.v)) != GAI4_OK) return st;
    if (num_tokens * (q_heads / kv_heads) > 0x7fffffff) return GAI4_ERR_UNSUPPORTED;   // 32-bit row numbers
    if (num_tokens == 0) return GAI4_OK;
    if (!q || !out || !block_table || !kv_lens || !cu_q) return GAI4_ERR_INVALID_ARG;
    if (q_token_stride < q_heads * head_dim || out_token_stride < q_heads * head_dim) return GAI4_ERR_INVALID_ARG;
    const uintptr_t e = (uintptr_t)elem_bytes(dtype);
    if (!aligned_to(q, e) || !aligned_to(out, e) || !aligned_to(block_table, 4) || !aligned_to(kv_lens, 4) ||
        !aligned_to(cu_q, 4) || !aligned_to(lse, 4))
        return GAI4_ERR_MISALIGNED;
    L.group = (int)(q_heads / kv_heads);
    if (!workspace || workspace_bytes < attention_workspace(head_dim, dtype)) return GAI4_ERR_WORKSPACE;
    if (!aligned_to(workspace, 16)) return GAI4_ERR_MISALIGNED;
    L.q = q;
    L.q_stride = q_token_stride;
    L.table = block_table;
    L.max_blocks = max_blocks;
    L.kv_lens = kv_lens;
    L.cu_q = cu_q;
    L.out = out;
    L.out_stride = out_token_stride;
    L.lse = lse;
    L.batch = (int)batch;
    L.num_tokens = num_tokens;
    L.max_q_len = std::min(max_q_len, num_tokens);   // (times the group: below 2^31)
    L.scale = scale;
    L.window = std::min<int64_t>(window, 0x7fffffff);   // no position is beyond it, and position - window stays in 64 bits
    L.workspace = workspace;
    L.status = status_ptr();
    L.spin_limit = 2000000000LL;   // ~1 s of SM clock per wait
    if (!L.status) return GAI4_ERR_CUDA;
    cudaStream_t cs = (cudaStream_t)stream;
    if (dtype == GAI4_F32) return done(launch_kv_attention_f32(L, cs));
    if (L.max_q_len * L.group > kManyRows) return done(launch_kv_attention_tc(L, cs));
    return done(dtype == GAI4_F16 ? launch_kv_attention_f16(L, cs) : launch_kv_attention_bf16(L, cs));
}

}  // extern "C"
