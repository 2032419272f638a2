// kv_attention_f32.cu -- attention over the 4-bit cache, f32 activations.
#include "kv_attention.cuh"

namespace gai4 {
cudaError_t launch_kv_attention_f32(const KvAttnLaunch& L, cudaStream_t s) { return kvs::launch_type<F32>(L, s); }
}  // namespace gai4
