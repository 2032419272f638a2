// kv_attention_f16.cu -- attention over the 4-bit cache, f16 activations.
#include "kv_attention.cuh"

namespace gai4 {
cudaError_t launch_kv_attention_f16(const KvAttnLaunch& L, cudaStream_t s) { return kvs::launch_type<F16>(L, s); }
}  // namespace gai4
