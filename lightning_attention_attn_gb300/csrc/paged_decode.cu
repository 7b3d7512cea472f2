// Attention of one new token per request over its whole cache; the kernels are in
// paged_attention.cuh.
#include "paged_attention.cuh"

namespace la {

cudaError_t paged_decode(const PagedDecodeArgs &a, bool bf16, bool q_f32) {
    if (a.head_dim == 128) return dispatch<Kv::kOwn, 128>(a, bf16, q_f32);
    if (a.head_dim == 64) return dispatch<Kv::kOwn, 64>(a, bf16, q_f32);
    return cudaErrorNotSupported;
}

}  // namespace la
