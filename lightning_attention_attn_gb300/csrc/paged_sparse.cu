// Attention of one new token per request over chosen pages of its cache: the kernels of
// paged_attention.cuh, which go by a list of blocks for each request and key-value head instead
// of all of the request's blocks.  The entries that count are known from the length alone, so
// units and ranges are those of a cache of that many full pages; rows of a page
// behind the request's last token are absent, as those of an absent page.
#include "paged_attention.cuh"

namespace la {

cudaError_t paged_sparse_decode(const PagedDecodeArgs &a, bool bf16) {
    if (a.head_dim == 128) return dispatch<Kv::kChosen, 128>(a, bf16);
    if (a.head_dim == 64) return dispatch<Kv::kChosen, 64>(a, bf16);
    return cudaErrorNotSupported;
}

}  // namespace la
