// Instantiations of the attention kernel for trees of drafts: per-token 4-bit caches.
#include "shared_kernel.cuh"

namespace pkv {

template <int D, bool BF>
static const void* of(bool few) {
  return few ? reinterpret_cast<const void*>(&shared_attention_kernel<D, KV_U4T, BF, kFewDrafts>)
             : reinterpret_cast<const void*>(&shared_attention_kernel<D, KV_U4T, BF, kDraftRows>);
}

const void* tree_kernel_u4t(int D, bool bf, bool few) {
  return D == 64 ? (bf ? of<64, true>(few) : of<64, false>(few)) : (bf ? of<128, true>(few) : of<128, false>(few));
}

}  // namespace pkv
