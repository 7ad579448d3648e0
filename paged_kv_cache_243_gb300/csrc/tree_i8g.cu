// Instantiations of the attention kernel for trees of drafts: per-group INT8 caches.
#include "shared_kernel.cuh"

namespace pkv {

template <int D, bool BF>
static const void* of(bool few) {
  return few ? reinterpret_cast<const void*>(&shared_attention_kernel<D, KV_I8G, BF, kFewDrafts>)
             : reinterpret_cast<const void*>(&shared_attention_kernel<D, KV_I8G, BF, kDraftRows>);
}

const void* tree_kernel_i8g(int D, bool bf, bool few) {
  return D == 64 ? (bf ? of<64, true>(few) : of<64, false>(few)) : (bf ? of<128, true>(few) : of<128, false>(few));
}

}  // namespace pkv
