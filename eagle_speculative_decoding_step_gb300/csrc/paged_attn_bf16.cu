// Instantiations of the paged attention kernel for bf16 queries (bf16 and 8-bit caches).
#include "paged_attn.cuh"

namespace spec {
namespace pa {
Kernel kernel_bf16(bool e4m3, int hd, int G) {
  return e4m3 ? pick16<__nv_bfloat16, true>(hd, G) : pick16<__nv_bfloat16, false>(hd, G);
}
}  // namespace pa
}  // namespace spec

// per-unit log setter of the instrumented build (no-op otherwise)
SPEC_TL_SETTER(paged_attn_bf16)
