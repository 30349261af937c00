// Instantiations of the paged attention kernel for fp16 queries (fp16 and 8-bit caches).
#include "paged_attn.cuh"

namespace spec {
namespace pa {
Kernel kernel_f16(bool e4m3, int hd, int G) {
  return e4m3 ? pick16<__half, true>(hd, G) : pick16<__half, false>(hd, G);
}
}  // namespace pa
}  // namespace spec

// per-unit log setter of the instrumented build (no-op otherwise)
SPEC_TL_SETTER(paged_attn_f16)
