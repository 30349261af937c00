// Chunk attention on tcgen05: f16 rows.
#include "chunk_attn_tc.cuh"

namespace spec {
namespace ca {

TcFn tc_kernel_f16(bool f8, int mode) { return tc_kernel_of<__half>(f8, mode); }

}  // namespace ca
}  // namespace spec

// per-unit log setter of the instrumented build (no-op otherwise)
SPEC_TL_SETTER(chunk_attn_f16)
