// Chunk attention on tcgen05: bf16 rows.
#include "chunk_attn_tc.cuh"

namespace spec {
namespace ca {

TcFn tc_kernel_bf16(bool f8, int mode) { return tc_kernel_of<__nv_bfloat16>(f8, mode); }

}  // namespace ca
}  // namespace spec

// per-unit log setter of the instrumented build (no-op otherwise)
SPEC_TL_SETTER(chunk_attn_bf16)
