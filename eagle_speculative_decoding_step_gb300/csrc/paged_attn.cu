// Attention of one new token per request over the paged cache: plan, checks and
// launch, and the fp32 instantiations (the 16-bit ones have their own files).
//
// [NEURON] "KV Cache Sharing": the paged cache the draft layer and the target
// share; this is the decode step of a request that is not speculated on.
#include <algorithm>

#include "paged_attn.cuh"

namespace spec {
namespace pa {

Kernel kernel_f32(int hd, int) {
  if (hd <= 64) return kernel_of<F32Math<64>>();
  if (hd <= 128) return kernel_of<F32Math<128>>();
  return kernel_of<F32Math<256>>();
}

constexpr size_t kSmemMax = 227 * 1024;

static Kernel kernel_for(const spec_attn_desc& d) {
  const int G = d.n_q_heads / d.n_kv_heads;
  const bool e4m3 = d.kv_dtype == SPEC_DTYPE_E4M3;
  if (d.dtype == SPEC_DTYPE_F32) return kernel_f32(d.head_dim, G);
  return d.dtype == SPEC_DTYPE_BF16 ? kernel_bf16(e4m3, d.head_dim, G) : kernel_f16(e4m3, d.head_dim, G);
}

static int pow2_up(int x) {
  int p = 1;
  while (p < x) p <<= 1;
  return p;
}

// query tiles and splits do not depend on the heads of a tile
static void plan_queries(const Kernel& k, int G, Plan* p) {
  p->qtiles = (G + k.kq - 1) / k.kq;
  p->qt = std::min(pow2_up(p->qtiles), k.warps);
  p->qs = (p->qtiles + p->qt - 1) / p->qt;
}

static Plan make(const Kernel& k, const spec_attn_desc& d, int nh, int B) {
  Plan p{};
  plan_queries(k, d.n_q_heads / d.n_kv_heads, &p);
  p.nh = nh;
  p.kg = k.warps / (p.nh * p.qt);
  p.kt = p.kg * k.sub;
  p.hgq = d.n_kv_heads / p.nh * p.qs;
  p.row = p.nh * d.head_dim * k.es;
  p.stride = p.row + ((p.row / 16) % 2 == 0 ? 16 : 0);
  p.slots = (int)std::min<size_t>(kMaxSlots, (kSmemMax - 1024 - k.fixed(B)) / ((size_t)p.kt * p.stride));
  return p;
}

static Plan plan(const Kernel& k, const spec_attn_desc& d, int B, int max_len, int sms) {
  Plan q{};
  plan_queries(k, d.n_q_heads / d.n_kv_heads, &q);
  int nh = 1;
  while (d.n_kv_heads % (2 * nh) == 0 && 2 * nh * q.qt <= k.warps) nh *= 2;
  const int len = d.window > 0 ? std::min(d.window, max_len) : max_len;
  // the last CTA of a group to finish reads every piece of it: few heads a tile where few requests
  // are cut into many pieces
  while (nh > 1) {
    const Plan p = make(k, d, nh, B);
    const double tiles = (double)(len + p.kt - 1) / p.kt;
    const double pieces = std::min(tiles, std::max(1.0, (double)sms / ((double)B * p.hgq)));
    if (nh * pieces <= 40) break;
    nh /= 2;
  }
  return make(k, d, nh, B);
}

static bool check(const spec_attn_desc* d) {
  return d && d->n_q_heads > 0 && d->n_kv_heads > 0 && d->n_q_heads % d->n_kv_heads == 0 &&
         d->n_q_heads / d->n_kv_heads <= 128 && d->head_dim > 0 && d->head_dim % 16 == 0 && d->head_dim <= 256 &&
         d->window >= 0;
}
static bool check_types(const spec_attn_desc& d) {
  if (d.dtype < SPEC_DTYPE_F32 || d.dtype > SPEC_DTYPE_F16) return false;
  return d.kv_dtype == d.dtype || (d.kv_dtype == SPEC_DTYPE_E4M3 && d.dtype != SPEC_DTYPE_F32);
}

// Partial results come first, at the size of the largest instantiation (8 warps x 72 registers a
// lane), so that the counters lie in the same place for every descriptor and batch that shares the
// workspace and stay zero between calls.
static size_t part_bytes(int sms) { return (size_t)sms * 2 * 8 * 72 * 32 * 4; }

static size_t counter_bytes(const Kernel& k, const spec_attn_desc& d, int B) {
  Plan p{};
  plan_queries(k, d.n_q_heads / d.n_kv_heads, &p);
  return align_up((size_t)B * d.n_kv_heads * p.qs * 4, 256);
}

}  // namespace pa
}  // namespace spec

using namespace spec;

extern "C" size_t spec_attention_workspace_bytes(const spec_attn_desc* desc, int32_t max_B) {
  if (!pa::check(desc) || !pa::check_types(*desc) || max_B <= 0) return 0;
  const pa::Kernel k = pa::kernel_for(*desc);
  return kWsHeader + pa::part_bytes(sm_count()) + pa::counter_bytes(k, *desc, max_B);
}

extern "C" spec_status spec_paged_attention(const spec_attn_desc* desc, const void* q, int64_t q_ld, const spec_kv* kv,
                                            const int32_t* seq_len, int32_t B, int32_t max_len, void* out,
                                            int64_t out_ld, float* lse, void* ws, size_t ws_bytes,
                                            spec_stream_t stream) {
  if (!desc || !q || !kv || !kv->k || !kv->v || !kv->block_table || !seq_len || !out) return SPEC_ERR_ARG;
  const spec_attn_desc& d = *desc;
  if (!pa::check(desc) || B <= 0 || max_len < 0 || kv->block_size <= 0 || kv->max_blocks <= 0 ||
      kv->num_slots <= 0 || (long long)kv->max_blocks * kv->block_size >= (1ll << 31))
    return SPEC_ERR_SHAPE;
  if (!pa::check_types(d)) return SPEC_ERR_UNSUPPORTED;
  const bool e4m3 = d.kv_dtype == SPEC_DTYPE_E4M3;
  if (!(d.scale >= 0) || (e4m3 && !(d.k_scale > 0 && d.v_scale > 0))) return SPEC_ERR_ARG;
  const long long width = (long long)d.n_q_heads * d.head_dim;
  if (q_ld == 0) q_ld = width;
  if (out_ld == 0) out_ld = width;
  if (q_ld < width || out_ld < width) return SPEC_ERR_SHAPE;
  const int es = d.dtype == SPEC_DTYPE_F32 ? 4 : 2;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(kv->k, 16) || !aligned(kv->v, 16) || q_ld * es % 16 ||
      out_ld * es % 16)
    return SPEC_ERR_ALIGN;
  if (!ws || !aligned(ws, 256) || ws_bytes < spec_attention_workspace_bytes(desc, B)) return SPEC_ERR_WORKSPACE;
  const pa::Kernel k = pa::kernel_for(d);
  const int sms = sm_count();
  const int longest = max_len > 0 ? max_len : kv->max_blocks * kv->block_size;
  pa::Args g{};
  g.kv = *kv, g.q = q, g.out = out, g.lse = lse, g.seq_len = seq_len, g.q_ld = q_ld, g.out_ld = out_ld;
  g.nq = d.n_q_heads, g.nkv = d.n_kv_heads, g.G = d.n_q_heads / d.n_kv_heads, g.hd = d.head_dim, g.window = d.window;
  g.scale2 = (d.scale > 0 ? d.scale : 1.f / sqrtf((float)d.head_dim)) * (e4m3 ? d.k_scale : 1.f) * pa::kLog2e;
  g.v_scale = e4m3 ? d.v_scale : 1.f;
  g.part = reinterpret_cast<float*>(static_cast<char*>(ws) + kWsHeader);
  g.counters = reinterpret_cast<int*>(static_cast<char*>(ws) + kWsHeader + pa::part_bytes(sms));
  g.ws = ws;
  for (int b0 = 0; b0 < B; b0 += pa::kMaxB) {
    g.b0 = b0;
    g.B = std::min(B - b0, pa::kMaxB);
    g.p = pa::plan(k, d, g.B, longest, sms);
    const size_t smem = (size_t)g.p.slots * g.p.kt * g.p.stride + k.fixed(g.B);
    if (g.p.slots < 2) return SPEC_ERR_UNSUPPORTED;
    if (cudaFuncSetAttribute(k.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
      return SPEC_ERR_CUDA;
    launch_pdl(k.fn, dim3(sms), dim3(k.warps * 32 + 32), smem, stream, g);
  }
  return last_launch();
}

// per-unit log setter of the instrumented build (no-op otherwise)
SPEC_TL_SETTER(paged_attn)
