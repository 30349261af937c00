// Attention of one new token per request over the paged cache.
//
// [NEURON] "KV Cache Sharing": the paged cache the draft layer and the target
// share; this is the decode step of a request that is not speculated on.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace spec {

enum : unsigned { kTLPagedAttn = 26 };   // after common.cuh's ids

struct PaArgs {
  spec_attn_desc d;
  spec_kv kv;
  const void* q;
  void* out;
  float* lse;
  const int32_t* seq_len;
  long long q_ld, out_ld;
  int B, G;
  float scale;
  void* ws;
};

SPEC_DEV float val(float x) { return x; }
SPEC_DEV float val(__nv_bfloat16 x) { return __bfloat162float(x); }
SPEC_DEV float val(__half x) { return __half2float(x); }
SPEC_DEV float val(__nv_fp8_e4m3 x) { return (float)x; }
SPEC_DEV void put(float* p, float v) { *p = v; }
SPEC_DEV void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
SPEC_DEV void put(__half* p, float v) { *p = __float2half_rn(v); }

// A CTA per (request, kv head, up to 8 of its query heads); warps take keys in
// turn, lanes hold head_dim / 32 components; the warps' results are joined.
template <typename T, typename C>
__global__ void __launch_bounds__(256) paged_attention_kernel(const PaArgs g) {
  SPEC_TL(kTLPagedAttn);
  pdl_wait();
  pdl_trigger();
  constexpr int NQ = 8, ND = 8;
  const int b = blockIdx.z, h = blockIdx.y, q0 = blockIdx.x * NQ, nq = min(NQ, g.G - q0);
  const int hd = g.d.head_dim, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int nkv = g.d.n_kv_heads;
  int len = g.seq_len[b];
  const long long most = (long long)g.kv.max_blocks * g.kv.block_size;
  if (len < 0 || len > most) {
    if (tid == 0) report(g.ws, SPEC_ERR_DEVICE, b, len);
    len = len < 0 ? 0 : (int)most;
  }
  const int lo = g.d.window > 0 ? max(0, len - g.d.window) : 0;
  __shared__ float sm_m[8][NQ], sm_l[8][NQ], sm_o[8][256];
  float q[NQ][ND], o[NQ][ND], m[NQ], l[NQ];
  for (int i = 0; i < NQ; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int e = 0; e < ND; ++e) {
      const int c = lane + 32 * e;
      o[i][e] = 0.f;
      q[i][e] = i < nq && c < hd
                    ? val(static_cast<const T*>(g.q)[b * g.q_ld + (long long)(h * g.G + q0 + i) * hd + c]) : 0.f;
    }
  }
  for (int t = lo + warp; t < len; t += 8) {
    const long long slot = slot_of(g.kv, b, t);
    if (slot < 0) {
      if (lane == 0) report(g.ws, SPEC_ERR_DEVICE, b, t);
      continue;
    }
    const C* kr = static_cast<const C*>(g.kv.k) + (slot * nkv + h) * hd;
    const C* vr = static_cast<const C*>(g.kv.v) + (slot * nkv + h) * hd;
    float k[ND], v[ND];
#pragma unroll
    for (int e = 0; e < ND; ++e) {
      const int c = lane + 32 * e;
      k[e] = c < hd ? val(kr[c]) : 0.f;
      v[e] = c < hd ? val(vr[c]) : 0.f;
    }
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      float s = 0.f;
#pragma unroll
      for (int e = 0; e < ND; ++e) s = fmaf(q[i][e], k[e], s);
      s = warp_sum(s) * g.scale;
      const float mn = fmaxf(m[i], s), a = expf(m[i] - mn), p = expf(s - mn);
      m[i] = mn;
      l[i] = l[i] * a + p;
#pragma unroll
      for (int e = 0; e < ND; ++e) o[i][e] = fmaf(p, v[e], o[i][e] * a);
    }
  }
  for (int i = 0; i < NQ; ++i)
    if (lane == 0) {
      sm_m[warp][i] = m[i];
      sm_l[warp][i] = l[i];
    }
  const float vs = g.d.kv_dtype == SPEC_DTYPE_E4M3 ? g.d.v_scale : 1.f;
#pragma unroll
  for (int i = 0; i < NQ; ++i) {
    __syncthreads();
#pragma unroll
    for (int e = 0; e < ND; ++e) sm_o[warp][lane + 32 * e] = o[i][e];
    __syncthreads();
    if (i < nq) {
      float mm = -INFINITY, ll = 0.f, x = 0.f;
      for (int w = 0; w < 8; ++w) mm = fmaxf(mm, sm_m[w][i]);
      for (int w = 0; w < 8; ++w)
        if (sm_m[w][i] > -INFINITY) {
          const float a = expf(sm_m[w][i] - mm);
          ll += a * sm_l[w][i];
          x += a * sm_o[w][tid];
        }
      const int head = h * g.G + q0 + i;
      if (tid < hd) put(static_cast<T*>(g.out) + b * g.out_ld + (long long)head * hd + tid, ll > 0.f ? x / ll * vs : 0.f);
      if (tid == 0 && g.lse) g.lse[(long long)b * g.d.n_q_heads + head] = ll > 0.f ? mm + logf(ll) : -INFINITY;
    }
  }
}

static bool check_attn(const spec_attn_desc* d) {
  return d && d->n_q_heads > 0 && d->n_kv_heads > 0 && d->n_q_heads % d->n_kv_heads == 0 &&
         d->n_q_heads / d->n_kv_heads <= 128 && d->head_dim > 0 && d->head_dim % 16 == 0 && d->head_dim <= 256 &&
         d->window >= 0;
}

}  // namespace spec

using namespace spec;

extern "C" size_t spec_attention_workspace_bytes(const spec_attn_desc* desc, int32_t max_B) {
  if (!check_attn(desc) || max_B <= 0) return 0;
  return kWsHeader;
}

extern "C" spec_status spec_paged_attention(const spec_attn_desc* desc, const void* q, int64_t q_ld, const spec_kv* kv,
                                            const int32_t* seq_len, int32_t B, int32_t max_len, void* out,
                                            int64_t out_ld, float* lse, void* ws, size_t ws_bytes,
                                            spec_stream_t stream) {
  if (!desc || !q || !kv || !kv->k || !kv->v || !kv->block_table || !seq_len || !out) return SPEC_ERR_ARG;
  const spec_attn_desc& d = *desc;
  if (!check_attn(desc) || B <= 0 || B > 65535 || max_len < 0 || kv->block_size <= 0 || kv->max_blocks <= 0 ||
      kv->num_slots <= 0 || (long long)kv->max_blocks * kv->block_size >= (1ll << 31))
    return SPEC_ERR_SHAPE;
  if (d.dtype < SPEC_DTYPE_F32 || d.dtype > SPEC_DTYPE_F16) return SPEC_ERR_UNSUPPORTED;
  const bool e4m3 = d.kv_dtype == SPEC_DTYPE_E4M3 && d.dtype != SPEC_DTYPE_F32;
  if (d.kv_dtype != d.dtype && !e4m3) return SPEC_ERR_UNSUPPORTED;
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
  PaArgs g{};
  g.d = d, g.kv = *kv, g.q = q, g.out = out, g.lse = lse, g.seq_len = seq_len, g.q_ld = q_ld, g.out_ld = out_ld;
  g.B = B, g.G = d.n_q_heads / d.n_kv_heads, g.ws = ws;
  g.scale = (d.scale > 0 ? d.scale : 1.f / sqrtf((float)d.head_dim)) * (e4m3 ? d.k_scale : 1.f);
  const dim3 grid((g.G + 7) / 8, d.n_kv_heads, B);
  auto* kern = d.dtype == SPEC_DTYPE_F32 ? paged_attention_kernel<float, float>
               : d.dtype == SPEC_DTYPE_BF16
                   ? (e4m3 ? paged_attention_kernel<__nv_bfloat16, __nv_fp8_e4m3>
                           : paged_attention_kernel<__nv_bfloat16, __nv_bfloat16>)
                   : (e4m3 ? paged_attention_kernel<__half, __nv_fp8_e4m3> : paged_attention_kernel<__half, __half>);
  launch_pdl(kern, grid, dim3(256), 0, stream, g);
  return last_launch();
}

// per-unit log setter of the instrumented build (no-op otherwise)
SPEC_TL_SETTER(paged_attn)
