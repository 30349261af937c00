// Attention of one new token per request over the paged cache: plan, checks and
// launch, and the fp32 instantiations (the 16-bit ones have their own files).
//
// [NEURON] "KV Cache Sharing": the paged cache the draft layer and the target
// share; this is the decode step of a request that is not speculated on.
#include <algorithm>

#include "paged_attn.cuh"

namespace spec {
namespace pa {

Kernel kernel_f32(int hd, int G) {
  if (hd <= 64) return G <= 4 ? kernel_of<F32Math<64, 4>>() : kernel_of<F32Math<64, 8>>();
  if (hd <= 128) return G <= 4 ? kernel_of<F32Math<128, 4>>() : kernel_of<F32Math<128, 8>>();
  return G <= 4 ? kernel_of<F32Math<256, 4>>() : kernel_of<F32Math<256, 8>>();
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
  p->qt = std::min(pow2_up(p->qtiles), k.warps / k.vs);
  p->qs = (p->qtiles + p->qt - 1) / p->qt;
}

static Plan make(const Kernel& k, const spec_attn_desc& d, int nh, int B, int block_size) {
  Plan p{};
  plan_queries(k, d.n_q_heads / d.n_kv_heads, &p);
  p.nh = nh;
  p.kg = 1;
  while (2 * p.kg * p.nh * p.qt <= k.warps / k.vs) p.kg *= 2;
  p.kt = p.kg * k.sub;
  p.hgq = d.n_kv_heads / p.nh * p.qs;
  const int head = d.head_dim * k.es;
  const int chunks = (head + 127) / 128;
  p.swz = block_size % 8 == 0;
  if (p.swz) {
    p.run_lg = block_size % 16 == 0 && p.kt >= 16 ? 4 : 3;
    p.key_stride = 128;
    p.copies = head % 128 == 0 ? 1 : chunks;
    p.head_stride = (head % 128 == 0 ? chunks : 1) * (128 << p.run_lg);
    p.chunk_stride = (head % 128 == 0 ? 1 : p.nh) * (128 << p.run_lg);
    p.run_bytes = chunks * p.nh * (128 << p.run_lg);
    p.slot_bytes = (p.kt >> p.run_lg) * p.run_bytes;
  } else {
    p.run_lg = 8;                      // all keys of a tile are one run
    p.row = p.nh * head;
    p.key_stride = p.row + ((p.row / 16) % 2 == 0 ? 16 : 0);
    p.head_stride = head;
    p.chunk_stride = 128;
    p.slot_bytes = (int)align_up((size_t)p.kt * p.key_stride, 16);
  }
  p.full = d.head_dim == k.hd || (p.swz && chunks == (k.hd * k.es + 127) / 128);
  p.slots = (int)std::min<size_t>(kMaxSlots, (kSmemMax - 1024 - k.fixed(B)) / p.slot_bytes);
  return p;
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The cache as [nkv][chunks][slots][128 bytes], boxes of one run of slots over the tile's heads and all chunks.  Where
// a row is no multiple of 128 bytes a last chunk would run into the next head: there the view is [nkv][1][slots][row],
// copied in 128-byte steps.  What is past a row's or the cache's end reads as zeros.
static bool run_map(CUtensorMap* tm, const void* ptr, const spec_attn_desc& d, const spec_kv& kv, const Kernel& k,
                    const Plan& p) {
  static const EncodeTiledFn enc = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    const bool ok = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) ==
                        cudaSuccess && q == cudaDriverEntryPointSuccess;
    return ok ? reinterpret_cast<EncodeTiledFn>(f) : nullptr;
  }();
  if (!enc) return false;
  const CUtensorMapDataType type = d.kv_dtype == SPEC_DTYPE_F32    ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                   : d.kv_dtype == SPEC_DTYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                   : d.kv_dtype == SPEC_DTYPE_F16  ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                                   : CU_TENSOR_MAP_DATA_TYPE_UINT8;
  const cuuint64_t head = (cuuint64_t)d.head_dim * k.es;
  const cuuint32_t whole = head % 128 == 0 ? (cuuint32_t)(head / 128) : 1;
  cuuint64_t dims[4] = {head % 128 == 0 ? (cuuint64_t)(128 / k.es) : (cuuint64_t)d.head_dim, (cuuint64_t)kv.num_slots,
                        whole, (cuuint64_t)d.n_kv_heads};
  cuuint64_t strides[3] = {d.n_kv_heads * head, 128, head};
  cuuint32_t box[4] = {(cuuint32_t)(128 / k.es), 1u << p.run_lg, whole, (cuuint32_t)p.nh};
  cuuint32_t es[4] = {1, 1, 1, 1};
  // L2 fetches past a row's end what the row does not fill, and the next head's copy again (64 requests of 4000 keys,
  // 256 / 128 / 64 bytes: 8 heads of 80 bytes 110 / 89 / 93 us, 3 heads of 224 91 / 79 / 67; of 256: no difference)
  const CUtensorMapL2promotion ahead = head % 128 == 0 ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B
                                       : head < 128    ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B
                                                       : CU_TENSOR_MAP_L2_PROMOTION_L2_64B;
  return enc(tm, type, 4, const_cast<void*>(ptr), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, ahead,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Heads of a tile: the cheapest by share_out() with every request as long as the longest.  Small copies cost
// more where a request's heads are not all under way at once: 64 requests of up to 8190 keys, 8 heads of 256 bytes,
// 8 / 4 / 2 / 1 heads a tile, copies of 32 / 16 / 8 / 4 KB: 162 / 162 / 166 / 185 us (16 requests of 4000:
// 46.7 / 46.2 / 46.0 / 45.3); and always in 8 bits: 64 requests of 4000, copies of 16 / 8 / 4 / 2 KB 86 / 86 / 87 / 125 us.
static Plan plan(const Kernel& k, const spec_attn_desc& d, int B, int max_len, int block_size, int sms) {
  Plan q{}, best{};
  plan_queries(k, d.n_q_heads / d.n_kv_heads, &q);
  const int len = d.window > 0 ? std::min(d.window, max_len) : max_len;
  float least = 0.f;
  for (int nh = 1; nh * q.qt <= k.warps / k.vs; ++nh) {
    if (d.n_kv_heads % nh != 0) continue;
    const Plan p = make(k, d, nh, B, block_size);
    const int tiles = std::max(1, (len + p.kt - 1) / p.kt);
    const long long items = (long long)B * p.hgq, copy = (long long)(p.swz ? 1 << p.run_lg : 1) * nh * d.head_dim * k.es;
    int cuts;
    // Rows: tiles are smaller where warps are left over (3 or 5 heads), and a single key's copy wants 2 KB (64 requests
    // of 4000 keys, blocks of one slot, 8 heads of 256 bytes, copies of 2048 / 1024 / 512 / 256 bytes: 159 / 166 / 232 /
    // 361 us).  Runs: a smaller tile takes a warp as long as a whole one.
    const float form = p.swz ? (copy >= 16384 || (items <= sms && k.es > 1) ? 1.f : copy >= 8192 ? 1.08f : 1.25f)
                             : (copy >= 2048 ? 1.f : copy >= 1024 ? 1.2f : copy >= 512 ? 1.7f : 2.8f) *
                                   (float)(p.nh * p.qt * p.kg * k.vs) / (float)k.warps;
    const float cost = share_out(items * tiles, items, tiles, p.kg, sms, &cuts) * form;
    if (nh == 1 || cost < least) least = cost, best = p;
  }
  return best;
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

static int group_ints(int sms) { return (int)align_up((size_t)2 * sms, 64); }

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
  return kWsHeader + pa::part_bytes(sm_count()) + (size_t)pa::group_ints(sm_count()) * 4 +
          pa::counter_bytes(k, *desc, max_B);
}

extern "C" spec_status spec_paged_attention(const spec_attn_desc* desc, const void* q, int64_t q_ld, const spec_kv* kv,
                                            const int32_t* seq_len, int32_t B, int32_t max_len, void* out,
                                            int64_t out_ld, float* lse, void* ws, size_t ws_bytes,
                                            spec_stream_t stream) {
  if (!desc || !q || !kv || !kv->k || !kv->v || !kv->block_table || !seq_len || !out) return SPEC_ERR_ARG;
  const spec_attn_desc& d = *desc;
  if (!pa::check(desc) || B <= 0 || max_len < 0 || kv->block_size <= 0 || kv->max_blocks <= 0 ||
      kv->num_slots <= 0 || (long long)kv->max_blocks * kv->block_size >= (1ll << 30))
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
  if (!k.fits()) return SPEC_ERR_CUDA;
  const int sms = sm_count();
  const int longest = max_len > 0 ? max_len : kv->max_blocks * kv->block_size;
  pa::Args g{};
  g.kv = *kv, g.q = q, g.out = out, g.lse = lse, g.seq_len = seq_len, g.q_ld = q_ld, g.out_ld = out_ld;
  g.nq = d.n_q_heads, g.nkv = d.n_kv_heads, g.G = d.n_q_heads / d.n_kv_heads, g.hd = d.head_dim, g.window = d.window;
  g.scale2 = (d.scale > 0 ? d.scale : 1.f / sqrtf((float)d.head_dim)) * (e4m3 ? d.k_scale : 1.f) * pa::kLog2e;
  g.v_scale = e4m3 ? d.v_scale : 1.f;
  g.part = reinterpret_cast<float*>(static_cast<char*>(ws) + kWsHeader);
  g.group_counters = reinterpret_cast<int*>(static_cast<char*>(ws) + kWsHeader + pa::part_bytes(sms));
  g.counters = g.group_counters + pa::group_ints(sms);
  g.ws = ws;
  // a launch's tiles are counted in 32 bits: fewer requests of one where every table could be full of small tiles
  // (tables of over 2^23 tokens)
  const long long most_tiles = (long long)kv->max_blocks * kv->block_size / k.sub + 2;
  const int per = (int)std::min<long long>(pa::kMaxB, 0x7fffffff / most_tiles);
  for (int b0 = 0; b0 < B; b0 += per) {
    g.b0 = b0;
    g.B = std::min(B - b0, per);
    g.p = pa::plan(k, d, g.B, longest, kv->block_size, sms);
    const size_t smem = (size_t)g.p.slots * g.p.slot_bytes + k.fixed(g.B);
    if (g.p.slots < 2) return SPEC_ERR_UNSUPPORTED;
    if (g.p.swz && (!pa::run_map(&g.tmk, kv->k, d, *kv, k, g.p) || !pa::run_map(&g.tmv, kv->v, d, *kv, k, g.p)))
      return SPEC_ERR_CUDA;
    // always the same limit: another thread may be launching the same kernel with another plan
    if (cudaFuncSetAttribute(k.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)(pa::kSmemMax - 1024)) != cudaSuccess)
      return SPEC_ERR_CUDA;
    launch_pdl(k.fn, dim3(sms), dim3(k.warps * 32 + 128), smem, stream, g);
  }
  return last_launch();
}

// per-unit log setter of the instrumented build (no-op otherwise)
SPEC_TL_SETTER(paged_attn)
