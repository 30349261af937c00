// Attention of a chunk of new tokens per request over the paged cache: checks and
// launch, and the kernel on fp32 multiply-adds.
//
// [NEURON] "KV Cache Sharing": the paged cache the draft layer and the target
// share; this is a target's pass over several tokens of a request (a prompt's
// chunk, or a verified chain's tokens).
#include <algorithm>
#include <cmath>

#include "chunk_attn_tc.cuh"

namespace spec {
namespace ca {

// ---------------------------------------------------------------- kernel on fp32 multiply-adds
SPEC_DEV float4 load4(const float* p) { return __ldg(reinterpret_cast<const float4*>(p)); }

constexpr int kFmaThreads = 256, kFmaRows = 64, kFmaKeys = 64;
constexpr int kFmaEdges = kFmaRows / kFmaKeys + 2;     // edge tiles at either end of an item's keys

template <int HD> struct FmaSmem {
  Plan plan;
  alignas(16) float q[kFmaRows][HD + 4];
  float kv[kFmaKeys][HD + 4];                          // keys, then values
  float p[kFmaRows][kFmaKeys + 4];
  int slot[kFmaKeys];                                  // cache slot of a tile's keys, -1: none
  uint32_t poison[2 * kFmaEdges][kFmaKeys / 32];       // keys of edge tiles whose value is not finite
  int poisoned, last;
};

// Keys of a tile -> cache slots.  A block id outside the cache, or a slot past its end, is reported and left out.
SPEC_DEV int slot_for(const Args& g, const Item& it, int key) {
  if (key < it.lo || key >= it.hi) return -1;
  const long long s = slot_of(g.kv, g.b0 + it.b, key);
  if (s < 0) report(g.ws, SPEC_ERR_DEVICE, g.b0 + it.b, key);
  return (int)s;
}

// fp32 rows.  Bound by shared memory: 8 reads of 16 bytes for 64 multiply-adds of a thread (4 x 4 outputs).  8 chunks of
// 512-1024 tokens, 32 heads of 64 / 128 / 256 components: 25 / 27 / 19 TFLOP/s; 20 / 52 / 0 bytes a thread are spilled.
template <int HD> __global__ void __launch_bounds__(kFmaThreads)
    chunk_fma_kernel(const __grid_constant__ Args g) {
  SPEC_TL(kTLChunkAttn);
  constexpr int BM = kFmaRows, KT = kFmaKeys, NJ = HD / 64;
  extern __shared__ __align__(16) uint8_t raw[];
  FmaSmem<HD>& sm = *reinterpret_cast<FmaSmem<HD>*>(raw);
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  pdl_wait();
  pdl_trigger();
  make_plan<BM, KT>(g, sm.plan, tid, kFmaThreads);
  const Plan& plan = sm.plan;
  Walk<BM, KT> walk(g, plan);
  Item it;
  const float* kc = static_cast<const float*>(g.kv.k);
  const float* vc = static_cast<const float*>(g.kv.v);
  const int units = g.hd / 4;
  while (walk.next(it)) {
    __syncthreads();
    if (tid < 2 * kFmaEdges * (KT / 32)) (&sm.poison[0][0])[tid] = 0;
    if (tid == 0) sm.poisoned = 0;
    for (int i = tid; i < BM * (HD / 4); i += kFmaThreads) {
      const int r = i / (HD / 4), u = i % (HD / 4);
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < it.rows && u < units) {
        const int tok = (it.r0 + r) / g.G, head = it.h * g.G + (it.r0 + r) % g.G;
        v = load4(static_cast<const float*>(g.q) + (it.row0 + tok) * g.q_ld + (long long)head * g.hd + 4 * u);
      }
      *reinterpret_cast<float4*>(&sm.q[r][4 * u]) = v;
    }
    const Edges<KT> edges(g, it);
    float m[4], l[4], o[4][4 * NJ];
    int klo[4], khi[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      m[i] = -INFINITY, l[i] = 0.f;
      keys_of(g, it, ty + 16 * i, &klo[i], &khi[i]);
#pragma unroll
      for (int j = 0; j < 4 * NJ; ++j) o[i][j] = 0.f;
    }
    for (int k = it.k0; k < it.k1; ++k) {
      const int tile = it.tile0 + k, key0 = tile * KT;
      const bool edge = edges.has(tile);
      __syncthreads();
      if (tid < KT) sm.slot[tid] = slot_for(g, it, key0 + tid);
      __syncthreads();
      for (int i = tid; i < KT * (HD / 4); i += kFmaThreads) {
        const int r = i / (HD / 4), u = i % (HD / 4), s = sm.slot[r];
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (s >= 0 && u < units) v = load4(kc + ((long long)s * g.nkv + it.h) * g.hd + 4 * u);
        *reinterpret_cast<float4*>(&sm.kv[r][4 * u]) = v;
      }
      __syncthreads();
      float s[4][4] = {};
#pragma unroll 4
      for (int d = 0; d < HD; d += 4) {
        float4 a[4], b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = *reinterpret_cast<const float4*>(&sm.q[ty + 16 * i][d]);
#pragma unroll
        for (int j = 0; j < 4; ++j) b[j] = *reinterpret_cast<const float4*>(&sm.kv[tx + 16 * j][d]);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            s[i][j] += a[i].x * b[j].x + a[i].y * b[j].y + a[i].z * b[j].z + a[i].w * b[j].w;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float top = -INFINITY;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int key = key0 + tx + 16 * j;
          const bool seen = key >= klo[i] && key < khi[i] && sm.slot[tx + 16 * j] >= 0;
          s[i][j] = seen ? s[i][j] * g.scale2 : -INFINITY;
          top = fmaxf(top, s[i][j]);
        }
#pragma unroll
        for (int w = 8; w > 0; w >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
        // (nothing seen yet: m is -infinity and keep 0, whatever the first scores are)
        const float now = fmaxf(m[i], top), base = base_of(now), keep = exp2_fast(m[i] - base);
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float e = exp2_fast(s[i][j] - base);
          sum += e;
          sm.p[ty + 16 * i][tx + 16 * j] = e;
        }
#pragma unroll
        for (int w = 8; w > 0; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
        m[i] = now;
        l[i] = l[i] * keep + sum;
#pragma unroll
        for (int j = 0; j < 4 * NJ; ++j) o[i][j] *= keep;
      }
      __syncthreads();
      for (int i = tid; i < KT * (HD / 4); i += kFmaThreads) {
        const int r = i / (HD / 4), u = i % (HD / 4), s = sm.slot[r];
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (s >= 0 && u < units) {
          v = load4(vc + ((long long)s * g.nkv + it.h) * g.hd + 4 * u);
          // a value that is not finite must not reach the rows that do not attend to its key (0 * inf)
          if (edge && (not_finite(v.x) || not_finite(v.y) || not_finite(v.z) || not_finite(v.w))) {
            atomicOr(&sm.poison[edges.slot<kFmaEdges>(tile)][r / 32], 1u << (r % 32));
            sm.poisoned = 1;
            if (not_finite(v.x)) v.x = 0.f;
            if (not_finite(v.y)) v.y = 0.f;
            if (not_finite(v.z)) v.z = 0.f;
            if (not_finite(v.w)) v.w = 0.f;
          }
        }
        *reinterpret_cast<float4*>(&sm.kv[r][4 * u]) = v;
      }
      __syncthreads();
#pragma unroll 4
      for (int kk = 0; kk < KT; ++kk) {
        float p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = sm.p[ty + 16 * i][kk];
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          const float4 v = *reinterpret_cast<const float4*>(&sm.kv[kk][4 * tx + 64 * j]);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            o[i][4 * j] += p[i] * v.x, o[i][4 * j + 1] += p[i] * v.y;
            o[i][4 * j + 2] += p[i] * v.z, o[i][4 * j + 3] += p[i] * v.w;
          }
        }
      }
    }
    __syncthreads();
    if (sm.poisoned) {
      for (int e = 0; e < 2 * kFmaEdges; ++e)
        for (int w = 0; w < KT / 32; ++w)
          for (uint32_t bits = sm.poison[e][w]; bits; bits &= bits - 1) {
            const int key = edges.tile<kFmaEdges>(e) * KT + 32 * w + __ffs(bits) - 1;
            const long long s = slot_of(g.kv, g.b0 + it.b, key);
            for (int i = 0; i < 4; ++i) {
              if (key < klo[i] || key >= khi[i]) continue;
              for (int j = 0; j < NJ; ++j) {
                if (4 * tx + 64 * j >= g.hd) continue;
                const float4 v = load4(vc + (s * g.nkv + it.h) * g.hd + 4 * tx + 64 * j);
                const float x[4] = {v.x, v.y, v.z, v.w};
                for (int c = 0; c < 4; ++c)
                  if (not_finite(x[c])) o[i][4 * j + c] = NAN;
              }
            }
          }
    }
    if (it.k0 > 0 || it.k1 < it.tiles) {
      const Pieces pc(plan, it);
      const size_t piece = piece_floats(BM, g.hd);
      float* mine = g.part + pc.slot(blockIdx.x) * piece;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = ty + 16 * i;
#pragma unroll
        for (int j = 0; j < NJ; ++j)
          if (4 * tx + 64 * j < g.hd)
            *reinterpret_cast<float4*>(mine + ((size_t)(tx + 16 * j) * BM + r) * 4) =
                make_float4(o[i][4 * j], o[i][4 * j + 1], o[i][4 * j + 2], o[i][4 * j + 3]);
        if (tx == 0) mine[(size_t)BM * g.hd + r] = m[i], mine[(size_t)BM * (g.hd + 1) + r] = l[i];
      }
      __threadfence();
      __syncthreads();
      if (tid == 0) {
        int* counter = g.counters + (long long)it.h * plan.pairs[g.B] + plan.pairs[it.b] + it.t;
        const int before = atomicAdd(counter, 1);
        sm.last = before == pc.c1 - pc.c0;
        if (sm.last) *counter = 0;
      }
      __syncthreads();
      if (!sm.last) continue;
      __threadfence();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        m[i] = -INFINITY, l[i] = 0.f;
#pragma unroll
        for (int j = 0; j < 4 * NJ; ++j) o[i][j] = 0.f;
      }
      for (int c = pc.c0; c <= pc.c1; ++c) {
        const float* x = g.part + pc.slot(c) * piece;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = ty + 16 * i;
          const float mc = __ldcg(x + (size_t)BM * g.hd + r), lc = __ldcg(x + (size_t)BM * (g.hd + 1) + r);
          const float now = fmaxf(m[i], mc), base = base_of(now);
          const float a = exp2_fast(m[i] - base), b = exp2_fast(mc - base);    // (0 for a piece without keys of the row)
          m[i] = now;
          l[i] = l[i] * a + lc * b;
#pragma unroll
          for (int j = 0; j < NJ; ++j) {
            if (4 * tx + 64 * j >= g.hd) continue;
            const float4 v = __ldcg(reinterpret_cast<const float4*>(x + ((size_t)(tx + 16 * j) * BM + r) * 4));
            o[i][4 * j] = o[i][4 * j] * a + v.x * b, o[i][4 * j + 1] = o[i][4 * j + 1] * a + v.y * b;
            o[i][4 * j + 2] = o[i][4 * j + 2] * a + v.z * b, o[i][4 * j + 3] = o[i][4 * j + 3] * a + v.w * b;
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = ty + 16 * i;
      if (r >= it.rows) continue;
      const int tok = (it.r0 + r) / g.G, head = it.h * g.G + (it.r0 + r) % g.G;
      // l = 0: no key; a NaN stays one
      const float inv = l[i] == 0.f ? 0.f : g.v_scale / l[i];
      float* dst = static_cast<float*>(g.out) + (it.row0 + tok) * g.out_ld + (long long)head * g.hd;
#pragma unroll
      for (int j = 0; j < NJ; ++j)
        if (4 * tx + 64 * j < g.hd)
          *reinterpret_cast<float4*>(dst + 4 * tx + 64 * j) =
              make_float4(o[i][4 * j] * inv, o[i][4 * j + 1] * inv, o[i][4 * j + 2] * inv, o[i][4 * j + 3] * inv);
      if (g.lse && tx == 0)
        g.lse[(long long)(it.row0 + tok) * g.nq + head] = l[i] == 0.f ? -INFINITY : (m[i] + log2f(l[i])) * kLn2;
    }
  }
}

// ---------------------------------------------------------------- dispatch
struct Kernel {
  void (*fn)(Args);
  int rows, threads, per_sm;   // packed rows of an item; CTAs an SM
  size_t smem;
};

template <int HD> static Kernel fma_of() {
  return Kernel{chunk_fma_kernel<HD>, kFmaRows, kFmaThreads, HD > 128 ? 1 : 2, sizeof(FmaSmem<HD>)};
}
static Kernel fma_for(int hd) {
  return hd <= 64 ? fma_of<64>() : hd <= 128 ? fma_of<128>() : fma_of<256>();
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

// Pieces (two a CTA) come first, at the size of the largest kernel's, so that the counters lie in the same place for every call
// that shares the workspace and stay zero between calls.
static size_t part_bytes(int sms) { return align_up((size_t)sms * 2 * kPieceFloats * 4, 256); }

// Counters: an item has at least 64 packed rows, or ends its request; two of one with 256 rows.
static long long most_items(const spec_attn_desc& d, long long B, long long rows) {
  return d.n_kv_heads * (2 * B + (rows * (d.n_q_heads / d.n_kv_heads) + kFmaRows - 1) / kFmaRows);
}

// 128 packed rows where every request's fit them, over a 16-bit cache.  kOneQ / kTwoQ: 4 requests of 8 tokens and 200-256 keys
// 13.0 / 14.0 us; 16 of 32 tokens and 300-4000 keys 59 / 66; 64 single tokens of 4000 keys 194 / 222.  Over an 8-bit cache,
// where widening bounds both, 20.2 / 19.4 for the first of them and 393 / 310 for the last: always kTwoQ.
static int mode_for(const spec_attn_desc& d, int longest) {
  if (d.head_dim > 128) return kWide;
  return d.kv_dtype == d.dtype && (long long)longest * (d.n_q_heads / d.n_kv_heads) <= 128 ? kOneQ : kTwoQ;
}

static spec_status launch_fma(const spec_attn_desc& d, const Args& g, int sms, cudaStream_t st) {
  const Kernel k = fma_for(d.head_dim);
  if (cudaFuncSetAttribute(k.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)k.smem) != cudaSuccess) return SPEC_ERR_CUDA;
  return cuda_status(launch_pdl(k.fn, dim3(sms * k.per_sm), dim3(k.threads), k.smem, st, g));
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// ptr as [rows][heads][hd] with ld components from a row to the next, boxes of box_heads x box_rows x 64 (8 bits: x hd, as
// they lie); past a head's or the last row's end: zeros
static bool rows_map(CUtensorMap* tm, const void* ptr, int dtype, int hd, int heads, long long rows, long long ld, int box_heads,
                     int box_rows) {
  static const EncodeTiledFn enc = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    const bool ok = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) ==
                        cudaSuccess && q == cudaDriverEntryPointSuccess;
    return ok ? reinterpret_cast<EncodeTiledFn>(f) : nullptr;
  }();
  if (!enc) return false;
  cuuint64_t dims[3] = {(cuuint64_t)hd, (cuuint64_t)heads, (cuuint64_t)rows};
  const bool f8 = dtype == SPEC_DTYPE_E4M3;
  const cuuint64_t es_bytes = f8 ? 1 : 2;
  cuuint64_t strides[2] = {hd * es_bytes, ld * es_bytes};
  cuuint32_t box[3] = {f8 ? (cuuint32_t)hd : 64u, (cuuint32_t)box_heads, (cuuint32_t)box_rows};
  cuuint32_t es[3] = {1, 1, 1};
  const CUtensorMapDataType type = f8                          ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                   : dtype == SPEC_DTYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                              : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  return enc(tm, type, 3, const_cast<void*>(ptr), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
             f8 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

static spec_status launch_tc(const spec_attn_desc& d, const Args& g, int longest, int sms, cudaStream_t st) {
  const bool f8 = d.kv_dtype == SPEC_DTYPE_E4M3;
  const int mode = mode_for(d, longest);
  TcArgs a{};
  a.g = g;
  a.l = mode == kTwoQ ? layout<kTwoQ>(d.head_dim, f8) : mode == kOneQ ? layout<kOneQ>(d.head_dim, f8) : layout<kWide>(d.head_dim, f8);
  a.l.runs = g.kv.block_size % 16 == 0;
  const long long slot = (long long)d.n_kv_heads * d.head_dim;
  if (a.l.runs)
    for (int i = 0; i < 2; ++i)
      if (!rows_map(i ? &a.tmv : &a.tmk, i ? g.kv.v : g.kv.k, d.kv_dtype, d.head_dim, d.n_kv_heads, g.kv.num_slots, slot, 1, 16))
        return SPEC_ERR_CUDA;
  // (a row stride of 2^40 bytes and over is no tensor map's)
  a.l.q_boxes = 128 % g.G == 0 && g.q_ld < (1ll << 38);
  if (a.l.q_boxes && !rows_map(&a.tmq, g.q, d.dtype, d.head_dim, d.n_q_heads, g.n_rows, g.q_ld, g.G, 128 / g.G))
    return SPEC_ERR_CUDA;
  const TcFn fn = d.dtype == SPEC_DTYPE_BF16 ? tc_kernel_bf16(f8, mode) : tc_kernel_f16(f8, mode);
  if (!fn || cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kTcSmem) != cudaSuccess) return SPEC_ERR_CUDA;
  return cuda_status(launch_pdl(fn, dim3(sms), dim3(kTcThreads), a.l.smem, st, a));
}

}  // namespace ca
}  // namespace spec

using namespace spec;

extern "C" size_t spec_chunk_attention_workspace_bytes(const spec_attn_desc* desc, int32_t max_B, int32_t max_rows) {
  if (!ca::check(desc) || !ca::check_types(*desc) || max_B <= 0 || max_rows <= 0 ||
      (long long)max_rows * desc->n_q_heads >= (1ll << 31))
    return 0;
  return kWsHeader + ca::part_bytes(sm_count()) + align_up((size_t)ca::most_items(*desc, max_B, max_rows) * 4, 256);
}

extern "C" spec_status spec_chunk_attention(const spec_attn_desc* desc, const void* q, int64_t q_ld, const spec_kv* kv,
                                            const int32_t* cu_rows, const int32_t* seq_len, int32_t B, int32_t n_rows,
                                            int32_t max_chunk, int32_t max_len, void* out, int64_t out_ld, float* lse,
                                            void* ws, size_t ws_bytes, spec_stream_t stream) {
  if (!desc || !q || !kv || !kv->k || !kv->v || !kv->block_table || !cu_rows || !seq_len || !out) return SPEC_ERR_ARG;
  const spec_attn_desc& d = *desc;
  if (!ca::check(desc) || B <= 0 || n_rows <= 0 || max_chunk < 0 || max_len < 0 || kv->block_size <= 0 ||
      kv->max_blocks <= 0 || kv->num_slots <= 0 || (long long)kv->max_blocks * kv->block_size >= (1ll << 30))
    return SPEC_ERR_SHAPE;
  if (!ca::check_types(d)) return SPEC_ERR_UNSUPPORTED;
  const bool e4m3 = d.kv_dtype == SPEC_DTYPE_E4M3;
  if (!(d.scale >= 0) || std::isinf(d.scale) ||
      (e4m3 && !(d.k_scale > 0 && d.v_scale > 0 && std::isfinite(d.k_scale) && std::isfinite(d.v_scale))))
    return SPEC_ERR_ARG;
  const long long width = (long long)d.n_q_heads * d.head_dim;
  if (q_ld == 0) q_ld = width;
  if (out_ld == 0) out_ld = width;
  if (q_ld < width || out_ld < width) return SPEC_ERR_SHAPE;
  if ((long long)n_rows * d.n_q_heads >= (1ll << 31) || width >= (1ll << 30)) return SPEC_ERR_CAPACITY;
  const int es = d.dtype == SPEC_DTYPE_F32 ? 4 : 2;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(kv->k, 16) || !aligned(kv->v, 16) || q_ld * es % 16 ||
      out_ld * es % 16)
    return SPEC_ERR_ALIGN;
  if (!ws || !aligned(ws, 256) || ws_bytes < spec_chunk_attention_workspace_bytes(desc, B, n_rows)) return SPEC_ERR_WORKSPACE;
  const int sms = sm_count();
  const int longest = max_chunk > 0 ? std::min(max_chunk, n_rows) : n_rows;
  ca::Args g{};
  g.kv = *kv, g.q = q, g.out = out, g.lse = lse, g.cu = cu_rows, g.seq_len = seq_len, g.q_ld = q_ld, g.out_ld = out_ld;
  g.n_rows = n_rows, g.nq = d.n_q_heads, g.nkv = d.n_kv_heads, g.G = d.n_q_heads / d.n_kv_heads, g.hd = d.head_dim;
  g.window = d.window < kv->max_blocks * kv->block_size ? d.window : 0;
  g.scale2 = (d.scale > 0 ? d.scale : 1.f / sqrtf((float)d.head_dim)) * (e4m3 ? d.k_scale : 1.f) * ca::kLog2e;
  g.v_scale = e4m3 ? d.v_scale : 1.f;
  g.part = reinterpret_cast<float*>(static_cast<char*>(ws) + kWsHeader);
  g.counters = reinterpret_cast<int*>(static_cast<char*>(ws) + kWsHeader + ca::part_bytes(sms));
  g.ws = ws;
  for (int b0 = 0; b0 < B; b0 += ca::kMaxB) {
    g.b0 = b0;
    g.B = std::min(B - b0, ca::kMaxB);
    const spec_status r = d.dtype == SPEC_DTYPE_F32 ? ca::launch_fma(d, g, sms, stream) : ca::launch_tc(d, g, longest, sms, stream);
    if (r != SPEC_OK) return r;
  }
  return last_launch();
}

// per-unit log setter of the instrumented build (no-op otherwise)
SPEC_TL_SETTER(chunk_attn)
