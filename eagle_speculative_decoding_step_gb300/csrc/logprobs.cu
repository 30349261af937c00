// Log-probabilities of given tokens, with their ranks, the entropy of the
// distribution and its best alternatives, in one pass over the logits.
//
// The library's verifiers and selections answer with tokens; this is what a user
// is told about them (and about a prompt's own tokens).
#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "internal.h"

namespace spec {
namespace lp {

enum : unsigned { kTLLogprobs = 30 };    // after the other units' ids

constexpr int kThreads = 512, kVecs = 4; // 16-byte vectors a thread holds
constexpr int kMaxK = 32, kMaxV = 1 << 20;
constexpr int kRows = 4096;              // rows of a launch (their counters lie at the workspace's start)
constexpr int kCand = kThreads;          // candidates of a chunk that are ranked by counting
constexpr int kMaxChunks = 129;          // of a row of kMaxV fp32 logits
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

struct Args {
  const void* logits;
  long long ld;
  const int32_t* tok;
  float *logprob, *entropy, *lse, *top_logprob;
  int32_t *rank, *top_ids;
  int V, k, chunks, row0;
  int* counters;               // [kRows]
  float* rec;                  // [rows][chunks][record_floats(k)]: m, s, w, count, then (value, id) pairs
  void* ws;
};

__host__ __device__ inline int record_floats(int k) { return 4 + 2 * ((k + 1) & ~1); }   // multiples of 16 bytes

template <typename T> constexpr int vec_elems() { return 16 / (int)sizeof(T); }
template <typename T> static int chunks_of(int V) {
  const int per = kThreads * kVecs * vec_elems<T>();
  return (V + vec_elems<T>() - 1 + per - 1) / per;     // a row may begin inside a 16-byte unit
}

template <typename T> SPEC_DEV float to_float(T x);
template <> SPEC_DEV float to_float(float x) { return x; }
template <> SPEC_DEV float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
template <> SPEC_DEV float to_float(__half x) { return __half2float(x); }

// element e of a vector
template <typename T> SPEC_DEV float elem(const uint4& v, int e) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  if constexpr (sizeof(T) == 4) return __uint_as_float(w[e]);
  else if constexpr (std::is_same_v<T, __nv_bfloat16>) return __uint_as_float(e & 1 ? w[e >> 1] & 0xffff0000u : w[e >> 1] << 16);
  else {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[e >> 1]));
    return e & 1 ? f.y : f.x;
  }
}
template <typename T> SPEC_DEV uint32_t minus_inf() {
  if constexpr (sizeof(T) == 4) return 0xff800000u;
  else if constexpr (std::is_same_v<T, __nv_bfloat16>) return 0xff80u;
  else return 0xfc00u;
}
template <typename T> SPEC_DEV void set_masked(uint4& v, int e) {
  uint32_t* w = &v.x;
  if constexpr (sizeof(T) == 4) w[e] = minus_inf<T>();
  else w[e >> 1] = e & 1 ? (w[e >> 1] & 0xffffu) | minus_inf<T>() << 16 : (w[e >> 1] & 0xffff0000u) | minus_inf<T>();
}

// largest element, NaN if there is one
SPEC_DEV float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
template <typename T> SPEC_DEV float vec_max(const uint4& v) {
  if constexpr (sizeof(T) == 4) {
    return max_nan(max_nan(__uint_as_float(v.x), __uint_as_float(v.y)), max_nan(__uint_as_float(v.z), __uint_as_float(v.w)));
  } else {
    using T2 = std::conditional_t<std::is_same_v<T, __half>, __half2, __nv_bfloat162>;
    const T2* p = reinterpret_cast<const T2*>(&v);
    const T2 m = __hmax2_nan(__hmax2_nan(p[0], p[1]), __hmax2_nan(p[2], p[3]));
    return max_nan(to_float(m.x), to_float(m.y));
  }
}

SPEC_DEV bool before(float v, int id, float w, int jd) { return v > w || (v == w && id < jd); }

SPEC_DEV float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

struct Smem {
  float group[32];             // maxima of the 32 half-warps
  float red[3][16];
  float cv[kCand];
  int ci[kCand];
  float top_v[kMaxK];
  int top_i[kMaxK];
  int n, last;
  float out[4];                // m, s, w, count of the row
  float list_v[kMaxChunks * kMaxK];
  int list_i[kMaxChunks * kMaxK];
};

// What the row's record says, by the first threads.
SPEC_DEV void finish(const Args& g, int row, int tok, float xt, float m, float s, float w, int count, const float* tv,
                     const int* ti) {
  const float log_s = log2f(s) * kLn2;                 // of sum exp(x - m)
  if (threadIdx.x == 0) {
    const bool some = s > 0.f, has = tok >= 0 && xt > -INFINITY && some;
    if (g.logprob) g.logprob[row] = has ? (xt - m) - log_s : -INFINITY;
    if (g.rank) g.rank[row] = has ? count : -1;
    if (g.entropy) g.entropy[row] = some ? fmaxf(log_s - w / s * kLn2, 0.f) : 0.f;
    if (g.lse) g.lse[row] = some ? m + log_s : -INFINITY;
  }
  if ((int)threadIdx.x < g.k) {
    const int id = ti[threadIdx.x];
    g.top_ids[(long long)row * g.k + threadIdx.x] = id;
    g.top_logprob[(long long)row * g.k + threadIdx.x] = id >= 0 ? (tv[threadIdx.x] - m) - log_s : -INFINITY;
  }
}

// A CTA holds one chunk of one row in registers: its maximum, then the sums against
// it (no rescaling), the tokens before the given one, and its k best.  The k-th
// largest of 32 group maxima is a bound that k elements reach; in logits without an
// order about k ln 32 do, and they are ranked by counting.  The last CTA of a row to
// finish joins the chunks in their order (a counter, nobody waits).
template <typename T> __global__ void __launch_bounds__(kThreads, 2) logprobs_kernel(const __grid_constant__ Args g) {
  SPEC_TL(kTLLogprobs);
  constexpr int VE = vec_elems<T>();
  extern __shared__ __align__(16) uint8_t raw[];
  Smem& sm = *reinterpret_cast<Smem*>(raw);
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int local = blockIdx.x / g.chunks, chunk = blockIdx.x - local * g.chunks, row = g.row0 + local;
  const T* x = static_cast<const T*>(g.logits) + row * g.ld;
  const int skew = (int)((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(T));
  int tok = g.tok ? g.tok[row] : -1;
  if (tok < -1 || tok >= g.V) {
    if (tid == 0 && chunk == 0) report(g.ws, SPEC_ERR_DEVICE, row, tok);
    tok = -1;
  }
  float xt = tok >= 0 ? to_float(x[tok]) : -INFINITY;
  if (!(fabsf(xt) < INFINITY)) xt = -INFINITY;         // masked
  uint4 v[kVecs];
  int id0[kVecs];
  const uint32_t none = minus_inf<T>() | (sizeof(T) == 2 ? minus_inf<T>() << 16 : 0u);
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    id0[i] = ((chunk * kVecs + i) * kThreads + tid) * VE - skew;
    v[i] = make_uint4(none, none, none, none);
    if (id0[i] >= 0 && id0[i] + VE <= g.V) {
      asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                   : "=r"(v[i].x), "=r"(v[i].y), "=r"(v[i].z), "=r"(v[i].w) : "l"(x + id0[i]));
    }
  }
  // the row's first and last unit, where it does not fill them
#pragma unroll
  for (int i = 0; i < kVecs; ++i)
    if ((id0[i] < 0 && id0[i] + VE > 0) || (id0[i] < g.V && id0[i] + VE > g.V)) {
      const uint32_t* w = reinterpret_cast<const uint32_t*>(x);
      uint32_t* d = &v[i].x;
#pragma unroll
      for (int e = 0; e < VE; ++e)
        if (id0[i] + e >= 0 && id0[i] + e < g.V) {
          if constexpr (sizeof(T) == 4) d[e] = w[id0[i] + e];
          else {
            const uint32_t h = reinterpret_cast<const uint16_t*>(x)[id0[i] + e];
            d[e >> 1] = e & 1 ? (d[e >> 1] & 0xffffu) | h << 16 : (d[e >> 1] & 0xffff0000u) | h;
          }
        }
    }
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < kVecs; ++i) top = max_nan(top, vec_max<T>(v[i]));
  if (!(top < INFINITY)) {                             // NaN or +infinity: masked
    top = -INFINITY;
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        const float f = elem<T>(v[i], e);
        if (!(f < INFINITY)) set_masked<T>(v[i], e);
        else top = fmaxf(top, f);
      }
  }
  float half = top;
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) half = fmaxf(half, __shfl_xor_sync(0xffffffffu, half, o));
  if ((lane & 15) == 0) sm.group[2 * warp + (lane >> 4)] = half;
  if (tid == 0) sm.n = 0;
  if (tid < kMaxK) sm.top_v[tid] = -INFINITY, sm.top_i[tid] = -1;
  __syncthreads();
  const float mine = sm.group[lane], m_chunk = warp_max(mine);
  // ---- sums against the chunk's maximum, and the tokens before the given one
  const float m = m_chunk == -INFINITY ? 0.f : m_chunk;
  float s = 0.f, w = 0.f;
  int count = 0;
  // x > below(xt) is x >= xt
  const float above = xt > -INFINITY ? xt : INFINITY;
  const float from = xt > -INFINITY ? nextafterf(xt, -INFINITY) : INFINITY;
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const float th = id0[i] + VE <= tok ? from : above;
#pragma unroll
    for (int e = 0; e < VE; ++e) {
      const float f = elem<T>(v[i], e);
      const float t = fmaxf((f - m) * kLog2e, -1e4f);  // finite also where f is not: 0 * t = 0
      const float p = exp2_fast(t);
      s += p;
      w = fmaf(p, t, w);
      count += f > th;
    }
    if (id0[i] < tok && tok < id0[i] + VE) {           // the unit that the token is in
#pragma unroll
      for (int e = 0; e < VE; ++e) count += id0[i] + e < tok && elem<T>(v[i], e) == xt;
    }
  }
  s = warp_sum(s), w = warp_sum(w);
  count = __reduce_add_sync(0xffffffffu, count);
  if (lane == 0) sm.red[0][warp] = s, sm.red[1][warp] = w, sm.red[2][warp] = __int_as_float(count);
  // ---- the k best
  if (g.k > 0) {
    int place = 0;             // of this lane's group maximum among the 32
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      const float o = __shfl_sync(0xffffffffu, mine, j);
      place += before(o, j, mine, lane);
    }
    const unsigned at = __ballot_sync(0xffffffffu, place == g.k - 1);
    const float bound = __shfl_sync(0xffffffffu, mine, __ffs(at) - 1);
    if (top >= bound && top > -INFINITY) {
#pragma unroll
      for (int i = 0; i < kVecs; ++i)
#pragma unroll
        for (int e = 0; e < VE; ++e) {
          const float f = elem<T>(v[i], e);
          if (f >= bound && f > -INFINITY) {
            const int p = atomicAdd(&sm.n, 1);
            if (p < kCand) sm.cv[p] = f, sm.ci[p] = id0[i] + e;
          }
        }
    }
    __syncthreads();
    const int n = sm.n;
    if (n <= kCand) {
      if (tid < n) {
        const float f = sm.cv[tid];
        const int id = sm.ci[tid];
        int r = 0;
        for (int j = 0; j < n; ++j) r += before(sm.cv[j], sm.ci[j], f, id);
        if (r < g.k) sm.top_v[r] = f, sm.top_i[r] = id;
      }
    } else {
      // logits in an order, or mostly equal: the best one after the last, k times
      float pv = INFINITY;
      int pi = -1;
      for (int r = 0; r < g.k; ++r) {
        float bv = -INFINITY;
        int bi = 0x7fffffff;
#pragma unroll
        for (int i = 0; i < kVecs; ++i)
#pragma unroll
          for (int e = 0; e < VE; ++e) {
            const float f = elem<T>(v[i], e);
            if (f > -INFINITY && before(pv, pi, f, id0[i] + e) && before(f, id0[i] + e, bv, bi)) bv = f, bi = id0[i] + e;
          }
        warp_argmax(bv, bi);
        __syncthreads();
        if (lane == 0) sm.cv[warp] = bv, sm.ci[warp] = bi;
        __syncthreads();
        bv = sm.cv[lane & 15], bi = sm.ci[lane & 15];
        warp_argmax(bv, bi);
        if (tid == 0 && bv > -INFINITY) sm.top_v[r] = bv, sm.top_i[r] = bi;
        pv = bv, pi = bi;
      }
    }
  }
  __syncthreads();
  if (warp == 0) {
    s = lane < 16 ? sm.red[0][lane] : 0.f, w = lane < 16 ? sm.red[1][lane] : 0.f;
    count = lane < 16 ? __float_as_int(sm.red[2][lane]) : 0;
    s = warp_sum(s), w = warp_sum(w);
    count = __reduce_add_sync(0xffffffffu, count);
  }
  if (g.chunks == 1) {
    finish(g, row, tok, xt, m, s, w, count, sm.top_v, sm.top_i);
    return;
  }
  // ---- this chunk's record, and the row by the last one
  const int rf = record_floats(g.k);
  float* rec = g.rec + ((long long)local * g.chunks + chunk) * rf;
  if (tid == 0) __stcg(reinterpret_cast<float4*>(rec), make_float4(m_chunk, s, w, __int_as_float(count)));
  if (tid < g.k) __stcg(reinterpret_cast<float2*>(rec + 4 + 2 * tid), make_float2(sm.top_v[tid], __int_as_float(sm.top_i[tid])));
  __threadfence();
  __syncthreads();
  if (tid == 0) {
    sm.last = atomicAdd(&g.counters[local], 1) == g.chunks - 1;
    if (sm.last) g.counters[local] = 0;
  }
  __syncthreads();
  if (!sm.last) return;
  __threadfence();
  rec = g.rec + (long long)local * g.chunks * rf;
  const int lists = g.chunks * g.k;
  for (int i = tid; i < lists; i += kThreads) {
    const float2 e = __ldcg(reinterpret_cast<const float2*>(rec + (i / g.k) * rf + 4 + 2 * (i % g.k)));
    sm.list_v[i] = e.x, sm.list_i[i] = __float_as_int(e.y);
  }
  if (warp == 0) {
    float M = -INFINITY;
    for (int c = lane; c < g.chunks; c += 32) M = fmaxf(M, __ldcg(rec + c * rf));
    M = warp_max(M);
    const float base = M == -INFINITY ? 0.f : M;
    s = 0.f, w = 0.f, count = 0;
    for (int c = lane; c < g.chunks; c += 32) {
      const float4 r = __ldcg(reinterpret_cast<const float4*>(rec + c * rf));
      const float t = fmaxf((r.x - base) * kLog2e, -1e4f), p = exp2_fast(t);
      s += r.y * p;
      w += p * (r.z + r.y * t);                        // exponents against the row's maximum
      count += __float_as_int(r.w);
    }
    s = warp_sum(s), w = warp_sum(w);
    count = __reduce_add_sync(0xffffffffu, count);
    if (lane == 0) sm.out[0] = base, sm.out[1] = s, sm.out[2] = w, sm.out[3] = __int_as_float(count);
  }
  if (tid < kMaxK) sm.top_v[tid] = -INFINITY, sm.top_i[tid] = -1;
  __syncthreads();
  // an entry's place: its own, and in every other list (all are in order) by bisection
  for (int i = tid; i < lists; i += kThreads) {
    const float f = sm.list_v[i];
    const int id = sm.list_i[i], c = i / g.k;
    if (id < 0) continue;
    int r = i - c * g.k;
    for (int o = 0; o < g.chunks && r < g.k; ++o) {
      if (o == c) continue;
      int lo = 0, hi = g.k;
      while (lo < hi) {
        const int mid = (lo + hi) >> 1, j = o * g.k + mid;
        if (sm.list_i[j] >= 0 && before(sm.list_v[j], sm.list_i[j], f, id)) lo = mid + 1;
        else hi = mid;
      }
      r += lo;
    }
    if (r < g.k) sm.top_v[r] = f, sm.top_i[r] = id;
  }
  __syncthreads();
  finish(g, row, tok, xt, sm.out[0], sm.out[1], sm.out[2], __float_as_int(sm.out[3]), sm.top_v, sm.top_i);
}

template <typename T> static spec_status launch(Args g, int n, cudaStream_t st) {
  g.chunks = chunks_of<T>(g.V);
  const size_t smem = offsetof(Smem, list_v) + (g.chunks > 1 ? sizeof(float) * kMaxChunks * kMaxK * 2 : 0);
  if (cudaFuncSetAttribute(logprobs_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Smem)) != cudaSuccess)
    return SPEC_ERR_CUDA;
  for (int r0 = 0; r0 < n; r0 += kRows) {
    g.row0 = r0;
    if (launch_pdl(logprobs_kernel<T>, dim3((unsigned)(std::min(n - r0, kRows) * g.chunks)), dim3(kThreads), smem, st, g) !=
        cudaSuccess)
      return SPEC_ERR_CUDA;
  }
  return last_launch();
}

}  // namespace lp
}  // namespace spec

using namespace spec;

extern "C" size_t spec_token_logprobs_workspace_bytes(int32_t n, int32_t V, int32_t k) {
  if (n <= 0 || V <= 0 || V > lp::kMaxV || k < 0 || k > lp::kMaxK) return 0;
  // fp32 rows have the most chunks
  return kWsHeader + lp::kRows * sizeof(int) +
         align_up((size_t)std::min(n, lp::kRows) * lp::chunks_of<float>(V) * lp::record_floats(k) * sizeof(float), 256);
}

extern "C" spec_status spec_token_logprobs(int32_t n, int32_t V, int32_t dtype, const void* logits, int64_t ld,
                                           const int32_t* tok, int32_t k, float* logprob, int32_t* rank, float* entropy,
                                           float* lse, int32_t* top_ids, float* top_logprob, void* ws, size_t ws_bytes,
                                           spec_stream_t stream) {
  if (!logits || (k > 0 && (!top_ids || !top_logprob)) || (!tok && (logprob || rank))) return SPEC_ERR_ARG;
  if (n <= 0 || V <= 0 || k < 0 || k > lp::kMaxK) return SPEC_ERR_SHAPE;
  if (dtype < SPEC_DTYPE_F32 || dtype > SPEC_DTYPE_F16) return SPEC_ERR_UNSUPPORTED;
  if (V > lp::kMaxV) return SPEC_ERR_CAPACITY;
  if (ld == 0) ld = V;
  if (ld < V) return SPEC_ERR_SHAPE;
  if (!aligned(logits, dtype == SPEC_DTYPE_F32 ? 4 : 2)) return SPEC_ERR_ALIGN;
  if (!ws || !aligned(ws, 256) || ws_bytes < spec_token_logprobs_workspace_bytes(n, V, k)) return SPEC_ERR_WORKSPACE;
  lp::Args g{};
  g.logits = logits, g.ld = ld, g.tok = tok, g.logprob = logprob, g.rank = rank, g.entropy = entropy, g.lse = lse;
  g.top_ids = top_ids, g.top_logprob = top_logprob, g.V = V, g.k = k, g.ws = ws;
  g.counters = reinterpret_cast<int*>(static_cast<char*>(ws) + kWsHeader);
  g.rec = reinterpret_cast<float*>(static_cast<char*>(ws) + kWsHeader + lp::kRows * sizeof(int));
  return dtype == SPEC_DTYPE_F32    ? lp::launch<float>(g, n, stream)
         : dtype == SPEC_DTYPE_BF16 ? lp::launch<__nv_bfloat16>(g, n, stream)
                                    : lp::launch<__half>(g, n, stream);
}

// per-unit log setter of the instrumented build (no-op otherwise)
SPEC_TL_SETTER(logprobs)
