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

constexpr int kResident = 1024;          // threads of an SM
// Threads of a CTA.  More of them: fewer ends of parts, where the k best are found; fewer: their warps wait less for one
// another.  When it was chosen, 2048 rows of 151936 fp32 logits, k = 20, 256 / 512: 267 / 246 us; of 32000 f16, k = 5: 62 / 72.
template <typename T> constexpr int threads_of() { return sizeof(T) == 4 ? 512 : 256; }
constexpr int kHits = 1024;              // threads of a few tiles that hold candidates
constexpr int kMaxK = 32, kMaxV = 1 << 20;
constexpr int kRows = 4096;              // rows of a launch (their counters lie at the workspace's start)
constexpr int kMaxParts = 32;            // of a row
constexpr int kCand = 1024;              // candidates that a CTA keeps
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f, kLowest = -3.402823466e38f;

struct Args {
  const void* logits;
  long long ld;
  const int32_t* tok;
  float *logprob, *entropy, *lse, *top_logprob;
  int32_t *rank, *top_ids;
  int V, k, tiles, parts, row0;
  int* counters;               // [kRows]
  float* rec;                  // [rows][parts][record_floats(k)]: m, s, w, count, then (value, id) pairs
  void* ws;
};

__host__ __device__ inline int record_floats(int k) { return 4 + 2 * ((k + 1) & ~1); }   // multiples of 16 bytes

template <typename T> constexpr int vec_elems() { return 16 / (int)sizeof(T); }
// A tile is NV 16-byte units a thread; a row may begin inside one.
template <typename T, int NV> static int tiles_of(int V) {
  const int per = threads_of<T>() * NV * vec_elems<T>();
  return (V + vec_elems<T>() - 1 + per - 1) / per;
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
SPEC_DEV float max_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
template <typename T, int NV> SPEC_DEV float max_of(const uint4* v) {
  if constexpr (sizeof(T) == 4) {
    float a = -INFINITY, b = -INFINITY;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      a = max_nan(a, __uint_as_float(v[i].x), __uint_as_float(v[i].y));
      b = max_nan(b, __uint_as_float(v[i].z), __uint_as_float(v[i].w));
    }
    return max_nan(a, b);
  } else {
    using T2 = std::conditional_t<std::is_same_v<T, __half>, __half2, __nv_bfloat162>;
    const T2* p = reinterpret_cast<const T2*>(v);
    T2 m = p[0];
#pragma unroll
    for (int i = 1; i < 4 * NV; ++i) m = __hmax2_nan(m, p[i]);
    return max_nan(to_float(m.x), to_float(m.y));
  }
}

SPEC_DEV bool before(float v, int id, float w, int jd) { return v > w || (v == w && id < jd); }

SPEC_DEV float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// two floats in an instruction: the sums' loop is bound by what it issues
struct Two {
  unsigned long long x;
  SPEC_DEV Two() {}
  SPEC_DEV Two(float a, float b) { asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a), "f"(b)); }
  SPEC_DEV void get(float& a, float& b) const { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x)); }
};
SPEC_DEV Two add(Two a, Two b) {
  Two d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d.x) : "l"(a.x), "l"(b.x));
  return d;
}
SPEC_DEV Two mul(Two a, Two b) {
  Two d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d.x) : "l"(a.x), "l"(b.x));
  return d;
}
SPEC_DEV Two fma(Two a, Two b, Two c) {
  Two d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d.x) : "l"(a.x), "l"(b.x), "l"(c.x));
  return d;
}
// all ones where a > b
SPEC_DEV int greater(float a, float b) {
  int d;
  asm("set.gt.u32.f32 %0, %1, %2;" : "=r"(d) : "f"(a), "f"(b));
  return d;
}

// How many of a unit's elements are past a threshold: `or_at`: at it as well.  16-bit ones are compared in pairs, against
// the next smaller number of their type for "at or past".
template <typename T> struct Above;
template <> struct Above<float> {
  float th;
  SPEC_DEV Above(bool or_at, float x) : th(!(x > -INFINITY) ? INFINITY : or_at ? nextafterf(x, -INFINITY) : x) {}
  SPEC_DEV int count(const uint4& v) const {
    return -(greater(__uint_as_float(v.x), th) + greater(__uint_as_float(v.y), th) + greater(__uint_as_float(v.z), th) +
             greater(__uint_as_float(v.w), th));
  }
};
template <typename T, typename T2> struct Above16 {
  uint32_t th;
  SPEC_DEV Above16(bool or_at, uint32_t bits, uint32_t inf) {
    // the next smaller number: towards zero above it (the number of smallest magnitude below zero at zero), away from it below
    const uint32_t less = (bits & 0x7fffu) == 0 ? 0x8001u : bits & 0x8000u ? bits + 1 : bits - 1;
    const uint32_t b = bits == (inf | 0x8000u) ? inf : or_at ? less : bits;
    th = b | b << 16;
  }
  SPEC_DEV int count(const uint4& v) const {
    const T2 t = *reinterpret_cast<const T2*>(&th);
    const T2* p = reinterpret_cast<const T2*>(&v);
    // ones and zeros: exact sums
    const T2 n = __hadd2(__hadd2(__hgt2(p[0], t), __hgt2(p[1], t)), __hadd2(__hgt2(p[2], t), __hgt2(p[3], t)));
    return (int)(to_float(n.x) + to_float(n.y));
  }
};
template <> struct Above<__nv_bfloat16> : Above16<__nv_bfloat16, __nv_bfloat162> {
  SPEC_DEV Above(bool or_at, float x) : Above16(or_at, __bfloat16_as_ushort(__float2bfloat16_rn(x)), 0x7f80u) {}
};
template <> struct Above<__half> : Above16<__half, __half2> {
  SPEC_DEV Above(bool or_at, float x) : Above16(or_at, __half_as_ushort(__float2half_rn(x)), 0x7c00u) {}
};

struct Smem {
  float group[32];             // maxima of 32 groups of lanes
  float red[4][16];
  float2 cand[kCand];          // (value, id)
  float2 hit[kHits];           // (the thread's largest element, tile * kThreads + thread)
  float2 top[kMaxK];           // the k best so far, in order
  float bound;
  int n, hits, last;
  float out[4];                // m, s, w, count of the row
};

// sums against another reference: exponents t are clamped, so that 0 * t is 0
SPEC_DEV void rebase(float& s, float& w, float m, float to) {
  const float d = fmaxf((m - to) * kLog2e, -1e4f), f = exp2_fast(d);
  w = f * (w + s * d);
  s *= f;
}

// What the row's record says, by the first threads.
SPEC_DEV void finish(const Args& g, int row, int tok, float xt, float m, float s, float w, int count, const float2* top) {
  const float log_s = log2f(s) * kLn2;                 // of sum exp(x - m)
  if (threadIdx.x == 0) {
    const bool some = s > 0.f, has = tok >= 0 && xt > -INFINITY && some;
    if (g.logprob) g.logprob[row] = has ? (xt - m) - log_s : -INFINITY;
    if (g.rank) g.rank[row] = has ? count : -1;
    if (g.entropy) g.entropy[row] = some ? fmaxf(log_s - w / s * kLn2, 0.f) : 0.f;
    if (g.lse) g.lse[row] = some ? m + log_s : -INFINITY;
  }
  if ((int)threadIdx.x < g.k) {
    const float2 e = top[threadIdx.x];
    const int id = __float_as_int(e.y);
    g.top_ids[(long long)row * g.k + threadIdx.x] = id;
    g.top_logprob[(long long)row * g.k + threadIdx.x] = id >= 0 ? (e.x - m) - log_s : -INFINITY;
  }
}

// The k best of sm.cand[0, n) -> sm.top, in order; all threads.
template <int kThreads> SPEC_DEV void best_of(Smem& sm, int n, int k) {
  const int tid = threadIdx.x;
  if (tid < kMaxK) sm.top[tid] = make_float2(-INFINITY, __int_as_float(-1));
  __syncthreads();
  for (int i = tid; i < n; i += kThreads) {
    const float2 e = sm.cand[i];
    const int id = __float_as_int(e.y);
    int r = 0;
#pragma unroll 8
    for (int j = 0; j < n; ++j) {
      const float2 o = sm.cand[j];
      r += before(o.x, __float_as_int(o.y), e.x, id);
    }
    if (r < k) sm.top[r] = e;
  }
  __syncthreads();
}

// A CTA streams a part of a row in tiles that it holds in registers, the next tile's loads under way.  A thread's maximum,
// sum and first moment are its own until the end; exact sums against its running maximum.
// The k best: elements at or past a bound are candidates.  In the first tile the k-th largest of 32 group maxima is one
// (k elements reach it), then the k-th largest of the threads' maxima so far.  The stream only notes which threads' maxima
// reach the bound, and after 1, 4, 16, ... tiles forgets those below a new one; at the end the elements of the threads that
// are left, about k, are read again (from L2) and ranked by counting.  Where there are too many (logits in an order, or
// mostly equal) the part is searched k times.  The last CTA of a row to finish joins the parts in their order (a counter,
// nobody waits).
// 2048 rows of 151936 fp32 logits: k = 0 194-208 us (89-95 % of the copy bandwidth), k = 20 233; bf16, k = 0 and 5: 146 and 181 (13
// instructions an element, half of the issue slots' time, 224-232 bytes a thread spilled at 64 registers; fp32: none); of 32000 f16,
// k = 5: 52, mostly the ends of parts; 64 rows of 128256 bf16, k = 5: 15 us, a chain of dependent trips.
template <typename T, int NV> __global__ void __launch_bounds__(threads_of<T>(), kResident / threads_of<T>())
    logprobs_kernel(const __grid_constant__ Args g) {
  SPEC_TL(kTLLogprobs);
  constexpr int kThreads = threads_of<T>(), kWarps = kThreads / 32, VE = vec_elems<T>(), TILE = kThreads * NV * VE;
  __shared__ __align__(16) Smem sm;
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, k = g.k;
  const int local = blockIdx.x / g.parts, part = blockIdx.x - local * g.parts, row = g.row0 + local;
  const int t0 = (int)((long long)part * g.tiles / g.parts), t1 = (int)((long long)(part + 1) * g.tiles / g.parts);
  const T* x = static_cast<const T*>(g.logits) + row * g.ld;
  const int skew = (int)((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(T));
  const uint32_t none = minus_inf<T>() | (sizeof(T) == 2 ? minus_inf<T>() << 16 : 0u);
  const int mine0 = tid * VE - skew;   // id of the thread's first element in tile 0
  auto id_of = [&](int tile, int i) { return tile * TILE + i * (kThreads * VE) + mine0; };
  auto load = [&](int tile, uint4* v) {
    const int lo = tile * TILE - skew;
    if (lo >= 0 && lo + TILE <= g.V) {
      const T* at = x + (lo + tid * VE);
#pragma unroll
      for (int i = 0; i < NV; ++i)
        asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(v[i].x), "=r"(v[i].y), "=r"(v[i].z), "=r"(v[i].w) : "l"(at + i * (kThreads * VE)));
      return;
    }
    // the row's first or last tile: units that the row does not fill by elements
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int id = id_of(tile, i);
      v[i] = make_uint4(none, none, none, none);
      if (id >= 0 && id + VE <= g.V) {
        asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(v[i].x), "=r"(v[i].y), "=r"(v[i].z), "=r"(v[i].w) : "l"(x + id));
      } else if (id + VE > 0 && id < g.V) {
        uint32_t* d = &v[i].x;
#pragma unroll
        for (int e = 0; e < VE; ++e)
          if (id + e >= 0 && id + e < g.V) {
            if constexpr (sizeof(T) == 4) d[e] = reinterpret_cast<const uint32_t*>(x)[id + e];
            else {
              const uint32_t h = reinterpret_cast<const uint16_t*>(x)[id + e];
              d[e >> 1] = e & 1 ? (d[e >> 1] & 0xffffu) | h << 16 : (d[e >> 1] & 0xffff0000u) | h;
            }
          }
      }
    }
  };
  // the largest of the thread's elements; what is not finite becomes -infinity
  auto largest = [&](uint4* v) {
    float top = max_of<T, NV>(v);
    if (!(top < INFINITY)) {
      top = -INFINITY;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < VE; ++e) {
          const float f = elem<T>(v[i], e);
          if (!(f < INFINITY)) set_masked<T>(v[i], e);
          else top = fmaxf(top, f);
        }
    }
    return top;
  };
  uint4 v[NV], next[NV];
  load(t0, v);
  int tok = g.tok ? g.tok[row] : -1;
  if (tok < -1 || tok >= g.V) {
    if (tid == 0 && part == 0) report(g.ws, SPEC_ERR_DEVICE, row, tok);
    tok = -1;
  }
  float xt = tok >= 0 ? to_float(x[tok]) : -INFINITY;
  if (!(fabsf(xt) < INFINITY)) xt = -INFINITY;         // masked
  float m = -INFINITY, s = 0.f, w = 0.f, bound = INFINITY;
  int count = 0;
  if (tid == 0) sm.n = 0, sm.hits = 0;
  if (tid < kMaxK) sm.top[tid] = make_float2(-INFINITY, __int_as_float(-1));
  if (k > 0) {
    float group = largest(v);
#pragma unroll
    for (int o = kThreads / 64; o > 0; o >>= 1) group = fmaxf(group, __shfl_xor_sync(0xffffffffu, group, o));
    if (tid % (kThreads / 32) == 0) sm.group[tid / (kThreads / 32)] = group;
    __syncthreads();
    if (warp == 0) {
      const float mine = sm.group[lane];
      int place = 0;           // among the 32
#pragma unroll 8
      for (int j = 0; j < 32; ++j) place += before(sm.group[j], j, mine, lane);
      if (place == k - 1) sm.bound = mine;
    }
    __syncthreads();
    bound = fmaxf(sm.bound, kLowest);
  }
  auto step = [&](int tile, uint4* v, uint4* next) {
    if (tile + 1 < t1) load(tile + 1, next);
    const float top = largest(v);
    if (top >= bound) {
      const int p = atomicAdd(&sm.hits, 1);
      if (p < kHits) sm.hit[p] = make_float2(top, __int_as_float(tile * kThreads + tid));
    }
    // sums against the thread's maximum, and the tokens before the given one
    if (top > m) {
      if (m > -INFINITY) rebase(s, w, m, top);
      m = top;
    }
    const float base = m == -INFINITY ? 0.f : m;
    const Two neg(-base, -base), l2e(kLog2e, kLog2e);
    Two s2(0.f, 0.f), w2(0.f, 0.f);
    // (the tile that the token is in: below)
    const int lo = tile * TILE - skew;
    const Above<T> th(lo + TILE <= tok, xt);
    int n = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      n += th.count(v[i]);
#pragma unroll
      for (int e = 0; e < VE; e += 2) {
        float a, b;
        mul(add(Two(elem<T>(v[i], e), elem<T>(v[i], e + 1)), neg), l2e).get(a, b);
        a = fmaxf(a, -1e4f), b = fmaxf(b, -1e4f);      // finite also where x is not: 0 * t = 0
        const Two p(exp2_fast(a), exp2_fast(b));
        s2 = add(s2, p);
        w2 = fma(p, Two(a, b), w2);
      }
    }
    count += n;
    if (lo < tok && tok < lo + TILE) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < VE; ++e) count += id_of(tile, i) + e < tok && elem<T>(v[i], e) == xt;
    }
    float a, b;
    s2.get(a, b);
    s += a + b;
    w2.get(a, b);
    w += a + b;
  };
  int tile = t0;
  for (long long window = 1; tile < t1; window *= 4) {
    const int end = (int)min((long long)t1, t0 + window);
#pragma unroll 1
    for (; tile + 2 <= end; tile += 2) {
      step(tile, v, next);
      step(tile + 1, next, v);
    }
    if (tile < end) {
      step(tile, v, next);
#pragma unroll
      for (int i = 0; i < NV; ++i) v[i] = next[i];
      ++tile;
    }
    if (k == 0) continue;
    __syncthreads();
    int hits = sm.hits;
    if (hits <= kHits && tile < t1) {
      // the k-th largest of the noted maxima is a bound; threads below it are forgotten
      constexpr int PER = kHits / kThreads;
      float2 mine[PER];
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int h = tid + i * kThreads;
        if (h < hits) {
          mine[i] = sm.hit[h];
          int place = 0;
#pragma unroll 4
          for (int j = 0; j < hits; ++j) place += before(sm.hit[j].x, j, mine[i].x, h);
          if (place == k - 1) sm.bound = mine[i].x;
        }
      }
      __syncthreads();
      if (hits >= k) bound = fmaxf(sm.bound, kLowest);
      if (tid == 0) sm.hits = 0;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (tid + i * kThreads < hits && mine[i].x >= bound) sm.hit[atomicAdd(&sm.hits, 1)] = mine[i];
      __syncthreads();
      continue;
    }
    if (hits <= kHits) {
      // the end: the elements of the threads that are left (read again, from L2), one a lane
      constexpr int PER = NV * VE;
      for (int i = tid; i < hits * PER; i += kThreads) {
        const int h = __float_as_int(sm.hit[i / PER].y), q = i % PER;
        const int id = (h / kThreads) * TILE + (q / VE * kThreads + h % kThreads) * VE - skew + q % VE;
        if (id >= 0 && id < g.V) {
          const float f = to_float(x[id]);
          if (f >= bound && f < INFINITY) {
            const int p = atomicAdd(&sm.n, 1);
            if (p < kCand) sm.cand[p] = make_float2(f, __int_as_float(id));
          }
        }
      }
    }
    __syncthreads();
    const int n = sm.n;
    if (hits <= kHits && n <= kCand) {
      best_of<kThreads>(sm, n, k);
      break;
    }
    // Too many: the best one after the last, k times.
    bound = INFINITY;
    if (tile < t1) {
      // (no more threads are noted; the part is searched when its sums are done)
      if (tid == 0) sm.hits = kHits + 1;
      __syncthreads();
      continue;
    }
    float pv = INFINITY;
    int pi = -1;
    for (int r = 0; r < k; ++r) {
      float bv = -INFINITY;
      int bi = 0x7fffffff;
      for (int id = max(0, t0 * TILE - skew) + tid; id < min(g.V, t1 * TILE - skew); id += kThreads) {
        const float f = to_float(x[id]);
        if (f >= kLowest && f < INFINITY && before(pv, pi, f, id) && before(f, id, bv, bi)) bv = f, bi = id;
      }
      warp_argmax(bv, bi);
      __syncthreads();
      if (lane == 0) sm.red[0][warp] = bv, sm.red[1][warp] = __int_as_float(bi);
      __syncthreads();
      bv = sm.red[0][lane % kWarps], bi = __float_as_int(sm.red[1][lane % kWarps]);
      warp_argmax(bv, bi);
      if (tid == 0 && bv > -INFINITY) sm.top[r] = make_float2(bv, __int_as_float(bi));
      pv = bv, pi = bi;
    }
    __syncthreads();
  }
  // ---- the part's sums
  float M = warp_max(m);
  if (lane == 0) sm.red[0][warp] = M;
  __syncthreads();
  M = warp_max(sm.red[0][lane % kWarps]);
  const float base = M == -INFINITY ? 0.f : M;
  if (m > -INFINITY) rebase(s, w, m, base);
  s = warp_sum(s), w = warp_sum(w);
  count = __reduce_add_sync(0xffffffffu, count);
  if (lane == 0) sm.red[1][warp] = s, sm.red[2][warp] = w, sm.red[3][warp] = __int_as_float(count);
  __syncthreads();
  if (warp == 0) {
    s = warp_sum(lane < kWarps ? sm.red[1][lane] : 0.f), w = warp_sum(lane < kWarps ? sm.red[2][lane] : 0.f);
    count = __reduce_add_sync(0xffffffffu, lane < kWarps ? __float_as_int(sm.red[3][lane]) : 0);
  }
  if (g.parts == 1) {
    finish(g, row, tok, xt, base, s, w, count, sm.top);
    return;
  }
  // ---- its record, and the row by the last part to finish
  const int rf = record_floats(k);
  float* rec = g.rec + ((long long)local * g.parts + part) * rf;
  if (tid == 0) __stcg(reinterpret_cast<float4*>(rec), make_float4(M, s, w, __int_as_float(count)));
  if (tid < k) __stcg(reinterpret_cast<float2*>(rec + 4 + 2 * tid), sm.top[tid]);
  if (warp == 0) __threadfence();
  __syncthreads();
  if (tid == 0) {
    __threadfence();
    sm.last = atomicAdd(&g.counters[local], 1) == g.parts - 1;
    if (sm.last) g.counters[local] = 0;
  }
  __syncthreads();
  if (!sm.last) return;
  __threadfence();
  rec = g.rec + (long long)local * g.parts * rf;
  const int lists = g.parts * k;                       // at most kCand
  for (int i = tid; i < lists; i += kThreads)
    sm.cand[i] = __ldcg(reinterpret_cast<const float2*>(rec + (i / k) * rf + 4 + 2 * (i % k)));
  if (warp == 0) {
    float4 r = make_float4(-INFINITY, 0.f, 0.f, 0.f);
    if (lane < g.parts) r = __ldcg(reinterpret_cast<const float4*>(rec + lane * rf));
    M = warp_max(r.x);
    const float to = M == -INFINITY ? 0.f : M;
    if (r.x > -INFINITY) rebase(r.y, r.z, r.x, to);
    s = warp_sum(r.y), w = warp_sum(r.z);
    count = __reduce_add_sync(0xffffffffu, __float_as_int(r.w));
    if (lane == 0) sm.out[0] = to, sm.out[1] = s, sm.out[2] = w, sm.out[3] = __int_as_float(count);
  }
  if (tid < kMaxK) sm.top[tid] = make_float2(-INFINITY, __int_as_float(-1));
  __syncthreads();
  // an entry's place: its own, and in every other list (all are in order) by bisection
  for (int i = tid; i < lists; i += kThreads) {
    const float2 e = sm.cand[i];
    const int id = __float_as_int(e.y), c = i / k;
    if (id < 0) continue;
    int r = i - c * k;
    for (int o = 0; o < g.parts && r < k; ++o) {
      if (o == c) continue;
      int lo = 0, hi = k;
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        const float2 f = sm.cand[o * k + mid];
        if (__float_as_int(f.y) >= 0 && before(f.x, __float_as_int(f.y), e.x, id)) lo = mid + 1;
        else hi = mid;
      }
      r += lo;
    }
    if (r < k) sm.top[r] = e;
  }
  __syncthreads();
  finish(g, row, tok, xt, sm.out[0], sm.out[1], sm.out[2], __float_as_int(sm.out[3]), sm.top);
}

template <typename T, int NV> static spec_status launch_as(Args g, int n, int sms, cudaStream_t st) {
  g.tiles = tiles_of<T, NV>(g.V);
  // Parts of a row: so many that all CTAs run at once, and with long rows six times as many, for an even end
  const int slots = kResident / threads_of<T>() * sms;
  const int parts = std::max(slots / n, std::min((6 * slots + n - 1) / n, g.tiles / 8));
  g.parts = std::max(1, std::min({parts, g.tiles, kMaxParts}));
  for (int r0 = 0; r0 < n; r0 += kRows) {
    g.row0 = r0;
    if (launch_pdl(logprobs_kernel<T, NV>, dim3((unsigned)(std::min(n - r0, kRows) * g.parts)), dim3(threads_of<T>()), 0, st, g) !=
        cudaSuccess)
      return SPEC_ERR_CUDA;
  }
  return last_launch();
}

template <typename T> static spec_status launch(const Args& g, int n, cudaStream_t st) {
  // few rows: smaller tiles, on more SMs
  const int sms = sm_count();
  return (long long)n * tiles_of<T, 4>(g.V) < sms ? launch_as<T, 1>(g, n, sms, st) : launch_as<T, 4>(g, n, sms, st);
}

}  // namespace lp
}  // namespace spec

using namespace spec;

extern "C" size_t spec_token_logprobs_workspace_bytes(int32_t n, int32_t V, int32_t k) {
  if (n <= 0 || V <= 0 || V > lp::kMaxV || k < 0 || k > lp::kMaxK) return 0;
  return kWsHeader + lp::kRows * sizeof(int) +
         align_up((size_t)std::min(n, lp::kRows) * lp::kMaxParts * lp::record_floats(k) * sizeof(float), 256);
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
