// Attention of one new token per request over the paged cache: the kernel.  The
// translation units paged_attn_<type>.cu instantiate it, paged_attn.cu plans and
// launches.
#pragma once
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "tc_core.cuh"

namespace spec {
namespace pa {

enum : unsigned { kTLPagedAttn = 26 };   // after common.cuh's ids

constexpr int kMaxB = 2048;              // requests of one launch (their tile counts' prefix sums sit in shared memory)
constexpr int kMaxSlots = 16;            // ring slots
constexpr int kMaskWords = 8;            // validity words of a tile of at most 256 keys
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// How a call's work is cut (host, paged_attn.cu).
struct Plan {
  int nh;          // kv heads of a tile
  int qt;          // query tiles of a kv head (warps over the same keys)
  int kg;          // key groups: nh * qt * kg consumer warps
  int kt;          // keys of a tile
  int hgq;         // head groups x query splits of a request
  int qs;          // query splits (K/V is read once per split; 1 unless nq / nkv is large)
  int qtiles;      // query tiles of a kv head in all
  int row;         // bytes of one key's nh heads
  int stride;      // of rows in shared memory: an odd multiple of 16, so 8 rows hit 8 bank groups
  int slots;       // ring slots of kt * stride bytes
};

struct Args {
  spec_kv kv;
  Plan p;
  const void* q;
  void* out;
  float* lse;
  const int32_t* seq_len;
  long long q_ld, out_ld;
  int B, b0, nq, nkv, G, hd, window;
  float scale2;    // softmax scale (and k_scale) times log2(e)
  float v_scale;
  int* counters;   // [B, hgq]
  float* part;     // [grid, 2, warps, entry]
  void* ws;
};

// A consumer warp's running state for one (kv head, query tile): unnormalised
// outputs o, running maxima m (log2 units) and sums l, in the layout of its math.
// Register r of o belongs to statistics index st(r).
template <int NR_, int NM_> struct State {
  static constexpr int NR = NR_, NM = NM_;
  float o[NR], m[NM], l[NM];
};

SPEC_DEV float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// reference value of an exponent: finite also where nothing has been seen
SPEC_DEV float base_of(float m) { return m == -INFINITY ? 0.f : m; }

SPEC_DEV void bulk_row(uint32_t dst, const void* src, uint32_t bytes, uint32_t mbar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(mbar), "l"(policy)
      : "memory");
}

// ---------------------------------------------------------------- 16-bit products
SPEC_DEV void ldsm4(uint32_t a, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
SPEC_DEV void ldsm4t(uint32_t a, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
SPEC_DEV uint32_t movm(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
template <typename T> SPEC_DEV void mma(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  if constexpr (std::is_same_v<T, __half>)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <typename T> SPEC_DEV uint32_t pack(float lo, float hi) {
  if constexpr (std::is_same_v<T, __half>) {
    __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&h);
  } else {
    __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&h);
  }
}
template <typename T> SPEC_DEV float2 unpack(uint32_t x) {
  if constexpr (std::is_same_v<T, __half>) return __half22float2(*reinterpret_cast<__half2*>(&x));
  else return __bfloat1622float2(*reinterpret_cast<__nv_bfloat162*>(&x));
}
// two 8-bit values (low 16 bits of x) as two T; exact (T has every 8-bit value)
template <typename T> SPEC_DEV uint32_t widen(uint32_t x) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(x & 0xffffu), __NV_E4M3);
  const __half2 f = h;
  if constexpr (std::is_same_v<T, __half>) return *reinterpret_cast<const uint32_t*>(&f);
  const float2 y = __half22float2(f);
  return pack<T>(y.x, y.y);
}

// Scores and outputs of 16 keys x one kv head x 8 NT queries on warp-level matrix
// instructions, keys and head-dim components in the rows: S^T = K Q^T and
// O^T += V^T P^T.  The instruction's 8-wide side is the queries, of which a decode
// step has few; K rows and (transposed) V rows come out of shared memory as they
// lie.  tcgen05 would want 128 rows of one operand per 16 keys' work.
template <typename T, bool F8, int HD, int NT> struct MmaMath {
  using In = T;
  static constexpr int kSub = 16, kQ = 8 * NT, kEs = F8 ? 1 : 2, kWarps = HD > 128 ? 4 : 8;
  using S = State<HD / 16 * NT * 4, 2 * NT>;
  SPEC_DEV static int st(int r) { return ((r >> 2) % NT) * 2 + (r & 1); }
  // query and head-dim component of register r
  SPEC_DEV static int query(int r, int lane) { return ((r >> 2) % NT) * 8 + 2 * (lane & 3) + (r & 1); }
  SPEC_DEV static int comp(int r, int lane) {
    const int mt = (r >> 2) / NT, hi = (r >> 1) & 1;
    return mt * 16 + (F8 ? 2 * (lane >> 2) + hi : (lane >> 2) + 8 * hi);
  }
  SPEC_DEV static int stat_query(int i, int lane) { return (i >> 1) * 8 + 2 * (lane & 3) + (i & 1); }
  SPEC_DEV static bool stat_owner(int lane) { return lane < 4; }

  uint32_t qf[HD / 16][NT][2];
  uint32_t pf[NT][4];      // P^T operands: high parts of keys 0-7 and 8-15, low parts of both
  uint32_t vm;             // valid keys (16 bits)

  // queries of the tile: q points at the kv head's first query, n of them from q0 on exist
  SPEC_DEV void load_q(const Args& g, const T* q, int q0, int n, int lane, float*) {
    const int gq = lane >> 2, t = lane & 3;
#pragma unroll
    for (int ks = 0; ks < HD / 16; ++ks)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int i = nt * 8 + gq;
        qf[ks][nt][0] = qf[ks][nt][1] = 0;
        if (i < n && ks * 16 < g.hd) {
          const T* p = q + (long long)(q0 + i) * g.hd + ks * 16;
          if constexpr (F8) {       // component order of an 8-bit K row's words
            const uint2 x = *reinterpret_cast<const uint2*>(p + 4 * t);
            qf[ks][nt][0] = x.x;
            qf[ks][nt][1] = x.y;
          } else {
            qf[ks][nt][0] = *reinterpret_cast<const uint32_t*>(p + 2 * t);
            qf[ks][nt][1] = *reinterpret_cast<const uint32_t*>(p + 2 * t + 8);
          }
        }
      }
  }

  // scores of the 16 keys at shared address k (this warp's head), running statistics, weights
  SPEC_DEV void scores(const Args& g, uint32_t k, uint32_t mask, int lane, S& s, float*) {
    vm = mask & 0xffffu;
    if (vm == 0) return;
    float c[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) c[nt][0] = c[nt][1] = c[nt][2] = c[nt][3] = 0.f;
    const uint32_t a0 = k + (uint32_t)((lane & 15) * g.p.stride) + (lane >> 4) * 16;
    if constexpr (F8) {
#pragma unroll
      for (int kp = 0; kp < HD / 32; ++kp)
        if (kp * 32 < g.hd) {
          uint32_t r[4], a[4];
          ldsm4(a0 + kp * 32, r);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            if (kp * 32 + j * 16 >= g.hd) break;
            a[0] = widen<T>(r[2 * j]), a[1] = widen<T>(r[2 * j + 1]);
            a[2] = widen<T>(r[2 * j] >> 16), a[3] = widen<T>(r[2 * j + 1] >> 16);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma<T>(c[nt], a, qf[kp * 2 + j][nt][0], qf[kp * 2 + j][nt][1]);
          }
        }
    } else {
#pragma unroll
      for (int ks = 0; ks < HD / 16; ++ks)
        if (ks * 16 < g.hd) {
          uint32_t a[4];
          ldsm4(a0 + ks * 32, a);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma<T>(c[nt], a, qf[ks][nt][0], qf[ks][nt][1]);
        }
    }
    const bool k0 = vm >> (lane >> 2) & 1, k1 = vm >> ((lane >> 2) + 8) & 1;
    bool grew = false;
    float mn[2 * NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        c[nt][j] = k0 ? c[nt][j] * g.scale2 : -INFINITY;
        c[nt][2 + j] = k1 ? c[nt][2 + j] * g.scale2 : -INFINITY;
        float x = fmaxf(c[nt][j], c[nt][2 + j]);
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
        mn[nt * 2 + j] = fmaxf(s.m[nt * 2 + j], x);
        grew |= x > s.m[nt * 2 + j];
      }
    if (__any_sync(0xffffffffu, grew)) {
      float al[2 * NT];
#pragma unroll
      for (int i = 0; i < 2 * NT; ++i) {
        al[i] = exp2_fast(s.m[i] - base_of(mn[i]));
        s.m[i] = mn[i];
        s.l[i] *= al[i];
      }
#pragma unroll
      for (int r = 0; r < S::NR; ++r) s.o[r] *= al[st(r)];
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float b = base_of(s.m[nt * 2 + j]);
        c[nt][j] = exp2_fast(c[nt][j] - b);
        c[nt][2 + j] = exp2_fast(c[nt][2 + j] - b);
        s.l[nt * 2 + j] += c[nt][j] + c[nt][2 + j];
      }
      // a weight enters the second product as two 16-bit parts: one alone (2^-9 of it in bf16)
      // would cost as much as the output's own rounding
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t hi = pack<T>(c[nt][2 * h], c[nt][2 * h + 1]);
        const float2 f = unpack<T>(hi);
        pf[nt][h] = movm(hi);
        pf[nt][2 + h] = movm(pack<T>(c[nt][2 * h] - f.x, c[nt][2 * h + 1] - f.y));
      }
    }
  }

  SPEC_DEV void values(const Args& g, uint32_t v, int lane, S& s) {
    if (vm == 0) return;
    const int t2 = 2 * (lane & 3);
    // rows of keys that are not valid may hold anything: their bits are cleared
    const bool some = vm != 0xffffu;
    const uint32_t z0 = (vm >> t2 & 1 ? 0xffffu : 0) | (vm >> (t2 + 1) & 1 ? 0xffff0000u : 0);
    const uint32_t z1 = (vm >> (t2 + 8) & 1 ? 0xffffu : 0) | (vm >> (t2 + 9) & 1 ? 0xffff0000u : 0);
    auto step = [&](int mt, uint32_t* a) {
      if (some) a[0] &= z0, a[1] &= z0, a[2] &= z1, a[3] &= z1;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float* o = &s.o[(mt * NT + nt) * 4];
        mma<T>(o, a, pf[nt][0], pf[nt][1]);
        mma<T>(o, a, pf[nt][2], pf[nt][3]);
      }
    };
    if constexpr (F8) {
      const uint32_t a0 = v + (uint32_t)((lane & 15) * g.p.stride) + (lane >> 4) * 16;
#pragma unroll
      for (int cp = 0; cp < HD / 32; ++cp)
        if (cp * 32 < g.hd) {
          uint32_t r[4], a[4];
          ldsm4t(a0 + cp * 32, r);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            if (cp * 32 + j * 16 >= g.hd) break;
            // bytes (key, component): 00 01 10 11 -> component 0 of both keys, component 1 of both
            const uint32_t x = __byte_perm(r[2 * j], 0, 0x3120), y = __byte_perm(r[2 * j + 1], 0, 0x3120);
            a[0] = widen<T>(x), a[1] = widen<T>(x >> 16), a[2] = widen<T>(y), a[3] = widen<T>(y >> 16);
            step(cp * 2 + j, a);
          }
        }
    } else {
      const uint32_t a0 = v + (uint32_t)(((lane & 7) + (lane >> 4) * 8) * g.p.stride) + ((lane >> 3) & 1) * 16;
#pragma unroll
      for (int mt = 0; mt < HD / 16; ++mt)
        if (mt * 16 < g.hd) {
          uint32_t a[4];
          ldsm4t(a0 + mt * 32, a);
          step(mt, a);
        }
    }
  }
  // sums over the lanes that hold other keys of the same query
  SPEC_DEV void finish(S& s) {
#pragma unroll
    for (int i = 0; i < S::NM; ++i) {
      s.l[i] += __shfl_xor_sync(0xffffffffu, s.l[i], 4);
      s.l[i] += __shfl_xor_sync(0xffffffffu, s.l[i], 8);
      s.l[i] += __shfl_xor_sync(0xffffffffu, s.l[i], 16);
    }
  }
};

// The same for 32-bit caches on fp32 multiply-adds: 8 keys x 8 queries a step.
// Scores: lane = (key, quarter of the components); outputs: a lane holds
// components lane + 32 e (e < HD / 32) of every query.
template <int HD> struct F32Math {
  using In = float;
  static constexpr int kSub = 8, kQ = 8, kEs = 4, kWarps = HD > 128 ? 4 : 8;
  using S = State<8 * (HD / 32), 8>;
  SPEC_DEV static int st(int r) { return r / (HD / 32); }
  SPEC_DEV static int query(int r, int) { return r / (HD / 32); }
  SPEC_DEV static int comp(int r, int lane) { return lane + 32 * (r % (HD / 32)); }
  SPEC_DEV static int stat_query(int i, int) { return i; }
  SPEC_DEV static bool stat_owner(int lane) { return lane == 0; }
  // a warp's shared scratch: its queries, then the 8 x 8 weights of a step
  static constexpr int kScratch = 8 * HD + 64;

  uint32_t vm;
  SPEC_DEV void load_q(const Args& g, const float* q, int q0, int n, int lane, float* w) {
    __syncwarp();
    for (int i = 0; i < 8; ++i)
      for (int c = lane; c < g.hd; c += 32) w[i * g.hd + c] = i < n ? q[(long long)(q0 + i) * g.hd + c] : 0.f;
    __syncwarp();
  }
  SPEC_DEV void scores(const Args& g, uint32_t k, uint32_t mask, int lane, S& s, float* w) {
    vm = mask & 0xffu;
    if (vm == 0) return;
    const int key = lane & 7, part = lane >> 3;
    float c[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    const uint32_t row = k + (uint32_t)(key * g.p.stride);
    for (int ch = part; ch < g.hd / 4; ch += 4) {
      float4 x;
      asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w) : "r"(row + ch * 16) : "memory");
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float4 y = *reinterpret_cast<const float4*>(w + i * g.hd + ch * 4);
        c[i] = fmaf(x.x, y.x, fmaf(x.y, y.y, fmaf(x.z, y.z, fmaf(x.w, y.w, c[i]))));
      }
    }
    const bool ok = vm >> key & 1;
    bool grew = false;
    float mn[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      c[i] += __shfl_xor_sync(0xffffffffu, c[i], 8);
      c[i] += __shfl_xor_sync(0xffffffffu, c[i], 16);
      c[i] = ok ? c[i] * g.scale2 : -INFINITY;
      float x = c[i];
      x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
      x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
      x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
      mn[i] = fmaxf(s.m[i], x);
      grew |= x > s.m[i];
    }
    if (grew) {                               // the same in every lane
      float al[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        al[i] = exp2_fast(s.m[i] - base_of(mn[i]));
        s.m[i] = mn[i];
        s.l[i] *= al[i];
      }
#pragma unroll
      for (int r = 0; r < S::NR; ++r) s.o[r] *= al[st(r)];
    }
    float* pw = w + 8 * g.hd;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      c[i] = exp2_fast(c[i] - base_of(s.m[i]));
      if (part == 0) s.l[i] += c[i];          // lanes 0-7 sum their own keys; finish() adds them up
      if (part == (i >> 1)) pw[i * 8 + key] = c[i];
    }
    __syncwarp();
  }
  SPEC_DEV void values(const Args& g, uint32_t v, int lane, S& s, const float* w) {
    if (vm == 0) return;
    const float* pw = w + 8 * g.hd;
#pragma unroll
    for (int key = 0; key < 8; ++key) {
      if (!(vm >> key & 1)) continue;         // its row may hold anything
      const uint32_t row = v + (uint32_t)(key * g.p.stride);
#pragma unroll
      for (int e = 0; e < HD / 32; ++e)
        if (lane + 32 * e < g.hd) {
          float x;
          asm volatile("ld.shared.f32 %0, [%1];" : "=f"(x) : "r"(row + (lane + 32 * e) * 4) : "memory");
#pragma unroll
          for (int i = 0; i < 8; ++i) s.o[i * (HD / 32) + e] = fmaf(pw[i * 8 + key], x, s.o[i * (HD / 32) + e]);
        }
    }
  }
  SPEC_DEV void finish(S& s) {
#pragma unroll
    for (int i = 0; i < S::NM; ++i) s.l[i] = warp_sum(s.l[i]);
  }
};

template <typename M> constexpr int math_scratch() {
  if constexpr (std::is_same_v<typename M::In, float>) return M::kScratch;
  else return 0;
}
// floats of one warp's partial result in the workspace, and of the exchange area in
// shared memory (half of the warps write at a time)
template <typename M> constexpr int entry_floats() { return (M::S::NR + 2 * M::S::NM) * 32; }
template <typename M> constexpr int exchange_floats() { return M::kWarps / 2 * entry_floats<M>(); }
// shared memory besides the ring
template <typename M> constexpr size_t fixed_smem(int B) {
  return 1024 + (size_t)kMaxSlots * kMaskWords * 4 + (size_t)(B + 4) / 4 * 16 +
         4 * (size_t)(exchange_floats<M>() + M::kWarps * math_scratch<M>());
}

template <typename S> SPEC_DEV void reset(S& s) {
#pragma unroll
  for (int r = 0; r < S::NR; ++r) s.o[r] = 0.f;
#pragma unroll
  for (int i = 0; i < S::NM; ++i) s.m[i] = -INFINITY, s.l[i] = 0.f;
}
// s and another state of the same queries, m and l of which are at x[NR ..) of the lane's column
template <typename M, typename Get> SPEC_DEV void join(typename M::S& s, Get get) {
  using S = typename M::S;
  float a[S::NM], b[S::NM];
#pragma unroll
  for (int i = 0; i < S::NM; ++i) {
    const float m = get(S::NR + i), mn = fmaxf(s.m[i], m), base = base_of(mn);
    a[i] = exp2_fast(s.m[i] - base);
    b[i] = exp2_fast(m - base);
    s.m[i] = mn;
    s.l[i] = s.l[i] * a[i] + get(S::NR + S::NM + i) * b[i];
  }
#pragma unroll
  for (int r = 0; r < S::NR; ++r) s.o[r] = s.o[r] * a[M::st(r)] + get(r) * b[M::st(r)];
}

// The linear order of a launch's tiles: (request, head group, tile); CTA c owns
// tiles [c T / C, (c + 1) T / C).  Every CTA finds its range by bisection of the
// prefix sums of the requests' tile counts.
struct Walk {
  const int* pre;       // [B + 1] exclusive prefix sums of tile counts
  int hgq;
  long long idx, end;
  int b;
  // current piece: tiles [t0, t1) of head group hg of request b, which has nt
  int hg, t0, t1, nt;
  SPEC_DEV Walk(const int* pre_, int B, int hgq_, long long beg, long long end_) : pre(pre_), hgq(hgq_), idx(beg), end(end_) {
    int lo = 0, hi = B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if ((long long)pre[mid] * hgq <= beg) lo = mid;
      else hi = mid;
    }
    b = lo;
  }
  SPEC_DEV bool next() {
    if (idx >= end) return false;
    while ((long long)pre[b + 1] * hgq <= idx) ++b;
    nt = pre[b + 1] - pre[b];
    const long long off = idx - (long long)pre[b] * hgq;
    hg = (int)(off / nt);
    t0 = (int)(off - (long long)hg * nt);
    const long long n = end - idx < nt - t0 ? end - idx : nt - t0;
    t1 = t0 + (int)n;
    idx += n;
    return true;
  }
};

// One CTA per SM walks its share of the tiles.  A producer warp copies the rows of
// a tile's keys (kt keys x nh heads, whole rows of the cache: one bulk copy a key,
// whatever the block size) into a ring of shared-memory slots, K and V tiles in
// turn; each consumer warp takes 16 (8) keys of one head and one query tile of
// every tile.  Pieces of a (request, head group) that several CTAs share are left
// as partial results; the last CTA of such a group to finish joins them in CTA
// order, so results do not depend on timing.
template <typename M>
__global__ void __launch_bounds__(M::kWarps * 32 + 32, 1) paged_attention_kernel(const __grid_constant__ Args g) {
  SPEC_TL(kTLPagedAttn);
  using T = typename M::In;
  using S = typename M::S;
  constexpr int NW = M::kWarps;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const Plan& p = g.p;
  uint8_t* ring = smem_raw;
  uint64_t* bars = reinterpret_cast<uint64_t*>(ring + (size_t)p.slots * p.kt * p.stride);   // full[kMaxSlots], empty[kMaxSlots]
  volatile int* flags = reinterpret_cast<volatile int*>(bars + 2 * kMaxSlots);              // abort, last
  uint32_t* masks = reinterpret_cast<uint32_t*>(reinterpret_cast<uint8_t*>(bars) + 1024);
  float* exch = reinterpret_cast<float*>(masks + kMaxSlots * kMaskWords);
  float* mscr = exch + exchange_floats<M>();
  int* pre = reinterpret_cast<int*>(mscr + NW * math_scratch<M>());
  __shared__ int wsum[NW + 1];
  const uint32_t full0 = tc::su32(bars), empty0 = full0 + 8 * kMaxSlots;
  if (tid == 0) {
    for (int i = 0; i < p.slots; ++i) {
      tc::mbar_init(full0 + 8 * i, 1);
      tc::mbar_init(empty0 + 8 * i, NW);
    }
    flags[0] = 0;
    pre[0] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  pdl_wait();
  pdl_trigger();
  // tile counts of the requests (one empty tile where there is nothing to attend to, so that
  // every request is somebody's) and their prefix sums
  const long long most_l = (long long)g.kv.max_blocks * g.kv.block_size;
  const int most = (int)most_l;
  auto range = [&](int b, int& lo, int& len) {
    len = g.seq_len[g.b0 + b];
    len = len < 0 ? 0 : (len > most ? most : len);
    lo = g.window > 0 && len > g.window ? len - g.window : 0;
  };
  int carry = 0;
  for (int base = 0; base < g.B; base += NW * 32 + 32) {
    const int b = base + tid;
    int x = 0;
    if (b < g.B) {
      int lo, len;
      range(b, lo, len);
      x = max(1, (len - lo + p.kt - 1) / p.kt);
      if (blockIdx.x == 0) {
        const int n = g.seq_len[g.b0 + b];
        if (n < 0 || n > most) report(g.ws, SPEC_ERR_DEVICE, g.b0 + b, n);
      }
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) wsum[warp] = x;
    __syncthreads();
    int before = carry;
    for (int w = 0; w < NW + 1; ++w) {
      if (w < warp) before += wsum[w];
      carry += wsum[w];
    }
    if (b < g.B) pre[b + 1] = before + x;
    __syncthreads();
  }
  const long long total = (long long)pre[g.B] * p.hgq;
  const long long C = total < (long long)gridDim.x ? total : (long long)gridDim.x;
  const int cta = blockIdx.x;
  if (cta >= C) return;
  Walk w(pre, g.B, p.hgq, cta * total / C, (cta + 1) * total / C);
  const uint32_t ring0 = tc::su32(ring), slot_bytes = (uint32_t)(p.kt * p.stride);

  if (warp == NW) {
    // ------------------------------------------------------------ producer
    const uint64_t policy = tc::policy_evict_first();      // each K/V row is read once
    const long long row_all = (long long)g.nkv * g.hd * M::kEs;
    const char* kp = static_cast<const char*>(g.kv.k);
    const char* vp = static_cast<const char*>(g.kv.v);
    const int bs = g.kv.block_size, shift = (bs & (bs - 1)) == 0 ? __ffs(bs) - 1 : -1;
    int slot = 0, phase = 0, issued = 0;
    bool ok = true;
    constexpr int kPer = kMaskWords;                       // keys of a tile a lane handles
    while (ok && w.next()) {
      int lo, len;
      range(w.b, lo, len);
      const int32_t* table = g.kv.block_table + (long long)(g.b0 + w.b) * g.kv.max_blocks;
      const long long col = (long long)(w.hg / p.qs) * p.row;
      for (int t = w.t0; ok && t < w.t1; ++t) {
        const int key0 = lo + t * p.kt;
        // this tile's cache slots (-1: no key), before waiting for room
        int sl[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          sl[i] = -1;
          const int j = i * 32 + lane, key = key0 + j;
          if (j < p.kt && key < len) {
            const int blk = shift >= 0 ? key >> shift : key / bs;
            const int id = __ldcg(table + blk);
            const long long s = (long long)id * bs + (key - blk * bs);
            if (id >= 0 && s < g.kv.num_slots) sl[i] = (int)s;
            else report(g.ws, SPEC_ERR_DEVICE, g.b0 + w.b, key);
          }
        }
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          ok = tc::mbar_wait(empty0 + 8 * slot, phase ^ 1, const_cast<volatile int*>(flags));
          if (!__all_sync(0xffffffffu, ok)) {
            ok = false;
            break;
          }
          int n = 0;
#pragma unroll
          for (int i = 0; i < kPer; ++i)
            if (i * 32 < p.kt) {
              const uint32_t word = __ballot_sync(0xffffffffu, sl[i] >= 0);
              if (lane == 0) masks[slot * kMaskWords + i] = word;
              n += __popc(word);
            }
          if (lane == 0) tc::mbar_expect_tx(full0 + 8 * slot, (uint32_t)(n * p.row));
          __syncwarp();
          const char* src = (v ? vp : kp) + col;
#pragma unroll
          for (int i = 0; i < kPer; ++i)
            if (sl[i] >= 0)
              bulk_row(ring0 + slot * slot_bytes + (i * 32 + lane) * p.stride, src + sl[i] * row_all, p.row,
                       full0 + 8 * slot, policy);
          ++issued;
          if (++slot == p.slots) slot = 0, phase ^= 1;
        }
      }
    }
    if (!ok) {
      // a wait ran out: let the copies in flight land before leaving
      if (lane == 0) report(g.ws, SPEC_ERR_TIMEOUT);
      int sl = slot, ph = phase;
      for (int i = 0; i < (issued < p.slots ? issued : p.slots); ++i) {
        if (--sl < 0) sl = p.slots - 1, ph ^= 1;
        tc::mbar_wait(full0 + 8 * sl, ph, const_cast<volatile int*>(flags), false);
      }
    }
    return;
  }

  // -------------------------------------------------------------- consumers
  const int h = warp % p.nh, qi = warp / p.nh % p.qt, kgrp = warp / (p.nh * p.qt);
  const uint32_t off = (uint32_t)(kgrp * M::kSub * p.stride + h * g.hd * M::kEs);
  float* wscr = mscr + warp * math_scratch<M>();
  int slot = 0, phase = 0;
  M math;
  S s;
  auto sync = [] { asm volatile("bar.sync 1, %0;" ::"n"(NW * 32) : "memory"); };
  auto advance = [&] {
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(empty0 + 8 * slot);
    if (++slot == p.slots) slot = 0, phase ^= 1;
  };
  // the key groups' states into group 0's
  auto merge_groups = [&] {
    for (int half = p.kg >> 1; half > 0; half >>= 1) {
      const int pair = h + p.nh * (qi + p.qt * (kgrp & (half - 1)));     // < NW / 2
      float* x = exch + (size_t)pair * entry_floats<M>() + lane;
      if (kgrp >= half && kgrp < 2 * half) {
#pragma unroll
        for (int r = 0; r < S::NR; ++r) x[r * 32] = s.o[r];
#pragma unroll
        for (int i = 0; i < S::NM; ++i) x[(S::NR + i) * 32] = s.m[i], x[(S::NR + S::NM + i) * 32] = s.l[i];
      }
      sync();
      if (kgrp < half) join<M>(s, [&](int r) { return x[r * 32]; });
      sync();
    }
  };
  while (w.next()) {
    const int head = (w.hg / p.qs) * p.nh + h, qtile = (w.hg % p.qs) * p.qt + qi;
    const int q0 = qtile * M::kQ, nq = min(M::kQ, g.G - q0);       // <= 0: this warp has no queries
    const long long b = g.b0 + w.b;
    reset(s);
    if (nq > 0)
      math.load_q(g, static_cast<const T*>(g.q) + b * g.q_ld + (long long)head * g.G * g.hd, q0, nq, lane, wscr);
    for (int t = w.t0; t < w.t1; ++t) {
      bool ok = tc::mbar_wait(full0 + 8 * slot, phase, const_cast<volatile int*>(flags));
      if (ok && nq > 0) {
        const int k0 = kgrp * M::kSub;
        math.scores(g, ring0 + slot * slot_bytes + off, masks[slot * kMaskWords + (k0 >> 5)] >> (k0 & 31), lane, s, wscr);
      }
      advance();
      ok = tc::mbar_wait(full0 + 8 * slot, phase, const_cast<volatile int*>(flags)) && ok;
      if (ok && nq > 0) {
        if constexpr (math_scratch<M>() > 0) math.values(g, ring0 + slot * slot_bytes + off, lane, s, wscr);
        else math.values(g, ring0 + slot * slot_bytes + off, lane, s);
      }
      advance();
    }
    math.finish(s);
    merge_groups();
    if (w.t1 - w.t0 < w.nt) {
      // one of several pieces: leave it, and join them all if it is the last to come
      const long long i0 = (long long)pre[w.b] * p.hgq + (long long)w.hg * w.nt;
      const int c0 = (int)(((i0 + 1) * C - 1) / total), c1 = (int)(((i0 + w.nt) * C - 1) / total);
      auto entry = [&](int c) {                 // a CTA's first piece may have begun before it, its last may go on
        return g.part + (((long long)c * 2 + (c == c0)) * NW + h + p.nh * qi) * entry_floats<M>() + lane * 4;
      };
      if (kgrp == 0) {
        float* x = entry(cta);
#pragma unroll
        for (int r = 0; r < S::NR; r += 4) __stcg(reinterpret_cast<float4*>(x + r * 32), make_float4(s.o[r], s.o[r + 1], s.o[r + 2], s.o[r + 3]));
        float ml[2 * S::NM];
#pragma unroll
        for (int i = 0; i < S::NM; ++i) ml[i] = s.m[i], ml[S::NM + i] = s.l[i];
#pragma unroll
        for (int r = 0; r < 2 * S::NM; r += 4)
          __stcg(reinterpret_cast<float4*>(x + (S::NR + r) * 32), make_float4(ml[r], ml[r + 1], ml[r + 2], ml[r + 3]));
      }
      __threadfence();
      sync();
      if (tid == 0) {
        int* ctr = &g.counters[b * p.hgq + w.hg];
        const bool last = atomicAdd(ctr, 1) == c1 - c0;
        if (last) *ctr = 0;
        flags[1] = last;
      }
      sync();
      if (!flags[1]) continue;
      __threadfence();
      reset(s);
      for (int c = c0 + kgrp; c <= c1; c += p.kg) {
        const float* x = entry(c);
        float y[S::NR + 2 * S::NM];
#pragma unroll
        for (int r = 0; r < S::NR + 2 * S::NM; r += 4) {
          const float4 f = __ldcg(reinterpret_cast<const float4*>(x + r * 32));
          y[r] = f.x, y[r + 1] = f.y, y[r + 2] = f.z, y[r + 3] = f.w;
        }
        join<M>(s, [&](int r) { return y[r]; });
      }
      merge_groups();
    }
    if (kgrp == 0 && nq > 0) {
      T* out = static_cast<T*>(g.out) + b * g.out_ld + ((long long)head * g.G + q0) * g.hd;
      float inv[S::NM];
#pragma unroll
      for (int i = 0; i < S::NM; ++i) {
        inv[i] = s.l[i] == 0.f ? 0.f : g.v_scale / s.l[i];
        const int q = M::stat_query(i, lane);
        if (g.lse && M::stat_owner(lane) && q < nq)
          g.lse[b * g.nq + (long long)head * g.G + q0 + q] = s.l[i] == 0.f ? -INFINITY : (s.m[i] + log2f(s.l[i])) * kLn2;
      }
#pragma unroll
      for (int r = 0; r < S::NR; ++r) {
        const int q = M::query(r, lane), c = M::comp(r, lane);
        if (q < nq && c < g.hd) {
          const float x = s.o[r] * inv[M::st(r)];
          if constexpr (std::is_same_v<T, float>) out[(long long)q * g.hd + c] = x;
          else if constexpr (std::is_same_v<T, __half>) out[(long long)q * g.hd + c] = __float2half_rn(x);
          else out[(long long)q * g.hd + c] = __float2bfloat16_rn(x);
        }
      }
    }
  }
  if (tid == 0 && flags[0]) report(g.ws, SPEC_ERR_TIMEOUT);
}

// What the planner needs to know of an instantiation, and its launch.
struct Kernel {
  void (*fn)(Args);
  int warps, sub, kq, es;
  size_t (*fixed)(int);
};
template <typename M> Kernel kernel_of() {
  static_assert(M::kWarps * entry_floats<M>() <= 8 * 72 * 32, "a CTA's piece fits the workspace");
  return {paged_attention_kernel<M>, M::kWarps, M::kSub, M::kQ, M::kEs,
          [](int B) { return fixed_smem<M>(B); }};
}

Kernel kernel_bf16(bool e4m3, int hd, int G);
Kernel kernel_f16(bool e4m3, int hd, int G);
Kernel kernel_f32(int hd, int G);

// 8 queries a warp, 16 where a kv head has more than 8 (not above 128 components, where the state
// of 16 queries would not fit in registers)
template <typename T, bool F8> Kernel pick16(int hd, int G) {
  if (hd <= 64) return G <= 8 ? kernel_of<MmaMath<T, F8, 64, 1>>() : kernel_of<MmaMath<T, F8, 64, 2>>();
  if (hd <= 128) return G <= 8 ? kernel_of<MmaMath<T, F8, 128, 1>>() : kernel_of<MmaMath<T, F8, 128, 2>>();
  return kernel_of<MmaMath<T, F8, 256, 1>>();
}

}  // namespace pa
}  // namespace spec
