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
constexpr int kFlat = 8;                 // up to so many pieces are joined at once
constexpr int kMaskWords = 8;            // validity words of a tile of at most 256 keys
// Registers a thread of 8 + 4 warps is launched with, and those after the two kinds of warps have
// shared them out (kMoreRegs): 4 x 88 + 8 x 208 = 12 x 168.
constexpr int kLaunchRegs = 168, kProducerRegs = 88, kConsumerRegs = 208;
static_assert(4 * kProducerRegs + 8 * kConsumerRegs <= 12 * kLaunchRegs, "");
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// How a call's work is cut (host, paged_attn.cu).
struct Plan {
  int nh;          // kv heads of a tile
  int qt;          // query tiles of a kv head (warps over the same keys)
  int kg;          // key groups, a power of two: nh * qt * kg units of consumer warps, at most all of them
  int kt;          // keys of a tile
  int hgq;         // head groups x query splits of a request
  int qs;          // query splits (K/V is read once per split; 1 unless nq / nkv is large)
  int qtiles;      // query tiles of a kv head in all
  int slots;       // ring slots of slot_bytes each: one K or V tile
  int slot_bytes;
  // A tile in shared memory: 16-byte unit u of key j of head h lies at
  //   (j >> run_lg) * run_bytes + (j & (run - 1)) * key_stride + h * head_stride +
  //   (u >> 3) * chunk_stride + (((u & 7) << 4) ^ swizzle(j)).
  // Runs (block sizes that are multiples of 8): `run` consecutive slots of a block come as one tensor
  // copy of all of the tile's heads, [head][128-byte chunk][slot] in TMA's 128-byte swizzle (rows that
  // are no multiple of 128 bytes: one copy a chunk, [chunk][head][slot], zeros past the row's end).  Rows (other block sizes): one bulk copy a key, rows apart
  // by an odd multiple of 16 bytes, no swizzle.  Either way 8 keys' units are in 8 bank groups.
  int swz, run_lg, run_bytes, key_stride, head_stride, chunk_stride;
  int copies;      // tensor copies of a run: 1, or the 128-byte chunks of a head's row
  int row;         // rows: bytes of one key's nh heads
  int full;        // rows in shared memory have all the components that the kernel handles (zeros past the head's)
};

struct Args {
  CUtensorMap tmk, tmv;   // runs: [nkv][chunks][slots][128 bytes] views of the cache
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
  int* counters;         // [B, hgq]
  int* group_counters;   // [grid, 2]
  float* part;     // [grid, 2, warps, entry]
  void* ws;
};

// quotient and root of the cost model: the device's need only be the same in every CTA
__host__ __device__ inline float cost_div(float a, float b) {
#ifdef __CUDA_ARCH__
  return __fdividef(a, b);
#else
  return a / b;
#endif
}
__host__ __device__ inline float cost_sqrt(float x) {
#ifdef __CUDA_ARCH__
  float y;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
#else
  return sqrtf(x);
#endif
}

// What it costs, in tiles (64 KB, ~1.35 us), to leave n pieces of an item and join
// them: the exchange itself, a second level beyond kFlat pieces, and the pieces that
// the joining CTA reads one after another, its kg key groups taking turns.
__host__ __device__ inline float join_cost(int n, float per_kg) {
  if (n <= 1) return 0.f;
  const float reads = n > kFlat ? 2.f * cost_sqrt((float)n) + 1.f : (float)n;
  return (n > kFlat ? 2.5f : 1.5f) + 0.37f * fmaxf(reads * per_kg, 1.f);
}

// How `total` tiles of `items` (request, head group)s, the longest of `most` tiles, are
// shared out: in `cuts` equal pieces an item, a CTA each, or (cuts = 0) in equal
// shares of the tiles in a row, which begin and end inside items.  Returns the cost
// in tiles.  Measured: 16 requests of 1000 keys, 128 items of 8 tiles, 12.7 us whole,
// 17.5 in shares; 4 requests, 32 items of 8 tiles, 11.9 whole, 9.8 in 4 pieces each, 12.7
// in shares; 64 requests of up to 8190 keys, 128 items of 256 tiles, 160 us in shares.
//
// In fp32 throughout: every CTA works it out for itself before it can start.
__host__ __device__ inline float share_out(long long total_, long long items_, int most, int kg, int ctas, int* cuts) {
  const float total = (float)total_, items = (float)items_, used = fminf(total, (float)ctas), per_kg = cost_div(1.f, (float)kg);
  // merging the key groups; ~0.8 tiles for every further item that a share touches
  const float base = kg == 1 ? 0.f : kg == 2 ? 0.1f : kg == 4 ? 0.2f : 0.3f;
  float best = cost_div(total + 0.8f * items, used) + 2.f;
  const int pieces = (int)cost_div(used + 0.5f, items) + 1;
  best += join_cost(pieces > 2 ? pieces : 2, per_kg);
  *cuts = 0;
  if (items <= (float)ctas) {
    const int room = (int)cost_div((float)ctas + 0.5f, items), all = room < most ? room : most;
    const int few = all < kFlat ? all : kFlat;
    if ((float)most <= best) best = (float)most, *cuts = 1;
    const float c8 = ceilf(cost_div((float)most - 0.5f, (float)few)) + join_cost(few, per_kg);
    if (c8 < best) best = c8, *cuts = few;
    if (all > few) {
      const float ca = ceilf(cost_div((float)most - 0.5f, (float)all)) + join_cost(all, per_kg);
      if (ca < best) best = ca, *cuts = all;
    }
  }
  return best + base;
}

// A consumer warp's running state for one (kv head, query tile): unnormalised
// outputs o, references m (running maxima, or a constant below; log2 units) and sums l, in the layout of its math.
// Register r of o belongs to statistics index st(r).
template <int NR_, int NM_> struct State {
  static constexpr int NR = NR_, NM = NM_;
  alignas(8) float o[NR];
  float m[NM], l[NM];
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

SPEC_DEV void tma_run(uint32_t dst, const CUtensorMap* tm, uint32_t mbar, int x, int slot, int head, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3, %4, %5}], [%6], %7;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tm)), "r"(x), "r"(slot), "r"(0), "r"(head), "r"(mbar), "l"(policy)
      : "memory");
}

// Where a lane's key row is in a tile: offset, and the swizzle of its units.
struct Row {
  uint32_t off, x;
  SPEC_DEV Row(const Plan& p, int key, int head)
      : off((uint32_t)((key >> p.run_lg) * p.run_bytes + (key & ((1 << p.run_lg) - 1)) * p.key_stride +
                       head * p.head_stride)),
        x(p.swz ? (uint32_t)(key & 7) << 4 : 0u) {}
  SPEC_DEV Row() {}
};

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
// two 8-bit values (low 16 bits of x) as two f16; exact
SPEC_DEV uint32_t widen(uint32_t x) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(x & 0xffffu), __NV_E4M3);
  const __half2 f = h;
  return *reinterpret_cast<const uint32_t*>(&f);
}

// Scores and outputs of 16 keys x one kv head x 8 NT queries on warp-level matrix
// instructions, keys and head-dim components in the rows: S^T = K Q^T and
// O^T += V^T P^T.  The instruction's 8-wide side is the queries, of which a decode
// step has few; K rows and (transposed) V rows come out of shared memory as they
// lie.  tcgen05 would want 128 rows of one operand per 16 keys' work.
//
// Where a head's row is 128 bytes or less (and 8-bit rows of up to 256) a step takes U = 2
// tiles of 16 keys: the chain of dependent instructions is the same for twice the
// bytes.  Wider rows fill a ring slot with one.
//
// 8-bit caches are multiplied in f16, which their values convert to in one
// instruction (bf16 would take four).  bf16 queries are scaled by a power of two per
// query, their largest component to [2^14, 2^15): exact but for components 2^28 times
// smaller than that, and undone in the scores' scale.
template <typename T, bool F8, int HD, int NT> struct MmaMath {
  using In = T;
  static constexpr int kHd = HD;
  using P = std::conditional_t<F8, __half, T>;      // operands of the products
  static constexpr bool kScaled = F8 && std::is_same_v<T, __nv_bfloat16>;
  float qs[2 * NT];        // kScaled: scores' scale by query
  static constexpr int kEs = F8 ? 1 : 2, U = HD * kEs <= 128 || (F8 && HD > 128) ? 2 : 1;
  static constexpr int kSub = 16 * U, kQ = 8 * NT;
  // above 128 components two warps share keys and queries: both compute the scores, each half of the outputs
  static constexpr int kWarps = 8, VS = HD > 128 ? 2 : 1, MT = HD / 16 / VS;
  static constexpr bool kMoreRegs = NT == 2 && HD >= 128;
  using S = State<MT * NT * 4, 2 * NT>;
  // m is the largest score less kBelow: weights are up to 2^kBelow.  f16 has no exponents for small ones: with weights up
  // to 1, those under 2^-25 would be lost and those under 2^-14 held in steps of 2^-24 (a first key 14 above 1000 others,
  // its value zero: the output 8e-3 off).  2^15 is the largest power of two below f16's largest number.
  static constexpr float kBelow = std::is_same_v<P, __half> ? 15.f : 0.f;
  // register r = (mt NT + nt) 4 + 2 i + j: query nt 8 + 2 (lane & 3) + j, component mt 16 + (lane >> 2) + 8 i
  // (8-bit caches: mt 16 + 2 (lane >> 2) + i)
  SPEC_DEV static int st(int r) { return ((r >> 2) % NT) * 2 + (r & 1); }
  // outputs two components at a time
  SPEC_DEV static void write(const S& s, const float* inv, T* out, int hd, int nq, int lane, int vs) {
    if (hd == HD) write_as<true>(s, inv, out, HD, nq, lane, vs);
    else write_as<false>(s, inv, out, hd, nq, lane, vs);
  }
  template <bool FULL> SPEC_DEV static void write_as(const S& s, const float* inv, T* out, int hd, int nq, int lane, int vs) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      if (nt * 8 >= nq) break;
      if constexpr (F8) {
        T* o = out + (long long)(nt * 8 + 2 * t) * hd + vs * MT * 16 + 2 * g;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
          if (FULL || (vs * MT + mt) * 16 < hd)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const float* x = &s.o[(mt * NT + nt) * 4 + j];
              if (nt * 8 + 2 * t + j < nq)
                *reinterpret_cast<uint32_t*>(o + j * hd + mt * 16) = pack<T>(x[0] * inv[nt * 2 + j], x[2] * inv[nt * 2 + j]);
            }
      } else {
        // 8 components x 8 queries transposed: lane then has components 2 t, 2 t + 1 of query g
        T* o = out + (long long)(nt * 8 + g) * hd + vs * MT * 16 + 2 * t;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
          if (FULL || (vs * MT + mt) * 16 < hd)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float* x = &s.o[(mt * NT + nt) * 4 + 2 * i];
              const uint32_t y = movm(pack<T>(x[0] * inv[nt * 2], x[1] * inv[nt * 2 + 1]));
              if (nt * 8 + g < nq) *reinterpret_cast<uint32_t*>(o + mt * 16 + 8 * i) = y;
            }
      }
    }
  }
  SPEC_DEV static int stat_query(int i, int lane) { return (i >> 1) * 8 + 2 * (lane & 3) + (i & 1); }
  SPEC_DEV static bool stat_owner(int lane) { return lane < 4; }

  Row rk, rv;              // this lane's K row (units lane >> 4 and up) and V row
  uint32_t next;           // from one tile of 16 keys to the next
  SPEC_DEV void init(const Plan& p, int key0, int head, int lane, uint32_t) {
    rk = Row(p, key0 + (lane & 15), head);
    rk.x ^= (lane >> 4) << 4;
    next = Row(p, key0 + (lane & 15) + 16 * (U - 1), head).off - rk.off;
    rv = rk;
    if constexpr (!F8) {
      rv = Row(p, key0 + (lane & 7) + (lane >> 4) * 8, head);
      rv.x ^= ((lane >> 3) & 1) << 4;
    }
  }
  // address of units 2 i, 2 i + 1 (by lane) of a row
  SPEC_DEV static uint32_t unit2(const Plan& p, uint32_t row, uint32_t x, int i) {
    return row + (i >> 2) * p.chunk_stride + ((uint32_t)((i & 3) << 5) ^ x);
  }

  uint32_t qf[HD / 16][NT][2];
  uint32_t pf[U][NT][4];   // P^T operands: high parts of keys 0-7 and 8-15, low parts of both
  uint32_t vm;             // valid keys
  static constexpr uint32_t kAll = U == 2 ? 0xffffffffu : 0xffffu;

  // queries of the tile: q points at the kv head's first query, n of them from q0 on exist
  SPEC_DEV void load_q(const Args& g, const T* q, int q0, int n, int lane) {
    if (g.hd == HD) load_q_as<true>(q + (long long)q0 * HD, HD, n, lane);
    else load_q_as<false>(q + (long long)q0 * g.hd, g.hd, n, lane);
  }
  template <bool FULL> SPEC_DEV void load_q_as(const T* q, int hd, int n, int lane) {
    const int gq = lane >> 2, t = lane & 3;
#pragma unroll
    for (int ks = 0; ks < HD / 16; ++ks)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int i = nt * 8 + gq;
        qf[ks][nt][0] = qf[ks][nt][1] = 0;
        if (i < n && (FULL || ks * 16 < hd)) {
          const T* p = q + (long long)i * hd + ks * 16;
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
  // after load_q, once its values are needed
  SPEC_DEV void scale_q(const Args& g, int lane) {
    if constexpr (kScaled) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        uint32_t big = 0;           // largest magnitude: as integers, bf16 magnitudes compare like numbers
#pragma unroll
        for (int ks = 0; ks < HD / 16; ++ks)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t x = qf[ks][nt][h] & 0x7fff7fffu;
            big = max(big, max(x >> 16, x & 0xffffu));
          }
        big = max(big, __shfl_xor_sync(0xffffffffu, big, 1));
        big = max(big, __shfl_xor_sync(0xffffffffu, big, 2));
        // 2^(14 - exponent); 1 for a zero row or one that is not finite
        const int e = big == 0 || big >= 0x7f80u ? 127 + 14 : max((int)(big >> 7), 15);
        const float up = __uint_as_float((uint32_t)(127 + 14 + 127 - e) << 23), down = __uint_as_float((uint32_t)(e - 14) << 23);
#pragma unroll
        for (int ks = 0; ks < HD / 16; ++ks)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float2 f = unpack<T>(qf[ks][nt][h]);
            qf[ks][nt][h] = pack<P>(f.x * up, f.y * up);
          }
#pragma unroll
        for (int j = 0; j < 2; ++j) qs[2 * nt + j] = __shfl_sync(0xffffffffu, down, (2 * (lane & 3) + j) * 4) * g.scale2;
      }
    }
  }

  // one tile of 16 keys x 8 queries: two sums over alternate 16 components, so that two chains of
  // products run side by side
  static constexpr int A = U * NT == 1 ? 2 : 1;
  static constexpr int KS = F8 ? HD / 32 : HD / 16, VSTEPS = KS / VS;     // steps of 32 bytes of a row
  float ca[A][U][NT][4];   // scores of the tile whose keys were read last
  SPEC_DEV void clear() {
#pragma unroll
    for (int i = 0; i < A * U * NT * 4; ++i) (&ca[0][0][0][0])[i] = 0.f;
  }
  // FULL: rows have all HD components (no branches between the instructions of several steps)
  template <bool FULL> SPEC_DEV void dot_step(const Args& g, uint32_t k, int i) {
    if (!FULL && i * (HD / KS) >= g.hd) return;
    const uint32_t a0 = k + rk.off;
    uint32_t r[U][4];
#pragma unroll
    for (int u = 0; u < U; ++u) ldsm4(unit2(g.p, a0 + u * next, rk.x, i), r[u]);
    if constexpr (F8) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if (!FULL && i * 32 + j * 16 >= g.hd) break;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          uint32_t a[4];
          a[0] = widen(r[u][2 * j]), a[1] = widen(r[u][2 * j + 1]);
          a[2] = widen(r[u][2 * j] >> 16), a[3] = widen(r[u][2 * j + 1] >> 16);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma<P>(ca[A == 2 ? j : 0][u][nt], a, qf[i * 2 + j][nt][0], qf[i * 2 + j][nt][1]);
        }
      }
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma<P>(ca[i % A][u][nt], r[u], qf[i][nt][0], qf[i][nt][1]);
    }
  }
  // ALL: every key is valid
  template <bool FULL, bool ALL> SPEC_DEV void value_step(const Args& g, uint32_t v, S& s, int vs, int il, const uint32_t (*z)[2]) {
    const int i = vs * VSTEPS + il;
    if (!FULL && i * (HD / KS) >= g.hd) return;
    const uint32_t a0 = v + rv.off;
    uint32_t r[U][4];
#pragma unroll
    for (int u = 0; u < U; ++u) ldsm4t(unit2(g.p, a0 + u * next, rv.x, i), r[u]);
    auto step = [&](int mt, int u, uint32_t* a) {
      if (!ALL) a[0] &= z[u][0], a[1] &= z[u][0], a[2] &= z[u][1], a[3] &= z[u][1];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float* o = &s.o[(mt * NT + nt) * 4];
        mma<P>(o, a, pf[u][nt][0], pf[u][nt][1]);
        mma<P>(o, a, pf[u][nt][2], pf[u][nt][3]);
      }
    };
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if constexpr (F8) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          if (!FULL && i * 32 + j * 16 >= g.hd) break;
          // bytes (key, component): 00 01 10 11 -> component 0 of both keys, component 1 of both
          const uint32_t x = __byte_perm(r[u][2 * j], 0, 0x3120), y = __byte_perm(r[u][2 * j + 1], 0, 0x3120);
          uint32_t a[4] = {widen(x), widen(x >> 16), widen(y), widen(y >> 16)};
          step(il * 2 + j, u, a);
        }
      } else {
        step(il, u, r[u]);
      }
    }
  }
  // scores of this warp's keys in the K tile at shared address k
  SPEC_DEV void dots(const Args& g, uint32_t k, uint32_t mask) {
    if ((mask & kAll) == 0) return;
    clear();
    if (g.p.full) {
#pragma unroll
      for (int i = 0; i < KS; ++i) dot_step<true>(g, k, i);
    } else {
#pragma unroll
      for (int i = 0; i < KS; ++i) dot_step<false>(g, k, i);
    }
  }
  // that and values() of the tile before: two independent chains of instructions in one run without a branch
  SPEC_DEV bool can_run_both(const Args& g, uint32_t mask) const { return vm == kAll && (mask & kAll) == kAll && g.p.full; }
  SPEC_DEV void both(const Args& g, uint32_t k, uint32_t v, S& s, int vs) {
    clear();
#pragma unroll
    for (int i = 0; i < KS; ++i) {
      dot_step<true>(g, k, i);
      if (i % VS == 0) value_step<true, true>(g, v, s, vs, i / VS, nullptr);
    }
  }
  // scores become weights: running statistics
  SPEC_DEV void weights(const Args& g, uint32_t mask, int lane, S& s) {
    vm = mask & kAll;
    if (vm == 0) return;
    auto& c = ca[0];
    if constexpr (A == 2) {
#pragma unroll
      for (int i = 0; i < U * NT * 4; ++i) (&ca[0][0][0][0])[i] += (&ca[A - 1][0][0][0])[i];
    }
    bool grew = false;
    float mn[2 * NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float x = -INFINITY;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const uint32_t v = vm >> (16 * u + (lane >> 2));
          const float sc = kScaled ? qs[nt * 2 + j] : g.scale2;
          c[u][nt][j] = v & 1 ? c[u][nt][j] * sc : -INFINITY;
          c[u][nt][2 + j] = v >> 8 & 1 ? c[u][nt][2 + j] * sc : -INFINITY;
          x = fmaxf(x, fmaxf(c[u][nt][j], c[u][nt][2 + j]));
        }
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16)) - kBelow;
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
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float b = base_of(s.m[nt * 2 + j]);
          c[u][nt][j] = exp2_fast(c[u][nt][j] - b);
          c[u][nt][2 + j] = exp2_fast(c[u][nt][2 + j] - b);
          s.l[nt * 2 + j] += c[u][nt][j] + c[u][nt][2 + j];
        }
        // a weight enters the second product as two 16-bit parts: one alone (2^-8 of it in bf16)
        // would cost as much as the output's own rounding.  Two bf16 parts lose 2^-17 of it; two f16 parts 2^-23, or
        // where the lower one is subnormal 2^-25, 2^-40 of the largest weight (kBelow)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t hi = pack<P>(c[u][nt][2 * h], c[u][nt][2 * h + 1]);
          const float2 f = unpack<P>(hi);
          pf[u][nt][h] = movm(hi);
          pf[u][nt][2 + h] = movm(pack<P>(c[u][nt][2 * h] - f.x, c[u][nt][2 * h + 1] - f.y));
        }
      }
  }

  SPEC_DEV void values(const Args& g, uint32_t v, int lane, S& s, int vs) {
    if (vm == 0) return;
    const int t2 = 2 * (lane & 3);
    // rows of keys that are not valid may hold anything: their bits are cleared
    uint32_t z[U][2];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t b = vm >> (16 * u + 8 * h + t2);
        z[u][h] = (b & 1 ? 0xffffu : 0) | (b & 2 ? 0xffff0000u : 0);
      }
    if (g.p.full) {
#pragma unroll
      for (int i = 0; i < VSTEPS; ++i) value_step<true, false>(g, v, s, vs, i, z);
    } else {
#pragma unroll
      for (int i = 0; i < VSTEPS; ++i) value_step<false, false>(g, v, s, vs, i, z);
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

// The same for 32-bit caches on fp32 multiply-adds: 8 keys x NQ (4 or 8) queries a step.
// A row's components are spread over R lanes (16 up to 64 components, where each half of
// the warp takes 4 of the keys; else 32), so that a row is read from shared memory once for
// all queries.  The partial sums are added up over the lanes in a butterfly that halves
// their number at every step and leaves a lane with one key's NQ / 4 scores; a lane
// takes keys and queries in an order of its own (its number's bits flipped), so that what it
// keeps is always the first half.  Queries go in pairs through packed multiply-adds.
// Measured: 32 requests of 2000 keys on 8 heads of 128, 32 / 64 / 128 queries 83 / 103 / 186
// us (77 at the copy bandwidth): a warp's step runs its multiply-adds, shuffles and
// shared-memory reads one after another, each ~60 us of the 186 (above 8 queries two warps read the same rows).  (Lanes with a key each and queries in
// shared memory: 64 queries 127 us; three tf32 products per product 122.)
template <int HD, int NQ> struct F32Math {
  using In = float;
  static constexpr bool kMoreRegs = false;
  static constexpr int kHd = HD, kSub = 8, kQ = NQ, kEs = 4, kWarps = HD > 128 ? 4 : 8, VS = 1;
  static constexpr int R = HD <= 64 ? 16 : 32, E = HD / R, NP = NQ / 2, J = NQ / 4;   // a lane's components and own scores
  static constexpr int KK = 8 * R / 32;      // keys a lane looks at
  using S = State<NQ * E, NQ>;
  // register r of o: pair of queries, component, query of the pair
  SPEC_DEV static int reg(int i, int e) { return (i >> 1) * 2 * E + e * 2 + (i & 1); }
  SPEC_DEV static int st(int r) { return r / (2 * E) * 2 + (r & 1); }
  SPEC_DEV static int stat_query(int i, int) { return i; }
  SPEC_DEV static bool stat_owner(int lane) { return lane == 0; }
  // the first of components 4 u .. 4 u + 3 of a lane
  SPEC_DEV static int comp(int u, int lane) { return 4 * (u * R + (lane & (R - 1))); }
  SPEC_DEV static void write(const S& s, const float* inv, float* out, int hd, int nq, int lane, int) {
#pragma unroll
    for (int i = 0; i < NQ; ++i)
#pragma unroll
      for (int u = 0; u < E / 4; ++u)
        if (i < nq && comp(u, lane) < hd && lane < R)
          *reinterpret_cast<float4*>(out + (long long)i * hd + comp(u, lane)) =
              make_float4(s.o[reg(i, 4 * u)] * inv[i], s.o[reg(i, 4 * u + 1)] * inv[i], s.o[reg(i, 4 * u + 2)] * inv[i],
                          s.o[reg(i, 4 * u + 3)] * inv[i]);
  }
  static constexpr int kScratch = NQ * 8;    // a step's weights

  float2 qf[NP][E];        // place i: query i ^ flip(lane)
  float mo[J], lo[J];      // running maxima and this lane's sums of its own queries
  uint32_t vm, zero;       // valid keys; 16 bytes of zeros
  uint32_t koff[KK], voff[KK], upper;        // offsets of a lane's K and V rows; from u to u + 1
  bool in[E / 4];

  SPEC_DEV static int flip(int lane) { return (lane & 2 ? NQ / 2 : 0) | (lane & 1 ? NQ / 4 : 0); }
  SPEC_DEV void init(const Plan& p, int key0, int head, int lane, uint32_t zero_) {
    zero = zero_;
    const uint32_t byte = comp(0, lane) * 4, unit = (byte >> 7) * p.chunk_stride, x = byte & 127;
    upper = (R * 16 >> 7) * p.chunk_stride;
#pragma unroll
    for (int k = 0; k < KK; ++k) {
      const Row rk(p, key0 + (k ^ (lane >> 2)), head), rv(p, key0 + (R == 16 ? (lane >> 4) * 4 + k : k), head);
      koff[k] = rk.off + unit + (x ^ rk.x);
      voff[k] = rv.off + unit + (x ^ rv.x);
    }
  }
  SPEC_DEV void load_q(const Args& g, const float* q, int q0, int n, int lane) {
#pragma unroll
    for (int u = 0; u < E / 4; ++u) {
      in[u] = comp(u, lane) < g.hd;
#pragma unroll
      for (int i = 0; i < NQ; ++i) {
        const int j = i ^ flip(lane);
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (j < n && in[u]) x = *reinterpret_cast<const float4*>(q + (long long)(q0 + j) * g.hd + comp(u, lane));
        float* o = reinterpret_cast<float*>(&qf[i >> 1][4 * u]) + (i & 1);
        o[0] = x.x, o[2] = x.y, o[4] = x.z, o[6] = x.w;
      }
    }
  }
  SPEC_DEV void scale_q(const Args&, int) {
#pragma unroll
    for (int j = 0; j < J; ++j) mo[j] = -INFINITY, lo[j] = 0.f;
  }
  // a lane's components of a row (zeros past the head's end, or if the row is not wanted)
  SPEC_DEV void read(uint32_t row, bool wanted, float* x) const {
#pragma unroll
    for (int u = 0; u < E / 4; ++u) {
      const uint32_t a = in[u] && wanted ? row + u * upper : zero;
      asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];"
                   : "=f"(x[4 * u]), "=f"(x[4 * u + 1]), "=f"(x[4 * u + 2]), "=f"(x[4 * u + 3]) : "r"(a) : "memory");
    }
  }
  SPEC_DEV static float2 plus_other(float2 keep, float2 give, int o) {
    return __fadd2_rn(keep, make_float2(__shfl_xor_sync(0xffffffffu, give.x, o), __shfl_xor_sync(0xffffffffu, give.y, o)));
  }
  // dot products of a lane's components of key k
  SPEC_DEV void dots(uint32_t tile, int k, float2* d) const {
    float x[E];
    read(tile + koff[k], true, x);
#pragma unroll
    for (int i = 0; i < NP; ++i) d[i] = __fmul2_rn(make_float2(x[0], x[0]), qf[i][0]);
#pragma unroll
    for (int e = 1; e < E; ++e)
#pragma unroll
      for (int i = 0; i < NP; ++i) d[i] = __ffma2_rn(make_float2(x[e], x[e]), qf[i][e], d[i]);
  }
  SPEC_DEV void scores(const Args& g, uint32_t k, uint32_t mask, int lane, S& s, float* w) {
    vm = mask & 0xffu;
    if (vm == 0) return;
    float2 d[4][NP];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      dots(k, i, d[i]);
      if constexpr (R == 32) {
        float2 e[NP];
        dots(k, i + 4, e);
#pragma unroll
        for (int j = 0; j < NP; ++j) d[i][j] = plus_other(d[i][j], e[j], 16);
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < NP; ++j) d[i][j] = plus_other(d[i][j], d[i + 2][j], 8);
#pragma unroll
    for (int j = 0; j < NP; ++j) d[0][j] = plus_other(d[0][j], d[1][j], 4);
#pragma unroll
    for (int j = 0; j < NP / 2; ++j) d[0][j] = plus_other(d[0][j], d[0][j + NP / 2], 2);
    float c[J];                    // key lane >> 2, query J (lane & 3) + j
    if constexpr (J == 2) {
      const float2 x = plus_other(d[0][0], d[0][1], 1);
      c[0] = x.x, c[J - 1] = x.y;
    } else {
      c[0] = d[0][0].x + __shfl_xor_sync(0xffffffffu, d[0][0].y, 1);
    }
    const bool ok = vm >> (lane >> 2) & 1;
    bool grew = false;
    float mn[J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
      c[j] = ok ? c[j] * g.scale2 : -INFINITY;
      float x = c[j];
      x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
      x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
      x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
      mn[j] = fmaxf(mo[j], x);
      grew |= x > mo[j];
    }
    if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
      for (int j = 0; j < J; ++j) {
        lo[j] *= exp2_fast(mo[j] - base_of(mn[j]));
        mo[j] = mn[j];
      }
      float al[NQ];
#pragma unroll
      for (int i = 0; i < NQ; ++i) {
        const float m = __shfl_sync(0xffffffffu, mn[i % J], i / J);
        al[i] = exp2_fast(s.m[i] - base_of(m));
        s.m[i] = m;
      }
#pragma unroll
      for (int r = 0; r < S::NR; ++r) s.o[r] *= al[st(r)];
    }
    __syncwarp();
#pragma unroll
    for (int j = 0; j < J; ++j) {
      c[j] = exp2_fast(c[j] - base_of(mo[j]));
      lo[j] += c[j];
      w[J * lane + j] = c[j];      // [key][query]
    }
    __syncwarp();
  }
  SPEC_DEV void values(const Args& g, uint32_t v, int lane, S& s, const float* w) {
    if (vm == 0) return;
    const int key0 = R == 16 ? (lane >> 4) * 4 : 0;
    const uint32_t ok = vm >> key0;
#pragma unroll
    for (int k = 0; k < KK; ++k) {
      float x[E];
      float4 pr[NQ / 4];
      read(v + voff[k], ok >> k & 1, x);               // the row of a key that is not valid may hold anything
#pragma unroll
      for (int i = 0; i < NQ / 4; ++i) pr[i] = *reinterpret_cast<const float4*>(w + (key0 + k) * NQ + 4 * i);
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const float2 p2 = i & 1 ? make_float2(pr[i / 2].z, pr[i / 2].w) : make_float2(pr[i / 2].x, pr[i / 2].y);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          float2* o = reinterpret_cast<float2*>(&s.o[reg(2 * i, e)]);
          *o = __ffma2_rn(p2, make_float2(x[e], x[e]), *o);
        }
      }
    }
  }
  SPEC_DEV void finish(S& s) {
#pragma unroll
    for (int j = 0; j < J; ++j) {
      lo[j] += __shfl_xor_sync(0xffffffffu, lo[j], 4);
      lo[j] += __shfl_xor_sync(0xffffffffu, lo[j], 8);
      lo[j] += __shfl_xor_sync(0xffffffffu, lo[j], 16);
    }
#pragma unroll
    for (int i = 0; i < NQ; ++i) s.l[i] = __shfl_sync(0xffffffffu, lo[i % J], i / J);
    if constexpr (R == 16) {
#pragma unroll
      for (int r = 0; r < S::NR; ++r) s.o[r] += __shfl_xor_sync(0xffffffffu, s.o[r], 16);
    }
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
  return 2048 + (size_t)kMaxSlots * kMaskWords * 4 + (size_t)(2 * B + 4) / 4 * 16 +
         4 * (size_t)(exchange_floats<M>() + M::kWarps * math_scratch<M>());
}

template <typename S> SPEC_DEV void reset(S& s) {
#pragma unroll
  for (int r = 0; r < S::NR; ++r) s.o[r] = 0.f;
#pragma unroll
  for (int i = 0; i < S::NM; ++i) s.m[i] = -INFINITY, s.l[i] = 0.f;
}
// s and another state of the same queries: get(r) is its o[r], then its m and l
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

// a / b for 0 <= a, 0 < b: in fp32 where that is exact (a < 2^20: the quotient of a + 0.5 is at least 0.5 / b
// from an integer, and within 2^-21 of its value), which is quicker than the integer division
SPEC_DEV int quot(int a, int b) { return a < (1 << 20) ? (int)__fdividef((float)a + 0.5f, (float)b) : a / b; }

// The linear order of a launch's tiles: (request, head group, tile).  CTA c owns tiles
// [c T / C, (c + 1) T / C), or a piece of one item; pre [B + 1]: exclusive prefix sums of the
// requests' tile counts.  A Walk goes through the pieces that a CTA owns.
struct Walk {
  const int* pre;
  int hgq;
  long long left;       // tiles after the current piece
  bool first;
  // current piece: tiles [t0, t1) of head group hg of request b, which has nt
  int b, hg, t0, t1, nt;
  // from tile t of (b, hg)
  SPEC_DEV Walk(const int* pre_, int hgq_, int b_, int hg_, int t, long long tiles)
      : pre(pre_), hgq(hgq_), left(tiles), first(true), b(b_), hg(hg_), t0(t), t1(0), nt(pre_[b_ + 1] - pre_[b_]) {}
  SPEC_DEV bool next() {
    if (left <= 0) return false;
    if (!first) {
      t0 = 0;
      if (++hg == hgq) {
        hg = 0;
        ++b;
        nt = pre[b + 1] - pre[b];
      }
    }
    first = false;
    t1 = left < nt - t0 ? t0 + (int)left : nt;
    left -= t1 - t0;
    return true;
  }
};

// One CTA per SM walks its share of the tiles.  A producer warp each for K and V copies the
// rows of a tile's keys (kt keys x nh heads) into a ring of shared-memory slots, K and V
// tiles in turn; each consumer warp takes 16 or 32 (fp32: 8) keys of one head and one query tile of
// every tile.  Pieces of a (request, head group) that several CTAs share are left
// as partial results; the last CTA of such a group to finish joins them in CTA
// order, so results do not depend on timing.
//
// One pass over K and V with running maxima m and sums l (log2 units): o <- o 2^(m - m') + sum p v,
// p = 2^(s - m').  Bound by the bytes of K and V, which the ring (up to 220 KB an SM) keeps in
// flight.  Measured, 64 requests on 8 K/V heads of 128, 4 queries each: bf16, 4000 keys 155 us (6.75
// TB/s, the copy bandwidth), e4m3 87 (6.0 TB/s: the warps' chain from shared memory through the conversion
// and two products); one request of 131071 keys 85 (152 pieces and their join); 4 of 256 keys 7.3 (launch and
// ~10 dependent steps).  A tile's values and the next tile's scores run as one stretch of
// instructions without a branch, so that two independent chains fill each other's gaps (one after the other:
// e4m3 98 us; 256 components 224 -> 162).
template <typename M>
__global__ void __launch_bounds__(M::kWarps * 32 + 128, 1) paged_attention_kernel(const __grid_constant__ Args g) {
  SPEC_TL(kTLPagedAttn);
  using T = typename M::In;
  using S = typename M::S;
  constexpr int NW = M::kWarps;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const Plan& p = g.p;
  uint8_t* ring = smem_raw + ((1024u - (tc::su32(smem_raw) & 1023u)) & 1023u);
  uint64_t* bars = reinterpret_cast<uint64_t*>(ring + (size_t)p.slots * p.slot_bytes);   // full[kMaxSlots], empty[kMaxSlots]
  volatile int* flags = reinterpret_cast<volatile int*>(bars + 2 * kMaxSlots);              // abort, last
  float* zeros = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(bars) + 512);
  uint32_t* masks = reinterpret_cast<uint32_t*>(reinterpret_cast<uint8_t*>(bars) + 1024);
  float* exch = reinterpret_cast<float*>(masks + kMaxSlots * kMaskWords);
  float* mscr = exch + exchange_floats<M>();
  int* pre = reinterpret_cast<int*>(mscr + NW * math_scratch<M>());
  int* lens = pre + g.B + 1;
  __shared__ int wsum[NW + 4], wmax[NW + 4];
  const uint32_t full0 = tc::su32(bars), empty0 = full0 + 8 * kMaxSlots, zero0 = tc::su32(zeros);
  if (tid == 0) {
    for (int i = 0; i < p.slots; ++i) {
      tc::mbar_init(full0 + 8 * i, 1);
      tc::mbar_init(empty0 + 8 * i, M::kWarps);
    }
    if (p.swz) {
      asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&g.tmk)) : "memory");
      asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&g.tmv)) : "memory");
    }
    for (int i = 0; i < 4; ++i) zeros[i] = 0.f;
    flags[0] = 0;
    pre[0] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  // consumers: the keys, head and queries of a warp
  const int vs = warp % M::VS, unit = warp / M::VS;
  const int kq = quot(unit, p.nh), h = unit - kq * p.nh, kgrp = quot(kq, p.qt), qi = kq - kgrp * p.qt;
  const int k0 = kgrp * M::kSub;
  M math;
  if (warp < NW) math.init(p, k0, h, lane, zero0);
  pdl_wait();
  pdl_trigger();
  // tile counts of the requests (one empty tile where there is nothing to attend to, so that
  // every request is somebody's) and their prefix sums
  const long long most_l = (long long)g.kv.max_blocks * g.kv.block_size;
  const int most = (int)most_l;
  auto first_key = [&](int len) { return g.window > 0 && len > g.window ? len - g.window : 0; };
  constexpr int kThreads = NW * 32 + 128, kPerThread = (kMaxB + kThreads - 1) / kThreads;
  const int per = (g.B + kThreads - 1) / kThreads;
  int most_tiles = 0, mine = 0, own_tiles[kPerThread];
#pragma unroll
  for (int j = 0; j < kPerThread; ++j) {
    const int b = tid * per + j;
    own_tiles[j] = j < per && b < g.B ? g.seq_len[g.b0 + b] : 0;
  }
#pragma unroll
  for (int j = 0; j < kPerThread; ++j) {
    const int b = tid * per + j;
    if (j < per && b < g.B) {
      int len = own_tiles[j];
      if (len < 0 || len > most) {
        if (blockIdx.x == 0) report(g.ws, SPEC_ERR_DEVICE, g.b0 + b, len);
        len = len < 0 ? 0 : most;
      }
      lens[b] = len;
      int lo = first_key(len);
      if (p.swz) lo &= -1 << p.run_lg;       // tiles start with a run
      own_tiles[j] = max(1, quot(len - lo + p.kt - 1, p.kt));
      mine += own_tiles[j];
      most_tiles = max(most_tiles, own_tiles[j]);
    }
  }
  {
    int sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += y;
    }
    most_tiles = __reduce_max_sync(0xffffffffu, most_tiles);
    if (lane == 31) wsum[warp] = sum, wmax[warp] = most_tiles;
    __syncthreads();
    sum -= mine;
#pragma unroll
    for (int w = 0; w < NW + 4; ++w) {
      if (w < warp) sum += wsum[w];
      most_tiles = max(most_tiles, wmax[w]);
    }
#pragma unroll
    for (int j = 0; j < kPerThread; ++j)
      if (j < per && tid * per + j < g.B) pre[tid * per + j + 1] = sum += own_tiles[j];
    __syncthreads();
  }
  const long long total = (long long)pre[g.B] * p.hgq;
  const int cta = blockIdx.x;
  int cuts;
  share_out(total, (long long)g.B * p.hgq, most_tiles, p.kg, gridDim.x, &cuts);
  const long long C = total < (long long)gridDim.x ? total : (long long)gridDim.x;
  int b_at, hg_at = 0, t_at;
  long long tiles;
  if (cuts > 0) {
    const int item = quot(cta, cuts), piece = cta - item * cuts;
    b_at = quot(item, p.hgq);
    if (b_at >= g.B) return;
    hg_at = item - b_at * p.hgq;
    const int nt = pre[b_at + 1] - pre[b_at], n = min(cuts, nt);
    if (piece >= n) return;
    auto cut = [&](int i) { return nt < 4096 ? quot(nt * i, n) : (int)((long long)nt * i / n); };
    t_at = cut(piece);
    tiles = cut(piece + 1) - t_at;
  } else {
    if (cta >= C) return;
    const long long beg = cta * total / C;
    tiles = (cta + 1) * total / C - beg;
    int hi = g.B;
    b_at = 0;
    while (hi - b_at > 1) {
      const int mid = (b_at + hi) >> 1;
      if ((long long)pre[mid] * p.hgq <= beg) b_at = mid;
      else hi = mid;
    }
    const long long off = beg - (long long)pre[b_at] * p.hgq;
    const int nt = pre[b_at + 1] - pre[b_at];
    hg_at = off >> 31 ? (int)(off / nt) : quot((int)off, nt);
    t_at = (int)(off - (long long)hg_at * nt);
  }
  // the CTAs that have pieces of an item: the first, and how many
  auto owners = [&](int b, int hg, int nt, int* first) {
    if (cuts > 0) {
      *first = (b * p.hgq + hg) * cuts;
      return min(cuts, nt);
    }
    const long long i0 = (long long)pre[b] * p.hgq + (long long)hg * nt;
    *first = (int)(((i0 + 1) * C - 1) / total);
    return (int)(((i0 + nt) * C - 1) / total) - *first + 1;
  };
  Walk w(pre, p.hgq, b_at, hg_at, t_at, tiles);
  const uint32_t ring0 = tc::su32(ring), slot_bytes = (uint32_t)p.slot_bytes;

  if (warp >= NW) {
    // ------------------------------------------------------------ producers: K, V
    if constexpr (M::kMoreRegs) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kProducerRegs));
    // Rows have many small copies, which two warps issue in turn (a copy takes a warp ~80 cycles): the
    // second one waits and looks up like the first, which alone writes the masks and arrives.
    const int v = (warp - NW) & 1, second = (warp - NW) >> 1;
    if (second && p.swz) return;
    const uint64_t policy = tc::policy_evict_first();      // each K/V row is read once
    const long long row_all = (long long)g.nkv * g.hd * M::kEs;
    const int bs = g.kv.block_size, shift = (bs & (bs - 1)) == 0 ? __ffs(bs) - 1 : -1;
    const int run = 1 << p.run_lg, runs = p.kt >> p.run_lg, copies = runs * p.copies;
    int slot = v, phase = 0, issued = 0;                   // every second slot in turn is this warp's
    auto room = [&] { return __all_sync(0xffffffffu, tc::mbar_wait(empty0 + 8 * slot, phase ^ 1, const_cast<volatile int*>(flags))); };
    auto passed = [&] {
      ++issued;
      if ((slot += 2) >= p.slots) slot -= p.slots, phase ^= 1;
    };
    auto head_of_group = [&] { return (p.qs == 1 ? w.hg : w.hg / p.qs) * p.nh; };
    bool ok = true, have = w.next();
    int t = w.t0;
    // The table entries of the next tile are on their way while this one waits for room.
    if (p.swz) {
      // lane r has run r's block
      int len = 0, lo = 0, key = 0, head0 = 0, id = 0;
      const int32_t* table = nullptr;
      const int last_id = (g.kv.num_slots - 1) / bs;
      auto piece = [&] {
        len = lens[w.b];
        lo = first_key(len);
        key = (lo & -run) + t * p.kt + lane * run;         // of the lane's run
        head0 = head_of_group();
        table = g.kv.block_table + (long long)(g.b0 + w.b) * g.kv.max_blocks;
      };
      auto look = [&] { id = lane < runs && key < len ? table[shift >= 0 ? key >> shift : key / bs] : -1; };
      if (have) {
        piece();
        look();
      }
      const uint32_t whole_word = p.kt >= 32 ? 0xffffffffu : (1u << p.kt) - 1;
      const unsigned whole_runs = 0xffffffffu >> (32 - runs);
      while (have) {
        const int key_ = key, len_ = len, lo_ = lo, head_ = head0, id_ = id, b_ = w.b;
        if (++t < w.t1) {
          key += p.kt;
        } else if ((have = w.next())) {
          t = w.t0;
          piece();
        }
        if (have) look();
        if (!(ok = room())) break;
        const uint32_t full = full0 + 8 * slot, dst = ring0 + slot * slot_bytes;
        // the run's first cache slot (-1: none, or a block id out of range: its keys are left out), and how
        // many slots from there are in the cache
        int sl = -1, in_run = 0;
        if (lane < runs && key_ < len_) {
          const uint32_t s = (uint32_t)id_ * bs + (shift >= 0 ? key_ & (bs - 1) : key_ % bs);   // < 2^32 up to last_id
          if (id_ >= 0 && id_ <= last_id && s < (uint32_t)g.kv.num_slots)
            sl = (int)s, in_run = min(run, g.kv.num_slots - sl);
          else
            report(g.ws, SPEC_ERR_DEVICE, g.b0 + b_, key_);
        }
        const int key0 = key_ - lane * run;
        const unsigned there = __ballot_sync(0xffffffffu, sl >= 0);
        if (key0 >= lo_ && key0 + p.kt <= len_ && __all_sync(0xffffffffu, lane >= runs || in_run == run) && there == whole_runs) {
          if (lane * 32 < p.kt) masks[slot * kMaskWords + lane] = whole_word;
        } else {
          // a block that the cache's end cuts: its keys past the end are left out as well
          if (sl >= 0 && max(key_ + in_run, lo_) < min(key_ + run, len_)) report(g.ws, SPEC_ERR_DEVICE, g.b0 + b_, key_ + in_run);
          for (int i = 0; i * 32 < p.kt; ++i) {
            const int j = i * 32 + lane, k = key0 + j;
            const int have_r = __shfl_sync(0xffffffffu, in_run, (j >> p.run_lg) & 31);
            const uint32_t word = __ballot_sync(0xffffffffu, j < p.kt && k >= lo_ && k < len_ && (j & (run - 1)) < have_r);
            if (lane == 0) masks[slot * kMaskWords + i] = word;
          }
        }
        __syncwarp();
        if (lane == 0) tc::mbar_expect_tx(full, (uint32_t)(__popc(there) * p.run_bytes));
        __syncwarp();
        const CUtensorMap* tm = v ? &g.tmv : &g.tmk;
        if (p.copies == 1) {
          if (sl >= 0) tma_run(dst + lane * p.run_bytes, tm, full, 0, sl, head_, policy);
        } else {
          for (int base = 0; base < copies; base += 32) {
            const int i = base + lane, r = quot(i, p.copies), c = i - r * p.copies;
            const int s = __shfl_sync(0xffffffffu, sl, r & 31);
            if (i < copies && s >= 0) tma_run(dst + r * p.run_bytes + c * p.chunk_stride, tm, full, c * (128 / M::kEs), s, head_, policy);
          }
        }
        passed();
      }
    } else {
      constexpr int kPer = kMaskWords;                     // keys of a tile a lane handles
      struct Tile {
        int b, key0, len, head0;
        int id[kPer];        // id[i] is the block of key 32 i + lane
      };
      auto fetch = [&](Tile& x) {
        x.b = w.b;
        x.len = lens[w.b];
        x.key0 = first_key(x.len) + t * p.kt;
        x.head0 = head_of_group();
        const int32_t* table = g.kv.block_table + (long long)(g.b0 + w.b) * g.kv.max_blocks;
#pragma unroll
        for (int i = 0; i < kPer; ++i)
          if (i * 32 < p.kt) {
            const int key = x.key0 + i * 32 + lane;
            x.id[i] = i * 32 + lane < p.kt && key < x.len ? table[shift >= 0 ? key >> shift : key / bs] : 0;
          }
      };
      Tile x;
      if (have) fetch(x);
      while (have) {
        Tile y = x;          // (not initialised: 167 us in place of 160 for 64 requests of 4000 keys)
        if (++t >= w.t1 && (have = w.next())) t = w.t0;
        if (have) fetch(y);
        if (!(ok = room())) break;
        const uint32_t full = full0 + 8 * slot, dst = ring0 + slot * slot_bytes;
        // cache slot of a key (-1: none, or a block id out of range: the key is left out)
        auto slot_of_key = [&](int key, int id) {
          if (key >= x.len) return -1;
          const long long s = (long long)id * bs + (shift >= 0 ? key & (bs - 1) : key % bs);
          if (id >= 0 && s < g.kv.num_slots) return (int)s;
          report(g.ws, SPEC_ERR_DEVICE, g.b0 + x.b, key);
          return -1;
        };
        int sl[kPer], n = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i)
          if (i * 32 < p.kt) {
            sl[i] = i * 32 + lane < p.kt ? slot_of_key(x.key0 + i * 32 + lane, x.id[i]) : -1;
            const uint32_t word = __ballot_sync(0xffffffffu, sl[i] >= 0);
            if (lane == 0 && !second) masks[slot * kMaskWords + i] = word;
            n += __popc(word);
          }
        if (lane == 0 && !second) tc::mbar_expect_tx(full, (uint32_t)(n * p.row));
        __syncwarp();
        const char* src = static_cast<const char*>(v ? g.kv.v : g.kv.k) + (long long)x.head0 * g.hd * M::kEs;
#pragma unroll
        for (int i = 0; i < kPer; ++i)
          if (i * 32 < p.kt && sl[i] >= 0 && (lane & 1) == second)
            bulk_row(dst + (i * 32 + lane) * p.key_stride, src + sl[i] * row_all, p.row, full, policy);
        passed();
        x = y;
      }
    }
    if (!ok) {
      // a wait ran out: let the copies in flight land before leaving
      if (lane == 0) report(g.ws, SPEC_ERR_TIMEOUT);
      int sl = slot, ph = phase;
      for (int i = 0; i < min(issued, (p.slots + 1) / 2); ++i) {
        if ((sl -= 2) < 0) sl += p.slots, ph ^= 1;
        tc::mbar_wait(full0 + 8 * sl, ph, const_cast<volatile int*>(flags), false);
      }
    }
    return;
  }

  // -------------------------------------------------------------- consumers
  if constexpr (M::kMoreRegs) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kConsumerRegs));
  float* wscr = mscr + warp * math_scratch<M>();
  int slot = 0, phase = 0;
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
      const int pair = (h + p.nh * (qi + p.qt * (kgrp & (half - 1)))) * M::VS + vs;     // < NW / 2
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
  auto group = [&] { return p.qs == 1 ? w.hg : w.hg / p.qs; };
  auto query0 = [&] { return ((w.hg - group() * p.qs) * p.qt + qi) * M::kQ; };
  auto queries = [&] { return kgrp < p.kg ? min(M::kQ, g.G - query0()) : 0; };     // <= 0: none for this warp
  auto head_of = [&] { return group() * p.nh + h; };
  auto load_q = [&] {
    const int n = queries();
    if (n > 0)
      math.load_q(g, static_cast<const T*>(g.q) + (g.b0 + w.b) * g.q_ld + (long long)head_of() * g.G * g.hd,
                  query0(), n, lane);
  };
  // a piece's queries are loaded while the one before it is merged and written
  bool more = w.next();
  if (more) load_q();
  while (more) {
    const int head = head_of(), q0 = query0(), nq = queries();
    const long long b = g.b0 + w.b;
    const int piece_b = w.b, hg = w.hg, nt = w.nt;
    const bool whole = w.t1 - w.t0 == w.nt;
    reset(s);
    math.scale_q(g, lane);
    auto wait = [&](int sl, int ph) { return tc::mbar_wait(full0 + 8 * sl, ph, const_cast<volatile int*>(flags)); };
    auto mask_of = [&](int sl) { return masks[sl * kMaskWords + (k0 >> 5)] >> (k0 & 31); };
    if constexpr (std::is_same_v<T, float>) {
      for (int t = w.t0; t < w.t1; ++t) {
        bool ok = wait(slot, phase);
        if (ok && nq > 0) math.scores(g, ring0 + slot * slot_bytes, mask_of(slot), lane, s, wscr);
        advance();
        ok = wait(slot, phase) && ok;
        if (ok && nq > 0) math.values(g, ring0 + slot * slot_bytes, lane, s, wscr);
        advance();
      }
    } else {
      // a tile's values together with the next one's scores
      bool ok = wait(slot, phase);
      uint32_t mask = mask_of(slot);
      if (ok && nq > 0) math.dots(g, ring0 + slot * slot_bytes, mask);
      advance();
      for (int t = w.t0; t < w.t1; ++t) {
        if (ok && nq > 0) math.weights(g, mask, lane, s);
        ok = wait(slot, phase) && ok;
        const uint32_t v = ring0 + slot * slot_bytes;
        if (t + 1 == w.t1) {
          if (ok && nq > 0) math.values(g, v, lane, s, vs);
        } else {
          const int ks = slot + 1 == p.slots ? 0 : slot + 1;
          ok = wait(ks, ks == 0 ? phase ^ 1 : phase) && ok;
          mask = mask_of(ks);
          const uint32_t k = ring0 + ks * slot_bytes;
          if (ok && nq > 0) {
            if (math.can_run_both(g, mask)) {
              math.both(g, k, v, s, vs);
            } else {
              math.dots(g, k, mask);
              math.values(g, v, lane, s, vs);
            }
          }
          advance();
        }
        advance();
      }
    }
    math.finish(s);
    more = w.next();
    if (more) load_q();
    merge_groups();
    if (!whole) {
      // one of several pieces: leave it, and join them all if it is the last to come
      int c0;
      const int n = owners(piece_b, hg, nt, &c0);
      auto entry = [&](int i) {                 // piece i: a CTA's first piece may have begun before it, its last may go on
        return g.part + (((long long)(c0 + i) * 2 + (i == 0)) * NW + (h + p.nh * qi) * M::VS + vs) * entry_floats<M>() + lane * 4;
      };
      auto leave = [&](int i) {                 // this warp's state as piece i
        if (kgrp != 0) return;
        float* x = entry(i);
#pragma unroll
        for (int r = 0; r < S::NR; r += 4)
          __stcg(reinterpret_cast<float4*>(x + r * 32), make_float4(s.o[r], s.o[r + 1], s.o[r + 2], s.o[r + 3]));
        float ml[2 * S::NM];
#pragma unroll
        for (int k = 0; k < S::NM; ++k) ml[k] = s.m[k], ml[S::NM + k] = s.l[k];
#pragma unroll
        for (int r = 0; r < 2 * S::NM; r += 4)
          __stcg(reinterpret_cast<float4*>(x + (S::NR + r) * 32), make_float4(ml[r], ml[r + 1], ml[r + 2], ml[r + 3]));
      };
      auto last_of = [&](int* ctr, int count) { // whether this CTA is the last of `count` to come here
        sync();                                 // its pieces are written; the atomic releases them and acquires the others'
        if (tid == 0) {
          int before;
          asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;" : "=r"(before) : "l"(ctr) : "memory");
          if (before == count - 1) *ctr = 0;
          flags[1] = before == count - 1;
        }
        sync();
        return flags[1] != 0;
      };
      auto collect = [&](int i, int end, int step) {   // pieces i, i + step .. joined in order, key groups taking turns
        reset(s);
        for (i += kgrp * step; i < end; i += p.kg * step) {
          const float* x = entry(i);
          float4 f;
          join<M>(s, [&](int r) {
            if (r >= S::NR) return __ldcg(x + (r & ~3) * 32 + (r & 3));
            if (r % 4 == 0) f = __ldcg(reinterpret_cast<const float4*>(x + r * 32));
            return r % 4 == 0 ? f.x : r % 4 == 1 ? f.y : r % 4 == 2 ? f.z : f.w;
          });
        }
        merge_groups();
      };
      const int i = cta - c0;
      leave(i);
      // many pieces are joined in two levels, about sqrt(n) at a time: one CTA reads a piece in ~0.5 us
      int step = 1;
      if (n > kFlat) {
        while (step * step < n) ++step;
        const int first = i / step * step, end = min(first + step, n);
        if (!last_of(&g.group_counters[2 * (c0 + first) + (first == 0)], end - first)) continue;
        collect(first, end, 1);
        leave(first);
      }
      if (!last_of(&g.counters[b * p.hgq + hg], (n + step - 1) / step)) continue;
      collect(0, n, step);
    }
    if (kgrp == 0 && nq > 0) {
      T* out = static_cast<T*>(g.out) + b * g.out_ld + ((long long)head * g.G + q0) * g.hd;
      float inv[S::NM];
#pragma unroll
      for (int i = 0; i < S::NM; ++i) {
        inv[i] = s.l[i] == 0.f ? 0.f : g.v_scale / s.l[i];
        const int q = M::stat_query(i, lane);
        if (g.lse && vs == 0 && M::stat_owner(lane) && q < nq)
          g.lse[b * g.nq + (long long)head * g.G + q0 + q] = s.l[i] == 0.f ? -INFINITY : (s.m[i] + log2f(s.l[i])) * kLn2;
      }
      M::write(s, inv, out, g.hd, nq, lane, vs);
    }
  }
  if (tid == 0 && flags[0]) report(g.ws, SPEC_ERR_TIMEOUT);
}

// What the planner needs to know of an instantiation, and its launch.
struct Kernel {
  void (*fn)(Args);
  int warps, vs, sub, kq, es, hd;
  size_t (*fixed)(int);
  bool (*fits)();      // launched with the registers that its warps share out
};
template <typename M> Kernel kernel_of() {
  static_assert(M::kWarps * entry_floats<M>() <= 8 * 72 * 32, "a CTA's piece fits the workspace");
  return {paged_attention_kernel<M>, M::kWarps, M::VS, M::kSub, M::kQ, M::kEs, M::kHd,
          [](int B) { return fixed_smem<M>(B); },
          [] {
            static const bool ok = [] {      // a share above the launch's registers would be waited for without end
              cudaFuncAttributes a;
              return !M::kMoreRegs || (cudaFuncGetAttributes(&a, paged_attention_kernel<M>) == cudaSuccess &&
                                       M::kWarps == 8 && a.numRegs == kLaunchRegs);
            }();
            return ok;
          }};
}

Kernel kernel_bf16(bool e4m3, int hd, int G);
Kernel kernel_f16(bool e4m3, int hd, int G);
Kernel kernel_f32(int hd, int G);

// 8 queries a warp, 16 where a kv head has more than 8: keys are then read from shared memory once for
// all of them (32 requests of 4000 keys, 8 heads of 256, 128 queries, by 8 / by 16: 196 / 168 us, in 8
// bits 158 / 139; 192 components 191 / 127)
template <typename T, bool F8> Kernel pick16(int hd, int G) {
  if (hd <= 64) return G <= 8 ? kernel_of<MmaMath<T, F8, 64, 1>>() : kernel_of<MmaMath<T, F8, 64, 2>>();
  if (hd <= 128) return G <= 8 ? kernel_of<MmaMath<T, F8, 128, 1>>() : kernel_of<MmaMath<T, F8, 128, 2>>();
  if (hd <= 192) return G <= 8 ? kernel_of<MmaMath<T, F8, 192, 1>>() : kernel_of<MmaMath<T, F8, 192, 2>>();
  return G <= 8 ? kernel_of<MmaMath<T, F8, 256, 1>>() : kernel_of<MmaMath<T, F8, 256, 2>>();
}

}  // namespace pa
}  // namespace spec
