// Attention of a chunk of new tokens on tcgen05: the kernel.  The translation
// units chunk_attn_<type>.cu instantiate it.
//
// A CTA has 128 or 256 packed rows (chunk_attn.cuh) and streams its keys in tiles.
// Per tile and 128 rows one job: S = Q K^T into TMEM, the softmax warpgroup's
// weights back into TMEM over S, O += P V with P from TMEM.  A softmax thread owns
// a row: no shuffles, its maximum and sum in registers.
//   warps 0-3, 4-7   two softmax warpgroups
//   warps 8-11       K/V and Q into shared memory
//   warp 12          issues the MMAs
//   warp 13          asks for 8-bit K/V, which warps 8-11 widen
// While one warpgroup works on its scores, the tensor cores do the other's products.
//
// Bound by a job's chain: scores ready -> softmax (1400 cycles: a row's 128 exponentials are
// 512 of the special function units', two warps share one) -> products and the next scores
// (1024 of MMA, 1400 with their waits).  128 rows x 128 keys x 128 components: 3060 cycles for
// two jobs, of which the tensor pipe works 2048.  500 rows of 32 heads over 131071 keys 0.89-0.94 ms
// (1.14-1.20 PFLOP/s, 59-62 % of a measured cuBLAS bf16 product; the SM clock stays near
// 1.5 GHz under this load, as it does for cuBLAS), 16 chunks of 100-2048 tokens 0.92-0.95 ms from one GPU to another.
// Spilled, bytes a thread: kTwoQ 92, kOneQ 292, kWide 48 over 16-bit caches, kTwoQ 362-386, kWide 132-156 over 8-bit ones.
#pragma once
#include <type_traits>

#include "chunk_attn.cuh"
#include "tc_core.cuh"

namespace spec {
namespace ca {

// kTwoQ: 256 rows, a warpgroup for each half, every K/V tile used twice (shared memory gives the tensor cores
// 128 bytes a cycle: scores of 128 x 128 take all of it).  kOneQ: 128 rows, the warpgroups take turns at the
// tiles with an accumulator each, joined at the end.  kWide: head sizes above 128, whose accumulator leaves no
// room for a second one: 128 rows, tiles of 64 keys, one warpgroup (256 components: 800 TFLOP/s).
enum Mode { kTwoQ = 0, kOneQ = 1, kWide = 2 };

constexpr int kTcThreads = 512;
// 512 threads are launched with 128 registers each and share them out: 2 x 128 x 192 + 128 x 72 + 128 x 56
constexpr int kLaunchRegs = 128, kSoftmaxRegs = 192, kLoaderRegs = 72, kMmaRegs = 56;
static_assert(2 * kSoftmaxRegs + kLoaderRegs + kMmaRegs <= 4 * kLaunchRegs, "");
// dynamic shared memory of a launch, at most; the attribute is always this: another thread may be launching the same kernel
// with another head size
constexpr int kTcSmem = 208 * 1024;
constexpr int kMaxStages = 8, kTileBits = 8;
constexpr int kRawStages = 2;            // 8-bit tiles under way, before they are widened
// An item's masks are used again 8 items later: the streams are at most two items apart (one's next-but-one Q waits for the
// other's scores of the item before it) and the loader one ahead of the first, so that stream clears those of four items ago.
constexpr int kItems = 8;
constexpr int kHoldWord = 16;            // of the workspace's header, in words

template <int MODE> struct Shape {
  static constexpr int BM = MODE == kTwoQ ? 256 : 128, KT = MODE == kWide ? 64 : 128;
  static constexpr int NQ = BM / 128, EDGES = BM / KT + 2;
  static constexpr int O0 = 256, O1 = 384;             // TMEM columns; S buffers at 0 and KT
};

// dynamic shared memory: Q tiles, the ring of K/V stages, raw 8-bit tiles
struct Layout {
  int chunks;        // 64-component (128-byte) chunks of a head
  int q_bytes, stage_bytes, stages, raw_bytes;
  int smem;
  int runs;          // keys come in runs of 16 slots of a block, by tensor copies
  int q_boxes;       // rows of Q come in boxes of 128 / G tokens
};
template <int MODE> static inline Layout layout(int hd, bool f8) {
  using S = Shape<MODE>;
  Layout l;
  l.chunks = (hd + 63) / 64;
  l.q_bytes = S::BM * 128 * l.chunks;
  l.stage_bytes = S::KT * 128 * l.chunks;
  l.raw_bytes = f8 ? S::KT * hd : 0;
  const int room = kTcSmem - 1024 - l.q_bytes - kRawStages * l.raw_bytes;
  l.stages = room / l.stage_bytes < kMaxStages ? room / l.stage_bytes : kMaxStages;
  l.smem = 1024 + l.q_bytes + l.stages * l.stage_bytes + kRawStages * l.raw_bytes;
  return l;
}

struct TcArgs {
  CUtensorMap tmk, tmv;        // runs: [slots][nkv][hd] views of the cache, boxes of 16 slots x 64 components
  CUtensorMap tmq;             // q_boxes: [n_rows][nq][hd] of q, boxes of 128 packed rows x 64 components
  Args g;
  Layout l;
};

SPEC_DEV void cp16(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
SPEC_DEV void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> SPEC_DEV void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
SPEC_DEV void proxy_fence() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
SPEC_DEV uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
SPEC_DEV void sts128(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
template <int R> SPEC_DEV void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R)); }
template <int R> SPEC_DEV void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R)); }

// Whether a phase is over, at once (mbarrier.try_wait may hold the warp for a while).  The answer is the warp's: what follows
// is done by all lanes together.
SPEC_DEV bool test(uint64_t& bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(tc::su32(&bar)), "r"(parity)
      : "memory");
  return __all_sync(0xffffffffu, ok != 0);
}
// Bounded wait, in few instructions: the roles' loops share the SM's instruction cache.
SPEC_DEV bool wait_lane(uint64_t& bar, uint32_t parity, volatile int* abort) {
  const uint32_t a = tc::su32(&bar);
  if (tc::mbar_try(a, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
#pragma unroll 1
  while (!tc::mbar_try(a, parity)) {
    if (*abort) return false;
    if (globaltimer_ns() - t0 > tc::kWaitNs) {
      *abort = 1;
      return false;
    }
  }
  return true;
}
// The same for a whole warp, whose lanes get one answer: a lane that gave up alone would leave the others waiting for it at
// their next exchange.
SPEC_DEV bool wait_for(uint64_t& bar, uint32_t parity, volatile int* abort) {
  return __all_sync(0xffffffffu, wait_lane(bar, parity, abort));
}

SPEC_DEV void copy_run(uint32_t dst, const CUtensorMap* tm, uint32_t mbar, int x, int head, int slot, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tm)), "r"(x), "r"(head), "r"(slot), "r"(mbar), "l"(policy)
      : "memory");
}

// D[tmem] (+)= A[smem] * B[smem]^T; descriptors by their low halves, the high ones do not change
template <bool ACC> SPEC_DEV void mma_ss(uint32_t d, uint32_t a, uint32_t a_hi, uint32_t b, uint32_t b_hi, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .b64 x, y;\n\t.reg .pred p;\n\t"
      "mov.b64 x, {%1, %2};\n\tmov.b64 y, {%3, %4};\n\tsetp.ne.u32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %5, p;\n\t}" ::"r"(d),
      "r"(a), "r"(a_hi), "r"(b), "r"(b_hi), "r"(idesc), "n"(ACC ? 1 : 0)
      : "memory");
}
// D[tmem] (+)= A[tmem] * B[smem]
SPEC_DEV void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t b_hi, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .b64 y;\n\t.reg .pred p;\n\t"
      "mov.b64 y, {%2, %3};\n\tsetp.ne.u32 p, %5, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %4, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(b_hi), "r"(idesc), "r"(accumulate)
      : "memory");
}
SPEC_DEV void tmem_ld32(uint32_t a, uint32_t* u) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,"
      "%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[8]),
        "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15]), "=r"(u[16]), "=r"(u[17]),
        "=r"(u[18]), "=r"(u[19]), "=r"(u[20]), "=r"(u[21]), "=r"(u[22]), "=r"(u[23]), "=r"(u[24]), "=r"(u[25]),
        "=r"(u[26]), "=r"(u[27]), "=r"(u[28]), "=r"(u[29]), "=r"(u[30]), "=r"(u[31])
      : "r"(a));
}
SPEC_DEV void tmem_st16(uint32_t a, const uint32_t* u) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(a),
      "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]), "r"(u[8]), "r"(u[9]),
      "r"(u[10]), "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15])
      : "memory");
}
SPEC_DEV void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Values as an MN-major operand [keys][components]: 128-byte rows of 64 components, 8 keys a swizzle atom (1024 bytes: the
// stride along K), 64-component chunks lbo bytes apart.
SPEC_DEV uint64_t desc_values(uint32_t saddr, uint32_t lbo) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(lbo >> 4) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}
// D fp32; A and B of the same 16-bit type; b_mn: B's components are contiguous
template <typename T> SPEC_DEV uint32_t idesc_of(int N, bool b_mn) {
  const uint32_t f = std::is_same_v<T, __half> ? 0u : 1u;
  return (1u << 4) | (f << 7) | (f << 10) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | (8u << 24);
}

// two floats in an instruction
struct Two {
  unsigned long long x;
  SPEC_DEV Two() {}
  SPEC_DEV Two(float a, float b) { asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a), "f"(b)); }
  SPEC_DEV void get(float& a, float& b) const { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x)); }
};
SPEC_DEV Two add2(Two a, Two b) {
  Two d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d.x) : "l"(a.x), "l"(b.x));
  return d;
}
SPEC_DEV Two fma2(Two a, Two b, Two c) {
  Two d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d.x) : "l"(a.x), "l"(b.x), "l"(c.x));
  return d;
}
SPEC_DEV float max3(float a, uint32_t b, uint32_t c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(__uint_as_float(b)), "f"(__uint_as_float(c)));
  return d;
}

template <typename T> SPEC_DEV uint32_t pack2(float lo, float hi) {
  if constexpr (std::is_same_v<T, __half>) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}
// halves of x that are not finite, as 0xffff
template <typename T> SPEC_DEV uint32_t odd_halves(uint32_t x) {
  constexpr uint32_t e = std::is_same_v<T, __half> ? 0x7c00u : 0x7f80u;
  return ((x & e) == e ? 0xffffu : 0u) | ((x >> 16 & e) == e ? 0xffff0000u : 0u);
}
// four 8-bit values as four of T; exact
template <typename T> SPEC_DEV uint2 widen4(uint32_t x) {
  const __half2 a = __half2_raw(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(x & 0xffffu), __NV_E4M3));
  const __half2 b = __half2_raw(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(x >> 16), __NV_E4M3));
  if constexpr (std::is_same_v<T, __half>) {
    return make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  } else {
    const float2 x0 = __half22float2(a), x1 = __half22float2(b);
    return make_uint2(pack2<T>(x0.x, x0.y), pack2<T>(x1.x, x1.y));
  }
}

struct TcSmem {
  Plan plan;
  uint64_t full[kMaxStages], empty[kMaxStages], q_full, q_empty, drain, landed[4], raw_full[kRawStages], raw_empty[kRawStages], s_full[2], p_full[2][2], o_done[2], o_free[2], group[2];
  alignas(16) uint32_t bits[kTileBits][4];   // keys of a tile that are there
  uint32_t poison[kItems][2 * 6][4];   // keys of an item's edge tiles whose value is not finite
  int poisoned[kItems];
  alignas(16) uint32_t way_there[kRawStages][4];   // an 8-bit stage: its keys, and its info
  int way_info[kRawStages];
  int info[4][kTileBits];              // loader warps: what a stage under way needs when it has come
  float2 ml[2][128];
  int last[2];
  uint32_t tmem;
  int abort;
  int hold;                            // CTA + 1 that gets no keys (the workspace header's test hook)
};

// ---------------------------------------------------------------- loader
// Keys come in runs of 16 slots by tensor copies where the block size allows: boxes of 16 slots x 128 bytes, no thread's
// time.  Otherwise four warps copy a tile's rows in 16-byte pieces (cp.async): any block size, rows of any number of
// pieces, and 512 bytes an instruction; an SM takes about 27 bytes a cycle that way (8 chunks of 512-1024 tokens, blocks of
// 16 / 24 / 1 slots: 280 / 386 / 387 us).  U: pieces of a cache row, where that is 4, 8, 16 or 32 (a lane's piece and its step from row to row do
// not change then), or 0.
template <int N> struct Units {
  const int n, inv;                    // 2^16 / n rounded up: quotients of numbers below 2^11 are exact
  SPEC_DEV explicit Units(int n_) : n(N ? N : n_), inv(N ? 0 : (65536 + n_ - 1) / n_) {}
  SPEC_DEV int row(int i) const { return N ? i / (N ? N : 1) : (i * inv) >> 16; }
};

template <typename T, bool F8, int MODE> struct Loader {
  using S = Shape<MODE>;
  static constexpr int KT = S::KT, RW = KT / 4;        // key rows of a warp
  static constexpr int ES = F8 ? 1 : 2;
  static constexpr int kLag = 1;       // stages under way behind the newest

  // where 16-byte piece u of a row of 16-bit components is in a tile of `rows` rows
  static SPEC_DEV uint32_t place(int row, int u, int rows) {
    return (uint32_t)((u >> 3) * rows * 128 + row * 128 + (((u ^ row) & 7) << 4));
  }
  // A weight of 0 times a value that is not finite is a NaN in rows that do not attend to the key: in edge tiles such
  // components are zeros, and the rows that do attend to the key get theirs at the end.
  static SPEC_DEV void mark(TcSmem& sm, int info, int key) {
    atomicOr(&sm.poison[info >> 8][info & 255][key >> 5], 1u << (key & 31));
    sm.poisoned[info >> 8] = 1;
  }
  // rows r0 .. of a warp, whose slots (-1: none) its lanes hold
  template <int U> static SPEC_DEV void copy_rows(const char* base, uint32_t stride, int slot, uint32_t to, int r0, int lane,
                                                  int units) {
    const Units<U> un(units);
    const int n = RW * un.n;
    constexpr int B = U ? 8 : 2;                       // slots looked up together
    static_assert(!U || RW * U % (32 * B) == 0 || RW * U < 32 * B, "");
    const int i0 = lane, u0 = U ? lane % (U ? U : 1) : 0;
#pragma unroll 1
    for (int j = 0; j < n; j += 32 * B) {              // (every lane takes part in the shuffles)
      int s[B];
#pragma unroll
      for (int q = 0; q < B; ++q) s[q] = __shfl_sync(0xffffffffu, slot, un.row(i0 + j + 32 * q) & 31);
#pragma unroll
      for (int q = 0; q < B; ++q) {
        const int i = i0 + j + 32 * q, row = un.row(i), u = U ? u0 : i - row * un.n;
        const char* src = base + (uint64_t)(uint32_t)max(s[q], 0) * stride + u * 16;
        if (i < n) cp16(to + (F8 ? (uint32_t)((r0 + row) * un.n + u) * 16 : place(r0 + row, u, KT)), src, s[q] >= 0);
      }
    }
  }
  // 8-bit rows -> 16-bit ones in the ring, four pieces of a lane at a time (one warp's latencies are what this takes)
  template <int U> static SPEC_DEV void widen_rows(uint32_t from, uint32_t to, int r0, int lane, int units) {
    const Units<U> un(units);
    const int n = RW * un.n;
    constexpr int B = U ? U : 2;                       // U: RW U pieces are B 32 of them, or half of that
#pragma unroll 1
    for (int j = lane; j < n; j += 32 * B) {
      uint4 x[B];
#pragma unroll
      for (int q = 0; q < B; ++q)
        if (j + 32 * q < n) x[q] = lds128(from + (uint32_t)(r0 * un.n + j + 32 * q) * 16);
#pragma unroll
      for (int q = 0; q < B; ++q) {
        const int i = j + 32 * q, row = un.row(i), u = U ? lane % (U ? U : 1) : i - row * un.n;
        if (i >= n) break;
        const uint2 a = widen4<T>(x[q].x), b = widen4<T>(x[q].y), c = widen4<T>(x[q].z), d = widen4<T>(x[q].w);
        sts128(to + place(r0 + row, 2 * u, KT), make_uint4(a.x, a.y, b.x, b.y));
        sts128(to + place(r0 + row, 2 * u + 1, KT), make_uint4(c.x, c.y, d.x, d.y));
      }
    }
  }
  // Rows r0 .. of a tile in an edge (info), of which `there` are keys (others hold whatever the cache has there).  Looked
  // over first: the largest magnitude of the lane's pieces, NaN if there is one.
  static SPEC_DEV void clean_rows(TcSmem& sm, uint32_t at, int r0, int lane, int units, int info, uint32_t there) {
    using T2 = std::conditional_t<std::is_same_v<T, __half>, __half2, __nv_bfloat162>;
    const Units<0> un(units);
    const uint32_t zero = 0;
    T2 top = *reinterpret_cast<const T2*>(&zero);
#pragma unroll 8
    for (int i = lane; i < RW * units; i += 32) {
      const int row = un.row(i), u = i - row * units;
      const uint4 v = lds128(at + place(r0 + row, u, KT));
      const T2* x = reinterpret_cast<const T2*>(&v);
      top = __hmax2_nan(top, __hmax2_nan(__hmax2_nan(__habs2(x[0]), __habs2(x[1])), __hmax2_nan(__habs2(x[2]), __habs2(x[3]))));
    }
    if (!__any_sync(0xffffffffu, odd_halves<T>(*reinterpret_cast<const uint32_t*>(&top)) != 0)) return;
#pragma unroll 1
    for (int i = lane; i < RW * units; i += 32) {
      const int row = un.row(i), u = i - row * units;
      const uint32_t to = at + place(r0 + row, u, KT);
      uint4 v = lds128(to);
      const uint32_t a = odd_halves<T>(v.x), b = odd_halves<T>(v.y), c = odd_halves<T>(v.z), d = odd_halves<T>(v.w);
      if (a | b | c | d) {
        v.x &= ~a, v.y &= ~b, v.z &= ~c, v.w &= ~d;
        sts128(to, v);
        if (there >> row & 1u) mark(sm, info, r0 + row);
      }
    }
  }
  static SPEC_DEV void zero_rows(uint32_t at, int r0, int lane, int units, uint32_t which) {
    const Units<0> un(units);
#pragma unroll 1
    for (int i = lane; i < RW * units; i += 32) {
      const int row = un.row(i), u = i - row * units;
      if (which >> row & 1u) sts128(at + place(r0 + row, u, KT), make_uint4(0, 0, 0, 0));
    }
  }
  // Q by tensor copies: 128 packed rows are 128 / G tokens of G heads, in this order in a box (rows of other requests and
  // zeros past the last token among them).  Every warp arrives at q_full.
  static SPEC_DEV void copy_q(const TcArgs& a, TcSmem& sm, const Item& it, uint32_t q0, int warp, int lane) {
    const uint32_t bar = tc::su32(&sm.q_full);
    if (lane == 0) {
      if (warp == 0) {
        tc::mbar_expect_tx(bar, S::NQ * a.l.chunks * 16384);
        const int token = it.row0 + it.r0 / a.g.G, per = 128 / a.g.G;
        const uint64_t policy = tc::policy_evict_first();
#pragma unroll 1
        for (int i = 0; i < S::NQ * a.l.chunks; ++i) {
          const int t = i / a.l.chunks, c = i - t * a.l.chunks;
          copy_run(q0 + (uint32_t)i * 16384, &a.tmq, bar, 64 * c, it.h * a.g.G, token + t * per, policy);
        }
      } else {
        tc::mbar_arrive(bar);
      }
    }
    __syncwarp();
  }
  static SPEC_DEV void load_q(const Args& g, const Item& it, uint32_t q0, int chunks, int warp, int lane) {
    constexpr int RQ = S::BM / 4;                      // rows of a warp
    const Units<0> un(g.hd / 8);
    const T* q = static_cast<const T*>(g.q);
    for (int r0 = 0; r0 < RQ; r0 += 32) {
      const int r = warp * RQ + r0 + lane;
      long long off = -1;
      if (r < it.rows) {
        const int tok = (it.r0 + r) / g.G, head = it.h * g.G + (it.r0 + r) - tok * g.G;
        off = (it.row0 + tok) * g.q_ld + (long long)head * g.hd;
      }
#pragma unroll 2
      for (int j = 0; j < 32 * un.n; j += 32) {
        const int i = j + lane, row = un.row(i), u = i - row * un.n;
        const long long o = __shfl_sync(0xffffffffu, off, row);
        const int m = warp * RQ + r0 + row;
        cp16(q0 + (uint32_t)((m >> 7) * chunks * 16384) + place(m & 127, u, 128), q + max(o, 0ll) + 8 * u, o >= 0);
      }
    }
  }

  // Q of the next item, once the MMAs have read the last one's.  Every loader warp.
  static SPEC_DEV bool next_q(const TcArgs& a, TcSmem& sm, const Item& it, uint32_t q0, int warp, int lane, int items,
                              uint32_t& q_phase) {
    if (items > 0) {
      if (!wait_for(sm.q_empty, q_phase, &sm.abort)) return false;
      q_phase ^= 1u;
    }
    if (a.l.q_boxes) {
      copy_q(a, sm, it, q0, warp, lane);
    } else {
      load_q(a.g, it, q0, a.l.chunks, warp, lane);
      cp_commit();
      cp_wait<0>();
      proxy_fence();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(tc::su32(&sm.q_full));
    }
    return true;
  }
  // Gives up: Q's copies land first (or the limit passes).
  static SPEC_DEV void settle_q(const TcArgs& a, TcSmem& sm, int warp, int items) {
    if (a.l.q_boxes && warp == 0 && items > 0) tc::mbar_wait(tc::su32(&sm.q_full), (uint32_t)(items - 1) & 1u, &sm.abort, false);
  }

  // Where the keys of consecutive tiles are: the lane's key of a tile, its entry of the block table asked for a tile ahead.
  struct Keys {
    const Args& g;
    const int32_t* table;
    int b, lo, hi, key, block, in_block, e;
    bool mine;
    SPEC_DEV explicit Keys(const Args& g_) : g(g_) {}
    SPEC_DEV void begin(const Item& it, int first, bool mine_) {
      table = g.kv.block_table + (long long)(g.b0 + it.b) * g.kv.max_blocks;
      b = g.b0 + it.b, lo = it.lo, hi = it.hi, key = first, mine = mine_;
      block = key / g.kv.block_size, in_block = key % g.kv.block_size;
      ask();
    }
    SPEC_DEV void ask() { e = mine && key >= lo && key < hi ? __ldg(table + block) : -1; }
    // the key's slot, -1 for none; then the next tile's key
    SPEC_DEV int next(bool more, int step_b, int step_i, int kt) {
      int slot = -1;
      if (mine && key >= lo && key < hi) {
        const long long s = (long long)e * g.kv.block_size + in_block;
        if (s >= 0 && s < g.kv.num_slots) slot = (int)s;
        else report(g.ws, SPEC_ERR_DEVICE, b, key);
      }
      key += kt, block += step_b, in_block += step_i;
      if (in_block >= g.kv.block_size) in_block -= g.kv.block_size, ++block;
      if (more) ask();
      return slot;
    }
  };

  // 16-bit keys in runs of 16 slots: tensor copies, a lane a run and 64 components, that report to the MMA warp by themselves;
  // the values of edge tiles come by way of this warp.
  static SPEC_DEV void run_tensor(const TcArgs& a, TcSmem& sm, uint32_t q0, int warp, int lane) {
    const Args& g = a.g;
    const int chunks = a.l.chunks, stages = a.l.stages, units = g.hd / 8, r0 = warp * RW;
    const uint32_t stage_bytes = a.l.stage_bytes, ring0 = q0 + a.l.q_bytes;
    volatile int* abort = &sm.abort;
    Walk<S::BM, KT> walk(g, sm.plan);
    Item it;
    int tiles = 0, items = 0, stage = 0, filled = 0;
    uint32_t phase = 0, q_phase = 0, l_phase = 0;
    // this lane's copy: run and chunk
    const int run = lane / chunks, chunk = lane - run * chunks;
    const uint32_t lane_to = (uint32_t)(chunk * KT * 128 + (r0 + run * 16) * 128);
    const uint32_t run_mask = run < RW / 16 ? 0xffffu << (run * 16) : 0u;
    const uint64_t policy = tc::policy_evict_last();
    const int step_b = KT / g.kv.block_size, step_i = KT % g.kv.block_size;
    Keys at_key(g);
    bool ok = true;
    while (ok && walk.next(it)) {
      const Edges<KT> edges(g, it);
      at_key.begin(it, (it.tile0 + it.k0) * KT + r0 + lane, lane < RW);
      for (int k = it.k0; ok && k < it.k1; ++k, ++tiles) {
        const int slot = at_key.next(k + 1 < it.k1, step_b, step_i, KT);
        const uint32_t there = __ballot_sync(0xffffffffu, slot >= 0);
        if (lane == 0) {
          if constexpr (RW == 32) sm.bits[tiles % kTileBits][warp] = there;
          else reinterpret_cast<uint16_t*>(sm.bits[tiles % kTileBits])[warp] = (uint16_t)there;
        }
        // the slot that the lane's run begins with
        const uint32_t keys = there & run_mask;
        const int from = keys ? __ffs(keys) - 1 : 0;
        const int first = __shfl_sync(0xffffffffu, slot, from) - (from & 15);
        const uint32_t bytes = ((there & 0xffffu ? 1u : 0u) + (RW == 32 && there >> 16 ? 1u : 0u)) * chunks * 2048u;
        const uint32_t absent = (there & 0xffffu ? 0u : 0xffffu) | (RW == 32 && !(there >> 16) ? 0xffff0000u : 0u);
        const int tile = it.tile0 + k;
        const bool edge = edges.has(tile);
#pragma unroll 1
        for (int value = 0; value < 2; ++value) {
          if (!wait_for(sm.empty[stage], phase ^ 1u, abort)) {
            ok = false;
            break;
          }
          const uint32_t at = ring0 + (uint32_t)stage * stage_bytes;
          const bool by_way = value && edge;
          if (value && absent) {                       // nothing is copied there: weights of 0 must meet numbers
            zero_rows(at, r0, lane, units, absent);
            proxy_fence();
          }
          uint64_t& bar = by_way ? sm.landed[warp] : sm.full[stage];
          __syncwarp();
          if (lane == 0) tc::mbar_expect_tx(tc::su32(&bar), bytes);
          __syncwarp();
          if (keys) copy_run(at + lane_to, value ? &a.tmv : &a.tmk, tc::su32(&bar), 64 * chunk, it.h, first, policy);
          if (by_way) {
            __syncwarp();
            if (!wait_for(bar, l_phase, abort)) {
              ok = false;
              break;
            }
            l_phase ^= 1u;
            clean_rows(sm, at, r0, lane, units, (items % kItems) << 8 | edges.template slot<S::EDGES>(tile), there);
            proxy_fence();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(tc::su32(&sm.full[stage]));
          }
          filled = min(filled + 1, stages);
          if (++stage == stages) stage = 0, phase ^= 1u;
        }
        // Q, once the first keys are on their way
        if (k == it.k0 && ok) ok = next_q(a, sm, it, q0, warp, lane, items, q_phase);
      }
      ++items;
    }
    cp_wait<0>();
    if (!ok || sm.abort) {
      // gives up: the copies under way land first (or the limit passes)
      settle_q(a, sm, warp, items);
      for (int i = 0; i < filled; ++i) {
        if (--stage < 0) stage = stages - 1, phase ^= 1u;
        tc::mbar_wait(tc::su32(&sm.full[stage]), phase, abort, false);
      }
    }
  }

  // 8-bit keys in runs of 16 slots: one warp asks for them, as they lie, in raw stages ...
  static SPEC_DEV void ask_raw(const TcArgs& a, TcSmem& sm, uint32_t q0, int lane) {
    constexpr int N = KT / 32, RUNS = KT / 16;
    const Args& g = a.g;
    const uint32_t raw0 = q0 + a.l.q_bytes + (uint32_t)a.l.stages * a.l.stage_bytes;
    volatile int* abort = &sm.abort;
    Walk<S::BM, KT> walk(g, sm.plan);
    Item it;
    int tiles = 0, items = 0, raw = 0, asked = 0;
    uint32_t phase = 0;
    const uint64_t policy = tc::policy_evict_last();
    const int step_b = KT / g.kv.block_size, step_i = KT % g.kv.block_size;
    Keys at_key[4] = {Keys(g), Keys(g), Keys(g), Keys(g)};         // (N of them)
    bool ok = true;
    while (ok && walk.next(it)) {
      const Edges<KT> edges(g, it);
#pragma unroll
      for (int i = 0; i < N; ++i) at_key[i].begin(it, (it.tile0 + it.k0) * KT + 32 * i + lane, true);
      for (int k = it.k0; ok && k < it.k1; ++k, ++tiles) {
        uint32_t there[N], runs = 0, keys = 0;
        int first = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const int slot = at_key[i].next(k + 1 < it.k1, step_b, step_i, KT);
          there[i] = __ballot_sync(0xffffffffu, slot >= 0);
          // lane r: run r
          const uint32_t mine = lane >> 1 == i ? there[i] & 0xffffu << (16 * (lane & 1)) : 0u;
          const int from = mine ? __ffs(mine) - 1 : 0, s = __shfl_sync(0xffffffffu, slot, from);
          if (mine) first = s - (from & 15), keys = mine;
          runs += (there[i] & 0xffffu ? 1u : 0u) + (there[i] >> 16 ? 1u : 0u);
        }
        const int tile = it.tile0 + k;
        const int info = edges.has(tile) ? (items % kItems) << 8 | edges.template slot<S::EDGES>(tile) : -1;
#pragma unroll 1
        for (int value = 0; value < 2; ++value) {
          if (!wait_for(sm.raw_empty[raw], phase ^ 1u, abort)) {
            ok = false;
            break;
          }
          if (lane == 0) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
              sm.way_there[raw][i] = there[i];
              if (!value) sm.bits[tiles % kTileBits][i] = there[i];
            }
            sm.way_info[raw] = value ? info : -1;
            tc::mbar_expect_tx(tc::su32(&sm.raw_full[raw]), runs * 16u * g.hd);
          }
          __syncwarp();
          if (lane < RUNS && keys)
            copy_run(raw0 + (uint32_t)raw * a.l.raw_bytes + (uint32_t)(lane * 16 * g.hd), value ? &a.tmv : &a.tmk,
                     tc::su32(&sm.raw_full[raw]), 0, it.h, first, policy);
          __syncwarp();
          asked = min(asked + 1, kRawStages);
          if (++raw == kRawStages) raw = 0, phase ^= 1u;
        }
      }
      ++items;
    }
    if (!ok || sm.abort)
      for (int i = 0; i < asked; ++i) {
        if (--raw < 0) raw = kRawStages - 1, phase ^= 1u;
        tc::mbar_wait(tc::su32(&sm.raw_full[raw]), phase, abort, false);
      }
  }
  // ... and the loader warps widen them.
  static SPEC_DEV void run_widen(const TcArgs& a, TcSmem& sm, uint32_t q0, int warp, int lane) {
    const Args& g = a.g;
    const int stages = a.l.stages, units = g.hd / 8, r0 = warp * RW;
    const uint32_t stage_bytes = a.l.stage_bytes, ring0 = q0 + a.l.q_bytes, raw0 = ring0 + (uint32_t)stages * stage_bytes;
    volatile int* abort = &sm.abort;
    Walk<S::BM, KT> walk(g, sm.plan);
    Item it;
    int items = 0, stage = 0, raw = 0;
    uint32_t phase = 0, r_phase = 0, q_phase = 0;
    bool ok = true;
    while (ok && walk.next(it)) {
      const int jobs = 2 * (it.k1 - it.k0);            // K, V, K, V, ...
#pragma unroll 1
      for (int j = 0; ok && j < jobs; ++j) {
        ok = wait_for(sm.raw_full[raw], r_phase, abort) &&
             wait_for(sm.empty[stage], phase ^ 1u, abort);
        if (!ok) break;
        const uint32_t word = sm.way_there[raw][r0 / 32];
        const uint32_t there = RW == 32 ? word : word >> (r0 % 32) & 0xffffu;
        const int info = sm.way_info[raw];
        const uint32_t from = raw0 + (uint32_t)raw * a.l.raw_bytes, at = ring0 + (uint32_t)stage * stage_bytes;
        if (units == 16) widen_rows<8>(from, at, r0, lane, 8);
        else if (units == 8) widen_rows<4>(from, at, r0, lane, 4);
        else widen_rows<0>(from, at, r0, lane, units / 2);
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(tc::su32(&sm.raw_empty[raw]));
        const uint32_t absent = (there & 0xffffu ? 0u : 0xffffu) | (RW == 32 && !(there >> 16) ? 0xffff0000u : 0u);
        if (absent) {                                  // (whatever the raw stage held)
          zero_rows(at, r0, lane, units, absent);
          __syncwarp();
        }
        if (info >= 0) clean_rows(sm, at, r0, lane, units, info, there);
        proxy_fence();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(tc::su32(&sm.full[stage]));
        if (++raw == kRawStages) raw = 0, r_phase ^= 1u;
        if (++stage == stages) stage = 0, phase ^= 1u;
        // Q, once the first keys are there
        if (j == 0) ok = next_q(a, sm, it, q0, warp, lane, items, q_phase);
      }
      ++items;
    }
    cp_wait<0>();
    if (!ok || sm.abort) settle_q(a, sm, warp, items);
  }

  // One loop, a step of which either hands over the oldest stage under way or asks for the next one, so that each is in
  // the code once.
  static SPEC_DEV void run(const TcArgs& a, TcSmem& sm, uint32_t q0, int warp, int lane) {
    const Args& g = a.g;
    const int chunks = a.l.chunks, stages = a.l.stages, units = g.hd * ES / 16, r0 = warp * RW;
    const uint32_t stage_bytes = a.l.stage_bytes, raw_bytes = a.l.raw_bytes, ring0 = q0 + a.l.q_bytes,
                   raw0 = ring0 + (uint32_t)stages * stage_bytes, stride = (uint32_t)(g.nkv * g.hd * ES);
    volatile int* abort = &sm.abort;
    Walk<S::BM, KT> walk(g, sm.plan);
    Item it;
    it.k0 = it.k1 = 0;
    // stage: the next to be filled; f_stage: of the oldest copies under way (8 bits: raw, f_raw)
    int tiles = 0, items = 0, issued = 0, finished = 0, stage = 0, f_stage = 0, raw = 0, f_raw = 0, q_at = -1;
    uint32_t phase = 0, q_phase = 0;
    int k = 0, key = 0, e = -1, slot = -1, info = -1;
    int block = 0, in_block = 0;       // of the lane's key in the tile whose entry has been asked for
    const int step_b = KT / g.kv.block_size, step_i = KT % g.kv.block_size;
    const int32_t* table = nullptr;
    bool value = false, more = true, q_due = false;
    // A key's entry of the block table, asked for a tile ahead; -1 where no row attends to it.
    const bool mine = lane < RW;
    auto entry = [&](int key_) { return mine && key_ >= it.lo && key_ < it.hi ? __ldg(table + block) : -1; };
    Edges<KT> edges;
#pragma unroll 1
    for (;;) {
      if (!value && k == it.k1 && more && !q_due) {
        more = walk.next(it);
        if (more) {
          q_due = true;
          k = it.k0;
          key = (it.tile0 + k) * KT + r0 + lane;
          table = g.kv.block_table + (long long)(g.b0 + it.b) * g.kv.max_blocks;
          block = key / g.kv.block_size, in_block = key % g.kv.block_size;
          edges = Edges<KT>(g, it);
          e = entry(key);
        }
      }
      bool hand = issued - finished > kLag;
      if (hand) {
        cp_wait<kLag>();
      } else if (!more) {
        if (issued == finished) break;
        cp_wait<0>();
        hand = true;
      } else if (q_due || !F8) {
        // what has been asked for may be what frees the place that is waited for
        uint64_t& bar = q_due ? sm.q_empty : sm.empty[stage];
        const uint32_t parity = q_due ? q_phase : phase ^ 1u;
        if (!(q_due && items == 0) && !test(bar, parity)) {
          if (issued > finished) {
            cp_wait<0>();
            hand = true;
          } else if (!wait_for(bar, parity, abort)) {
            break;
          }
        }
      }
      if (hand) {
        // it has come: widened (8 bits), cleared of values that are not finite (in an edge tile), handed to the MMA thread
        const int edge = sm.info[warp][finished % kTileBits];
        if constexpr (F8) {
          if (!wait_for(sm.empty[stage], phase ^ 1u, abort)) break;
          const uint32_t from = raw0 + (uint32_t)f_raw * raw_bytes, to = ring0 + (uint32_t)stage * stage_bytes;
          if (units == 8) widen_rows<8>(from, to, r0, lane, units);
          else if (units == 4) widen_rows<4>(from, to, r0, lane, units);
          else widen_rows<0>(from, to, r0, lane, units);
          if (++f_raw == kRawStages) f_raw = 0;
        }
        if (edge >= 0) {
          __syncwarp();
          clean_rows(sm, ring0 + (uint32_t)(F8 ? stage : f_stage) * stage_bytes, r0, lane, g.hd / 8, edge, 0xffffffffu);   // (others are zeros)
        }
        proxy_fence();
        __syncwarp();
        if (lane == 0) {
          tc::mbar_arrive(tc::su32(&sm.full[F8 ? stage : f_stage]));
          if (finished == q_at) tc::mbar_arrive(tc::su32(&sm.q_full));
        }
        ++finished;
        if constexpr (F8) {
          if (++stage == stages) stage = 0, phase ^= 1u;
        } else {
          if (++f_stage == stages) f_stage = 0;
        }
        continue;
      }
      if (q_due) {
        if (items > 0) q_phase ^= 1u;
        ++items;
        q_due = false;
        if (a.l.q_boxes) {
          copy_q(a, sm, it, q0, warp, lane);
        } else {
          load_q(g, it, q0, chunks, warp, lane);
          q_at = issued;                               // comes with the next stage's copies
        }
        if (!F8 && !test(sm.empty[stage], phase ^ 1u)) continue;
      }
      if (!value) {                                    // a new tile: its slots
        const int tile = it.tile0 + k;
        slot = -1;
        if (mine && key >= it.lo && key < it.hi) {
          const long long s = (long long)e * g.kv.block_size + in_block;
          if (s >= 0 && s < g.kv.num_slots) slot = (int)s;
          else report(g.ws, SPEC_ERR_DEVICE, g.b0 + it.b, key);
        }
        if (k + 1 < it.k1) {
          block += step_b, in_block += step_i;
          if (in_block >= g.kv.block_size) in_block -= g.kv.block_size, ++block;
          e = entry(key + KT);
        }
        const uint32_t there = __ballot_sync(0xffffffffu, slot >= 0);
        if (lane == 0) {
          if constexpr (RW == 32) sm.bits[tiles % kTileBits][warp] = there;
          else reinterpret_cast<uint16_t*>(sm.bits[tiles % kTileBits])[warp] = (uint16_t)there;
        }
        info = edges.has(tile) ? ((items - 1) % kItems) << 8 | edges.template slot<S::EDGES>(tile) : -1;
      }
      const uint32_t to = F8 ? raw0 + (uint32_t)raw * raw_bytes : ring0 + (uint32_t)stage * stage_bytes;
      const char* base = static_cast<const char*>(value ? g.kv.v : g.kv.k) + (long long)it.h * g.hd * ES;
      if (units == 16) copy_rows<16>(base, stride, slot, to, r0, lane, units);
      else if (units == 8) copy_rows<8>(base, stride, slot, to, r0, lane, units);
      else copy_rows<0>(base, stride, slot, to, r0, lane, units);
      cp_commit();
      if (lane == 0) sm.info[warp][issued % kTileBits] = value ? info : -1;
      __syncwarp();
      ++issued;
      if constexpr (F8) {
        if (++raw == kRawStages) raw = 0;
      } else {
        if (++stage == stages) stage = 0, phase ^= 1u;
      }
      if (value) ++k, ++tiles, key += KT;
      value = !value;
    }
    cp_wait<0>();                                      // nothing in flight when the CTA ends, or gives up
    if (a.l.q_boxes && warp == 0 && items > 0 && sm.abort) tc::mbar_wait(tc::su32(&sm.q_full), (uint32_t)(items - 1) & 1u, abort, false);
  }
};

// ---------------------------------------------------------------- MMA warp
// The whole warp walks the items, with values that are the same in all lanes (uniform()), and one lane issues: a lane on a
// path of its own would move every operand of every instruction into uniform registers first (80 cycles an MMA).
SPEC_DEV int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }
SPEC_DEV bool elect_one() {
  uint32_t one;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
  return one != 0;
}
// Waits without an answer, so that the warp's path does not depend on it: after a timeout every wait returns at once, and
// what is issued meanwhile works on whatever is there.  (A path that does is 100 cycles longer a wait.)
SPEC_DEV void settle(uint64_t& bar, uint32_t parity, volatile int* abort) { (void)wait_lane(bar, parity, abort); }

// Jobs of an item, in the order of their MMAs: kTwoQ: (tile 0, rows 0-127), (tile 0, rows 128-255), (tile 1, ...), ...;
// otherwise the tiles, for two streams in turns (kOneQ) or one (kWide).  The products of job k with V, then the scores of
// job k + 2, which go over its weights: one warp for both streams, so that they stay half a period apart and their softmax
// warps do not all want the special function units at the same time.
// The weights of a job come in halves, so that the products begin with whichever half is there.
template <typename T, int MODE> SPEC_DEV void issue_mmas(const TcArgs& a, TcSmem& sm, uint32_t base_, uint32_t tmem_) {
  using S = Shape<MODE>;
  constexpr int KT = S::KT;
  const Args& g = a.g;
  const Layout& l = a.l;
  const uint32_t base = uniform(base_), tmem = uniform(tmem_), ring0 = base + l.q_bytes;
  const int ks = g.hd / 16;
  const uint32_t id_s = idesc_of<T>(KT, false), id_o = idesc_of<T>(g.hd, true);
  volatile int* abort = &sm.abort;
  Walk<S::BM, KT> walk(g, sm.plan);
  Item it;
  uint32_t q_phase = 0, p_phase = 0, free_phase = 0;   // (of two barriers: a bit each)
  // K and V tiles take turns in the ring; their next places, and what is added to a descriptor there
  int k_st = 0, v_st = 1;
  uint32_t k_ph = 0, v_ph = 0;
  const uint64_t q_desc = tc::desc_sw128(base), k_desc = tc::desc_sw128(ring0), v_desc = desc_values(ring0, KT * 128);
  const uint32_t q_lo = (uint32_t)q_desc, k_lo = (uint32_t)k_desc, v_lo = (uint32_t)v_desc;
  const uint32_t s_hi = (uint32_t)(k_desc >> 32), v_hi = (uint32_t)(v_desc >> 32), stage16 = (uint32_t)l.stage_bytes >> 4;
  bool first = true;
  while (__any_sync(0xffffffffu, walk.next(it)) && !__any_sync(0xffffffffu, *abort != 0)) {
    const int jobs = uniform((it.k1 - it.k0) * (MODE == kTwoQ ? 2 : 1));
    settle(sm.q_full, q_phase, abort);
    q_phase ^= 1u;
#pragma unroll 1
    for (int k = -2; k < jobs; ++k) {
      const int buf = k & 1;
      const bool last_use = MODE != kTwoQ || buf;      // of the K and V tiles
      if (k >= 0) {
        const int acc = MODE == kWide ? 0 : buf;
        const bool fresh = MODE == kWide ? k == 0 : k < 2;
        if (MODE != kTwoQ || !buf) settle(sm.full[v_st], v_ph, abort);
        if (fresh && !first) {         // the last item's accumulator has been read
          settle(sm.o_free[acc], free_phase >> acc & 1u, abort);
          free_phase ^= 1u << acc;
        }
        const uint32_t b = v_lo + v_st * stage16;
        const uint32_t d = tmem + (uint32_t)(acc ? S::O1 : S::O0), p = tmem + (uint32_t)(buf * KT);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          settle(sm.p_full[buf][h], p_phase >> buf & 1u, abort);
          tc::tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int i = 0; i < KT / 32; ++i) {
              const int kk = h * (KT / 32) + i;
              mma_ts(d, p + 8 * kk, b + (kk * 2048 >> 4), v_hi, id_o, kk > 0 ? 1u : fresh ? 0u : 1u);
            }
            if (h && last_use) tc::tc_commit(tc::su32(&sm.empty[v_st]));
            if (h && (MODE == kWide || k >= jobs - 2)) tc::tc_commit(tc::su32(&sm.o_done[acc]));
          }
          __syncwarp();
        }
        p_phase ^= 1u << buf;
        if (last_use) {
          v_st += 2;
          if (v_st >= l.stages) v_st -= l.stages, v_ph ^= 1u;
        }
      }
      if (k + 2 < jobs) {
        if (MODE != kTwoQ || !buf) {
          settle(sm.full[k_st], k_ph, abort);
          tc::tc_fence_after();
        }
        if (elect_one()) {
          uint32_t qa = q_lo + (MODE == kTwoQ ? (uint32_t)(buf * l.chunks) * (16384 >> 4) : 0u), kb = k_lo + k_st * stage16;
          const uint32_t d = tmem + (uint32_t)(buf * KT);
          mma_ss<false>(d, qa, s_hi, kb, s_hi, id_s);
#pragma unroll 1
          for (int c = 0, n = ks; c < l.chunks; ++c, n -= 4, qa += 16384 >> 4, kb += KT * 128 >> 4) {
            if (c) mma_ss<true>(d, qa, s_hi, kb, s_hi, id_s);
            if (n > 1) mma_ss<true>(d, qa + 2, s_hi, kb + 2, s_hi, id_s);
            if (n > 2) mma_ss<true>(d, qa + 4, s_hi, kb + 4, s_hi, id_s);
            if (n > 3) mma_ss<true>(d, qa + 6, s_hi, kb + 6, s_hi, id_s);
          }
          tc::tc_commit(tc::su32(&sm.s_full[buf]));
          if (last_use) tc::tc_commit(tc::su32(&sm.empty[k_st]));
          if (k + 2 == jobs - 1) tc::tc_commit(tc::su32(&sm.q_empty));
        }
        __syncwarp();
        if (last_use) {
          k_st += 2;
          if (k_st >= l.stages) k_st -= l.stages, k_ph ^= 1u;
        }
      }
    }
    // (kOneQ with a single tile: the second accumulator is not used, nor waited for)
    if (MODE == kOneQ && jobs == 1 && !first) {
      settle(sm.o_free[1], free_phase >> 1, abort);
      free_phase ^= 2u;
    }
    first = false;
  }
  // the copies' stages and TMEM are given back only when every MMA has ended
  if (elect_one()) tc::tc_commit(tc::su32(&sm.drain));
  __syncwarp();
  tc::mbar_wait(tc::su32(&sm.drain), 0, abort, false);
}

// ---------------------------------------------------------------- softmax warpgroups
// Weights are 2^(s - m + kShift) against a reference m, which follows the running maximum only when that has gone more
// than kSlack past it: then the sums and outputs are rescaled, as they seldom are.  f16 weights stay below 2^15 and lose
// what is under 2^-34 of the largest; bf16 has fp32's exponents.  A weight goes into the product with V as one 16-bit number,
// rounded: 2^-8 (bf16) or 2^-11 of it is lost at most, as of an output by its own rounding, and what different keys lose does not
// add up in one direction (against 64 bits 0.0021-0.0023 of the output, 0.0017 by its rounding alone; f16 0.00030 / 0.00021).  A second part
// of each weight would be half as much tensor work again.  The sum l is of the weights as they were before.
template <typename T> struct Weights {
  static constexpr bool kHalf = std::is_same_v<T, __half>;
  static constexpr float kShift = kHalf ? 10.f : 0.f, kSlack = kHalf ? 5.f : 8.f;
};

template <typename T, bool F8, int MODE> struct Softmax {
  using S = Shape<MODE>;
  using W = Weights<T>;
  static constexpr int KT = S::KT, BM = S::BM;
  const Args& g;
  TcSmem& sm;
  const int w, warp, lane, row;        // warpgroup, its warp, and the thread's row of 128
  const uint32_t tm;                   // TMEM with the warp's lanes
  float m = -INFINITY, l = 0.f;
  bool counted = false;                // the item's piece has been counted

  SPEC_DEV Softmax(const Args& g_, TcSmem& sm_, uint32_t tmem, int w_, int warp_, int lane_)
      : g(g_), sm(sm_), w(w_), warp(warp_), lane(lane_), row(warp_ * 32 + lane_), tm(tmem + ((uint32_t)(warp_ * 32) << 16)) {}

  // The warps that write an item together: a warpgroup, or both (kOneQ).  Bounded as every wait.
  uint32_t group_phase = 0;
  SPEC_DEV bool group_sync() {
    uint64_t& bar = sm.group[MODE == kOneQ ? 0 : w];
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(tc::su32(&bar));
    const bool ok = wait_for(bar, group_phase, &sm.abort);
    group_phase ^= 1u;
    __syncwarp();
    return ok;
  }
  SPEC_DEV void arrive(uint64_t& bar) {
    tc::tc_fence_before();
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(tc::su32(&bar));
  }

  // bits of the tile's keys 32 i .. 32 i + 31 that are in [lo, hi) (of the tile)
  static SPEC_DEV uint32_t span(int lo, int hi, int i) {
    const int a = min(max(lo - 32 * i, 0), 32), b = min(max(hi - 32 * i, 0), 32);
    const uint32_t below_b = b == 32 ? 0xffffffffu : (1u << b) - 1u, below_a = a == 32 ? 0xffffffffu : (1u << a) - 1u;
    return below_b & ~below_a;
  }

  // One tile: scores in an S buffer -> weights there, handed over by halves.  o0: the accumulator; fresh: nothing is in it.
  // done: waits until the products of the last tile are in the accumulator (kWide).
  template <typename Done> SPEC_DEV void tile(const Edges<KT>& edges, int tile, int bits, int buf, uint32_t o0, bool fresh,
                                              int klo, int khi, Done&& done) {
    const uint32_t at = tm + (uint32_t)(buf * KT);
    __syncwarp();
    const uint4 there = *reinterpret_cast<const uint4*>(sm.bits[bits]);
    const uint32_t all = KT == 128 ? there.x & there.y & there.z & there.w : there.x & there.y;
    if (edges.has(tile) || all != 0xffffffffu) {
      const int key0 = tile * KT;
#pragma unroll 1
      for (int i = 0; i < KT / 32; ++i) {
        const uint32_t seen = span(klo - key0, khi - key0, i) & (i == 0 ? there.x : i == 1 ? there.y : i == 2 ? there.z : there.w);
        if (__all_sync(0xffffffffu, seen == 0xffffffffu)) continue;
        uint32_t s[32];
        tmem_ld32(at + 32 * i, s);
        tc::tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 32; ++j) s[j] = seen & (1u << j) ? s[j] : 0xff800000u;
        tmem_st16(at + 32 * i, s);
        tmem_st16(at + 32 * i + 16, s + 16);
      }
      tmem_st_wait();
    }
    uint32_t x[KT];
#pragma unroll
    for (int i = 0; i < KT / 32; ++i) tmem_ld32(at + 32 * i, x + 32 * i);
    tc::tmem_ld_wait();
    float t0 = -INFINITY, t1 = -INFINITY, t2 = -INFINITY, t3 = -INFINITY;
#pragma unroll
    for (int j = 0; j < KT; j += 8) {
      t0 = max3(t0, x[j], x[j + 1]), t1 = max3(t1, x[j + 2], x[j + 3]);
      t2 = max3(t2, x[j + 4], x[j + 5]), t3 = max3(t3, x[j + 6], x[j + 7]);
    }
    const float now = fmaxf(fmaxf(fmaxf(t0, t1), fmaxf(t2, t3)) * g.scale2, m);
    bool in = fresh;
    if (fresh) {
      m = now;
    } else if (__any_sync(0xffffffffu, now > m + W::kSlack)) {
      const float f = m == -INFINITY ? 1.f : exp2_fast(m - now);
      if (!done()) return;
      in = true;
      tc::tmem_ld_wait();
      tc::tc_fence_after();
#pragma unroll 1
      for (int c = 0; c < g.hd; c += 16) {
        uint32_t o[16];
        tc::tmem_ld16(tm + o0 + c, o);
        tc::tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
        tmem_st16(tm + o0 + c, o);
      }
      l *= f;
      m = now;
    }
    const float base = W::kShift - base_of(m);
    const Two b2(base, base), scale(g.scale2, g.scale2);
    Two sum(0.f, 0.f);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int i = h * (KT / 64); i < (h + 1) * (KT / 64); ++i) {
        uint32_t p[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          float u, v;
          fma2(Two(__uint_as_float(x[32 * i + 2 * j]), __uint_as_float(x[32 * i + 2 * j + 1])), scale, b2).get(u, v);
          u = exp2_fast(u), v = exp2_fast(v);
          sum = add2(sum, Two(u, v));
          p[j] = pack2<T>(u, v);
        }
        tmem_st16(at + 16 * i, p);
      }
      tmem_st_wait();
      if (h == 1 && !in) done();           // (every phase is waited for in its turn)
      arrive(sm.p_full[buf][h]);
    }
    float u, v;
    sum.get(u, v);
    l += u + v;
  }

  // A value that is not finite, of a key of an edge tile that the row attends to
  SPEC_DEV void mend(const Item& it, int item, int klo, int khi, int c0, float* o) {
#pragma unroll 1
    for (int e = 0; e < 2 * S::EDGES; ++e)
#pragma unroll 1
      for (int i = 0; i < KT / 32; ++i)
#pragma unroll 1
        for (uint32_t b = sm.poison[item][e][i]; b; b &= b - 1) {
          const int key = Edges<KT>(g, it).template tile<S::EDGES>(e) * KT + 32 * i + __ffs(b) - 1;
          if (key < klo || key >= khi) continue;
          const long long at = (slot_of(g.kv, g.b0 + it.b, key) * g.nkv + it.h) * g.hd + c0;
          uint32_t odd = 0;
#pragma unroll 1
          for (int j = 0; j < 16; ++j) {
            float v;
            if constexpr (F8) v = (float)static_cast<const __nv_fp8_e4m3*>(g.kv.v)[at + j];
            else v = (float)static_cast<const T*>(g.kv.v)[at + j];
            odd |= not_finite(v) ? 1u << j : 0u;
          }
#pragma unroll
          for (int j = 0; j < 16; ++j) o[j] = odd >> j & 1u ? NAN : o[j];
        }
  }

  // 16 components of the row's unnormalised output, or 32
  SPEC_DEV void take(float* o, int c, float f0, float f1, bool two, bool more) {
    __syncwarp();
    const uint32_t o0 = tm + (MODE == kTwoQ && w ? S::O1 : S::O0) + c;
    uint32_t a[32];
    tc::tmem_ld16(o0, a);
    if (more) tc::tmem_ld16(o0 + 16, a + 16);
    if (MODE == kOneQ && two) {
      uint32_t b[32];
      tc::tmem_ld16(tm + S::O1 + c, b);
      if (more) tc::tmem_ld16(tm + S::O1 + c + 16, b + 16);
      tc::tmem_ld_wait();
#pragma unroll
      for (int j = 0; j < 32; ++j) o[j] = fmaf(__uint_as_float(b[j]), f1, __uint_as_float(a[j]) * f0);
    } else {
      tc::tmem_ld_wait();
#pragma unroll
      for (int j = 0; j < 32; ++j) o[j] = MODE == kOneQ ? __uint_as_float(a[j]) * f0 : __uint_as_float(a[j]);
    }
  }

  static SPEC_DEV void write(T* dst, const float* o, float inv) {
    uint32_t u[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) u[j] = pack2<T>(o[2 * j] * inv, o[2 * j + 1] * inv);
    reinterpret_cast<uint4*>(dst)[0] = make_uint4(u[0], u[1], u[2], u[3]);
    reinterpret_cast<uint4*>(dst)[1] = make_uint4(u[4], u[5], u[6], u[7]);
  }

  // 16 components of the rows of a warp, a row a lane: two lanes exchange pieces of 16 bytes, so that a store writes 32 bytes
  // of each of 16 rows instead of 16 of each of 32 (8 chunks of 512-1024 tokens 287 -> 279 us, 32 of 100-300 tokens
  // 114 -> 109; four lanes, 64 bytes of 8 rows: as much, but 1-3 % more where items are long, from the code).  Not kOneQ,
  // whose few rows are written sooner without (4 chunks of 8 tokens 13.0 / 14.2).
  // at: the lane's piece of the pair's rows (NULL: not written).
  static SPEC_DEV void write_rows(T* const (&at)[2], int c, const float* o, float inv, bool odd) {
    uint32_t u[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) u[j] = pack2<T>(o[2 * j] * inv, o[2 * j + 1] * inv);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t x = __shfl_xor_sync(0xffffffffu, odd ? u[j] : u[4 + j], 1);
      if (odd) u[j] = x;
      else u[4 + j] = x;
    }
    if (at[0]) *reinterpret_cast<uint4*>(at[0] + c) = make_uint4(u[0], u[1], u[2], u[3]);
    if (at[1]) *reinterpret_cast<uint4*>(at[1] + c) = make_uint4(u[4], u[5], u[6], u[7]);
  }

  // The item's rows, or their piece; the last piece to come joins all.
  SPEC_DEV bool finish(const Item& it, int item, int klo, int khi) {
    const bool two = MODE == kOneQ && it.k1 - it.k0 > 1;
    float f0 = 1.f, f1 = 0.f;
    if (MODE == kOneQ) {
      // the warpgroups' halves of the keys -> each writes half of the components
      sm.ml[w][row] = make_float2(m, l);
      if (!group_sync()) return false;
      const float2 o = sm.ml[1 - w][row];
      const float m0 = w ? o.x : m, m1 = w ? m : o.x, l0 = w ? o.y : l, l1 = w ? l : o.y;
      m = fmaxf(m0, m1);
      f0 = m0 == -INFINITY ? 1.f : exp2_fast(m0 - base_of(m)), f1 = m1 == -INFINITY ? 1.f : exp2_fast(m1 - base_of(m));
      l = l0 * f0 + l1 * f1;
      if (!group_sync()) return false;     // (read before the next item's are written)
    }
    const int steps = g.hd / 16, half = (steps + 1) / 2;
    const int c0 = MODE == kOneQ && w ? 16 * half : 0, c1 = MODE == kOneQ && !w ? 16 * half : g.hd;
    const int r = MODE == kTwoQ ? w * 128 + row : row;
    const bool valid = r < it.rows, poisoned = sm.poisoned[item] != 0;
    const int tok = (it.r0 + r) / g.G, head = it.h * g.G + (it.r0 + r) - tok * g.G;
    T* dst = static_cast<T*>(g.out) + (it.row0 + tok) * g.out_ld + (long long)head * g.hd;
    float* lse = g.lse && c0 == 0 ? g.lse + (long long)(it.row0 + tok) * g.nq + head : nullptr;
    const bool whole = it.k0 == 0 && it.k1 == it.tiles;
    const float inv = l == 0.f ? 0.f : g.v_scale / l;
    const size_t piece = piece_floats(BM, g.hd);
    float* mine = g.part + (whole ? 0 : 2 * blockIdx.x + (it.k0 > 0 ? 0 : 1)) * piece;
    const bool odd = lane & 1;
    T* at[2];
    if (MODE != kOneQ && whole) {
      T* const own = valid ? dst : nullptr;
      T* const other = reinterpret_cast<T*>(__shfl_xor_sync(0xffffffffu, reinterpret_cast<unsigned long long>(own), 1));
      at[0] = odd ? other : own, at[1] = odd ? own : other;
      if (odd) at[0] = at[0] ? at[0] + 8 : nullptr, at[1] = at[1] ? at[1] + 8 : nullptr;
    }
#pragma unroll 1
    for (int c = c0; c < c1; c += 32) {
      const bool more = c + 16 < c1;
      float o[32];
      take(o, c, f0, f1, two, more);
      if (poisoned && valid) {
        mend(it, item, klo, khi, c, o);
        if (more) mend(it, item, klo, khi, c + 16, o + 16);
      }
      if (MODE != kOneQ && whole) {
        write_rows(at, c, o, inv, odd);
        if (more) write_rows(at, c + 16, o + 16, inv, odd);
      }
      if (MODE == kOneQ && whole && valid) {
        write(dst + c, o, inv);
        if (more) write(dst + c + 16, o + 16, inv);
      }
      if (valid && !whole)
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j < 4 || more)
            *reinterpret_cast<float4*>(mine + ((size_t)(c / 4 + j) * BM + r) * 4) =
                make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
    }
    if (whole) {
      if (valid && lse) *lse = l == 0.f ? -INFINITY : (m - W::kShift + log2f(l)) * kLn2;
      release();
      return true;
    }
    const Pieces pc(sm.plan, it);
    if (valid && c0 == 0) mine[(size_t)BM * g.hd + r] = m, mine[(size_t)BM * (g.hd + 1) + r] = l;
    release();
    __threadfence();
    const int slot = MODE == kOneQ ? 0 : w;
    if (!group_sync()) return false;
    if (counts()) sm.last[slot] = count(it, pc);
    if (!group_sync()) return false;
    const bool last = sm.last[slot] != 0;
    if (!group_sync()) return false;       // (read before the next item's is written)
    if (last) join(it, pc);
    return true;
  }

  // The thread that counts the warpgroups' pieces of an item, and whether this is the last to come.
  SPEC_DEV bool counts() const { return row == 0 && (MODE != kOneQ || w == 0); }
  SPEC_DEV bool count(const Item& it, const Pieces& pc) {
    const long long at = (long long)it.h * sm.plan.pairs[g.B] + sm.plan.pairs[it.b] + it.t;
    int* counter = g.counters + (MODE == kTwoQ ? 2 * at + w : at);
    const bool last = atomicAdd(counter, 1) == pc.c1 - pc.c0;
    if (last) *counter = 0;
    counted = true;
    return last;
  }
  // After a wait that ran out: what is left of the share counts as pieces that have come, so that all counters are at zero
  // when the launch ends.
  SPEC_DEV void give_up(Walk<BM, KT>& walk, Item& it) {
    if (!counts()) return;
    do {
      if (!counted && (it.k0 > 0 || it.k1 < it.tiles)) count(it, Pieces(sm.plan, it));
      counted = false;
    } while (walk.next(it));
  }

  // All pieces of the item's rows, in their order; 16 components of a row a thread at a time.
  SPEC_DEV void join(const Item& it, const Pieces& pc) {
    __threadfence();
    const int base = MODE == kTwoQ ? w * 128 : 0, rows = MODE == kTwoQ ? min(128, it.rows - base) : it.rows;
    const int tid = MODE == kOneQ ? w * 128 + row : row, threads = MODE == kOneQ ? 256 : 128;
    const size_t piece = piece_floats(BM, g.hd);
#pragma unroll 1
    for (int task = tid; task < rows * (g.hd / 16); task += threads) {
      const int r = base + task % rows, c = task / rows * 16;
      float M = -INFINITY;
#pragma unroll 4
      for (int p = pc.c0; p <= pc.c1; ++p) M = fmaxf(M, __ldcg(g.part + pc.slot(p) * piece + (size_t)BM * g.hd + r));
      float L = 0.f, o[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) o[j] = 0.f;
#pragma unroll 4
      for (int p = pc.c0; p <= pc.c1; ++p) {
        const float* x = g.part + pc.slot(p) * piece;
        const float mc = __ldcg(x + (size_t)BM * g.hd + r), lc = __ldcg(x + (size_t)BM * (g.hd + 1) + r);
        float4 v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = __ldcg(reinterpret_cast<const float4*>(x + ((size_t)(c / 4 + j) * BM + r) * 4));
        const float f = mc == -INFINITY ? 1.f : exp2_fast(mc - base_of(M));   // (1: of zeros)
        L = fmaf(lc, f, L);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          o[4 * j] = fmaf(v[j].x, f, o[4 * j]), o[4 * j + 1] = fmaf(v[j].y, f, o[4 * j + 1]);
          o[4 * j + 2] = fmaf(v[j].z, f, o[4 * j + 2]), o[4 * j + 3] = fmaf(v[j].w, f, o[4 * j + 3]);
        }
      }
      const int tok = (it.r0 + r) / g.G, head = it.h * g.G + (it.r0 + r) - tok * g.G;
      write(static_cast<T*>(g.out) + (it.row0 + tok) * g.out_ld + (long long)head * g.hd + c, o, L == 0.f ? 0.f : g.v_scale / L);
      if (g.lse && c == 0)
        g.lse[(long long)(it.row0 + tok) * g.nq + head] = L == 0.f ? -INFINITY : (M - W::kShift + log2f(L)) * kLn2;
    }
  }
  // the accumulators have been read
  SPEC_DEV void release() {
    if (MODE == kTwoQ) {
      arrive(sm.o_free[w]);
    } else {
      arrive(sm.o_free[0]);
      if (MODE == kOneQ) arrive(sm.o_free[1]);
    }
  }

  SPEC_DEV void run() {
    volatile int* abort = &sm.abort;
    Walk<BM, KT> walk(g, sm.plan);
    Item it;
    uint32_t s_phase[2] = {0, 0}, o_phase[2] = {0, 0};
    int tiles = 0, items = 0;
    auto item_done = [&]() -> bool {
      const int nt = it.k1 - it.k0, item = items % kItems;
      int klo, khi;
      keys_of(g, it, MODE == kTwoQ ? w * 128 + row : row, &klo, &khi);
      const Edges<KT> edges(g, it);
      m = -INFINITY, l = 0.f;
      bool fresh = true;
      for (int k = MODE == kOneQ ? w : 0; k < nt; k += MODE == kOneQ ? 2 : 1) {
        const int buf = MODE == kWide ? k & 1 : w;
        if (!wait_for(sm.s_full[buf], s_phase[buf], abort)) return false;
        s_phase[buf] ^= 1u;
        tc::tc_fence_after();
        bool ok = true;
        tile(edges, it.tile0 + it.k0 + k, (tiles + k) % kTileBits, buf,
             MODE == kWide ? S::O0 : w ? S::O1 : S::O0, fresh, klo, khi, [&] {
               // kTwoQ, kOneQ: the scores were asked for after those products
               if (MODE == kWide) ok = wait_for(sm.o_done[0], o_phase[0] ^ (uint32_t)((k - 1) & 1), abort);
               return ok;
             });
        if (!ok) return false;
        fresh = false;
      }
      if (MODE == kTwoQ) {
        if (!wait_for(sm.o_done[w], o_phase[w], abort)) return false;
        o_phase[w] ^= 1u;
      } else if (MODE == kOneQ) {
        if (!wait_for(sm.o_done[0], o_phase[0], abort)) return false;
        o_phase[0] ^= 1u;
        if (nt > 1) {
          if (!wait_for(sm.o_done[1], o_phase[1], abort)) return false;
          o_phase[1] ^= 1u;
        }
      } else {
        // a phase a tile
        if (!wait_for(sm.o_done[0], o_phase[0] ^ (uint32_t)((nt - 1) & 1), abort)) return false;
        o_phase[0] ^= (uint32_t)(nt & 1);
      }
      tc::tc_fence_after();
      const bool ok = finish(it, item, klo, khi);
      __syncwarp();
      if (!ok) return false;
      if (w == 0) {
        const int old = (items + kItems - 4) % kItems;
        if (row < 2 * 6 * 4) (&sm.poison[old][0][0])[row] = 0;
        if (row == 0) sm.poisoned[old] = 0;
      }
      ++items;
      tiles += nt;
      return true;
    };
    while (walk.next(it)) {
      counted = false;
      if (!item_done()) {
        give_up(walk, it);
        return;
      }
    }
  }
};

template <typename T, bool F8, int MODE> __global__ void __launch_bounds__(kTcThreads, 1)
    chunk_tc_kernel(const __grid_constant__ TcArgs a) {
  SPEC_TL(kTLChunkAttn);
  using S = Shape<MODE>;
  extern __shared__ uint8_t dyn[];
  __shared__ __align__(16) TcSmem sm;
  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
  const uint32_t base = (tc::su32(dyn) + 1023u) & ~1023u;
  if (tid == 0) {
    sm.abort = 0;
    for (int i = 0; i < kMaxStages; ++i) {
      tc::mbar_init(tc::su32(&sm.full[i]), 4);
      tc::mbar_init(tc::su32(&sm.empty[i]), 1);
    }
    tc::mbar_init(tc::su32(&sm.q_full), 4);
    tc::mbar_init(tc::su32(&sm.q_empty), 1);
    tc::mbar_init(tc::su32(&sm.drain), 1);
    for (int i = 0; i < 4; ++i) tc::mbar_init(tc::su32(&sm.landed[i]), 1);
    for (int i = 0; i < kRawStages; ++i) {
      tc::mbar_init(tc::su32(&sm.raw_full[i]), 1);
      tc::mbar_init(tc::su32(&sm.raw_empty[i]), 4);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(tc::su32(&sm.s_full[i]), 1);
      tc::mbar_init(tc::su32(&sm.p_full[i][0]), 4);
      tc::mbar_init(tc::su32(&sm.p_full[i][1]), 4);
      tc::mbar_init(tc::su32(&sm.o_done[i]), 1);
      tc::mbar_init(tc::su32(&sm.o_free[i]), MODE == kOneQ ? 8 : 4);
      tc::mbar_init(tc::su32(&sm.group[i]), MODE == kOneQ ? 8 : 4);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  for (int i = tid; i < kItems * 2 * 6 * 4; i += kTcThreads) (&sm.poison[0][0][0])[i] = 0;
  if (tid < kItems) sm.poisoned[tid] = 0;
  if (warp == 0) {
    tc::tmem_alloc(tc::su32(&sm.tmem), 512);
    tc::tmem_relinquish();
  }
  pdl_wait();
  pdl_trigger();
  // (asked for before the plan's own reads, and looked at after them)
  const int hold = tid == 0 ? __ldcg(static_cast<const int*>(a.g.ws) + kHoldWord) : 0;
  make_plan<S::BM, S::KT>(a.g, sm.plan, tid, kTcThreads);
  if (tid == 0) sm.hold = hold;
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = sm.tmem;
  if (warp < 8) {
    regs_inc<kSoftmaxRegs>();
    if (MODE != kWide || warp < 4) Softmax<T, F8, MODE>(a.g, sm, tmem, warp >> 2, warp & 3, lane).run();
  } else if (warp < 12) {
    regs_dec<kLoaderRegs>();
    if (sm.hold == (int)blockIdx.x + 1) {}             // every wait for them runs out
    else if (a.l.runs && F8) Loader<T, F8, MODE>::run_widen(a, sm, base, warp - 8, lane);
    else if (a.l.runs) Loader<T, F8, MODE>::run_tensor(a, sm, base, warp - 8, lane);
    else Loader<T, F8, MODE>::run(a, sm, base, warp - 8, lane);
  } else {
    regs_dec<kMmaRegs>();
    if (warp == 12) issue_mmas<T, MODE>(a, sm, base, tmem);
    else if (F8 && warp == 13 && a.l.runs) Loader<T, F8, MODE>::ask_raw(a, sm, base, lane);
  }
  tc::tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, 512);
  }
  if (tid == 0 && sm.abort) report(a.g.ws, SPEC_ERR_TIMEOUT, blockIdx.x, 0);
}

static_assert(kTcSmem + sizeof(TcSmem) <= 227 * 1024, "");

typedef void (*TcFn)(TcArgs);
// by type (chunk_attn_<type>.cu); NULL where the kernel is not launched with the registers that its warpgroups share out
// (a share above them would be waited for without end)
TcFn tc_kernel_bf16(bool f8, int mode);
TcFn tc_kernel_f16(bool f8, int mode);

template <typename T, bool F8, int MODE> TcFn checked() {
  static const bool ok = [] {
    cudaFuncAttributes a;
    return cudaFuncGetAttributes(&a, chunk_tc_kernel<T, F8, MODE>) == cudaSuccess && a.numRegs == kLaunchRegs;
  }();
  return ok ? chunk_tc_kernel<T, F8, MODE> : nullptr;
}

template <typename T> TcFn tc_kernel_of(bool f8, int mode) {
  if (f8) return mode == kTwoQ ? checked<T, true, kTwoQ>() : checked<T, true, kWide>();
  return mode == kTwoQ ? checked<T, false, kTwoQ>() : mode == kOneQ ? checked<T, false, kOneQ>() : checked<T, false, kWide>();
}

}  // namespace ca
}  // namespace spec
