// Attention of a chunk of new tokens on tcgen05: the kernel.  The translation
// units chunk_attn_<type>.cu instantiate it.
//
// A CTA has 128 or 256 packed rows (chunk_attn.cuh) and streams its keys in tiles.
// Per tile and 128 rows one job: S = Q K^T into TMEM, the softmax warpgroup's
// weights back into TMEM over S, O += P V with P from TMEM.  A softmax thread owns
// a row: no shuffles, its maximum and sum in registers.
//   warps 0-3, 4-7   two softmax warpgroups
//   warps 8-11       K/V and Q into shared memory (any block size, any alignment of runs)
//   warp 12          one thread issues all MMAs
// The MMA thread keeps two S buffers in flight: while a warpgroup works on one job's
// scores, the tensor cores do the other's products.
#pragma once
#include <type_traits>

#include "chunk_attn.cuh"
#include "tc_core.cuh"

namespace spec {
namespace ca {

// kTwoQ: 256 rows, a warpgroup for each half, every K/V tile used twice.  kOneQ: 128 rows, the warpgroups
// take turns at the tiles with an accumulator each, joined at the end.  kWide: head sizes above 128, whose
// accumulator leaves no room for a second one: 128 rows, tiles of 64 keys, one warpgroup.
enum Mode { kTwoQ = 0, kOneQ = 1, kWide = 2 };

constexpr int kTcThreads = 512;
// 512 threads are launched with 128 registers each and share them out: 2 x 128 x 200 + 128 x 72 + 128 x 40
constexpr int kSoftmaxRegs = 200, kLoaderRegs = 72, kMmaRegs = 40;
static_assert(2 * kSoftmaxRegs + kLoaderRegs + kMmaRegs <= 4 * 128, "");
constexpr int kMaxStages = 8, kTileBits = 8;
constexpr int kRawStages = 2;            // 8-bit tiles under way, before they are widened
// An item's masks are used again 8 items later: the loader is at most two items ahead of a warpgroup, and the
// warpgroups at most one apart, so the first of them may clear those of two items ago.
constexpr int kItems = 8;

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
};
template <int MODE> static inline Layout layout(int hd, bool f8) {
  using S = Shape<MODE>;
  Layout l;
  l.chunks = (hd + 63) / 64;
  l.q_bytes = S::BM * 128 * l.chunks;
  l.stage_bytes = S::KT * 128 * l.chunks;
  l.raw_bytes = f8 ? S::KT * hd : 0;
  const int room = 208 * 1024 - 1024 - l.q_bytes - kRawStages * l.raw_bytes;
  l.stages = room / l.stage_bytes < kMaxStages ? room / l.stage_bytes : kMaxStages;
  l.smem = 1024 + l.q_bytes + l.stages * l.stage_bytes + kRawStages * l.raw_bytes;
  return l;
}

struct TcArgs {
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

// D[tmem] (+)= A[tmem] * B[smem]
SPEC_DEV void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
SPEC_DEV void tmem_ld32(uint32_t a, float* r) {
  uint32_t* u = reinterpret_cast<uint32_t*>(r);
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

template <typename T> SPEC_DEV uint32_t pack2(float lo, float hi) {
  if constexpr (std::is_same_v<T, __half>) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}
template <typename T> SPEC_DEV float2 unpack2(uint32_t x) {
  if constexpr (std::is_same_v<T, __half>) return __half22float2(*reinterpret_cast<const __half2*>(&x));
  else return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&x));
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
  uint64_t full[kMaxStages], empty[kMaxStages], q_full, q_empty, drain, s_full[2], p_full[2], o_done[2], o_free[2], group[2];
  alignas(16) uint32_t bits[kTileBits][4];   // keys of a tile that are there
  uint32_t poison[kItems][2 * 6][4];   // keys of an item's edge tiles whose value is not finite
  int poisoned[kItems];
  int info[4][kTileBits];              // loader warps: what a stage under way needs when it has come
  float2 ml[2][128];
  int last[2];
  uint32_t tmem;
  int abort;
};

// ---------------------------------------------------------------- loader
template <typename T, bool F8, int MODE> struct Loader {
  using S = Shape<MODE>;
  static constexpr int KT = S::KT, RW = KT / 4;        // key rows of a warp
  static constexpr int EW = 16 / (F8 ? 1 : 2);         // components of 16 bytes of the cache
  static constexpr int kLag = F8 ? kRawStages - 1 : 2; // stages under way behind the newest
  const Args& g;
  const Layout& l;
  TcSmem& sm;
  uint32_t q0, ring0, raw0;
  int warp, lane, units, inv;          // 16-byte units of a cache row, and 2^16 / units rounded up
  int issued = 0, finished = 0, stage = 0, f_stage = 0;
  uint32_t phase = 0;
  int raw = 0, f_raw = 0, q_at = -1;   // the stage that the item's Q came with
  bool ok = true;

  SPEC_DEV Loader(const TcArgs& a, TcSmem& s, uint32_t base, int w, int ln)
      : g(a.g), l(a.l), sm(s), q0(base), ring0(base + a.l.q_bytes), raw0(base + a.l.q_bytes + a.l.stages * a.l.stage_bytes),
        warp(w), lane(ln) {
    units = g.hd / EW;
    inv = (65536 + units - 1) / units;
  }
  // rows of 16-byte units: row of item i (i < 32 * 32)
  SPEC_DEV int row_of(int i) const { return (i * inv) >> 16; }
  SPEC_DEV uint32_t place(int row, int u) const {      // of a 16-bit 16-byte unit in a stage
    return (uint32_t)((u >> 3) * KT * 128 + row * 128 + (((u ^ row) & 7) << 4));
  }
  SPEC_DEV bool wait(uint64_t& bar, uint32_t parity) {
    const uint32_t a = tc::su32(&bar);
    if (tc::mbar_try(a, parity)) return true;
    drain();                                           // what has been asked for may be what frees the stage
    return tc::mbar_wait(a, parity, &sm.abort);
  }
  SPEC_DEV void drain() {
    while (finished < issued && ok) {
      cp_wait<0>();
      finish();
    }
  }
  // Copies of the next stage, K or V of the tile whose slots the lanes hold.
  SPEC_DEV void issue(const void* cache, int slot, int h, int info) {
    if constexpr (!F8) {
      if (ok && !wait(sm.empty[stage], phase ^ 1u)) ok = false;
    }
    if (!ok) return;
    const uint32_t to = F8 ? raw0 + (uint32_t)raw * l.raw_bytes : ring0 + (uint32_t)stage * l.stage_bytes;
    const char* c = static_cast<const char*>(cache);
    for (int i = lane; i < RW * units + lane; i += 32) {   // (every lane takes part in the shuffles)
      const int row = min(row_of(i), RW - 1), u = i - row * units;
      const int s = __shfl_sync(0xffffffffu, slot, row);
      if (i < RW * units) {
        const long long at = (((long long)max(s, 0) * g.nkv + h) * units + u) * 16;
        const uint32_t dst = F8 ? to + (uint32_t)((warp * RW + row) * units + u) * 16 : to + place(warp * RW + row, u);
        cp16(dst, c + at, s >= 0);
      }
    }
    cp_commit();
    if (lane == 0) sm.info[warp][issued % kTileBits] = info;
    __syncwarp();
    ++issued;
    if constexpr (F8) {
      if (++raw == kRawStages) raw = 0;
    } else {
      if (++stage == l.stages) stage = 0, phase ^= 1u;
    }
    if (issued - finished > kLag) {
      cp_wait<kLag>();
      finish();
    }
  }
  // The oldest stage under way has come: widened (8 bits), cleared of values that are not finite (info: in an edge tile),
  // handed to the MMA thread.
  SPEC_DEV void finish() {
    const int info = sm.info[warp][finished % kTileBits];
    if constexpr (F8) {
      // (not through wait(): it must not come back here)
      if (!tc::mbar_wait(tc::su32(&sm.empty[stage]), phase ^ 1u, &sm.abort)) {
        ok = false;
        return;
      }
      const uint32_t from = raw0 + (uint32_t)f_raw * l.raw_bytes, to = ring0 + (uint32_t)stage * l.stage_bytes;
      for (int i = lane; i < RW * units; i += 32) {
        const int row = row_of(i), u = i - row * units, r = warp * RW + row;
        const uint4 x = lds128(from + (uint32_t)(r * units + u) * 16);
        const uint2 a = widen4<T>(x.x), b = widen4<T>(x.y), c = widen4<T>(x.z), d = widen4<T>(x.w);
        uint4 lo = make_uint4(a.x, a.y, b.x, b.y), hi = make_uint4(c.x, c.y, d.x, d.y);
        if (info >= 0) lo = clean(lo, info, r), hi = clean(hi, info, r);
        sts128(to + place(r, 2 * u), lo);
        sts128(to + place(r, 2 * u + 1), hi);
      }
      if (++f_raw == kRawStages) f_raw = 0;
    } else if (info >= 0) {
      const uint32_t at = ring0 + (uint32_t)f_stage * l.stage_bytes;
      for (int i = lane; i < RW * units; i += 32) {    // the units that this lane copied
        const int row = row_of(i), u = i - row * units, r = warp * RW + row;
        const uint32_t a = at + place(r, u);
        sts128(a, clean(lds128(a), info, r));
      }
    }
    proxy_fence();
    __syncwarp();
    if (lane == 0) {
      tc::mbar_arrive(tc::su32(&sm.full[F8 ? stage : f_stage]));
      if (finished == q_at) tc::mbar_arrive(tc::su32(&sm.q_full));
    }
    if (finished == q_at) q_at = -1;
    ++finished;
    if constexpr (F8) {
      if (++stage == l.stages) stage = 0, phase ^= 1u;
    } else {
      if (++f_stage == l.stages) f_stage = 0;
    }
  }
  // A weight of 0 times a value that is not finite is a NaN in rows that do not attend to the key: in edge tiles such
  // components are zeros, and the rows that do attend to the key get theirs at the end.
  SPEC_DEV uint4 clean(uint4 v, int info, int key) {
    const uint32_t a = odd_halves<T>(v.x), b = odd_halves<T>(v.y), c = odd_halves<T>(v.z), d = odd_halves<T>(v.w);
    if (a | b | c | d) {
      const int item = info >> 8, e = info & 255;
      atomicOr(&sm.poison[item][e][key >> 5], 1u << (key & 31));
      sm.poisoned[item] = 1;
      v.x &= ~a, v.y &= ~b, v.z &= ~c, v.w &= ~d;
    }
    return v;
  }
  SPEC_DEV void load_q(const Item& it) {
    constexpr int RQ = S::BM / 4;                      // rows of a warp
    const int qu = g.hd / 8, qinv = (65536 + qu - 1) / qu;
    const T* q = static_cast<const T*>(g.q);
    for (int r0 = 0; r0 < RQ; r0 += 32) {
      const int r = warp * RQ + r0 + lane;
      long long off = -1;
      if (r < it.rows) {
        const int tok = (it.r0 + r) / g.G, head = it.h * g.G + (it.r0 + r) - tok * g.G;
        off = (it.row0 + tok) * g.q_ld + (long long)head * g.hd;
      }
      for (int i = lane; i < 32 * qu + lane; i += 32) {
        const int row = min((i * qinv) >> 16, 31), u = i - row * qu;
        const long long o = __shfl_sync(0xffffffffu, off, row);
        if (i < 32 * qu) {
          const int m = warp * RQ + r0 + row, t = m >> 7, mr = m & 127;
          cp16(q0 + (uint32_t)(t * l.chunks * 16384 + (u >> 3) * 16384 + mr * 128 + (((u ^ mr) & 7) << 4)),
               q + max(o, 0ll) + 8 * u, o >= 0);
        }
      }
    }
    q_at = issued;                                     // with the next stage's copies
  }
  SPEC_DEV void run() {
    Walk<S::BM, KT> walk(g, sm.plan);
    Item it;
    int tiles = 0, items = 0;
    uint32_t q_phase = 0;
    while (ok && walk.next(it)) {
      const int im = items % kItems;
      if (items > 0) {
        if (!wait(sm.q_empty, q_phase)) break;
        q_phase ^= 1u;
      }
      ++items;
      load_q(it);
      for (int k = it.k0; ok && k < it.k1; ++k, ++tiles) {
        const int tile = it.tile0 + k, key = tile * KT + warp * RW + lane;
        int slot = -1;
        if (lane < RW && key >= it.lo && key < it.hi) {
          const long long s = slot_of(g.kv, g.b0 + it.b, key);
          slot = (int)s;
          if (s < 0) report(g.ws, SPEC_ERR_DEVICE, g.b0 + it.b, key);
        }
        const uint32_t there = __ballot_sync(0xffffffffu, slot >= 0);
        if (lane == 0) {
          if constexpr (RW == 32) sm.bits[tiles % kTileBits][warp] = there;
          else reinterpret_cast<uint16_t*>(sm.bits[tiles % kTileBits])[warp] = (uint16_t)there;
        }
        const bool edge = edge_tile(g, it, tile, KT);
        issue(g.kv.k, slot, it.h, -1);
        issue(g.kv.v, slot, it.h, edge ? im << 8 | edge_slot<S::EDGES, KT>(g, it, tile) : -1);
      }
    }
    drain();
    cp_wait<0>();                                      // nothing in flight when the CTA ends, or gives up
  }
};

// ---------------------------------------------------------------- MMA thread
template <typename T, int MODE> SPEC_DEV void issue_mmas(const TcArgs& a, TcSmem& sm, uint32_t base, uint32_t tmem) {
  using S = Shape<MODE>;
  constexpr int KT = S::KT;
  const Args& g = a.g;
  const Layout& l = a.l;
  const uint32_t ring0 = base + l.q_bytes;
  const int ks = g.hd / 16;
  const uint32_t id_s = idesc_of<T>(KT, false), id_o = idesc_of<T>(g.hd, true);
  volatile int* abort = &sm.abort;
  Walk<S::BM, KT> walk(g, sm.plan);
  Item it;
  uint32_t q_phase = 0, p_phase[2] = {0, 0}, free_phase[2] = {0, 0};
  int tile0 = 0;               // tiles before the item's
  bool first = true, ok = true;
  while (ok && walk.next(it)) {
    const int nt = it.k1 - it.k0, jobs = MODE == kTwoQ ? 2 * nt : nt;
    if (!tc::mbar_wait(tc::su32(&sm.q_full), q_phase, abort)) break;
    q_phase ^= 1u;
    auto scores = [&](int k) {
      const int t = tile0 + (MODE == kTwoQ ? k >> 1 : k), idx = 2 * t, st = idx % l.stages;
      if (!tc::mbar_wait(tc::su32(&sm.full[st]), (uint32_t)(idx / l.stages) & 1u, abort)) return false;
      tc::tc_fence_after();
      const uint32_t q = base + (MODE == kTwoQ ? (uint32_t)(k & 1) * l.chunks * 16384 : 0u);
      const uint64_t da = tc::desc_sw128(q), db = tc::desc_sw128(ring0 + (uint32_t)st * l.stage_bytes);
      const uint32_t d = tmem + (uint32_t)((k & 1) * KT);
      for (int kk = 0; kk < ks; ++kk)
        tc::tc_mma(d, da + (uint64_t)(((kk >> 2) * 16384 + (kk & 3) * 32) >> 4),
                   db + (uint64_t)(((kk >> 2) * KT * 128 + (kk & 3) * 32) >> 4), id_s, kk > 0);
      tc::tc_commit(tc::su32(&sm.s_full[k & 1]));
      if (MODE != kTwoQ || (k & 1)) tc::tc_commit(tc::su32(&sm.empty[st]));
      if (k == jobs - 1) tc::tc_commit(tc::su32(&sm.q_empty));
      return true;
    };
    ok = scores(0) && (jobs < 2 || scores(1));
    for (int k = 0; ok && k < jobs; ++k) {
      const int buf = k & 1, acc = MODE == kWide ? 0 : buf;
      if (!(ok = tc::mbar_wait(tc::su32(&sm.p_full[buf]), p_phase[buf], abort))) break;
      p_phase[buf] ^= 1u;
      const bool fresh = MODE == kWide ? k == 0 : k < 2;
      // the last item's accumulator has been read
      if (fresh && !first) {
        if (!(ok = tc::mbar_wait(tc::su32(&sm.o_free[acc]), free_phase[acc], abort))) break;
        free_phase[acc] ^= 1u;
      }
      const int t = tile0 + (MODE == kTwoQ ? k >> 1 : k), idx = 2 * t + 1, st = idx % l.stages;
      if (!(ok = tc::mbar_wait(tc::su32(&sm.full[st]), (uint32_t)(idx / l.stages) & 1u, abort))) break;
      tc::tc_fence_after();
      const uint64_t db = desc_values(ring0 + (uint32_t)st * l.stage_bytes, KT * 128);
      const uint32_t d = tmem + (uint32_t)(acc ? S::O1 : S::O0), p = tmem + (uint32_t)(buf * KT);
#pragma unroll
      for (int kk = 0; kk < KT / 16; ++kk)
        tc_mma_ts(d, p + 8 * kk, db + (uint64_t)(kk * 2048 >> 4), id_o, !fresh || kk > 0);
      if (MODE != kTwoQ || buf) tc::tc_commit(tc::su32(&sm.empty[st]));
      if (MODE == kWide || k >= jobs - 2) tc::tc_commit(tc::su32(&sm.o_done[acc]));
      if (k + 2 < jobs) ok = scores(k + 2);
    }
    // (kOneQ with a single tile: the second accumulator is not used, nor waited for)
    if (MODE == kOneQ && jobs == 1 && ok && !first) {
      ok = tc::mbar_wait(tc::su32(&sm.o_free[1]), free_phase[1], abort);
      free_phase[1] ^= 1u;
    }
    first = false;
    tile0 += nt;
  }
  // the copies' stages and TMEM are given back only when every MMA has ended
  tc::tc_commit(tc::su32(&sm.drain));
  tc::mbar_wait(tc::su32(&sm.drain), 0, abort, false);
}

// ---------------------------------------------------------------- softmax warpgroups
// Weights are 2^(s - m + kShift) against a reference m, which follows the running maximum only when that has gone more
// than kSlack past it: then the sums and outputs are rescaled, as they seldom are.  f16 weights stay below 2^15 and lose
// what is under 2^-34 of the largest; bf16 has fp32's exponents.
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

  SPEC_DEV Softmax(const Args& g_, TcSmem& sm_, uint32_t tmem, int w_, int warp_, int lane_)
      : g(g_), sm(sm_), w(w_), warp(warp_), lane(lane_), row(warp_ * 32 + lane_), tm(tmem + ((uint32_t)(warp_ * 32) << 16)) {}

  // The warps that write an item together: a warpgroup, or both (kOneQ).  Bounded as every wait.
  uint32_t group_phase = 0;
  SPEC_DEV bool group_sync() {
    const uint32_t a = tc::su32(&sm.group[MODE == kOneQ ? 0 : w]);
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(a);
    const bool ok = tc::mbar_wait(a, group_phase, &sm.abort);
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

  // One tile: scores in TMEM columns s0 -> weights there.  o0: the accumulator; fresh: nothing is in it.
  // done: waits until the products of the last tile are in the accumulator (kWide).
  template <typename Done> SPEC_DEV void tile(const Item& it, int tile, int bits, uint32_t s0, uint32_t o0, bool fresh,
                                              int klo, int khi, Done&& done) {
    float s[KT];
    __syncwarp();
#pragma unroll
    for (int i = 0; i < KT / 32; ++i) tmem_ld32(tm + s0 + 32 * i, s + 32 * i);
    tc::tmem_ld_wait();
    const uint4 there = *reinterpret_cast<const uint4*>(sm.bits[bits]);
    const uint32_t all = KT == 128 ? there.x & there.y & there.z & there.w : there.x & there.y;
    if (edge_tile(g, it, tile, KT) || all != 0xffffffffu) {
      const int key0 = tile * KT;
#pragma unroll
      for (int i = 0; i < KT / 32; ++i) {
        const uint32_t seen = span(klo - key0, khi - key0, i) & (i == 0 ? there.x : i == 1 ? there.y : i == 2 ? there.z : there.w);
#pragma unroll
        for (int j = 0; j < 32; ++j) s[32 * i + j] = seen & (1u << j) ? s[32 * i + j] : -INFINITY;
      }
    }
    float top[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
    for (int i = 4; i < KT; ++i) top[i & 3] = fmaxf(top[i & 3], s[i]);
    const float now = fmaxf(fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * g.scale2, m);
    bool in = fresh;
    if (fresh) {
      m = now;
    } else if (__any_sync(0xffffffffu, now > m + W::kSlack)) {
      const float f = m == -INFINITY ? 1.f : exp2_fast(m - now);
      if (!done()) return;
      in = true;
      tc::tc_fence_after();
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
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < KT / 32; ++i) {
      uint32_t p[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const float a = exp2_fast(fmaf(s[32 * i + 2 * j], g.scale2, base));
        const float b = exp2_fast(fmaf(s[32 * i + 2 * j + 1], g.scale2, base));
        sum[(2 * j) & 3] += a, sum[(2 * j + 1) & 3] += b;
        p[j] = pack2<T>(a, b);
      }
      tmem_st16(tm + s0 + 16 * i, p);
    }
    tmem_st_wait();
    l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
    if (!in) done();                       // every phase is waited for in its turn
  }

  // A value that is not finite, of a key of an edge tile that the row attends to
  SPEC_DEV void mend(const Item& it, int item, int klo, int khi, int c0, float* o) {
    for (int e = 0; e < 2 * S::EDGES; ++e)
      for (int i = 0; i < KT / 32; ++i)
        for (uint32_t b = sm.poison[item][e][i]; b; b &= b - 1) {
          const int key = edge_tile_of<S::EDGES, KT>(g, it, e) * KT + 32 * i + __ffs(b) - 1;
          if (key < klo || key >= khi) continue;
          const long long at = (slot_of(g.kv, g.b0 + it.b, key) * g.nkv + it.h) * g.hd + c0;
          for (int j = 0; j < 16; ++j) {
            float v;
            if constexpr (F8) v = (float)static_cast<const __nv_fp8_e4m3*>(g.kv.v)[at + j];
            else v = (float)static_cast<const T*>(g.kv.v)[at + j];
            if (not_finite(v)) o[j] = NAN;
          }
        }
  }

  // 16 components of the row's unnormalised output
  SPEC_DEV void take(float* o, int c, float f0, float f1, bool two) {
    __syncwarp();
    uint32_t a[16];
    if (MODE == kTwoQ) {
      tc::tmem_ld16(tm + (w ? S::O1 : S::O0) + c, a);
      tc::tmem_ld_wait();
#pragma unroll
      for (int j = 0; j < 16; ++j) o[j] = __uint_as_float(a[j]);
    } else {
      tc::tmem_ld16(tm + S::O0 + c, a);
      uint32_t b[16];
      if (MODE == kOneQ && two) tc::tmem_ld16(tm + S::O1 + c, b);
      tc::tmem_ld_wait();
#pragma unroll
      for (int j = 0; j < 16; ++j) o[j] = __uint_as_float(a[j]) * f0;
      if (MODE == kOneQ && two)
#pragma unroll
        for (int j = 0; j < 16; ++j) o[j] = fmaf(__uint_as_float(b[j]), f1, o[j]);
    }
  }

  SPEC_DEV void write(const Item& it, int r, int c, const float* o, float inv) {
    const int tok = (it.r0 + r) / g.G, head = it.h * g.G + (it.r0 + r) - tok * g.G;
    uint4* dst = reinterpret_cast<uint4*>(static_cast<T*>(g.out) + (it.row0 + tok) * g.out_ld + (long long)head * g.hd + c);
    uint32_t u[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) u[j] = pack2<T>(o[2 * j] * inv, o[2 * j + 1] * inv);
    dst[0] = make_uint4(u[0], u[1], u[2], u[3]);
    dst[1] = make_uint4(u[4], u[5], u[6], u[7]);
  }
  SPEC_DEV void write_lse(const Item& it, int r, float m_, float l_) {
    if (!g.lse) return;
    const int tok = (it.r0 + r) / g.G, head = it.h * g.G + (it.r0 + r) - tok * g.G;
    g.lse[(long long)(it.row0 + tok) * g.nq + head] = l_ == 0.f ? -INFINITY : (m_ - W::kShift + log2f(l_)) * kLn2;
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
    const Pieces pc(sm.plan, it);
    if (pc.c0 == pc.c1) {
      const float inv = l == 0.f ? 0.f : g.v_scale / l;
      for (int c = c0; c < c1; c += 16) {
        float o[16];
        take(o, c, f0, f1, two);
        if (poisoned && valid) mend(it, item, klo, khi, c, o);
        if (valid) write(it, r, c, o, inv);
      }
      if (valid && c0 == 0) write_lse(it, r, m, l);
      release();
      return true;
    }
    const size_t piece = piece_floats(BM, g.hd);
    float* mine = g.part + pc.slot(sm.plan, it, blockIdx.x) * piece;
    for (int c = c0; c < c1; c += 16) {
      float o[16];
      take(o, c, f0, f1, two);
      if (poisoned && valid) mend(it, item, klo, khi, c, o);
      if (valid)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *reinterpret_cast<float4*>(mine + ((size_t)(c / 4 + j) * BM + r) * 4) =
              make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
    }
    if (valid && c0 == 0) mine[(size_t)BM * g.hd + r] = m, mine[(size_t)BM * (g.hd + 1) + r] = l;
    release();
    __threadfence();
    const int slot = MODE == kOneQ ? 0 : w;
    if (!group_sync()) return false;
    if (row == 0 && (MODE != kOneQ || w == 0)) {
      const long long at = (long long)it.h * sm.plan.pairs[g.B] + sm.plan.pairs[it.b] + it.t;
      int* counter = g.counters + (MODE == kTwoQ ? 2 * at + w : at);
      const int before = atomicAdd(counter, 1);
      sm.last[slot] = before == pc.c1 - pc.c0;
      if (sm.last[slot]) *counter = 0;
    }
    if (!group_sync()) return false;
    const bool last = sm.last[slot] != 0;
    if (!group_sync()) return false;       // (read before the next item's is written)
    if (!last || !valid) return true;
    __threadfence();
    float M = -INFINITY;
    for (int c = pc.c0; c <= pc.c1; ++c)
      M = fmaxf(M, __ldcg(g.part + pc.slot(sm.plan, it, c) * piece + (size_t)BM * g.hd + r));
    float L = 0.f;
    for (int c = pc.c0; c <= pc.c1; ++c) {
      const float* x = g.part + pc.slot(sm.plan, it, c) * piece + (size_t)BM * g.hd + r;
      const float mc = __ldcg(x);
      L += __ldcg(x + BM) * (mc == -INFINITY ? 0.f : exp2_fast(mc - base_of(M)));
    }
    const float inv = L == 0.f ? 0.f : g.v_scale / L;
    for (int c = c0; c < c1; c += 16) {
      float o[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) o[j] = 0.f;
      for (int p = pc.c0; p <= pc.c1; ++p) {
        const float* x = g.part + pc.slot(sm.plan, it, p) * piece;
        const float mc = __ldcg(x + (size_t)BM * g.hd + r), f = mc == -INFINITY ? 1.f : exp2_fast(mc - base_of(M));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float4 v = __ldcg(reinterpret_cast<const float4*>(x + ((size_t)(c / 4 + j) * BM + r) * 4));
          o[4 * j] = fmaf(v.x, f, o[4 * j]), o[4 * j + 1] = fmaf(v.y, f, o[4 * j + 1]);
          o[4 * j + 2] = fmaf(v.z, f, o[4 * j + 2]), o[4 * j + 3] = fmaf(v.w, f, o[4 * j + 3]);
        }
      }
      write(it, r, c, o, inv);
    }
    if (c0 == 0) write_lse(it, r, M, L);
    return true;
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
    while (walk.next(it)) {
      const int nt = it.k1 - it.k0, item = items % kItems;
      int klo, khi;
      keys_of(g, it, MODE == kTwoQ ? w * 128 + row : row, &klo, &khi);
      m = -INFINITY, l = 0.f;
      bool fresh = true;
      for (int k = MODE == kOneQ ? w : 0; k < nt; k += MODE == kOneQ ? 2 : 1) {
        const int buf = MODE == kWide ? k & 1 : w;
        if (!tc::mbar_wait(tc::su32(&sm.s_full[buf]), s_phase[buf], abort)) return;
        s_phase[buf] ^= 1u;
        tc::tc_fence_after();
        bool ok = true;
        tile(it, it.tile0 + it.k0 + k, (tiles + k) % kTileBits, (uint32_t)(buf * KT),
             MODE == kWide ? S::O0 : w ? S::O1 : S::O0, fresh, klo, khi, [&] {
               // kTwoQ, kOneQ: the scores were asked for after those products
               if (MODE == kWide) ok = tc::mbar_wait(tc::su32(&sm.o_done[0]), o_phase[0] ^ (uint32_t)((k - 1) & 1), abort);
               return ok;
             });
        if (!ok) return;
        arrive(sm.p_full[buf]);
        fresh = false;
      }
      if (MODE == kTwoQ) {
        if (!tc::mbar_wait(tc::su32(&sm.o_done[w]), o_phase[w], abort)) return;
        o_phase[w] ^= 1u;
      } else if (MODE == kOneQ) {
        if (!tc::mbar_wait(tc::su32(&sm.o_done[0]), o_phase[0], abort)) return;
        o_phase[0] ^= 1u;
        if (nt > 1) {
          if (!tc::mbar_wait(tc::su32(&sm.o_done[1]), o_phase[1], abort)) return;
          o_phase[1] ^= 1u;
        }
      } else {
        // a phase a tile
        if (!tc::mbar_wait(tc::su32(&sm.o_done[0]), o_phase[0] ^ (uint32_t)((nt - 1) & 1), abort)) return;
        o_phase[0] ^= (uint32_t)(nt & 1);
      }
      tc::tc_fence_after();
      const bool ok = finish(it, item, klo, khi);
      __syncwarp();
      if (!ok) return;
      if (w == 0) {
        const int old = (items + kItems - 2) % kItems;
        if (row < 2 * 6 * 4) (&sm.poison[old][0][0])[row] = 0;
        if (row == 0) sm.poisoned[old] = 0;
      }
      ++items;
      tiles += nt;
    }
  }
};

template <typename T, bool F8, int MODE> __global__ void __launch_bounds__(kTcThreads, 1)
    chunk_tc_kernel(const __grid_constant__ TcArgs a) {
  SPEC_TL(kTLChunkAttn);
  using S = Shape<MODE>;
  extern __shared__ uint8_t dyn[];
  __shared__ __align__(16) TcSmem sm;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
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
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(tc::su32(&sm.s_full[i]), 1);
      tc::mbar_init(tc::su32(&sm.p_full[i]), 4);
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
  make_plan<S::BM, S::KT>(a.g, sm.plan, tid, kTcThreads);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = sm.tmem;
  if (warp < 8) {
    regs_inc<kSoftmaxRegs>();
    if (MODE != kWide || warp < 4) Softmax<T, F8, MODE>(a.g, sm, tmem, warp >> 2, warp & 3, lane).run();
  } else if (warp < 12) {
    regs_dec<kLoaderRegs>();
    Loader<T, F8, MODE>(a, sm, base, warp - 8, lane).run();
  } else {
    regs_dec<kMmaRegs>();
    if (warp == 12 && lane == 0) issue_mmas<T, MODE>(a, sm, base, tmem);
    __syncwarp();
  }
  tc::tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, 512);
  }
  if (tid == 0 && sm.abort) report(a.g.ws, SPEC_ERR_TIMEOUT, blockIdx.x, 0);
}

typedef void (*TcFn)(TcArgs);
// by type (chunk_attn_<type>.cu)
TcFn tc_kernel_bf16(bool f8, int mode);
TcFn tc_kernel_f16(bool f8, int mode);

template <typename T> TcFn tc_kernel_of(bool f8, int mode) {
  if (f8) return mode == kTwoQ ? chunk_tc_kernel<T, true, kTwoQ> : mode == kOneQ ? chunk_tc_kernel<T, true, kOneQ>
                                                                             : chunk_tc_kernel<T, true, kWide>;
  return mode == kTwoQ ? chunk_tc_kernel<T, false, kTwoQ> : mode == kOneQ ? chunk_tc_kernel<T, false, kOneQ>
                                                                       : chunk_tc_kernel<T, false, kWide>;
}

}  // namespace ca
}  // namespace spec
