// Attention of a chunk of new tokens per request over the paged cache: how a
// call's work is cut and shared out, and how pieces of an item are joined.
//
// The n new tokens of a request and the G query heads of a kv head make n * G
// packed rows (row r: token r / G, head r % G of the group), all over the same
// keys.  An item is one kv head and BM consecutive packed rows; its keys come in
// tiles of KT.  Items lie in a row (kv head, request, packed rows), and the CTAs
// of a launch take equal shares of all tiles in that row: a share begins and ends
// inside items, so few items over a long context are split, and many items end
// at the same time.
#pragma once
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "internal.h"

namespace spec {
namespace ca {

enum : unsigned { kTLChunkAttn = 29 };   // after the other units' ids

constexpr int kMaxB = 1024;              // requests of a launch
constexpr int kWhole = 4;                // tiles of an item that is not cut while there are CTAs for all
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

struct Args {
  spec_kv kv;
  const void* q;
  void* out;
  float* lse;                  // [n_rows, nq] or NULL
  const int32_t *cu, *seq_len;
  long long q_ld, out_ld;
  int B, b0, n_rows, nq, nkv, G, hd, window;
  float scale2;                // softmax scale (and k_scale) times log2(e)
  float v_scale;
  float* part;                 // [grid][2] pieces of piece_floats()
  int* counters;               // [nkv][items of a kv head], zero between calls
  void* ws;
};

// a piece: unnormalised outputs [hd / 4][BM][4], references m [BM], sums l [BM]
__host__ __device__ inline size_t piece_floats(int bm, int hd) { return (size_t)bm * (hd + 2); }

constexpr size_t kPieceFloats = 256 * (128 + 2);   // of an SM's CTAs together, the largest: 256 rows of 128 components

struct Req {
  int row0, n, len;            // first row, new tokens, tokens in the cache
};

// What a launch's arrays say of request b, with bad values clamped.
SPEC_DEV Req request(const Args& g, int b, bool* bad = nullptr) {
  const int a = g.cu[g.b0 + b], e = g.cu[g.b0 + b + 1], len = g.seq_len[g.b0 + b];
  Req r;
  r.row0 = min(max(a, 0), g.n_rows);
  r.n = min(max(e, r.row0), g.n_rows) - r.row0;
  r.len = min(max(len, 0), g.kv.max_blocks * g.kv.block_size);
  if (bad) *bad = r.row0 != a || r.row0 + r.n != e || r.len != len;
  return r;
}

// One item's share in a CTA: tiles [k0, k1) of its `tiles`.
struct Item {
  int h, b, t;
  int row0, r0, rows;          // the request's first row; the first packed row and how many
  int first;                   // cache index of the request's first new token
  int lo, hi;                  // keys that any row attends to: [lo, hi)
  int tile0, tiles;            // key tiles: tile0 .. tile0 + tiles - 1
  int k0, k1;
  long long pos;               // place of the item's first tile in the row of all tiles
};

template <int BM, int KT> SPEC_DEV void geometry(const Args& g, const Req& r, int t, Item& it) {
  it.t = t;
  it.row0 = r.row0;
  it.r0 = t * BM;
  it.rows = min(BM, r.n * g.G - it.r0);
  it.first = r.len - r.n;
  const int p0 = it.first + it.r0 / g.G, p1 = it.first + (it.r0 + it.rows - 1) / g.G;
  it.hi = max(0, p1 + 1);
  it.lo = g.window > 0 ? max(0, min(p0 - g.window + 1, it.hi)) : 0;
  it.tile0 = it.lo / KT;
  it.tiles = max(1, (it.hi + KT - 1) / KT - it.tile0);
}

// The launch's plan, in shared memory of every CTA.
struct Plan {
  long long work[kMaxB + 1];   // prefix sums of the tiles of a kv head by request
  int pairs[kMaxB + 1];        // prefix sums of the items of a kv head by request
  long long total, begin, end; // tiles in all, and this CTA's
  int ctas;
  int longest;                 // tiles of an item, at most
  bool whole;                  // an item a CTA
  int h, b, t, off;            // where this CTA begins
};

SPEC_DEV int owner(const Plan& p, long long x) { return (int)(((x + 1) * p.ctas - 1) / p.total); }

// All threads of the block.  A few thousand integers at most are read, from L2.  Where rows fall from a request to the
// next, requests overlap, and their items may be more than there are counters: then none has any.
template <int BM, int KT> SPEC_DEV void make_plan(const Args& g, Plan& p, int tid, int threads) {
  int falls = 0;
#pragma unroll 1
  for (int b = tid; b < g.B; b += threads) {
    bool bad;
    falls |= g.cu[g.b0 + b + 1] < g.cu[g.b0 + b];
    const Req r = request(g, b, &bad);
    if (bad && blockIdx.x == 0) report(g.ws, SPEC_ERR_DEVICE, g.b0 + b, r.len);
    p.pairs[b + 1] = (int)(((long long)r.n * g.G + BM - 1) / BM);
    p.work[b + 1] = 0;
  }
  if (tid == 0) p.pairs[0] = 0, p.work[0] = 0, p.longest = 0;
  falls = __syncthreads_or(falls);
  if (tid < 32) {
    int run = 0;
#pragma unroll 1
    for (int b0 = 0; b0 < g.B; b0 += 32) {
      int x = b0 + tid < g.B && !falls ? p.pairs[b0 + tid + 1] : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (tid >= o) x += y;
      }
      if (b0 + tid < g.B) p.pairs[b0 + tid + 1] = run + x;
      run += __shfl_sync(0xffffffffu, x, 31);
    }
  }
  __syncthreads();
  const int items = p.pairs[g.B];
#pragma unroll 1
  for (int i = tid; i < items; i += threads) {
    int lo = 0, hi = g.B;      // the request whose items hold i
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (p.pairs[mid] <= i) lo = mid;
      else hi = mid;
    }
    Item it;
    geometry<BM, KT>(g, request(g, lo), i - p.pairs[lo], it);
    atomicAdd(reinterpret_cast<unsigned long long*>(&p.work[lo + 1]), (unsigned long long)it.tiles);
    atomicMax(&p.longest, it.tiles);
  }
  __syncthreads();
  if (tid < 32) {
    long long run = 0;
#pragma unroll 1
    for (int b0 = 0; b0 < g.B; b0 += 32) {
      long long x = b0 + tid < g.B ? p.work[b0 + tid + 1] : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (tid >= o) x += y;
      }
      if (b0 + tid < g.B) p.work[b0 + tid + 1] = run + x;
      run += __shfl_sync(0xffffffffu, x, 31);
    }
    __syncwarp();
    const long long one = run, total = one * g.nkv, all_items = (long long)items * g.nkv;
    const int c = blockIdx.x;
    // Short items that have a CTA each stay whole: 32 items of 2 or 3 tiles, in shares of one tile 16.3 us,
    // whole 13.0.
    const bool whole = all_items <= gridDim.x && p.longest <= kWhole;
    const int ctas = whole ? (int)max(1ll, all_items) : (int)max(1ll, min((long long)gridDim.x, total));
    long long begin = c < ctas ? total * c / ctas : total, end = c < ctas ? total * (c + 1) / ctas : total;
    int h = 0, b = 0, t = 0;
    long long rem = 0;
    if (whole) {
      begin = end = 0;
      if (c < all_items) {
        h = c / items;
        const int i = c - h * items;
        int lo = 0, hi = g.B;
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (p.pairs[mid] <= i) lo = mid;
          else hi = mid;
        }
        b = lo, t = i - p.pairs[lo];
        Item it;
        geometry<BM, KT>(g, request(g, b), t, it);
        end = it.tiles;
      }
    } else if (begin < end) {
      h = (int)(begin / one);
      rem = begin - h * one;
      int lo = 0, hi = g.B;    // the last request whose prefix is at or below: it has tiles
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.work[mid] <= rem) lo = mid;
        else hi = mid;
      }
      b = lo;
      rem -= p.work[b];
      const Req r = request(g, b);
      const int n = p.pairs[b + 1] - p.pairs[b];
#pragma unroll 1
      for (int t0 = 0; t0 < n; t0 += 32) {
        Item it;
        it.tiles = 0;
        if (t0 + tid < n) geometry<BM, KT>(g, r, t0 + tid, it);
        int x = it.tiles;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, x, o);
          if (tid >= o) x += y;
        }
        const int all = __shfl_sync(0xffffffffu, x, 31);
        if (rem >= all) {
          rem -= all;
          continue;
        }
        const int who = __ffs(__ballot_sync(0xffffffffu, x > rem)) - 1;
        t = t0 + who;
        rem -= __shfl_sync(0xffffffffu, x - it.tiles, who);
        break;
      }
    }
    if (tid == 0) {
      p.total = total, p.begin = begin, p.end = end, p.ctas = ctas, p.whole = whole;
      p.h = h, p.b = b, p.t = t, p.off = (int)rem;
    }
  }
  __syncthreads();
}

// The items of this CTA's share, in order; every role walks them for itself.
template <int BM, int KT> struct Walk {
  const Args& g;
  const Plan& p;
  int h, b, t, off;
  long long at;
  SPEC_DEV Walk(const Args& g_, const Plan& p_) : g(g_), p(p_), h(p_.h), b(p_.b), t(p_.t), off(p_.off), at(p_.begin) {}
  SPEC_DEV bool next(Item& it) {
    if (at >= p.end) return false;
    while (p.pairs[b + 1] - p.pairs[b] <= t) {
      t = 0;
      if (++b == g.B) b = 0, ++h;
    }
    it.h = h, it.b = b;
    geometry<BM, KT>(g, request(g, b), t, it);
    it.k0 = off;
    it.k1 = (int)min((long long)it.tiles, off + (p.end - at));
    it.pos = at - off;
    at += it.k1 - it.k0;
    off = 0;
    ++t;
    return true;
  }
};

// Where the pieces of an item are: CTAs c0 .. c1, each in its first or second slot.
struct Pieces {
  int c0, c1;
  SPEC_DEV Pieces(const Plan& p, const Item& it)
      : c0(p.whole ? 0 : owner(p, it.pos)), c1(p.whole ? 0 : owner(p, it.pos + it.tiles - 1)) {}
  // (the first CTA's share begins before the item or with it, the others' inside)
  SPEC_DEV int slot(int c) const { return 2 * c + (c == c0 ? 1 : 0); }
};

// keys that packed row r of an item attends to: [lo, hi)
SPEC_DEV void keys_of(const Args& g, const Item& it, int r, int* lo, int* hi) {
  const int p = it.first + (it.r0 + r) / g.G;
  *hi = p + 1;
  *lo = g.window > 0 ? max(0, p + 1 - g.window) : 0;
}

// An item's edge tiles: those that some row does not attend to all keys of.  By number: the ones at its newest keys,
// then (from EDGES on) the ones at its window's start.
template <int KT> struct Edges {
  int from, below, tile_a, tile_b;     // keys at or past `from`, and below `below`, are not for all rows
  SPEC_DEV Edges() {}
  SPEC_DEV Edges(const Args& g, const Item& it) {
    const int p0 = it.first + it.r0 / g.G, p1 = it.first + (it.r0 + it.rows - 1) / g.G;
    from = p0 + 1;
    below = g.window > 0 ? p1 + 1 - g.window : 0;
    tile_a = max(0, from) / KT;
    tile_b = it.tile0;
  }
  SPEC_DEV bool has(int tile) const { return (tile + 1) * KT > from || tile * KT < below; }
  template <int EDGES> SPEC_DEV int slot(int tile) const { return (tile + 1) * KT > from ? tile - tile_a : EDGES + tile - tile_b; }
  template <int EDGES> SPEC_DEV int tile(int slot) const { return slot < EDGES ? tile_a + slot : tile_b + slot - EDGES; }
};

// reference of the exponents: finite also where nothing has been seen
SPEC_DEV float base_of(float m) { return m == -INFINITY ? 0.f : m; }
SPEC_DEV float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// One component of 16 or 32 bits that is not finite
SPEC_DEV bool not_finite(float x) { return !(fabsf(x) <= 3.402823466e38f); }

}  // namespace ca
}  // namespace spec
