// Beam search over the paged cache: the selection over beams and vocabulary, and
// the reordering of the beams' states (block tables, the partial block's K/V rows,
// token histories).
//
// The sources draft greedily or as a tree; a request decoded with beams is not
// speculated on ([NEURON] "Rejection Sampling" verifies one continuation), so its
// steps run through these calls on the same cache.
#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "internal.h"

namespace spec {

enum : unsigned { kTLBeamSelect = 27, kTLBeamReorder = 28 };   // after common.cuh's ids

// ---------------------------------------------------------------- selection
// Within a beam the order of scores is the order of logits, so a row's chunk needs
// only its W largest logits and its sum of exponentials: one pass over the logits,
// bound by their bytes.  Each warp streams tiles of 1024 logits into registers, the
// next tile's loads on their way while it works on one, with no barrier in the loop.
// A lane's 32 logits of a tile are a group, whose maximum the running sum needs
// anyway; it goes to shared memory.  The W largest logits lie in the W groups with
// the largest maxima, so the search for them is over 1/32 of the chunk, and only the
// few groups that are left are read again.  The last chunk of a request to finish (a
// counter, nobody waits) merges the request.
//
// log sum exp = m + log(sum of e^(x - m)), m the running maximum.  Measured: 32 x 8 rows of 151936 of random
// logits, fp32 33.6 us (4.6 TB/s; the stream ~23, a chunk's end ~5 under load: bound, second look at the kept
// groups, counter; the request's merge ~3), bf16 23; 4 rows of 128256 8.5 us, all latency: the first loads,
// the chunk's end, counter and merge are ~12 dependent trips to memory or across the block.
//
// Which lane has which element of a tile does not depend on the row's alignment, and
// rows are cut into equal chunks, so equal rows give equal sums and tie as they
// should.
constexpr int kSelWarps = 4, kSelThreads = kSelWarps * 32;
constexpr int kSelElems = 32;                               // logits of a group
constexpr int kSelTile = 32 * kSelElems;
constexpr int kSelChunk = 128 * kSelTile;                   // at most in a chunk
constexpr int kSelCap = 512;                                // entries of a candidate list
constexpr float kLog2e = 1.4426950408889634f;

// the requests' counters lie in the same place whatever a call's sizes (B W < 2^16), so that calls of
// any sizes share a workspace
constexpr size_t kSelCounterBytes = 65536 * 4;

struct SelArgs {
  int B, W, V, nch, chunk, eos;
  long long ld;
  const void* logits;
  const float* score;
  const int32_t* done;
  int32_t *parent, *tok, *done_out;
  float* score_out;
  int* counters;      // [B]
  float2* stats;      // [B * W, nch]  largest logit r, sum of exp(x - r)
  float2* cand;       // [B * W, nch, W]  logit, token id (bits)
};

SPEC_DEV bool finite(float x) { return fabsf(x) <= 3.402823466e38f; }
SPEC_DEV float cvt(float x) { return x; }
SPEC_DEV float cvt(__nv_bfloat16 x) { return __bfloat162float(x); }
SPEC_DEV float cvt(__half x) { return __half2float(x); }
SPEC_DEV float pow2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Values are ordered as unsigned integers (0 is below every number and stands for no
// candidate): fp64 comparisons would go through the slow fp64 units.  -0 equals +0.
SPEC_DEV uint32_t key_of(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);
  return x == -INFINITY ? 0u : ((u >> 31) ? ~u : u | 0x80000000u);
}
SPEC_DEV float value_of(uint32_t k) { return k == 0 ? -INFINITY : __uint_as_float((k >> 31) ? k & 0x7fffffffu : ~k); }
SPEC_DEV uint64_t key_of(double x) {
  const uint64_t u = (uint64_t)__double_as_longlong(x + 0.0);
  return (u >> 63) ? ~u : u | 0x8000000000000000ull;
}
SPEC_DEV double value_of(uint64_t k) {
  return __longlong_as_double((long long)((k >> 63) ? k & 0x7fffffffffffffffull : ~k));
}
// a place in the order: larger value first, then smaller index
template <typename K> SPEC_DEV bool ahead(K v, int i, K w, int j) { return v > w || (v == w && i < j); }

struct SelShared {
  uint64_t key[kSelCap], entry[kSelCap];
  int idx[kSelCap];
  uint64_t kred[kSelWarps];
  uint32_t bound[kSelWarps];
  int ired[kSelWarps];
  float fred[2][kSelWarps];
  int count, groups, last;
  float border;
  float score[32];    // of the request's beams; -infinity: none
  int done[32];
  double lse[32];
};

// A lower bound of the block's k-th largest value from the threads' maxima: a warp's
// k-th largest is reached by k values, and so is the largest of those over the warps.
// In two steps, the caller's barrier between them.
SPEC_DEV void leave_bound(uint32_t mine, int k, SelShared& sm) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int rank = 0;
#pragma unroll
  for (int o = 1; o < 32; ++o) {
    const uint32_t w = __shfl_sync(0xffffffffu, mine, (lane + o) & 31);
    rank += w > mine || (w == mine && ((lane + o) & 31) < lane);
  }
  if (rank == k - 1) sm.bound[warp] = mine;
}
SPEC_DEV uint32_t block_bound(const SelShared& sm) {
  uint32_t b = sm.bound[0];
#pragma unroll
  for (int w = 1; w < kSelWarps; ++w) b = max(b, sm.bound[w]);
  return b;
}

// The block's k best of `lists` lists of up to k (key, index) entries, each in
// descending order: get(place, index) is the key of an entry, lists one after another, 0 past a list's end;
// first(e, place, index) the same of the e-th that a thread can hold.
// They go, in order, to the front of the shared list; sm.count is how many there are.
// Entries at or above a bound are collected and ranked by counting; if those overflow
// the list, k rounds of block-wide maxima.  The bound comes from the threads' maxima
// over all entries where those can be held in registers between the two looks, else
// over the lists' heads, so that only lists whose head reaches it are read (16 beams:
// 512 entries 28.8 us against 35.7 by heads; 2560 entries 17.1 by heads against 35.8 by all entries).
constexpr int kHeld = 8;
SPEC_DEV bool can_hold(int k, int lists) { return lists * k <= kHeld * kSelThreads; }
template <typename First, typename Get> SPEC_DEV void block_best(int k, int lists, First first, Get get, SelShared& sm) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) sm.count = sm.groups = 0;
  auto keep = [&](uint64_t x, int i) {
    const int at = atomicAdd(&sm.count, 1);
    if (at < kSelCap) sm.key[at] = x, sm.idx[at] = i;
  };
  auto shared_bound = [&](uint64_t mine) {
    leave_bound((uint32_t)(mine >> 32), k, sm);                // of the keys' upper halves
    __syncthreads();
    const uint64_t bound = (uint64_t)block_bound(sm) << 32;
    return bound == 0 ? (uint64_t)1 : bound;
  };
  int open = 0;                                                // lists that were read
  uint64_t mine = 0;
  if (can_hold(k, lists)) {
    uint64_t held[kHeld];
    int at_of[kHeld];
#pragma unroll
    for (int e = 0; e < kHeld; ++e) {
      const int at = tid + e * kSelThreads;
      held[e] = 0;
      if (at < lists * k) held[e] = first(e, at, at_of[e]);
      mine = held[e] > mine ? held[e] : mine;
    }
    const uint64_t bound = shared_bound(mine);
#pragma unroll
    for (int e = 0; e < kHeld; ++e)
      if (held[e] >= bound) keep(held[e], at_of[e]);
  } else {
    for (int l = tid; l < lists; l += kSelThreads) {
      int i;
      const uint64_t x = get(l * k, i);
      mine = x > mine ? x : mine;
    }
    const uint64_t bound = shared_bound(mine);
    if (mine >= bound)
      for (int l = tid; l < lists; l += kSelThreads) {
        int i;
        if (get(l * k, i) < bound) continue;
        const int at = atomicAdd(&sm.groups, 1);
        if (at < kSelCap) sm.entry[at] = (uint64_t)l;
      }
    __syncthreads();
    open = sm.groups;
    for (int e = tid; e < min(open, kSelCap) * k; e += kSelThreads) {
      int i;
      const uint64_t x = get((int)sm.entry[e / k] * k + e % k, i);
      if (x >= bound) keep(x, i);
    }
  }
  __syncthreads();
  int count = sm.count;
  if (count > kSelCap || open > kSelCap) {
    uint64_t pv = ~0ull;
    int pi = -1;
    for (count = 0; count < k; ++count) {
      uint64_t v = 0;
      int at = 0x7fffffff;
      for (int e = tid; e < lists * k; e += kSelThreads) {
        int i;
        const uint64_t x = get(e, i);
        if (x > 0 && ahead(pv, pi, x, i) && ahead(x, i, v, at)) v = x, at = i;
      }
      for (int o = 16; o > 0; o >>= 1) {
        const uint64_t w = __shfl_xor_sync(0xffffffffu, v, o);
        const int j = __shfl_xor_sync(0xffffffffu, at, o);
        if (ahead(w, j, v, at)) v = w, at = j;
      }
      __syncthreads();
      if (lane == 0) sm.kred[warp] = v, sm.ired[warp] = at;
      __syncthreads();
      v = sm.kred[0], at = sm.ired[0];
      for (int w = 1; w < kSelWarps; ++w)
        if (ahead(sm.kred[w], sm.ired[w], v, at)) v = sm.kred[w], at = sm.ired[w];
      if (v == 0) break;
      if (tid == 0) sm.key[count] = v, sm.idx[count] = at;
      pv = v;
      pi = at;
    }
    __syncthreads();
    if (tid == 0) sm.count = count;
    __syncthreads();
    return;
  }
  constexpr int kPer = kSelCap / kSelThreads;
  uint64_t v[kPer];
  int i[kPer], rank[kPer];
#pragma unroll
  for (int e = 0; e < kPer; ++e) {
    const int a = tid + e * kSelThreads;
    rank[e] = k;
    if (a < count) {
      v[e] = sm.key[a];
      i[e] = sm.idx[a];
      rank[e] = 0;
#pragma unroll 4
      for (int b = 0; b < count; ++b) rank[e] += ahead(sm.key[b], sm.idx[b], v[e], i[e]);
    }
  }
  __syncthreads();
#pragma unroll
  for (int e = 0; e < kPer; ++e)
    if (rank[e] < k) sm.key[rank[e]] = v[e], sm.idx[rank[e]] = i[e];
  if (tid == 0) sm.count = min(count, k);
  __syncthreads();
}

// A tile's logits as a lane holds them: loads of 16 bytes (single elements where the
// row is not aligned to that), consecutive lanes side by side.
template <typename T> struct SelTile {
  static constexpr int P = 16 / sizeof(T), N = kSelElems / P;
  uint4 raw[N];
  // element e of lane `lane`
  SPEC_DEV static int pos(int e, int lane) { return (e / P) * 32 * P + lane * P + e % P; }
  // n: elements of the tile that exist; the others become the type's -infinity.  A row off the 16-byte
  // grid is read in words, a 16-bit one off the 4-byte grid in words that straddle its elements (not where
  // that would reach over the row's ends: `inner`, an element before the tile and one after it are the row's)
  SPEC_DEV void load(const T* p, int n, bool inner) {
    const int lane = threadIdx.x & 31;
    const uint32_t off = (uint32_t)reinterpret_cast<uintptr_t>(p);
    if (n >= kSelTile && (off & 15) == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) raw[i] = __ldcs(reinterpret_cast<const uint4*>(p + pos(i * P, lane)));
    } else if (n >= kSelTile && (off & 3) == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const uint32_t* q = reinterpret_cast<const uint32_t*>(p + pos(i * P, lane));
        raw[i] = make_uint4(q[0], q[1], q[2], q[3]);
      }
    } else if (n >= kSelTile && inner) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const uint32_t* q = reinterpret_cast<const uint32_t*>(p + pos(i * P, lane) - 1);
        uint32_t w[5];
#pragma unroll
        for (int j = 0; j < 5; ++j) w[j] = q[j];
        raw[i] = make_uint4(__funnelshift_r(w[0], w[1], 16), __funnelshift_r(w[1], w[2], 16),
                            __funnelshift_r(w[2], w[3], 16), __funnelshift_r(w[3], w[4], 16));
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        T v[P];
#pragma unroll
        for (int j = 0; j < P; ++j) v[j] = pos(i * P + j, lane) < n ? p[pos(i * P + j, lane)] : lowest();
        raw[i] = *reinterpret_cast<const uint4*>(v);
      }
    }
  }
  SPEC_DEV static T lowest() {
    if constexpr (sizeof(T) == 4) return -INFINITY;
    else if constexpr (std::is_same_v<T, __half>) return __ushort_as_half(0xfc00);
    else return __ushort_as_bfloat16(0xff80);
  }
  SPEC_DEV void values(float* x) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const T* v = reinterpret_cast<const T*>(&raw[i]);
#pragma unroll
      for (int j = 0; j < P; ++j) x[i * P + j] = cvt(v[j]);
    }
  }
};

template <typename T>
__global__ void __launch_bounds__(kSelThreads, 4) beam_select_kernel(const SelArgs g) {
  SPEC_TL(kTLBeamSelect);
  pdl_wait();
  pdl_trigger();
  __shared__ SelShared sm;
  extern __shared__ float maxima[];         // [groups of a chunk]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ch = blockIdx.x, row = blockIdx.y, b = row / g.W, W = g.W;
  if (tid < W) {
    const float sc = g.score[b * W + tid];
    sm.score[tid] = finite(sc) ? sc : -INFINITY;
    sm.done[tid] = g.done[b * W + tid];
  }
  __syncthreads();
  const int beam = row - b * W;
  const bool live = sm.score[beam] > -INFINITY && sm.done[beam] == 0;
  if (live) {
    const T* src = static_cast<const T*>(g.logits) + (long long)row * g.ld;
    const int c0 = ch * g.chunk, c1 = min(g.V, c0 + g.chunk);
    float r = -INFINITY, s = 0.f;           // this lane's largest logit and sum of exp(x - r)
    constexpr int kAhead = sizeof(T) == 4 ? 1 : 2;             // tiles on their way: 4 KB a warp
    constexpr int kStep = kSelWarps * kSelTile;
    SelTile<T> next[kAhead];
    const int mine = c0 + warp * kSelTile;
    auto fetch = [&](SelTile<T>& x, int at) { x.load(src + at, c1 - at, at > 0 && at + kSelTile < g.V); };
#pragma unroll
    for (int a = 0; a < kAhead; ++a)
      if (mine + a * kStep < c1) fetch(next[a], mine + a * kStep);
    for (int base0 = mine; base0 < c1; base0 += kAhead * kStep) {
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {
        const int base = base0 + a * kStep, then = base + kAhead * kStep;
        if (base >= c1) break;
        float x[kSelElems], m = -INFINITY;
        next[a].values(x);
        if (then < c1) fetch(next[a], then);
#pragma unroll
        for (int e = 0; e < kSelElems; ++e) m = fmaxf(m, x[e]);
        auto total = [&](float ref) {
          float a0 = 0.f, a1 = 0.f;
#pragma unroll
          for (int e = 0; e < kSelElems; e += 2) {
            a0 += pow2((x[e] - ref) * kLog2e);
            a1 += pow2((x[e + 1] - ref) * kLog2e);
          }
          return a0 + a1;
        };
        // a NaN or +infinity (not finite: masked) shows up in the sum
        float rn = fmaxf(r, m), add = total(rn == -INFINITY ? 0.f : rn);
        if (!(add <= 2.f * kSelElems)) {
          m = -INFINITY;
#pragma unroll
          for (int e = 0; e < kSelElems; ++e) {
            x[e] = finite(x[e]) ? x[e] : -INFINITY;
            m = fmaxf(m, x[e]);
          }
          rn = fmaxf(r, m);
          add = total(rn == -INFINITY ? 0.f : rn);
        }
        s = r == -INFINITY ? add : fmaf(s, pow2((r - rn) * kLog2e), add);
        r = rn;
        maxima[((base - c0) / kSelTile) * 32 + lane] = m;
      }
    }
    // the chunk's sum, relative to its largest logit; a bound of its W-th largest group maximum
    // from the lanes' largest
    const float rw = warp_max(r);
    s = warp_sum(r == -INFINITY ? 0.f : s * pow2((r - rw) * kLog2e));
    if (lane == 0) sm.fred[0][warp] = rw, sm.fred[1][warp] = s;
    if (tid == 0) sm.count = sm.groups = 0;
    leave_bound(key_of(r), W, sm);
    __syncthreads();
    if (tid == 0) {
      float R = sm.fred[0][0], S = 0.f;
      for (int w = 1; w < kSelWarps; ++w) R = fmaxf(R, sm.fred[0][w]);
      for (int w = 0; w < kSelWarps; ++w)
        if (sm.fred[0][w] > -INFINITY) S += sm.fred[1][w] * pow2((sm.fred[0][w] - R) * kLog2e);
      g.stats[(long long)row * g.nch + ch] = make_float2(R, S);
    }
    // the W groups with the largest maxima (and those that equal the last of them), each lane among its own
    const float bound = value_of(block_bound(sm));
    if (r >= bound && r > -INFINITY) {
      const int groups = (c1 - c0 + kSelTile - 1) / kSelTile * 32;
#pragma unroll 4
      for (int i = tid; i < groups; i += kSelThreads) {
        const float m = maxima[i];
        if (m >= bound && m > -INFINITY) {
          const int at = atomicAdd(&sm.groups, 1);
          if (at < kSelCap) sm.idx[at] = i, sm.key[at] = (uint64_t)key_of(m) << 32 | (uint32_t)at;
        }
      }
    }
    __syncthreads();
    const int found = sm.groups;
    if (tid == 0 && found < W) sm.border = -INFINITY;
    if (found >= W && found <= kSelCap)
      for (int a = tid; a < found; a += kSelThreads) {
        const uint64_t v = sm.key[a];
        int rank = 0;
#pragma unroll 8
        for (int i = 0; i < found; ++i) rank += sm.key[i] > v;
        if (rank == W - 1) sm.border = value_of((uint32_t)(v >> 32));
      }
    if (tid == 0 && found > kSelCap) sm.border = bound;
    __syncthreads();
    const float border = sm.border;
    // an entry: key and index (the smaller first) in one integer
    auto entry = [&](int i) -> uint64_t {
      const float x = cvt(src[i]);
      return finite(x) && x >= border ? (uint64_t)key_of(x) << 32 | (uint32_t)~i : 0ull;
    };
    // their logits that reach the border: the warps take a group each in turn, the lanes its elements
    int kept = 0;
    if (found <= kSelCap) {
      // places of the groups that are kept, in list order; a warp's are read kBatch at a time
      constexpr int kBatch = 4;
      for (int a = 0; a < found; a += 32) {
        const bool in = a + lane < found && maxima[sm.idx[a + lane]] >= border;
        unsigned who = __ballot_sync(0xffffffffu, in);
        while (who != 0) {
          int at[kBatch];
          uint64_t v[kBatch];
#pragma unroll
          for (int e = 0; e < kBatch; ++e) {
            at[e] = c1;
            for (; who != 0 && kept % kSelWarps != warp; who &= who - 1) ++kept;
            if (who == 0) continue;
            const int grp = sm.idx[a + __ffs(who) - 1];
            at[e] = c0 + (grp >> 5) * kSelTile + SelTile<T>::pos(lane, grp & 31);
            who &= who - 1;
            ++kept;
          }
#pragma unroll
          for (int e = 0; e < kBatch; ++e) v[e] = at[e] < c1 ? entry(at[e]) : 0ull;
#pragma unroll
          for (int e = 0; e < kBatch; ++e) {
            const unsigned hit = __ballot_sync(0xffffffffu, v[e] != 0);
            if (hit == 0) continue;
            int to = 0;
            if (lane == 0) to = atomicAdd(&sm.count, __popc(hit));
            to = __shfl_sync(0xffffffffu, to, 0) + __popc(hit & ((1u << lane) - 1));
            if (v[e] != 0 && to < kSelCap) sm.entry[to] = v[e];
          }
        }
      }
    }
    __syncthreads();
    int count = sm.count;
    float2* out = g.cand + ((long long)row * g.nch + ch) * W;
    auto put = [&](int rank, uint64_t v) { out[rank] = make_float2(value_of((uint32_t)(v >> 32)), __int_as_float(~(int)(uint32_t)v)); };
    if (found <= kSelCap && count <= kSelCap) {
      for (int a = tid; a < count; a += kSelThreads) {
        const uint64_t v = sm.entry[a];
        int rank = 0;
#pragma unroll 8
        for (int i = 0; i < count; ++i) rank += sm.entry[i] > v;
        if (rank < W) put(rank, v);
      }
    } else {
      // long runs of equal values: W rounds of block-wide maxima over the chunk
      uint64_t last = ~0ull;
      for (count = 0; count < W; ++count) {
        uint64_t v = 0;
        for (int i = c0 + tid; i < c1; i += kSelThreads) {
          const uint64_t x = entry(i);
          v = x < last && x > v ? x : v;
        }
        for (int o = 16; o > 0; o >>= 1) {
          const uint64_t x = __shfl_xor_sync(0xffffffffu, v, o);
          v = x > v ? x : v;
        }
        __syncthreads();
        if (lane == 0) sm.kred[warp] = v;
        __syncthreads();
        for (int w = 0; w < kSelWarps; ++w) v = sm.kred[w] > v ? sm.kred[w] : v;
        if (v == 0) break;
        if (tid == 0) put(count, v);
        last = v;
      }
    }
    if (tid >= count && tid < W) out[tid] = make_float2(-INFINITY, __int_as_float(0x7fffffff));
  }
  // the request's last CTA merges
  __syncthreads();
  if (tid == 0) {
    int before;
    asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;" : "=r"(before) : "l"(&g.counters[b]) : "memory");
    sm.last = before == W * g.nch - 1;
    if (sm.last) g.counters[b] = 0;
  }
  __syncthreads();
  if (!sm.last) return;
  // the candidates: W lists of each chunk of each beam; on their way while the sums are added up
  const float2* cand = g.cand + (long long)b * W * g.nch * W;
  const int lists = W * g.nch;
  float2 early[kHeld];
  if (can_hold(W, lists)) {
#pragma unroll
    for (int e = 0; e < kHeld; ++e) {
      early[e] = make_float2(-INFINITY, 0.f);
      if (tid + e * kSelThreads < lists * W) early[e] = __ldcg(&cand[tid + e * kSelThreads]);
    }
  }
  // log-sum-exp of every live beam: log2 of the sum with its exponent apart, so that fp32 is enough
  for (int j = warp; j < W; j += kSelWarps) {
    if (sm.score[j] == -INFINITY || sm.done[j] != 0) continue;
    const float2* st = g.stats + (long long)(b * W + j) * g.nch;
    float R = -INFINITY, s = 0.f;
    for (int c = lane; c < g.nch; c += 32) {
      const float2 v = __ldcg(&st[c]);
      const float rn = fmaxf(R, v.x);
      if (rn > -INFINITY) s = s * pow2((R - rn) * kLog2e) + v.y * pow2((v.x - rn) * kLog2e);
      R = rn;
    }
    const float rw = warp_max(R);
    s = warp_sum(R > -INFINITY ? s * pow2((R - rw) * kLog2e) : 0.f);
    if (lane == 0) {
      double l = 0;
      if (s > 0.f) {
        const int e = (int)(__float_as_uint(s) >> 23) - 127;
        l = (double)rw + (double)((float)e) * 0.6931471805599453 +
            (double)(log2f(__uint_as_float(__float_as_uint(s) - ((uint32_t)e << 23))) * 0.69314718f);
      }
      sm.lse[j] = l;
    }
  }
  __syncthreads();
  // scored in fp64
  const float per_beam = (float)(g.nch * W);
  auto scored = [&](int at, float2 x, int& i) -> uint64_t {
    // at / (nch W) in fp32: exact below 2^20
    const int j = at < (1 << 20) ? (int)__fdividef((float)at + 0.5f, per_beam) : at / (g.nch * W);
    const float sc = sm.score[j];
    if (sc == -INFINITY) return 0;
    if (sm.done[j] != 0) {
      i = j * g.V + max(g.eos, 0);
      return at == j * g.nch * W ? key_of((double)sc) : 0;
    }
    if (!(x.x > -INFINITY)) return 0;
    i = j * g.V + __float_as_int(x.y);
    return key_of((double)sc + ((double)x.x - sm.lse[j]));
  };
  block_best(
      W, lists, [&](int e, int at, int& i) { return scored(at, early[e], i); },
      [&](int at, int& i) { return scored(at, __ldcg(&cand[at]), i); }, sm);
  if (tid < W) {
    const int o = b * W + tid;
    if (tid < sm.count) {
      const int i = sm.idx[tid], j = i / g.V;
      const bool fin = sm.done[j] != 0;
      const int t = fin ? g.eos : i - j * g.V;
      g.parent[o] = j;
      g.tok[o] = t;
      g.score_out[o] = (float)value_of(sm.key[tid]);
      g.done_out[o] = fin || t == g.eos;
    } else {
      g.parent[o] = tid;
      g.tok[o] = -1;
      g.score_out[o] = -INFINITY;
      g.done_out[o] = 1;
    }
  }
}

constexpr int kSelSms = 152;
// chunks of a row: the same for every row of a call
static int sel_chunks(int B, int W, int V, int* chunk) {
  constexpr int kStep = kSelWarps * kSelTile;
  const int steps = (V + kStep - 1) / kStep;
  // one chunk an SM (a chunk's end costs ~3 us: 32 x 8 rows of 151936 in fp32, 2 / 4 chunks a row 33.6 / 37.5 us), of
  // at least two steps (merging: 4 rows of 128256 in fp32, 16 / 32 / 64 chunks 8.5 / 9.0 / 9.2 us)
  int want = std::min((kSelSms + B * W - 1) / (B * W), (steps + 1) / 2);
  want = std::max(want, (steps + kSelChunk / kStep - 1) / (kSelChunk / kStep));
  const int per = (steps + want - 1) / want;
  *chunk = per * kStep;
  return (steps + per - 1) / per;
}

// Chunks of all rows, at most, of any batch up to B: fewer rows are cut into more chunks each.  It grows with each of
// the three sizes.
static size_t sel_most_chunks(int B, int W, int V) {
  constexpr int kStep = kSelWarps * kSelTile;
  const long long rows = (long long)B * W, steps = (V + kStep - 1) / kStep;
  return (size_t)std::max(std::min(kSelSms + rows - 1, rows * ((steps + 1) / 2)),
                          rows * ((steps + kSelChunk / kStep - 1) / (kSelChunk / kStep)));
}

// ---------------------------------------------------------------- reordering
constexpr int kMaxLayers = 64;
struct ReorderArgs {
  spec_beam_state s;
  int n_layers, row_bytes, num_blocks, lanes;      // lanes: threads of a copy
  void* k[kMaxLayers];
  void* v[kMaxLayers];
  void* ws;
};

// What a child does with the block that its next token goes to.
struct Tail {
  int parent, n, at, rest;
  int block;       // that block (-1: none)
  int from;        // block whose first `rest` slots are copied into it (-1: none)
  int spare;       // the child's spare block afterwards
};

SPEC_DEV Tail beam_tail(const ReorderArgs& g, int row, bool tell) {
  const spec_beam_state& s = g.s;
  const int b = row / s.W, j = row - b * s.W;
  Tail t;
  t.parent = s.parent[row];
  if (t.parent < 0 || t.parent >= s.W) {
    if (tell) report(g.ws, SPEC_ERR_DEVICE, row, t.parent);
    t.parent = j;
  }
  t.n = s.seq_len[b];
  const int P = s.prompt_blocks[b];
  t.spare = s.spare_in[row];
  t.block = t.from = -1;
  t.at = 0;
  t.rest = 0;
  if (t.n < 0 || P < 0 || (long long)P * s.block_size > t.n) {
    if (tell) report(g.ws, SPEC_ERR_DEVICE, row, t.n);
    t.n = 0;
    return t;
  }
  t.at = t.n / s.block_size;
  t.rest = t.n - t.at * s.block_size;
  if (t.at >= s.max_blocks) {
    if (tell) report(g.ws, SPEC_ERR_CAPACITY, row, t.n);
    t.at = s.max_blocks;
    return t;
  }
  auto checked = [&](int id) {
    if ((unsigned)id < (unsigned)g.num_blocks) return id;
    if (tell) report(g.ws, SPEC_ERR_DEVICE, row, id);
    return -1;
  };
  if (t.rest == 0) {
    const long long o = (long long)P + s.W + (long long)(t.at - P) * s.W + j;
    if (o >= s.owned_ld) {
      if (tell) report(g.ws, SPEC_ERR_CAPACITY, row, (int)o);
      return t;
    }
    t.block = checked(s.owned[(long long)b * s.owned_ld + o]);
    return t;
  }
  const int mine = s.table_in[(long long)row * s.max_blocks + t.at];
  if (t.parent == j) {
    t.block = checked(mine);
    return t;
  }
  t.block = checked(t.spare);
  t.from = checked(s.table_in[((long long)b * s.W + t.parent) * s.max_blocks + t.at]);
  t.spare = mine;
  if (t.block < 0 || t.from < 0) t.block = t.from = -1;
  return t;
}

// Grid (part, row): part 0 writes the row's integers, the others copy the partial
// block's K or V rows, 256 / lanes (layer, K or V)s each; the rows are contiguous
// (slots of a block follow one another).  A copy's source is some beam's current block
// and its target a spare block, and no block is both.  Bound by the copies' bytes where they are many
// (128 beams, 32 layers, up to 32 KB each of K and V: 22.5 us), else by three dependent reads (4 beams: 2.9 us).
__global__ void __launch_bounds__(256) beam_reorder_kernel(const __grid_constant__ ReorderArgs g) {
  SPEC_TL(kTLBeamReorder);
  pdl_wait();
  pdl_trigger();
  const spec_beam_state& s = g.s;
  const int row = blockIdx.y, part = blockIdx.x, tid = threadIdx.x;
  const Tail t = beam_tail(g, row, part == 0 && tid == 0);
  if (part == 0) {
    const long long src = (long long)(row / s.W) * s.W + t.parent;
    const int32_t* in = s.table_in + src * s.max_blocks;
    int32_t* out = s.table_out + (long long)row * s.max_blocks;
    for (int i = tid; i < s.max_blocks; i += 256) out[i] = i < t.at ? in[i] : (i == t.at ? t.block : -1);
    if (s.hist_out) {
      const int32_t* hi = s.hist_in + src * s.hist_ld;
      int32_t* ho = s.hist_out + (long long)row * s.hist_ld;
      for (int i = tid; i < s.hist_ld; i += 256) ho[i] = i < t.n ? hi[i] : (i == t.n ? s.tok[row] : -1);
      if (tid == 0 && t.n >= s.hist_ld) report(g.ws, SPEC_ERR_CAPACITY, row, t.n);
    }
    if (tid == 0) {
      s.spare_out[row] = t.spare;
      s.slots[row] = t.block < 0 ? -1 : t.block * s.block_size + t.rest;
    }
    return;
  }
  const int copy = (part - 1) * (256 / g.lanes) + tid / g.lanes, me = tid % g.lanes;
  if (t.from < 0 || copy >= 2 * g.n_layers) return;
  char* base = static_cast<char*>(copy & 1 ? g.v[copy >> 1] : g.k[copy >> 1]);
  const long long block_bytes = (long long)s.block_size * g.row_bytes;
  const char* from = base + t.from * block_bytes;
  char* to = base + t.block * block_bytes;
  const int bytes = t.rest * g.row_bytes;
  if (((reinterpret_cast<uintptr_t>(base) | g.row_bytes) & 15) == 0) {
    const uint4* f = reinterpret_cast<const uint4*>(from);
    uint4* o = reinterpret_cast<uint4*>(to);
    const int n = bytes >> 4;
    for (int i0 = me; i0 < n; i0 += 4 * g.lanes) {
      uint4 x[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (i0 + j * g.lanes < n) x[j] = __ldcs(f + i0 + j * g.lanes);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (i0 + j * g.lanes < n) o[i0 + j * g.lanes] = x[j];
    }
  } else {
    for (int i = me; i < bytes; i += g.lanes) to[i] = from[i];
  }
}

}  // namespace spec

using namespace spec;

static size_t sel_bytes(size_t chunks, int W) {
  return kWsHeader + kSelCounterBytes + align_up(chunks * 8, 256) + align_up(chunks * W * 8, 256);
}

extern "C" size_t spec_beam_workspace_bytes(int32_t B, int32_t W, int32_t V) {
  if (B <= 0 || W <= 0 || W > 32 || V <= 0 || (long long)W * V >= (1ll << 30)) return 0;
  return sel_bytes(sel_most_chunks(B, W, V), W);
}

extern "C" spec_status spec_beam_select(int32_t B, int32_t W, int32_t V, int32_t dtype, const void* logits, int64_t ld,
                                        const float* score, const int32_t* done, int32_t eos, int32_t* parent,
                                        int32_t* tok, float* score_out, int32_t* done_out, void* ws, size_t ws_bytes,
                                        spec_stream_t stream) {
  if (!logits || !score || !done || !parent || !tok || !score_out || !done_out) return SPEC_ERR_ARG;
  if (score == score_out || done == done_out) return SPEC_ERR_ARG;
  if (dtype < SPEC_DTYPE_F32 || dtype > SPEC_DTYPE_F16) return SPEC_ERR_UNSUPPORTED;
  if (spec_beam_workspace_bytes(B, W, V) == 0 || eos >= V || (long long)B * W > 65535) return SPEC_ERR_SHAPE;
  if (ld == 0) ld = V;
  if (ld < V) return SPEC_ERR_SHAPE;
  if (!aligned(logits, dtype == SPEC_DTYPE_F32 ? 4 : 2)) return SPEC_ERR_ALIGN;
  int chunk;
  const int nch = sel_chunks(B, W, V, &chunk);
  if (!ws || !aligned(ws, 256) || ws_bytes < sel_bytes((size_t)B * W * nch, W)) return SPEC_ERR_WORKSPACE;
  char* p = static_cast<char*>(ws) + kWsHeader;
  SelArgs g{};
  g.B = B, g.W = W, g.V = V, g.nch = nch, g.chunk = chunk, g.eos = eos < 0 ? -1 : eos, g.ld = ld;
  g.logits = logits, g.score = score, g.done = done;
  g.parent = parent, g.tok = tok, g.done_out = done_out, g.score_out = score_out;
  g.counters = reinterpret_cast<int*>(p);
  p += kSelCounterBytes;
  g.stats = reinterpret_cast<float2*>(p);
  p += align_up((size_t)B * W * nch * 8, 256);
  g.cand = reinterpret_cast<float2*>(p);
  auto* kern = dtype == SPEC_DTYPE_F32 ? beam_select_kernel<float>
               : dtype == SPEC_DTYPE_BF16 ? beam_select_kernel<__nv_bfloat16> : beam_select_kernel<__half>;
  launch_pdl(kern, dim3(nch, B * W), dim3(kSelThreads), (size_t)chunk / kSelElems * 4, stream, g);
  return last_launch();
}

extern "C" spec_status spec_beam_reorder(const spec_beam_state* st, int32_t n_layers, const spec_kv* kv,
                                         int32_t row_bytes, void* ws, spec_stream_t stream) {
  if (!st || !kv) return SPEC_ERR_ARG;
  const spec_beam_state& s = *st;
  if (!s.parent || !s.tok || !s.seq_len || !s.prompt_blocks || !s.owned || !s.table_in || !s.table_out ||
      !s.spare_in || !s.spare_out || !s.slots || (s.hist_in == nullptr) != (s.hist_out == nullptr))
    return SPEC_ERR_ARG;
  if (s.table_in == s.table_out || s.spare_in == s.spare_out || (s.hist_in && s.hist_in == s.hist_out))
    return SPEC_ERR_ARG;
  if (s.B <= 0 || s.W <= 0 || s.W > 32 || (long long)s.B * s.W > 65535 || s.block_size <= 0 || s.max_blocks <= 0 ||
      s.owned_ld <= 0 || (s.hist_in && s.hist_ld <= 0) || n_layers <= 0 || n_layers > kMaxLayers || row_bytes <= 0 ||
      (long long)row_bytes * s.block_size >= (1ll << 31))
    return SPEC_ERR_SHAPE;
  if (ws && !aligned(ws, 256)) return SPEC_ERR_WORKSPACE;
  ReorderArgs g{};
  g.s = s;
  g.n_layers = n_layers;
  g.row_bytes = row_bytes;
  g.num_blocks = 0x7fffffff;
  g.ws = ws;
  for (int i = 0; i < n_layers; ++i) {
    if (!kv[i].k || !kv[i].v) return SPEC_ERR_ARG;
    if (kv[i].block_size != s.block_size || kv[i].num_slots < s.block_size) return SPEC_ERR_SHAPE;
    g.num_blocks = std::min(g.num_blocks, kv[i].num_slots / s.block_size);
    g.k[i] = kv[i].k;
    g.v[i] = kv[i].v;
  }
  const long long block_bytes = (long long)s.block_size * row_bytes;
  // few lanes for small blocks, whose copies would leave most of a CTA idle (384 beams, 36 layers, 6 KB blocks, 32 / 64 /
  // 128 / 256 lanes 12.0 / 16.1 / 27.9 / 51.0 us; 144 beams, 24 layers, 16 KB 14.1 / 10.2 / 10.6 / 15.7; 128 beams, 32
  // layers, 32 KB 26.6 / 23.3 / 22.3 / 25.5), all of them where there are few copies (4 beams, 1 layer 4.6 / 3.5 / 3.2 / 2.9)
  g.lanes = 2ll * n_layers * s.B * s.W <= 4 * sm_count() ? 256 : block_bytes <= 8192 ? 32 : block_bytes <= 16384 ? 64 : 128;
  const int per = 256 / g.lanes;
  launch_pdl(beam_reorder_kernel, dim3(1 + (2 * n_layers + per - 1) / per, s.B * s.W), dim3(256), 0, stream, g);
  return last_launch();
}

// per-unit log setter of the instrumented build (no-op otherwise)
SPEC_TL_SETTER(beam)
