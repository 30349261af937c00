// Beam search over the paged cache: the selection over beams and vocabulary, and
// the reordering of the beams' states (block tables, the partial block's K/V rows,
// token histories).
//
// The sources draft greedily or as a tree; a request decoded with beams is not
// speculated on ([NEURON] "Rejection Sampling" verifies one continuation), so its
// steps run through these calls on the same cache.
#include <cuda_fp16.h>

#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace spec {

enum : unsigned { kTLBeamSelect = 27, kTLBeamReorder = 28 };   // after common.cuh's ids

// ---------------------------------------------------------------- selection
// Within a beam the order of scores is the order of logits, so a row's chunk needs
// only its W largest logits, its maximum and its sum of exponentials: one pass
// over the logits, which stay in registers between the three uses.  The last
// chunk of a request to finish (a counter, nobody waits) merges.
constexpr int kSelThreads = 256, kSelWarps = kSelThreads / 32;
constexpr int kSelElems = 32;                               // logits a thread holds
constexpr int kSelChunk = kSelThreads * kSelElems;
constexpr int kSelCap = 1024;                               // entries of a candidate list
constexpr float kLog2e = 1.4426950408889634f;

struct SelArgs {
  int B, W, V, nch, eos;
  long long ld;
  const void* logits;
  const float* score;
  const int32_t* done;
  int32_t *parent, *tok, *done_out;
  float* score_out;
  int* counters;      // [B]
  float2* stats;      // [B * W, nch]  maximum, sum of exp(x - maximum)
  float2* cand;       // [B * W, nch, W]  logit, token id (bits)
};

SPEC_DEV float finite_or_mask(float x) { return fabsf(x) <= 3.402823466e38f ? x : -INFINITY; }
SPEC_DEV float cvt(float x) { return x; }
SPEC_DEV float cvt(__nv_bfloat16 x) { return __bfloat162float(x); }
SPEC_DEV float cvt(__half x) { return __half2float(x); }

// a place in the order: larger value first, then smaller index
template <typename F> SPEC_DEV bool ahead(F v, int i, F w, int j) { return v > w || (v == w && i < j); }

// The k-th largest of the block's thread maxima by warps: each warp's k-th largest
// lane value is reached by at least k values of the block, and so is the largest of
// those over the warps: a lower bound of the block's k-th largest value.
template <typename F> SPEC_DEV F block_bound(F v, int k, F* red) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int rank = 0;
#pragma unroll
  for (int o = 1; o < 32; ++o) {
    const F w = __shfl_sync(0xffffffffu, v, (lane + o) & 31);
    rank += w > v || (w == v && ((lane + o) & 31) < lane);
  }
  if (rank == k - 1) red[warp] = v;
  __syncthreads();
  F b = red[0];
#pragma unroll
  for (int w = 1; w < kSelWarps; ++w) b = red[w] > b ? red[w] : b;
  __syncthreads();
  return b;
}

struct SelShared {
  float fred[kSelWarps];
  double dred[kSelWarps];
  double val[kSelCap];
  int idx[kSelCap];
  int count, last;
  double lse[32];
};

// Best (value, index) of the block strictly after (pv, pi); every thread gets it.
template <typename F, typename Get> SPEC_DEV void block_next(F pv, int pi, int n, Get get, SelShared& sm, F& bv, int& bi) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  F v = (F)-INFINITY;
  int at = 0x7fffffff;
  for (int e = 0; e < n; ++e) {
    F x;
    int i;
    get(e, x, i);
    if (x > (F)-INFINITY && ahead(pv, pi, x, i) && ahead(x, i, v, at)) {
      v = x;
      at = i;
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const F w = __shfl_xor_sync(0xffffffffu, v, o);
    const int j = __shfl_xor_sync(0xffffffffu, at, o);
    if (ahead(w, j, v, at)) {
      v = w;
      at = j;
    }
  }
  __syncthreads();
  if (lane == 0) {
    sm.dred[warp] = (double)v;
    sm.idx[warp] = at;
  }
  __syncthreads();
  bv = (F)sm.dred[0];
  bi = sm.idx[0];
#pragma unroll
  for (int w = 1; w < kSelWarps; ++w)
    if (ahead((F)sm.dred[w], sm.idx[w], bv, bi)) {
      bv = (F)sm.dred[w];
      bi = sm.idx[w];
    }
  __syncthreads();
}

// The k best entries of the block's n-per-thread values, in order, each handed to
// emit(rank, value, index) by one thread (ranks without an entry are not handed out).
// Values at or above the bound are collected and ranked by counting; a list that
// overflows (long runs of equal values) is replaced by k rounds of block-wide
// maxima.  Returns the number of entries.
template <typename F, typename Get, typename Emit>
SPEC_DEV int block_top(int k, int n, Get get, Emit emit, SelShared& sm, F* red) {
  F mine = (F)-INFINITY;
  for (int e = 0; e < n; ++e) {
    F x;
    int i;
    get(e, x, i);
    mine = x > mine ? x : mine;
  }
  if (threadIdx.x == 0) sm.count = 0;
  const F bound = block_bound<F>(mine, k, red);       // ends with a barrier
  for (int e = 0; e < n; ++e) {
    F x;
    int i;
    get(e, x, i);
    if (x >= bound && x > (F)-INFINITY) {
      const int at = atomicAdd(&sm.count, 1);
      if (at < kSelCap) {
        sm.val[at] = (double)x;
        sm.idx[at] = i;
      }
    }
  }
  __syncthreads();
  const int count = sm.count;
  if (count <= kSelCap) {
    for (int a = threadIdx.x; a < count; a += kSelThreads) {
      const double v = sm.val[a];
      const int i = sm.idx[a];
      int rank = 0;
      for (int b = 0; b < count; ++b) rank += ahead(sm.val[b], sm.idx[b], v, i);
      if (rank < k) emit(rank, (F)v, i);
    }
    __syncthreads();
    return min(count, k);
  }
  __syncthreads();
  F pv = (F)INFINITY;
  int pi = -1, r = 0;
  for (; r < k; ++r) {
    F v;
    int i;
    block_next<F>(pv, pi, n, get, sm, v, i);
    if (!(v > (F)-INFINITY)) break;
    if (threadIdx.x == 0) emit(r, v, i);
    pv = v;
    pi = i;
  }
  __syncthreads();
  return r;
}

template <typename T>
__global__ void __launch_bounds__(kSelThreads) beam_select_kernel(const SelArgs g) {
  SPEC_TL(kTLBeamSelect);
  pdl_wait();
  pdl_trigger();
  __shared__ SelShared sm;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ch = blockIdx.x, row = blockIdx.y, b = row / g.W, W = g.W;
  const float my_score = g.score[row];
  const bool live = fabsf(my_score) <= 3.402823466e38f && g.done[row] == 0;
  if (live) {
    // element e of thread t is logit base + (e / P) * (256 P) + t * P + e % P whatever the row's
    // alignment (P elements are 16 bytes), so equal rows give equal sums
    constexpr int P = 16 / sizeof(T);
    const T* src = static_cast<const T*>(g.logits) + (long long)row * g.ld;
    const int base = ch * kSelChunk;
    float x[kSelElems];
    const bool vec = (reinterpret_cast<uintptr_t>(src) & 15) == 0;
#pragma unroll
    for (int i = 0; i < kSelElems / P; ++i) {
      const int v0 = base + (i * kSelThreads + tid) * P;
      if (vec && v0 + P <= g.V) {
        const uint4 raw = __ldcs(reinterpret_cast<const uint4*>(src + v0));
        const T* p = reinterpret_cast<const T*>(&raw);
#pragma unroll
        for (int j = 0; j < P; ++j) x[i * P + j] = finite_or_mask(cvt(p[j]));
      } else {
#pragma unroll
        for (int j = 0; j < P; ++j) x[i * P + j] = v0 + j < g.V ? finite_or_mask(cvt(src[v0 + j])) : -INFINITY;
      }
    }
    float m = -INFINITY;
#pragma unroll
    for (int e = 0; e < kSelElems; ++e) m = fmaxf(m, x[e]);
    m = warp_max(m);
    if (lane == 0) sm.fred[warp] = m;
    __syncthreads();
    m = sm.fred[0];
#pragma unroll
    for (int w = 1; w < kSelWarps; ++w) m = fmaxf(m, sm.fred[w]);
    // x - m first: at a type's lowest values m * log2(e) would overflow
    const float ms = m > -INFINITY ? m : 0.f;
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < kSelElems; ++e) s += exp2f((x[e] - ms) * kLog2e);
    s = warp_sum(s);
    __syncthreads();
    if (lane == 0) sm.fred[warp] = s;
    __syncthreads();
    if (tid == 0) {
      s = 0.f;
      for (int w = 0; w < kSelWarps; ++w) s += sm.fred[w];
      g.stats[(long long)row * g.nch + ch] = make_float2(m, s);
    }
    __syncthreads();
    float2* out = g.cand + ((long long)row * g.nch + ch) * W;
    const int got = block_top<float>(
        W, kSelElems,
        [&](int e, float& v, int& i) {
          v = x[e];
          i = base + ((e / P) * kSelThreads + tid) * P + e % P;
        },
        [&](int r, float v, int i) { out[r] = make_float2(v, __int_as_float(i)); }, sm, sm.fred);
    if (tid >= got && tid < W) out[tid] = make_float2(-INFINITY, __int_as_float(0x7fffffff));
  }
  // the request's last CTA merges
  __threadfence();
  __syncthreads();
  if (tid == 0) sm.last = atomicAdd(&g.counters[b], 1) == W * g.nch - 1;
  __syncthreads();
  if (!sm.last) return;
  __threadfence();
  if (tid == 0) g.counters[b] = 0;
  // log-sum-exp of every live beam, in fp64
  for (int j = warp; j < W; j += kSelWarps) {
    const float2* st = g.stats + (long long)(b * W + j) * g.nch;
    const float sc = g.score[b * W + j];
    if (!(fabsf(sc) <= 3.402823466e38f) || g.done[b * W + j] != 0) continue;
    float m = -INFINITY;
    for (int c = lane; c < g.nch; c += 32) m = fmaxf(m, __ldcg(&st[c]).x);
    m = warp_max(m);
    double s = 0;
    if (m > -INFINITY)
      for (int c = lane; c < g.nch; c += 32) {
        const float2 v = __ldcg(&st[c]);
        if (v.x > -INFINITY) s += (double)v.y * exp((double)v.x - (double)m);
      }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) sm.lse[j] = m > -INFINITY ? (double)m + log(s) : 0.0;
  }
  __syncthreads();
  // candidates of the request: W beams x nch chunks x W, scored in fp64
  const int per = g.nch * W, all = W * per, n = (all + kSelThreads - 1) / kSelThreads;
  auto get = [&](int e, double& v, int& i) {
    const int k = e * kSelThreads + tid;
    v = -INFINITY;
    i = 0x7fffffff;
    if (k >= all) return;
    const int j = k / per, c = k - j * per;
    const float sc = g.score[b * W + j];
    if (!(fabsf(sc) <= 3.402823466e38f)) return;
    if (g.done[b * W + j] != 0) {
      if (c == 0) {
        v = (double)sc;
        i = j * g.V + max(g.eos, 0);
      }
      return;
    }
    const float2 x = __ldcg(&g.cand[(long long)(b * W + j) * per + c]);
    if (!(x.x > -INFINITY)) return;
    v = (double)sc + ((double)x.x - sm.lse[j]);
    i = j * g.V + __float_as_int(x.y);
  };
  const int got = block_top<double>(
      W, n, get,
      [&](int r, double v, int i) {
        const int j = i / g.V, o = b * W + r;
        const bool fin = g.done[b * W + j] != 0;
        const int t = fin ? g.eos : i - j * g.V;
        g.parent[o] = j;
        g.tok[o] = t;
        g.score_out[o] = (float)v;
        g.done_out[o] = fin || t == g.eos;
      },
      sm, sm.dred);
  if (tid >= got && tid < W) {
    const int o = b * W + tid;
    g.parent[o] = tid;
    g.tok[o] = -1;
    g.score_out[o] = -INFINITY;
    g.done_out[o] = 1;
  }
}

static int sel_chunks(int V) { return (V + kSelChunk - 1) / kSelChunk; }

// ---------------------------------------------------------------- reordering
constexpr int kMaxLayers = 64;
struct ReorderArgs {
  spec_beam_state s;
  int n_layers, row_bytes, num_blocks;
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

// Grid (part, row): part 0 writes the row's integers, part 1 + 2 * layer + (0 or
// 1) copies the partial block's K or V rows, which are contiguous (slots of a
// block follow one another).  A copy's source is some beam's current block and its
// target a spare block, and no block is both.
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
  if (t.from < 0) return;
  const int layer = (part - 1) >> 1;
  char* base = static_cast<char*>((part - 1) & 1 ? g.v[layer] : g.k[layer]);
  const long long block_bytes = (long long)s.block_size * g.row_bytes;
  const char* from = base + t.from * block_bytes;
  char* to = base + t.block * block_bytes;
  const int bytes = t.rest * g.row_bytes;
  if (((reinterpret_cast<uintptr_t>(base) | g.row_bytes) & 15) == 0) {
    const uint4* f = reinterpret_cast<const uint4*>(from);
    uint4* o = reinterpret_cast<uint4*>(to);
#pragma unroll 4
    for (int i = tid; i < bytes >> 4; i += 256) o[i] = __ldcs(f + i);
  } else {
    for (int i = tid; i < bytes; i += 256) to[i] = from[i];
  }
}

}  // namespace spec

using namespace spec;

extern "C" size_t spec_beam_workspace_bytes(int32_t B, int32_t W, int32_t V) {
  if (B <= 0 || W <= 0 || W > 32 || V <= 0 || (long long)W * V >= (1ll << 30)) return 0;
  const size_t n = (size_t)B * W * sel_chunks(V);
  return kWsHeader + align_up((size_t)B * 4, 256) + align_up(n * 8, 256) + align_up(n * W * 8, 256);
}

extern "C" spec_status spec_beam_select(int32_t B, int32_t W, int32_t V, int32_t dtype, const void* logits, int64_t ld,
                                        const float* score, const int32_t* done, int32_t eos, int32_t* parent,
                                        int32_t* tok, float* score_out, int32_t* done_out, void* ws, size_t ws_bytes,
                                        spec_stream_t stream) {
  if (!logits || !score || !done || !parent || !tok || !score_out || !done_out) return SPEC_ERR_ARG;
  if (score == score_out || done == done_out) return SPEC_ERR_ARG;
  if (dtype < SPEC_DTYPE_F32 || dtype > SPEC_DTYPE_F16) return SPEC_ERR_UNSUPPORTED;
  const size_t need = spec_beam_workspace_bytes(B, W, V);
  if (need == 0 || eos >= V || (long long)B * W > 65535) return SPEC_ERR_SHAPE;
  if (ld == 0) ld = V;
  if (ld < V) return SPEC_ERR_SHAPE;
  if (!aligned(logits, dtype == SPEC_DTYPE_F32 ? 4 : 2)) return SPEC_ERR_ALIGN;
  if (!ws || !aligned(ws, 256) || ws_bytes < need) return SPEC_ERR_WORKSPACE;
  const int nch = sel_chunks(V);
  char* p = static_cast<char*>(ws) + kWsHeader;
  SelArgs g{};
  g.B = B, g.W = W, g.V = V, g.nch = nch, g.eos = eos < 0 ? -1 : eos, g.ld = ld;
  g.logits = logits, g.score = score, g.done = done;
  g.parent = parent, g.tok = tok, g.done_out = done_out, g.score_out = score_out;
  g.counters = reinterpret_cast<int*>(p);
  p += align_up((size_t)B * 4, 256);
  g.stats = reinterpret_cast<float2*>(p);
  p += align_up((size_t)B * W * nch * 8, 256);
  g.cand = reinterpret_cast<float2*>(p);
  auto* kern = dtype == SPEC_DTYPE_F32 ? beam_select_kernel<float>
               : dtype == SPEC_DTYPE_BF16 ? beam_select_kernel<__nv_bfloat16> : beam_select_kernel<__half>;
  launch_pdl(kern, dim3(nch, B * W), dim3(kSelThreads), 0, stream, g);
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
  launch_pdl(beam_reorder_kernel, dim3(1 + 2 * n_layers, s.B * s.W), dim3(256), 0, stream, g);
  return last_launch();
}

// per-unit log setter of the instrumented build (no-op otherwise)
SPEC_TL_SETTER(beam)
