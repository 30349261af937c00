// Requests that share blocks of the paged cache: forked, released, and the cache
// compacted.
//
// [NEURON] "KV Cache Sharing": the paged cache and its block tables; here the
// blocks of one request are held by several (samples of one prompt).
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace spec {
namespace bl {

enum : unsigned { kTLFork = 31, kTLRelease, kTLCompact, kTLBlockCopy };   // after the other units' ids

// The state is a few hundred thousand integers and its steps depend on one another:
// one cluster works on it, with hardware barriers between the steps instead of
// launches (fork of 3 rows 8.4 us with its copies, release 10, compaction of 200 blocks 13).
constexpr int kCtas = 8, kThreads = 1024, kAll = kCtas * kThreads, kWarps = kAll / 32;
constexpr int kMaxB = 8192, kMaxLayers = 64;
constexpr int kBatch = 4;                                // table entries a lane has under way
constexpr int kCopyThreads = 256, kPiece = 32768;        // bytes that a CTA copies at a time

struct Scratch {               // in the workspace, after the header
  int moves;                   // blocks to copy
  int abort;
  int at_border;               // blocks in use below `used`
  int pad;
  int count[kCtas];
};
constexpr size_t kScratch = 256;

struct Args {
  spec_block_state s;
  int n;                       // forks
  const int32_t *src, *dst, *drop;
  Scratch* sc;
  int *a, *b, *c;              // [num_blocks] each (a: also [B])
  int4* moves;                 // (from slot, to slot, slots, 0)
  void* ws;
};

SPEC_DEV void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
SPEC_DEV int cap_of(const spec_block_state& s) { return s.max_blocks * s.block_size; }
SPEC_DEV int blocks_of(const spec_block_state& s, int len) { return (len + s.block_size - 1) / s.block_size; }
SPEC_DEV bool length_ok(const spec_block_state& s, int len) { return len >= 0 && len <= cap_of(s); }
SPEC_DEV bool id_ok(const spec_block_state& s, int id) { return id >= 0 && id < s.num_blocks; }
SPEC_DEV int free_count(const Args& g, int gt) {
  const int n = *g.s.n_free_in, m = min(max(n, 0), g.s.num_blocks);
  if (gt == 0 && n != m) report(g.ws, SPEC_ERR_DEVICE, -1, n);
  return m;
}

// dst = src, where the update is not in place
SPEC_DEV void carry(int32_t* dst, const int32_t* src, long long n, int gt, int all = kAll) {
  if (dst != src)
    for (long long i = gt; i < n; i += all) dst[i] = src[i];
}

// exclusive prefix sums of a[0, n) in shared memory, in place; returns the sum
SPEC_DEV int scan(int* a, int n, int* red) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, per = (n + kThreads - 1) / kThreads;
  const int i0 = min(n, tid * per), i1 = min(n, i0 + per);
  __syncthreads();
  int sum = 0;
  for (int i = i0; i < i1; ++i) sum += a[i];
  int x = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) red[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int y = red[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int z = __shfl_up_sync(0xffffffffu, y, o);
      if (lane >= o) y += z;
    }
    red[lane] = y;
  }
  __syncthreads();
  int run = x - sum + (warp > 0 ? red[warp - 1] : 0);
  for (int i = i0; i < i1; ++i) {
    const int y = a[i];
    a[i] = run;
    run += y;
  }
  const int total = red[31];
  __syncthreads();
  return total;
}

// ---------------------------------------------------------------- fork
__global__ void __cluster_dims__(kCtas, 1, 1) __launch_bounds__(kThreads, 1) fork_kernel(const __grid_constant__ Args g) {
  SPEC_TL(kTLFork);
  pdl_wait();
  pdl_trigger();
  extern __shared__ int sm[];
  __shared__ int red[32];
  const spec_block_state& s = g.s;
  const int tid = threadIdx.x, gt = blockIdx.x * kThreads + tid, lane = tid & 31, warp = gt >> 5, n = g.n, mb = s.max_blocks;
  int *nth = sm, *len = sm + n, *first = g.a;            // len: of the fork's source, -1: refused
  const int n_free = free_count(g, gt);
  for (int i = gt; i < s.B; i += kAll) first[i] = 0;
  carry(s.table_out, s.table_in, (long long)s.B * mb, gt);
  carry(s.len_out, s.len_in, s.B, gt);
  carry(s.shared_out, s.shared_in, s.num_blocks, gt);
  carry(s.free_out, s.free_in, s.num_blocks, gt);
  cluster_sync();
  // the first fork to name an empty row gets it
  for (int i = gt; i < n; i += kAll) {
    const int d = g.dst[i];
    if (d >= 0 && d < s.B) atomicMax(&first[d], n - i);
  }
  cluster_sync();
  // every CTA for itself: which forks are served, and their places in the pool
  for (int i = tid; i < n; i += kThreads) {
    const int a = g.src[i], d = g.dst[i];
    int l = -1;
    if (a >= 0 && a < s.B && d >= 0 && d < s.B && __ldcg(&first[d]) == n - i && s.len_in[d] == 0 && length_ok(s, s.len_in[a]))
      l = s.len_in[a];
    else if (blockIdx.x == 0) report(g.ws, SPEC_ERR_DEVICE, a, d);
    len[i] = l;
    nth[i] = l > 0 && l % s.block_size > 0;
  }
  const int need = scan(nth, n, red);
  if (gt == 0 && need > n_free) report(g.ws, SPEC_ERR_CAPACITY, need, n_free);
  cluster_sync();                                        // all lengths are read
  for (int i = warp; i < n; i += kWarps) {
    const int l = len[i], a = g.src[i], d = g.dst[i], whole = l / s.block_size, rest = l % s.block_size;
    int4 move = make_int4(0, 0, 0, 0);
    if (l >= 0 && (rest == 0 || nth[i] < n_free)) {      // (l = 0: a row of entries -1)
      int fresh = -1;
      if (rest > 0) {
        const int place = n_free - 1 - nth[i];
        fresh = s.free_in[place];
        __syncwarp();
        if (lane == 0) s.free_out[place] = -1;
      }
      const int32_t* from = s.table_in + (long long)a * mb;
      int32_t* to = s.table_out + (long long)d * mb;
      for (int j = lane; j < mb; j += 32) {
        int id = -1;
        if (j < whole || (j == whole && rest > 0)) {
          id = from[j];
          if (!id_ok(s, id)) {
            report(g.ws, SPEC_ERR_DEVICE, a, id);
            id = -1;
          }
          if (j < whole) {
            if (id >= 0) atomicAdd(&s.shared_out[id], 1);
          } else {
            const bool ok = id_ok(s, fresh);
            if (!ok) report(g.ws, SPEC_ERR_DEVICE, d, fresh);
            if (ok && id >= 0) move = make_int4(id * s.block_size, fresh * s.block_size, rest, 0);
            id = ok ? fresh : -1;
          }
        }
        to[j] = id;
      }
      if (lane == 0) s.len_out[d] = l;
    }
    const unsigned who = __ballot_sync(0xffffffffu, move.z > 0);
    if (who ? lane == __ffs(who) - 1 : lane == 0) g.moves[i] = move;
  }
  if (gt == 0) {
    g.sc->moves = n;
    *s.n_free_out = n_free - min(need, n_free);
  }
}

// ---------------------------------------------------------------- release
// Where the steps of a release run: all threads of one cluster, or of a launch each.
struct Place {
  int gt, all, warp, warps, lane;
};

// By block: the rows that let go of it, and the last of their entries (in row, then block order), 0: none.
SPEC_DEV void release_clear(const Args& g, const Place& p) {
  const spec_block_state& s = g.s;
  const int n_free = free_count(g, p.gt);
  for (int i = p.gt; i < s.num_blocks; i += p.all) g.a[i] = 0, g.b[i] = 0;
  if (p.gt == 0) g.sc->moves = n_free;                   // (n_free_out may be n_free_in)
  carry(s.shared_out, s.shared_in, s.num_blocks, p.gt, p.all);
  carry(s.free_out, s.free_in, n_free, p.gt, p.all);
}

SPEC_DEV void release_count(const Args& g, const Place& p) {
  const spec_block_state& s = g.s;
  const int mb = s.max_blocks;
  for (int b = p.warp; b < s.B; b += p.warps) {
    const int l = s.len_in[b];
    if (g.drop[b] == 0) continue;
    if (!length_ok(s, l)) {
      if (p.lane == 0) report(g.ws, SPEC_ERR_DEVICE, b, l);
      continue;
    }
    const int have = blocks_of(s, l);
    for (int j0 = p.lane; j0 < have; j0 += 32 * kBatch) {
      int id[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) id[i] = j0 + 32 * i < have ? s.table_in[(long long)b * mb + j0 + 32 * i] : 0;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        if (j0 + 32 * i >= have) break;
        if (!id_ok(s, id[i])) {
          report(g.ws, SPEC_ERR_DEVICE, b, id[i]);
          continue;
        }
        atomicAdd(&g.a[id[i]], 1);
        atomicMax(&g.b[id[i]], b * mb + j0 + 32 * i + 1);
      }
    }
  }
}

// Blocks that each row gives back.
SPEC_DEV void release_rows(const Args& g, const Place& p) {
  const spec_block_state& s = g.s;
  const int mb = s.max_blocks;
  for (int b = p.warp; b < s.B; b += p.warps) {
    const int l = s.len_in[b];
    int mine = 0;
    if (g.drop[b] != 0 && length_ok(s, l)) {
      const int have = blocks_of(s, l);
      for (int j0 = p.lane; j0 < have; j0 += 32 * kBatch) {
        int id[kBatch], last[kBatch], gone[kBatch], held[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          id[i] = j0 + 32 * i < have ? s.table_in[(long long)b * mb + j0 + 32 * i] : -1;
          if (!id_ok(s, id[i])) id[i] = -1;
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int at = max(id[i], 0);
          last[i] = __ldcg(&g.b[at]), gone[i] = __ldcg(&g.a[at]), held[i] = s.shared_in[at];
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) mine += id[i] >= 0 && last[i] == b * mb + j0 + 32 * i + 1 && gone[i] > held[i];
      }
    }
    mine = __reduce_add_sync(0xffffffffu, mine);
    if (p.lane == 0) g.c[b] = mine;
  }
}

// Every CTA for itself: the rows' places in the pool; then its rows.
SPEC_DEV void release_write(const Args& g, const Place& p, int* sm, int* red) {
  const spec_block_state& s = g.s;
  const int mb = s.max_blocks, n_free = __ldcg(&g.sc->moves);
  for (int b = threadIdx.x; b < s.B; b += kThreads) sm[b] = __ldcg(&g.c[b]);
  const int total = scan(sm, s.B, red);
  if (p.gt == 0 && n_free + total > s.num_blocks) report(g.ws, SPEC_ERR_DEVICE, n_free, total);
  for (int b = p.warp; b < s.B; b += p.warps) {
    const int l = s.len_in[b];
    const bool drop = g.drop[b] != 0 && length_ok(s, l);
    const int have = drop ? blocks_of(s, l) : 0;
    int at = n_free + sm[b];
    if (drop || s.table_out != s.table_in)
      for (int j0 = p.lane; j0 - p.lane < mb; j0 += 32 * kBatch) {
        const long long e = (long long)b * mb + j0;
        int id[kBatch], last[kBatch], gone[kBatch], held[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) id[i] = j0 + 32 * i < mb ? s.table_in[e + 32 * i] : -1;
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int k = j0 + 32 * i < have && id_ok(s, id[i]) ? id[i] : 0;
          last[i] = __ldcg(&g.b[k]), gone[i] = __ldcg(&g.a[k]), held[i] = s.shared_in[k];
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int j = j0 + 32 * i;
          bool freed = false;
          if (j < have && id_ok(s, id[i]) && last[i] == b * mb + j + 1) {      // (one entry of a block only)
            freed = gone[i] > held[i];
            if (gone[i] > held[i] + 1) report(g.ws, SPEC_ERR_DEVICE, id[i], gone[i]);
            s.shared_out[id[i]] = freed ? 0 : held[i] - gone[i];
          }
          const unsigned who = __ballot_sync(0xffffffffu, freed);
          const int place = at + __popc(who & ((1u << p.lane) - 1));
          if (freed && place < s.num_blocks) s.free_out[place] = id[i];
          at += __popc(who);
          if (j < mb) {
            if (drop) s.table_out[e + 32 * i] = -1;
            else if (s.table_out != s.table_in) s.table_out[e + 32 * i] = id[i];
          }
        }
      }
    __syncwarp();
    if (p.lane == 0) s.len_out[b] = drop ? 0 : l;
  }
  const int now = min(n_free + total, s.num_blocks);
  if (s.free_out != s.free_in)
    for (int i = now + p.gt; i < s.num_blocks; i += p.all) s.free_out[i] = -1;
  if (p.gt == 0) *s.n_free_out = now;
}

SPEC_DEV Place place_of(int ctas) {
  Place p;
  p.gt = blockIdx.x * kThreads + threadIdx.x, p.all = ctas * kThreads;
  p.warp = p.gt >> 5, p.warps = p.all >> 5, p.lane = p.gt & 31;
  return p;
}

__global__ void __cluster_dims__(kCtas, 1, 1) __launch_bounds__(kThreads, 1) release_kernel(const __grid_constant__ Args g) {
  SPEC_TL(kTLRelease);
  pdl_wait();
  pdl_trigger();
  extern __shared__ int sm[];
  __shared__ int red[32];
  const Place p = place_of(kCtas);
  release_clear(g, p);
  cluster_sync();
  release_count(g, p);
  cluster_sync();
  release_rows(g, p);
  cluster_sync();
  release_write(g, p, sm, red);
}

// A step a launch, on all SMs
template <int STEP> __global__ void __launch_bounds__(kThreads, 1) release_step_kernel(const __grid_constant__ Args g) {
  SPEC_TL(kTLRelease);
  pdl_wait();
  pdl_trigger();
  extern __shared__ int sm[];
  __shared__ int red[32];
  const Place p = place_of(gridDim.x);
  if (STEP == 0) release_clear(g, p);
  if (STEP == 1) release_count(g, p);
  if (STEP == 2) release_rows(g, p);
  if (STEP == 3) release_write(g, p, sm, red);
}

// ---------------------------------------------------------------- compact
__global__ void __cluster_dims__(kCtas, 1, 1) __launch_bounds__(kThreads, 1) compact_kernel(const __grid_constant__ Args g) {
  SPEC_TL(kTLCompact);
  pdl_wait();
  pdl_trigger();
  __shared__ int red[32];
  __shared__ int tile[4 * kThreads];
  const spec_block_state& s = g.s;
  const int tid = threadIdx.x, gt = blockIdx.x * kThreads + tid, lane = tid & 31, warp = gt >> 5, mb = s.max_blocks;
  const int N = s.num_blocks;
  int *used = g.a, *place = g.b, *where = g.c;
  const int n_free = free_count(g, gt);
  for (int i = gt; i < N; i += kAll) used[i] = 0;
  if (gt == 0) g.sc->abort = 0;
  carry(s.shared_out, s.shared_in, N, gt);
  carry(s.len_out, s.len_in, s.B, gt);
  cluster_sync();
  for (int b = warp; b < s.B; b += kWarps) {
    const int l = s.len_in[b];
    if (!length_ok(s, l)) {
      report(g.ws, SPEC_ERR_DEVICE, b, l);
      g.sc->abort = 1;
      continue;
    }
    const int have = blocks_of(s, l);
#pragma unroll 4
    for (int j = lane; j < have; j += 32) {
      const int id = s.table_in[(long long)b * mb + j];
      if (id_ok(s, id)) used[id] = 1;
      else {
        report(g.ws, SPEC_ERR_DEVICE, b, id);
        g.sc->abort = 1;
      }
    }
  }
  cluster_sync();
  // CTA c has ids [i0, i1)
  const int per = (N + kCtas - 1) / kCtas, i0 = min(N, (int)blockIdx.x * per), i1 = min(N, i0 + per);
  {
    int c = 0;
    for (int i = i0 + tid; i < i1; i += kThreads) c += __ldcg(&used[i]);
    c = __reduce_add_sync(0xffffffffu, c);
    if (lane == 0) red[tid >> 5] = c;
    __syncthreads();
    if (tid < 32) {
      c = __reduce_add_sync(0xffffffffu, red[tid]);
      if (tid == 0) g.sc->count[blockIdx.x] = c;
    }
  }
  cluster_sync();
  int U = 0, run = 0;
  for (int c = 0; c < kCtas; ++c) {
    const int x = __ldcg(&g.sc->count[c]);
    if (c < (int)blockIdx.x) run += x;
    U += x;
  }
  // blocks that no row and not the pool holds are someone else's: then nothing moves
  const bool go = U + n_free == N && __ldcg(&g.sc->abort) == 0;
  if (gt == 0 && U + n_free != N) report(g.ws, SPEC_ERR_CAPACITY, U, n_free);
  // Of an id, the used ones below it.  place[k]: the k-th unused id below U (k < holes), and the used ids from U on at
  // their rank among all used ones, which begins at U - holes.
  if (gt == 0 && U == N) g.sc->at_border = U;
  for (int t0 = i0; t0 < i1; t0 += 4 * kThreads) {
    const int m = min(4 * kThreads, i1 - t0);
    for (int i = tid; i < m; i += kThreads) tile[i] = __ldcg(&used[t0 + i]);
    const int all = scan(tile, m, red);
    for (int i = tid; i < m; i += kThreads) {
      const int id = t0 + i, below = run + tile[i];
      const bool u = __ldcg(&used[id]) != 0;
      if (id == U) g.sc->at_border = below;
      if (id < U && !u) place[id - below] = id;
      if (id >= U && u) where[below] = id;
    }
    __syncthreads();
    run += all;
  }
  cluster_sync();
  const int border = __ldcg(&g.sc->at_border), holes = go ? U - border : 0;
  for (int k = gt; k < holes; k += kAll) {
    const int from = __ldcg(&where[border + k]), to = __ldcg(&place[k]);
    g.moves[k] = make_int4(from * s.block_size, to * s.block_size, s.block_size, 0);
    used[from] = -1 - to;                                // where it goes
    s.shared_out[to] = s.shared_in[from];
    s.shared_out[from] = 0;
  }
  cluster_sync();
  for (int b = warp; b < s.B; b += kWarps) {
    const int l = s.len_in[b], have = length_ok(s, l) ? blocks_of(s, l) : 0;
    for (int j = lane; j < mb; j += 32) {
      const long long e = (long long)b * mb + j;
      const int id = s.table_in[e];
      if (!go) {
        if (s.table_out != s.table_in) s.table_out[e] = id;
        continue;
      }
      const int to = j < have ? __ldcg(&used[id]) : 0;
      if (j >= have) s.table_out[e] = -1;
      else if (to < 0) s.table_out[e] = -1 - to;
      else if (s.table_out != s.table_in) s.table_out[e] = id;
    }
  }
  if (go) {
    for (int i = gt; i < N; i += kAll) s.free_out[i] = i < N - U ? N - 1 - i : -1;
  } else {
    carry(s.free_out, s.free_in, N, gt);
  }
  if (gt == 0) {
    g.sc->moves = holes;
    *s.n_free_out = n_free;
  }
}

// ---------------------------------------------------------------- copies
struct CopyArgs {
  void* base[2 * kMaxLayers];  // K and V of each layer
  int n_bases, row_bytes;
  int pieces;                  // of a whole block
  const Scratch* sc;
  const int4* moves;
};

// A block's slots are one piece of memory in each K and V: kPiece bytes of it a CTA at a
// time, 8 vectors a thread under way.  Bound by the copy bandwidth (1.2 GB moved within
// the cache: 390-403 us from one GPU to another, 91-94 % of it).  Sources are never another move's target.
template <typename V> __global__ void __launch_bounds__(kCopyThreads) block_copy_kernel(const __grid_constant__ CopyArgs g) {
  SPEC_TL(kTLBlockCopy);
  pdl_wait();
  pdl_trigger();
  constexpr int U = 8;
  const int moves = g.sc->moves;
  const long long all = (long long)moves * g.n_bases * g.pieces;
  for (long long u = blockIdx.x; u < all; u += gridDim.x) {
    const int piece = (int)(u % g.pieces);
    const long long w = u / g.pieces;
    const int base = (int)(w % g.n_bases);
    const int4 m = g.moves[w / g.n_bases];
    const long long bytes = (long long)m.z * g.row_bytes, from = (long long)piece * kPiece;
    if (from >= bytes) continue;
    const int n = (int)(min(bytes - from, (long long)kPiece) / (long long)sizeof(V));
    const V* src = reinterpret_cast<const V*>(static_cast<char*>(g.base[base]) + (long long)m.x * g.row_bytes + from);
    V* dst = reinterpret_cast<V*>(static_cast<char*>(g.base[base]) + (long long)m.y * g.row_bytes + from);
    for (int i = threadIdx.x; i < n; i += U * kCopyThreads) {
      V v[U];
#pragma unroll
      for (int j = 0; j < U; ++j)
        if (i + j * kCopyThreads < n) v[j] = __ldcs(src + i + j * kCopyThreads);
#pragma unroll
      for (int j = 0; j < U; ++j)
        if (i + j * kCopyThreads < n) __stcs(dst + i + j * kCopyThreads, v[j]);
    }
  }
}

// ---------------------------------------------------------------- checks
static spec_status check(const spec_block_state* s) {
  if (!s || !s->table_in || !s->table_out || !s->len_in || !s->len_out || !s->shared_in || !s->shared_out || !s->free_in ||
      !s->free_out || !s->n_free_in || !s->n_free_out)
    return SPEC_ERR_ARG;
  if (s->B <= 0 || s->block_size <= 0 || s->max_blocks <= 0 || s->num_blocks <= 0) return SPEC_ERR_SHAPE;
  if (s->B > kMaxB || (long long)s->max_blocks * s->block_size >= (1ll << 30) ||
      (long long)s->B * s->max_blocks * s->block_size >= (1ll << 30) || (long long)s->num_blocks * s->block_size >= (1ll << 30))
    return SPEC_ERR_CAPACITY;
  return SPEC_OK;
}

static spec_status check_ws(const spec_block_state* s, const void* ws, size_t ws_bytes) {
  return ws && aligned(ws, 256) && ws_bytes >= spec_block_state_workspace_bytes(s->B, s->num_blocks) ? SPEC_OK
                                                                                                    : SPEC_ERR_WORKSPACE;
}

static spec_status check_kv(const spec_block_state* s, int n_layers, const spec_kv* kv, int row_bytes) {
  if (!kv) return SPEC_ERR_ARG;
  if (n_layers <= 0 || n_layers > kMaxLayers || row_bytes <= 0) return SPEC_ERR_SHAPE;
  for (int i = 0; i < n_layers; ++i) {
    if (!kv[i].k || !kv[i].v) return SPEC_ERR_ARG;
    if (kv[i].block_size != s->block_size || kv[i].num_slots < (long long)s->num_blocks * s->block_size) return SPEC_ERR_SHAPE;
  }
  return SPEC_OK;
}

static Args args(const spec_block_state* s, void* ws) {
  Args g{};
  g.s = *s;
  g.ws = ws;
  char* p = static_cast<char*>(ws) + kWsHeader;
  g.sc = reinterpret_cast<Scratch*>(p);
  g.moves = reinterpret_cast<int4*>(p + kScratch);
  g.a = reinterpret_cast<int*>(g.moves + std::max(s->B, s->num_blocks));
  g.b = g.a + std::max(s->B, s->num_blocks);
  g.c = g.b + std::max(s->B, s->num_blocks);
  return g;
}

static spec_status plan(void (*kern)(Args), const Args& g, size_t smem, int ctas, cudaStream_t st) {
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 2 * kMaxB * (int)sizeof(int)) != cudaSuccess)
    return SPEC_ERR_CUDA;
  return cuda_status(launch_pdl(kern, dim3(ctas), dim3(kThreads), smem, st, g));
}

static spec_status copy(const Args& g, int n_layers, const spec_kv* kv, int row_bytes, long long most, cudaStream_t st) {
  CopyArgs c{};
  c.n_bases = 2 * n_layers, c.row_bytes = row_bytes, c.sc = g.sc, c.moves = g.moves;
  c.pieces = (int)(((long long)g.s.block_size * row_bytes + kPiece - 1) / kPiece);
  bool a16 = row_bytes % 16 == 0, a4 = row_bytes % 4 == 0;
  for (int i = 0; i < n_layers; ++i) {
    c.base[2 * i] = kv[i].k, c.base[2 * i + 1] = kv[i].v;
    a16 = a16 && aligned(kv[i].k, 16) && aligned(kv[i].v, 16);
    a4 = a4 && aligned(kv[i].k, 4) && aligned(kv[i].v, 4);
  }
  const long long units = most * c.n_bases * c.pieces;
  const dim3 grid((unsigned)std::min<long long>(units, 8ll * sm_count()));
  auto kern = a16 ? block_copy_kernel<float4> : a4 ? block_copy_kernel<int> : block_copy_kernel<unsigned char>;
  return cuda_status(launch_pdl(kern, grid, dim3(kCopyThreads), 0, st, c));
}

}  // namespace bl
}  // namespace spec

using namespace spec;

extern "C" size_t spec_block_state_workspace_bytes(int32_t B, int32_t num_blocks) {
  if (B <= 0 || B > bl::kMaxB || num_blocks <= 0) return 0;
  return kWsHeader + bl::kScratch + (size_t)std::max(B, num_blocks) * (sizeof(int4) + 3 * sizeof(int));
}

extern "C" spec_status spec_block_fork(const spec_block_state* st, int32_t n, const int32_t* src, const int32_t* dst,
                                       int32_t n_layers, const spec_kv* kv, int32_t row_bytes, void* ws, size_t ws_bytes,
                                       spec_stream_t stream) {
  if (!src || !dst) return SPEC_ERR_ARG;
  spec_status r = bl::check(st);
  if (r == SPEC_OK) r = bl::check_kv(st, n_layers, kv, row_bytes);
  if (r != SPEC_OK) return r;
  if (n <= 0 || n > st->B) return SPEC_ERR_SHAPE;
  if ((r = bl::check_ws(st, ws, ws_bytes)) != SPEC_OK) return r;
  bl::Args g = bl::args(st, ws);
  g.n = n, g.src = src, g.dst = dst;
  if ((r = bl::plan(bl::fork_kernel, g, (size_t)n * 2 * sizeof(int), bl::kCtas, stream)) != SPEC_OK) return r;
  if ((r = bl::copy(g, n_layers, kv, row_bytes, n, stream)) != SPEC_OK) return r;
  return last_launch();
}

extern "C" spec_status spec_block_release(const spec_block_state* st, const int32_t* drop, void* ws, size_t ws_bytes,
                                          spec_stream_t stream) {
  if (!drop) return SPEC_ERR_ARG;
  spec_status r = bl::check(st);
  if (r == SPEC_OK) r = bl::check_ws(st, ws, ws_bytes);
  if (r != SPEC_OK) return r;
  bl::Args g = bl::args(st, ws);
  g.drop = drop;
  // A row a warp.  Rows that one cluster's warps hold: its barriers are cheaper than launches; more: a launch a step, whose SMs
  // are more.  Cluster / launches, 32 rows of up to 138 entries 10.5 / 12.2 us; 128 of 264: 19.5 / 20.5; 256 of 138, 264, 451:
  // 14.0 / 15.4, 21.5 / 22.3, 33.9 / 32.2; 512 of 138, 451: 21.9 / 16.3, 57 / 35.7.
  if (st->B <= bl::kWarps) {
    r = bl::plan(bl::release_kernel, g, (size_t)st->B * sizeof(int), bl::kCtas, stream);
  } else {
    void (*const steps[])(bl::Args) = {bl::release_step_kernel<0>, bl::release_step_kernel<1>, bl::release_step_kernel<2>,
                                       bl::release_step_kernel<3>};
    const int ctas = std::min(sm_count(), (st->B + 31) / 32 * 4);
    for (auto step : steps)
      if ((r = bl::plan(step, g, (size_t)st->B * sizeof(int), ctas, stream)) != SPEC_OK) return r;
  }
  return r != SPEC_OK ? r : last_launch();
}

extern "C" spec_status spec_block_compact(const spec_block_state* st, int32_t n_layers, const spec_kv* kv, int32_t row_bytes,
                                          void* ws, size_t ws_bytes, spec_stream_t stream) {
  spec_status r = bl::check(st);
  if (r == SPEC_OK) r = bl::check_kv(st, n_layers, kv, row_bytes);
  if (r == SPEC_OK) r = bl::check_ws(st, ws, ws_bytes);
  if (r != SPEC_OK) return r;
  bl::Args g = bl::args(st, ws);
  if ((r = bl::plan(bl::compact_kernel, g, 0, bl::kCtas, stream)) != SPEC_OK) return r;
  if ((r = bl::copy(g, n_layers, kv, row_bytes, st->num_blocks, stream)) != SPEC_OK) return r;
  return last_launch();
}

// per-unit log setter of the instrumented build (no-op otherwise)
SPEC_TL_SETTER(blocks)
