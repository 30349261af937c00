// Block tables and slot maps from request lengths, and the K/V append that the
// slots are for.
//
// [NEURON] "KV Cache Sharing" and "EagleProposer": a paged cache addressed by
// block tables, slot_mapping built from them for the tokens of a step.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "internal.h"

namespace spec {

enum : unsigned { kTLTables = 24, kTLAppend = 25 };   // after common.cuh's ids

// ---------------------------------------------------------------- block tables
constexpr int kTabThreads = 512;
constexpr int kTabMaxB = 8192;

struct TabArgs {
  int B, bs, mb, num_blocks, cap;
  const int32_t *len_old, *len_new, *table_in, *free_in, *n_free_in;
  int32_t *table_out, *free_out, *n_free_out, *len_out, *cu_new, *slots, *pos;
  void* ws;
};

// index of the first entry of the ascending a[0, n) above x (n if none)
SPEC_DEV int first_above(const int* a, int n, int x) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (a[mid] > x) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

// One launch.  Every CTA computes the prefix sums of all requests for itself (a
// few thousand integers, read from L2), then takes its share of the pool
// entries, table entries and tokens.  A block taken from the pool is *delivered*
// by the thread that reads it: it finds the request that the block goes to by
// bisection of the prefix sums and writes that table entry and the slots of the
// block's tokens.  So every pool entry and every released table entry is read by
// one thread only, which writes to it afterwards, and the update is safe in
// place without a grid-wide barrier.  What all CTAs read and one of them
// replaces (len_old, n_free_in) is written by the last CTA to have read it.
// Bound by latency (lengths, scan, bisection, table entry, slots): 64 requests that grow by a few tokens 4.0 us,
// 512 requests with 0.8 million new tokens 8.4 us, 1.7 of them at the copy bandwidth.
__global__ void __launch_bounds__(kTabThreads) block_tables_kernel(const TabArgs g) {
  SPEC_TL(kTLTables);
  pdl_wait();
  pdl_trigger();
  extern __shared__ int tab_sm[];
  const int B = g.B, bs = g.bs, mb = g.mb;
  int* s_old = tab_sm;             // clamped lengths
  int* s_new = s_old + B;
  int* s_rel = s_new + B;          // inclusive prefix sums: blocks released,
  int* s_need = s_rel + B;         // blocks asked for,
  int* s_cnt = s_need + B;         // tokens asked for
  __shared__ int wsum[3][kTabThreads / 32];
  __shared__ int s_last;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool first_cta = blockIdx.x == 0;

  int n_free = *g.n_free_in;
  if (n_free < 0 || n_free > g.num_blocks) {
    if (first_cta && tid == 0) report(g.ws, SPEC_ERR_DEVICE, -1, n_free);
    n_free = n_free < 0 ? 0 : g.num_blocks;
  }
  int carry[3] = {0, 0, 0};
  for (int base = 0; base < B; base += kTabThreads) {
    const int b = base + tid;
    int x[3] = {0, 0, 0};
    if (b < B) {
      int o = g.len_old[b], n = g.len_new[b];
      const int most = mb * bs;
      if (o < 0 || o > most || n < 0 || n > most) {
        if (first_cta) report(g.ws, SPEC_ERR_DEVICE, b, n);
        o = o < 0 ? 0 : (o > most ? most : o);
        n = o;
      }
      s_old[b] = o;
      s_new[b] = n;
      const int have = (o + bs - 1) / bs, want = (n + bs - 1) / bs;
      x[0] = max(have - want, 0);
      x[1] = max(want - have, 0);
      x[2] = max(n - o, 0);
    }
#pragma unroll
    for (int i = 0; i < 3; ++i) {
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x[i], o);
        if (lane >= o) x[i] += y;
      }
      if (lane == 31) wsum[i][warp] = x[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      const int w = lane < kTabThreads / 32 ? wsum[i][lane] : 0;
      const int before = __reduce_add_sync(0xffffffffu, lane < warp ? w : 0);
      const int all = __reduce_add_sync(0xffffffffu, w);
      x[i] += carry[i] + before;
      carry[i] += all;
    }
    if (b < B) {
      s_rel[b] = x[0];
      s_need[b] = x[1];
      s_cnt[b] = x[2];
    }
    __syncthreads();
  }
  const int avail = n_free + carry[0], total = carry[2];
  // requests are served while their needs fit; the needs' prefix sums ascend, so the
  // served ones (and those that need nothing) are the requests before `cut`
  const int cut = carry[1] <= avail ? B : first_above(s_need, B, avail);
  const int taken = cut > 0 ? s_need[cut - 1] : 0;
  const int left = avail - taken;
  auto have_of = [&](int b) { return (s_old[b] + bs - 1) / bs; };
  auto is_served = [&](int b) { return b < cut || (b > 0 && s_need[b] == s_need[b - 1]); };
  auto want_of = [&](int b) { return is_served(b) ? (s_new[b] + bs - 1) / bs : have_of(b); };

  // this CTA has read what is replaced at the end; the answer is not looked at before that
  int* ctr = reinterpret_cast<int*>(static_cast<char*>(g.ws) + kWsHeader);
  int arrived = 0;
  if (tid == 0) asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;" : "=r"(arrived) : "l"(ctr) : "memory");

  const int gt = blockIdx.x * kTabThreads + tid, gn = gridDim.x * kTabThreads;
  // The warps take the four kinds of work below one after another, a kind beginning with the warp at which the
  // one before it ended: a warp has one or two pieces of one kind rather than the latencies of all four
  // (512 requests, 0.8 million new tokens: then 3 CTAs an SM: 13.8 -> 11.8 us).
  const int warps = gn >> 5;
  int begun = 0;
  auto first_piece = [&](long long pieces) {
    const int at = (gt >> 5) - begun;
    begun = (int)((begun + pieces) % warps);
    return at < 0 ? at + warps : at;
  };
  const bool out_of_place = g.table_out != g.table_in, pool_moves = g.free_out != g.free_in;
  auto on16 = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; };
  const bool vec_pool = on16(g.free_in) && on16(g.free_out);
  const bool vec_table = mb % 4 == 0 && on16(g.table_in) && on16(g.table_out);
  // the j-th id of the pool with the released blocks on top
  auto pool_id = [&](int j) {
    int id;
    if (j < n_free) {
      id = g.free_in[j];
    } else {
      const int r = j - n_free, b = first_above(s_rel, B, r);
      const int start = b > 0 ? s_rel[b - 1] : 0;
      const long long e = (long long)b * mb + (s_new[b] + bs - 1) / bs + (r - start);
      id = g.table_in[e];
      if (!out_of_place) g.table_out[e] = -1;
    }
    if ((unsigned)id >= (unsigned)g.num_blocks) {
      report(g.ws, SPEC_ERR_DEVICE, j, id);
      id = -1;
    }
    return id;
  };
  // what stays in the pool (an entry of the free list that stays where it is is not
  // written in place), and -1 past its end; four entries a thread
  for (int j0 = 128 * first_piece((g.num_blocks + 127) >> 7) + 4 * lane; j0 < g.num_blocks; j0 += 4 * gn) {
    const bool four = pool_moves && j0 + 4 <= g.num_blocks && vec_pool;
    if (four && j0 + 4 <= min(left, n_free)) {
      *reinterpret_cast<int4*>(g.free_out + j0) = *reinterpret_cast<const int4*>(g.free_in + j0);
    } else if (four && j0 >= left) {
      *reinterpret_cast<int4*>(g.free_out + j0) = make_int4(-1, -1, -1, -1);
    } else {
      for (int j = j0; j < min(j0 + 4, g.num_blocks); ++j) {
        if (j < left) {
          if (j >= n_free) g.free_out[j] = pool_id(j);
          else if (pool_moves) g.free_out[j] = g.free_in[j];
        } else if (pool_moves) {
          g.free_out[j] = -1;
        }
      }
    }
  }
  // deliveries: a lane takes a block and finds whose it is, then 2^lg lanes write a block's slots
  int lg = 0;
  while (lg < 5 && (1 << lg) < bs) ++lg;
  const int part = lane & ((1 << lg) - 1);
  constexpr int kTake = 16;                          // blocks of a warp (8 / 16 / 32: 9.9 / 8.7 / 9.0 us for 512 requests as below)
  for (int base = first_piece((taken + kTake - 1) / kTake) * kTake; base < taken; base += warps * kTake) {
    const int i = lane < kTake ? base + lane : taken;  // the i-th block taken
    int id = -1, first = 0, end = 0, to = 0;         // tokens [first, end) of the block, slot entry of token 0
    int e = 0;
    if (i < taken) {
      const int j = avail - 1 - i;
      id = pool_id(j);
      if (!pool_moves && j < n_free) g.free_out[j] = -1;
      const int b = first_above(s_need, B, i);
      e = have_of(b) + i - (b > 0 ? s_need[b - 1] : 0);
      g.table_out[(long long)b * mb + e] = id;
      to = (b > 0 ? s_cnt[b - 1] : 0) - s_old[b];
      first = max(s_old[b], e * bs);
      end = min(s_new[b], (e + 1) * bs);
    }
    const int valid = min(kTake, taken - base);
    for (int from0 = 0; from0 < valid; from0 += 32 >> lg) {
      const int from = (from0 + (lane >> lg)) & 31;
      const int id_ = __shfl_sync(0xffffffffu, id, from), end_ = __shfl_sync(0xffffffffu, end, from);
      const int to_ = __shfl_sync(0xffffffffu, to, from), e0 = __shfl_sync(0xffffffffu, e, from) * bs;
      for (int t = __shfl_sync(0xffffffffu, first, from) + part; t < end_; t += 1 << lg)
        if (to_ + t < g.cap) {
          g.slots[to_ + t] = id_ < 0 ? -1 : id_ * bs + (t - e0);
          if (g.pos) g.pos[to_ + t] = t;
        }
    }
  }
  // kept entries, and -1 past a request's blocks: a warp takes 128 entries of a row
  if (out_of_place) {
    const int segs = (mb + 127) >> 7;
    for (int task = first_piece((long long)B * segs); task < B * segs; task += warps) {
      const int b = task / segs, i0 = (task - b * segs) * 128 + 4 * lane, want = want_of(b), keep = min(have_of(b), want);
      const int32_t* in = g.table_in + (long long)b * mb + i0;
      int32_t* out = g.table_out + (long long)b * mb + i0;
      if (vec_table && i0 + 4 <= keep) {
        *reinterpret_cast<int4*>(out) = *reinterpret_cast<const int4*>(in);
      } else if (vec_table && i0 >= want && i0 + 4 <= mb) {
        *reinterpret_cast<int4*>(out) = make_int4(-1, -1, -1, -1);
      } else {
        for (int i = 0; i < 4 && i0 + i < mb; ++i) {
          if (i0 + i < keep) out[i] = in[i];
          else if (i0 + i >= want) out[i] = -1;
        }
      }
    }
  }
  // tokens of blocks that were there before, a warp a request; all tokens of a request
  // that is not served
  for (int b = first_piece(B); b < B; b += warps) {
    const int o = s_old[b], off = (b > 0 ? s_cnt[b - 1] : 0) - o;
    const bool ok = is_served(b);
    const int end = ok ? min(s_new[b], have_of(b) * bs) : s_new[b];
    if (o >= end) continue;
    int id = -1;
    if (ok) {
      id = g.table_in[(long long)b * mb + o / bs];
      if ((unsigned)id >= (unsigned)g.num_blocks) {
        if (lane == 0) report(g.ws, SPEC_ERR_DEVICE, b, id);
        id = -1;
      }
    }
    for (int t = o + lane; t < end; t += 32)
      if (off + t < g.cap) {
        g.slots[off + t] = id < 0 ? -1 : id * bs + t % bs;
        if (g.pos) g.pos[off + t] = t;
      }
  }
  for (int k = total + gt; k < g.cap; k += gn) {
    g.slots[k] = -1;
    if (g.pos) g.pos[k] = 0;
  }
  // by the last CTA to have read them: the lengths, the pool's size, the prefix sums
  if (tid == 0) {
    s_last = arrived == (int)gridDim.x - 1;
    if (s_last) *ctr = 0;
  }
  __syncthreads();
  if (!s_last) return;
  if (tid == 0) {
    *g.n_free_out = min(left, g.num_blocks);
    if (carry[1] > avail || total > g.cap) report(g.ws, SPEC_ERR_CAPACITY, carry[1], avail);
    if (left > g.num_blocks) report(g.ws, SPEC_ERR_DEVICE, left, g.num_blocks);
    g.cu_new[0] = 0;
  }
  for (int b = tid; b < B; b += kTabThreads) {
    g.cu_new[b + 1] = s_cnt[b];
    g.len_out[b] = is_served(b) ? s_new[b] : s_old[b];
  }
}

// ---------------------------------------------------------------- K/V append
template <typename T> struct alignas(sizeof(T) == 1 ? 8 : 16) Vec8 { T v[8]; };   // eight elements: 32, 16 or 8 bytes

SPEC_DEV float to_f(float x) { return x; }
SPEC_DEV float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
SPEC_DEV float to_f(__half x) { return __half2float(x); }

// Value in the cache's type.  E4M3: the fp32 quotient x / scale, then one rounding to
// nearest even, saturating.  The quotient itself takes more instructions than the
// copy can hide, so it is only taken where it matters: with a power of two for scale
// the product with its reciprocal is the quotient; otherwise the product is within 2
// steps of it, and rounds the same way unless it lies next to a border between two
// 8-bit values (a middle of the 20 bits that are dropped, or a number too small for
// the type's normal ones).  A scale whose reciprocal fp32 holds in fewer bits or not at all
// has NaN for it (reciprocal()), and the quotient is taken every time.
template <typename T, typename C, bool EXACT> SPEC_DEV C stored(T x, float scale, float inv) {
  if constexpr (sizeof(C) == 1) {
    float y = to_f(x) * inv;
    if constexpr (!EXACT) {
      const uint32_t past = (__float_as_uint(y) + 4u - 0x80000u) & 0xfffffu;
      if (past < 8u || !(fabsf(y) >= 0.015625f)) y = __fdiv_rn(to_f(x), scale);
    }
    return __nv_cvt_float_to_fp8(y, __NV_SATFINITE, __NV_E4M3);
  } else {
    return x;
  }
}
SPEC_DEV float reciprocal(float s) {
  return s >= 1.17549435e-38f && s <= 8.50705917e37f ? 1.f / s : NAN;      // 2^-126 .. 2^126
}
static bool power_of_two(float s) {
  int e;
  return frexpf(s, &e) == 0.5f && e > -120 && e < 120;
}

// Rows to slots, bound by the bytes moved.  2^lg lanes share a row (as many as it
// has vectors of eight elements, at most a warp), blockIdx.y picks K or V.  Measured: 32768 rows of 1024 bf16,
// slices of a fused product, into 8 bits 27.9 us (7.2 TB/s: the last writes stay in L2), 256 rows 1.8 us.
template <typename T, typename C, bool VEC, bool EXACT>
__global__ void __launch_bounds__(256) cache_append_kernel(const T* __restrict__ k, const T* __restrict__ v,
                                                           long long k_ld, long long v_ld,
                                                           const int32_t* __restrict__ slots, int n,
                                                           C* __restrict__ ck, C* __restrict__ cv, int width,
                                                           int num_slots, float k_scale, float v_scale, int lg,
                                                           void* ws) {
  SPEC_TL(kTLAppend);
  pdl_wait();
  pdl_trigger();
  const T* __restrict__ src = blockIdx.y ? v : k;
  C* __restrict__ dst = blockIdx.y ? cv : ck;
  const float scale = blockIdx.y ? v_scale : k_scale, inv = reciprocal(scale);
  const int per = 1 << lg, part = threadIdx.x & (per - 1);
  const long long row = (long long)blockIdx.x * (256 >> lg) + (threadIdx.x >> lg);
  if (row >= n) return;
  const T* s = src + row * (blockIdx.y ? v_ld : k_ld);
  if constexpr (VEC) {
    // four vectors on their way before the slot is looked at
    constexpr int kBatch = 4;
    const int nv = width >> 3;
    int slot = 0;
    for (int i0 = part; i0 < nv; i0 += kBatch * per) {
      Vec8<T> x[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j)
        if (i0 + j * per < nv) {
          const uint4* p = reinterpret_cast<const uint4*>(s + 8 * (i0 + j * per));
          uint4* q = reinterpret_cast<uint4*>(&x[j]);
          q[0] = __ldcs(p);
          if constexpr (sizeof(T) == 4) q[1] = __ldcs(p + 1);
        }
      if (i0 == part) {
        slot = slots[row];
        if (slot < 0 || slot >= num_slots) {
          if (slot != -1 && part == 0) report(ws, SPEC_ERR_DEVICE, (int)row, slot);
          return;
        }
      }
      C* d = dst + (long long)slot * width;
#pragma unroll
      for (int j = 0; j < kBatch; ++j)
        if (i0 + j * per < nv) {
          Vec8<C> o;
#pragma unroll
          for (int e = 0; e < 8; ++e) o.v[e] = stored<T, C, EXACT>(x[j].v[e], scale, inv);
          C* w = d + 8 * (i0 + j * per);
          if constexpr (sizeof(C) == 1) {
            *reinterpret_cast<uint2*>(w) = *reinterpret_cast<uint2*>(&o);
          } else {
            reinterpret_cast<uint4*>(w)[0] = reinterpret_cast<uint4*>(&o)[0];
            if constexpr (sizeof(C) == 4) reinterpret_cast<uint4*>(w)[1] = reinterpret_cast<uint4*>(&o)[1];
          }
        }
    }
  } else {
    const int slot = slots[row];
    if (slot < 0 || slot >= num_slots) {
      if (slot != -1 && part == 0) report(ws, SPEC_ERR_DEVICE, (int)row, slot);
      return;
    }
    C* d = dst + (long long)slot * width;
    for (int i = part; i < width; i += per) d[i] = stored<T, C, EXACT>(s[i], scale, inv);
  }
}

template <typename T, typename C>
static void launch_append(const spec_attn_desc& d, const void* k, long long k_ld, const void* v, long long v_ld,
                          const int32_t* slots, int n, const spec_kv& kv, void* ws, cudaStream_t st) {
  const int width = d.n_kv_heads * d.head_dim;
  int lg = 0;
  while (lg < 5 && (8 << lg) < width) ++lg;
  const bool vec = (k_ld * (long long)sizeof(T)) % 16 == 0 && (v_ld * (long long)sizeof(T)) % 16 == 0 && aligned(k, 16) &&
                   aligned(v, 16) && aligned(kv.k, 16) && aligned(kv.v, 16);
  const int rows = 256 >> lg;
  const dim3 grid((n + rows - 1) / rows, 2);
  auto* kern = vec ? cache_append_kernel<T, C, true, true> : cache_append_kernel<T, C, false, true>;
  if constexpr (sizeof(C) == 1)
    if (!power_of_two(d.k_scale) || !power_of_two(d.v_scale))
      kern = vec ? cache_append_kernel<T, C, true, false> : cache_append_kernel<T, C, false, false>;
  launch_pdl(kern, grid, dim3(256), 0, st, (const T*)k, (const T*)v, k_ld, v_ld, slots, n, (C*)kv.k, (C*)kv.v, width,
             (int)kv.num_slots, d.k_scale, d.v_scale, lg, ws);
}

}  // namespace spec

using namespace spec;

extern "C" size_t spec_block_tables_workspace_bytes(int32_t B) {
  return B <= 0 || B > kTabMaxB ? 0 : kWsHeader + 256;
}

extern "C" spec_status spec_block_tables(int32_t B, int32_t block_size, int32_t max_blocks, int32_t num_blocks,
                                         const int32_t* len_old, const int32_t* len_new, const int32_t* table_in,
                                         int32_t* table_out, const int32_t* free_in, const int32_t* n_free_in,
                                         int32_t* free_out, int32_t* n_free_out, int32_t* len_out, int32_t* cu_new,
                                         int32_t* slots, int32_t* pos, int32_t slots_cap, void* ws, size_t ws_bytes,
                                         spec_stream_t stream) {
  if (B <= 0 || block_size <= 0 || max_blocks <= 0 || num_blocks <= 0 || slots_cap <= 0) return SPEC_ERR_SHAPE;
  if (!len_old || !len_new || !table_in || !table_out || !free_in || !n_free_in || !free_out || !n_free_out ||
      !len_out || !cu_new || !slots)
    return SPEC_ERR_ARG;
  // token indices, slots, places in the slot map and pool positions (free and released ids together) are 32-bit integers
  const long long limit = 1ll << 30;
  if (B > kTabMaxB || (long long)max_blocks * block_size >= limit ||
      (long long)B * ((long long)max_blocks * block_size) >= limit || (long long)num_blocks * block_size >= limit ||
      slots_cap >= limit)
    return SPEC_ERR_CAPACITY;
  if (!ws || !aligned(ws, 256) || ws_bytes < spec_block_tables_workspace_bytes(B)) return SPEC_ERR_WORKSPACE;
  TabArgs a{B, block_size, max_blocks, num_blocks, slots_cap, len_old, len_new, table_in, free_in, n_free_in,
            table_out, free_out, n_free_out, len_out, cu_new, slots, pos, ws};
  // a CTA per 1024 items it may have to touch, up to two an SM: every CTA scans the requests for itself
  // (64 requests of 8000 tokens 4.1 / 4.0 / 4.6 us with 512 / 1024 / 2048 items a CTA; 512 requests, 0.8 million new
  // tokens, 1 / 2 / 3 CTAs an SM 10.2 / 8.7 / 10.7 us)
  const long long items = (table_out != table_in ? (long long)B * max_blocks : 0) + num_blocks + slots_cap;
  const int grid = (int)std::min<long long>(std::max<long long>(1, items / 1024), 2 * sm_count());
  const size_t smem = (size_t)5 * B * 4;
  if (smem > 47 * 1024 && cudaFuncSetAttribute(block_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               5 * kTabMaxB * 4) != cudaSuccess)
    return SPEC_ERR_CUDA;
  launch_pdl(block_tables_kernel, dim3(grid), dim3(kTabThreads), smem, stream, a);
  return last_launch();
}

extern "C" spec_status spec_cache_append(const spec_attn_desc* desc, const void* k, const void* v, int64_t ld,
                                         const int32_t* slots, int32_t n, const spec_kv* kv, void* ws,
                                         spec_stream_t stream) {
  return spec_cache_append_strided(desc, k, ld, v, ld, slots, n, kv, ws, stream);
}

extern "C" spec_status spec_cache_append_strided(const spec_attn_desc* desc, const void* k, int64_t k_ld, const void* v,
                                                 int64_t v_ld, const int32_t* slots, int32_t n, const spec_kv* kv,
                                                 void* ws, spec_stream_t stream) {
  if (!desc || !k || !v || !slots || !kv || !kv->k || !kv->v) return SPEC_ERR_ARG;
  const spec_attn_desc& d = *desc;
  if (d.n_kv_heads <= 0 || d.head_dim <= 0 || d.head_dim % 16 || d.head_dim > 256 || n <= 0 || kv->num_slots <= 0)
    return SPEC_ERR_SHAPE;
  if (d.dtype < SPEC_DTYPE_F32 || d.dtype > SPEC_DTYPE_F16) return SPEC_ERR_UNSUPPORTED;
  const bool e4m3 = d.kv_dtype == SPEC_DTYPE_E4M3 && d.dtype != SPEC_DTYPE_F32;
  if (d.kv_dtype != d.dtype && !e4m3) return SPEC_ERR_UNSUPPORTED;
  if (e4m3 && !(d.k_scale > 0 && d.v_scale > 0)) return SPEC_ERR_ARG;
  const long long width = (long long)d.n_kv_heads * d.head_dim;
  if (width >= (1ll << 30)) return SPEC_ERR_SHAPE;
  if (k_ld == 0) k_ld = width;
  if (v_ld == 0) v_ld = width;
  if (k_ld < width || v_ld < width) return SPEC_ERR_SHAPE;
  const size_t es = d.dtype == SPEC_DTYPE_F32 ? 4 : 2;
  if (!aligned(k, es) || !aligned(v, es) || (!e4m3 && (!aligned(kv->k, es) || !aligned(kv->v, es))))
    return SPEC_ERR_ALIGN;
  if (ws && !aligned(ws, 256)) return SPEC_ERR_WORKSPACE;
  if (d.dtype == SPEC_DTYPE_F32) launch_append<float, float>(d, k, k_ld, v, v_ld, slots, n, *kv, ws, stream);
  else if (d.dtype == SPEC_DTYPE_BF16 && !e4m3)
    launch_append<__nv_bfloat16, __nv_bfloat16>(d, k, k_ld, v, v_ld, slots, n, *kv, ws, stream);
  else if (d.dtype == SPEC_DTYPE_BF16)
    launch_append<__nv_bfloat16, uint8_t>(d, k, k_ld, v, v_ld, slots, n, *kv, ws, stream);
  else if (!e4m3) launch_append<__half, __half>(d, k, k_ld, v, v_ld, slots, n, *kv, ws, stream);
  else launch_append<__half, uint8_t>(d, k, k_ld, v, v_ld, slots, n, *kv, ws, stream);
  return last_launch();
}

// per-unit log setter of the instrumented build (no-op otherwise)
SPEC_TL_SETTER(tables)
