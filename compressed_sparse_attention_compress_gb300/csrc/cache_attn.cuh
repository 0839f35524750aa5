// cache_attn.cuh -- what the two cache attention kernels share: how the work is
// divided among the CTAs, the operations on codes, and how pieces become rows.
//
// Work.  R (query, head) rows that read one KV head form an item: 2^lq queries of
// one sequence x their G heads, or a part of one query's heads when G > R.  An
// item's keys are cut into tiles of 128; all tiles of all items, in order, are
// divided evenly among a grid that fills the GPU, so ragged batches and single
// long sequences load it alike.  An item that one CTA holds whole is written at
// once; the pieces of the others go to the workspace and a second, small kernel
// joins them in order (no atomics: the same bits every run).
//
// Sums.  With t = log2 scores and V scale 2^e, the value products use the weights
// 2^(t + e - M + kBase), M = max(t + e) as of the last time that a term exceeded it
// by kSlack, as halves; so neither the range of the scores nor that of the block
// scales leaves a half's range.  l = sum 2^t comes from the unrounded weights,
// held in float32 against 2^(M - kBase - e0), e0 the first key's e.  Where an e
// lies 60 or more from e0 that could leave float32, and the terms are summed
// against a maximum of their own ("far").
#pragma once

#include <math.h>

#include "cache.cuh"
#include "ws_sync.cuh"

namespace csa {
namespace cache_attn {

using ws::ex2;

constexpr int kTile = 128;             // keys of a tile
constexpr float kBase = 7.f;           // largest weight in the products when M is exact: 2^kBase ...
constexpr float kSlack = 8.f;          // ... and M may lag by this much (a half ends below 2^16)
constexpr float kNone = -3e38f;        // M before the first key
constexpr uint32_t kNoRow = 0xffffffffu;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// The rounding error of pack_f16x2, as halves.
__device__ __forceinline__ uint32_t rest_f16x2(uint32_t hi, float a, float b) {
  const float2 f = f16x2_to_float2(hi);
  return pack_f16x2(a - f.x, b - f.y);
}
__device__ __forceinline__ uint32_t widen_lo(uint32_t w) { return e4m3x2_to_f16x2((uint16_t)w); }
__device__ __forceinline__ uint32_t widen_hi(uint32_t w) { return e4m3x2_to_f16x2((uint16_t)(w >> 16)); }
// Exponent of a power of two.
__device__ __forceinline__ float exponent_of(float s) { return (float)((int)(__float_as_uint(s) >> 23) - 127); }
// Any NaN code (0x7f with either sign) among four.
__device__ __forceinline__ bool has_nan4(uint32_t w) { return (((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) != 0; }

// The same codes, NaN as 0.
__device__ __forceinline__ uint32_t without_nan4(uint32_t w) {
  const uint32_t nan = ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
  return w & ~(nan | (nan - (nan >> 7)));
}

struct Plan {  // what every CTA derives from the arguments
  int lq;      // queries of an item: 1 << lq
  int parts;   // items of one query group and KV head: ceil(G / R) when G > R
  int subs;    // H_kv * parts
  int slots;   // query groups, at most
  int cost;    // what an item costs beside its tiles, in tiles: queries, the first maxima, rows written
};

struct Slot {  // a query group
  int b, row0, nq, p0;  // sequence, first packed row, queries, position of the first
  int ct, rt;           // tiles of compressed entries, of raw rows
  int vis, w0;          // last query's visible entries (listed: k_pad); first raw position of the tiles
  bool bad;
};

// The order is in units: an item's `cost`, then one for each of its tiles.  Without the cost, CTAs that got the
// many short items of a prompt's first rows ran 38% longer than the mean.
struct Share {  // a CTA's units [u0, u1) of all `total`, and the slot that u0 lies in, which begins at slot_at
  int64_t total, grid, u0, u1, slot_at;
  int slot, cost;
  __device__ __forceinline__ int64_t of(int64_t cta) const { return cta >= grid ? total : total * cta / grid; }
};

// What every part of a kernel looks its work up in, in shared memory.
struct Context {
  CacheAttnArgs a;
  Plan pl;
  Share sh;
  int R;
};

// Query group `s`: sequences' groups start at floor(cu / 2^lq) + b, which leaves
// every sequence room for ceil(L / 2^lq).  nq = 0: none.
__device__ __forceinline__ Slot find_slot(const Context* ctx, const int32_t* cu, const int32_t* pos0, int s) {
  const CacheAttnArgs& a = ctx->a;
  const int lq = ctx->pl.lq;
  Slot r{};
  int lo = 0, hi = a.B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if ((cu[mid] >> lq) + mid <= s) lo = mid; else hi = mid - 1;
  }
  const int row0 = cu[lo], L = cu[lo + 1] - row0;
  const int64_t first = (int64_t)(s - ((row0 >> lq) + lo)) << lq;
  if (first < 0 || first >= L || row0 < 0 || (int64_t)row0 + L > a.T_cap) return r;
  r.b = lo;
  r.row0 = row0 + (int)first;
  r.nq = min(L - (int)first, 1 << lq);
  const int64_t end = (int64_t)pos0[lo] + L;
  r.bad = pos0[lo] < 0 || end > INT32_MAX || (a.raw.k && end > a.raw.cap) || (a.cmp.k && (int)end / a.r > a.cmp.cap);
  if (r.bad) {
    r.ct = 1;
    return r;
  }
  r.p0 = pos0[lo] + (int)first;
  const int p1 = r.p0 + r.nq - 1;
  if (a.cmp.k) {
    r.vis = a.idx ? a.k_pad : (p1 + 1) / a.r;
    r.ct = (r.vis + kTile - 1) / kTile;
  }
  if (a.raw.k) {
    r.w0 = max(0, r.p0 - a.window + 1) & ~15;  // 16 keys lie in one block
    r.rt = (p1 - r.w0) / kTile + 1;
  }
  if (r.ct + r.rt == 0) r.ct = 1;  // nothing in sight: the rows are still written
  return r;
}

// The same out of line, where a smaller kernel is worth more (setmaxnreg allows no calls).
static __device__ __noinline__ Slot call_find_slot(const Context* ctx, const int32_t* cu, const int32_t* pos0, int s) {
  return find_slot(ctx, cu, pos0, s);
}

// One piece of an item in the workspace: O [R][D], then m, M, l [R].
template <int D> __host__ __device__ constexpr int piece_floats(int R) { return R * (D + 4); }

// A row's joined sums: its lse is written, and its O is to be multiplied by both factors.
__device__ __forceinline__ float2 finish_factors(const CacheAttnArgs& a, int at, float m, float M, float l) {
  if (a.sink) {  // it joins the sum and has no value row
    const float s2 = __ldg(a.sink + at % a.H) * kLog2e, top = fmaxf(m, s2);
    l = l * ex2(m - top) + (s2 > kNone ? ex2(s2 - top) : 0.f);
    m = top;
  }
  if (a.lse) a.lse[at] = l == 0.f ? -INFINITY : (m + __log2f(l)) * kLn2;
  if (M == kNone && l == l) return make_float2(0.f, 0.f);  // no key in sight
  const float f = ex2(0.5f * (M - kBase - m));             // 2^(M - kBase - m) in two halves
  return make_float2(f, f / l);
}
template <typename T>
__device__ __forceinline__ void store_out(const CacheAttnArgs& a, int at, int D, int d4, float4 v, float2 f) {
  v.x = v.x * f.x * f.y, v.y = v.y * f.x * f.y, v.z = v.z * f.x * f.y, v.w = v.w * f.x * f.y;
  T* out = static_cast<T*>(a.out) + (int64_t)at * D + 4 * d4;
  if (sizeof(T) == 4) *reinterpret_cast<float4*>(out) = v;
  else *reinterpret_cast<uint2*>(out) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
}

// Every thread of the CTA; `scratch` is shared memory that is free until then.
template <int kThreads, bool kCalls>
__device__ __forceinline__ void split_tiles(const CacheAttnArgs& a, const Plan& pl, int R, Context* ctx,
                                            uint8_t* scratch, int scratch_bytes) {
  __shared__ int64_t s_sum[2][kThreads / 32];
  __shared__ int64_t s_at;
  __shared__ int s_slot;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int32_t* cu = a.cu;
  const int32_t* pos0 = a.pos0;
  if (tid == 0) {
    ctx->a = a;
    ctx->pl = pl;
    ctx->R = R;
  }
  if ((2 * (int64_t)a.B + 1) * 4 <= scratch_bytes) {  // searched by every thread
    int32_t* s_cu = reinterpret_cast<int32_t*>(scratch);
    for (int i = tid; i <= a.B; i += kThreads) {
      s_cu[i] = __ldg(a.cu + i);
      if (i < a.B) s_cu[a.B + 1 + i] = __ldg(a.pos0 + i);
    }
    cu = s_cu;
    pos0 = s_cu + a.B + 1;
  }
  __syncthreads();
  const int n_slots = a.B > 0 ? pl.slots : 0;
  const int per = (n_slots + kThreads - 1) / kThreads;
  const int slot0 = min(tid * per, n_slots), slot1 = min(slot0 + per, n_slots);
  int64_t mine = 0, items = 0;
  for (int s = slot0; s < slot1; ++s) {
    const Slot x = kCalls ? call_find_slot(ctx, cu, pos0, s) : find_slot(ctx, cu, pos0, s);
    if (x.nq) {
      mine += (int64_t)(x.ct + x.rt) * pl.subs;
      items += pl.subs;
    }
  }
  int64_t incl = mine, incl_items = items;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, incl, o), vi = __shfl_up_sync(0xffffffffu, incl_items, o);
    if (lane >= o) {
      incl += v;
      incl_items += vi;
    }
  }
  if (lane == 31) {
    s_sum[0][warp] = incl;
    s_sum[1][warp] = incl_items;
  }
  __syncthreads();
  Share sh;
  sh.total = 0;
  int64_t all_items = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) {
      incl += s_sum[0][w];
      incl_items += s_sum[1][w];
    }
    sh.total += s_sum[0][w];
    all_items += s_sum[1][w];
  }
  // Up to a tile a CTA, tiles alone are shared.  Above, the cost counts at once (from 2 tiles a CTA: 48 tokens
  // with 64 listed heads 25.7 us, from one 23.9).
  sh.cost = sh.total >= gridDim.x ? pl.cost : 0;
  sh.total += sh.cost * all_items;
  mine += sh.cost * items;
  incl += sh.cost * incl_items;
  sh.grid = min((int64_t)gridDim.x, sh.total);  // CTAs that get a unit or more; the rest none
  sh.u0 = sh.of(blockIdx.x);
  sh.u1 = sh.of((int64_t)blockIdx.x + 1);
  if (sh.u0 < sh.u1 && incl - mine <= sh.u0 && sh.u0 < incl) {
    int64_t at = incl - mine;
    int s = slot0;
    while (true) {
      const Slot x = kCalls ? call_find_slot(ctx, cu, pos0, s) : find_slot(ctx, cu, pos0, s);
      const int64_t n = x.nq ? (int64_t)(x.ct + x.rt + sh.cost) * pl.subs : 0;
      if (sh.u0 < at + n) break;
      at += n;
      ++s;
    }
    s_slot = s;
    s_at = at;
  }
  __syncthreads();
  if (tid == 0) {
    sh.slot = sh.u0 < sh.u1 ? s_slot : 0;
    sh.slot_at = sh.u0 < sh.u1 ? s_at : 0;
    ctx->sh = sh;
  }
  __syncthreads();
}

struct Item {
  Slot x;
  int sub, kvh, h0, heads;   // which part; KV head; first head; heads of a query in this item
  int t0, t1, n_tiles;       // this CTA's tiles of the item's
  int vis;                   // entries that its first query sees
  int64_t item0;             // its first tile in the whole order
};

// The items of a CTA's share, one after the other.
struct Items {
  int64_t u, slot_at;
  int slot;
};
template <bool kCalls>
__device__ __forceinline__ bool next_item(const Context* ctx, Items* st, Item* out) {
  const CacheAttnArgs& a = ctx->a;
  const int R = ctx->R, parts = ctx->pl.parts, subs = ctx->pl.subs, G = a.H / a.H_kv;
  while (st->u < ctx->sh.u1) {
    Item& it = *out;
    it.x = kCalls ? call_find_slot(ctx, a.cu, a.pos0, st->slot) : find_slot(ctx, a.cu, a.pos0, st->slot);
    it.n_tiles = it.x.nq ? it.x.ct + it.x.rt : 0;
    const int cost = ctx->sh.cost, units = it.x.nq ? it.n_tiles + cost : 0;
    const int64_t n = (int64_t)units * subs;
    if (st->u >= st->slot_at + n) {
      st->slot_at += n;
      ++st->slot;
      continue;
    }
    it.sub = (int)((st->u - st->slot_at) / units);
    it.item0 = st->slot_at + (int64_t)it.sub * units + cost;
    it.t0 = (int)max(st->u - it.item0, (int64_t)0);
    it.t1 = (int)min(ctx->sh.u1 - it.item0, (int64_t)it.n_tiles);
    if (it.t1 <= 0) break;  // the share ends before its first tile
    it.kvh = it.sub / parts;
    it.h0 = it.kvh * G + (it.sub % parts) * R;
    it.heads = min(it.kvh * G + G - it.h0, G > R ? R : G);
    it.vis = it.x.bad || !a.cmp.k ? 0 : (it.x.p0 + 1) / a.r;
    st->u = it.item0 + it.t1;
    return true;
  }
  return false;
}

static __device__ __noinline__ bool call_next_item(const Context* ctx, Items* st, Item* out) {
  return next_item<true>(ctx, st, out);
}

// Position of key k of an item's tile t (-1: none), before a listed one is checked.
__device__ __forceinline__ int key_position(const CacheAttnArgs& a, const Item& it, int t, int k) {
  const Slot& x = it.x;
  if (x.bad || t >= it.t1) return -1;
  if (t < x.ct) {
    const int e = t * kTile + k;
    return e < x.vis ? (a.idx ? __ldg(a.idx + (int64_t)x.row0 * a.k_pad + e) : e) : -1;
  }
  const int p = x.w0 + (t - x.ct) * kTile + k;
  return p >= x.p0 - a.window + 1 && p < x.p0 + x.nq ? p : -1;
}
// That position once checked; problems raise the status.
__device__ __forceinline__ int checked_position(const CacheAttnArgs& a, const Item& it, int t, int pos) {
  if (t >= it.x.ct || !a.idx || pos < 0) return pos;
  const int64_t e = (int64_t)pos - (a.cu_cmp ? __ldg(a.cu_cmp + it.x.b) : 0);
  if (e >= 0 && e < it.vis) return (int)e;
  raise_status(a.status, CSA_ERR_DEVICE_BOUNDS);
  return -1;
}
__device__ __forceinline__ int table_entry(const CacheAttnArgs& a, const Item& it, int t, int pos) {
  const CacheView& c = t < it.x.ct ? a.cmp : a.raw;
  return pos >= 0 ? __ldg(c.table + (int64_t)it.x.b * c.max_blocks + (pos >> c.log_block)) : 0;
}
// Its row in the cache: (block * H_kv + head) * block rows + row.
__device__ __forceinline__ uint32_t cache_row(const CacheAttnArgs& a, const Item& it, int t, int pos, int blk) {
  const CacheView& c = t < it.x.ct ? a.cmp : a.raw;
  if (pos < 0) return kNoRow;
  if (blk >= 0 && blk < c.n_blocks)
    return ((uint32_t)(blk * a.H_kv + it.kvh) << c.log_block) + (pos & ((1 << c.log_block) - 1));
  raise_status(a.status, CSA_ERR_DEVICE_BOUNDS);
  return kNoRow;
}

// Notes an item that goes on in later CTAs: its rows, its part, the CTA of its last tile.
__device__ __forceinline__ void note_split(const Context* ctx, int row0, int nq, int sub, int64_t item0, int n_tiles,
                                        int4* meta) {
  const Share& sh = ctx->sh;
  const int64_t last = item0 + n_tiles - 1;
  int64_t cta = (last * sh.grid) / sh.total;
  while (sh.of(cta + 1) <= last) ++cta;
  while (sh.of(cta) > last) --cta;
  *meta = make_int4(row0, nq, sub, (int)cta);
}

// Rows that belong to no sequence: zeros, lse -inf.
template <typename T, int D>
__device__ __forceinline__ void capacity_rows(const CacheAttnArgs& a, int t, int n_t) {  // thread t of n_t of the CTA
  const int r0 = max(__ldg(a.cu + a.B), 0);
  T* out = static_cast<T*>(a.out);
  const int64_t n = ((int64_t)a.T_cap - r0) * a.H, step = (int64_t)gridDim.x * n_t;
  for (int64_t i = (int64_t)blockIdx.x * n_t + t; i < n * (D / 8); i += step) {
    uint4* o = reinterpret_cast<uint4*>(out + (int64_t)r0 * a.H * D) + i * (sizeof(T) / 2);
    o[0] = make_uint4(0, 0, 0, 0);
    if (sizeof(T) == 4) o[1] = make_uint4(0, 0, 0, 0);
  }
  if (a.lse)
    for (int64_t i = (int64_t)blockIdx.x * n_t + t; i < n; i += step)
      a.lse[(int64_t)r0 * a.H + i] = -INFINITY;
}

// Joins the pieces of the item that begins in CTA blockIdx.x's share and goes on
// in later ones; a warp per row.  Lanes hold the pieces' factors, 32 at a time, so that
// the rows' loads depend on nothing (one sequence of 128K rows has 57 pieces an item).
constexpr int kJoinWarps = 4;
template <typename T, int D, int R>
__global__ void __launch_bounds__(32 * kJoinWarps)
cache_attn_join_kernel(const CacheAttnArgs a, const Plan pl, const float* __restrict__ ws_o,
                       const int4* __restrict__ ws_meta) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4 meta = ws_meta[blockIdx.x];
  if (meta.x < 0) return;
  const int lane = threadIdx.x & 31, r = blockIdx.y * kJoinWarps + (threadIdx.x >> 5);
  const int G = a.H / a.H_kv, sub = meta.z, first = blockIdx.x, last = meta.w;
  const int kvh = sub / pl.parts, h0 = kvh * G + (sub % pl.parts) * R;
  const int heads = min(kvh * G + G - h0, G > R ? R : G);
  const int qi = G > R ? 0 : r / G, h = G > R ? r : r % G;
  if (qi >= meta.y || h >= heads) return;
  auto piece = [&](int cta) { return ws_o + ((int64_t)cta * 2 + (cta == first ? 1 : 0)) * piece_floats<D>(R); };
  float m = kNone, M = kNone;
  for (int k = first + lane; k <= last; k += 32) {
    m = fmaxf(m, piece(k)[R * D + r]);
    M = fmaxf(M, piece(k)[R * D + R + r]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  }
  float l = 0.f;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  const int d4 = lane % (D / 4);
  for (int k0 = first; k0 <= last; k0 += 32) {
    float f = 0.f;
    if (k0 + lane <= last) {
      const float* p = piece(k0 + lane) + R * D + r;
      f = ex2(p[R] - M);
      l += p[2 * R] * ex2(p[0] - m);
    }
    const int n = min(last - k0 + 1, 32);
#pragma unroll 1
    for (int j0 = 0; j0 < n; j0 += 8) {
      float4 x[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        x[j] = j0 + j < n ? *reinterpret_cast<const float4*>(piece(k0 + j0 + j) + r * D + 4 * d4)
                          : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float fj = __shfl_sync(0xffffffffu, f, j0 + j);
        v.x += x[j].x * fj, v.y += x[j].y * fj, v.z += x[j].z * fj, v.w += x[j].w * fj;
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  const int at = (meta.x + qi) * a.H + h0 + h;
  if (lane < D / 4) store_out<T>(a, at, D, d4, v, finish_factors(a, at, m, M, l));
}

// A CTA holds 2^lq queries of G heads, or a part of a query's heads.
inline Plan make_plan(const CacheAttnArgs& a, int R, int cost) {
  const int G = a.H / a.H_kv;
  Plan pl{};
  while (!a.idx && (2 << pl.lq) * G <= R) ++pl.lq;
  pl.parts = G > R ? (G + R - 1) / R : 1;
  pl.subs = a.H_kv * pl.parts;
  pl.slots = (a.T_cap >> pl.lq) + a.B;
  pl.cost = cost;
  return pl;
}

// The workspace: a word group per CTA on the item that begins there and goes on,
// two pieces per CTA, and `warps` warps' far sums.
struct Scratch {
  int4* meta;
  float* pieces;
  float* far;
};
template <int D> inline Scratch scratch_of(void* ws, int grid, int R) {
  Scratch s;
  s.meta = static_cast<int4*>(ws);
  s.pieces = reinterpret_cast<float*>(s.meta + grid);
  s.far = s.pieces + (size_t)grid * 2 * piece_floats<D>(R);
  return s;
}
inline size_t scratch_bytes(int grid, int R, int d, int warps) {
  return (size_t)grid * (sizeof(int4) + sizeof(float) * ((size_t)R * (2 * (d + 4)) + (size_t)warps * 2 * R));
}

}  // namespace cache_attn
}  // namespace csa
