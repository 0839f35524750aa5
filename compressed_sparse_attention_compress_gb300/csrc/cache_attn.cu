// cache_attn.cu -- attention of new query rows over the 8-bit serving cache
// (csa_cache_attn_fwd): cached compressed entries (every visible one, or those
// listed) and a window of cached raw rows in one softmax.
//
// Work.  R = 16 or 32 (query, head) rows that read one KV head form an item:
// 2^lq queries of one sequence x their G heads, or a part of one query's heads
// when G > R.  An item's keys are cut into tiles of 64; all tiles of all items,
// in order, are divided evenly among a grid that fills the GPU, so ragged
// batches and single long sequences load it alike.  An item that one CTA holds
// whole is written at once; the pieces of the others go to the workspace and a
// second, small kernel joins them in order (no atomics: the same bits every run).
//
// A tile.  Each of the four warps takes 16 of its keys through a ring of its own
// (cp.async, no CTA-wide barrier): codes are widened to halves in registers
// (exact), S = Q K^T and O += P V run on m16n8k16 products with float32 sums.
// A decode step moves 2 d bytes per key and head against 4 d G FLOP, so with up
// to 16 rows a tile it is bound by HBM, and codes go from shared memory straight
// into product fragments: a thread's 16 consecutive codes of a K row serve four
// k-steps (the order of the dims within a product is free), and four V rows are
// interleaved bytewise before widening.
//
// Numbers.  A query row is scaled by a power of two so that its largest element
// is in [2^14, 2^15): bf16 queries are then exact as halves down to 2^-38 of it.
// float32 queries and weights go in as two halves (22 bits).  With t = log2
// scores and V scale 2^e: l = sum 2^(t - m) with m = max t in float32; the value
// products use w = 2^(t + e - M + 15), M = max(t + e), as halves, so neither the
// range of the scores nor that of the block scales leaves a half's range.
#include <math.h>

#include "cache.cuh"
#include "ws_sync.cuh"

namespace csa {

namespace {

using ws::ex2;

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kStep = 16;              // keys of a warp's step
constexpr int kTile = kStep * kWarps;  // keys of a tile
constexpr int kSeqSmem = 1024;         // so many sequences' offsets are kept in shared memory
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint4& a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}
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
__device__ __forceinline__ float2 lds_f2(uint32_t a) {
  float2 v;
  asm volatile("ld.shared.v2.f32 {%0,%1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ void cp_async_4_zfill(uint32_t dst, const void* src, bool valid) {
  const int n = valid ? 4 : 0;
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;\n" ::"r"(dst), "l"(src), "r"(n));
}
// Any NaN code (0x7f with either sign) among four.
__device__ __forceinline__ bool has_nan4(uint32_t w) { return (((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) != 0; }

// Byte offset of 16-byte chunk `ch` of row `row` in a 16-row tile of codes.  The
// chunks of a 128-byte line are permuted so that the eight lanes of a 16-byte
// read phase hit all banks: K reads take four chunks of two neighbouring rows,
// V reads a chunk pair of every other row.
template <int D> __device__ __forceinline__ int code_offset(int row, int ch) {
  if (D == 128) return row * 128 + ((ch ^ (((row >> 1) & 1) << 1 | (((row >> 2) ^ row) & 1) << 2)) << 4);
  const int line = row >> 1;
  return line * 128 + ((((row & 1) * 4 + ch) ^ ((line & 3) << 1)) << 4);
}

struct Plan {  // what every CTA derives from the arguments
  int lq;      // queries of an item: 1 << lq
  int parts;   // items of one query group and KV head: ceil(G / R) when G > R
  int subs;    // H_kv * parts
  int slots;   // query groups, at most
};

struct Slot {  // a query group
  int b, row0, nq, p0;  // sequence, first packed row, queries, position of the first
  int ct, rt;           // tiles of compressed entries, of raw rows
  int vis, w0;          // last query's visible entries (listed: k_pad); first raw position of the tiles
  bool bad;
};

// Query group `s`: sequences' groups start at floor(cu / 2^lq) + b, which leaves
// every sequence room for ceil(L / 2^lq).  nq = 0: none.
__device__ __forceinline__ Slot find_slot(const CacheAttnArgs& a, const Plan& pl, const int32_t* cu,
                                          const int32_t* pos0, int s) {
  Slot r{};
  int lo = 0, hi = a.B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if ((cu[mid] >> pl.lq) + mid <= s) lo = mid; else hi = mid - 1;
  }
  const int row0 = cu[lo], L = cu[lo + 1] - row0;
  const int64_t first = (int64_t)(s - ((row0 >> pl.lq) + lo)) << pl.lq;
  if (first < 0 || first >= L || row0 < 0 || (int64_t)row0 + L > a.T_cap) return r;
  r.b = lo;
  r.row0 = row0 + (int)first;
  r.nq = min(L - (int)first, 1 << pl.lq);
  const int64_t end = (int64_t)pos0[lo] + L;
  r.bad = pos0[lo] < 0 || end > INT32_MAX || (a.raw.k && end > a.raw.cap) || (a.cmp.k && end / a.r > a.cmp.cap);
  if (r.bad) {
    r.ct = 1;
    return r;
  }
  r.p0 = pos0[lo] + (int)first;
  const int p1 = r.p0 + r.nq - 1;
  if (a.cmp.k) {
    r.vis = a.idx ? a.k_pad : (int)(((int64_t)p1 + 1) / a.r);
    r.ct = (r.vis + kTile - 1) / kTile;
  }
  if (a.raw.k) {
    r.w0 = max(0, r.p0 - a.window + 1) & ~(kStep - 1);  // a step's 16 keys lie in one block
    r.rt = (p1 - r.w0) / kTile + 1;
  }
  if (r.ct + r.rt == 0) r.ct = 1;  // nothing in sight: the rows are still written
  return r;
}

template <int D, int MT, bool kSplit, bool kShared> struct Layout {
  static constexpr int R = 16 * MT;
  static constexpr int kCodes = kStep * D;                                   // bytes of 16 rows
  static constexpr int kStage = kCodes * (kShared ? 1 : 2) + 2 * kStep * 4;  // K, V, their scales
  // copies of kStages - 1 steps are in flight: 96 KB an SM at 128 dims with separate V
  static constexpr int kStages = D == 128 && !kShared && MT == 1 ? 3 : 4;
  static constexpr int kRing = kStages * kStage * kWarps;
  static constexpr int kMerge = kWarps * R * D * 4;
  static constexpr int kBuf = kRing > kMerge ? kRing : kMerge;
  static constexpr int kQ = MT * (D / 16) * 32 * 16 * (kSplit ? 2 : 1);      // query fragments
  static constexpr int kSmem = kBuf + kQ;
  static constexpr bool kQRegs = MT == 1 && !kSplit;                         // fragments held in registers
};

// One piece of an item in the workspace: O [R][D], then m, M, l [R].
template <int D> __host__ __device__ constexpr int piece_floats(int R) { return R * (D + 4); }

// A row's result from its joined sums: four dims of it, and with the first ones its lse.
template <typename T, int D>
__device__ __forceinline__ void finish_row(const CacheAttnArgs& a, int at, int d4, float4 v, float m, float M, float l) {
  if (a.sink) {  // it joins the sum and has no value row
    const float s2 = __ldg(a.sink + at % a.H) * kLog2e, top = fmaxf(m, s2);
    if (top > -INFINITY) {
      l = (m == -INFINITY ? l : l * ex2(m - top)) + ex2(s2 - top);
      m = top;
    }
  }
  if (M == -INFINITY && l == l) v = make_float4(0.f, 0.f, 0.f, 0.f);  // no key in sight
  else {
    const float f = ex2(0.5f * (M - 15.f - m)), f2 = f / l;           // 2^(M - 15 - m) in two halves
    v.x = v.x * f * f2, v.y = v.y * f * f2, v.z = v.z * f * f2, v.w = v.w * f * f2;
  }
  T* out = static_cast<T*>(a.out) + (int64_t)at * D + 4 * d4;
  if (sizeof(T) == 4) *reinterpret_cast<float4*>(out) = v;
  else *reinterpret_cast<uint2*>(out) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
  if (d4 == 0 && a.lse) a.lse[at] = l == 0.f ? -INFINITY : (m + __log2f(l)) * kLn2;
}

template <typename T, int D, int MT, bool kShared>
__global__ void __launch_bounds__(kThreads, MT == 1 ? 3 : 2)
cache_attn_kernel(const CacheAttnArgs a, const Plan pl, float* __restrict__ ws_o, int4* __restrict__ ws_meta) {
  constexpr bool kSplit = sizeof(T) == 4;
  using L = Layout<D, MT, kSplit, kShared>;
  constexpr int R = L::R, kStages = L::kStages;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ int s_cu[kSeqSmem + 1], s_pos[kSeqSmem];
  __shared__ int64_t s_sum[kWarps];
  __shared__ int64_t s_at;
  __shared__ int s_slot;
  __shared__ float s_qf[R];                       // a row's query is q * 2^-e; 2^e
  __shared__ int s_p[R];                          // a row's position, -1: no such row
  __shared__ int s_out[R];                        // and its place: packed row * H + head
  __shared__ float s_m[kWarps][R], s_M[kWarps][R], s_l[kWarps][R];

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, c = lane & 3;
  const int G = a.H / a.H_kv;
  const uint32_t buf = smem_u32(smem), qbuf = buf + L::kBuf;
  asm volatile("griddepcontrol.launch_dependents;");

  // ---- this CTA's share of the tiles ----
  const int32_t* cu = a.cu;
  const int32_t* pos0 = a.pos0;
  if (a.B <= kSeqSmem) {
    for (int i = tid; i <= a.B; i += kThreads) {
      s_cu[i] = __ldg(a.cu + i);
      if (i < a.B) s_pos[i] = __ldg(a.pos0 + i);
    }
    __syncthreads();
    cu = s_cu;
    pos0 = s_pos;
  }
  const int n_slots = a.B > 0 ? pl.slots : 0;
  const int per = (n_slots + kThreads - 1) / kThreads;
  const int slot0 = min(tid * per, n_slots), slot1 = min(slot0 + per, n_slots);
  int64_t mine = 0;
  for (int s = slot0; s < slot1; ++s) {
    const Slot x = find_slot(a, pl, cu, pos0, s);
    if (x.nq) mine += (int64_t)(x.ct + x.rt) * pl.subs;
  }
  int64_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) s_sum[warp] = incl;
  __syncthreads();
  int64_t total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) incl += s_sum[w];
    total += s_sum[w];
  }
  const int64_t grid = min((int64_t)gridDim.x, total);  // CTAs that get a tile or more; the rest none
  auto share = [&](int64_t cta) { return cta >= grid ? total : total * cta / grid; };
  const int64_t u0 = share(blockIdx.x), u1 = share((int64_t)blockIdx.x + 1);
  if (tid == 0) ws_meta[blockIdx.x] = make_int4(-1, 0, 0, 0);
  if (u0 < u1 && incl - mine <= u0 && u0 < incl) {
    int64_t at = incl - mine;
    int s = slot0;
    while (true) {
      const Slot x = find_slot(a, pl, cu, pos0, s);
      const int64_t n = x.nq ? (int64_t)(x.ct + x.rt) * pl.subs : 0;
      if (u0 < at + n) break;
      at += n;
      ++s;
    }
    s_slot = s;
    s_at = at;
  }
  __syncthreads();

  // ---- rows that belong to no sequence ----
  {
    const int r0 = max(__ldg(a.cu + a.B), 0);
    T* out = static_cast<T*>(a.out);
    const int64_t n = ((int64_t)a.T_cap - r0) * a.H;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + tid; i < n * (D / 8); i += (int64_t)gridDim.x * kThreads) {
      uint4* o = reinterpret_cast<uint4*>(out + (int64_t)r0 * a.H * D) + i * (sizeof(T) / 2);
      o[0] = make_uint4(0, 0, 0, 0);
      if (sizeof(T) == 4) o[1] = make_uint4(0, 0, 0, 0);
    }
    if (a.lse)
      for (int64_t i = (int64_t)blockIdx.x * kThreads + tid; i < n; i += (int64_t)gridDim.x * kThreads)
        a.lse[(int64_t)r0 * a.H + i] = -INFINITY;
  }

  const uint32_t ring = buf + warp * (kStages * L::kStage);
  // lane constants of the fragment reads
  int off_k[D / 64], off_v[2];
#pragma unroll
  for (int h = 0; h < D / 64; ++h) off_k[h] = code_offset<D>(g, c + 4 * h);
#pragma unroll
  for (int e = 0; e < 2; ++e)
    off_v[e] = D == 128 ? code_offset<D>(2 * c + e, g) : code_offset<D>(2 * c + e, g >> 1) + (g & 1) * 8;

  int64_t u = u0;
  int slot = u0 < u1 ? s_slot : 0;
  int64_t slot_at = u0 < u1 ? s_at : 0;
  while (u < u1) {
    // ---- the next item: query group, KV head, part of the heads, tiles [t0, t1) ----
    Slot x = find_slot(a, pl, cu, pos0, slot);
    const int64_t n_tiles = x.nq ? x.ct + x.rt : 0;
    if (u >= slot_at + n_tiles * pl.subs) {
      slot_at += n_tiles * pl.subs;
      ++slot;
      continue;
    }
    const int sub = (int)((u - slot_at) / n_tiles);
    const int64_t item0 = slot_at + sub * n_tiles;
    const int t0 = (int)(u - item0), t1 = (int)min(u1 - item0, n_tiles);
    const int kvh = sub / pl.parts, h0 = kvh * G + (sub % pl.parts) * R;
    const int heads = min(kvh * G + G - h0, G > R ? R : G);  // heads of a query in this item
    if (x.bad && tid == 0) raise_status(a.status, CSA_ERR_DEVICE_BOUNDS);

    // step t of this warp: 16 keys; its rows are resolved a step before the copies are issued
    auto position = [&](int t) -> int {  // of key lane & 15; -1: not there
      const int k = t * kTile + warp * kStep + (lane & 15);
      if (x.bad || t >= t1) return -1;
      if (t < x.ct) {
        if (k >= x.vis) return -1;
        if (!a.idx) return k;
        const int v = __ldg(a.idx + (int64_t)x.row0 * a.k_pad + k);
        if (v < 0) return -1;
        const int64_t e = (int64_t)v - (a.cu_cmp ? __ldg(a.cu_cmp + x.b) : 0);
        if (e >= 0 && e < ((int64_t)x.p0 + 1) / a.r) return (int)e;
        raise_status(a.status, CSA_ERR_DEVICE_BOUNDS);
        return -1;
      }
      const int p = x.w0 + k - x.ct * kTile;
      return p >= x.p0 - a.window + 1 && p < x.p0 + x.nq ? p : -1;
    };
    auto block_of = [&](int t, int pos) -> int {
      return pos >= 0 ? cache_block(t < x.ct ? a.cmp : a.raw, x.b, pos, a.status) : -1;
    };
    auto copy = [&](int t, int pos, int blk) {
      if (t < t1) {
        const CacheView& cc = t < x.ct ? a.cmp : a.raw;
        const uint32_t st = ring + (t % kStages) * L::kStage;
        const int bh = blk >= 0 ? blk * a.H_kv + kvh : -1;
        const int r = pos & ((1 << cc.log_block) - 1);
        constexpr int kPerRow = D / 16, kRowsPer = 32 / kPerRow;
#pragma unroll
        for (int i = 0; i < kStep / kRowsPer; ++i) {
          const int row = lane / kPerRow + i * kRowsPer, ch = lane % kPerRow;
          const int rb = __shfl_sync(0xffffffffu, bh, row), rr = __shfl_sync(0xffffffffu, r, row);
          const int64_t off = rb >= 0 ? ((((int64_t)rb << cc.log_block) + rr) * D + ch * 16) : 0;
          cp_async_16_zfill(st + code_offset<D>(row, ch), cc.k + off, rb >= 0);
          if (!kShared) cp_async_16_zfill(st + L::kCodes + code_offset<D>(row, ch), cc.v + off, rb >= 0);
        }
        const float* sc = lane < 16 || kShared ? cc.k_scale : cc.v_scale;
        cp_async_4_zfill(st + L::kStage - 2 * kStep * 4 + lane * 4, sc + max(bh, 0), bh >= 0);
      }
      cp_async_commit();
    };
    int pos_c, blk_c, pos_n;  // rows of the step to copy next, positions of the one after it
    {
      int pos[kStages], blk[kStages];
#pragma unroll
      for (int i = 0; i < kStages; ++i) pos[i] = position(t0 + i);
#pragma unroll
      for (int i = 0; i < kStages; ++i) blk[i] = block_of(t0 + i, pos[i]);
#pragma unroll
      for (int i = 0; i < kStages - 1; ++i) copy(t0 + i, pos[i], blk[i]);
      pos_c = pos[kStages - 1];
      blk_c = blk[kStages - 1];
      pos_n = position(t0 + kStages);
    }

    // ---- queries as product fragments, one warp a 16-row tile ----
    if (warp < MT) {
      float amax[2] = {0.f, 0.f};
      const T* src[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = warp * 16 + g + 8 * e;
        const int qi = G > R ? 0 : r / G, h = G > R ? r : r % G;
        const bool real = qi < x.nq && h < heads;
        const int at = real ? (x.row0 + qi) * a.H + h0 + h : -1;
        if (c == 0) {
          s_p[r] = real ? x.p0 + qi : -1;
          s_out[r] = at;
        }
        src[e] = at >= 0 ? static_cast<const T*>(a.q) + (int64_t)(x.row0 + qi) * a.H * D + (int64_t)(h0 + h) * D : nullptr;
      }
      float v[2][D / 4];  // this thread's 16-element chunks c (and c + 4)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int i = 0; i < D / 4; i += 4) {
          float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
          if (src[e]) {
            const T* p = src[e] + 16 * (c + 4 * (i / 16)) + i % 16;
            if (kSplit) {
              f = __ldg(reinterpret_cast<const float4*>(p));
            } else {
              const uint2 w = __ldg(reinterpret_cast<const uint2*>(p));
              f = make_float4(bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y));
            }
          }
          v[e][i] = f.x, v[e][i + 1] = f.y, v[e][i + 2] = f.z, v[e][i + 3] = f.w;
        }
#pragma unroll
        for (int i = 0; i < D / 4; ++i)
          if (fabsf(v[e][i]) < INFINITY) amax[e] = fmaxf(amax[e], fabsf(v[e][i]));
        amax[e] = fmaxf(amax[e], __shfl_xor_sync(0xffffffffu, amax[e], 1));
        amax[e] = fmaxf(amax[e], __shfl_xor_sync(0xffffffffu, amax[e], 2));
      }
      float inv[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        // largest element to [2^14, 2^15), as far as 2^e and 2^-e are normal numbers
        const int ex = max((int)(__float_as_uint(amax[e]) >> 23) - 127 - 14, -113);
        inv[e] = pow2i(-ex);
        if (c == 0) s_qf[warp * 16 + g + 8 * e] = pow2i(ex);
      }
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        uint4 hi, lo;
        uint32_t* hw = reinterpret_cast<uint32_t*>(&hi);
        uint32_t* lw = reinterpret_cast<uint32_t*>(&lo);
#pragma unroll
        for (int w = 0; w < 4; ++w) {  // a0: row g, first pair; a1: row g + 8; a2, a3: second pair
          const int e = w & 1, i = ks * 4 + (w >> 1) * 2;
          const float f0 = v[e][i] * inv[e], f1 = v[e][i + 1] * inv[e];
          hw[w] = pack_f16x2(f0, f1);
          lw[w] = rest_f16x2(hw[w], f0, f1);
        }
        const uint32_t at = qbuf + ((warp * (D / 16) + ks) * 32 + lane) * 16;
        asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(hi.x), "r"(hi.y), "r"(hi.z), "r"(hi.w));
        if (kSplit)
          asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at + L::kQ / 2), "r"(lo.x), "r"(lo.y), "r"(lo.z),
                       "r"(lo.w));
      }
    }
    __syncthreads();
    uint4 qr[L::kQRegs ? D / 16 : 1];
    if (L::kQRegs) {
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) qr[ks] = lds128(qbuf + (ks * 32 + lane) * 16);
    }
    float qf[MT][2], m[MT][2], M[MT][2], l[MT][2], o[MT][D / 8][4];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        qf[mt][e] = s_qf[mt * 16 + g + 8 * e];
        m[mt][e] = M[mt][e] = -INFINITY;
        l[mt][e] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < D / 8; ++i) o[mt][i][0] = o[mt][i][1] = o[mt][i][2] = o[mt][i][3] = 0.f;
    }
    const float scale_log2 = a.scale * kLog2e;

    for (int t = t0; t < t1; ++t) {
      cp_async_wait<kStages - 2>();
      __syncwarp();
      copy(t + kStages - 1, pos_c, blk_c);
      pos_c = pos_n;
      blk_c = block_of(t + kStages, pos_n);
      pos_n = position(t + kStages + 1);
      const uint32_t st = ring + (t % kStages) * L::kStage;
      const uint32_t sc = st + L::kStage - 2 * kStep * 4;
      float ks[4], ev[4];  // keys 2c, 2c + 1, 8 + 2c, 9 + 2c
      {
        const float2 k0 = lds_f2(sc + 8 * c), k1 = lds_f2(sc + 32 + 8 * c);
        const float2 v0 = lds_f2(sc + 64 + 8 * c), v1 = lds_f2(sc + 96 + 8 * c);
        ks[0] = k0.x, ks[1] = k0.y, ks[2] = k1.x, ks[3] = k1.y;
        ev[0] = v0.x, ev[1] = v0.y, ev[2] = v1.x, ev[3] = v1.y;
      }
      if (!__any_sync(0xffffffffu, fmaxf(fmaxf(ks[0], ks[1]), fmaxf(ks[2], ks[3])) > 0.f)) continue;  // no key here
#pragma unroll
      for (int i = 0; i < 4; ++i) ev[i] = (float)((int)(__float_as_uint(ev[i]) >> 23) - 127);
      // ---- S = Q K^T ----
      float s[MT][2][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int j = 0; j < 2; ++j) s[mt][j][0] = s[mt][j][1] = s[mt][j][2] = s[mt][j][3] = 0.f;
#pragma unroll
      for (int h = 0; h < D / 64; ++h) {
        const uint4 k0 = lds128(st + off_k[h]), k1 = lds128(st + off_k[h] + 8 * D);
        const uint32_t w0[4] = {k0.x, k0.y, k0.z, k0.w}, w1[4] = {k1.x, k1.y, k1.z, k1.w};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const uint32_t b00 = widen_lo(w0[w]), b01 = widen_hi(w0[w]), b10 = widen_lo(w1[w]), b11 = widen_hi(w1[w]);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            const uint32_t at = qbuf + ((mt * (D / 16) + h * 4 + w) * 32 + lane) * 16;
            const uint4 q = L::kQRegs ? qr[L::kQRegs ? h * 4 + w : 0] : lds128(at);
            mma_f16(s[mt][0], q, b00, b01);
            mma_f16(s[mt][1], q, b10, b11);
            if (kSplit) {
              const uint4 ql = lds128(at + L::kQ / 2);
              mma_f16(s[mt][0], ql, b00, b01);
              mma_f16(s[mt][1], ql, b10, b11);
            }
          }
        }
      }
      // ---- log2 scores, masks ----
      bool seen[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        seen[i] = ks[i] > 0.f;
        ks[i] *= scale_log2;
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int key = 2 * j + (e & 1);
            s[mt][j][e] = seen[key] ? s[mt][j][e] * ks[key] * qf[mt][e >> 1] : -INFINITY;
          }
      // a step that some of the item's queries see and others do not
      const bool entries = t < x.ct;
      const int first = entries ? t * kTile + warp * kStep : x.w0 + (t - x.ct) * kTile + warp * kStep;
      auto sees = [&](int p, int pos) {  // entry / row pos, query at p
        return entries ? pos < ((int64_t)p + 1) / a.r : pos <= p && pos > p - a.window;
      };
      bool mixed = false;
      if (x.nq > 1) {
        const int p1 = x.p0 + x.nq - 1;
        mixed = !sees(x.p0, first + kStep - 1) || !(entries || first > p1 - a.window);
        if (mixed) {
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int p = s_p[mt * 16 + g + 8 * e];
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (!sees(p, first + (i >> 1) * 8 + 2 * c + (i & 1))) s[mt][i >> 1][2 * e + (i & 1)] = -INFINITY;
            }
        }
      }
      // ---- softmax: l against m, the products' weights against M ----
      uint4 pa[MT], pl_[MT];
      bool grew = false;
      float beta[MT][2];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        float w[2][4];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float t4[4], u4[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            t4[i] = s[mt][i >> 1][2 * e + (i & 1)];
            u4[i] = t4[i] + ev[i];
          }
          float tm = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3]));
          float um = fmaxf(fmaxf(u4[0], u4[1]), fmaxf(u4[2], u4[3]));
          tm = fmaxf(tm, __shfl_xor_sync(0xffffffffu, tm, 1));
          um = fmaxf(um, __shfl_xor_sync(0xffffffffu, um, 1));
          tm = fmaxf(tm, __shfl_xor_sync(0xffffffffu, tm, 2));
          um = fmaxf(um, __shfl_xor_sync(0xffffffffu, um, 2));
          const float mn = fmaxf(m[mt][e], tm), Mn = fmaxf(M[mt][e], um);
          const float mu = mn == -INFINITY ? 0.f : mn, Mu = Mn == -INFINITY ? 0.f : Mn;
          float sum = 0.f;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            sum += ex2(t4[i] - mu);
            w[e][i] = ex2(u4[i] - Mu + 15.f);
          }
          l[mt][e] = l[mt][e] * ex2(m[mt][e] - mu) + sum;
          beta[mt][e] = ex2(M[mt][e] - Mu);
          grew |= Mn > M[mt][e];
          m[mt][e] = mn;
          M[mt][e] = Mn;
        }
        pa[mt] = make_uint4(pack_f16x2(w[0][0], w[0][1]), pack_f16x2(w[1][0], w[1][1]), pack_f16x2(w[0][2], w[0][3]),
                            pack_f16x2(w[1][2], w[1][3]));
        if (kSplit)
          pl_[mt] = make_uint4(rest_f16x2(pa[mt].x, w[0][0], w[0][1]), rest_f16x2(pa[mt].y, w[1][0], w[1][1]),
                               rest_f16x2(pa[mt].z, w[0][2], w[0][3]), rest_f16x2(pa[mt].w, w[1][2], w[1][3]));
      }
      if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int i = 0; i < D / 8; ++i) {
            o[mt][i][0] *= beta[mt][0];
            o[mt][i][1] *= beta[mt][0];
            o[mt][i][2] *= beta[mt][1];
            o[mt][i][3] *= beta[mt][1];
          }
      }
      // ---- O += P V: keys 2c, 2c + 1, 8 + 2c, 9 + 2c; column n of product i is dim n D / 8 + i ----
      constexpr int kWords = D / 32;
      uint32_t v[4][kWords];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t at = st + (kShared ? 0 : L::kCodes) + off_v[k & 1] + (k >> 1) * 8 * D;
        if (D == 128) {
          const uint4 q = lds128(at);
          v[k][0] = q.x, v[k][1] = q.y, v[k][kWords - 2] = q.z, v[k][kWords - 1] = q.w;
        } else {
          const uint2 q = lds64(at);
          v[k][0] = q.x, v[k][1] = q.y;
        }
      }
      bool nan = false;  // a NaN row that only some queries see must not reach the others as 0 * NaN
      if (mixed) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int w = 0; w < kWords; ++w) nan |= has_nan4(v[k][w]);
        nan = __any_sync(0xffffffffu, nan);
      }
#pragma unroll
      for (int w = 0; w < kWords; ++w) {
        uint32_t y0[2], y1[2];
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          y0[hh] = __byte_perm(v[0][w], v[1][w], hh ? 0x7362 : 0x5140);
          y1[hh] = __byte_perm(v[2][w], v[3][w], hh ? 0x7362 : 0x5140);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t b0 = (i & 1) ? widen_hi(y0[i >> 1]) : widen_lo(y0[i >> 1]);
          const uint32_t b1 = (i & 1) ? widen_hi(y1[i >> 1]) : widen_lo(y1[i >> 1]);
          if (!nan) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              mma_f16(o[mt][4 * w + i], pa[mt], b0, b1);
              if (kSplit) mma_f16(o[mt][4 * w + i], pl_[mt], b0, b1);
            }
          } else {  // query by query, without the rows that it does not see
            for (int qi = 0; qi < x.nq; ++qi) {
              uint32_t z0 = b0, z1 = b1;
              const int k0 = first + 2 * c, p = x.p0 + qi;
              if (!sees(p, k0)) z0 &= 0xffff0000u;
              if (!sees(p, k0 + 1)) z0 &= 0x0000ffffu;
              if (!sees(p, k0 + 8)) z1 &= 0xffff0000u;
              if (!sees(p, k0 + 9)) z1 &= 0x0000ffffu;
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) {
                float d[4] = {0.f, 0.f, 0.f, 0.f};
                mma_f16(d, pa[mt], z0, z1);
                if (kSplit) mma_f16(d, pl_[mt], z0, z1);
                if (s_p[mt * 16 + g] == p) o[mt][4 * w + i][0] += d[0], o[mt][4 * w + i][1] += d[1];
                if (s_p[mt * 16 + g + 8] == p) o[mt][4 * w + i][2] += d[2], o[mt][4 * w + i][3] += d[3];
              }
            }
          }
        }
      }
    }
    cp_async_wait<0>();

    // ---- join the four warps ----
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float sum = l[mt][e];
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        const int r = mt * 16 + g + 8 * e;
        if (c == 0) {
          s_m[warp][r] = m[mt][e];
          s_M[warp][r] = M[mt][e];
          s_l[warp][r] = sum;
        }
      }
    __syncthreads();  // the rings are free, too
    float* acc = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = mt * 16 + g + 8 * e;
        float top = s_M[0][r];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) top = fmaxf(top, s_M[w][r]);
        const float f = M[mt][e] == -INFINITY ? 0.f : ex2(M[mt][e] - top);
        // columns 2c and 2c + 1 of products 0 .. D / 8 - 1: dims [2c D/8, (2c + 2) D/8)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < D / 8; i += 4) {
            float4 v = make_float4(o[mt][i][2 * e + h], o[mt][i + 1][2 * e + h], o[mt][i + 2][2 * e + h],
                                   o[mt][i + 3][2 * e + h]);
            if (f == 0.f) v = make_float4(0.f, 0.f, 0.f, 0.f);
            v.x *= f, v.y *= f, v.z *= f, v.w *= f;
            *reinterpret_cast<float4*>(acc + (warp * R + r) * D + (2 * c + h) * (D / 8) + i) = v;
          }
      }
    __syncthreads();
    const bool whole = t0 == 0 && t1 == n_tiles;
    float* piece = ws_o + ((int64_t)blockIdx.x * 2 + (t0 == 0 ? 1 : 0)) * piece_floats<D>(R);
    for (int i = tid; i < R * (D / 4); i += kThreads) {
      const int r = i / (D / 4), d4 = i % (D / 4);
      const int at = s_out[r];
      if (at < 0) continue;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      float mm = -INFINITY, MM = -INFINITY, ll = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float4 f = *reinterpret_cast<const float4*>(acc + (w * R + r) * D + 4 * d4);
        v.x += f.x, v.y += f.y, v.z += f.z, v.w += f.w;
        mm = fmaxf(mm, s_m[w][r]);
        MM = fmaxf(MM, s_M[w][r]);
      }
#pragma unroll
      for (int w = 0; w < kWarps; ++w) ll += s_m[w][r] == -INFINITY ? s_l[w][r] : s_l[w][r] * ex2(s_m[w][r] - mm);
      if (!whole) {
        *reinterpret_cast<float4*>(piece + r * D + 4 * d4) = v;
        if (d4 == 0) {
          piece[R * D + r] = mm;
          piece[R * D + R + r] = MM;
          piece[R * D + 2 * R + r] = ll;
        }
        continue;
      }
      finish_row<T, D>(a, at, d4, v, mm, MM, ll);
    }
    if (!whole && t0 == 0 && tid == 0) {
      // the pieces of this item: this one, then the first pieces of the CTAs up to that of its last tile
      const int64_t last = item0 + n_tiles - 1;
      int64_t cta = (last * grid) / total;
      while (share(cta + 1) <= last) ++cta;
      while (share(cta) > last) --cta;
      ws_meta[blockIdx.x] = make_int4(x.row0, x.nq, sub, (int)cta);
    }
    __syncthreads();  // s_out, s_m and the buffers are taken again
    u = item0 + t1;
  }
}

// Joins the pieces of the item that begins in CTA blockIdx.x's share and goes on
// in later ones; a warp per row.
template <typename T, int D, int R>
__global__ void __launch_bounds__(kThreads)
cache_attn_join_kernel(const CacheAttnArgs a, const Plan pl, const float* __restrict__ ws_o,
                       const int4* __restrict__ ws_meta) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4 meta = ws_meta[blockIdx.x];
  if (meta.x < 0) return;
  const int lane = threadIdx.x & 31, r = blockIdx.y * kWarps + (threadIdx.x >> 5);
  const int G = a.H / a.H_kv, sub = meta.z, first = blockIdx.x, last = meta.w;
  const int kvh = sub / pl.parts, h0 = kvh * G + (sub % pl.parts) * R;
  const int heads = min(kvh * G + G - h0, G > R ? R : G);
  const int qi = G > R ? 0 : r / G, h = G > R ? r : r % G;
  if (qi >= meta.y || h >= heads) return;
  auto piece = [&](int cta) { return ws_o + ((int64_t)cta * 2 + (cta == first ? 1 : 0)) * piece_floats<D>(R); };
  float m = -INFINITY, M = -INFINITY;
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
#pragma unroll 4
  for (int k = first; k <= last; ++k) {
    const float* p = piece(k);
    const float4 x = *reinterpret_cast<const float4*>(p + r * D + 4 * d4);
    const float pm = p[R * D + r], pM = p[R * D + R + r], q = p[R * D + 2 * R + r];
    l += pm == -INFINITY ? q : q * ex2(pm - m);
    if (pM > -INFINITY) {
      const float f = ex2(pM - M);
      v.x += x.x * f, v.y += x.y * f, v.z += x.z * f, v.w += x.w * f;
    }
  }
  if (lane < D / 4) finish_row<T, D>(a, (meta.x + qi) * a.H + h0 + h, d4, v, m, M, l);
}

// Two row tiles a CTA where a KV head's queries fill them: more than 16 heads a
// group, or several queries a sequence (each key is then widened once for 32 rows).
int row_tiles(int T_cap, int B, int G, bool listed, bool fp32) {
  return !fp32 && (G > 16 || (!listed && (int64_t)T_cap > 4 * (int64_t)B)) ? 2 : 1;
}
constexpr int ctas_per_sm(int mt) { return mt == 1 ? 3 : 2; }

size_t ws_bytes(int sm_count, int mt, int d) {
  const size_t grid = (size_t)sm_count * ctas_per_sm(mt);
  return grid * (sizeof(int4) + 2 * sizeof(float) * (size_t)(16 * mt) * (d + 4));
}

template <typename T, int D, int MT, bool kShared>
cudaError_t run(const CacheAttnArgs& a, int sm_count, cudaStream_t stream) {
  using L = Layout<D, MT, sizeof(T) == 4, kShared>;
  const int G = a.H / a.H_kv;
  Plan pl{};
  while (!a.idx && (2 << pl.lq) * G <= L::R) ++pl.lq;
  pl.parts = G > L::R ? (G + L::R - 1) / L::R : 1;
  pl.subs = a.H_kv * pl.parts;
  pl.slots = (a.T_cap >> pl.lq) + a.B;
  const int grid = sm_count * ctas_per_sm(MT);
  int4* meta = static_cast<int4*>(a.ws);
  float* pieces = reinterpret_cast<float*>(meta + grid);
  cudaError_t e = cudaFuncSetAttribute(cache_attn_kernel<T, D, MT, kShared>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmem);
  if (e != cudaSuccess) return e;
  cache_attn_kernel<T, D, MT, kShared><<<grid, kThreads, L::kSmem, stream>>>(a, pl, pieces, meta);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid, L::R / kWarps);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;  // its launch overlaps the first kernel
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, cache_attn_join_kernel<T, D, L::R>, a, pl, (const float*)pieces, (const int4*)meta);
}

template <typename T, int D>
cudaError_t choose(const CacheAttnArgs& a, int sm_count, cudaStream_t stream) {
  const bool shared = (a.cmp.k ? a.cmp.v : a.raw.v) == nullptr;
  if (row_tiles(a.T_cap, a.B, a.H / a.H_kv, a.idx != nullptr, sizeof(T) == 4) == 2) {
    if constexpr (sizeof(T) == 2)
      return shared ? run<T, D, 2, true>(a, sm_count, stream) : run<T, D, 2, false>(a, sm_count, stream);
  }
  return shared ? run<T, D, 1, true>(a, sm_count, stream) : run<T, D, 1, false>(a, sm_count, stream);
}

}  // namespace

size_t cache_attn_workspace(int sm_count, int T_cap, int H, int H_kv, int d) {
  if (T_cap <= 0) return 0;
  return ws_bytes(sm_count, 2, d) > ws_bytes(sm_count, 1, d) ? ws_bytes(sm_count, 2, d) : ws_bytes(sm_count, 1, d);
}

cudaError_t launch_cache_attn(const CacheAttnArgs& a, bool fp32, int sm_count, cudaStream_t stream) {
  if (a.T_cap <= 0) return cudaSuccess;
  if (a.d == 64)
    return fp32 ? choose<float, 64>(a, sm_count, stream) : choose<__nv_bfloat16, 64>(a, sm_count, stream);
  return fp32 ? choose<float, 128>(a, sm_count, stream) : choose<__nv_bfloat16, 128>(a, sm_count, stream);
}

}  // namespace csa
