// cache_attn.cu -- attention of new query rows over the 8-bit serving cache
// (csa_cache_attn_fwd): cached compressed entries (every visible one, or those
// listed) and a window of cached raw rows in one softmax.
//
// Items of R = 16 or 32 (query, head) rows.
//
// A tile.  Each of the four warps takes 32 of its keys at a time through a ring of its own
// (cp.async, no CTA-wide barrier): codes are widened to halves in registers
// (exact), S = Q K^T and O += P V run on m16n8k16 products with float32 sums.
// A decode step moves 2 d bytes per key and head against 4 d G FLOP, so with up
// to 16 rows a tile it is bound by HBM, and codes go from shared memory straight
// into product fragments: a thread's 16 consecutive codes of a K row serve four
// k-steps (the order of the dims within a product is free), and four V rows are
// interleaved bytewise before widening.  32 sequences of 2K to 32K rows, 64 heads on 8
// KV heads: 204 us, 84% of the rate of a plain copy; one sequence of 128K rows, split
// over the whole GPU, 71 us (56%: the start, and pieces joined by a second kernel).
//
// Numbers.  A query row is scaled by a power of two so that its largest element
// is in [2^14, 2^15): bf16 queries are then exact as halves down to 2^-38 of it.
// float32 queries and weights go in as two halves (22 bits).
#include <math.h>

#include "cache_attn.cuh"

namespace csa {

namespace {

using namespace cache_attn;

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kStep = 32;              // keys of a warp's step
constexpr int kAhead = 4;              // steps whose rows are looked up together
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint4& a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float lds_f(uint32_t a) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a));
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
// Byte offset of 16-byte chunk `ch` of row `row` in a 16-row tile of codes.  The
// chunks of a 128-byte line are permuted so that the eight lanes of a 16-byte
// read phase hit all banks: K reads take four chunks of two neighbouring rows,
// V reads a chunk pair of every other row.
template <int D> __device__ __forceinline__ int code_offset(int row, int ch) {
  if (D == 128) return row * 128 + ((ch ^ (((row >> 1) & 1) << 1 | (((row >> 2) ^ row) & 1) << 2)) << 4);
  const int line = row >> 1;
  return line * 128 + ((((row & 1) * 4 + ch) ^ ((line & 3) << 1)) << 4);
}

// Notes the dims in which rows r see a NaN among the 16 V rows at `at` (half hf of a
// step whose first key is `first`): rare, so small rather than fast.
template <int D, int R>
__device__ __noinline__ void note_nans(uint32_t at, int hf, int first, bool entries, int window, const int* s_p,
                                       const int* s_vis, uint32_t* s_nan, int lane) {
  for (int i = lane; i < 16 * D; i += 32) {
    const int key = 16 * hf + i / D, d = i % D;
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(at + code_offset<D>(key, d / 16) + d % 16));
    if ((v & 0x7f) != 0x7f) continue;
    const int pos = first + key;
    for (int r = 0; r < R; ++r)
      if (entries ? pos < s_vis[r] : pos <= s_p[r] && pos > s_p[r] - window)
        atomicOr(s_nan + (r * D + d) / 32, 1u << (d % 32));
  }
  __syncwarp();
}

template <int D, int MT, bool kSplit, bool kShared> struct Layout {
  static constexpr int R = 16 * MT;
  static constexpr int kCodes = kStep * D;                                   // bytes of a step's rows
  static constexpr int kStage = kCodes * (kShared ? 1 : 2) + 2 * kStep * 4;  // K, V, their scales
  // copies of kStages - 1 steps are in flight: 96 KB an SM at 128 dims with separate V and three CTAs
  static constexpr int kStages = D == 128 && !kShared ? 2 : 4;
  static constexpr int kRing = kStages * kStage * kWarps;
  static constexpr int kMerge = kWarps * R * D * 4;
  static constexpr int kSums = 3 * kWarps * R * 4;                           // each warp's m, M, l behind them
  static constexpr int kBuf = kRing > kMerge + kSums ? kRing : kMerge + kSums;
  static constexpr int kQ = MT * (D / 16) * 32 * 16 * (kSplit ? 2 : 1);      // query fragments
  static constexpr int kRows = kBuf + kQ;                                    // rows of the next steps
  static constexpr int kSmem = kRows + kWarps * kAhead * kStep * 4;      // three CTAs an SM fit with MT = 1
};

template <typename T, int D, int MT, bool kShared>
__global__ void __launch_bounds__(kThreads, MT == 1 ? 3 : 2)
cache_attn_kernel(const CacheAttnArgs a, const Plan pl, float* __restrict__ ws_o, int4* __restrict__ ws_meta,
                  float* ws_far) {
  constexpr bool kSplit = sizeof(T) == 4;
  using L = Layout<D, MT, kSplit, kShared>;
  constexpr int R = L::R, kStages = L::kStages;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Context s_ctx;
  __shared__ float s_qf[R];                       // a row's query is q * 2^-e; 2^e
  __shared__ int s_p[R], s_vis[R];                // a row's position (-1: no such row), the entries that it sees
  __shared__ uint32_t s_nan[R * D / 32];          // dims of a row that a NaN reached (see note_nans)
  __shared__ int s_nans;
  __shared__ int s_out[R];                        // and its place: packed row * H + head

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, c = lane & 3;
  const int G = a.H / a.H_kv;
  const uint32_t buf = smem_u32(smem), qbuf = buf + L::kBuf;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // for what ran before on the stream
  asm volatile("griddepcontrol.launch_dependents;");

  if (tid == 0) ws_meta[blockIdx.x] = make_int4(-1, 0, 0, 0);
  split_tiles<kThreads, true>(a, pl, R, &s_ctx, smem, L::kBuf);
  capacity_rows<T, D>(a, tid, kThreads);

  const uint32_t ring = buf + warp * (kStages * L::kStage);
  uint32_t* rows = reinterpret_cast<uint32_t*>(smem + L::kRows) + warp * (kAhead * kStep);
  // lane constants of the fragment reads
  int off_k[D / 64], off_v[2];
#pragma unroll
  for (int h = 0; h < D / 64; ++h) off_k[h] = code_offset<D>(g, c + 4 * h);
#pragma unroll
  for (int e = 0; e < 2; ++e)
    off_v[e] = D == 128 ? code_offset<D>(2 * c + e, g) : code_offset<D>(2 * c + e, g >> 1) + (g & 1) * 8;
  float* far_m = ws_far + ((int64_t)blockIdx.x * kWarps + warp) * (2 * R);  // log2 maximum and sum of far steps
  float* far_l = far_m + R;
  const float scale_log2 = fabsf(a.scale) * kLog2e;  // its sign is put into the queries

  Items items{s_ctx.sh.u0, s_ctx.sh.slot_at, s_ctx.sh.slot};
  Item found;
  while (call_next_item(&s_ctx, &items, &found)) {
    const Item it = found;
    const Slot& x = it.x;
    const int t0 = it.t0, t1 = it.t1;
    if (x.bad && tid == 0) raise_status(a.status, CSA_ERR_DEVICE_BOUNDS);

    // Cache rows (block * H_kv + head) * block + row of the keys of steps [t, t + kAhead)
    // of this warp, a lane a key: the list and table reads of all steps are in flight together.
    auto look_up = [&](int t) {
      int pos[kAhead], blk[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) pos[i] = key_position(a, it, t + i, warp * kStep + lane);
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        pos[i] = checked_position(a, it, t + i, pos[i]);
        blk[i] = table_entry(a, it, t + i, pos[i]);
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) rows[i * kStep + lane] = cache_row(a, it, t + i, pos[i], blk[i]);
    };
    auto copy = [&](int n) {  // codes and scales of step t0 + n into its stage
      const int t = t0 + n;
      if (t < t1) {
        const uint32_t* from = rows + (n % kAhead) * kStep;
        const CacheView& cc = t < x.ct ? a.cmp : a.raw;
        const uint32_t st = ring + (n % kStages) * L::kStage;
        constexpr int kPerRow = D / 16, kRowsPer = 32 / kPerRow;
        const int r0 = lane / kPerRow, ch = lane % kPerRow;
        const uint8_t* k = cc.k + ch * 16;
        const uint8_t* v = kShared ? nullptr : cc.v + ch * 16;
#pragma unroll
        for (int i = 0; i < kStep / kRowsPer; ++i) {
          const uint32_t row = from[r0 + i * kRowsPer];
          const uint64_t off = row == kNoRow ? 0 : (uint64_t)row * D;
          const uint32_t dst = st + code_offset<D>(r0 + i * kRowsPer, ch);
          cp_async_16_zfill(dst, k + off, row != kNoRow);
          if (!kShared) cp_async_16_zfill(dst + L::kCodes, v + off, row != kNoRow);
        }
        const uint32_t row = from[lane], bh = row == kNoRow ? 0 : row >> cc.log_block;
        const uint32_t dst = st + L::kStage - 2 * kStep * 4 + lane * 4;
        cp_async_4_zfill(dst, cc.k_scale + bh, row != kNoRow);
        if (!kShared) cp_async_4_zfill(dst + kStep * 4, cc.v_scale + bh, row != kNoRow);
      }
      cp_async_commit();
    };
    // the queries as product fragments, one warp a 16-row tile
    auto take_queries = [&]() {
      if (warp == kWarps - 1) {
        for (int i = lane; i < R * D / 32; i += 32) s_nan[i] = 0;
        if (lane == 0) s_nans = 0;
      }
      if (warp < MT) {
        float v[2][D / 4];  // this thread's 16-element chunks c (and c + 4) of rows g, g + 8
        float inv[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = warp * 16 + g + 8 * e;
          const int qi = G > R ? 0 : r / G, h = G > R ? r : r % G;
          const bool real = qi < x.nq && h < it.heads;
          if (c == 0) {
            s_p[r] = real ? x.p0 + qi : -1;
            s_vis[r] = real && a.cmp.k ? (x.p0 + qi + 1) / a.r : 0;
            s_out[r] = real ? (x.row0 + qi) * a.H + it.h0 + h : -1;
          }
          const T* src = static_cast<const T*>(a.q) + ((int64_t)(x.row0 + qi) * a.H + it.h0 + h) * D;
          float amax = 0.f;
#pragma unroll
          for (int i = 0; i < D / 4; i += 4) {
            float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
            if (real) {
              const T* p = src + 16 * (c + 4 * (i / 16)) + i % 16;
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
            if (fabsf(v[e][i]) < INFINITY) amax = fmaxf(amax, fabsf(v[e][i]));
          amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
          amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
          // largest element to [2^14, 2^15), as far as 2^e and 2^-e are normal numbers
          const int ex = max((int)(__float_as_uint(amax) >> 23) - 127 - 14, -113);
          inv[e] = a.scale < 0.f ? -pow2i(-ex) : pow2i(-ex);
          if (c == 0) s_qf[r] = pow2i(ex);
        }
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int w = 0; w < 4; ++w) {  // row g, first pair; row g + 8; their second pairs
            const int e = w & 1, i = ks * 4 + (w >> 1) * 2;
            const float f0 = v[e][i] * inv[e], f1 = v[e][i + 1] * inv[e];
            hi[w] = pack_f16x2(f0, f1);
            lo[w] = rest_f16x2(hi[w], f0, f1);
          }
          const uint32_t at = qbuf + ((warp * (D / 16) + ks) * 32 + lane) * 16;
          asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(hi[0]), "r"(hi[1]), "r"(hi[2]), "r"(hi[3]));
          if (kSplit)
            asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at + L::kQ / 2), "r"(lo[0]), "r"(lo[1]),
                         "r"(lo[2]), "r"(lo[3]));
        }
      }
    };
    float qf[MT][2], M[MT][2], l[MT][2], o[MT][D / 8][4];
    float e0 = 0.f;         // l is of 2^(t + e0 - M + kBase), e0 the first key's V exponent
    bool any_key = false, any_far = false;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        M[mt][e] = kNone;
        l[mt][e] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < D / 8; ++i) o[mt][i][0] = o[mt][i][1] = o[mt][i][2] = o[mt][i][3] = 0.f;
    }

    // kStages - 1 rounds that only copy, then a round a step
    for (int n = 1 - kStages; n < t1 - t0; ++n) {
      const int next = n + kStages - 1;
      cp_async_wait<kStages - 2>();
      __syncwarp();
      if (next % kAhead == 0 && t0 + next < t1) {
        look_up(t0 + next);
        __syncwarp();
      }
      copy(next);
      if (n < 0) {
        if (n == -1) {
          take_queries();
          __syncthreads();
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int e = 0; e < 2; ++e) qf[mt][e] = s_qf[mt * 16 + g + 8 * e];
        }
        continue;
      }
      const int t = t0 + n;
      const uint32_t st = ring + (n % kStages) * L::kStage;
      const uint32_t sc = st + L::kStage - 2 * kStep * 4;
      // each key's score factor and V exponent, in place of its scales
      bool uniform, far;    // one V scale in each half of the step (a block's); a V scale far from e0
      float ie[2];
      {
        const float ks = lds_f(sc + 4 * lane), vs = kShared ? ks : lds_f(sc + kStep * 4 + 4 * lane);
        const uint32_t there = __ballot_sync(0xffffffffu, ks > 0.f);
        if (there == 0) continue;
        const float ev = exponent_of(vs);
        if (!any_key) e0 = __shfl_sync(0xffffffffu, ev, __ffs(there) - 1);
        any_key = true;
        far = __any_sync(0xffffffffu, ks > 0.f && fabsf(ev - e0) > 60.f);
        const float ev0 = __shfl_sync(0xffffffffu, ev, 0), ev1 = __shfl_sync(0xffffffffu, ev, 16);
        ie[0] = ex2(e0 - ev0);
        ie[1] = ex2(e0 - ev1);
        uniform = __all_sync(0xffffffffu, ks > 0.f && ev == (lane < 16 ? ev0 : ev1));
        asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(sc + 8 * lane), "f"(ks * scale_log2),
                     "f"(ks > 0.f ? ev : -INFINITY)
                     : "memory");
        __syncwarp();
      }

      // ---- S = Q K^T ----
      float s[MT][4][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[mt][j][0] = s[mt][j][1] = s[mt][j][2] = s[mt][j][3] = 0.f;
#pragma unroll
      for (int h = 0; h < D / 64; ++h) {
        uint32_t kw[4][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint4 k = lds128(st + off_k[h] + j * 8 * D);
          kw[j][0] = k.x, kw[j][1] = k.y, kw[j][2] = k.z, kw[j][3] = k.w;
        }
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          uint4 q[MT], ql[MT];
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            const uint32_t at = qbuf + ((mt * (D / 16) + h * 4 + w) * 32 + lane) * 16;
            q[mt] = lds128(at);
            if (kSplit) ql[mt] = lds128(at + L::kQ / 2);
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t b0 = widen_lo(kw[j][w]), b1 = widen_hi(kw[j][w]);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              mma_f16(s[mt][j], q[mt], b0, b1);
              if (kSplit) mma_f16(s[mt][j], ql[mt], b0, b1);
            }
          }
        }
      }

      // a step that some of the item's queries see and others do not
      const bool entries = t < x.ct;
      const int first = t * kTile + warp * kStep + (entries ? 0 : x.w0 - x.ct * kTile);
      bool mixed = false;
      if (x.nq > 1)
        mixed = entries ? first + kStep > it.vis : first + kStep - 1 > x.p0 || first <= x.p0 + x.nq - 1 - a.window;

      // ---- softmax: s becomes u = t + e, then the weights 2^(u - M + kBase) ----
      float ev[8];  // keys 8 j + 2 c, + 1
      {
        float ks[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint4 k = lds128(sc + 64 * j + 16 * c);
          ks[2 * j] = __uint_as_float(k.x), ev[2 * j] = __uint_as_float(k.y);
          ks[2 * j + 1] = __uint_as_float(k.z), ev[2 * j + 1] = __uint_as_float(k.w);
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              s[mt][j][i] = fmaf(s[mt][j][i] * ks[2 * j + (i & 1)], qf[mt][i >> 1], ev[2 * j + (i & 1)]);
      }
      if (mixed) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int r = mt * 16 + g + 8 * e, p = s_p[r];
            const int from = (entries ? 0 : p - a.window + 1) - first, to = (entries ? s_vis[r] : p + 1) - first;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int at = (i >> 1) * 8 + 2 * c + (i & 1);
              if (at < from || at >= to) s[mt][i >> 1][2 * e + (i & 1)] = -INFINITY;
            }
          }
      }
      {
        float top[MT][2];
        bool grow = false;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float v = fmaxf(s[mt][0][2 * e], s[mt][0][2 * e + 1]);
#pragma unroll
            for (int j = 1; j < 4; ++j) v = fmaxf(v, fmaxf(s[mt][j][2 * e], s[mt][j][2 * e + 1]));
            top[mt][e] = v;
            grow |= v > M[mt][e] + kSlack;
          }
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            float f[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float v = fmaxf(top[mt][e], __shfl_xor_sync(0xffffffffu, top[mt][e], 1));
              v = fmaxf(M[mt][e], fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2)));
              f[e] = ex2(M[mt][e] - v);
              l[mt][e] *= f[e];
              M[mt][e] = v;
            }
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
              o[mt][i][0] *= f[0];
              o[mt][i][1] *= f[0];
              o[mt][i][2] *= f[1];
              o[mt][i][3] *= f[1];
            }
          }
        }
      }
      if (far) {  // block scales 2^60 apart: this step's part of the sums in sums of their own
        if (!any_far) {
          for (int i = lane; i < R; i += 32) far_m[i] = kNone, far_l[i] = 0.f;
          __syncwarp();
        }
        any_far = true;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int r = mt * 16 + g + 8 * e;
            float top = kNone, sum = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (ev[i] > -INFINITY) top = fmaxf(top, s[mt][i >> 1][2 * e + (i & 1)] - ev[i]);
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(far_m[r], fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2)));
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (ev[i] > -INFINITY) sum += ex2(s[mt][i >> 1][2 * e + (i & 1)] - ev[i] - top);
            sum += __shfl_xor_sync(0xffffffffu, sum, 1);
            sum += __shfl_xor_sync(0xffffffffu, sum, 2);
            if (c == 0) {
              far_l[r] = far_l[r] * ex2(far_m[r] - top) + sum;
              far_m[r] = top;
            }
          }
        __syncwarp();
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float shift = kBase - M[mt][e];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float& w = s[mt][i >> 1][2 * e + (i & 1)];
            w = ex2(w + shift);
          }
        }
      if (far) {
      } else if (uniform) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf)
              l[mt][e] = fmaf((s[mt][2 * hf][2 * e] + s[mt][2 * hf][2 * e + 1]) +
                                  (s[mt][2 * hf + 1][2 * e] + s[mt][2 * hf + 1][2 * e + 1]),
                              ie[hf], l[mt][e]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float f = ev[i] > -INFINITY ? ex2(e0 - ev[i]) : 0.f;
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int e = 0; e < 2; ++e) l[mt][e] = fmaf(s[mt][i >> 1][2 * e + (i & 1)], f, l[mt][e]);
        }
      }
      uint4 pa[MT][2], pb[MT][2];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const float(&w0)[4] = s[mt][2 * hf];
          const float(&w1)[4] = s[mt][2 * hf + 1];
          uint4& p = pa[mt][hf];
          p = make_uint4(pack_f16x2(w0[0], w0[1]), pack_f16x2(w0[2], w0[3]), pack_f16x2(w1[0], w1[1]),
                         pack_f16x2(w1[2], w1[3]));
          if (kSplit)
            pb[mt][hf] = make_uint4(rest_f16x2(p.x, w0[0], w0[1]), rest_f16x2(p.y, w0[2], w0[3]),
                                    rest_f16x2(p.z, w1[0], w1[1]), rest_f16x2(p.w, w1[2], w1[3]));
        }

      // ---- O += P V, 16 keys at a time: 2c, 2c + 1, 8 + 2c, 9 + 2c of them a thread;
      //      column n of product i is dim n D / 8 + i ----
      constexpr int kWords = D / 32;
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        uint32_t v[4][kWords];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t at = st + (kShared ? 0 : L::kCodes) + off_v[k & 1] + (2 * hf + (k >> 1)) * 8 * D;
          if (D == 128) {
            const uint4 q = lds128(at);
            v[k][0] = q.x, v[k][1] = q.y, v[k][kWords - 2] = q.z, v[k][kWords - 1] = q.w;
          } else {
            const uint2 q = lds64(at);
            v[k][0] = q.x, v[k][1] = q.y;
          }
        }
        if (mixed) {  // a NaN that only some queries see must not reach the others as 0 * NaN: noted, and taken as 0
          bool nan = false;
#pragma unroll
          for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int w = 0; w < kWords; ++w) nan |= has_nan4(v[k][w]);
          if (__any_sync(0xffffffffu, nan)) {
            note_nans<D, R>(st + (kShared ? 0 : L::kCodes), hf, first, entries, a.window, s_p, s_vis, s_nan, lane);
            if (lane == 0) s_nans = 1;
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
              for (int w = 0; w < kWords; ++w) v[k][w] = without_nan4(v[k][w]);
          }
        }
#pragma unroll
        for (int w = 0; w < kWords; ++w) {
          const uint32_t y[2][2] = {{__byte_perm(v[0][w], v[1][w], 0x5140), __byte_perm(v[0][w], v[1][w], 0x7362)},
                                    {__byte_perm(v[2][w], v[3][w], 0x5140), __byte_perm(v[2][w], v[3][w], 0x7362)}};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t b0 = (i & 1) ? widen_hi(y[0][i >> 1]) : widen_lo(y[0][i >> 1]);
            const uint32_t b1 = (i & 1) ? widen_hi(y[1][i >> 1]) : widen_lo(y[1][i >> 1]);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              mma_f16(o[mt][4 * w + i], pa[mt][hf], b0, b1);
              if (kSplit) mma_f16(o[mt][4 * w + i], pb[mt][hf], b0, b1);
            }
          }
        }
      }
    }
    cp_async_wait<0>();

    // ---- join the four warps ----
    __syncthreads();  // the rings are free
    float* acc = reinterpret_cast<float*>(smem);
    float(*s_m)[R] = reinterpret_cast<float(*)[R]>(smem + L::kMerge);
    float(*s_M)[R] = s_m + kWarps;
    float(*s_l)[R] = s_M + kWarps;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float sum = l[mt][e];
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        const int r = mt * 16 + g + 8 * e;
        float m = M[mt][e] == kNone ? kNone : M[mt][e] - kBase - e0;  // the sum is sum * 2^m
        if (any_far) {
          const float top = fmaxf(m, far_m[r]);
          sum = sum * ex2(m - top) + far_l[r] * ex2(far_m[r] - top);
          m = top;
        }
        if (c == 0) {
          s_m[warp][r] = m;
          s_M[warp][r] = M[mt][e];
          s_l[warp][r] = sum;
        }
      }
    __syncthreads();
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = mt * 16 + g + 8 * e;
        float top = s_M[0][r];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) top = fmaxf(top, s_M[w][r]);
        const float f = ex2(M[mt][e] - top);
        // columns 2c and 2c + 1 of products 0 .. D / 8 - 1: dims [2c D/8, (2c + 2) D/8)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < D / 8; i += 4) {
            float4 v = make_float4(o[mt][i][2 * e + h], o[mt][i + 1][2 * e + h], o[mt][i + 2][2 * e + h],
                                   o[mt][i + 3][2 * e + h]);
            v.x *= f, v.y *= f, v.z *= f, v.w *= f;
            *reinterpret_cast<float4*>(acc + (warp * R + r) * D + (2 * c + h) * (D / 8) + i) = v;
          }
      }
    __syncthreads();
    const bool whole = t0 == 0 && t1 == it.n_tiles;
    float* piece = ws_o + ((int64_t)blockIdx.x * 2 + (t0 == 0 ? 1 : 0)) * piece_floats<D>(R);
    for (int i = tid; i < R * (D / 4); i += kThreads) {
      const int r = i / (D / 4), d4 = i % (D / 4);
      const int at = s_out[r];
      if (at < 0) continue;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      float mm = kNone, MM = kNone, ll = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float4 f = *reinterpret_cast<const float4*>(acc + (w * R + r) * D + 4 * d4);
        v.x += f.x, v.y += f.y, v.z += f.z, v.w += f.w;
        mm = fmaxf(mm, s_m[w][r]);
        MM = fmaxf(MM, s_M[w][r]);
      }
#pragma unroll
      for (int w = 0; w < kWarps; ++w) ll += s_l[w][r] * ex2(s_m[w][r] - mm);
      if (s_nans) {
        const uint32_t bits = s_nan[(r * D + 4 * d4) / 32] >> (4 * d4 % 32);
        if (bits & 1) v.x = NAN;
        if (bits & 2) v.y = NAN;
        if (bits & 4) v.z = NAN;
        if (bits & 8) v.w = NAN;
      }
      if (!whole) {
        *reinterpret_cast<float4*>(piece + r * D + 4 * d4) = v;
        if (d4 == 0) {
          piece[R * D + r] = mm;
          piece[R * D + R + r] = MM;
          piece[R * D + 2 * R + r] = ll;
        }
        continue;
      }
      store_out<T>(a, at, D, d4, v, finish_factors(a, at, mm, MM, ll));
    }
    if (!whole && t0 == 0 && tid == 0)  // its pieces: this one, then the first ones of the CTAs up to its last tile's
      note_split(&s_ctx, x.row0, x.nq, it.sub, it.item0, it.n_tiles, ws_meta + blockIdx.x);
    __syncthreads();  // s_out, s_m and the buffers are taken again
  }
}

// Rows that an item can fill: the heads of a group, and without a list the queries of
// a sequence on average.  The forms below are for 16, 32, 64 and 128 of them; a larger
// one widens a key once for more rows, and its empty rows cost what full ones do.
// Measured, us, with separate V (16 sequences of 2K to 8K rows, 32 heads, 128 dims; 16 and
// 32 rows on mma.sync, 64 and 128 on tcgen05), by the rows that there are:
//    16: 53 (as 32: 69, as 64: 88)     32: 71 (as 16: 82, as 64: 89)
//    64: 53 (as 32: 70, as 128: 76)   128: 80 (as 64: 86)   256: 127 (as 64: 154, as 32: 217)
// where V is K (24 sequences of 4K to 25K entries): 16: 38 (as 64: 43), 32: as 64 42 (as 32: 47);
// 512 listed entries of 48 sequences: 16: 21.3 (as 64: 22.3), 32: as 64 22.5 (as 32: 23.7);
// 64 dims: 16: 38 (as 32: 49), 32: 49 (as 16: 60).
int64_t rows_of_item(int T_cap, int B, int G, bool listed) {
  return listed || B <= 0 ? G : ((int64_t)T_cap + B - 1) / B * G;
}
int row_tiles(int64_t rows) { return rows > 16 ? 2 : 1; }  // bf16; float32 has one, in two halves
constexpr int ctas_per_sm(int mt) { return mt == 1 ? 3 : 2; }

template <typename T, int D, int MT, bool kShared>
cudaError_t run(const CacheAttnArgs& a, int sm_count, cudaStream_t stream) {
  using L = Layout<D, MT, sizeof(T) == 4, kShared>;
  // an item costs as much as 5 tiles beside its own (32 sequences with 8 KV heads: 220 us with 0, 208 with 3, 204 so,
  // 206 with 8; 24 dense sequences with 16 heads 46, 41, 38, 38)
  const Plan pl = make_plan(a, L::R, 5);
  const int grid = sm_count * ctas_per_sm(MT);
  const Scratch sc = scratch_of<D>(a.ws, grid, L::R);
  cudaError_t e = cudaFuncSetAttribute(cache_attn_kernel<T, D, MT, kShared>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmem);
  if (e != cudaSuccess) return e;
  if ((e = launch_after(cache_attn_kernel<T, D, MT, kShared>, dim3(grid), dim3(kThreads), L::kSmem, stream, a, pl,
                        sc.pieces, sc.meta, sc.far)) != cudaSuccess)
    return e;
  return launch_after(cache_attn_join_kernel<T, D, L::R>, dim3(grid, L::R / kJoinWarps), dim3(32 * kJoinWarps), 0, stream, a, pl,
                      (const float*)sc.pieces, (const int4*)sc.meta);
}

// Rows of an item on tcgen05 (cache_attn_tc.cu), or 0.
int tc_rows(int64_t rows, bool shared, int d, bool fp32) {
  return fp32 || d != 128 || rows <= (shared ? 16 : 32) ? 0 : rows <= 64 ? 64 : 128;
}

template <typename T, int D>
cudaError_t choose(const CacheAttnArgs& a, int64_t rows, int sm_count, cudaStream_t stream) {
  const bool shared = (a.cmp.k ? a.cmp.v : a.raw.v) == nullptr;
  if constexpr (sizeof(T) == 2) {
    if (row_tiles(rows) == 2) {
      if (!shared) return run<T, D, 2, false>(a, sm_count, stream);
      if constexpr (D == 64) return run<T, D, 2, true>(a, sm_count, stream);  // 128 dims: on tcgen05
    }
  }
  return shared ? run<T, D, 1, true>(a, sm_count, stream) : run<T, D, 1, false>(a, sm_count, stream);
}

}  // namespace

size_t cache_attn_workspace(int sm_count, int T_cap, int H, int H_kv, int d) {
  if (T_cap <= 0) return 0;
  size_t n = cache_attn_tc_workspace(sm_count);
  for (int mt = 1; mt <= 2; ++mt) {
    const size_t k = scratch_bytes(sm_count * ctas_per_sm(mt), 16 * mt, d, kWarps);
    if (k > n) n = k;
  }
  return n;
}

cudaError_t launch_cache_attn(const CacheAttnArgs& a, bool fp32, int sm_count, cudaStream_t stream) {
  if (a.T_cap <= 0) return cudaSuccess;
  const int64_t rows = rows_of_item(a.T_cap, a.B, a.H / a.H_kv, a.idx != nullptr);
  if (const int tc = tc_rows(rows, (a.cmp.k ? a.cmp.v : a.raw.v) == nullptr, a.d, fp32)) return launch_cache_attn_tc(a, tc, sm_count, stream);
  if (a.d == 64)
    return fp32 ? choose<float, 64>(a, rows, sm_count, stream) : choose<__nv_bfloat16, 64>(a, rows, sm_count, stream);
  return fp32 ? choose<float, 128>(a, rows, sm_count, stream) : choose<__nv_bfloat16, 128>(a, rows, sm_count, stream);
}

}  // namespace csa
