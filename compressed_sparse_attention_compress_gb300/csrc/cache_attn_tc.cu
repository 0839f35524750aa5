// cache_attn_tc.cu -- attention over the 8-bit serving cache on tcgen05 tensor
// cores: 128 dims, bf16 queries, many (query, head) rows per KV head (64 shared
// heads of a decode step, or the queries of a chunk).
//
// With 64 rows a key takes 64 x 4 x 128 FLOP against its 128 to 256 bytes: what bounds
// this form is neither HBM nor the tensor pipe (18% busy in prompt chunks, 420 TFLOP/s
// there, 300 in dense decode) but the softmax's chain of dependent steps per tile (loads
// from tensor memory, a vote, exponentials, P^T, a barrier) and, in small calls, the first
// pass through the code.  Tiles are transposed as in the training kernels, the 128 keys on
// the lanes of tensor memory:
//   S^T[key, r]  = K[key, :] . Q[r, :]        (M = 128, N = 64 or 128, K = 128 dims)
//   O^T[dim, r] += V^T[dim, key] P^T[key, r]  (M = 128, N, K = 128 keys)
// so a thread owns a key: its block scales and its place in the mask are scalars.
// Roles, one CTA per SM:
//   8 converter warps: look rows up (list, table), load a tile's codes into registers
//     while the one before is in use, widen them to halves (exact) into swizzled
//     operand tiles, K a tile ahead of V, and leave each key's score factor and V
//     exponent beside them; they meet only at mbarriers;
//   1 warp issues S^T, 1 warp O^T: one issuer in one order had each product wait for
//     what the other one waits for (prompt chunks 494 us, with two issuers 452 us);
//   1 warp finds the CTA's items ahead of their use;
//   8 softmax warps: (key, half of the rows); weights as halves into P^T, the sums per
//     row in registers, with 128 rows in tensor memory (reduced over keys once per item).
// Twice as many softmax warps with a quarter of the rows each were slower (dense decode
// 66 against 57 us, prompt chunks 612 against 455 us), and so were two softmax groups that
// take the tiles in turn: the kernel then waits for code more than for products.
// The query rows of an item are scaled by one power of two, the largest element to
// [2^14, 2^15): exact as halves down to 2^-32 of it.
#include "cache_attn.cuh"
#include "tcgen05.cuh"

namespace csa {

namespace {

using namespace cache_attn;
using namespace ws;

constexpr int kDim = 128;
constexpr int kSoftWarps = 8, kConvWarps = 8;
constexpr int kSoftThreads = 32 * kSoftWarps, kConvThreads = 32 * kConvWarps;
constexpr int kMmaWarp = kSoftWarps + kConvWarps;
constexpr int kThreads = 32 * (kMmaWarp + 4);  // whole warpgroups; one of the last one's warps has no part
constexpr int kConvKeys = kTile / kConvWarps;  // keys of a converter warp
// Registers a thread: 640 threads are launched with 96 each (61,440); 256 x 120 + 256 x 88 + 128 x 56 = 60,416.
constexpr int kSoftRegs = 120, kConvRegs = 88, kMmaRegs = 56;
constexpr int kSoftBar = 1, kHalfBar = 2;  // named barriers; the last and the next one: half of the rows each
constexpr int kRing = 4;                    // tiles (items) whose key factors (NaN notes) can be in use at once
constexpr int kAhead = 4;                   // tiles whose rows are looked up together
constexpr float kUnset = 1e9f;              // a row's shift before its first key: any score then asks for a maximum
constexpr uint32_t kRegion = kTile * 128;   // 128 keys x 64 halves
constexpr uint32_t kTileBytes = 2 * kRegion;

template <int N, bool kShared> struct Tc {
  // K (or K = V) tiles, as many as fit: dense decode 51.3 us with three, 50.0 with four (two tiles' codes
  // on their way in registers instead of one: slower again, 50.9)
  static constexpr int kStK = kShared ? (N == 64 ? 4 : 3) : 2;
  static constexpr int kStV = kShared ? 0 : 2;
  static constexpr int kQBufs = N == 128 && !kShared ? 1 : 2;
  static constexpr uint32_t kQRegion = N * 128;                 // N rows x 64 halves
  static constexpr uint32_t kQBytes = 2 * kQRegion;
  static constexpr uint32_t kVOff = kStK * kTileBytes;
  static constexpr uint32_t kQOff = kVOff + kStV * kTileBytes;
  static constexpr uint32_t kPOff = kQOff + kQBufs * kQBytes;
  static constexpr uint32_t kSmem = kPOff + (N / 64) * kRegion;
  static constexpr uint32_t kCols = N == 64 ? 256 : 512;        // S^T twice, O^T; with N = 128 the sums
  static constexpr int kPasses = N / 64;                        // of 32 rows a thread
};

// kind::f16 instruction descriptor with half operands.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, int a_mn, int b_mn) {
  return (1u << 4) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ void sts128(uint32_t at, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
__device__ __forceinline__ float tmem_ld1_sync(uint32_t at) {
  uint32_t r;
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];\ntcgen05.wait::ld.sync.aligned;\n" : "=r"(r) : "r"(at) : "memory");
  return __uint_as_float(r);
}
__device__ __forceinline__ void tmem_ld32f_sync(uint32_t at, float (&v)[32]) {
  uint32_t r[32];
  tc::tmem_ld32_sync(at, r);
#pragma unroll
  for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]);
}
__device__ __forceinline__ void tmem_st32f(uint32_t at, const float (&v)[32]) {
#pragma unroll
  for (int c = 0; c < 32; c += 16) {
    uint32_t r[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) r[j] = __float_as_uint(v[c + j]);
    tc::tmem_st16(at + c, r);
  }
  tc::tmem_wait_st();
}
__device__ __forceinline__ bool has_nan16(uint4 v) {
  return has_nan4(v.x) || has_nan4(v.y) || has_nan4(v.z) || has_nan4(v.w);
}
__device__ __forceinline__ uint4 without_nan16(uint4 v) {
  return make_uint4(without_nan4(v.x), without_nan4(v.y), without_nan4(v.z), without_nan4(v.w));
}
__device__ __forceinline__ int ord_of(float f) {
  const int i = __float_as_int(f);
  return i >= 0 ? i : i ^ 0x7FFFFFFF;
}
__device__ __forceinline__ float float_of(int i) { return __int_as_float(i >= 0 ? i : i ^ 0x7FFFFFFF); }

// Sums of 32 values per thread over a warp: lane l gets that of value l.
__device__ __forceinline__ float warp_sum32(float (&v)[32], int lane) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const bool upper = (lane & o) != 0;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      if (j < o) {
        const float send = upper ? v[j] : v[j + o], keep = upper ? v[j + o] : v[j];
        v[j] = keep + __shfl_xor_sync(0xffffffffu, send, o);
      }
    }
  }
  return v[0];
}

// Whether some of the item's queries see a key of tile t that others do not.
__device__ __forceinline__ bool mixed_tile(const CacheAttnArgs& a, const Item& it, int t, int& first) {
  const Slot& x = it.x;
  const bool entries = t < x.ct;
  first = entries ? t * kTile : x.w0 + (t - x.ct) * kTile;
  if (x.nq <= 1) return false;
  return entries ? first + kTile > it.vis : first + kTile - 1 > x.p0 || first <= x.p0 + x.nq - 1 - a.window;
}

template <int N, bool kShared>
__global__ void __launch_bounds__(kThreads, 1)
cache_attn_tc_kernel(const CacheAttnArgs a, const Plan pl, float* __restrict__ ws_o, int4* __restrict__ ws_meta) {
  using C = Tc<N, kShared>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ Context s_ctx;
  __shared__ uint32_t s_tmem;
  __shared__ __align__(8) uint64_t s_kfull[C::kStK], s_kempty[C::kStK], s_vfull[2], s_vempty[2], s_qfull[2],
      s_qempty[2], s_sfull[2], s_sfree[2], s_par_full[kRing], s_ifull[kRing], s_iempty[kRing],
      s_pfull, s_odone, s_ofree, s_drain[2], s_qmaxed;
  __shared__ Item s_item[kRing];                           // t1 < 0: no more
  __shared__ __align__(8) float2 s_par[kRing][kTile];      // score factor, V exponent (-inf: no key)
  __shared__ uint32_t s_rows[kConvWarps][2 * kAhead][kConvKeys];  // cache rows of the next tiles
  __shared__ uint32_t s_nan[kRing][N * kDim / 32];         // dims of a row that a NaN reached, by item
  __shared__ int s_nans[kRing];
  __shared__ float s_qmax[2][kConvWarps];
  __shared__ __align__(16) float s_shift[N];               // kBase - M
  __shared__ float s_M[N], s_alpha[N], s_f[N], s_f2[N];
  __shared__ int s_wmax[4][64];
  __shared__ float s_m[4][N], s_l[4][N];
  __shared__ int2 s_sees[2][N];                            // entries, raw rows that a row sees: first, how many
  __shared__ int s_out[N];
  __shared__ float2 s_far[kSoftWarps][N / 2];              // reference and sum of a warp's far keys
  __shared__ int s_abort;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const int G = a.H / a.H_kv;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // for what ran before on the stream
  asm volatile("griddepcontrol.launch_dependents;");

  if (tid == 0) {
    for (int i = 0; i < C::kStK; ++i) {
      mbar_init(smem_u32(&s_kfull[i]), kConvWarps);
      mbar_init(smem_u32(&s_kempty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&s_vfull[i]), kConvWarps);
      mbar_init(smem_u32(&s_vempty[i]), 1);
      mbar_init(smem_u32(&s_qfull[i]), kConvWarps);
      mbar_init(smem_u32(&s_qempty[i]), 1);
      mbar_init(smem_u32(&s_sfull[i]), 1);
      mbar_init(smem_u32(&s_sfree[i]), kSoftWarps);
    }
    for (int i = 0; i < kRing; ++i) {
      mbar_init(smem_u32(&s_par_full[i]), kConvWarps);
      mbar_init(smem_u32(&s_ifull[i]), 1);
      mbar_init(smem_u32(&s_iempty[i]), kConvWarps + kSoftWarps + 2);
      s_nans[i] = 0;
    }
    mbar_init(smem_u32(&s_pfull), kSoftWarps);
    mbar_init(smem_u32(&s_odone), 1);
    mbar_init(smem_u32(&s_qmaxed), kConvWarps);
    mbar_init(smem_u32(&s_ofree), kSoftWarps);
    mbar_init(smem_u32(&s_drain[0]), 1);
    mbar_init(smem_u32(&s_drain[1]), 1);
    fence_mbar_init();
    s_abort = 0;
    ws_meta[blockIdx.x] = make_int4(-1, 0, 0, 0);
  }
  for (int i = tid; i < kRing * (N * kDim / 32); i += kThreads) (&s_nan[0][0])[i] = 0;
  if (warp == kMmaWarp) {
    tc::tmem_alloc(smem_u32(&s_tmem), C::kCols);
    tc::tmem_relinquish();
  }
  split_tiles<kThreads, false>(a, pl, N, &s_ctx, smem_raw, (int)C::kSmem);
  capacity_rows<__nv_bfloat16, kDim>(a, tid, kThreads);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = s_tmem;
  volatile int* abort_flag = &s_abort;
  int* status = a.status;

  // the n-th item of this CTA, once it is known: waited for by every thread that takes part
  auto item_ready = [&](uint32_t n) { return mbar_wait_bounded(smem_u32(&s_ifull[n % kRing]), n / kRing & 1u, status); };

  if (warp >= kSoftWarps && warp < kMmaWarp) {
    // =================== converters: warp w has keys 16 w .. 16 w + 15 of every tile ===================
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kConvRegs));
    const int w = warp - kSoftWarps, ct = tid - kSoftThreads;
    const int sub = (lane >> 2) & 3, ch = (lane & 3) | (lane >> 4) << 2;  // row of a group of four, 16-code chunk:
    uint32_t k = 0;                                  // eight lanes' stores then fall into different banks
    bool dead = false;
    for (uint32_t n_item = 0; !dead; ++n_item) {
      if ((dead = __any_sync(0xffffffffu, !item_ready(n_item) || *abort_flag != 0))) break;
      const Item& it = s_item[n_item % kRing];
      if (it.t1 < 0) break;
      if (it.x.bad && ct == 0) raise_status(status, CSA_ERR_DEVICE_BOUNDS);
      const int t0 = it.t0, t1 = it.t1;
      auto look_up = [&](int t) {
        constexpr int kLoads = kAhead * kConvKeys / 32;  // a lane: one key of every other tile
        const int key = lane % kConvKeys, off = lane / kConvKeys;
        int pos[kLoads], blk[kLoads];
#pragma unroll
        for (int i = 0; i < kLoads; ++i) pos[i] = key_position(a, it, t + 2 * i + off, kConvKeys * w + key);
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
          pos[i] = checked_position(a, it, t + 2 * i + off, pos[i]);
          blk[i] = table_entry(a, it, t + 2 * i + off, pos[i]);
        }
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
          const uint32_t row = cache_row(a, it, t + 2 * i + off, pos[i], blk[i]);
          s_rows[w][(t - t0 + 2 * i + off) % (2 * kAhead)][key] = row;
          if (row != kNoRow) {  // a row is a line: it comes to L2 while the tiles before it are in use
            const CacheView& cc = t + 2 * i + off < it.x.ct ? a.cmp : a.raw;
            asm volatile("prefetch.global.L2 [%0];" ::"l"(cc.k + (uint64_t)row * kDim));
            if (!kShared) asm volatile("prefetch.global.L2 [%0];" ::"l"(cc.v + (uint64_t)row * kDim));
          }
        }
        __syncwarp();
      };
      constexpr int kChunks = kConvKeys / 4;
      struct Unit {  // codes of a warp's rows, kChunks chunks a thread, and the scales of row lane % kConvKeys
        uint4 c[kChunks];
        float ks, vs;  // vs: where V has scales of its own
      };
      auto load = [&](Unit& un, int t, bool is_v) {
        if (t >= t1) return;
        const CacheView& cc = t < it.x.ct ? a.cmp : a.raw;
        const uint32_t* rows = s_rows[w][(t - t0) % (2 * kAhead)];
        const uint8_t* src = (is_v ? cc.v : cc.k) + ch * 16;
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
          const uint32_t row = rows[4 * i + sub];
          un.c[i] = row == kNoRow ? make_uint4(0, 0, 0, 0)
                                  : __ldg(reinterpret_cast<const uint4*>(src + (uint64_t)row * kDim));
        }
        if (!is_v) {
          const uint32_t row = rows[lane % kConvKeys];
          un.ks = row == kNoRow ? 0.f : __ldg(cc.k_scale + (row >> cc.log_block));
          if (!kShared) un.vs = row == kNoRow ? 0.f : __ldg(cc.v_scale + (row >> cc.log_block));
        }
      };
      auto store = [&](const Unit& un, uint32_t tile) {
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
          const uint4 v = un.c[i];
          const int row = kConvKeys * w + 4 * i + sub;
          const uint32_t at = tile + (ch >> 2) * kRegion;
          sts128(at + tc::sw128_offset(row, (ch & 3) * 2), widen_lo(v.x), widen_hi(v.x), widen_lo(v.y), widen_hi(v.y));
          sts128(at + tc::sw128_offset(row, (ch & 3) * 2 + 1), widen_lo(v.z), widen_hi(v.z), widen_lo(v.w), widen_hi(v.w));
        }
      };
      Unit uk, uv;
      auto query = [&](int at) -> uint4 {  // 8 dims of row at / 16
        const int r = at >> 4, qi = G > N ? 0 : r / G, h = G > N ? r : r % G;
        if (qi >= it.x.nq || h >= it.heads) return make_uint4(0, 0, 0, 0);
        return __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) +
                                                    ((int64_t)(it.x.row0 + qi) * a.H + it.h0 + h) * kDim) + (at & 15));
      };
      // 64 rows stay in registers between the maximum and the products' form (a call for one token: 18.0 -> 16.8 us);
      // 128 are read twice
      constexpr int kIter = N * 16 / kConvThreads;
      uint4 held[N == 64 ? kIter : 1];
      if (N == 64) {
#pragma unroll
        for (int i = 0; i < kIter; ++i) held[N == 64 ? i : 0] = query(ct + i * kConvThreads);
      }
      look_up(t0);
      load(uk, t0, false);
      if (!kShared) load(uv, t0, true);

      // the item's queries
      const uint32_t qb = n_item % C::kQBufs;
      bool ok = true;
      float qf;
      {
        float amax = 0.f;
#pragma unroll(N == 64 ? kIter : 4)
        for (int i = 0; i < kIter; ++i) {
          const uint4 u = N == 64 ? held[N == 64 ? i : 0] : query(ct + i * kConvThreads);
          const uint32_t v[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float x = fabsf(bf16_lo(v[j])), y = fabsf(bf16_hi(v[j]));
            if (x < INFINITY) amax = fmaxf(amax, x);
            if (y < INFINITY) amax = fmaxf(amax, y);
          }
        }
        amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));
        if (lane == 0) {
          s_qmax[n_item & 1u][w] = amax;
          mbar_arrive(smem_u32(&s_qmaxed));
        }
        ok = mbar_wait_bounded(smem_u32(&s_qmaxed), n_item & 1u, status) &&
             mbar_wait_bounded(smem_u32(&s_qempty[qb]), (n_item / C::kQBufs & 1u) ^ 1u, status);
        if ((dead = __any_sync(0xffffffffu, !ok))) break;
#pragma unroll
        for (int i = 0; i < kConvWarps; ++i) amax = fmaxf(amax, s_qmax[n_item & 1u][i]);
        const int ex = max((int)(__float_as_uint(amax) >> 23) - 127 - 14, -113);
        const float mul = a.scale < 0.f ? -pow2i(-ex) : pow2i(-ex);
        qf = pow2i(ex) * fabsf(a.scale) * kLog2e;
        const uint32_t to = base + C::kQOff + qb * C::kQBytes;
#pragma unroll(N == 64 ? kIter : 2)
        for (int i = 0; i < kIter; ++i) {
          const int at = ct + i * kConvThreads;
          const uint4 u = N == 64 ? held[N == 64 ? i : 0] : query(at);
          sts128(to + ((at & 15) >> 3) * C::kQRegion + tc::sw128_offset(at >> 4, at & 7),
                 pack_f16x2(bf16_lo(u.x) * mul, bf16_hi(u.x) * mul), pack_f16x2(bf16_lo(u.y) * mul, bf16_hi(u.y) * mul),
                 pack_f16x2(bf16_lo(u.z) * mul, bf16_hi(u.z) * mul), pack_f16x2(bf16_lo(u.w) * mul, bf16_hi(u.w) * mul));
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&s_qfull[qb]));
      }

      // the next tile's codes are loaded as soon as this one's are stored
      auto put_k = [&](int t, uint32_t k) {
        const uint32_t st = k % C::kStK;
        ok = mbar_wait_bounded(smem_u32(&s_kempty[st]), (k / C::kStK & 1u) ^ 1u, status);
        if ((dead = __any_sync(0xffffffffu, !ok || *abort_flag != 0))) return;
        float ev = uk.ks > 0.f ? exponent_of(kShared ? uk.ks : uk.vs) : -INFINITY;
        int first;
        if (kShared && mixed_tile(a, it, t, first)) {  // a NaN that only some queries see: its key's scores become NaN, its values 0
          uint32_t rows = 0;
#pragma unroll
          for (int i = 0; i < kChunks; ++i) {
            const uint32_t b = __ballot_sync(0xffffffffu, has_nan16(uk.c[i]));
#pragma unroll
            for (int r = 0; r < 4; ++r)
              if (b & (0x000f000fu << (4 * r))) rows |= 1u << (4 * i + r);
            uk.c[i] = without_nan16(uk.c[i]);
          }
          if (rows >> lane % kConvKeys & 1) ev = NAN;
        }
        if (lane < kConvKeys) s_par[k % kRing][kConvKeys * w + lane] = make_float2(uk.ks * qf, ev);
        store(uk, base + st * kTileBytes);
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(smem_u32(&s_par_full[k % kRing]));
          mbar_arrive(smem_u32(&s_kfull[st]));
        }
        load(uk, t + 1, false);
      };
      auto put_v = [&](int t, uint32_t k) {
        const uint32_t sv = k & 1u;
        ok = mbar_wait_bounded(smem_u32(&s_vempty[sv]), (k >> 1 & 1u) ^ 1u, status);
        if ((dead = __any_sync(0xffffffffu, !ok || *abort_flag != 0))) return;
        int first;
        if (mixed_tile(a, it, t, first)) {  // such a NaN in V: noted for the rows that see it, and taken as 0
#pragma unroll
          for (int i = 0; i < kChunks; ++i) {
            if (has_nan16(uv.c[i])) {
              const int pos = first + kConvKeys * w + 4 * i + sub;
#pragma unroll 1
              for (int j = 0; j < 16 * N; ++j) {  // dim j % 16 of the chunk, row j / 16
                const int d = j & 15, r = j >> 4, p = it.x.p0 + (G > N ? 0 : r / G);
                const uint32_t v = d < 4 ? uv.c[i].x : d < 8 ? uv.c[i].y : d < 12 ? uv.c[i].z : uv.c[i].w;
                if ((v >> (8 * (d & 3)) & 0x7f) == 0x7f &&
                    (t < it.x.ct ? pos < (p + 1) / a.r : pos <= p && pos > p - a.window))
                  atomicOr(&s_nan[n_item % kRing][(r * kDim + ch * 16 + d) / 32], 1u << ((ch * 16 + d) % 32));
              }
              s_nans[n_item % kRing] = 1;
              uv.c[i] = without_nan16(uv.c[i]);
            }
          }
        }
        store(uv, base + C::kVOff + sv * kTileBytes);
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&s_vfull[sv]));
        load(uv, t + 1, true);
      };
      if (!kShared) put_k(t0, k);
      for (int t = t0; t < t1 && !dead; ++t, ++k) {
        if ((t - t0) % kAhead == 0 && t + kAhead < t1) look_up(t + kAhead);
        if (kShared) {
          put_k(t, k);
        } else {  // K a tile ahead of V: S^T of the next tile does not wait for room for this one's V
          if (t + 1 < t1) put_k(t + 1, k + 1);
          if (!dead) put_v(t, k);
        }
      }
      if (dead) break;
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&s_iempty[n_item % kRing]));
    }
    if (dead) *abort_flag = 1;
  } else if (warp >= kMmaWarp) {
    // =================== products ===================
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kMmaRegs));
    if (warp == kMmaWarp && lane == 0) {
      // S^T
      constexpr uint32_t kId = idesc_f16(kTile, N, 0, 0);
      const uint64_t dk0 = tc::smem_desc_sw128(base, 16, 1024);
      const uint64_t dq0 = tc::smem_desc_sw128(base + C::kQOff, 16, 1024);
      int t = 0, t1 = 0;
      uint32_t n = 0;  // items begun
      bool ok = true;
      for (uint32_t k = 0; *abort_flag == 0; ++k) {
        const bool first = t == t1;
        if (first) {
          if (!(ok = item_ready(n))) break;
          t = s_item[n % kRing].t0;
          t1 = s_item[n % kRing].t1;
          mbar_arrive(smem_u32(&s_iempty[n % kRing]));
          ++n;
          if (t1 < 0) break;
        }
        ++t;
        const uint32_t st = k % C::kStK, qb = (n - 1) % C::kQBufs, g = k & 1u;
        ok = mbar_wait_bounded(smem_u32(&s_kfull[st]), k / C::kStK & 1u, status);
        if (first) ok = ok && mbar_wait_bounded(smem_u32(&s_qfull[qb]), (n - 1) / C::kQBufs & 1u, status);
        if (k >= 2) ok = ok && mbar_wait_bounded(smem_u32(&s_sfree[g]), ((k >> 1) - 1) & 1u, status);
        if (!ok) break;
        tc::fence_after_sync();
        tc::fence_proxy_async_smem();  // for the tiles' and P^T's plain stores, which the barriers made visible here
        const uint64_t dk = dk0 + ((st * kTileBytes) >> 4), dq = dq0 + ((qb * C::kQBytes) >> 4);
#pragma unroll
        for (int ks = 0; ks < kDim / 16; ++ks)
          tc::mma_bf16(tmem + g * N, dk + (((ks >> 2) * kRegion + (ks & 3) * 32) >> 4),
                       dq + (((ks >> 2) * C::kQRegion + (ks & 3) * 32) >> 4), kId, ks > 0 ? 1u : 0u);
        tc::mma_commit(smem_u32(&s_sfull[g]));
        if (!kShared) tc::mma_commit(smem_u32(&s_kempty[st]));
        if (t == t1) tc::mma_commit(smem_u32(&s_qempty[qb]));
      }
      if (!ok) *abort_flag = 1;
      tc::mma_commit(smem_u32(&s_drain[0]));  // every product has completed before tensor memory is freed
      mbar_wait_bounded(smem_u32(&s_drain[0]), 0, status);
    } else if (warp == kMmaWarp + 2 && lane == 0) {
      // O^T; an issuer of its own, because in one order with S^T each waits for what the other waits for
      constexpr uint32_t kId = idesc_f16(kDim, N, 1, 1);
      const uint64_t dv0 = tc::smem_desc_sw128(base + (kShared ? 0 : C::kVOff), kRegion, 1024);
      const uint64_t dp = tc::smem_desc_sw128(base + C::kPOff, N == 64 ? 1024 : kRegion, 1024);
      int t = 0, t1 = 0;
      uint32_t n = 0;  // items begun
      bool ok = true;
      for (uint32_t k = 0; *abort_flag == 0; ++k) {
        const bool first = t == t1;
        if (first) {
          if (!(ok = item_ready(n))) break;
          t = s_item[n % kRing].t0;
          t1 = s_item[n % kRing].t1;
          mbar_arrive(smem_u32(&s_iempty[n % kRing]));
          ++n;
          if (t1 < 0) break;
        }
        ++t;
        const uint32_t st = kShared ? k % C::kStK : k & 1u;
        ok = mbar_wait_bounded(smem_u32(&s_pfull), k & 1u, status);
        if (!kShared) ok = ok && mbar_wait_bounded(smem_u32(&s_vfull[st]), k >> 1 & 1u, status);
        if (first && n > 1) ok = ok && mbar_wait_bounded(smem_u32(&s_ofree), (n - 2) & 1u, status);  // O^T has been read
        if (!ok) break;
        tc::fence_after_sync();
        tc::fence_proxy_async_smem();  // for the tiles' and P^T's plain stores, which the barriers made visible here
        const uint64_t dv = dv0 + ((st * kTileBytes) >> 4);
#pragma unroll
        for (int ks = 0; ks < kTile / 16; ++ks)
          tc::mma_bf16(tmem + 2 * N, dv + ((ks * 2048) >> 4), dp + ((ks * 2048) >> 4), kId, first && ks == 0 ? 0u : 1u);
        tc::mma_commit(smem_u32(&s_odone));
        tc::mma_commit(kShared ? smem_u32(&s_kempty[st]) : smem_u32(&s_vempty[st]));
      }
      if (!ok) *abort_flag = 1;
      tc::mma_commit(smem_u32(&s_drain[1]));
      mbar_wait_bounded(smem_u32(&s_drain[1]), 0, status);
    } else if (warp == kMmaWarp + 1 && lane == 0) {
      // =================== the CTA's items, found ahead of their use ===================
      Items items{s_ctx.sh.u0, s_ctx.sh.slot_at, s_ctx.sh.slot};
      for (uint32_t n = 0;; ++n) {
        if (!mbar_wait_bounded(smem_u32(&s_iempty[n % kRing]), (n / kRing & 1u) ^ 1u, status) || *abort_flag) {
          *abort_flag = 1;
          break;
        }
        const bool more = next_item<false>(&s_ctx, &items, &s_item[n % kRing]);
        if (!more) s_item[n % kRing].t1 = -1;
        mbar_arrive(smem_u32(&s_ifull[n % kRing]));
        if (!more) break;
      }
    }
  } else {
    // =================== softmax: warp = (half of the rows, lane quadrant), thread = key ===================
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
    const int quad = warp & 3, hh = warp >> 2, key = quad * 32 + lane;
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
    const int r0 = hh * (N / 2);  // first row of this half
    const uint32_t prow = base + C::kPOff + (N == 128 ? hh * kRegion : 0);
    uint32_t k = 0;
    bool dead = false;
    for (uint32_t n_item = 0; !dead; ++n_item) {
      if ((dead = bar_or(kSoftBar, kSoftThreads, !item_ready(n_item) || *abort_flag != 0))) break;
      const Item& it = s_item[n_item % kRing];
      if (it.t1 < 0) break;
      const Slot& x = it.x;
      const int t0 = it.t0, t1 = it.t1;
      if (tid < N) {
        const int qi = G > N ? 0 : tid / G, h = G > N ? tid : tid % G;
        const bool real = qi < x.nq && h < it.heads;
        const int p = x.p0 + qi;
        s_sees[0][tid] = make_int2(0, real && a.cmp.k ? (p + 1) / a.r : 0);
        s_sees[1][tid] = make_int2(p - a.window + 1, real ? a.window : 0);
        s_out[tid] = real ? (x.row0 + qi) * a.H + it.h0 + h : -1;
        s_M[tid] = kNone;
        s_shift[tid] = kUnset;
      }
      bar_sync(kSoftBar, kSoftThreads);
      float l[32];  // this key's part of the rows' sums; two passes keep theirs in tensor memory in between
#pragma unroll
      for (int j = 0; j < 32; ++j) l[j] = 0.f;
      float e0 = 0.f;
      bool any_key = false, any_far = false;
      for (int t = t0; t < t1 && !dead; ++t, ++k) {
        int first;
        const bool mixed = mixed_tile(a, it, t, first), entries = t < x.ct;
        bool good = mbar_wait_bounded(smem_u32(&s_par_full[k % kRing]), k / kRing & 1u, status);
        const float2 par = s_par[k % kRing][key];
        const float kq = par.x, ev = par.y;
        const uint32_t there = __ballot_sync(0xffffffffu, ev > -INFINITY);
        if (!any_key && there) {
          e0 = __shfl_sync(0xffffffffu, ev, __ffs(there) - 1);
          any_key = true;
        }
        const bool far = ev > -INFINITY && fabsf(ev - e0) > 60.f;
        const float ie = ev == -INFINITY || far ? 0.f : ev == ev ? ex2(e0 - ev) : 1.f;  // NaN reaches l by the weights
        const bool warp_far = __any_sync(0xffffffffu, far);
        good = good && mbar_wait_bounded(smem_u32(&s_sfull[k & 1u]), k >> 1 & 1u, status);
        tc::fence_after_sync();
        bool pv_waited = k == 0;
        const uint64_t kq2 = f2_pack(kq, kq), ev2 = f2_pack(ev, ev), ie2 = f2_pack(ie, ie);
#pragma unroll 1
        for (int ps = 0; ps < C::kPasses; ++ps) {
          const int rb = r0 + 32 * ps;
          const uint32_t t_s = tmem + lane_off + (k & 1u) * N + rb, t_o = tmem + lane_off + 2 * N + rb,
                         t_l = tmem + lane_off + 3 * N + rb;
          float u[32];
          {
            uint32_t rs[32];
            tc::tmem_ld32_sync(t_s, rs);
            if (C::kPasses > 1) {
#pragma unroll
              for (int j = 0; j < 32; ++j) l[j] = 0.f;
              if (t > t0) tmem_ld32f_sync(t_l, l);
            }
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
              const float4 sf = *reinterpret_cast<const float4*>(s_shift + rb + j);
              f2_unpack(f2_fma(f2_pack(__uint_as_float(rs[j]), __uint_as_float(rs[j + 1])), kq2,
                               f2_add(ev2, f2_pack(sf.x, sf.y))), u[j], u[j + 1]);
              f2_unpack(f2_fma(f2_pack(__uint_as_float(rs[j + 2]), __uint_as_float(rs[j + 3])), kq2,
                               f2_add(ev2, f2_pack(sf.z, sf.w))), u[j + 2], u[j + 3]);
            }
          }
          if (mixed) {
            const int2* sees = s_sees[entries ? 0 : 1] + rb;
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if ((uint32_t)(first + key - sees[j].x) >= (uint32_t)sees[j].y) u[j] = -INFINITY;
          }
          float top = u[0];
#pragma unroll
          for (int j = 1; j < 32; ++j) top = fmaxf(top, u[j]);
          const bool bad = !good || *abort_flag != 0;
          if (bar_or(kHalfBar + hh, kSoftThreads / 2, top > kBase + kSlack || bad)) {
            // the references move to the maxima over the tile's keys
            {
              uint32_t rs[32];
              tc::tmem_ld32_sync(t_s, rs);
#pragma unroll
              for (int j = 0; j < 32; ++j) u[j] = u[j] == -INFINITY ? u[j] : fmaf(__uint_as_float(rs[j]), kq, ev);
            }
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              const int v = __reduce_max_sync(0xffffffffu, ord_of(u[j] == u[j] ? u[j] : -INFINITY));
              if (lane == 0) s_wmax[quad][hh * 32 + j] = v;
            }
            bool done = true;
            if (!pv_waited) done = mbar_wait_bounded(smem_u32(&s_odone), (k - 1) & 1u, status);
            pv_waited = true;
            if (bar_or(kHalfBar + hh, kSoftThreads / 2, bad || !done)) {
              dead = true;
              break;
            }
            tc::fence_after_sync();
            if (quad == 0) {
              const int r = rb + lane;
              const float old = s_M[r];
              float v = old;
#pragma unroll
              for (int q = 0; q < 4; ++q) v = fmaxf(v, float_of(s_wmax[q][hh * 32 + lane]));
              s_alpha[r] = ex2(old - v);
              s_M[r] = v;
              s_shift[r] = v == kNone ? kUnset : kBase - v;
            }
            bar_sync(kHalfBar + hh, kSoftThreads / 2);
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              u[j] += s_shift[rb + j];
              l[j] *= s_alpha[rb + j];
            }
            if (t > t0) {
#pragma unroll 1
              for (int c0 = 0; c0 < 32; c0 += 16) {
                uint32_t ro[16];
                tc::tmem_ld16_sync(t_o + c0, ro);
#pragma unroll
                for (int j = 0; j < 16; ++j) ro[j] = __float_as_uint(__uint_as_float(ro[j]) * s_alpha[rb + c0 + j]);
                tc::tmem_st16(t_o + c0, ro);
              }
              tc::tmem_wait_st();
            }
          }
          if (warp_far) {  // these keys' terms go to sums in shared memory that move their own reference; rare, so not unrolled
            if (!any_far) s_far[warp][32 * ps + lane] = make_float2(kNone, 0.f);
            if (ps == C::kPasses - 1) any_far = true;
            __syncwarp();
#pragma unroll 1
            for (int j = 0; j < 32; ++j) {
              const int2 sees = s_sees[entries ? 0 : 1][rb + j];
              float s = tmem_ld1_sync(t_s + j) * kq;
              if (!far || (mixed && (uint32_t)(first + key - sees.x) >= (uint32_t)sees.y)) s = -INFINITY;
              const float2 was = s_far[warp][32 * ps + j];
              float high = fmaxf(s, was.x);
#pragma unroll 1
              for (int o = 16; o > 0; o >>= 1) high = fmaxf(high, __shfl_xor_sync(0xffffffffu, high, o));
              float sum = ex2(s - high);
#pragma unroll 1
              for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
              if (lane == 0) s_far[warp][32 * ps + j] = make_float2(high, was.y * ex2(was.x - high) + sum);
            }
          }
          if (ps == C::kPasses - 1) {  // S^T may be overwritten
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&s_sfree[k & 1u]));
          }
          // the weights: unrounded into the sums, as halves into P^T (free once the previous O^T products are done)
          if (!pv_waited && !mbar_wait_bounded(smem_u32(&s_odone), (k - 1) & 1u, status)) *abort_flag = 1;
          pv_waited = true;
          tc::fence_after_sync();
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t pk[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int at = c * 8 + 2 * j;
              const float w0 = ex2(u[at]), w1 = ex2(u[at + 1]);
              pk[j] = pack_f16x2(w0, w1);
              f2_unpack(f2_fma(f2_pack(w0, w1), ie2, f2_pack(l[at], l[at + 1])), l[at], l[at + 1]);
            }
            const int chunk = N == 64 ? hh * 4 + c : ps * 4 + c;
            sts128(prow + tc::sw128_offset(key, chunk), pk[0], pk[1], pk[2], pk[3]);
          }
          if (C::kPasses > 1) tmem_st32f(t_l, l);
        }
        if (dead) break;
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&s_pfull));
      }
      // ---- the item's rows ----
      const bool done = !dead && mbar_wait_bounded(smem_u32(&s_odone), (k - 1) & 1u, status);
      dead = bar_or(kSoftBar, kSoftThreads, !done || *abort_flag != 0);
      if (dead) break;
      tc::fence_after_sync();
#pragma unroll 1
      for (int ps = 0; ps < C::kPasses; ++ps) {
        const int r = r0 + 32 * ps + lane;
        if (C::kPasses > 1) tmem_ld32f_sync(tmem + lane_off + 3 * N + r0 + 32 * ps, l);
        float sum = warp_sum32(l, lane);
        float m = any_key && s_M[r] > kNone ? s_M[r] - kBase - e0 : kNone;  // the sum is sum * 2^m
        if (any_far) {
          __syncwarp();
          const float2 o = s_far[warp][32 * ps + lane];
          const float top = fmaxf(m, o.x);
          sum = sum * ex2(m - top) + o.y * ex2(o.x - top);
          m = top;
        }
        s_m[quad][r] = m;
        s_l[quad][r] = sum;
      }
      bar_sync(kSoftBar, kSoftThreads);
      const bool whole = t0 == 0 && t1 == it.n_tiles;
      float* piece = ws_o + ((int64_t)blockIdx.x * 2 + (t0 == 0 ? 1 : 0)) * piece_floats<kDim>(N);
      if (tid < N) {
        float m = kNone, sum = 0.f;
#pragma unroll
        for (int q = 0; q < 4; ++q) m = fmaxf(m, s_m[q][tid]);
#pragma unroll
        for (int q = 0; q < 4; ++q) sum += s_l[q][tid] * ex2(s_m[q][tid] - m);
        const int at = s_out[tid];
        s_f[tid] = s_f2[tid] = 1.f;
        if (at >= 0 && whole) {
          const float2 f = finish_factors(a, at, m, s_M[tid], sum);
          s_f[tid] = f.x;
          s_f2[tid] = f.y;
        } else if (at >= 0) {
          piece[N * kDim + tid] = m;
          piece[N * kDim + N + tid] = s_M[tid];
          piece[N * kDim + 2 * N + tid] = sum;
        }
      }
      bar_sync(kSoftBar, kSoftThreads);
      const bool nans = s_nans[n_item % kRing] != 0;
#pragma unroll 1
      for (int c0 = 0; c0 < N / 2; c0 += 8) {
        uint32_t ro[8];
        tc::tmem_ld8_sync(tmem + lane_off + 2 * N + r0 + c0, ro);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int r = r0 + c0 + j, at = s_out[r];
          const float v = __uint_as_float(ro[j]) * s_f[r] * s_f2[r];
          if (at >= 0) {
            if (whole) static_cast<__nv_bfloat16*>(a.out)[(int64_t)at * kDim + key] = __float2bfloat16(v);
            else piece[r * kDim + key] = v;
          }
        }
      }
      if (nans) {  // what the converters took as 0
#pragma unroll 1
        for (int j = 0; j < N / 2; ++j) {
          const int r = r0 + j, at = s_out[r];
          if (at >= 0 && (s_nan[n_item % kRing][(r * kDim + key) / 32] >> (key % 32) & 1)) {
            if (whole) static_cast<__nv_bfloat16*>(a.out)[(int64_t)at * kDim + key] = __float2bfloat16(NAN);
            else piece[r * kDim + key] = NAN;
          }
        }
      }
      if (!whole && t0 == 0 && tid == 0)
        note_split(&s_ctx, x.row0, x.nq, it.sub, it.item0, it.n_tiles, ws_meta + blockIdx.x);
      tc::fence_before_sync();
      bar_sync(kSoftBar, kSoftThreads);
      if (nans) {  // the notes are taken again four items on
        for (int i = tid; i < N * kDim / 32; i += kSoftThreads) s_nan[n_item % kRing][i] = 0;
        if (tid == 0) s_nans[n_item % kRing] = 0;
        bar_sync(kSoftBar, kSoftThreads);
      }
      if (lane == 0) {
        mbar_arrive(smem_u32(&s_ofree));
        mbar_arrive(smem_u32(&s_iempty[n_item % kRing]));
      }
    }
    if (dead) *abort_flag = 1;
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == kMmaWarp) tc::tmem_dealloc(tmem, C::kCols);
}

template <int N, bool kShared>
cudaError_t run(const CacheAttnArgs& a, int sm_count, cudaStream_t stream) {
  using C = Tc<N, kShared>;
  // an item costs as much as 6 or 4 tiles beside its own (prompt chunks: 444 us with 0, 396 with 2, 354 so, 368 with 14)
  const Plan pl = make_plan(a, N, N == 128 ? 6 : 4);
  const Scratch sc = scratch_of<kDim>(a.ws, sm_count, N);
  const size_t smem = C::kSmem + 1024;
  cudaError_t e = cudaFuncSetAttribute(cache_attn_tc_kernel<N, kShared>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)smem);
  if (e != cudaSuccess) return e;
  if ((e = launch_after(cache_attn_tc_kernel<N, kShared>, dim3(sm_count), dim3(kThreads), smem, stream, a, pl,
                        sc.pieces, sc.meta)) != cudaSuccess)
    return e;
  return launch_after(cache_attn_join_kernel<__nv_bfloat16, kDim, N>, dim3(sm_count, N / kJoinWarps), dim3(32 * kJoinWarps), 0, stream, a, pl,
                      (const float*)sc.pieces, (const int4*)sc.meta);
}

}  // namespace

size_t cache_attn_tc_workspace(int sm_count) { return cache_attn::scratch_bytes(sm_count, 128, kDim, 0); }

cudaError_t launch_cache_attn_tc(const CacheAttnArgs& a, int rows, int sm_count, cudaStream_t stream) {
  const bool shared = (a.cmp.k ? a.cmp.v : a.raw.v) == nullptr;
  if (rows == 64) return shared ? run<64, true>(a, sm_count, stream) : run<64, false>(a, sm_count, stream);
  return shared ? run<128, true>(a, sm_count, stream) : run<128, false>(a, sm_count, stream);
}

}  // namespace csa
