// cache.cu -- rows quantised into the 8-bit serving cache as they arrive, and
// read back (csa_cache_write, csa_cache_read).
//
// Write.  One item is one (sequence, block, head, K or V): the rows of the call
// that fall into that block, and the codes that the block already holds before
// them.  s = 2^e is the smallest with max|x| <= 448 s; appended rows take
// max(s_old, s), and when that grew the earlier codes are multiplied by s_old / s
// (a power of two: exact above E4M3's subnormals).  One item owns its scale and
// its codes, so nothing is atomic and results do not depend on order.
// Bound by HBM: each row is read once (kept in registers between the maximum and
// the conversion) and each code written once.  Few rows per sequence (a decode
// step) are bound by latency: a warp per item then, 8 items a CTA.
//
// Read.  value = code * scale, one rounding; bound by HBM.
#include "cache.cuh"

namespace csa {

namespace {

constexpr int kThreads = 256;
constexpr int kKeep = 4;  // 8-element chunks that a thread holds between the two passes

// Eight consecutive elements, as they are stored.
template <typename T> struct Chunk;
template <> struct Chunk<__nv_bfloat16> {
  uint4 u;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = __ldg(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[2 * i] = bf16_lo(w[i]), v[2 * i + 1] = bf16_hi(w[i]);
  }
};
template <> struct Chunk<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = __ldg(reinterpret_cast<const float4*>(p));
    b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
};

// First slot of sequence b: consecutive sequences are at least as far apart as
// the blocks that the earlier one's rows can touch.
__device__ __forceinline__ int64_t slot_base(int32_t cu, int b, int lg) {
  return ((int64_t)cu >> lg) + 2 * (int64_t)b;
}

struct Owner {
  int b, row0, row1, p0;
  int64_t base;
};

// The last sequence b with slot_base <= slot, by a whole warp: one round of
// loads up to 31 sequences, 32 ways a round above.
__device__ __forceinline__ Owner slot_owner(const int32_t* cu, const int32_t* pos0, int B, int lg, int64_t slot,
                                            int lane) {
  Owner o;
  if (B < 32) {
    const int cv = lane <= B ? __ldg(cu + lane) : 0, pv = lane < B ? __ldg(pos0 + lane) : 0;
    o.b = max(__popc(__ballot_sync(0xffffffffu, lane < B && slot_base(cv, lane, lg) <= slot)) - 1, 0);
    o.row0 = __shfl_sync(0xffffffffu, cv, o.b);
    o.row1 = __shfl_sync(0xffffffffu, cv, o.b + 1);
    o.p0 = __shfl_sync(0xffffffffu, pv, o.b);
  } else {
    int lo = 0, n = B;
    while (n > 1) {
      const int step = (n + 31) / 32, at = lane * step;
      const bool le = at < n && slot_base(__ldg(cu + lo + at), lo + at, lg) <= slot;
      const int skip = max(__popc(__ballot_sync(0xffffffffu, le)) - 1, 0) * step;
      lo += skip;
      n = min(step, n - skip);
    }
    o.b = lo;
    o.row0 = __ldg(cu + lo);
    o.row1 = __ldg(cu + lo + 1);
    o.p0 = __ldg(pos0 + lo);
  }
  o.base = slot_base(o.row0, o.b, lg);
  return o;
}

// kWarpItems: a warp per item, 8 items a CTA (few rows per sequence); else a CTA
// per item, whose threads hold kKeep chunks each of a full block.
template <typename T, int D, bool kWarpItems>
__global__ void __launch_bounds__(kWarpItems ? kThreads : 512)
cache_write_kernel(CacheView c, const T* __restrict__ x_k, const T* __restrict__ x_v, const int32_t* __restrict__ cu,
                   const int32_t* __restrict__ pos0, int B, int T_cap, int64_t n_items, int* status) {
  constexpr int kChunks = D / 8;
  __shared__ float s_max[16];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int t = kWarpItems ? lane : threadIdx.x, n_t = kWarpItems ? 32 : blockDim.x;
  const int64_t item = kWarpItems ? (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5) : blockIdx.x;
  if (item >= n_items) return;
  const int kinds = c.v ? 2 : 1;
  const int h = (int)(item % c.H_kv);
  const bool is_v = (item / c.H_kv) % kinds != 0;
  const int64_t slot = item / (c.H_kv * kinds);
  const int lg = c.log_block, P = 1 << lg;

  const Owner o = slot_owner(cu, pos0, B, lg, slot, lane);
  const int row0 = o.row0, L = o.row1 - row0, p0 = o.p0;
  if (L <= 0 || row0 < 0 || (int64_t)row0 + L > T_cap) return;
  if (p0 < 0 || (int64_t)p0 + L > c.cap) {
    if (t == 0) raise_status(status, CSA_ERR_DEVICE_BOUNDS);
    return;
  }
  const int64_t nth = slot - o.base;
  const int64_t j = (p0 >> lg) + nth;  // block of the sequence
  if (nth < 0 || (j << lg) >= (int64_t)p0 + L) return;
  const int first = (int)(j << lg);  // position of the block's first row
  const int lo = max(p0 - first, 0), hi = min(p0 + L - first, P);
  const int n = (hi - lo) * kChunks;
  const T* x = (is_v ? x_v : x_k) + (((int64_t)row0 + first + lo - p0) * c.H_kv + h) * D;
  const int64_t stride = (int64_t)c.H_kv * D;

  Chunk<T> v[kKeep];
  auto load = [&](int base) {
#pragma unroll
    for (int k = 0; k < kKeep; ++k) {
      const int i = base + t + k * n_t;
      if (i < n) v[k].load(x + (i / kChunks) * stride + (i % kChunks) * 8);
    }
  };
  load(0);
  const int blk = cache_block(c, o.b, first, status);
  if (blk < 0) return;
  uint8_t* codes = (is_v ? c.v : c.k) + ((int64_t)blk * c.H_kv + h) * ((int64_t)P * D);
  float* scale = (is_v ? c.v_scale : c.k_scale) + (int64_t)blk * c.H_kv + h;
  const float old_s = lo > 0 ? *scale : 0.f;

  float amax = 0.f;
  for (int base = 0; base < n; base += n_t * kKeep) {
    if (base > 0) load(base);
#pragma unroll
    for (int k = 0; k < kKeep; ++k) {
      if (base + t + k * n_t < n) {
        float f[8];
        v[k].get(f);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (fabsf(f[e]) < INFINITY) amax = fmaxf(amax, fabsf(f[e]));
      }
    }
  }
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, s));
  if (!kWarpItems) {
    if (lane == 0) s_max[threadIdx.x >> 5] = amax;
    __syncthreads();
    for (int w = 0; w < (n_t >> 5); ++w) amax = fmaxf(amax, s_max[w]);
  }
  const float need = pow2i(e4m3_scale_exponent(amax));
  const float new_s = lo > 0 ? fmaxf(old_s, need) : need;

  if (lo > 0 && new_s > old_s) {  // the codes before the new rows, under the larger scale
    const float f = old_s / new_s;
    uint4* row = reinterpret_cast<uint4*>(codes);
    for (int i = t; i < lo * (D / 16); i += n_t) {
      uint4 u = row[i];
      uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 a = f16x2_to_float2(e4m3x2_to_f16x2((uint16_t)w[e]));
        const float2 d = f16x2_to_float2(e4m3x2_to_f16x2((uint16_t)(w[e] >> 16)));
        w[e] = (uint32_t)e4m3x2_from_floats(a.x * f, a.y * f) |
               (uint32_t)e4m3x2_from_floats(d.x * f, d.y * f) << 16;
      }
      row[i] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  const float inv = 1.f / new_s;  // a power of two
  for (int base = 0; base < n; base += n_t * kKeep) {
    if (n > n_t * kKeep) load(base);  // more rows than the registers held
#pragma unroll
    for (int k = 0; k < kKeep; ++k) {
      const int i = base + t + k * n_t;
      if (i < n) {
        float f[8];
        v[k].get(f);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = fabsf(f[e]) < INFINITY ? f[e] * inv : NAN;
        const uint32_t w0 = (uint32_t)e4m3x2_from_floats(f[0], f[1]) | (uint32_t)e4m3x2_from_floats(f[2], f[3]) << 16;
        const uint32_t w1 = (uint32_t)e4m3x2_from_floats(f[4], f[5]) | (uint32_t)e4m3x2_from_floats(f[6], f[7]) << 16;
        *reinterpret_cast<uint2*>(codes + (lo + i / kChunks) * D + (i % kChunks) * 8) = make_uint2(w0, w1);
      }
    }
  }
  if (t == 0) *scale = new_s;
}

constexpr int kReadRows = 16;  // packed rows of a CTA

template <typename T> __device__ __forceinline__ void store16(T* p, const float (&v)[16]);
template <> __device__ __forceinline__ void store16<__nv_bfloat16>(__nv_bfloat16* p, const float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
    reinterpret_cast<uint4*>(p)[i] =
        make_uint4(pack_bf16x2(v[8 * i], v[8 * i + 1]), pack_bf16x2(v[8 * i + 2], v[8 * i + 3]),
                   pack_bf16x2(v[8 * i + 4], v[8 * i + 5]), pack_bf16x2(v[8 * i + 6], v[8 * i + 7]));
}
template <> __device__ __forceinline__ void store16<float>(float* p, const float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    reinterpret_cast<float4*>(p)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
cache_read_kernel(CacheView c, const int32_t* __restrict__ cu, const int32_t* __restrict__ pos0, int B, int T_cap,
                  T* __restrict__ k_out, T* __restrict__ v_out, int* status) {
  constexpr int kChunks = D / 16;
  __shared__ int s_blk[kReadRows], s_row[kReadRows];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t row0 = (int64_t)blockIdx.x * kReadRows;
  const int rows = (int)min((int64_t)kReadRows, T_cap - row0);
  if ((int)threadIdx.x < rows) {
    const int row = (int)row0 + threadIdx.x;
    int blk = -1, r = 0;
    const int b = owner_sequence(cu, B, row);
    if (b >= 0) {
      const int s0 = __ldg(cu + b), p0 = __ldg(pos0 + b);
      const int64_t end = (int64_t)p0 + (__ldg(cu + b + 1) - s0);
      if (p0 < 0 || end > c.cap || row < s0 || (int64_t)p0 + row - s0 >= end) {
        raise_status(status, CSA_ERR_DEVICE_BOUNDS);
      } else {
        const int p = p0 + row - s0;
        blk = cache_block(c, b, p, status);
        r = p & ((1 << c.log_block) - 1);
      }
    }
    s_blk[threadIdx.x] = blk;
    s_row[threadIdx.x] = r;
  }
  __syncthreads();
  const int per_kind = rows * c.H_kv * kChunks;
  for (int i = threadIdx.x; i < per_kind * (v_out ? 2 : 1); i += kThreads) {
    const bool is_v = i >= per_kind;
    const int u = is_v ? i - per_kind : i;
    const int ch = u % kChunks, h = (u / kChunks) % c.H_kv, rr = u / (kChunks * c.H_kv);
    const int blk = s_blk[rr];
    float v[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) v[e] = 0.f;
    if (blk >= 0) {
      const int64_t bh = (int64_t)blk * c.H_kv + h;
      const uint4 q = __ldg(reinterpret_cast<const uint4*>((is_v ? c.v : c.k) + ((bh << c.log_block) + s_row[rr]) * D) + ch);
      const float s = __ldg((is_v ? c.v_scale : c.k_scale) + bh);
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 a = f16x2_to_float2(e4m3x2_to_f16x2((uint16_t)w[e]));
        const float2 d = f16x2_to_float2(e4m3x2_to_f16x2((uint16_t)(w[e] >> 16)));
        v[4 * e] = a.x * s, v[4 * e + 1] = a.y * s, v[4 * e + 2] = d.x * s, v[4 * e + 3] = d.y * s;
      }
    }
    store16((is_v ? v_out : k_out) + ((row0 + rr) * c.H_kv + h) * D + ch * 16, v);
  }
}

template <typename T, int D>
cudaError_t write_launch(const CacheView& c, const void* x_k, const void* x_v, const int32_t* cu, const int32_t* pos0, int B,
                  int T_cap, int* status, cudaStream_t stream) {
  const int64_t slots = ((int64_t)T_cap >> c.log_block) + 2 * (int64_t)B;
  const int64_t items = slots * c.H_kv * (c.v ? 2 : 1);
  const T* k = static_cast<const T*>(x_k);
  const T* v = static_cast<const T*>(x_v);
  if (T_cap <= 4 * (int64_t)B)
    return launch_after(cache_write_kernel<T, D, true>, dim3((unsigned)((items + 7) / 8)), dim3(kThreads), 0, stream,
                        c, k, v, cu, pos0, B, T_cap, items, status);
  return launch_after(cache_write_kernel<T, D, false>, dim3((unsigned)items), dim3((D / 8 << c.log_block) / kKeep), 0,
                      stream, c, k, v, cu, pos0, B, T_cap, items, status);
}

template <typename T, int D>
cudaError_t read_launch(const CacheView& c, const int32_t* cu, const int32_t* pos0, int B, int T_cap, void* k_out,
                 void* v_out, int* status, cudaStream_t stream) {
  return launch_after(cache_read_kernel<T, D>, dim3((unsigned)(((int64_t)T_cap + kReadRows - 1) / kReadRows)),
                      dim3(kThreads), 0, stream, c, cu, pos0, B, T_cap, static_cast<T*>(k_out),
                      static_cast<T*>(v_out), status);
}

}  // namespace

cudaError_t launch_cache_write(const CacheView& c, const void* x_k, const void* x_v, const int32_t* cu,
                               const int32_t* pos0, int B, int T_cap, bool fp32, int* status, cudaStream_t stream) {
  if (B <= 0 || T_cap <= 0) return cudaSuccess;
  if (c.d == 64)
    return fp32 ? write_launch<float, 64>(c, x_k, x_v, cu, pos0, B, T_cap, status, stream)
         : write_launch<__nv_bfloat16, 64>(c, x_k, x_v, cu, pos0, B, T_cap, status, stream);
  return fp32 ? write_launch<float, 128>(c, x_k, x_v, cu, pos0, B, T_cap, status, stream)
         : write_launch<__nv_bfloat16, 128>(c, x_k, x_v, cu, pos0, B, T_cap, status, stream);
}

cudaError_t launch_cache_read(const CacheView& c, const int32_t* cu, const int32_t* pos0, int B, int T_cap, bool fp32,
                              void* k_out, void* v_out, int* status, cudaStream_t stream) {
  if (T_cap <= 0) return cudaSuccess;
  if (c.d == 64)
    return fp32 ? read_launch<float, 64>(c, cu, pos0, B, T_cap, k_out, v_out, status, stream)
         : read_launch<__nv_bfloat16, 64>(c, cu, pos0, B, T_cap, k_out, v_out, status, stream);
  return fp32 ? read_launch<float, 128>(c, cu, pos0, B, T_cap, k_out, v_out, status, stream)
         : read_launch<__nv_bfloat16, 128>(c, cu, pos0, B, T_cap, k_out, v_out, status, stream);
}

}  // namespace csa
