// cache.cu -- rows quantised into the 8-bit serving cache as they arrive, and
// read back (csa_cache_write, csa_cache_read).
//
// Write.  One item is one (sequence, block, head, K or V): the rows of the call
// that fall into that block, and the codes that the block already holds before
// them.  s = 2^e is the smallest with max|x| <= 448 s; appended rows take
// max(s_old, s), and when that grew the earlier codes are multiplied by s_old / s
// (a power of two: exact above E4M3's subnormals).  One item owns its scale and
// its codes, so nothing is atomic and results do not depend on order.
// Each row is read once (kept in registers between the maximum and the conversion)
// and each code written once: bound by HBM, once the instructions are few enough.
// At ten an element (a test for infinities each, 64-bit divisions per item) issue
// was the bound: 117 us for 16 prompts of 1K to 16K rows (4 heads, K and V, 128
// dims); with maxima on bf16 pairs as bits and rare infinities apart 81 us, 85% of
// the rate of a plain copy.  Up to 16 rows a sequence a warp takes an item, 8 items
// a CTA: 64 sequences with 1, 4, 16 rows 5 to 6 us against 7.7, 7.9, 8.8 us.
//
// Read.  value = code * scale, one rounding; bound by HBM, four bytes written for one
// read with float32: 46 us for 8 prefixes of 3K to 16K rows (72% of the copy rate).
// What is left is the look-up of a CTA's rows before its first load; a grid that
// stays resident and looks the next rows up meanwhile was no faster (48 us).
#include "cache.cuh"

namespace csa {

namespace {

constexpr int kThreads = 256;
constexpr int kKeep = 4;  // 8-element chunks that a thread holds between the two passes

__device__ __forceinline__ void mul2(float& a, float& b, float m) {  // both products in one instruction
  asm("{\n .reg .b64 x, y;\n mov.b64 x, {%0, %1};\n mov.b64 y, {%2, %2};\n mul.rn.f32x2 x, x, y;\n mov.b64 {%0, %1}, x;\n}"
      : "+f"(a), "+f"(b) : "f"(m));
}
constexpr uint32_t kInfBits = 0x7f800000u;

// Eight consecutive elements, as they are stored.  top: the largest |x| as float32 bits, which
// compare like numbers; from kInfBits on, an element is not finite.
template <typename T> struct Chunk;
template <> struct Chunk<__nv_bfloat16> {
  uint4 u;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = __ldg(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[2 * i] = bf16_lo(w[i]), v[2 * i + 1] = bf16_hi(w[i]);
  }
  __device__ __forceinline__ uint32_t top() const {
    const uint32_t a = max2(max2(u.x & 0x7fff7fffu, u.y & 0x7fff7fffu), max2(u.z & 0x7fff7fffu, u.w & 0x7fff7fffu));
    return max(a << 16, a & 0xffff0000u);
  }
  static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t m;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(a), "r"(b));
    return m;
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
  __device__ __forceinline__ uint32_t top() const {
    float v[8];
    get(v);
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
    return m;
  }
};

// First slot of sequence b: consecutive sequences are at least as far apart as
// the blocks that the earlier one's rows can touch.
__device__ __forceinline__ int slot_base(int32_t cu, int b, int lg) { return (cu >> lg) + 2 * b; }

struct Owner {
  int b, row0, row1, p0, base;
};

// The last sequence b with slot_base <= slot, by a whole warp: one round of
// loads up to 31 sequences, 32 ways a round above.
__device__ __forceinline__ Owner slot_owner(const int32_t* cu, const int32_t* pos0, int B, int lg, int slot,
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
// per item, whose threads hold kKeep chunks each of a full block (four CTAs of 64 rows
// x 128 dims an SM in bf16: 81 us, with three 83, with the two of 64 registers 104).
template <typename T, int D, bool kWarpItems>
__global__ void __launch_bounds__(kWarpItems ? kThreads : 512, kWarpItems ? 4 : sizeof(T) == 2 ? 4 : 2)
cache_write_kernel(CacheView c, const T* __restrict__ x_k, const T* __restrict__ x_v, const int32_t* __restrict__ cu,
                   const int32_t* __restrict__ pos0, int B, int T_cap, uint32_t n_items, int* status) {
  constexpr int kChunks = D / 8;
  __shared__ uint32_t s_max[16];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int t = kWarpItems ? lane : threadIdx.x, n_t = kWarpItems ? 32 : blockDim.x;
  const uint32_t item = kWarpItems ? blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5) : blockIdx.x;
  if (item >= n_items) return;
  const uint32_t parts = c.v ? 2 * c.H_kv : c.H_kv;
  const int slot = (int)(item / parts);
  int h = (int)(item - slot * parts);
  const bool is_v = h >= c.H_kv;
  if (is_v) h -= c.H_kv;
  const int lg = c.log_block, P = 1 << lg;

  const Owner o = slot_owner(cu, pos0, B, lg, slot, lane);
  const int row0 = o.row0, L = o.row1 - row0, p0 = o.p0;
  if (L <= 0 || row0 < 0 || (int64_t)row0 + L > T_cap) return;
  if (p0 < 0 || (int64_t)p0 + L > c.cap) {
    if (t == 0) raise_status(status, CSA_ERR_DEVICE_BOUNDS);
    return;
  }
  const int nth = slot - o.base;
  const int64_t j = (int64_t)(p0 >> lg) + nth;  // block of the sequence
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

  uint32_t most = 0;     // of the finite elements
  bool special = false;  // others among this thread's
  for (int base = 0; base < n; base += n_t * kKeep) {
    if (base > 0) load(base);
#pragma unroll
    for (int k = 0; k < kKeep; ++k) {
      if (base + t + k * n_t < n) {
        uint32_t m = v[k].top();
        if (m >= kInfBits) {
          special = true;
          m = 0;
          float f[8];
          v[k].get(f);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (fabsf(f[e]) < INFINITY) m = max(m, __float_as_uint(fabsf(f[e])));
        }
        most = max(most, m);
      }
    }
  }
  most = __reduce_max_sync(0xffffffffu, most);
  if (!kWarpItems) {
    if (lane == 0) s_max[threadIdx.x >> 5] = most;
    __syncthreads();
    for (int w = 0; w < (n_t >> 5); ++w) most = max(most, s_max[w]);
  }
  const float amax = __uint_as_float(most);
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
        for (int e = 0; e < 8; e += 2) mul2(f[e], f[e + 1], inv);
        if (special) {  // an infinity becomes NaN; a NaN is one already
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (!(fabsf(f[e]) < INFINITY)) f[e] = NAN;
        }
        const uint32_t w0 = (uint32_t)e4m3x2_from_floats(f[0], f[1]) | (uint32_t)e4m3x2_from_floats(f[2], f[3]) << 16;
        const uint32_t w1 = (uint32_t)e4m3x2_from_floats(f[4], f[5]) | (uint32_t)e4m3x2_from_floats(f[6], f[7]) << 16;
        *reinterpret_cast<uint2*>(codes + (lo + i / kChunks) * D + (i % kChunks) * 8) = make_uint2(w0, w1);
      }
    }
  }
  if (t == 0) *scale = new_s;
}

constexpr int kReadRows = 16;  // packed rows of a CTA
constexpr int kReadAhead = 2;  // chunks of 8 codes that a thread has in flight

template <typename T> __device__ __forceinline__ void store8(T* p, const float (&v)[8]);
template <> __device__ __forceinline__ void store8<__nv_bfloat16>(__nv_bfloat16* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) =
      make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}
template <> __device__ __forceinline__ void store8<float>(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
cache_read_kernel(CacheView c, const int32_t* __restrict__ cu, const int32_t* __restrict__ pos0, int B, int T_cap,
                  T* __restrict__ k_out, T* __restrict__ v_out, int* status) {
  constexpr int kChunks = D / 8;
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
  const int row_chunks = c.H_kv * kChunks, per_kind = rows * row_chunks, n = v_out ? 2 * per_kind : per_kind;
  for (int i0 = threadIdx.x; i0 < n; i0 += kThreads * kReadAhead) {  // K's chunks, then V's
    uint2 q[kReadAhead];
    float s[kReadAhead];
#pragma unroll
    for (int k = 0; k < kReadAhead; ++k) {
      const int at = i0 + k * kThreads, i = at < per_kind ? at : at - per_kind;
      q[k] = make_uint2(0, 0);
      s[k] = 0.f;
      if (at < n) {
        const int ch = i % kChunks, rr = i / row_chunks, h = (i - rr * row_chunks) / kChunks, blk = s_blk[rr];
        if (blk >= 0) {
          const int64_t bh = (int64_t)blk * c.H_kv + h;
          q[k] = __ldg(reinterpret_cast<const uint2*>((at < per_kind ? c.k : c.v) +
                                                      ((bh << c.log_block) + s_row[rr]) * D) + ch);
          s[k] = __ldg((at < per_kind ? c.k_scale : c.v_scale) + bh);
        }
      }
    }
#pragma unroll
    for (int k = 0; k < kReadAhead; ++k) {
      const int at = i0 + k * kThreads;
      if (at < n) {
        const uint32_t w[2] = {q[k].x, q[k].y};
        float v[8];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float2 x = f16x2_to_float2(e4m3x2_to_f16x2((uint16_t)w[e]));
          const float2 y = f16x2_to_float2(e4m3x2_to_f16x2((uint16_t)(w[e] >> 16)));
          v[4 * e] = x.x * s[k], v[4 * e + 1] = x.y * s[k], v[4 * e + 2] = y.x * s[k], v[4 * e + 3] = y.y * s[k];
        }
        T* out = at < per_kind ? k_out + (int64_t)at * 8 : v_out + (int64_t)(at - per_kind) * 8;
        store8(out + row0 * c.H_kv * D, v);
      }
    }
  }
}

template <typename T, int D>
cudaError_t write_launch(const CacheView& c, const void* x_k, const void* x_v, const int32_t* cu, const int32_t* pos0, int B,
                  int T_cap, int* status, cudaStream_t stream) {
  const int64_t slots = ((int64_t)T_cap >> c.log_block) + 2 * (int64_t)B;
  const int64_t items = slots * c.H_kv * (c.v ? 2 : 1);
  const T* k = static_cast<const T*>(x_k);
  const T* v = static_cast<const T*>(x_v);
  if (T_cap <= 16 * (int64_t)B)
    return launch_after(cache_write_kernel<T, D, true>, dim3((unsigned)((items + 7) / 8)), dim3(kThreads), 0, stream,
                        c, k, v, cu, pos0, B, T_cap, (uint32_t)items, status);
  return launch_after(cache_write_kernel<T, D, false>, dim3((unsigned)items), dim3((D / 8 << c.log_block) / kKeep), 0,
                      stream, c, k, v, cu, pos0, B, T_cap, (uint32_t)items, status);
}

template <typename T, int D>
cudaError_t read_launch(const CacheView& c, const int32_t* cu, const int32_t* pos0, int B, int T_cap, void* k_out,
                 void* v_out, int* status, cudaStream_t stream) {
  return launch_after(cache_read_kernel<T, D>, dim3((unsigned)(((int64_t)T_cap + kReadRows - 1) / kReadRows)),
                      dim3(kThreads), 0, stream, c, cu, pos0, B, T_cap, static_cast<T*>(k_out), static_cast<T*>(v_out), status);
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
