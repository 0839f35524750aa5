// cache_attn.cu -- attention of new query rows over the 8-bit serving cache
// (csa_cache_attn_fwd): cached compressed entries (every visible one, or those
// listed) and a window of cached raw rows in one softmax.
//
// One CTA per (query row, KV head); tiles of 64 keys are widened to float32 in
// shared memory, scores, weights and sums are float32.
#include <math.h>

#include "cache.cuh"

namespace csa {

namespace {

constexpr int kThreads = 256;
constexpr int kTile = 64;

template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
cache_attn_kernel(CacheAttnArgs a) {
  extern __shared__ __align__(16) float sm[];
  const int G = a.H / a.H_kv;
  float* sQ = sm;                       // [G][D]
  float* sO = sQ + G * D;               // [G][D]
  float* sX = sO + G * D;               // [kTile][D + 1]
  float* sP = sX + kTile * (D + 1);     // [G][kTile]
  float* sM = sP + G * kTile;           // [G] running maximum
  float* sL = sM + G;                   // [G] running sum
  float* sA = sL + G;                   // [G] rescale of this tile
  __shared__ int s_blk[kTile], s_row[kTile];
  const int tid = threadIdx.x;
  const int row = blockIdx.x, kvh = blockIdx.y;
  const T* q = static_cast<const T*>(a.q);
  T* out = static_cast<T*>(a.out);
  const int h0 = kvh * G;
  const int b = owner_sequence(a.cu, a.B, row);
  int p = -1;
  if (b >= 0) {
    const int s0 = __ldg(a.cu + b), L = __ldg(a.cu + b + 1) - s0, p0 = __ldg(a.pos0 + b);
    const int64_t end = (int64_t)p0 + L;
    bool ok = p0 >= 0 && row >= s0 && row < s0 + L;
    ok = ok && (!a.raw.k || end <= a.raw.cap) && (!a.cmp.k || end / a.r <= a.cmp.cap) && end <= INT32_MAX;
    if (ok) p = p0 + row - s0;
    else if (tid == 0) raise_status(a.status, CSA_ERR_DEVICE_BOUNDS);
  }
  const int vis = p >= 0 && a.cmp.k ? (int)(((int64_t)p + 1) / a.r) : 0;
  const int n_cmp = p < 0 ? 0 : (a.idx ? a.k_pad : vis);
  const int w0 = p >= 0 && a.raw.k ? max(0, p - a.window + 1) : 0;
  const int n_raw = p >= 0 && a.raw.k ? p - w0 + 1 : 0;
  const int ct = (n_cmp + kTile - 1) / kTile, tiles = ct + (n_raw + kTile - 1) / kTile;
  for (int i = tid; i < G * D; i += kThreads) {
    sQ[i] = to_f32(q[((int64_t)row * a.H + h0) * D + i]);
    sO[i] = 0.f;
  }
  for (int g = tid; g < G; g += kThreads) sM[g] = -INFINITY, sL[g] = 0.f;
  for (int it = 0; it < tiles; ++it) {
    const CacheView& c = it < ct ? a.cmp : a.raw;
    __syncthreads();
    if (tid < kTile) {
      int pos = -1;
      if (it < ct) {
        const int s = it * kTile + tid;
        if (s < n_cmp) {
          pos = s;
          if (a.idx) {
            pos = __ldg(a.idx + (int64_t)row * a.k_pad + s);
            if (pos >= 0) {
              const int64_t e = (int64_t)pos - (a.cu_cmp ? __ldg(a.cu_cmp + b) : 0);
              pos = e >= 0 && e < vis ? (int)e : -1;
              if (pos < 0) raise_status(a.status, CSA_ERR_DEVICE_BOUNDS);
            }
          }
        }
      } else {
        const int s = (it - ct) * kTile + tid;
        if (s < n_raw) pos = w0 + s;
      }
      const int blk = pos >= 0 ? cache_block(c, b, pos, a.status) : -1;
      s_blk[tid] = blk;
      s_row[tid] = pos & ((1 << c.log_block) - 1);
    }
    __syncthreads();
    auto widen = [&](const uint8_t* codes, const float* scale) {
      for (int i = tid; i < kTile * D; i += kThreads) {
        const int k = i / D, e = i % D, blk = s_blk[k];
        float v = 0.f;
        if (blk >= 0) {
          const int64_t bh = (int64_t)blk * c.H_kv + kvh;
          const uint16_t code = __ldg(codes + ((bh << c.log_block) + s_row[k]) * D + e);
          v = f16x2_to_float2(e4m3x2_to_f16x2(code)).x * __ldg(scale + bh);
        }
        sX[k * (D + 1) + e] = v;
      }
    };
    widen(c.k, c.k_scale);
    __syncthreads();
    for (int i = tid; i < G * kTile; i += kThreads) {
      const int g = i / kTile, k = i % kTile;
      float s = 0.f;
      for (int e = 0; e < D; ++e) s = fmaf(sQ[g * D + e], sX[k * (D + 1) + e], s);
      sP[i] = s_blk[k] >= 0 ? s * a.scale : -INFINITY;
    }
    __syncthreads();
    for (int g = tid; g < G; g += kThreads) {
      float m = sM[g], l = 0.f;
      for (int k = 0; k < kTile; ++k) m = fmaxf(m, sP[g * kTile + k]);
      const float ref = m == -INFINITY ? 0.f : m;
      for (int k = 0; k < kTile; ++k) {
        const float e = expf(sP[g * kTile + k] - ref);
        sP[g * kTile + k] = e;
        l += e;
      }
      sA[g] = expf(sM[g] - ref);
      sL[g] = sL[g] * sA[g] + l;
      sM[g] = m;
    }
    if (c.v) widen(c.v, c.v_scale);
    __syncthreads();
    for (int i = tid; i < G * D; i += kThreads) {
      const int g = i / D, e = i % D;
      float o = sO[i] * sA[g];
      for (int k = 0; k < kTile; ++k) o = fmaf(sP[g * kTile + k], sX[k * (D + 1) + e], o);
      sO[i] = o;
    }
  }
  __syncthreads();
  for (int g = tid; g < G; g += kThreads) {
    float m = sM[g], l = sL[g], f = 1.f;
    if (a.sink && b >= 0) {
      const float s = __ldg(a.sink + h0 + g), n = fmaxf(m, s);
      f = m == -INFINITY ? 0.f : expf(m - n);
      l = l * f + (s == -INFINITY ? 0.f : expf(s - n));
      m = n;
    }
    sA[g] = l > 0.f || l != l ? f / l : 0.f;
    if (a.lse) a.lse[(int64_t)row * a.H + h0 + g] = l > 0.f || l != l ? m + logf(l) : -INFINITY;
  }
  __syncthreads();
  for (int i = tid; i < G * D; i += kThreads)
    out[((int64_t)row * a.H + h0) * D + i] = from_f32<T>(sA[i / D] == 0.f ? 0.f : sO[i] * sA[i / D]);
}

template <typename T, int D>
cudaError_t run(const CacheAttnArgs& a, cudaStream_t stream) {
  const int G = a.H / a.H_kv;
  const size_t smem = sizeof(float) * (2 * (size_t)G * D + kTile * (D + 1) + (size_t)G * kTile + 3 * G);
  cudaError_t e = cudaFuncSetAttribute(cache_attn_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  cache_attn_kernel<T, D><<<dim3(a.T_cap, a.H_kv), kThreads, smem, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

size_t cache_attn_workspace(int, int, int, int, int) { return 0; }

cudaError_t launch_cache_attn(const CacheAttnArgs& a, bool fp32, int, cudaStream_t stream) {
  if (a.T_cap <= 0) return cudaSuccess;
  if (a.d == 64) return fp32 ? run<float, 64>(a, stream) : run<__nv_bfloat16, 64>(a, stream);
  return fp32 ? run<float, 128>(a, stream) : run<__nv_bfloat16, 128>(a, stream);
}

}  // namespace csa
