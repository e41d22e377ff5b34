// layer_norm.cuh -- layer norm of a feature map's channels, forward and backward.
//
//   mu = mean_c x,  v = mean_c (x - mu)^2,  r = 1 / sqrt(v + eps),  xh = (x - mu) r
//   y = gamma xh + beta
//   g = gamma dy,  dx = r (g - mean_c g - xh mean_c (g xh)) (+ dres)
//   dgamma = sum_rows dy xh,  dbeta = sum_rows dy
//
// A row is read once: a group of threads (a warp, or a 256-thread CTA for
// wide rows) holds it in registers as vectors of V elements, vector
// t + threads * i in thread t, so every load of a warp is one contiguous run.
// The variance is the mean of the squared deviations from the mean already
// found (not E x^2 - mu^2, which cancels where |mu| is far above the spread).
// Everything is fp32 between the load and the store; y and dx are rounded
// once, to the features' type.
//
// Both kernels are bound by HBM: the grid is a few CTAs per SM that walk the
// rows, each warp with kRows rows' loads in flight at once.
#pragma once

#include <cuda_bf16.h>

#include "ptx.cuh"

namespace rib {

constexpr int kLnThreads = 256;
constexpr int kLnWarps = kLnThreads / 32;
constexpr int kLnMaxC = 8192;
constexpr int G_LN_IN = 160, G_LN_OUT = 161, G_LN_STAT = 162, G_LN_PART = 163;

struct LnParams {
  const void* x;
  const void* dy;
  const void* dres;
  const float* gamma;
  const float* beta;
  float* mean;        // forward: out (may be null); backward: in
  float* rstd;
  void* out;          // y, or dx
  float* part;        // [gridDim.x][2][C]: dgamma, dbeta partials (null: not wanted)
  int rows, C;
  float eps;
};

// V consecutive elements as fp32
template <typename T, int V>
struct LnVec;
template <>
struct LnVec<__nv_bfloat16, 8> {
  typedef uint4 raw;
  static __device__ __forceinline__ raw load(const void* p, size_t i) {
    return __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + i));
  }
  static __device__ __forceinline__ raw zero() { return make_uint4(0, 0, 0, 0); }
  static __device__ __forceinline__ void get(const raw& r, float (&f)[8]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      f[2 * e] = __uint_as_float(w[e] << 16);
      f[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ void store(void* p, size_t i, const float (&f)[8]) {
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p) + i) =
        make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                   pack_bf16x2(f[6], f[7]));
  }
};
template <>
struct LnVec<float, 4> {
  typedef float4 raw;
  static __device__ __forceinline__ raw load(const void* p, size_t i) {
    return __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p) + i));
  }
  static __device__ __forceinline__ raw zero() { return make_float4(0.f, 0.f, 0.f, 0.f); }
  static __device__ __forceinline__ void get(const raw& r, float (&f)[4]) {
    f[0] = r.x; f[1] = r.y; f[2] = r.z; f[3] = r.w;
  }
  static __device__ __forceinline__ void store(void* p, size_t i, const float (&f)[4]) {
    *reinterpret_cast<float4*>(static_cast<float*>(p) + i) = make_float4(f[0], f[1], f[2], f[3]);
  }
};
template <>
struct LnVec<__nv_bfloat16, 1> {
  typedef __nv_bfloat16 raw;
  static __device__ __forceinline__ raw load(const void* p, size_t i) {
    return static_cast<const __nv_bfloat16*>(p)[i];
  }
  static __device__ __forceinline__ raw zero() { return __float2bfloat16_rn(0.f); }
  static __device__ __forceinline__ void get(const raw& r, float (&f)[1]) {
    f[0] = __bfloat162float(r);
  }
  static __device__ __forceinline__ void store(void* p, size_t i, const float (&f)[1]) {
    static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(f[0]);
  }
};
template <>
struct LnVec<float, 1> {
  typedef float raw;
  static __device__ __forceinline__ raw load(const void* p, size_t i) {
    return static_cast<const float*>(p)[i];
  }
  static __device__ __forceinline__ raw zero() { return 0.f; }
  static __device__ __forceinline__ void get(const raw& r, float (&f)[1]) { f[0] = r; }
  static __device__ __forceinline__ void store(void* p, size_t i, const float (&f)[1]) {
    static_cast<float*>(p)[i] = f[0];
  }
};

__device__ __forceinline__ float ln_warp_sum(float v) {
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
  return v;
}

// Sum over the group that holds a row: a warp, or the CTA (through shared
// memory, the warps' sums added in warp order by every thread; `buf` holds
// kLnWarps values and is not reused before the next barrier but one).
template <bool CTA>
__device__ __forceinline__ float ln_group_sum(float v, float* buf) {
  v = ln_warp_sum(v);
  if constexpr (CTA) {
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int w = 0; w < kLnWarps; ++w) v += buf[w];
  }
  return v;
}

// gamma or beta of one vector (1 or 0 where the pointer is null)
template <int V>
__device__ __forceinline__ void ln_weight(const float* p, int c, bool in, float fill,
                                          float (&f)[V]) {
#pragma unroll
  for (int e = 0; e < V; ++e) f[e] = (p && in) ? __ldg(p + c + e) : fill;
}

// Rows a group works on at once: as many as keep about 16 fp32 values of x
// per thread in flight.
template <int V, int NV, bool CTA>
__host__ __device__ constexpr int ln_rows() {
  return CTA ? 1 : (V * NV <= 8 ? 4 : V * NV <= 16 ? 2 : 1);
}

// -------------------------------------------------------------- forward
// grid: a few CTAs per SM (ln_grid), block kLnThreads.
template <typename T, int V, int NV, bool CTA>
__global__ void __launch_bounds__(kLnThreads) layer_norm_fwd_kernel(const LnParams p) {
  using L = LnVec<T, V>;
  constexpr int R = ln_rows<V, NV, CTA>();
  constexpr int G = CTA ? kLnThreads : 32;
  __shared__ float buf[2][kLnWarps];
  const int t = CTA ? threadIdx.x : threadIdx.x & 31;
  const int C = p.C;
  const size_t elems = static_cast<size_t>(p.rows) * C;
  const float inv_c = 1.f / static_cast<float>(C);
  const long long group = CTA ? blockIdx.x : blockIdx.x * kLnWarps + (threadIdx.x >> 5);
  const long long groups = CTA ? gridDim.x : static_cast<long long>(gridDim.x) * kLnWarps;
  // the weights stay in registers over the rows when they are few
  constexpr bool kKeep = V * NV <= 16;
  float gk[kKeep ? NV : 1][V], bk[kKeep ? NV : 1][V];
  if constexpr (kKeep) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (t + G * i) * V;
      ln_weight<V>(p.gamma, c, c < C, 1.f, gk[i]);
      ln_weight<V>(p.beta, c, c < C, 0.f, bk[i]);
    }
  }
  for (long long r0 = group * R; r0 < p.rows; r0 += groups * R) {
    typename L::raw raw[R][NV];
#pragma unroll
    for (int k = 0; k < R; ++k)
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (t + G * i) * V;
        const size_t at = static_cast<size_t>(r0 + k) * C + c;
        raw[k][i] = (c < C && r0 + k < p.rows && rib_guard(at + V - 1, elems, G_LN_IN))
                        ? L::load(p.x, at)
                        : L::zero();
      }
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const long long r = r0 + k;
      if (r >= p.rows) break;
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float f[V];
        L::get(raw[k][i], f);
#pragma unroll
        for (int e = 0; e < V; ++e) s += f[e];
      }
      const float mu = ln_group_sum<CTA>(s, buf[0]) * inv_c;
      float q = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const bool in = (t + G * i) * V < C;
        float f[V];
        L::get(raw[k][i], f);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float d = in ? f[e] - mu : 0.f;
          q = fmaf(d, d, q);
        }
      }
      const float var = ln_group_sum<CTA>(q, buf[1]) * inv_c;
      const float rs = rsqrtf(var + p.eps);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (t + G * i) * V;
        float f[V], g[V], b[V];
        L::get(raw[k][i], f);
        if constexpr (kKeep) {
#pragma unroll
          for (int e = 0; e < V; ++e) { g[e] = gk[i][e]; b[e] = bk[i][e]; }
        } else {
          ln_weight<V>(p.gamma, c, c < C, 1.f, g);
          ln_weight<V>(p.beta, c, c < C, 0.f, b);
        }
#pragma unroll
        for (int e = 0; e < V; ++e) f[e] = fmaf((f[e] - mu) * rs, g[e], b[e]);
        const size_t at = static_cast<size_t>(r) * C + c;
        if (c < C && rib_guard(at + V - 1, elems, G_LN_OUT)) L::store(p.out, at, f);
      }
      if (t == 0 && rib_guard(static_cast<size_t>(r), static_cast<size_t>(p.rows), G_LN_STAT)) {
        if (p.mean) p.mean[r] = mu;
        if (p.rstd) p.rstd[r] = rs;
      }
    }
  }
}

// -------------------------------------------------------------- backward
// Each thread sums dgamma and dbeta of its own columns over the rows its
// group walks; the CTA's warps are then added in warp order through shared
// memory and the CTA's sums go to the workspace, where reduce_rows_kernel
// adds the CTAs in order: the same result on every run.
// Dynamic shared memory: kLnWarps * 2 * C floats for warp groups when the
// sums are wanted, else none.
template <typename T, int V, int NV, bool CTA>
__global__ void __launch_bounds__(kLnThreads) layer_norm_bwd_kernel(const LnParams p) {
  using L = LnVec<T, V>;
  constexpr int R = V * NV <= 8 && !CTA ? 2 : 1;
  constexpr int G = CTA ? kLnThreads : 32;
  __shared__ float buf[2][2][kLnWarps];
  extern __shared__ float ln_sums[];
  const int t = CTA ? threadIdx.x : threadIdx.x & 31;
  const int C = p.C;
  const size_t elems = static_cast<size_t>(p.rows) * C;
  const float inv_c = 1.f / static_cast<float>(C);
  const long long group = CTA ? blockIdx.x : blockIdx.x * kLnWarps + (threadIdx.x >> 5);
  const long long groups = CTA ? gridDim.x : static_cast<long long>(gridDim.x) * kLnWarps;
  float sg[NV][V], sb[NV][V];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < V; ++e) sg[i][e] = sb[i][e] = 0.f;
  constexpr bool kKeep = V * NV <= 16;
  float gk[kKeep ? NV : 1][V];
  if constexpr (kKeep) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (t + G * i) * V;
      ln_weight<V>(p.gamma, c, c < C, 1.f, gk[i]);
    }
  }
  int turn = 0;
  for (long long r0 = group * R; r0 < p.rows; r0 += groups * R) {
    typename L::raw xr[R][NV], dr[R][NV], ar[R][NV];
    float mu[R], rs[R];
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const bool row = r0 + k < p.rows;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (t + G * i) * V;
        const size_t at = static_cast<size_t>(r0 + k) * C + c;
        const bool in = row && c < C && rib_guard(at + V - 1, elems, G_LN_IN);
        xr[k][i] = in ? L::load(p.x, at) : L::zero();
        dr[k][i] = in ? L::load(p.dy, at) : L::zero();
        ar[k][i] = in && p.dres ? L::load(p.dres, at) : L::zero();
      }
      mu[k] = row ? __ldg(p.mean + r0 + k) : 0.f;
      rs[k] = row ? __ldg(p.rstd + r0 + k) : 0.f;
    }
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const long long r = r0 + k;
      if (r >= p.rows) break;
      float s1 = 0.f, s2 = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (t + G * i) * V;
        float x[V], d[V], g[V];
        L::get(xr[k][i], x);
        L::get(dr[k][i], d);
        if constexpr (kKeep) {
#pragma unroll
          for (int e = 0; e < V; ++e) g[e] = gk[i][e];
        } else {
          ln_weight<V>(p.gamma, c, c < C, 1.f, g);
        }
        const bool in = c < C;
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float xh = in ? (x[e] - mu[k]) * rs[k] : 0.f;
          const float gd = d[e] * g[e];
          sg[i][e] = fmaf(d[e], xh, sg[i][e]);
          sb[i][e] += d[e];
          s1 += gd;
          s2 = fmaf(gd, xh, s2);
        }
      }
      // two buffers in turn: a thread may still read this row's sums while
      // the fastest one writes the next row's
      float* b0 = buf[turn][0];
      float* b1 = buf[turn][1];
      turn ^= 1;
      if constexpr (CTA) {
        s1 = ln_warp_sum(s1);
        s2 = ln_warp_sum(s2);
        if ((threadIdx.x & 31) == 0) {
          b0[threadIdx.x >> 5] = s1;
          b1[threadIdx.x >> 5] = s2;
        }
        __syncthreads();
        s1 = s2 = 0.f;
#pragma unroll
        for (int w = 0; w < kLnWarps; ++w) {
          s1 += b0[w];
          s2 += b1[w];
        }
      } else {
        s1 = ln_warp_sum(s1);
        s2 = ln_warp_sum(s2);
      }
      const float m1 = s1 * inv_c, m2 = s2 * inv_c;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (t + G * i) * V;
        float x[V], d[V], a[V], g[V];
        L::get(xr[k][i], x);
        L::get(dr[k][i], d);
        L::get(ar[k][i], a);
        if constexpr (kKeep) {
#pragma unroll
          for (int e = 0; e < V; ++e) g[e] = gk[i][e];
        } else {
          ln_weight<V>(p.gamma, c, c < C, 1.f, g);
        }
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float xh = (x[e] - mu[k]) * rs[k];
          a[e] = fmaf(rs[k], fmaf(-xh, m2, fmaf(d[e], g[e], -m1)), a[e]);
        }
        const size_t at = static_cast<size_t>(r) * C + c;
        if (c < C && rib_guard(at + V - 1, elems, G_LN_OUT)) L::store(p.out, at, a);
      }
    }
  }
  if (!p.part) return;
  float* mine = p.part + static_cast<size_t>(blockIdx.x) * 2 * C;
  const size_t part_n = static_cast<size_t>(gridDim.x) * 2 * C;
  const size_t part_0 = static_cast<size_t>(blockIdx.x) * 2 * C;
  if constexpr (CTA) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const int c = (t + G * i) * V + e;
        if (c < C && rib_guard(part_0 + C + c, part_n, G_LN_PART)) {
          mine[c] = sg[i][e];
          mine[C + c] = sb[i][e];
        }
      }
  } else {
    float* w = ln_sums + static_cast<size_t>(threadIdx.x >> 5) * 2 * C;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const int c = (t + G * i) * V + e;
        if (c < C) {
          w[c] = sg[i][e];
          w[C + c] = sb[i][e];
        }
      }
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * C; c += kLnThreads) {
      float s = 0.f;
#pragma unroll
      for (int k = 0; k < kLnWarps; ++k) s += ln_sums[static_cast<size_t>(k) * 2 * C + c];
      if (rib_guard(part_0 + c, part_n, G_LN_PART)) mine[c] = s;
    }
  }
}

// -------------------------------------------------------------- sums of partials
// out[c] = sum_r part[r][c], r in order within each of kLnWarps interleaved
// row classes, the classes then added in order: deterministic.  Columns
// [0, n0) go to out0, [n0, n0 + n1) to out1 (either may be null).
// grid ceil((n0 + n1) / 32), block kLnThreads.
__global__ void __launch_bounds__(kLnThreads)
    reduce_rows_kernel(const float* part, int rows, int n0, float* out0, int n1, float* out1) {
  __shared__ float sums[kLnWarps][32];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int n = n0 + n1, c = blockIdx.x * 32 + lane;
  const size_t total = static_cast<size_t>(rows) * n;
  float s = 0.f;
  if (c < n) {
#pragma unroll 8
    for (int r = w; r < rows; r += kLnWarps) {
      const size_t at = static_cast<size_t>(r) * n + c;
      if (rib_guard(at, total, G_LN_PART)) s += part[at];
    }
  }
  sums[w][lane] = s;
  __syncthreads();
  if (w == 0 && c < n) {
    s = 0.f;
#pragma unroll
    for (int k = 0; k < kLnWarps; ++k) s += sums[k][lane];
    if (c < n0) {
      if (out0) out0[c] = s;
    } else if (out1) {
      out1[c - n0] = s;
    }
  }
}

}  // namespace rib
