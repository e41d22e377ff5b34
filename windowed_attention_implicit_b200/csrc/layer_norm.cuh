// layer_norm.cuh -- layer norm of a feature map's channels, forward and backward.
//
//   mu = mean_c x,  v = mean_c (x - mu)^2,  r = 1 / sqrt(v + eps),  xh = (x - mu) r
//   y = gamma xh + beta
//   g = gamma dy,  dx = r (g - mean_c g - xh mean_c (g xh)) (+ dres)
//   dgamma = sum_rows dy xh,  dbeta = sum_rows dy
//
// The variance is the mean of the squared deviations from the mean already
// found (not E x^2 - mu^2, which cancels where |mu| is far above the spread).
// Everything is fp32 between the load and the store; y and dx are rounded
// once, to the features' type.  Bound by HBM.
//
// ln_async_kernel (up to 1024 channels): every warp runs its own pipeline over
// blocks of a few rows.  Rows are contiguous, so a block is one run of bytes
// whatever the channel count, odd ones included: a bulk copy brings it into
// one of two or three shared-memory stages, the warp works on it there, writes
// y (or dx) over x (or dy) and a bulk copy takes it back.  With three stages the
// next blocks are in flight meanwhile, without holding registers; with two (the
// fp32 backward of 525 to 780 single elements, whose three do not fit) the next
// block's copy starts when this one's results have left, and its latency shows.
// No warp waits for another.  L lanes hold a row as vectors of V elements, vector j + L i in lane
// j, so 192 channels of bf16 use all 32 lanes (four rows of eight lanes, three
// vectors each) where a lane per vector would idle a quarter of them.
// Measured, bf16, 192 channels: forward of 294912 rows 38 to 40 us (226 MB, 5.8
// TB/s), backward of 147456 with a second gradient 41 us (226 MB and the sums);
// fp32, 333 channels, backward of 9217 rows 20 us for 49 MB: DRAM 22 % and issue 32
// % busy, so latency at nine warps an SM, single elements by way of shared memory.
//
// ln_row_*_kernel (wider rows, the fp32 backward of more than 780 channels
// that are not whole vectors, or pointers off a 16-byte address): a group of
// threads (a CTA above 1024 channels, else a warp) holds a row in registers.
#pragma once

#include <cuda_bf16.h>

#include "ptx.cuh"

namespace rib {

constexpr int kLnThreads = 256;
constexpr int kLnWarps = kLnThreads / 32;
constexpr int kLnMaxC = 8192;
constexpr int G_LN_IN = 160, G_LN_OUT = 161, G_LN_STAT = 162, G_LN_PART = 163;

// Programmatic dependent launch: a kernel lets the next one's blocks start as
// soon as SMs are free (at its own start: these kernels fill the SMs in one
// wave), and each kernel waits for the one before it, complete with its
// writes, before it touches global memory.  Only launch latency and a
// kernel's set-up overlap the one before.  Every block of a kernel launched
// this way calls it, so that kernels stay ordered one after the other.
// What such a kernel reads may thus be written while it is already there: it
// reads by plain loads behind the wait (and by TMA), never by the non-coherent
// path, which takes data that is constant for the whole life of a kernel.
__device__ __forceinline__ void pdl_wait() {
  asm volatile("griddepcontrol.launch_dependents;\n\tgriddepcontrol.wait;" ::: "memory");
}

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

// V consecutive elements as fp32 (plain loads, not the read-only path: y may
// be x, and dx dy or dres)
template <typename T, int V>
struct LnVec;
template <>
struct LnVec<__nv_bfloat16, 8> {
  typedef uint4 raw;
  static __device__ __forceinline__ raw load(const void* p, size_t i) {
    return *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + i);
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
    return *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
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
  for (int e = 0; e < V; ++e) f[e] = (p && in) ? p[c + e] : fill;
}

// Rows a group works on at once: as many as keep about 16 fp32 values of x
// per thread in flight.
template <int V, int NV, bool CTA>
__host__ __device__ constexpr int ln_rows() {
  return CTA ? 1 : (V * NV <= 8 ? 4 : V * NV <= 16 ? 2 : 1);
}

// -------------------------------------------------------------- forward
// grid: a few CTAs per SM (plan_ln), block kLnThreads.
template <typename T, int V, int NV, bool CTA>
__global__ void __launch_bounds__(kLnThreads) ln_row_fwd_kernel(const LnParams p) {
  using L = LnVec<T, V>;
  constexpr int R = ln_rows<V, NV, CTA>();
  constexpr int G = CTA ? kLnThreads : 32;
  __shared__ float buf[2][kLnWarps];
  pdl_wait();
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
__global__ void __launch_bounds__(kLnThreads) ln_row_bwd_kernel(const LnParams p) {
  using L = LnVec<T, V>;
  constexpr int R = V * NV <= 8 && !CTA ? 2 : 1;
  constexpr int G = CTA ? kLnThreads : 32;
  __shared__ float buf[2][2][kLnWarps];
  extern __shared__ float ln_sums[];
  pdl_wait();
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
      mu[k] = row ? p.mean[r0 + k] : 0.f;
      rs[k] = row ? p.rstd[r0 + k] : 0.f;
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

// -------------------------------------------------------------- blocks of rows
constexpr int kLnMaxStages = 3;
constexpr int SITE_LN = 45;

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void bulk_store(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst),
               "r"(smem_u32(src)), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void bulk_store_wait_read_one() {
  asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
}

struct LnBlocks {
  int rows;              // rows of a block
  uint32_t bytes;        // its bytes in shared memory (a multiple of 128)
  int warps;             // per CTA
  int stages;            // 2 or 3
  uint64_t wait_limit_ns;
};

// Slot i of a lane: what it holds of a row at a time, as P packed fp32 pairs,
// to and from shared memory.  Whole vectors: vector j + L i (V elements, V / 2
// pairs).  Single elements (V = 1): elements j + 2 L i and j + 2 L i + L as one
// pair.  `row` is the row's first byte; elements beyond C read as zero
// and are not written (a vector beyond C is not asked for).
template <typename T, int V, int L>
struct LnSlot;
template <int L>
struct LnSlot<__nv_bfloat16, 8, L> {
  static constexpr int P = 4;
  static __device__ __forceinline__ void get(const uint8_t* row, int i, int j, int, uint64_t (&f)[4]) {
    const uint4 r = *reinterpret_cast<const uint4*>(row + 16 * (j + L * i));
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int e = 0; e < 4; ++e)
      f[e] = pk2(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xffff0000u));
  }
  static __device__ __forceinline__ void put(uint8_t* row, int i, int j, int, const uint64_t (&f)[4]) {
    *reinterpret_cast<uint4*>(row + 16 * (j + L * i)) =
        make_uint4(pack_bf16x2(lo2(f[0]), hi2(f[0])), pack_bf16x2(lo2(f[1]), hi2(f[1])),
                   pack_bf16x2(lo2(f[2]), hi2(f[2])), pack_bf16x2(lo2(f[3]), hi2(f[3])));
  }
};
template <int L>
struct LnSlot<float, 4, L> {
  static constexpr int P = 2;
  static __device__ __forceinline__ void get(const uint8_t* row, int i, int j, int, uint64_t (&f)[2]) {
    const float4 r = *reinterpret_cast<const float4*>(row + 16 * (j + L * i));
    f[0] = pk2(r.x, r.y);
    f[1] = pk2(r.z, r.w);
  }
  static __device__ __forceinline__ void put(uint8_t* row, int i, int j, int, const uint64_t (&f)[2]) {
    *reinterpret_cast<float4*>(row + 16 * (j + L * i)) =
        make_float4(lo2(f[0]), hi2(f[0]), lo2(f[1]), hi2(f[1]));
  }
};
template <typename T, int L>
struct LnSlot<T, 1, L> {
  static constexpr int P = 1;
  static __device__ __forceinline__ void get(const uint8_t* row, int i, int j, int C, uint64_t (&f)[1]) {
    const T* r = reinterpret_cast<const T*>(row);
    const int c = j + 2 * L * i;
    f[0] = pk2(c < C ? static_cast<float>(r[c]) : 0.f, c + L < C ? static_cast<float>(r[c + L]) : 0.f);
  }
  static __device__ __forceinline__ void put(uint8_t* row, int i, int j, int C, const uint64_t (&f)[1]) {
    T* r = reinterpret_cast<T*>(row);
    const int c = j + 2 * L * i;
    if (c < C) r[c] = static_cast<T>(lo2(f[0]));   // to nearest
    if (c + L < C) r[c + L] = static_cast<T>(hi2(f[0]));
  }
};
// column of half h of pair e of slot i
template <int V, int L>
__device__ __forceinline__ int ln_column(int i, int j, int e, int h) {
  return V == 1 ? j + 2 * L * i + L * h : (j + L * i) * V + 2 * e + h;
}

template <int L>
__device__ __forceinline__ float ln_lane_sum(float v) {
#pragma unroll
  for (int m = L / 2; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
  return v;
}
__device__ __forceinline__ float ln_pair_sum(uint64_t v) { return lo2(v) + hi2(v); }
__device__ __forceinline__ uint64_t ln_both(float v) { return pk2(v, v); }

// gamma or beta of vector `vec` from shared memory.  The vectors' first four
// floats lie together and their last four behind all of those, so that
// neighbouring lanes read neighbouring 16 bytes.
template <int V>
__device__ __forceinline__ int ln_weight_slot(int c, int C) {
  return V == 8 ? (c & 4 ? C / 2 : 0) + (c >> 3) * 4 + (c & 3) : c;
}
template <int V, int L, int P>
__device__ __forceinline__ void ln_weight_get(const float* w, int i, int j, int C, uint64_t (&f)[P]) {
  if constexpr (V == 1) {
    const int c = j + 2 * L * i;
    f[0] = pk2(c < C ? w[c] : 0.f, c + L < C ? w[c + L] : 0.f);
  } else {
#pragma unroll
    for (int h = 0; h < V / 4; ++h) {
      const float4 r = *reinterpret_cast<const float4*>(w + h * (C / 2) + 4 * (j + L * i));
      f[2 * h] = pk2(r.x, r.y);
      f[2 * h + 1] = pk2(r.z, r.w);
    }
  }
}

// grid: CTAs that fit the SMs; block 32 * q.warps; dynamic shared memory:
// gamma (and beta) [C] fp32, then each warp's stages, then its barriers.  At
// the end of the backward the stages hold the warps' sums.
template <typename T, int V, int NV, int L, bool BWD>
__global__ void __launch_bounds__(BWD ? 384 : 512)
    ln_async_kernel(const LnParams p, const LnBlocks q) {
  using LP = LnSlot<T, V, L>;
  constexpr int P = LP::P;
  constexpr int G = 32 / L;   // rows side by side
  // rows whose chains of shuffles run interleaved, where the registers allow
  constexpr int RR = (L == 32 || V == 1) && NV * P <= 8 ? 2 : 1;
  constexpr uint32_t ES = sizeof(T);
  extern __shared__ __align__(128) uint8_t ln_smem[];
  __shared__ int abort_flag;
  volatile int* ab = &abort_flag;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int j = lane & (L - 1), grp = lane / L;
  const int C = p.C, arrays = BWD ? (p.dres ? 3 : 2) : 1;
  const uint32_t w_bytes = (static_cast<uint32_t>(BWD ? 1 : 2) * 4 * C + 127u) & ~127u;
  const uint32_t warp_bytes = q.stages * arrays * q.bytes;
  float* s_gamma = reinterpret_cast<float*>(ln_smem);
  float* s_beta = s_gamma + C;
  uint8_t* mine = ln_smem + w_bytes + warp * warp_bytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(ln_smem + w_bytes + q.warps * warp_bytes) +
                   warp * kLnMaxStages;
  if (threadIdx.x == 0) abort_flag = 0;
  if (lane == 0) {
    for (int i = 0; i < q.stages; ++i) mbar_init(&full[i], 1);
    fence_mbarrier_init();
  }
  pdl_wait();
  for (int c = threadIdx.x; c < C; c += blockDim.x) {
    s_gamma[ln_weight_slot<V>(c, C)] = p.gamma ? p.gamma[c] : 1.f;
    if (!BWD) s_beta[ln_weight_slot<V>(c, C)] = p.beta ? p.beta[c] : 0.f;
  }
  __syncthreads();
  const float inv_c = 1.f / static_cast<float>(C);
  const uint32_t row_bytes = C * ES;
  const int blocks = (p.rows + q.rows - 1) / q.rows;
  const int step = gridDim.x * q.warps, first = warp * gridDim.x + blockIdx.x;
  const uint8_t* src[3] = {static_cast<const uint8_t*>(p.x), static_cast<const uint8_t*>(p.dy),
                           static_cast<const uint8_t*>(p.dres)};
  uint8_t* out = static_cast<uint8_t*>(p.out);
  const size_t all_bytes = static_cast<size_t>(p.rows) * row_bytes;
  auto rows_of = [&](int b) { return min(q.rows, p.rows - b * q.rows); };
  auto at = [&](int b) { return static_cast<size_t>(b) * (q.rows * row_bytes); };
  // A block of rows of an odd size begins off a 16-byte address (the tensors
  // themselves do not): it lies in its stage as it lies in memory, behind the
  // bytes of the row before it up to the last 16-byte address.
  auto lead_of = [&](int b) { return V == 1 ? static_cast<uint32_t>(at(b)) & 15u : 0u; };
  auto stage = [&](int s, int a) { return mine + (s * arrays + a) * q.bytes; };
  // Starts block b's copies into stage s, whole 16 bytes; up to 15 bytes that
  // the tensor has behind its last 16-byte address are copied by the lanes.
  auto load = [&](int b, int s) {
    const uint32_t bytes = rows_of(b) * row_bytes;
    if constexpr (V != 1) {
      if (lane == 0) {
        mbar_arrive_expect_tx(&full[s], arrays * bytes);
        for (int a = 0; a < arrays; ++a) bulk_load(stage(s, a), src[a] + at(b), bytes, &full[s]);
      }
    } else {
      const size_t from = at(b) - lead_of(b), end = at(b) + bytes;
      const size_t to = min((end + 15) & ~static_cast<size_t>(15), all_bytes & ~static_cast<size_t>(15));
      const uint32_t whole = to > from ? static_cast<uint32_t>(to - from) : 0u;
      if (from + whole < end) {
        for (int a = 0; a < arrays; ++a)
          if (from + whole + lane * ES < end && rib_guard(from + whole + lane * ES, all_bytes, G_LN_IN))
            reinterpret_cast<T*>(stage(s, a) + whole)[lane] =
                reinterpret_cast<const T*>(src[a] + from + whole)[lane];
        __syncwarp();
      }
      if (lane == 0) {
        mbar_arrive_expect_tx(&full[s], arrays * whole);
        for (int a = 0; a < arrays && whole; ++a)
          bulk_load(stage(s, a), src[a] + from, whole, &full[s]);
      }
    }
  };
  // the rows' statistics, lane r holding row r of the next block
  float mu_next = 0.f, rs_next = 0.f;
  auto load_stats = [&](int b) {
    if (BWD && b < blocks && lane < rows_of(b)) {
      const size_t r = static_cast<size_t>(b) * q.rows + lane;
      if (rib_guard(r, p.rows, G_LN_STAT)) {
        mu_next = p.mean[r];
        rs_next = p.rstd[r];
      }
    }
  };
  [[maybe_unused]] uint64_t sg[BWD ? NV : 1][P], sb[BWD ? NV : 1][P];
  if constexpr (BWD) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < P; ++e) sg[i][e] = sb[i][e] = 0ull;
  }
  bool ok = true;
  int loaded = 0, ahead = first;   // blocks whose copies were started; the next one
  for (; loaded < q.stages - 1 && ahead < blocks; ahead += step, ++loaded) load(ahead, loaded);
  load_stats(first);
  int s = 0, s_load = q.stages - 1;
  uint32_t ph = 0;
  int n = 0;
  for (int b = first; b < blocks; b += step, ++n) {
    const float mu_b = mu_next, rs_b = rs_next;
    load_stats(b + step);
    if (!(ok = warp_wait(&full[s], ph, ab, q.wait_limit_ns, SITE_LN))) break;
    const int rows = rows_of(b);
    const uint32_t lead = lead_of(b);
    uint8_t* x0 = stage(s, 0) + lead;
    for (int r0 = 0; r0 < rows; r0 += G * RR) {
      uint32_t off[RR];
      bool in_row[RR];
#pragma unroll
      for (int k = 0; k < RR; ++k) {
        in_row[k] = r0 + grp + G * k < rows;
        off[k] = (r0 + grp + G * k) * row_bytes;
      }
      if constexpr (!BWD) {
        uint64_t f[RR][NV][P];
        float mu[RR], rs[RR];
#pragma unroll
        for (int k = 0; k < RR; ++k) {
          uint64_t sum = 0ull;
#pragma unroll
          for (int i = 0; i < NV; ++i) {
            if (in_row[k] && ln_column<V, L>(i, j, 0, 0) < C) {
              LP::get(x0 + off[k], i, j, C, f[k][i]);
            } else {
#pragma unroll
              for (int e = 0; e < P; ++e) f[k][i][e] = 0ull;
            }
#pragma unroll
            for (int e = 0; e < P; ++e) sum = fadd2(sum, f[k][i][e]);
          }
          mu[k] = ln_pair_sum(sum);
        }
#pragma unroll
        for (int k = 0; k < RR; ++k) mu[k] = ln_lane_sum<L>(mu[k]) * inv_c;
#pragma unroll
        for (int k = 0; k < RR; ++k) {
          uint64_t sq = 0ull;
#pragma unroll
          for (int i = 0; i < NV; ++i) {
            if (ln_column<V, L>(i, j, 0, 0) >= C) continue;
            // an element beyond C stays zero
            const uint64_t neg =
                pk2(-mu[k], V == 1 && ln_column<V, L>(i, j, 0, 1) >= C ? 0.f : -mu[k]);
#pragma unroll
            for (int e = 0; e < P; ++e) {
              f[k][i][e] = fadd2(f[k][i][e], neg);
              sq = ffma2(f[k][i][e], f[k][i][e], sq);
            }
          }
          rs[k] = ln_pair_sum(sq);
        }
#pragma unroll
        for (int k = 0; k < RR; ++k) rs[k] = rsqrtf(ln_lane_sum<L>(rs[k]) * inv_c + p.eps);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          if (ln_column<V, L>(i, j, 0, 0) >= C) continue;
          uint64_t g[P], bt[P];
          ln_weight_get<V, L>(s_gamma, i, j, C, g);
          ln_weight_get<V, L>(s_beta, i, j, C, bt);
#pragma unroll
          for (int k = 0; k < RR; ++k) {
#pragma unroll
            for (int e = 0; e < P; ++e)
              f[k][i][e] = ffma2(fmul2(f[k][i][e], ln_both(rs[k])), g[e], bt[e]);
            if (in_row[k]) LP::put(x0 + off[k], i, j, C, f[k][i]);
          }
        }
#pragma unroll
        for (int k = 0; k < RR; ++k) {
          const size_t row = static_cast<size_t>(b) * q.rows + r0 + grp + G * k;
          if (j == 0 && in_row[k] && rib_guard(row, p.rows, G_LN_STAT)) {
            if (p.mean) p.mean[row] = mu[k];
            if (p.rstd) p.rstd[row] = rs[k];
          }
        }
      } else {
        uint8_t* d0 = stage(s, 1) + lead;
        float mu[RR], rs[RR], m1[RR], m2[RR];
        uint64_t xc[RR][NV][P], gd[RR][NV][P];   // x - mean, gamma dy
#pragma unroll
        for (int k = 0; k < RR; ++k) {
          mu[k] = __shfl_sync(0xffffffffu, mu_b, (r0 + grp + G * k) & 31);
          rs[k] = __shfl_sync(0xffffffffu, rs_b, (r0 + grp + G * k) & 31);
        }
#pragma unroll
        for (int k = 0; k < RR; ++k) {
          uint64_t s1 = 0ull, s2 = 0ull;
#pragma unroll
          for (int i = 0; i < NV; ++i) {
            if (!in_row[k] || ln_column<V, L>(i, j, 0, 0) >= C) continue;
            uint64_t d[P], g[P];
            LP::get(x0 + off[k], i, j, C, xc[k][i]);
            LP::get(d0 + off[k], i, j, C, d);   // zero beyond C, so its terms vanish
            ln_weight_get<V, L>(s_gamma, i, j, C, g);
#pragma unroll
            for (int e = 0; e < P; ++e) {
              xc[k][i][e] = fadd2(xc[k][i][e], ln_both(-mu[k]));
              gd[k][i][e] = fmul2(d[e], g[e]);
              const uint64_t xh = fmul2(xc[k][i][e], ln_both(rs[k]));
              sg[i][e] = ffma2(d[e], xh, sg[i][e]);
              sb[i][e] = fadd2(sb[i][e], d[e]);
              s1 = fadd2(s1, gd[k][i][e]);
              s2 = ffma2(gd[k][i][e], xh, s2);
            }
          }
          m1[k] = ln_pair_sum(s1);
          m2[k] = ln_pair_sum(s2);
        }
#pragma unroll
        for (int k = 0; k < RR; ++k) {
          m1[k] = ln_lane_sum<L>(m1[k]) * inv_c;
          m2[k] = ln_lane_sum<L>(m2[k]) * inv_c;
        }
#pragma unroll
        for (int k = 0; k < RR; ++k) {
          // dx = r (g - m1 - (r m2) (x - mean)) + dres: r m2, not r^2 m2, which is beyond
          // fp32 for rows of spread below 1e-19
          const uint64_t kg = ln_both(rs[k]), kx = ln_both(-rs[k] * m2[k]), k1 = ln_both(-m1[k]);
#pragma unroll
          for (int i = 0; i < NV; ++i) {
            if (!in_row[k] || ln_column<V, L>(i, j, 0, 0) >= C) continue;
            uint64_t a[P];
            if (arrays == 3) {
              LP::get(stage(s, 2) + lead + off[k], i, j, C, a);
            } else {
#pragma unroll
              for (int e = 0; e < P; ++e) a[e] = 0ull;
            }
#pragma unroll
            for (int e = 0; e < P; ++e)
              a[e] = ffma2(kg, ffma2(kx, xc[k][i][e], fadd2(gd[k][i][e], k1)), a[e]);
            LP::put(d0 + off[k], i, j, C, a);
          }
        }
      }
    }
    fence_proxy_async_smem();
    __syncwarp();
    {
      const uint8_t* res = stage(s, BWD ? 1 : 0);   // lies there as byte at(b) - lead does
      const uint32_t bytes = rows * row_bytes;
      uint32_t head = 0, whole = bytes;   // bytes before the first 16-byte address; in whole 16s
      if constexpr (V == 1) {
        head = min((16u - lead) & 15u, bytes);
        whole = (bytes - head) & ~15u;
        const uint32_t edge = lane < 8 ? lane * ES : head + whole + (lane - 8) * ES;
        if ((lane < 8 ? edge < head : lane < 16 && edge < bytes) &&
            rib_guard(at(b) + edge, all_bytes, G_LN_OUT))
          *reinterpret_cast<T*>(out + at(b) + edge) = *reinterpret_cast<const T*>(res + lead + edge);
      }
      if (lane == 0) {
        if (whole) bulk_store(out + at(b) + head, res + lead + head, whole);
        tma_store_commit();
        // the stage that the next copies go to, that of the block before this
        // one, has been read
        bulk_store_wait_read_one();
      }
      __syncwarp();
    }
    if (ahead < blocks) {
      load(ahead, s_load);
      ++loaded;
      ahead += step;
      if (++s_load == q.stages) s_load = 0;
    }
    if (++s == q.stages) {
      s = 0;
      ph ^= 1;
    }
  }
  if (!ok && lane == 0) {   // copies in flight land before the CTA exits
    volatile int no_abort = 0;
    for (int i = n; i < loaded; ++i)
      mbar_wait(&full[i % q.stages], (i / q.stages) & 1, &no_abort, 200000000ull, SITE_LN);
  }
  if (lane == 0) tma_store_wait_all();
  if constexpr (BWD) {
    if (!p.part) return;
    // sum over the rows' lane groups, then over the warps in order
    __syncthreads();   // every warp is done with its stages
    float* sums = reinterpret_cast<float*>(ln_smem + w_bytes);   // [warps][2][C]
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < P; ++e) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float g = h ? hi2(sg[i][e]) : lo2(sg[i][e]), t = h ? hi2(sb[i][e]) : lo2(sb[i][e]);
#pragma unroll
          for (int m = L; m < 32; m <<= 1) {
            g += __shfl_xor_sync(0xffffffffu, g, m);
            t += __shfl_xor_sync(0xffffffffu, t, m);
          }
          const int c = ln_column<V, L>(i, j, e, h);
          if (grp == 0 && c < C) {
            sums[(2 * warp) * C + c] = g;
            sums[(2 * warp + 1) * C + c] = t;
          }
        }
      }
    __syncthreads();
    const size_t part_0 = static_cast<size_t>(blockIdx.x) * 2 * C;
    for (int c = threadIdx.x; c < 2 * C; c += blockDim.x) {
      float v = 0.f;
      for (int w = 0; w < q.warps; ++w) v += sums[2 * w * C + c];
      if (rib_guard(part_0 + c, static_cast<size_t>(gridDim.x) * 2 * C, G_LN_PART))
        p.part[part_0 + c] = v;
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
  pdl_wait();
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
