// few_rows.cuh -- projections of up to eight rows (single tokens), forward.
//
//   linear   y = act(x W^T + bias) + residual
//   gated    h = act(x Wg^T + bg) (x Wu^T + bu)
//
// The gated form is the first half of the feed-forward block; its h goes to the
// second product in fp32, since no tensor core wants it in bf16 here and it is
// read from L2 (two rows of 16 channels, 1512 hidden: error 2.7e-3 with h in bf16).
//
// With so few rows a product is one read of the weights, and a tensor-core
// tile of 128 rows would spend its time on tile set-up: here a warp takes two
// weight rows (the gate's and the other projection's of one hidden channel),
// its lanes read them in 16-byte pieces, 512 bytes a warp at a time, and
// keep fp32 sums for every row of x, which the whole grid reads from L1 / L2.
// The lanes' sums are added in a fixed tree.
#pragma once

#include "gemm.cuh"

namespace rib {

constexpr int kFewRows = 8;
constexpr int kFewThreads = 128;
constexpr int G_FEW_W = 177, G_FEW_X = 178, G_FEW_OUT = 179;

struct FewParams {
  const void* x;              // bf16, or fp32 (X32)
  const __nv_bfloat16 *w, *residual;
  const float* bias;
  __nv_bfloat16* pre;
  void* y;                    // bf16, or fp32 (GATED)
  int rows, K, N;
};

__device__ __forceinline__ void few_unpack(const uint4& r, float (&f)[8]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    f[2 * e] = __uint_as_float(w[e] << 16);
    f[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
  }
}

// Eight elements of x from element `at`
template <bool X32>
__device__ __forceinline__ void few_load(const void* x, size_t at, float (&f)[8]) {
  if constexpr (X32) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(x) + at);
    const float4 a = p[0], b = p[1];
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  } else {
    few_unpack(*reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(x) + at), f);
  }
}

// R: rows of x held (the first p.rows of them are real).
// grid ceil(outputs / (2 or 1 per warp) / 4), block kFewThreads.
template <int R, int ACT, bool GATED, bool X32>
__global__ void __launch_bounds__(kFewThreads) few_rows_kernel(const FewParams p) {
  constexpr int U = R <= 2 ? 4 : 2;   // 16-byte pieces of each weight row in flight
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int job = blockIdx.x * (kFewThreads / 32) + (threadIdx.x >> 5);
  const int n0 = GATED ? job : 2 * job;
  if (n0 >= p.N) return;
  const int n1 = GATED ? p.N + job : min(n0 + 1, p.N - 1);
  const size_t w_n = static_cast<size_t>(GATED ? 2 : 1) * p.N * p.K;
  const size_t x_n = static_cast<size_t>(p.rows) * p.K;
  const size_t w0 = static_cast<size_t>(n0) * p.K, w1 = static_cast<size_t>(n1) * p.K;
  float acc[2][R];
#pragma unroll
  for (int r = 0; r < R; ++r) acc[0][r] = acc[1][r] = 0.f;
  for (int k0 = 8 * lane; k0 < p.K; k0 += 256 * U) {
    uint4 a[U], b[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = k0 + 256 * u;
      const bool in = k < p.K && rib_guard(w1 + k + 7, w_n, G_FEW_W);
      a[u] = in ? *reinterpret_cast<const uint4*>(p.w + w0 + k) : make_uint4(0, 0, 0, 0);
      b[u] = in ? *reinterpret_cast<const uint4*>(p.w + w1 + k) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = k0 + 256 * u;
      if (k >= p.K) break;
      float fa[8], fb[8];
      few_unpack(a[u], fa);
      few_unpack(b[u], fb);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const size_t at = static_cast<size_t>(r) * p.K + k;
        if (r >= p.rows || !rib_guard(at + 7, x_n, G_FEW_X)) continue;
        float fx[8];
        few_load<X32>(p.x, at, fx);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          acc[0][r] = fmaf(fa[e], fx[e], acc[0][r]);
          acc[1][r] = fmaf(fb[e], fx[e], acc[1][r]);
        }
      }
    }
  }
  // after the tree every lane holds every sum; lane l writes row l % R of
  // output l / R
  float mine = 0.f, other = 0.f;
#pragma unroll
  for (int c = 0; c < 2; ++c)
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float v = acc[c][r];
#pragma unroll
      for (int m = 16; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
      if (GATED) {
        if (lane == r) (c ? other : mine) = v;
      } else if (lane == c * R + r) {
        mine = v;
      }
    }
  const int row = GATED ? lane : lane % R, n = GATED ? n0 : n0 + lane / R;
  if (lane >= (GATED ? R : 2 * R) || row >= p.rows || n >= p.N) return;
  const size_t at = static_cast<size_t>(row) * p.N + n;
  if (!rib_guard(at, static_cast<size_t>(p.rows) * p.N, G_FEW_OUT)) return;
  const float z = mine + (p.bias ? p.bias[n] : 0.f);
  float v, slope;
  act_both<ACT>(z, v, slope);
  if constexpr (GATED) {
    static_cast<float*>(p.y)[at] = v * (other + (p.bias ? p.bias[p.N + n] : 0.f));
  } else {
    if (p.pre) p.pre[at] = __float2bfloat16_rn(z);
    if (p.residual) v += __bfloat162float(p.residual[at]);
    static_cast<__nv_bfloat16*>(p.y)[at] = __float2bfloat16_rn(v);
  }
}

}  // namespace rib
