// gemm.cuh -- matrix products of the layer's projections on tcgen05 tensor
// cores, bf16 operands and fp32 accumulation, with the work around each
// product in its epilogue.
//
//   kLinear   z = x W^T + b,  y = act(z) + residual   (x [M][K], W [N][K])
//   kDx       y = x W + residual                       (x [M][K], W [K][N])
//   kGated    y = act(x Wg^T + bg) (x Wu^T + bu)       (W [2][N][K])
//   dw_kernel dW = dz^T x, db = sum_rows dz            (dz [R][N], x [R][K])
//
// gemm_kernel is persistent and warp-specialised: warp 16 feeds a ring of
// 64-deep operand tiles by TMA, warp 17 issues the MMAs of 128 x bn tiles
// into one of two accumulators in tensor memory, warps 0-15 are the epilogue
// of the other one.  Operand tiles are rows of 128 bytes in the 128-byte
// swizzle, the layout the tensor core reads without bank conflicts; rows and
// channels outside the matrices are the TMA's zero fill, and outputs outside
// are clipped by the TMA store, so any M and any N, K that are multiples of
// 8 (a 16-byte row pitch) run without a special case.
//
// What bounds the products, and what they take (x and weights in L2 at the small
// sizes):
//   147456 x 192 -> 576         42 us, 226 MB: HBM
//   147456 x 768 -> 192 (dx)    51 us, 283 MB: HBM
//   8192 x 4096 -> 4096        172 us, 1.60 PFLOP/s: tensor cores
//   5003 x 1032 -> 2056         25 us, with gelu and a residual 30: a dozen
//     microseconds of set-up, fill and last epilogue, then the tensor cores
//     (rows of 2064 bytes cost four of them: their 128-byte pieces straddle lines)
//   8192 x 1024 -> 2 x 2816, gated, gelu  68 us, 1.39 PFLOP/s: tensor cores
#pragma once

#include "layer_norm.cuh"   // pdl_wait
#include "ptx.cuh"

namespace rib {

constexpr int SITE_GEMM = 50, SITE_DW = 51, SITE_FFN = 52;
constexpr int G_GEMM_BIAS = 171, G_DW_PART = 172, G_DW_RED = 173,
              G_DZ_IN = 174, G_DZ_OUT = 175, G_FFN_PART = 176;

enum GemmMode { kLinear = 0, kDx = 1, kGated = 2 };
enum ActKind { kActNone = 0, kActGelu = 1, kActSilu = 2 };

// ---------------------------------------------------------------- 2-D / 3-D TMA
__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* map, uint64_t* bar,
                                            int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1)
      : "memory");
}
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, const void* src, int c0,
                                             int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
          reinterpret_cast<uint64_t>(map)),
      "r"(smem_u32(src)), "r"(c0), "r"(c1)
      : "memory");
}
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, const void* src, int c0,
                                             int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
          reinterpret_cast<uint64_t>(map)),
      "r"(smem_u32(src)), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}

// The warp's number, from lane 0: the compiler then knows that branches on it
// are taken by whole warps and keeps what they compute in uniform registers,
// where the tensor core's descriptors have to be.
__device__ __forceinline__ int warp_index() {
  return __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);
}

// Behind the last barrier of a CTA whose waits ran out: a load issued by a
// producer that had already left could still be on its way into the CTA's
// shared memory, so it stays for far longer than a load takes.
__device__ __forceinline__ void settle(volatile int* aborted) {
  if (!*aborted) return;
  for (const uint64_t t0 = globaltimer_ns(); globaltimer_ns() - t0 < 2000000ull;) {
  }
}

// ---------------------------------------------------------------- CTA pairs
// Two CTAs of a cluster work as one 256-row tile (cta_group::2): each holds
// its 128 rows of A and of the accumulator and half of B; CTA 0 issues the
// MMAs, which read both shared memories.
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// Address of CTA `rank`'s copy of a shared variable, for remote arrivals.
__device__ __forceinline__ uint32_t cluster_addr(const void* p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
// An arrival on a barrier of the other CTA that hands over tensor memory, and
// nothing else: what it orders are tensor-memory reads and writes, which the
// tcgen05 fence before it and the one after the wait order, so CTA scope will do.
// It does not order shared memory for the other CTA: that takes a release and an
// acquire at cluster scope, and the release waits for all earlier stores, about
// 2400 cycles.
__device__ __forceinline__ void mbar_arrive_remote(uint32_t addr) {
  asm volatile("mbarrier.arrive.release.cta.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}
// A load into this CTA's shared memory that reports to `bar`, a barrier of
// either CTA of the pair.
__device__ __forceinline__ void tma_load_2d_pair(void* dst, const CUtensorMap* map, uint32_t bar,
                                                 int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".cta_group::2 [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1)
      : "memory");
}
template <int CG>
__device__ __forceinline__ void pair_tmem_alloc(uint32_t* dst, uint32_t cols) {
  if constexpr (CG == 1) {
    tmem_alloc(dst, cols);
    tmem_relinquish();
  } else {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(dst)),
                 "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
}
template <int CG>
__device__ __forceinline__ void pair_tmem_dealloc(uint32_t addr, uint32_t cols) {
  if constexpr (CG == 1)
    tmem_dealloc(addr, cols);
  else
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols)
                 : "memory");
}
template <int CG>
__device__ __forceinline__ void pair_umma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                          uint32_t accumulate) {
  if constexpr (CG == 1)
    umma_ss_elect(d, a, b, idesc, accumulate);
  else
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Four MMAs D (+)= A_k B_k, the descriptors advanced by a_step and b_step (units
// of 16 bytes), from one election: `first_acc` = 0 makes the first overwrite D.
// The issuing warp is a serial resource of these kernels: with an election and
// a wait per MMA and k-step it took about 580 cycles for the 4 x 96 of a
// k-step of 192 columns.
#define RIB_CHAIN4(cg)                                                        \
  asm volatile(                                                               \
      "{\n\t.reg .pred p, e, t;\n\t.reg .b64 a, b, sa, sb;\n\t"             \
      "setp.ne.b32 p, %6, 0;\n\t"                                            \
      "setp.eq.b32 t, %5, %5;\n\t"                                           \
      "cvt.u64.u32 sa, %2;\n\t cvt.u64.u32 sb, %4;\n\t"                     \
      "elect.sync _|e, 0xffffffff;\n\t"                                      \
      "@e tcgen05.mma.cta_group::" cg ".kind::f16 [%0], %1, %3, %5, p;\n\t"  \
      "add.s64 a, %1, sa;\n\t add.s64 b, %3, sb;\n\t"                       \
      "@e tcgen05.mma.cta_group::" cg ".kind::f16 [%0], a, b, %5, t;\n\t"    \
      "add.s64 a, a, sa;\n\t add.s64 b, b, sb;\n\t"                         \
      "@e tcgen05.mma.cta_group::" cg ".kind::f16 [%0], a, b, %5, t;\n\t"    \
      "add.s64 a, a, sa;\n\t add.s64 b, b, sb;\n\t"                         \
      "@e tcgen05.mma.cta_group::" cg ".kind::f16 [%0], a, b, %5, t;\n\t}" ::"r"(d), \
      "l"(a), "r"(a_step), "l"(b), "r"(b_step), "r"(idesc), "r"(first_acc)    \
      : "memory")
template <int CG>
__device__ __forceinline__ void pair_umma4(uint32_t d, uint64_t a, uint32_t a_step, uint64_t b,
                                           uint32_t b_step, uint32_t idesc, uint32_t first_acc) {
  if constexpr (CG == 1)
    RIB_CHAIN4("1");
  else
    RIB_CHAIN4("2");
}
#undef RIB_CHAIN4
// `steps` (1 .. 4) of them
template <int CG>
__device__ __forceinline__ void pair_umma_steps(int steps, uint32_t d, uint64_t a, uint32_t a_step,
                                                uint64_t b, uint32_t b_step, uint32_t idesc,
                                                uint32_t first_acc) {
  if (steps == 4) {
    pair_umma4<CG>(d, a, a_step, b, b_step, idesc, first_acc);
  } else {
    for (int s = 0; s < steps; ++s)
      pair_umma<CG>(d, a + static_cast<uint64_t>(a_step) * s, b + static_cast<uint64_t>(b_step) * s,
                    idesc, s > 0 ? 1u : first_acc);
  }
}

// Four MMAs D (+)= A_k B_k of a pair with A in tensor memory, each CTA's 128 rows
// in its own lanes: 16 bf16 channels a step in 8 columns, 16 columns from one
// step to the next; B's descriptor advances by b_step.  One election.
__device__ __forceinline__ void pair_umma_ts4(uint32_t d, uint32_t a, uint64_t b, uint32_t b_step,
                                              uint32_t idesc, uint32_t first_acc) {
  asm volatile(
      "{\n\t.reg .pred p, e, t;\n\t.reg .b64 b, sb;\n\t.reg .b32 a;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "setp.eq.b32 t, %4, %4;\n\t"
      "cvt.u64.u32 sb, %3;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %4, p;\n\t"
      "add.s32 a, %1, 16;\n\t add.s64 b, %2, sb;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], [a], b, %4, t;\n\t"
      "add.s32 a, a, 16;\n\t add.s64 b, b, sb;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], [a], b, %4, t;\n\t"
      "add.s32 a, a, 16;\n\t add.s64 b, b, sb;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], [a], b, %4, t;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(b_step), "r"(idesc), "r"(first_acc)
      : "memory");
}
// `steps` (1 .. 4) of them
__device__ __forceinline__ void pair_umma_ts_steps(int steps, uint32_t d, uint32_t a, uint64_t b,
                                                   uint32_t b_step, uint32_t idesc,
                                                   uint32_t first_acc) {
  if (steps == 4) {
    pair_umma_ts4(d, a, b, b_step, idesc, first_acc);
  } else {
    for (int s = 0; s < steps; ++s)
      asm volatile(
          "{\n\t.reg .pred p, e;\n\t"
          "setp.ne.b32 p, %4, 0;\n\t"
          "elect.sync _|e, 0xffffffff;\n\t"
          "@e tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
          "r"(a + 16 * s), "l"(b + static_cast<uint64_t>(b_step) * s), "r"(idesc),
          "r"(s > 0 ? 1u : first_acc)
          : "memory");
  }
}

// Waits of the issuing warp on a ring of barriers.  The next barrier is tested
// before the MMAs of the present one are issued, so its answer is there when
// it is asked for (test_wait: try_wait may sleep until the phase completes,
// with the MMAs not yet issued behind it).
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
struct RingWait {
  bool ready = false;
  __device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, volatile int* ab,
                                       uint64_t lim, int site) {
    return __all_sync(0xffffffffu, ready) || warp_wait(bar, parity, ab, lim, site);
  }
  __device__ __forceinline__ void peek(uint64_t* bar, uint32_t parity) {
    ready = mbar_test(bar, parity);
  }
};

// Arrives on `bar` (in both CTAs of a pair) when the MMAs issued so far are done.
template <int CG>
__device__ __forceinline__ void pair_commit(uint64_t* bar) {
  if constexpr (CG == 1)
    umma_commit_elect(bar);
  else
    asm volatile(
        "{\n\t.reg .pred e;\n\t.reg .b16 m;\n\t"
        "mov.b16 m, 3;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster"
        ".b64 [%0], m;\n\t}" ::"r"(smem_u32(bar))
        : "memory");
}

// ---------------------------------------------------------------- activations
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

constexpr float kLog2e = 1.4426950408889634f;

// Forward values, two elements (or four) at a time: the epilogue's issue slots
// and the 16 lanes of the special-function unit bound the products of few
// channels, so the work goes to packed fp32 and as few special functions as
// the accuracy allows.
//
// gelu(z) = z Phi(z) = max(z, 0) - t Q, t = |z|, Q = erfc(t / sqrt 2) / 2 =
// e^(-t^2/2) R(t), and R = k P(k) with k = 1 / (1 + c t) and a polynomial P
// (fit_gelu_poly.py).  The fit is relative, 4.6e-6, and holds as far as Q is a
// normal number: for z < 0 the result is -t Q itself, and its bf16 step is
// relative.  (A polynomial in t on [0, 6] with absolute bounds left up to 4 % of
// that result there.)  One reciprocal serves four elements, 1/a = b c d / (a b c
// d), with t capped at 16, where the exponential is 0, so that the factors lie
// within [1, 6] and an infinite z gives no NaN.
__device__ __forceinline__ void gelu_quad(uint64_t& z01, uint64_t& z23) {
  const float z[4] = {lo2(z01), hi2(z01), lo2(z23), hi2(z23)};
  float m[4];   // -t
#pragma unroll
  for (int i = 0; i < 4; ++i) m[i] = fmaxf(-fabsf(z[i]), -16.f);
  const uint64_t m01 = pk2(m[0], m[1]), m23 = pk2(m[2], m[3]);
  const uint64_t c = pk2(-0.31f, -0.31f), one = pk2(1.f, 1.f);
  const uint64_t a01 = ffma2(m01, c, one), a23 = ffma2(m23, c, one);
  const float p01 = lo2(a01) * hi2(a01), p23 = lo2(a23) * hi2(a23);
  const float r = rcp_approx(p01 * p23);
  const float r01 = r * p23, r23 = r * p01;   // 1 / (a0 a1), 1 / (a2 a3)
  const uint64_t k01 = fmul2(pk2(hi2(a01), lo2(a01)), pk2(r01, r01));
  const uint64_t k23 = fmul2(pk2(hi2(a23), lo2(a23)), pk2(r23, r23));
  const uint64_t h = pk2(-0.5f * kLog2e, -0.5f * kLog2e);
  const uint64_t x01 = fmul2(fmul2(z01, h), z01), x23 = fmul2(fmul2(z23, h), z23);
  const uint64_t e01 = pk2(ex2_approx(lo2(x01)), ex2_approx(hi2(x01)));
  const uint64_t e23 = pk2(ex2_approx(lo2(x23)), ex2_approx(hi2(x23)));
  auto poly = [](uint64_t k) {
    uint64_t p = ffma2(k, pk2(-0.0739237592f, -0.0739237592f), pk2(0.180433989f, 0.180433989f));
    p = ffma2(p, k, pk2(0.0157634765f, 0.0157634765f));
    p = ffma2(p, k, pk2(0.133419752f, 0.133419752f));
    p = ffma2(p, k, pk2(0.120443746f, 0.120443746f));
    p = ffma2(p, k, pk2(0.123860478f, 0.123860478f));
    return fmul2(p, k);
  };
  z01 = ffma2(fmul2(poly(k01), e01), m01, pk2(fmaxf(z[0], 0.f), fmaxf(z[1], 0.f)));
  z23 = ffma2(fmul2(poly(k23), e23), m23, pk2(fmaxf(z[2], 0.f), fmaxf(z[3], 0.f)));
}

// silu(z) = z / (1 + e^-z) = max(z, 0) - |z| f with E = e^-|z| <= 1 and f = E / (1
// + E), exact in both tails; the four reciprocals come from one: 1/a = b c d /
// (a b c d), every factor within [1, 2].  (-|z| is bounded so that a NaN of one
// element stays out of the others; its own comes back through the maximum,
// which keeps it.)
__device__ __forceinline__ float max0_nan(float x) {
  float y;
  asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void silu_quad(uint64_t& z01, uint64_t& z23) {
  const float z[4] = {lo2(z01), hi2(z01), lo2(z23), hi2(z23)};
  float m[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) m[i] = fmaxf(-fabsf(z[i]), -103.f);
  const uint64_t k = pk2(kLog2e, kLog2e), one = pk2(1.f, 1.f);
  const uint64_t m01 = pk2(m[0], m[1]), m23 = pk2(m[2], m[3]);
  const uint64_t x01 = fmul2(m01, k), x23 = fmul2(m23, k);
  const float e0 = ex2_approx(lo2(x01)), e1 = ex2_approx(hi2(x01));
  const float e2 = ex2_approx(lo2(x23)), e3 = ex2_approx(hi2(x23));
  const uint64_t a01 = fadd2(pk2(e0, e1), one), a23 = fadd2(pk2(e2, e3), one);
  const float p01 = lo2(a01) * hi2(a01), p23 = lo2(a23) * hi2(a23);
  const float r = rcp_approx(p01 * p23);
  const float r01 = r * p23, r23 = r * p01;   // 1 / (a0 a1), 1 / (a2 a3)
  const uint64_t f01 = fmul2(pk2(e0 * hi2(a01), e1 * lo2(a01)), pk2(r01, r01));
  const uint64_t f23 = fmul2(pk2(e2 * hi2(a23), e3 * lo2(a23)), pk2(r23, r23));
  z01 = ffma2(m01, f01, pk2(max0_nan(z[0]), max0_nan(z[1])));
  z23 = ffma2(m23, f23, pk2(max0_nan(z[2]), max0_nan(z[3])));
}

template <int ACT>
__device__ __forceinline__ void act_quad(uint64_t& z01, uint64_t& z23) {
  if constexpr (ACT == kActGelu) {
    gelu_quad(z01, z23);
  } else if constexpr (ACT == kActSilu) {
    silu_quad(z01, z23);
  }
}

// act(z) and act'(z) for the backward, to fp32 accuracy (the bias gradients
// are fp32 sums of what is formed from them), and the value for few rows.
// gelu: as above with a longer polynomial, Q to 4e-7 of itself; the slope is Phi +
// z phi, from the same exponential.
template <int ACT>
__device__ __forceinline__ void act_both(float z, float& a, float& da) {
  if constexpr (ACT == kActGelu) {
    const float cap = fminf(fmaxf(z, -16.f), 16.f), t = fabsf(cap);
    const float k = rcp_approx(fmaf(t, 0.3f, 1.f));
    const float e = ex2_approx(z * z * (-0.5f * kLog2e));
    float p = fmaf(k, 0.0357484072f, -0.157488391f);
    p = fmaf(p, k, 0.206804186f);
    p = fmaf(p, k, -0.0540565774f);
    p = fmaf(p, k, 0.128734082f);
    p = fmaf(p, k, 0.0998697057f);
    p = fmaf(p, k, 0.12075948f);
    p = fmaf(p, k, 0.11962904f);
    const float q = p * k * e;
    a = fmaf(-t, q, fmaxf(z, 0.f));
    da = fmaf(cap, 0.3989422804f * e, z > 0.f ? 1.f - q : q);
  } else if constexpr (ACT == kActSilu) {
    // z is bounded in its products with what vanishes there, so that an infinite
    // one gives the limits (0 and 0, or infinity and 1), as silu_quad does
    const float s = rcp_approx(1.f + ex2_approx(-kLog2e * z));
    a = fmaxf(z, -1e4f) * s;
    da = fmaf(fminf(a, 1e4f), 1.f - s, s);
  } else {
    a = z;
    da = 1.f;
  }
}

// 16 columns' bias (fp32, from column `col` of n), zero outside or without one
__device__ __forceinline__ void bias16(const float* bias, int col, int n, float4 (&b)[4]) {
  if (bias && col + 16 <= n) {
#pragma unroll
    for (int e = 0; e < 4; ++e) b[e] = reinterpret_cast<const float4*>(bias + col)[e];
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      b[e] = bias && col + 4 * e < n &&
                     rib_guard(static_cast<size_t>(col) + 4 * e + 3, n, G_GEMM_BIAS)
                 ? reinterpret_cast<const float4*>(bias + col)[e]
                 : make_float4(0.f, 0.f, 0.f, 0.f);
  }
}

// ---------------------------------------------------------------- the product
constexpr int kGemmThreads = 576;
constexpr int kGemmEpiWarps = 16, kGemmTmaWarp = 16, kGemmMmaWarp = 17;
constexpr uint32_t kGemmATile = 128u * 128u;        // 128 rows x 64 channels
constexpr uint32_t kGemmUnit = 32u * 64u;           // an epilogue unit: 32 rows x 32 bf16 columns
constexpr uint32_t kGemmStaging = kGemmEpiWarps * kGemmUnit;
constexpr int kGemmMaxStages = 10;

struct GemmParams {
  const float* bias;               // [N], or [2][N] for kGated; may be null
  int M, N, K;
  int bn;                          // columns of a B tile in shared memory (64 .. 256)
  int m_tiles, n_tiles;
  int splits;                      // the row tiles of one column tile go to `splits` items
  int k_steps, stages;
  uint32_t a_bytes;                // of a k-step's x tile (rows that are not loaded are not stored)
  int b_resident;                  // the column tile's weights stay in shared memory
  uint64_t wait_limit_ns;
};

struct GemmBars {
  uint64_t full[kGemmMaxStages], empty[kGemmMaxStages];
  uint64_t acc_full[2], acc_free[2], b_full, b_free, drain, res[kGemmEpiWarps];
  uint32_t tmem;
  int abort_flag;
};

// Bytes of one k-step of B in one CTA: bn columns, or half of them in a pair
// (whole 64-column atoms where the columns are the leading dimension).
__host__ __device__ __forceinline__ uint32_t gemm_b_bytes(int mode, int cg, int bn) {
  const int cols = cg == 1 ? bn : mode == kDx ? (bn / 2 + 63) / 64 * 64 : bn / 2;
  return static_cast<uint32_t>(cols) * 128u;
}

__host__ __device__ __forceinline__ size_t gemm_smem_bytes(uint32_t b_bytes, int stages,
                                                           int k_steps, bool resident, bool res) {
  return 1024 + static_cast<size_t>(stages) * (kGemmATile + (resident ? 0 : b_bytes)) +
         (resident ? static_cast<size_t>(k_steps) * b_bytes : 0) +
         (res ? 2 : 1) * kGemmStaging + sizeof(GemmBars);
}

// Columns of y that one tile gives: half of the B tile for kGated (the other
// half is the second projection's).
template <int MODE>
__device__ __forceinline__ int gemm_tile_cols(const GemmParams& p) {
  return MODE == kGated ? p.bn / 2 : p.bn;
}

// MMA columns of the column tile at n0: a last tile narrower than bn takes a
// narrower MMA (16 columns per CTA at a time).
template <int MODE, int CG>
__device__ __forceinline__ int gemm_mma_cols(const GemmParams& p, int n0) {
  constexpr int unit = 16 * CG;
  return MODE == kGated ? p.bn : min(p.bn, (p.N - n0 + unit - 1) / unit * unit);
}

// Loads this CTA's share of the B tile at column n0, k-step k (64 deep), to
// `dst`; `bar` is the barrier that counts it.
template <int MODE, int CG>
__device__ __forceinline__ void gemm_load_b(uint8_t* dst, const CUtensorMap* tm_b, uint64_t* bar,
                                            uint32_t pair_bar, const GemmParams& p, int n0, int k,
                                            uint32_t rank) {
  auto load = [&](uint8_t* d, int c0, int c1) {
    if constexpr (CG == 1)
      tma_load_2d(d, tm_b, bar, c0, c1);
    else
      tma_load_2d_pair(d, tm_b, pair_bar, c0, c1);
  };
  if constexpr (MODE == kGated) {
    if constexpr (CG == 1) {
      load(dst, 64 * k, n0);
      load(dst + p.bn * 64, 64 * k, p.N + n0);
    } else {   // CTA 0 holds the gate's rows, CTA 1 the other projection's
      load(dst, 64 * k, rank * p.N + n0);
    }
  } else {
    const int c0 = n0 + (CG == 2 ? rank * gemm_mma_cols<MODE, CG>(p, n0) / 2 : 0);
    if constexpr (MODE == kLinear) {
      load(dst, 64 * k, c0);
    } else {
      const int chunks = gemm_b_bytes(MODE, CG, p.bn) / 8192;
      for (int c = 0; c < chunks; ++c) load(dst + c * 8192, c0 + 64 * c, 64 * k);
    }
  }
}

// Work item i: column tile i % n_tiles, row tiles (of 128 CG rows) i / n_tiles +
// splits * j.  Items that run at the same time so share their x rows (one read
// from HBM serves all column tiles), and a CTA keeps its column tile's weights.
// CG = 2: the CTA pairs of clusters of two; an MMA of 256 rows reads each
// CTA's half of B once for both, so B's shared-memory reads and its loads from
// L2 halve (the MMA of 128 x 256 alone takes 96 of the 128 bytes per clock of
// shared memory).
// grid CG * min(items, SMs / CG), block kGemmThreads, dynamic smem
// gemm_smem_bytes().
template <int MODE, int ACT, bool RES, bool PRE, int CG>
__global__ void __launch_bounds__(kGemmThreads, 1)
    gemm_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                const __grid_constant__ CUtensorMap tm_y,
                const __grid_constant__ CUtensorMap tm_pre,
                const __grid_constant__ CUtensorMap tm_res, const GemmParams p) {
  extern __shared__ uint8_t gemm_raw[];
  uint8_t* base = gemm_raw + ((1024u - (smem_u32(gemm_raw) & 1023u)) & 1023u);
  const uint32_t b_bytes = gemm_b_bytes(MODE, CG, p.bn);
  const uint32_t stage_bytes = kGemmATile + (p.b_resident ? 0u : b_bytes);
  uint8_t* s_res = base + p.stages * stage_bytes;
  uint8_t* s_stage = s_res + (p.b_resident ? p.k_steps * b_bytes : 0u);
  GemmBars& bb = *reinterpret_cast<GemmBars*>(s_stage + (RES ? 2 : 1) * kGemmStaging);
  volatile int* ab = &bb.abort_flag;
  // the gated epilogue spills with the warp's number uniform (106 us for 101 us
  // at 25600 x 288 x 2 x 1152 and the product after it)
  const int warp = MODE == kGated ? threadIdx.x >> 5 : warp_index(), lane = threadIdx.x & 31;
  const uint32_t rank = CG == 2 ? cluster_rank() : 0u;
  const int worker = blockIdx.x / CG, workers = gridDim.x / CG;
  const int tn = gemm_tile_cols<MODE>(p);
  const int items = p.n_tiles * p.splits;
  const int my_row = 128 * rank;   // of the tile's 128 CG rows
  const uint64_t lim = p.wait_limit_ns;
  if (threadIdx.x == 0) {
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(&bb.full[i], 1);
      mbar_init(&bb.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bb.acc_full[i], 1);
      mbar_init(&bb.acc_free[i], CG * kGemmEpiWarps);
    }
    mbar_init(&bb.b_full, 1);
    mbar_init(&bb.b_free, 1);
    mbar_init(&bb.drain, 1);
    for (int i = 0; i < kGemmEpiWarps; ++i) mbar_init(&bb.res[i], 1);
    bb.abort_flag = 0;
    fence_mbarrier_init();
  }
  if (warp == kGemmTmaWarp && lane == 0) {
    tma_prefetch_desc(&tm_a);
    tma_prefetch_desc(&tm_b);
    tma_prefetch_desc(&tm_y);
  }
  if (CG == 2) cluster_sync();   // the other CTA's barriers are ready too
  if (warp == kGemmMmaWarp) pair_tmem_alloc<CG>(&bb.tmem, 512);
  pdl_wait();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bb.tmem;

  if (warp == kGemmTmaWarp) {
    // ---------------------------------------------------------- TMA producer
    // In a pair both CTAs load their shares; CTA 0's barriers count all bytes.
    if (lane == 0) {
      bool ok = true;
      int q = 0, st = 0, n_item = 0;   // running load number, its stage
      uint32_t ph = 1;                 // parity of the previous use of the stage
      const uint32_t pair_b = CG == 2 ? cluster_addr(&bb.b_full, 0) : 0u;
      for (int it = worker; ok && it < items; it += workers, ++n_item) {
        const int n0 = (it % p.n_tiles) * tn;
        if (p.b_resident) {
          if (n_item > 0 && !(ok = mbar_wait(&bb.b_free, (n_item - 1) & 1, ab, lim, SITE_GEMM)))
            break;
          if (rank == 0) mbar_arrive_expect_tx(&bb.b_full, CG * p.k_steps * b_bytes);
          for (int k = 0; k < p.k_steps; ++k)
            gemm_load_b<MODE, CG>(s_res + k * b_bytes, &tm_b, &bb.b_full, pair_b, p, n0, k, rank);
        }
        for (int m = it / p.n_tiles; ok && m < p.m_tiles; m += p.splits)
          for (int k = 0; k < p.k_steps; ++k) {
            if (q >= p.stages && !(ok = mbar_wait(&bb.empty[st], ph, ab, lim, SITE_GEMM))) break;
            uint8_t* sa = base + st * stage_bytes;
            if (rank == 0)
              mbar_arrive_expect_tx(&bb.full[st], CG * (p.a_bytes + stage_bytes - kGemmATile));
            uint32_t pair_f = 0u;
            if constexpr (CG == 1) {
              tma_load_2d(sa, &tm_a, &bb.full[st], 64 * k, 128 * m);
            } else {
              pair_f = cluster_addr(&bb.full[st], 0);
              tma_load_2d_pair(sa, &tm_a, pair_f, 64 * k, 256 * m + my_row);
            }
            if (!p.b_resident)
              gemm_load_b<MODE, CG>(sa + kGemmATile, &tm_b, &bb.full[st], pair_f, p, n0, k, rank);
            ++q;
            if (++st == p.stages) {
              st = 0;
              ph ^= 1;
            }
          }
      }
      if (*ab) {
        // loads still in flight land before the CTA exits (in a pair, CTA 0's
        // barriers see both CTAs' and the CTAs leave together)
        volatile int no_abort = 0;
        if (rank == 0) {
          if (p.b_resident && n_item > 0)
            mbar_wait(&bb.b_full, (n_item - 1) & 1, &no_abort, 200000000ull, SITE_GEMM);
          for (int i = max(0, q - p.stages); i < q; ++i)
            mbar_wait(&bb.full[i % p.stages], (i / p.stages) & 1, &no_abort, 200000000ull,
                      SITE_GEMM);
        } else {
          // CTA 0 may have stopped counting: far longer than a load takes
          for (const uint64_t t0 = globaltimer_ns(); globaltimer_ns() - t0 < 2000000ull;) {
          }
        }
      }
    }
  } else if (warp == kGemmMmaWarp) {
    // ---------------------------------------------------------- MMA issue
    if (rank == 0) {
      const int last_steps = (p.K - 64 * (p.k_steps - 1) + 15) / 16;
      bool ok = true;
      int st = 0, t = 0, n_item = 0;
      uint32_t ph = 0;
      RingWait ring;
      for (int it = worker; ok && it < items; it += workers, ++n_item) {
        const int n0 = (it % p.n_tiles) * tn;
        const uint32_t idesc =
            make_idesc_bf16(128 * CG, gemm_mma_cols<MODE, CG>(p, n0), false, MODE == kDx);
        if (p.b_resident && !(ok = warp_wait(&bb.b_full, n_item & 1, ab, lim, SITE_GEMM))) break;
        for (int m = it / p.n_tiles; ok && m < p.m_tiles; m += p.splits, ++t) {
          const int a = t & 1;
          if (t >= 2 && !(ok = warp_wait(&bb.acc_free[a], ((t >> 1) - 1) & 1, ab, lim, SITE_GEMM)))
            break;
          for (int k = 0; k < p.k_steps; ++k) {
            if (!(ok = ring.wait(&bb.full[st], ph, ab, lim, SITE_GEMM))) break;
            tc_fence_after();
            const uint32_t sa = smem_u32(base + st * stage_bytes);
            const uint32_t sb = p.b_resident ? smem_u32(s_res + k * b_bytes) : sa + kGemmATile;
            // K-major: a K = 16 step is 32 bytes along the rows; MN-major
            // (kDx): it is 16 rows of 128 bytes, 64-column chunks 8 KB apart
            const uint64_t ad = make_sdesc(sa, 16, 1024, kLayoutSW128);
            const uint64_t bd = MODE == kDx ? make_sdesc(sb, 8192, 1024, kLayoutSW128)
                                            : make_sdesc(sb, 16, 1024, kLayoutSW128);
            uint64_t* done = &bb.empty[st];
            if (++st == p.stages) {
              st = 0;
              ph ^= 1;
            }
            ring.peek(&bb.full[st], ph);
            pair_umma_steps<CG>(k + 1 == p.k_steps ? last_steps : 4, tmem + 256 * a, ad, 2, bd,
                                MODE == kDx ? 128 : 2, idesc, k > 0 ? 1u : 0u);
            pair_commit<CG>(done);
          }
          if (ok) pair_commit<CG>(&bb.acc_full[a]);
        }
        if (ok && p.b_resident) pair_commit<CG>(&bb.b_free);
      }
      // every MMA issued above completes before the tensor memory is freed
      pair_commit<CG>(&bb.drain);
      volatile int no_abort = 0;
      mbar_wait(&bb.drain, 0, &no_abort, 200000000ull, SITE_GEMM);
    }
  } else {
    // ---------------------------------------------------------- epilogue
    // A tile's columns fall into units of 32; warp w takes TMEM lane quarter
    // w % 4 (rows 32 (w % 4) .. of the tile) of the units that come to its group
    // w / 4 as the groups take turns over all units of all tiles.  Sixteen
    // warps of few registers, because a unit is a chain of latencies (tensor
    // memory, special functions): four warps per scheduler fill each other's
    // gaps.  Outputs leave through the warp's 2 KB of shared memory (rows of
    // 64 bytes, 64-byte swizzle) and a TMA store, the residual comes in the
    // same way, one unit ahead.
    const int quarter = warp & 3, group = warp >> 2;
    uint8_t* sg = s_stage + warp * kGemmUnit;
    uint8_t* sr = sg + kGemmStaging;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    // this lane's 16-byte granule g of its row
    auto cell = [&](uint8_t* base, int g) {
      return reinterpret_cast<uint4*>(base + lane * 64 + ((g ^ ((lane >> 1) & 3)) << 4));
    };
    // the accumulator's columns are read: to the CTA that issues the MMAs
    auto free_acc = [&](int a) {
      if constexpr (CG == 1)
        mbar_arrive(&bb.acc_free[a]);
      else
        mbar_arrive_remote(cluster_addr(&bb.acc_free[a], 0));
    };
    int t = 0;
    int turn = 0;          // group whose turn the tile's first unit is
    uint32_t res_ph = 0;   // parity of the next residual unit
    bool ok = true, res_ahead = false;
    auto load_res = [&](int m, int col) {   // one unit ahead; rows and columns outside are zeros
      if (lane == 0) {
        mbar_arrive_expect_tx(&bb.res[warp], kGemmUnit);
        tma_load_2d(sr, &tm_res, &bb.res[warp], col, 128 * CG * m + my_row + 32 * quarter);
      }
      res_ahead = true;
    };
    for (int it = worker; ok && it < items; it += workers) {
      const int n0 = (it % p.n_tiles) * tn;
      const int units = (min(tn, p.N - n0) + 31) / 32;
      for (int m = it / p.n_tiles; ok && m < p.m_tiles; m += p.splits, ++t) {
        const int a = t & 1;
        const int row0 = 128 * CG * m + my_row + 32 * quarter;
        const int first = (group - turn) & 3;
        turn = (turn + units) & 3;
        // the group's first unit of the next row tile of this item
        const int next_m = m + p.splits, next_first = (group - turn) & 3;
        if (RES && !res_ahead && first < units && row0 < p.M) load_res(m, n0 + 32 * first);
        if (!(ok = warp_wait(&bb.acc_full[a], (t >> 1) & 1, ab, lim, SITE_GEMM))) break;
        tc_fence_after();
        const uint32_t acc = tmem + 256 * a + lane_off;
        for (int u = first; ok && u < units; u += 4) {
          const int col = n0 + 32 * u;
          uint32_t out[16];
          [[maybe_unused]] uint32_t pre[PRE ? 16 : 1];
          if constexpr (RES) {
            if (row0 < p.M) {
              if (!(ok = warp_wait(&bb.res[warp], res_ph, ab, lim, SITE_GEMM))) break;
              res_ph ^= 1;
              res_ahead = false;
            }
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {   // 16 columns at a time
            uint32_t v[16];
            [[maybe_unused]] uint32_t w[16];
            tmem_ld_x16(acc + 32 * u + 16 * h, v);
            if constexpr (MODE == kGated) tmem_ld_x16(acc + tn + 32 * u + 16 * h, w);
            [[maybe_unused]] float4 b[4], c[4];
            if constexpr (MODE != kDx) bias16(p.bias, col + 16 * h, p.N, b);
            if constexpr (MODE == kGated)
              bias16(p.bias ? p.bias + p.N : nullptr, col + 16 * h, p.N, c);
            tmem_wait_ld();
            reg_fence_x16(v);
            if constexpr (MODE == kGated) reg_fence_x16(w);
            if (h == 1 && u + 4 >= units) {   // this warp has read its last columns
              tc_fence_before();
              __syncwarp();
              if (lane == 0) free_acc(a);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              auto f = [](uint32_t x) { return __uint_as_float(x); };
              uint64_t z01 = pk2(f(v[4 * e]), f(v[4 * e + 1]));
              uint64_t z23 = pk2(f(v[4 * e + 2]), f(v[4 * e + 3]));
              if constexpr (MODE != kDx) {
                z01 = fadd2(z01, pk2(b[e].x, b[e].y));
                z23 = fadd2(z23, pk2(b[e].z, b[e].w));
              }
              if constexpr (PRE) {
                pre[8 * h + 2 * e] = pack_bf16x2(lo2(z01), hi2(z01));
                pre[8 * h + 2 * e + 1] = pack_bf16x2(lo2(z23), hi2(z23));
              }
              act_quad<ACT>(z01, z23);
              if constexpr (MODE == kGated) {
                z01 = fmul2(z01, fadd2(pk2(f(w[4 * e]), f(w[4 * e + 1])), pk2(c[e].x, c[e].y)));
                z23 = fmul2(z23, fadd2(pk2(f(w[4 * e + 2]), f(w[4 * e + 3])), pk2(c[e].z, c[e].w)));
              }
              if constexpr (RES) {
                const uint2 r = *(reinterpret_cast<const uint2*>(cell(sr, 2 * h + (e >> 1))) + (e & 1));
                z01 = fadd2(z01, pk2(f(r.x << 16), f(r.x & 0xffff0000u)));
                z23 = fadd2(z23, pk2(f(r.y << 16), f(r.y & 0xffff0000u)));
              }
              out[8 * h + 2 * e] = pack_bf16x2(lo2(z01), hi2(z01));
              out[8 * h + 2 * e + 1] = pack_bf16x2(lo2(z23), hi2(z23));
            }
          }
          if (row0 < p.M) {
            auto put = [&](const uint32_t(&w)[16], const CUtensorMap* map) {
              if (lane == 0) tma_store_wait_read_all();   // the last store has read the buffer
              __syncwarp();
#pragma unroll
              for (int g = 0; g < 4; ++g)
                *cell(sg, g) = make_uint4(w[4 * g], w[4 * g + 1], w[4 * g + 2], w[4 * g + 3]);
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) {
                tma_store_2d(map, sg, col, row0);
                tma_store_commit();
              }
            };
            if constexpr (PRE) put(pre, &tm_pre);
            put(out, &tm_y);
            if constexpr (RES) {   // every lane has read its residual (put's barriers)
              if (u + 4 < units)
                load_res(m, col + 128);
              else if (next_m < p.m_tiles && next_first < units && row0 + 128 * CG * p.splits < p.M)
                load_res(next_m, n0 + 32 * next_first);
            }
          }
        }
        if (first >= units) {   // no unit of this tile for this warp
          tc_fence_before();
          __syncwarp();
          if (lane == 0) free_acc(a);
        }
      }
    }
    if (RES && !ok && res_ahead && lane == 0) {   // a residual load in flight lands first
      volatile int no_abort = 0;
      mbar_wait(&bb.res[warp], res_ph, &no_abort, 200000000ull, SITE_GEMM);
    }
    // the stores are complete before the kernel's work is considered done
    if (lane == 0) tma_store_wait_all();
  }
  tc_fence_before();
  __syncthreads();
  settle(ab);
  // neither CTA of a pair leaves while the other may still read its shared
  // memory or arrive on its barriers
  if (CG == 2) cluster_sync();
  if (warp == kGemmMmaWarp) {
    tc_fence_after();
    pair_tmem_dealloc<CG>(tmem, 512);
  }
}

// ---------------------------------------------------------------- dW, db
// dW[n][k] = sum_r dz[r][n] x[r][k] and db[n] = sum_r dz[r][n]: the rows are
// the contraction, so both operands are MN-major (64 rows of 64 channels are
// one canonical 8 KB atom column).  A CTA takes a tile of up to 256 x 192 of dW
// (accumulators of 128 rows) and a range of the rows; the ranges' partial
// sums go to the workspace and dw_reduce_kernel adds them in order.  db is
// one more column of the product: a block of ones stands behind x's channels
// in each stage, so the sum of the bf16 dz costs 16 of 208 MMA columns and no
// pass over dz.
//
// The tensor core truncates when it adds to its accumulator, so a long chain
// of additions drifts towards zero: 188 of them (3000 rows) left dW with a
// relative error of 3.3e-6.  Every kDwFlush stages (32 additions) the epilogue
// warps therefore move the accumulators into fp32 registers, added to
// nearest, and the next chain starts from zero: 0.6e-6, as a plain fp32 sum,
// for a stall of about a tenth of the MMAs' time, which the loads hide.
//
// Bound by HBM and, at its ends, by latency: 147456 rows of 192 x 768 take 52 us
// (283 MB, 5.4 TB/s) and 8 us of reduction, of 192 x 576 46 us (226 MB), of 520 x
// 1480 with 3001 rows 11 us where the bytes are 1.8.
constexpr int kDwThreads = 384;   // warps 0-7 epilogue, 8 TMA, 9 MMA, two idle
constexpr int kDwBn = 192;
constexpr int kDwFlush = 8;
constexpr uint32_t kDwAtom = 8192;                       // 64 rows x 64 channels
constexpr int kDwMaxStages = 8;
// Registers (setmaxnreg): 256 x 224 + 128 x 56 = 64512 = 384 x 168 at launch.
constexpr int kDwEpiRegs = 224, kDwOtherRegs = 56;

struct DwParams {
  int rows, N, K;
  int a_chunks, b_chunks;          // 64-channel chunks of a tile: dz (2 .. 4), x (1 .. 3)
  int m_tiles, n_tiles, splits, stages;
  int steps, steps_per_split;      // 64-row steps, in all and per split
  int part;                        // tm_part is written: the partials, or with one split an fp32 dW
  __nv_bfloat16* out16;            // one split and a bf16 dW
  float* part_db;                  // [splits][N]; null: no db
  uint64_t wait_limit_ns;
};

struct DwBars {
  uint64_t full[kDwMaxStages], empty[kDwMaxStages], acc_full, acc_free, drain;
  uint32_t tmem;
  int abort_flag;
};

__host__ __device__ __forceinline__ uint32_t dw_stage_bytes(int a_chunks, int b_chunks) {
  return static_cast<uint32_t>(a_chunks + b_chunks + 1) * kDwAtom;   // dz, x, ones
}
__host__ __device__ __forceinline__ size_t dw_smem_bytes(int a_chunks, int b_chunks, int stages) {
  return 1024 + static_cast<size_t>(stages) * dw_stage_bytes(a_chunks, b_chunks) + sizeof(DwBars);
}

// grid m_tiles * n_tiles * splits, block kDwThreads, dynamic smem dw_smem_bytes().
// tm_z: dz [rows][N], tm_x: x [rows][K], boxes of 64 channels x 64 rows; tm_part:
// part [splits][N][K], boxes 32 x 32 x 1; 128-byte swizzle.
__global__ void __launch_bounds__(kDwThreads, 1)
    dw_kernel(const __grid_constant__ CUtensorMap tm_z, const __grid_constant__ CUtensorMap tm_x,
              const __grid_constant__ CUtensorMap tm_part, const DwParams p) {
  extern __shared__ uint8_t dwg_raw[];
  uint8_t* base = dwg_raw + ((1024u - (smem_u32(dwg_raw) & 1023u)) & 1023u);
  const uint32_t stage_bytes = dw_stage_bytes(p.a_chunks, p.b_chunks);
  const uint32_t b_off = p.a_chunks * kDwAtom;
  DwBars& bb = *reinterpret_cast<DwBars*>(base + p.stages * stage_bytes);
  volatile int* ab = &bb.abort_flag;
  const int warp = warp_index(), lane = threadIdx.x & 31;
  const int tiles = p.m_tiles * p.n_tiles;
  const int tile = blockIdx.x % tiles, split = blockIdx.x / tiles;
  const int m0 = (tile / p.n_tiles) * 64 * p.a_chunks, k0 = (tile % p.n_tiles) * 64 * p.b_chunks;
  const int a_chunks = min(p.a_chunks, (p.N - m0 + 63) / 64);
  const int b_chunks = min(p.b_chunks, (p.K - k0 + 63) / 64);
  const int blocks = p.a_chunks > 2 && p.N - m0 > 128 ? 2 : 1;
  const bool with_db = p.part_db != nullptr && k0 == 0;
  const int s0 = split * p.steps_per_split, s1 = min(p.steps, s0 + p.steps_per_split);
  const uint64_t lim = p.wait_limit_ns;
  if (threadIdx.x == 0) {
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(&bb.full[i], 1);
      mbar_init(&bb.empty[i], 1);
    }
    mbar_init(&bb.acc_full, 1);
    mbar_init(&bb.acc_free, 4 * blocks);
    mbar_init(&bb.drain, 1);
    bb.abort_flag = 0;
    fence_mbarrier_init();
  }
  if (with_db) {
    // ones behind x's atoms (every element: the swizzle does not matter)
    for (int i = threadIdx.x; i < p.stages * 512; i += kDwThreads)
      *reinterpret_cast<uint4*>(base + (i / 512) * stage_bytes + b_off + b_chunks * kDwAtom +
                                (i % 512) * 16) =
          make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u);
    fence_proxy_async_smem();
  }
  if (warp == 9) {
    tmem_alloc(&bb.tmem, 512);
    tmem_relinquish();
  }
  pdl_wait();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bb.tmem;
  if (warp < 8) {
    // ---------------------------------------------------------- epilogue
    // warp w: rows 32 (w % 4) .. of block w / 4, every column
    regs_inc<kDwEpiRegs>();
    if ((warp >> 2) < blocks) {
      const int blk = warp >> 2;
      const int n = m0 + 128 * blk + 32 * (warp & 3) + lane;
      const uint32_t acc = tmem + 256 * blk + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
      float sum[kDwBn], sum_db = 0.f;
#pragma unroll
      for (int c = 0; c < kDwBn; ++c) sum[c] = 0.f;
      bool ok = true;
      int f = 0;
      for (int s = s0; s < s1; s += kDwFlush, ++f) {
        if (!(ok = warp_wait(&bb.acc_full, f & 1, ab, lim, SITE_DW))) break;
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < kDwBn / 16; ++c) {
          if (c >= 4 * b_chunks) continue;
          uint32_t v[16];
          tmem_ld_x16(acc + 16 * c, v);
          tmem_wait_ld();
          reg_fence_x16(v);
#pragma unroll
          for (int e = 0; e < 16; ++e) sum[16 * c + e] += __uint_as_float(v[e]);
        }
        if (with_db) {
          uint32_t v[16];
          tmem_ld_x16(acc + 64 * b_chunks, v);
          tmem_wait_ld();
          reg_fence_x16(v);
          sum_db += __uint_as_float(v[0]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bb.acc_free);
      }
      // this thread's row of the tile (a tile of three chunks ends inside its
      // second block, whose other rows are the next tile's)
      const int n_end = min(p.N, m0 + 64 * p.a_chunks);
      const size_t row = static_cast<size_t>(split) * p.N + n;
      if (ok && p.part && n - lane < n_end) {
        // fp32: 32 columns at a time through shared memory, whose stages are
        // all consumed, and a bulk store: a row per lane, stored directly, would
        // be half sectors all over the rows
        uint8_t* sg = base + warp * 8192;
#pragma unroll
        for (int c = 0; c < kDwBn / 32; ++c) {
          if (c >= 2 * b_chunks || k0 + 32 * c >= p.K) continue;
          uint8_t* dst = sg + (c & 1) * 4096 + lane * 128;   // 128-byte swizzle
          if (lane == 0 && c >= 2) bulk_store_wait_read_one();
          __syncwarp();
#pragma unroll
          for (int e = 0; e < 8; ++e)
            *reinterpret_cast<float4*>(dst + ((e ^ (lane & 7)) << 4)) =
                make_float4(sum[32 * c + 4 * e], sum[32 * c + 4 * e + 1], sum[32 * c + 4 * e + 2],
                            sum[32 * c + 4 * e + 3]);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_3d(&tm_part, sg + (c & 1) * 4096, k0 + 32 * c, n, split);
            tma_store_commit();
          }
        }
      }
      if (ok && n < n_end) {
        const size_t all = static_cast<size_t>(p.N) * p.K;
#pragma unroll
        for (int c = 0; c < kDwBn / 4; ++c) {
          const int k = k0 + 4 * c;
          const size_t at = row * p.K + k;   // one split
          if (!p.out16 || c >= 16 * b_chunks || k >= p.K || !rib_guard(at + 3, all, G_DW_PART))
            continue;
          *reinterpret_cast<uint2*>(p.out16 + at) =
              make_uint2(pack_bf16x2(sum[4 * c], sum[4 * c + 1]),
                         pack_bf16x2(sum[4 * c + 2], sum[4 * c + 3]));
        }
        if (with_db && rib_guard(row, static_cast<size_t>(p.splits) * p.N, G_DW_PART))
          p.part_db[row] = sum_db;
      }
      if (lane == 0) tma_store_wait_all();
    }
  } else {
    regs_dec<kDwOtherRegs>();
    bool ok = true;
    if (warp == 8) {
      // -------------------------------------------------------- TMA producer
      if (lane == 0) {
        int q = 0, st = 0;
        uint32_t ph = 1;
        for (int s = s0; s < s1; ++s, ++q) {
          if (q >= p.stages && !(ok = mbar_wait(&bb.empty[st], ph, ab, lim, SITE_DW))) break;
          uint8_t* sa = base + st * stage_bytes;
          mbar_arrive_expect_tx(&bb.full[st], (a_chunks + b_chunks) * kDwAtom);
          for (int c = 0; c < a_chunks; ++c)
            tma_load_2d(sa + c * kDwAtom, &tm_z, &bb.full[st], m0 + 64 * c, 64 * s);
          for (int c = 0; c < b_chunks; ++c)
            tma_load_2d(sa + b_off + c * kDwAtom, &tm_x, &bb.full[st], k0 + 64 * c, 64 * s);
          if (++st == p.stages) {
            st = 0;
            ph ^= 1;
          }
        }
        if (*ab) {
          volatile int no_abort = 0;
          for (int i = max(0, q - p.stages); i < q; ++i)
            mbar_wait(&bb.full[i % p.stages], (i / p.stages) & 1, &no_abort, 200000000ull, SITE_DW);
        }
      }
    } else if (warp == 9) {
      // -------------------------------------------------------- MMA issue
      const uint32_t idesc = make_idesc_bf16(128, 64 * b_chunks + (with_db ? 16 : 0), true, true);
      int q = 0, st = 0, f = 0;
      uint32_t ph = 0;
      RingWait ring;
      for (int s = s0; ok && s < s1; ++s, ++q) {
        const bool fresh = q % kDwFlush == 0;
        if (fresh && q > 0) {   // the last chain's sums leave tensor memory
          umma_commit_elect(&bb.acc_full);
          if (!(ok = warp_wait(&bb.acc_free, f & 1, ab, lim, SITE_DW))) break;
          ++f;
        }
        if (!(ok = ring.wait(&bb.full[st], ph, ab, lim, SITE_DW))) break;
        tc_fence_after();
        const uint32_t sa = smem_u32(base + st * stage_bytes);
        const uint64_t bd = make_sdesc(sa + b_off, kDwAtom, 1024, kLayoutSW128);
        uint64_t* done = &bb.empty[st];
        if (++st == p.stages) {
          st = 0;
          ph ^= 1;
        }
        ring.peek(&bb.full[st], ph);
        for (int b = 0; b < blocks; ++b)
          pair_umma4<1>(tmem + 256 * b, make_sdesc(sa + 2 * b * kDwAtom, kDwAtom, 1024, kLayoutSW128),
                        128, bd, 128, idesc, fresh ? 0u : 1u);
        umma_commit_elect(done);
      }
      if (ok) umma_commit_elect(&bb.acc_full);
      umma_commit_elect(&bb.drain);
      volatile int no_abort = 0;
      mbar_wait(&bb.drain, 0, &no_abort, 200000000ull, SITE_DW);
    }
  }
  tc_fence_before();
  __syncthreads();
  settle(ab);
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// db and dW = the sums of their partials.  Groups of threads take a run of the
// partials each, in order, and the groups' sums are added in order: for db,
// whose partials may be another kernel's and many more, sixteen groups (in the
// first db_blocks blocks), for dW four.  nb4 = N / 4 float4 of db, n4 = N K / 4
// of dW (none when there is one split); dW fp32 or rounded to bf16 once.
// grid db_blocks + ceil(n4 / 64), db_blocks = ceil(nb4 / 16), block 256.
__global__ void __launch_bounds__(256)
    dw_reduce_kernel(const float* part, const float* part_db, int dw_splits, int db_splits,
                     size_t n4, size_t nb4, float* out32, __nv_bfloat16* out16, float* db) {
  __shared__ float4 sums[256];
  pdl_wait();
  const unsigned db_blocks = static_cast<unsigned>((nb4 + 15) / 16);
  const bool is_db = blockIdx.x < db_blocks;
  const int cols = is_db ? 16 : 64, groups = 256 / cols;
  const int col = threadIdx.x % cols, group = threadIdx.x / cols;
  const size_t i = static_cast<size_t>(blockIdx.x - (is_db ? 0u : db_blocks)) * cols + col;
  const float* src = is_db ? part_db : part;
  const int splits = is_db ? db_splits : dw_splits;
  const size_t n = 4 * (is_db ? nb4 : n4), at0 = 4 * i;
  const bool in = at0 < n;
  const int per = (splits + groups - 1) / groups, k1 = min(splits, (group + 1) * per);
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (in) {
#pragma unroll 4
    for (int k = group * per; k < k1; ++k) {
      const size_t at = static_cast<size_t>(k) * n + at0;
      if (!rib_guard(at + 3, static_cast<size_t>(splits) * n, G_DW_RED)) continue;
      const float4 v = *reinterpret_cast<const float4*>(src + at);
      s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
    }
  }
  sums[threadIdx.x] = s;
  __syncthreads();
  if (group != 0 || !in) return;
  for (int g = 1; g < groups; ++g) {
    const float4 v = sums[g * cols + col];
    s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
  }
  if (is_db)
    *reinterpret_cast<float4*>(db + at0) = s;
  else if (out32)
    *reinterpret_cast<float4*>(out32 + at0) = s;
  else
    *reinterpret_cast<uint2*>(out16 + at0) = make_uint2(pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w));
}

// ---------------------------------------------------------------- dz
// dz = dy act'(pre), rounded to bf16 for the products that follow (their
// operands are bf16), and per-row-range column sums of the unrounded fp32
// dz.  A thread keeps one channel octet over its rows.  With pre null dz is
// dy itself and only the sums are formed.
// grid (ceil(N / 256), row splits), block 256: 32 octets x 8 row slots.
struct DzParams {
  const __nv_bfloat16* dy;
  const __nv_bfloat16* pre;   // null: act none, sums only
  __nv_bfloat16* dz;
  float* part;                // [gridDim.y][N]; null: no sums
  int rows, N;
};

template <int ACT>
__global__ void __launch_bounds__(256) dz_kernel(const DzParams p) {
  __shared__ float sums[8][256];
  pdl_wait();
  const int oct = threadIdx.x & 31, slot = threadIdx.x >> 5;
  const int c = blockIdx.x * 256 + 8 * oct;
  const size_t n = static_cast<size_t>(p.rows) * p.N;
  float acc[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) acc[e] = 0.f;
  const bool in = c < p.N;
  constexpr int B = 4;   // rows in flight per thread
  const long long step = 8ll * gridDim.y;
  for (long long r0 = slot + 8ll * blockIdx.y; in && r0 < p.rows; r0 += B * step) {
    uint4 dv[B], zv[B];
#pragma unroll
    for (int k = 0; k < B; ++k) {
      const long long r = r0 + k * step;
      const size_t at = static_cast<size_t>(r) * p.N + c;
      const bool ok = r < p.rows && rib_guard(at + 7, n, G_DZ_IN);
      dv[k] = ok ? *reinterpret_cast<const uint4*>(p.dy + at) : make_uint4(0, 0, 0, 0);
      zv[k] = ok && ACT != kActNone ? *reinterpret_cast<const uint4*>(p.pre + at)
                                    : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int k = 0; k < B; ++k) {
      const long long r = r0 + k * step;
      if (r >= p.rows) break;
      const uint32_t dw[4] = {dv[k].x, dv[k].y, dv[k].z, dv[k].w};
      const uint32_t zw[4] = {zv[k].x, zv[k].y, zv[k].z, zv[k].w};
      uint32_t o[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float d0 = __uint_as_float(dw[e] << 16), d1 = __uint_as_float(dw[e] & 0xffff0000u);
        if constexpr (ACT != kActNone) {
          float a, g0, g1;
          act_both<ACT>(__uint_as_float(zw[e] << 16), a, g0);
          act_both<ACT>(__uint_as_float(zw[e] & 0xffff0000u), a, g1);
          d0 *= g0;
          d1 *= g1;
          o[e] = pack_bf16x2(d0, d1);
        }
        acc[2 * e] += d0;
        acc[2 * e + 1] += d1;
      }
      if constexpr (ACT != kActNone) {
        const size_t at = static_cast<size_t>(r) * p.N + c;
        if (rib_guard(at + 7, n, G_DZ_OUT))
          *reinterpret_cast<uint4*>(p.dz + at) = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
  }
  if (!p.part) return;
#pragma unroll
  for (int e = 0; e < 8; ++e) sums[slot][8 * oct + e] = acc[e];
  __syncthreads();
  const int col = blockIdx.x * 256 + threadIdx.x;
  if (col < p.N) {
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) s += sums[k][threadIdx.x];
    const size_t at = static_cast<size_t>(blockIdx.y) * p.N + col;
    if (rib_guard(at, static_cast<size_t>(gridDim.y) * p.N, G_DW_PART)) p.part[at] = s;
  }
}

}  // namespace rib
