// ffn.cuh -- backward of the gated feed-forward block's inner half.
//
// Forward (gemm.cuh, kGated and kLinear):
//   g = x Wg^T + bg,  u = x Wu^T + bu,  h = act(g) u,  y = h Wo^T + bo + residual
// This kernel recomputes g and u from x (nothing but x is kept from the
// forward: keeping them would cost 8 bytes of HBM traffic per hidden element,
// recomputing them 4 C FLOPs, which is less time up to C of about 500 and
// never more than a third of the backward), forms dh = dy Wo beside them,
// and writes what the remaining products read:
//   h,  dg = dh u act'(g),  du = dh act(g)      (bf16, the products' operands)
//   sum over rows of dg and du                  (fp32, before the rounding)
// One tile is 128 rows x 64 hidden channels with three accumulators (g | u as
// one MMA of 128 columns, then dh), two sets of them in tensor memory; the
// warp roles are gemm.cuh's with eight epilogue warps.
//
// 147456 rows, 192 channels, 384 hidden: 107 us for 453 MB, 4.2 TB/s; the whole
// backward reads and writes 1190 MB in 262 us, 4.5 TB/s.
// Nor epilogue (without its arithmetic 117 us for 119, before the following) nor
// stores (102 without any) bound it but the latency of x and dy, read once per
// column tile, mostly from L2: so the staging takes 16 columns at a time and a
// fourth stage of x and dy fits beside the resident weights (119 -> 107 us; the
// next kernel then meets more writes still on their way: 265 -> 262 in all).
// The tensor core truncates when it adds to its accumulator, so g, u and dh drift
// towards zero with the channels that are added up in one chain (dw_kernel), and
// the bias gradients, fp32 sums of what is formed from them, with them: 2.1e-6 at
// 1024 channels, a plain fp32 sum 0.4e-6.  Beyond kFfnChain k-steps the chains are
// therefore cut (CHUNKED): each piece is a tile of its own to the MMA warp, and the
// epilogue warps add the pieces to nearest, g and u in the tensor memory beside
// the accumulators, dh in registers: 0.65e-6, for 4 % of the whole backward
// (8192 rows of 1024, 2816 hidden: 406 -> 421 us).
// Not kept: sixteen epilogue warps (124), tiles of 256 x 128 by CTA pairs, which
// halve those reads but hold their accumulators longer (132).
#pragma once

#include "gemm.cuh"

namespace rib {

constexpr int kFfnThreads = 320;
constexpr int kFfnCols = 64;                              // hidden channels of a tile
constexpr uint32_t kFfnA = 2u * kGemmATile;               // x and dy, 64 channels deep
constexpr uint32_t kFfnB = 3u * 8192u;                    // Wg, Wu (K-major), Wo (MN-major)
constexpr uint32_t kFfnOut = 32u * 32u;                   // a warp's staging: 32 rows x 16 columns
constexpr uint32_t kFfnStaging = 8u * 3u * kFfnOut;
constexpr int kFfnMaxStages = 6;
constexpr int kFfnChain = 8;                              // k-steps (4 additions each) of one chain
constexpr int kFfnPiece = 6;                              // at most, where chains are cut

struct FfnBwdParams {
  const float* b_in;      // [2][H]; may be null
  float* part;            // [splits * 4][2][H] column sums of dg, du; null: not wanted
  int M, C, H;
  int m_tiles, n_tiles, splits, k_steps, stages, b_resident;
  int piece;              // k-steps of a chain (CHUNKED)
  uint64_t wait_limit_ns;
};

struct FfnBars {
  uint64_t full[kFfnMaxStages], empty[kFfnMaxStages];
  uint64_t acc_full[2], acc_free[2], b_full, b_free, drain;
  uint32_t tmem;
  int abort_flag;
};

__host__ __device__ __forceinline__ size_t ffn_bwd_smem_bytes(int stages, int k_steps,
                                                              bool resident) {
  return 1024 + static_cast<size_t>(stages) * (kFfnA + (resident ? 0 : kFfnB)) +
         (resident ? static_cast<size_t>(k_steps) * kFfnB : 0) + kFfnStaging + sizeof(FfnBars);
}

// Sums 16 columns over the warp's 32 rows (lane = row): each step sends half
// of the columns to the partner lane and keeps the other half, so 16 shuffles
// do what 80 would column by column.  Lane l ends with column l / 2.
__device__ __forceinline__ float col_sum16(float (&v)[16], int lane) {
#pragma unroll
  for (int w = 8; w >= 1; w >>= 1) {
    const int mask = 2 * w;
    const bool up = (lane & mask) != 0;
#pragma unroll
    for (int i = 0; i < w; ++i) {
      const float send = up ? v[i] : v[i + w];
      const float keep = up ? v[i + w] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, send, mask);
    }
  }
  return v[0] + __shfl_xor_sync(0xffffffffu, v[0], 1);
}

__device__ __forceinline__ void ffn_load_b(uint8_t* dst, const CUtensorMap* tm_in,
                                           const CUtensorMap* tm_out, uint64_t* bar, int H,
                                           int n0, int k) {
  tma_load_2d(dst, tm_in, bar, 64 * k, n0);
  tma_load_2d(dst + 8192, tm_in, bar, 64 * k, H + n0);
  tma_load_2d(dst + 16384, tm_out, bar, n0, 64 * k);
}

// Work items and grid as in gemm_kernel.  tm_x, tm_dy: [M][C], boxes 64 x
// 128; tm_in: w_in [2 H][C], boxes 64 x 64; tm_out: w_out [C][H], boxes 64 x
// 64 (all 128-byte swizzle); tm_h: h [M][H], boxes 16 x 32, tm_d: dg | du
// [M][2][H], boxes 16 x 1 x 32 (32-byte swizzle).
template <int ACT, bool CHUNKED>
__global__ void __launch_bounds__(kFfnThreads, 1)
    ffn_bwd_kernel(const __grid_constant__ CUtensorMap tm_x,
                   const __grid_constant__ CUtensorMap tm_dy,
                   const __grid_constant__ CUtensorMap tm_in,
                   const __grid_constant__ CUtensorMap tm_out,
                   const __grid_constant__ CUtensorMap tm_h,
                   const __grid_constant__ CUtensorMap tm_d, const FfnBwdParams p) {
  extern __shared__ uint8_t ffn_raw[];
  uint8_t* base = ffn_raw + ((1024u - (smem_u32(ffn_raw) & 1023u)) & 1023u);
  const uint32_t stage_bytes = kFfnA + (p.b_resident ? 0u : kFfnB);
  uint8_t* s_res = base + p.stages * stage_bytes;
  uint8_t* s_stage = s_res + (p.b_resident ? p.k_steps * kFfnB : 0u);
  FfnBars& bb = *reinterpret_cast<FfnBars*>(s_stage + kFfnStaging);
  volatile int* ab = &bb.abort_flag;
  const int warp = warp_index(), lane = threadIdx.x & 31;
  const int items = p.n_tiles * p.splits;
  const int piece = CHUNKED ? p.piece : p.k_steps;
  const uint64_t lim = p.wait_limit_ns;
  if (threadIdx.x == 0) {
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(&bb.full[i], 1);
      mbar_init(&bb.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bb.acc_full[i], 1);
      mbar_init(&bb.acc_free[i], 8);
    }
    mbar_init(&bb.b_full, 1);
    mbar_init(&bb.b_free, 1);
    mbar_init(&bb.drain, 1);
    bb.abort_flag = 0;
    fence_mbarrier_init();
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

  if (warp == 8) {
    // ---------------------------------------------------------- TMA producer
    if (lane == 0) {
      bool ok = true;
      int q = 0, st = 0, n_item = 0;
      uint32_t ph = 1;
      for (int it = blockIdx.x; ok && it < items; it += gridDim.x, ++n_item) {
        const int n0 = (it % p.n_tiles) * kFfnCols;
        if (p.b_resident) {
          if (n_item > 0 && !(ok = mbar_wait(&bb.b_free, (n_item - 1) & 1, ab, lim, SITE_FFN)))
            break;
          mbar_arrive_expect_tx(&bb.b_full, p.k_steps * kFfnB);
          for (int k = 0; k < p.k_steps; ++k)
            ffn_load_b(s_res + k * kFfnB, &tm_in, &tm_out, &bb.b_full, p.H, n0, k);
        }
        for (int m = it / p.n_tiles; ok && m < p.m_tiles; m += p.splits)
          for (int k = 0; k < p.k_steps; ++k) {
            if (q >= p.stages && !(ok = mbar_wait(&bb.empty[st], ph, ab, lim, SITE_FFN))) break;
            uint8_t* sa = base + st * stage_bytes;
            mbar_arrive_expect_tx(&bb.full[st], stage_bytes);
            tma_load_2d(sa, &tm_x, &bb.full[st], 64 * k, 128 * m);
            tma_load_2d(sa + kGemmATile, &tm_dy, &bb.full[st], 64 * k, 128 * m);
            if (!p.b_resident)
              ffn_load_b(sa + kFfnA, &tm_in, &tm_out, &bb.full[st], p.H, n0, k);
            ++q;
            if (++st == p.stages) {
              st = 0;
              ph ^= 1;
            }
          }
      }
      if (*ab) {
        volatile int no_abort = 0;
        if (p.b_resident && n_item > 0)
          mbar_wait(&bb.b_full, (n_item - 1) & 1, &no_abort, 200000000ull, SITE_FFN);
        for (int i = max(0, q - p.stages); i < q; ++i)
          mbar_wait(&bb.full[i % p.stages], (i / p.stages) & 1, &no_abort, 200000000ull, SITE_FFN);
      }
    }
  } else if (warp == 9) {
    // ---------------------------------------------------------- MMA issue
    const int last_steps = (p.C - 64 * (p.k_steps - 1) + 15) / 16;
    const uint32_t id_gu = make_idesc_bf16(128, 128, false, false);
    const uint32_t id_dh = make_idesc_bf16(128, 64, false, true);
    bool ok = true;
    int st = 0, t = 0, n_item = 0;
    uint32_t ph = 0;
    RingWait ring;
    for (int it = blockIdx.x; ok && it < items; it += gridDim.x, ++n_item) {
      if (p.b_resident && !(ok = warp_wait(&bb.b_full, n_item & 1, ab, lim, SITE_FFN))) break;
      for (int m = it / p.n_tiles; ok && m < p.m_tiles; m += p.splits)
        for (int k0 = 0; ok && k0 < p.k_steps; k0 += piece, ++t) {   // t: chains so far
          const int a = t & 1;
          if (t >= 2 && !(ok = warp_wait(&bb.acc_free[a], ((t >> 1) - 1) & 1, ab, lim, SITE_FFN)))
            break;
          const int k1 = min(k0 + piece, p.k_steps);
          for (int k = k0; k < k1; ++k) {
            if (!(ok = ring.wait(&bb.full[st], ph, ab, lim, SITE_FFN))) break;
            tc_fence_after();
            const uint32_t sa = smem_u32(base + st * stage_bytes);
            const uint32_t sb = p.b_resident ? smem_u32(s_res + k * kFfnB) : sa + kFfnA;
            const uint64_t xd = make_sdesc(sa, 16, 1024, kLayoutSW128);
            const uint64_t yd = make_sdesc(sa + kGemmATile, 16, 1024, kLayoutSW128);
            const uint64_t wd = make_sdesc(sb, 16, 1024, kLayoutSW128);
            const uint64_t od = make_sdesc(sb + 16384, 8192, 1024, kLayoutSW128);
            const int steps = k + 1 == p.k_steps ? last_steps : 4;
            uint64_t* done = &bb.empty[st];
            if (++st == p.stages) {
              st = 0;
              ph ^= 1;
            }
            ring.peek(&bb.full[st], ph);
            const uint32_t acc = k > k0 ? 1u : 0u;
            pair_umma_steps<1>(steps, tmem + 256 * a, xd, 2, wd, 2, id_gu, acc);
            pair_umma_steps<1>(steps, tmem + 256 * a + 128, yd, 2, od, 128, id_dh, acc);
            umma_commit_elect(done);
          }
          if (ok) umma_commit_elect(&bb.acc_full[a]);
        }
      if (ok && p.b_resident) umma_commit_elect(&bb.b_free);
    }
    umma_commit_elect(&bb.drain);
    volatile int no_abort = 0;
    mbar_wait(&bb.drain, 0, &no_abort, 200000000ull, SITE_FFN);
  } else {
    // ---------------------------------------------------------- epilogue
    // warp w: tile rows 32 (w % 4) .., hidden channels 32 (w / 4) ..
    const int quarter = warp & 3, half = warp >> 2;
    uint8_t* sg = s_stage + warp * 3 * kFfnOut;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const size_t part_n = static_cast<size_t>(p.splits) * 8 * p.H;
    int t = 0;
    bool ok = true;
    for (int it = blockIdx.x; ok && it < items; it += gridDim.x) {
      const int n0 = (it % p.n_tiles) * kFfnCols + 32 * half;   // this warp's first channel
      const int split = it / p.n_tiles;
      float sum_g[2] = {0.f, 0.f}, sum_u[2] = {0.f, 0.f};
      for (int m = split; m < p.m_tiles; m += p.splits, ++t) {
        // the pieces before a tile's last one: added up, g and u in the columns
        // behind the accumulators (which only this warp touches)
        [[maybe_unused]] float dh[CHUNKED ? 32 : 1];
        const uint32_t sum_gu = tmem + 192 + lane_off + 32 * half;   // g; u 256 columns on
        if constexpr (CHUNKED) {
          for (int k1 = piece; k1 < p.k_steps; k1 += piece, ++t) {
            const int b = t & 1;
            if (!(ok = warp_wait(&bb.acc_full[b], (t >> 1) & 1, ab, lim, SITE_FFN))) break;
            tc_fence_after();
            const uint32_t acc = tmem + 256 * b + lane_off + 32 * half;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t g[16], u[16], d[16];
              tmem_ld_x16(acc + 16 * h, g);
              tmem_ld_x16(acc + 64 + 16 * h, u);
              tmem_ld_x16(acc + 128 + 16 * h, d);
              if (k1 > piece) {
                uint32_t sg[16], su[16];
                tmem_ld_x16(sum_gu + 16 * h, sg);
                tmem_ld_x16(sum_gu + 256 + 16 * h, su);
                tmem_wait_ld();
                reg_fence_x16(g);
                reg_fence_x16(u);
                reg_fence_x16(d);
                reg_fence_x16(sg);
                reg_fence_x16(su);
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                  g[e] = __float_as_uint(__uint_as_float(g[e]) + __uint_as_float(sg[e]));
                  u[e] = __float_as_uint(__uint_as_float(u[e]) + __uint_as_float(su[e]));
                  dh[16 * h + e] += __uint_as_float(d[e]);
                }
              } else {
                tmem_wait_ld();
                reg_fence_x16(g);
                reg_fence_x16(u);
                reg_fence_x16(d);
#pragma unroll
                for (int e = 0; e < 16; ++e) dh[16 * h + e] = __uint_as_float(d[e]);
              }
              tmem_st_x16(sum_gu + 16 * h, g);
              tmem_st_x16(sum_gu + 256 + 16 * h, u);
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bb.acc_free[b]);
          }
          if (!ok) break;
        }
        const int a = t & 1;
        const int row0 = 128 * m + 32 * quarter;
        if (!(ok = warp_wait(&bb.acc_full[a], (t >> 1) & 1, ab, lim, SITE_FFN))) break;
        tc_fence_after();
        const uint32_t acc = tmem + 256 * a + lane_off + 32 * half;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t g[16], u[16], d[16];
          tmem_ld_x16(acc + 16 * h, g);
          tmem_ld_x16(acc + 64 + 16 * h, u);
          tmem_ld_x16(acc + 128 + 16 * h, d);
          if constexpr (CHUNKED) {
            uint32_t pg[16], pu[16];
            tmem_ld_x16(sum_gu + 16 * h, pg);
            tmem_ld_x16(sum_gu + 256 + 16 * h, pu);
            tmem_wait_ld();
            reg_fence_x16(g);
            reg_fence_x16(u);
            reg_fence_x16(d);
            reg_fence_x16(pg);
            reg_fence_x16(pu);
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              g[e] = __float_as_uint(__uint_as_float(g[e]) + __uint_as_float(pg[e]));
              u[e] = __float_as_uint(__uint_as_float(u[e]) + __uint_as_float(pu[e]));
              d[e] = __float_as_uint(__uint_as_float(d[e]) + dh[16 * h + e]);
            }
          } else {
            tmem_wait_ld();
            reg_fence_x16(g);
            reg_fence_x16(u);
            reg_fence_x16(d);
          }
          if (h == 1) {   // the accumulators are in registers
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bb.acc_free[a]);
          }
          float dg[16], du[16];
          uint32_t hw[8], gw[8], uw[8];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int col = n0 + 16 * h + 4 * e;
            float4 bg = make_float4(0.f, 0.f, 0.f, 0.f), bu = bg;
            if (p.b_in && col < p.H &&
                rib_guard(static_cast<size_t>(p.H) + col + 3, 2ull * p.H, G_GEMM_BIAS)) {
              bg = *reinterpret_cast<const float4*>(p.b_in + col);
              bu = *reinterpret_cast<const float4*>(p.b_in + p.H + col);
            }
            const float b4[4] = {bg.x, bg.y, bg.z, bg.w}, c4[4] = {bu.x, bu.y, bu.z, bu.w};
            float hv[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int j = 4 * e + i;
              const float uv = __uint_as_float(u[j]) + c4[i], dv = __uint_as_float(d[j]);
              float av, sl;
              act_both<ACT>(__uint_as_float(g[j]) + b4[i], av, sl);
              hv[i] = av * uv;
              dg[j] = dv * uv * sl;
              du[j] = dv * av;
            }
            hw[2 * e] = pack_bf16x2(hv[0], hv[1]);
            hw[2 * e + 1] = pack_bf16x2(hv[2], hv[3]);
            gw[2 * e] = pack_bf16x2(dg[4 * e], dg[4 * e + 1]);
            gw[2 * e + 1] = pack_bf16x2(dg[4 * e + 2], dg[4 * e + 3]);
            uw[2 * e] = pack_bf16x2(du[4 * e], du[4 * e + 1]);
            uw[2 * e + 1] = pack_bf16x2(du[4 * e + 2], du[4 * e + 3]);
          }
          if (lane == 0) tma_store_wait_read_all();   // the last stores have read the staging
          __syncwarp();
          // rows of 32 bytes, 32-byte swizzle: granule XOR (row / 4) % 2
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            uint8_t* dst = sg + lane * 32 + ((e ^ ((lane >> 2) & 1)) << 4);
            *reinterpret_cast<uint4*>(dst) =
                make_uint4(hw[4 * e], hw[4 * e + 1], hw[4 * e + 2], hw[4 * e + 3]);
            *reinterpret_cast<uint4*>(dst + kFfnOut) =
                make_uint4(gw[4 * e], gw[4 * e + 1], gw[4 * e + 2], gw[4 * e + 3]);
            *reinterpret_cast<uint4*>(dst + 2 * kFfnOut) =
                make_uint4(uw[4 * e], uw[4 * e + 1], uw[4 * e + 2], uw[4 * e + 3]);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0 && row0 < p.M && n0 + 16 * h < p.H) {
            tma_store_2d(&tm_h, sg, n0 + 16 * h, row0);
            tma_store_3d(&tm_d, sg + kFfnOut, n0 + 16 * h, 0, row0);
            tma_store_3d(&tm_d, sg + 2 * kFfnOut, n0 + 16 * h, 1, row0);
            tma_store_commit();
          }
          if (p.part) {
            // rows beyond M: x and dy are the TMA's zeros, so dh = 0 and they
            // add nothing
            sum_g[h] += col_sum16(dg, lane);
            sum_u[h] += col_sum16(du, lane);
          }
        }
      }
      if (ok && p.part && (lane & 1) == 0) {
        // one row of partials per (split, quarter)
        const size_t row = (static_cast<size_t>(split) * 4 + quarter) * 2 * p.H;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int col = n0 + 16 * h + (lane >> 1);
          if (col < p.H && rib_guard(row + p.H + col, part_n, G_FFN_PART)) {
            p.part[row + col] = sum_g[h];
            p.part[row + p.H + col] = sum_u[h];
          }
        }
      }
    }
    if (lane == 0) tma_store_wait_all();
  }
  tc_fence_before();
  __syncthreads();
  settle(ab);
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace rib
