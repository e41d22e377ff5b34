// ffn_fused.cuh -- the gated feed-forward block's forward in one kernel, for
// up to 256 channels:
//   y = (act(x Wg^T + bg) (x Wu^T + bu)) Wo^T + bo + residual
//
// A pair of CTAs (cta_group::2, gemm.cuh) owns 256 rows.  Their x stays in
// shared memory and their y (256 x C) in tensor memory while the pair walks
// the hidden channels 64 at a time: an MMA of 128 columns gives the chunk's
// gate and other projection (GU), the epilogue warps turn it into 64 columns of
// h, and a second MMA adds h Wo^T to y (Y).  h never reaches HBM: at 192 channels
// and 384 hidden ones that is 226 of 396 MB.  What is read again per row tile are
// the weights, from L2; each CTA of a pair reads half.
//
// h lies in tensor memory, where Y takes its A operand from: each warp writes
// its 16 channels of h (bf16 pairs, 8 columns, one step of the MMA) over the
// 16 gate columns that it has just read, in its own CTA's lanes.  That makes
// the hand-over to CTA 0, which issues the MMAs for both, one of tensor memory
// only, ordered by the tcgen05 fences around the arrival and the wait.  (Through
// shared memory, CTA 1's h would have to be published to CTA 0 at cluster
// scope, which took 107 us of 147456 x 192 x 384 rows for 86, by a relay in each
// CTA as by releases from every warp.)
//
// Order of the work, with chunk g of all the pair's chunks:
//   MMA        GU(0), GU(1), Y(0), GU(2), Y(1), GU(3), ...   GU(g + 2) takes the
//              columns of h(g) and so waits for Y(g); the epilogue has GU(g + 1)
//              meanwhile, and is much the longer
//   epilogue   h(0), h(1), ...; y of a row tile after the first h of the next
//              one; y leaves tensor memory before it is worked on, so that the
//              next tile's Y can start, and its residual is loaded one chunk
//              ahead
// Two accumulators of 128 columns for GU and h, one of C for y.
#pragma once

#include "gemm.cuh"

namespace rib {

constexpr int SITE_FUSED = 53;
constexpr int kFusedMaxC = 256;
constexpr int kFusedMaxRing = 4;

struct FusedParams {
  const float* b_in;    // [2][H] or null
  const float* b_out;   // [C] or null
  int M, C, H;
  int m_tiles, chunks, k_steps, ring;
  uint64_t wait_limit_ns;
};

struct FusedBars {
  uint64_t x_full, x_free, y_full, y_free;
  uint64_t in_full[kFusedMaxRing], in_free[kFusedMaxRing];
  uint64_t out_full[kFusedMaxRing], out_free[kFusedMaxRing];
  uint64_t gu_full[2], h_full[2], y_done[2];
  uint64_t drain, res[kGemmEpiWarps];
  uint32_t tmem;
  int abort_flag;
};

// MMA columns of y: whole 16 columns in each CTA.
__host__ __device__ __forceinline__ int fused_cols(int C) { return (C + 31) / 32 * 32; }
__host__ __device__ __forceinline__ uint32_t fused_in_bytes(int C) { return (C + 63) / 64 * 8192u; }
__host__ __device__ __forceinline__ uint32_t fused_out_bytes(int C) { return fused_cols(C) / 2 * 128u; }
__host__ __device__ __forceinline__ size_t fused_smem_bytes(int C, int ring) {
  return 1024 + static_cast<size_t>((C + 63) / 64) * kGemmATile +
         static_cast<size_t>(ring) * (fused_in_bytes(C) + fused_out_bytes(C)) + kGemmStaging +
         sizeof(FusedBars);
}

// tm_x: [M][C], boxes 64 x 128; tm_in: w_in [2 H][C], boxes 64 x 64; tm_out: w_out
// [C][H], boxes 64 x fused_cols(C) / 2 (128-byte swizzle); tm_y, tm_res: [M][C],
// boxes 32 x 32 (64-byte swizzle).
// grid 2 * min(m_tiles, SMs / 2) in clusters of two, block kGemmThreads, dynamic
// smem fused_smem_bytes().
template <int ACT, bool RES>
__global__ void __launch_bounds__(kGemmThreads, 1)
    ffn_fused_kernel(const __grid_constant__ CUtensorMap tm_x,
                     const __grid_constant__ CUtensorMap tm_in,
                     const __grid_constant__ CUtensorMap tm_out,
                     const __grid_constant__ CUtensorMap tm_y,
                     const __grid_constant__ CUtensorMap tm_res, const FusedParams p) {
  extern __shared__ uint8_t fused_raw[];
  uint8_t* s_x = fused_raw + ((1024u - (smem_u32(fused_raw) & 1023u)) & 1023u);
  const uint32_t in_bytes = fused_in_bytes(p.C), out_bytes = fused_out_bytes(p.C);
  const uint32_t x_bytes = p.k_steps * kGemmATile;
  uint8_t* s_in = s_x + x_bytes;
  uint8_t* s_out = s_in + p.ring * in_bytes;
  uint8_t* s_stage = s_out + p.ring * out_bytes;
  FusedBars& bb = *reinterpret_cast<FusedBars*>(s_stage + kGemmStaging);
  volatile int* ab = &bb.abort_flag;
  const int warp = warp_index(), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int pair = blockIdx.x / 2, pairs = gridDim.x / 2;
  const int tiles = (p.m_tiles - pair + pairs - 1) / pairs;   // this pair's row tiles
  const uint64_t lim = p.wait_limit_ns;
  if (threadIdx.x == 0) {
    mbar_init(&bb.x_full, 1);
    mbar_init(&bb.x_free, 1);
    mbar_init(&bb.y_full, 1);
    mbar_init(&bb.y_free, 2 * kGemmEpiWarps);
    for (int i = 0; i < p.ring; ++i) {
      mbar_init(&bb.in_full[i], 1);
      mbar_init(&bb.in_free[i], 1);
      mbar_init(&bb.out_full[i], 1);
      mbar_init(&bb.out_free[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bb.gu_full[i], 1);
      mbar_init(&bb.h_full[i], 2 * kGemmEpiWarps);
      mbar_init(&bb.y_done[i], 1);
    }
    mbar_init(&bb.drain, 1);
    for (int i = 0; i < kGemmEpiWarps; ++i) mbar_init(&bb.res[i], 1);
    bb.abort_flag = 0;
    fence_mbarrier_init();
  }
  if (warp == kGemmTmaWarp && lane == 0) {
    tma_prefetch_desc(&tm_x);
    tma_prefetch_desc(&tm_in);
    tma_prefetch_desc(&tm_out);
  }
  cluster_sync();   // the other CTA's barriers are ready too
  if (warp == kGemmMmaWarp) pair_tmem_alloc<2>(&bb.tmem, 512);
  pdl_wait();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bb.tmem;   // y at 0, GU (and h over it) at 256 and 384

  if (warp == kGemmTmaWarp) {
    // ---------------------------------------------------------- TMA producer
    // Both CTAs load their halves; CTA 0's barriers count all bytes.
    if (lane == 0) {
      bool ok = true;
      int st = 0, g = 0, t = 0;   // ring slot, chunks and tiles loaded so far
      uint32_t ph = 1;
      const uint32_t half = fused_cols(p.C) / 2;
      for (; ok && t < tiles; ++t) {
        const int row = 256 * (pair + t * pairs) + 128 * rank;
        if (t > 0 && !(ok = mbar_wait(&bb.x_free, (t - 1) & 1, ab, lim, SITE_FUSED))) break;
        if (rank == 0) mbar_arrive_expect_tx(&bb.x_full, 2 * x_bytes);
        const uint32_t bx = cluster_addr(&bb.x_full, 0);
        for (int k = 0; k < p.k_steps; ++k)
          tma_load_2d_pair(s_x + k * kGemmATile, &tm_x, bx, 64 * k, row);
        for (int c = 0; c < p.chunks; ++c, ++g) {
          if (g >= p.ring && !(ok = mbar_wait(&bb.in_free[st], ph, ab, lim, SITE_FUSED))) break;
          if (rank == 0) mbar_arrive_expect_tx(&bb.in_full[st], 2 * in_bytes);
          const uint32_t bi = cluster_addr(&bb.in_full[st], 0);
          for (int k = 0; k < p.k_steps; ++k)   // CTA 0: the gate's rows, CTA 1: the other's
            tma_load_2d_pair(s_in + st * in_bytes + k * 8192, &tm_in, bi, 64 * k,
                             rank * p.H + 64 * c);
          if (g >= p.ring && !(ok = mbar_wait(&bb.out_free[st], ph, ab, lim, SITE_FUSED))) break;
          if (rank == 0) mbar_arrive_expect_tx(&bb.out_full[st], 2 * out_bytes);
          tma_load_2d_pair(s_out + st * out_bytes, &tm_out, cluster_addr(&bb.out_full[st], 0),
                           64 * c, rank * half);
          if (++st == p.ring) {
            st = 0;
            ph ^= 1;
          }
        }
      }
    }
  } else if (warp == kGemmMmaWarp) {
    // ---------------------------------------------------------- MMA issue
    if (rank == 0) {
      const uint32_t id_gu = make_idesc_bf16(256, 128, false, false);
      const uint32_t id_y = make_idesc_bf16(256, fused_cols(p.C), false, false);
      const int last_c = (p.C - 64 * (p.k_steps - 1) + 15) / 16;
      const int last_h = (p.H - 64 * (p.chunks - 1) + 15) / 16;
      const int total = tiles * p.chunks;
      bool ok = true;
      int st_in = 0, st_out = 0;
      uint32_t ph_in = 0, ph_out = 0;
      RingWait ring;
      // y += h Wo^T of chunk g
      auto issue_y = [&](int g, int c, int t) {
        if (c == 0 && t > 0 && !(ok = warp_wait(&bb.y_free, (t - 1) & 1, ab, lim, SITE_FUSED))) return;
        if (!(ok = warp_wait(&bb.out_full[st_out], ph_out, ab, lim, SITE_FUSED))) return;
        if (!(ok = warp_wait(&bb.h_full[g & 1], (g >> 1) & 1, ab, lim, SITE_FUSED))) return;
        tc_fence_after();
        pair_umma_ts_steps(c + 1 == p.chunks ? last_h : 4, tmem, tmem + 256 + 128 * (g & 1),
                           make_sdesc(smem_u32(s_out + st_out * out_bytes), 16, 1024, kLayoutSW128),
                           2, id_y, c > 0 ? 1u : 0u);
        pair_commit<2>(&bb.y_done[g & 1]);
        pair_commit<2>(&bb.out_free[st_out]);
        if (c + 1 == p.chunks) pair_commit<2>(&bb.y_full);
        if (++st_out == p.ring) {
          st_out = 0;
          ph_out ^= 1;
        }
      };
      int c = 0, t = 0, c_y = 0, t_y = 0;   // chunk and tile of the next GU and Y
      for (int g = 0; ok && g <= total; ++g) {
        if (g < total) {
          if (c == 0 && !(ok = warp_wait(&bb.x_full, t & 1, ab, lim, SITE_FUSED))) break;
          if (!(ok = ring.wait(&bb.in_full[st_in], ph_in, ab, lim, SITE_FUSED))) break;
          // Y(g - 2) has read h from the columns (and the epilogue has left them)
          if (g >= 2 && !(ok = warp_wait(&bb.y_done[g & 1], ((g >> 1) - 1) & 1, ab, lim, SITE_FUSED)))
            break;
          tc_fence_after();
          const uint32_t sa = smem_u32(s_x), sb = smem_u32(s_in + st_in * in_bytes);
          for (int k = 0; k < p.k_steps; ++k)
            pair_umma_steps<2>(k + 1 == p.k_steps ? last_c : 4, tmem + 256 + 128 * (g & 1),
                               make_sdesc(sa + k * kGemmATile, 16, 1024, kLayoutSW128), 2,
                               make_sdesc(sb + k * 8192, 16, 1024, kLayoutSW128), 2, id_gu,
                               k > 0 ? 1u : 0u);
          pair_commit<2>(&bb.gu_full[g & 1]);
          pair_commit<2>(&bb.in_free[st_in]);
          if (++c == p.chunks) {
            pair_commit<2>(&bb.x_free);
            c = 0;
            ++t;
          }
          if (++st_in == p.ring) {
            st_in = 0;
            ph_in ^= 1;
          }
          ring.peek(&bb.in_full[st_in], ph_in);
        }
        if (g > 0) {
          issue_y(g - 1, c_y, t_y);
          if (++c_y == p.chunks) {
            c_y = 0;
            ++t_y;
          }
        }
      }
      pair_commit<2>(&bb.drain);
      volatile int no_abort = 0;
      mbar_wait(&bb.drain, 0, &no_abort, 200000000ull, SITE_FUSED);
    }
  } else {
    // ---------------------------------------------------------- epilogue
    // warp w: rows 32 (w % 4) .. of the CTA's 128; of a chunk the 16 hidden
    // channels of its group w / 4, of y the units of 32 columns that come to
    // its group in turn
    const int quarter = warp & 3, group = warp >> 2;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    uint8_t* sg = s_stage + warp * kGemmUnit;
    auto cell = [&](int q) {   // granule q of this lane's row
      return reinterpret_cast<uint4*>(sg + lane * 64 + ((q ^ ((lane >> 1) & 3)) << 4));
    };
    auto to_leader = [&](uint64_t* bar) {
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(cluster_addr(bar, 0));
    };
    const int units = (p.C + 31) / 32;   // of y; at most two come to a group
    bool ok = true;
    // The row tile whose y is being finished: its rows, the next unit (none at
    // `units` or beyond) and whether that unit's residual is on its way.
    int y_row = 0, y_unit = units, turn = 0;
    uint32_t res_ph = 0;
    bool res_ahead = false;
    auto start_res = [&]() {
      if (!RES || y_unit >= units || y_row >= p.M || res_ahead) return;
      res_ahead = true;
      if (lane == 0) {
        tma_store_wait_read_all();   // the last store has read the buffer
        mbar_arrive_expect_tx(&bb.res[warp], kGemmUnit);
        tma_load_2d(sg, &tm_res, &bb.res[warp], 32 * y_unit, y_row);
      }
    };
    // the next unit of y
    auto finish_unit = [&]() {
      const int u = y_unit;
      const bool in = y_row < p.M;
      start_res();
      if (RES && in) {
        if (!(ok = warp_wait(&bb.res[warp], res_ph, ab, lim, SITE_FUSED))) return;
        res_ph ^= 1;
        res_ahead = false;
      }
      y_unit += 4;
      uint32_t out[16];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t v[16];
        tmem_ld_x16(tmem + lane_off + 32 * u + 16 * h, v);
        float4 b[4];
        bias16(p.b_out, 32 * u + 16 * h, p.C, b);
        tmem_wait_ld();
        reg_fence_x16(v);
        if (h == 1 && y_unit >= units) {   // this warp's columns of y are read
          tc_fence_before();
          to_leader(&bb.y_free);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          auto f = [](uint32_t x) { return __uint_as_float(x); };
          uint64_t z01 = fadd2(pk2(f(v[4 * e]), f(v[4 * e + 1])), pk2(b[e].x, b[e].y));
          uint64_t z23 = fadd2(pk2(f(v[4 * e + 2]), f(v[4 * e + 3])), pk2(b[e].z, b[e].w));
          if constexpr (RES) {
            const uint2 r = *(reinterpret_cast<const uint2*>(cell(2 * h + (e >> 1))) + (e & 1));
            z01 = fadd2(z01, pk2(f(r.x << 16), f(r.x & 0xffff0000u)));
            z23 = fadd2(z23, pk2(f(r.y << 16), f(r.y & 0xffff0000u)));
          }
          out[8 * h + 2 * e] = pack_bf16x2(lo2(z01), hi2(z01));
          out[8 * h + 2 * e + 1] = pack_bf16x2(lo2(z23), hi2(z23));
        }
      }
      if (!in) return;
      if (!RES && lane == 0) tma_store_wait_read_all();
      __syncwarp();
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *cell(q) = make_uint4(out[4 * q], out[4 * q + 1], out[4 * q + 2], out[4 * q + 3]);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        tma_store_2d(&tm_y, sg, 32 * u, y_row);
        tma_store_commit();
      }
    };
    const int total = tiles * p.chunks;
    int c = 0, t = 0;
    // one step more than there are chunks: the last tile's y
    for (int g = 0; ok && g <= total; ++g) {
      start_res();   // of a second unit, the first one's store has long been read
      if (g < total) {
        const int col = 64 * c + 16 * group;
        const uint32_t acc = tmem + 256 + 128 * (g & 1) + lane_off + 16 * group;
        float4 bg[4], bu[4];
        bias16(p.b_in, col, p.H, bg);
        bias16(p.b_in ? p.b_in + p.H : nullptr, col, p.H, bu);
        if (!(ok = warp_wait(&bb.gu_full[g & 1], (g >> 1) & 1, ab, lim, SITE_FUSED))) break;
        tc_fence_after();
        uint32_t v[16], w[16], out[8];
        tmem_ld_x16(acc, v);
        tmem_ld_x16(acc + 64, w);
        tmem_wait_ld();
        reg_fence_x16(v);
        reg_fence_x16(w);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          auto f = [](uint32_t x) { return __uint_as_float(x); };
          uint64_t z01 = fadd2(pk2(f(v[4 * e]), f(v[4 * e + 1])), pk2(bg[e].x, bg[e].y));
          uint64_t z23 = fadd2(pk2(f(v[4 * e + 2]), f(v[4 * e + 3])), pk2(bg[e].z, bg[e].w));
          act_quad<ACT>(z01, z23);
          z01 = fmul2(z01, fadd2(pk2(f(w[4 * e]), f(w[4 * e + 1])), pk2(bu[e].x, bu[e].y)));
          z23 = fmul2(z23, fadd2(pk2(f(w[4 * e + 2]), f(w[4 * e + 3])), pk2(bu[e].z, bu[e].w)));
          // beyond H the gate's columns are the other projection's: h is zero
          const bool in = col + 4 * e < p.H;
          out[2 * e] = in ? pack_bf16x2(lo2(z01), hi2(z01)) : 0u;
          out[2 * e + 1] = in ? pack_bf16x2(lo2(z23), hi2(z23)) : 0u;
        }
        tmem_st_x8(acc, out);
        tmem_wait_st();
        tc_fence_before();
        to_leader(&bb.h_full[g & 1]);
      }
      // a unit of the previous tile's y behind each of this tile's first
      // chunks, all that is left behind the last chunk
      if (c == 0 && g > 0) {
        if (!(ok = warp_wait(&bb.y_full, (t - 1) & 1, ab, lim, SITE_FUSED))) break;
        tc_fence_after();
        if (y_unit >= units) to_leader(&bb.y_free);   // no unit for this warp
      }
      if (g > 0 && y_unit < units) finish_unit();
      const bool last = c + 1 == p.chunks || g == total;
      while (ok && last && g > 0 && t > 0 && y_unit < units) finish_unit();
      if (!ok) break;
      if (c + 1 == p.chunks && g < total) {   // this tile's y comes next
        y_row = 256 * (pair + t * pairs) + 128 * static_cast<int>(rank) + 32 * quarter;
        y_unit = (group - turn) & 3;
        turn = (turn + units) & 3;
        start_res();
      }
      if (++c == p.chunks) {
        c = 0;
        ++t;
      }
    }
    if (RES && res_ahead && lane == 0) {   // after a failure: the load in flight lands first
      volatile int no_abort = 0;
      mbar_wait(&bb.res[warp], res_ph, &no_abort, 200000000ull, SITE_FUSED);
    }
    if (lane == 0) tma_store_wait_all();
  }
  tc_fence_before();
  __syncthreads();
  settle(ab);
  cluster_sync();
  if (warp == kGemmMmaWarp) {
    tc_fence_after();
    pair_tmem_dealloc<2>(tmem, 512);
  }
}

}  // namespace rib
