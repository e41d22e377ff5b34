// layer_api.cuh -- entry points of the layer's other operators: layer norm,
// linear projections, the gated feed-forward block (include/rib.h).  Host
// side only: validation, launch shapes, tensor maps, workspace carving.
// Included once, at the end of rib.cu, whose helpers it uses.
#pragma once

#include <algorithm>
#include <initializer_list>

#include "layer_norm.cuh"
#include "gemm.cuh"
#include "ffn.cuh"
#include "few_rows.cuh"
#include "ffn_fused.cuh"

namespace rib {
namespace {

// ---------------------------------------------------------------- launches

// Launches a kernel that calls pdl_wait(), optionally in clusters.
template <typename... Args>
int launch(void (*kernel)(Args...), dim3 grid, int block, size_t smem, cudaStream_t st, int cluster,
           Args... args) {
  cudaLaunchAttribute attr[2] = {};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  if (cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess) return RIB_OK;
  cudaGetLastError();
  return RIB_ERR_CUDA;
}

// ---------------------------------------------------------------- shapes

constexpr int kMaxChannels = 65536;
constexpr int kMaxRows = 1 << 30;

int check_product(int rows, int K, int N) {
  if (rows < 0 || K <= 0 || N <= 0) return RIB_ERR_ARG;
  if (K % 8 || N % 8 || K > kMaxChannels || N > kMaxChannels || rows > kMaxRows)
    return RIB_ERR_UNSUPPORTED;
  return RIB_OK;
}

int check_act(int act) {
  return act == RIB_ACT_NONE || act == RIB_ACT_GELU || act == RIB_ACT_SILU ? RIB_OK : RIB_ERR_ARG;
}

int div_up(long long a, long long b) { return static_cast<int>((a + b - 1) / b); }

// How many items the row tiles of one column tile are dealt to: the count
// with the fewest tiles on the busiest CTA, the smallest such (fewer items
// reload fewer weights), at most 2 sms.  Only the most items that finish in
// 1, 2, ... rounds can be best, and of those the fewest with as few row tiles
// each: a search over every count took 9 of 18 us of a call on the host.
int pick_splits(int m_tiles, int n_tiles, int sms) {
  const int most = std::min(m_tiles, 2 * sms);
  int best = 1;
  long long best_cost = -1;
  for (int rounds = div_up(n_tiles, sms);; ++rounds) {
    const int s = static_cast<int>(std::min<long long>(most, (long long)rounds * sms / n_tiles));
    const int per = div_up(m_tiles, s);
    const long long cost = (long long)div_up((long long)n_tiles * s, sms) * per;
    if (best_cost < 0 || cost < best_cost) {
      best_cost = cost;
      best = div_up(m_tiles, per);
    }
    if (s == most) return best;
  }
}

struct GemmPlan {
  int cg, bn, a_rows, m_tiles, n_tiles, splits, k_steps, stages, grid;
  bool resident;
  size_t smem;
};

GemmPlan plan_gemm(int mode, int M, int N, int K, bool res, int sms) {
  GemmPlan g{};
  g.k_steps = div_up(K, 64);
  const bool gated = mode == kGated;
  const int unit = gated ? 128 : 64;             // bn is a multiple of this
  const int cols = gated ? 2 * N : N;
  // One CTA or a pair per tile, and the tile width: the least work on the
  // busiest worker, tiles times a tile's cost, its columns plus a fixed part
  // (the x rows that every column tile reads again, the pipeline's ends) worth
  // about 48 columns.  A pair, whose MMA shares B, runs a tile better the more
  // k-steps it has: 147456 x 384 -> 192 33 us (one CTA: 38), 8192 x 4096 -> 4096
  // with a residual 197 us (229), 5003 x 1032 -> 2056 28.4 us (34.6); at three
  // k-steps its longer hand-over costs more than that (147456 x 192 -> 576
  // 46.2 us, one CTA 42.7).
  long long best = -1;
  for (int cg = 1; cg <= 2; ++cg) {
    if (cg == 2 && M <= 128) break;
    const int m_tiles = div_up(M, 128 * cg), workers = sms / cg;
    for (int bn = unit; bn <= 256; bn += unit) {
      const int n_tiles = div_up(cols, bn), splits = pick_splits(m_tiles, n_tiles, workers);
      const long long cost = (long long)div_up((long long)n_tiles * splits, workers) *
                             div_up(m_tiles, splits) * (bn + (cg == 1 ? 48 : 24 + 120 / g.k_steps));
      if (best < 0 || cost < best) {
        best = cost;
        g.cg = cg;
        g.bn = bn;
        g.m_tiles = m_tiles;
        g.n_tiles = n_tiles;
        g.splits = splits;
      }
    }
  }
  g.grid = std::min(g.n_tiles * g.splits, sms / g.cg) * g.cg;
  // a lone row tile of few rows is loaded as such
  g.a_rows = g.cg == 1 && M < 128 ? div_up(M, 8) * 8 : 128;
  const size_t b = gemm_b_bytes(mode, g.cg, g.bn);
  const size_t room = kSmemMax - gemm_smem_bytes(0, 0, 0, false, res);
  // weights stay in shared memory over an item's row tiles when at least
  // four stages of x still fit beside them
  g.resident = g.m_tiles >= 2 * g.splits && g.k_steps * b + 4 * kGemmATile <= room;
  const size_t left = room - (g.resident ? g.k_steps * b : 0);
  g.stages = static_cast<int>(left / (kGemmATile + (g.resident ? 0 : b)));
  if (g.stages > kGemmMaxStages) g.stages = kGemmMaxStages;
  g.smem = gemm_smem_bytes((uint32_t)b, g.stages, g.k_steps, g.resident, res);
  return g;
}

// bf16 [rows][cols] as a 2-D map with boxes of box_cols x box_rows
int map_2d(CUtensorMap* m, const void* base, uint64_t rows, uint64_t cols, uint32_t box_cols,
           uint32_t box_rows, CUtensorMapSwizzle sw = CU_TENSOR_MAP_SWIZZLE_128B) {
  const uint64_t dims[2] = {cols, rows};
  const uint64_t strides[1] = {2 * cols};
  const uint32_t box[2] = {box_cols, box_rows};
  return make_map(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base, dims, strides, box, sw);
}

template <int MODE, int ACT, bool RES, bool PRE, int CG>
int launch_gemm_as(int kid, const GemmPlan& g, const void* a, const void* b, const float* bias,
                const void* residual, void* pre, void* y, int M, int N, int K, cudaStream_t st) {
  CUtensorMap ta, tb, ty, tp, tr;
  int rc = map_2d(&ta, a, M, K, 64, g.a_rows);
  if (!rc)
    rc = MODE == kLinear ? map_2d(&tb, b, N, K, 64, g.bn / CG)
         : MODE == kGated ? map_2d(&tb, b, 2ull * N, K, 64, g.bn / 2)
                          : map_2d(&tb, b, K, N, 64, 64);
  if (!rc) rc = map_2d(&ty, y, M, N, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B);
  if (!rc) rc = map_2d(&tp, pre ? pre : y, M, N, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B);
  if (!rc)
    rc = map_2d(&tr, residual ? residual : y, M, N, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B);
  if (rc) return rc;
  GemmParams p{};
  p.bias = bias;
  p.M = M; p.N = N; p.K = K;
  p.bn = g.bn;
  p.m_tiles = g.m_tiles; p.n_tiles = g.n_tiles; p.splits = g.splits;
  p.a_bytes = 128u * g.a_rows;
  p.k_steps = g.k_steps; p.stages = g.stages; p.b_resident = g.resident;
  p.wait_limit_ns = g_wait_limit_ns;
  auto kernel = gemm_kernel<MODE, ACT, RES, PRE, CG>;
  if ((rc = set_smem(kernel, g.smem))) return rc;
  TraceScope ts(kid, st);
  return launch(kernel, dim3(g.grid), kGemmThreads, g.smem, st, CG, ta, tb, ty, tp, tr, p);
}

// The epilogue's optional reads and writes are template arguments: an absent
// one costs no instructions.
template <int MODE, int ACT>
int launch_gemm(int kid, const GemmPlan& g, const void* a, const void* b, const float* bias,
                const void* residual, void* pre, void* y, int M, int N, int K, cudaStream_t st) {
#define RIB_GEMM(res, save)                                                                       \
  return g.cg == 2 ? launch_gemm_as<MODE, ACT, res, save, 2>(kid, g, a, b, bias, residual, pre, y, \
                                                             M, N, K, st)                         \
                   : launch_gemm_as<MODE, ACT, res, save, 1>(kid, g, a, b, bias, residual, pre, y, \
                                                             M, N, K, st)
  if constexpr (MODE == kLinear) {
    if (residual && pre) RIB_GEMM(true, true);
    if (pre) RIB_GEMM(false, true);
  }
  if constexpr (MODE != kGated) {
    if (residual) RIB_GEMM(true, false);
  }
  RIB_GEMM(false, false);
#undef RIB_GEMM
}

template <int MODE>
int launch_gemm_act(int act, int kid, const GemmPlan& g, const void* a, const void* b,
                    const float* bias, const void* residual, void* pre, void* y, int M, int N,
                    int K, cudaStream_t st) {
  switch (act) {
    case RIB_ACT_GELU:
      return launch_gemm<MODE, kActGelu>(kid, g, a, b, bias, residual, pre, y, M, N, K, st);
    case RIB_ACT_SILU:
      return launch_gemm<MODE, kActSilu>(kid, g, a, b, bias, residual, pre, y, M, N, K, st);
    default:
      return launch_gemm<MODE, kActNone>(kid, g, a, b, bias, residual, pre, y, M, N, K, st);
  }
}

// ---------------------------------------------------------------- few rows

// One or two rows are a read of the weights (1024 -> 4096: 2.9 us for one row,
// 9.7 on the tensor cores; 4096 -> 4096: 21 us for two, 27); more rows cost
// this kernel fp32 work in proportion: four of 1024 -> 4096 take 6.0 us (9.9),
// four of 4096 -> 4096 35.8 us (27.5), eight of 4096 -> 1024 29 us (24).
bool few_rows_win(int rows, int K, int N) {
  return rows <= 2 || (rows <= kFewRows && (long long)rows * K * N <= 1ll << 24);
}

template <int ACT, bool GATED, bool X32>
int launch_few_as(const FewParams& p, cudaStream_t st) {
  const int per_block = kFewThreads / 32 * (GATED ? 1 : 2);
  const int grid = div_up(p.N, per_block);
  TraceScope ts(K_FEW_ROWS, st);
  auto kernel = p.rows == 1   ? few_rows_kernel<1, ACT, GATED, X32>
                : p.rows == 2 ? few_rows_kernel<2, ACT, GATED, X32>
                : p.rows <= 4 ? few_rows_kernel<4, ACT, GATED, X32>
                              : few_rows_kernel<8, ACT, GATED, X32>;
  return launch(kernel, dim3(grid), kFewThreads, 0, st, 1, p);
}

FewParams few_params(const void* x, const void* w, const float* bias, const void* residual, void* pre,
                     void* y, int rows, int N, int K) {
  FewParams p{};
  p.x = x;
  p.w = static_cast<const __nv_bfloat16*>(w);
  p.residual = static_cast<const __nv_bfloat16*>(residual);
  p.bias = bias;
  p.pre = static_cast<__nv_bfloat16*>(pre);
  p.y = y;
  p.rows = rows; p.K = K; p.N = N;
  return p;
}

template <bool GATED>
int launch_few(int act, const FewParams& p, cudaStream_t st) {
  return act == RIB_ACT_GELU   ? launch_few_as<kActGelu, GATED, false>(p, st)
         : act == RIB_ACT_SILU ? launch_few_as<kActSilu, GATED, false>(p, st)
                               : launch_few_as<kActNone, GATED, false>(p, st);
}

struct DwPlan {
  int a_chunks, b_chunks, stages, m_tiles, n_tiles, splits, steps, per_split;
  size_t part, part_db;   // bytes
};

// dW [N][K] over `rows` rows: the tile's height (the one that divides N best)
// and the number of row ranges.  More ranges shorten the rows' loop and
// lengthen the sum of the partials; the estimate of both that is minimised
// takes 0.15 us per 8 KB atom loaded (or the MMAs' 0.32 us per 64 rows and
// accumulator, if longer) and 4 TB/s for partials written and read.
DwPlan plan_dw(int rows, int N, int K, int sms) {
  DwPlan d{};
  d.steps = div_up(rows, 64);
  d.b_chunks = std::min(kDwBn / 64, div_up(K, 64));
  d.n_tiles = div_up(K, 64 * d.b_chunks);
  const unsigned most = d.steps;
  double best = -1.0;
  for (int ac = 2; ac <= 4; ++ac) {
    const int m_tiles = div_up(N, 64 * ac);
    const long long tiles = (long long)m_tiles * d.n_tiles;
    const double step = std::max(0.15 * (ac + d.b_chunks), 0.32 * (ac > 2 ? 2 : 1));
    for (unsigned s = 1; s <= most && (s == 1 || tiles * s <= 2ll * sms); ++s) {
      const unsigned per = (most + s - 1) / s;   // 32 bits: the divisions are the loop's time
      const double cost = (static_cast<unsigned>(tiles * s) + sms - 1) / sms * (per + 4) * step +
                          (s > 1 ? 2.0 + (double)s * N * K * 8.0 / 4.0e6 : 0.0);
      if (best < 0 || cost < best) {
        best = cost;
        d.a_chunks = ac;
        d.m_tiles = m_tiles;
        d.per_split = per;
        d.splits = div_up(d.steps, per);   // no empty range
      }
    }
  }
  d.stages = std::min<int>(kDwMaxStages, (kSmemMax - dw_smem_bytes(0, 0, 0)) /
                                             dw_stage_bytes(d.a_chunks, d.b_chunks));
  d.part = d.splits > 1 ? align256((size_t)d.splits * N * K * 4) : 0;
  d.part_db = align256((size_t)d.splits * N * 4);
  return d;
}

// dW = dz^T x (fp32, or bf16) and, with db, its column sums.
int launch_dw_reduce(const float* part, int splits, size_t n4, const float* part_db, int db_splits,
                     size_t nb4, float* out32, __nv_bfloat16* out16, float* db, cudaStream_t st) {
  TraceScope ts(K_DW_RED, st);
  return launch(dw_reduce_kernel, dim3(div_up(nb4, 16) + div_up(n4, 64)), 256, 0, st, 1, part,
                part_db, splits, db_splits, n4, nb4, out32, out16, db);
}

// db_rows: the partials of db that part_db holds already, or 0: the product
// forms them
int launch_dw(const DwPlan& d, const void* dz, const void* x, int rows, int N, int K, void* dw,
              int dw_dtype, float* db, void* part, void* part_db, int db_rows, cudaStream_t st) {
  CUtensorMap tz, tx;
  int rc = map_2d(&tz, dz, rows, N, 64, 64);
  if (!rc) rc = map_2d(&tx, x, rows, K, 64, 64);
  if (rc) return rc;
  const bool f32 = dw_dtype == RIB_DTYPE_F32, direct = d.splits == 1;
  DwParams p{};
  p.rows = rows; p.N = N; p.K = K;
  p.a_chunks = d.a_chunks; p.b_chunks = d.b_chunks;
  p.m_tiles = d.m_tiles; p.n_tiles = d.n_tiles; p.splits = d.splits; p.stages = d.stages;
  p.steps = d.steps; p.steps_per_split = d.per_split;
  float* out = static_cast<float*>(direct ? (f32 ? dw : nullptr) : part);
  CUtensorMap tp = tz;   // not looked at without `out`
  if (out) {
    const uint64_t dims[3] = {(uint64_t)K, (uint64_t)N, (uint64_t)d.splits};
    const uint64_t strides[2] = {4ull * K, 4ull * N * K};
    const uint32_t box[3] = {32, 32, 1};
    if ((rc = make_map(&tp, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, out, dims, strides, box,
                       CU_TENSOR_MAP_SWIZZLE_128B)))
      return rc;
  }
  p.part = out != nullptr;
  p.out16 = direct && !f32 ? static_cast<__nv_bfloat16*>(dw) : nullptr;
  p.part_db = !db || db_rows ? nullptr : direct ? db : static_cast<float*>(part_db);
  p.wait_limit_ns = g_wait_limit_ns;
  const size_t smem = dw_smem_bytes(d.a_chunks, d.b_chunks, d.stages);
  if ((rc = set_smem(dw_kernel, smem))) return rc;
  {
    TraceScope ts(K_DW, st);
    rc = launch(dw_kernel, dim3(d.m_tiles * d.n_tiles * d.splits), kDwThreads, smem, st, 1, tz, tx, tp,
                p);
    if (rc) return rc;
  }
  const size_t n4 = direct ? 0 : (size_t)N * K / 4, nb4 = db && (db_rows || !direct) ? N / 4 : 0;
  if (n4 + nb4 == 0) return rc;
  return launch_dw_reduce(out, d.splits, n4, static_cast<const float*>(part_db),
                          db_rows ? db_rows : d.splits, nb4, f32 ? static_cast<float*>(dw) : nullptr,
                          f32 ? nullptr : static_cast<__nv_bfloat16*>(dw), db, st);
}

int launch_reduce_rows(const float* part, int rows, int n0, float* out0, int n1, float* out1,
                       cudaStream_t st) {
  TraceScope ts(K_ROWS_RED, st);
  return launch(reduce_rows_kernel, dim3(div_up(n0 + n1, 32)), kLnThreads, 0, st, 1, part, rows,
                n0, out0, n1, out1);
}

bool aligned16_all(std::initializer_list<const void*> ptrs) {
  for (const void* q : ptrs)
    if (!aligned16(q)) return false;
  return true;
}

// ---------------------------------------------------------------- overlaps

struct Span {
  const void* p;   // may be null
  size_t bytes;
};

bool overlap(const Span& a, const Span& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x && y && x < y + b.bytes && y < x + a.bytes;
}
// An output on memory that the call still reads or writes otherwise.
bool clash(const Span& out, std::initializer_list<Span> others) {
  for (const Span& o : others)
    if (overlap(out, o)) return true;
  return false;
}
// The same where the output may take the other's place, element for element.
bool clash_unless_same(const Span& out, std::initializer_list<Span> others) {
  for (const Span& o : others)
    if (out.p != o.p && overlap(out, o)) return true;
  return false;
}

// ---------------------------------------------------------------- layer norm

// How one call runs: the asynchronous kernel's vector width, vectors per
// lane, lanes per row and block, or (lanes == 0) a row kernel; and the grid,
// which is also the number of dgamma / dbeta partials.
struct LnPlan {
  int vec, nv, lanes, grid;
  LnBlocks q;
  size_t smem;
};

LnPlan plan_ln(int rows, int C, int es, bool bwd, bool aligned, int sms) {
  LnPlan n{};
  const int arrays = bwd ? 3 : 1;   // also without dres: the sums then run in the same order
  const int v = 16 / es;
  n.vec = aligned && C % v == 0 ? v : 1;
  // (also the backward of more than 768 single elements of bf16, though it spills:
  // 60000 x 777 204 us, by the row kernels 419; x 1001 259 for 508; of fp32 up to
  // 780, where the stages still fit, 777 227 for 313)
  if (aligned && C <= 1024) {
    const int vecs = C / n.vec;
    // as few lanes per row as keep four vectors (or pairs of single elements) a
    // lane (backward of 122931 x 10 15 us, with all 32 lanes 72; x 100 57 for 77)
    if (n.vec == 1) {
      n.lanes = vecs <= 64 ? 8 : vecs <= 128 ? 16 : 32;
      n.nv = div_up(vecs, 2 * n.lanes);
      n.nv = n.nv <= 2 && n.lanes == 8 ? 2
             : n.nv <= 4                ? 4
             : n.nv <= 8                ? (n.nv + 1) / 2 * 2
                                        : (n.nv + 3) / 4 * 4;
    } else {
      n.lanes = vecs <= 16 ? 4 : vecs <= 32 ? 8 : vecs <= 64 ? 16 : 32;
      n.nv = div_up(vecs, n.lanes);
      if (n.nv > 4) n.nv = n.nv <= 8 ? 8 : 16;
    }
    // A block: whole groups of rows, 32 rows at most (a lane holds a row's
    // statistics).  Measured at 192 channels of bf16: the forward
    // is best at four rows (1.5 KB; 40.0 us for 294912 rows, 44 at sixteen), the
    // backward at eight (3 KB of each array; 42 us with the sums for 147456
    // rows, 56 at four: its fixed work per block is larger).
    // single elements: two groups of rows interleaved
    const int unit = 32 / n.lanes * (n.vec == 1 ? 2 : 1);
    n.q.rows = std::min(std::max(1, (bwd ? 9216 : 2048) / (arrays * unit * C * es)) * unit, 32);
    n.q.bytes = (n.q.rows * C * es + (n.vec == 1 ? 32 : 0) + 127) & ~127;
    const size_t weights = ((bwd ? 1 : 2) * 4 * C + 127) & ~127;
    for (n.q.stages = kLnMaxStages; n.q.stages >= 2; --n.q.stages) {
      const size_t per_warp = (size_t)n.q.stages * arrays * n.q.bytes + kLnMaxStages * 8;
      // two CTAs per SM where their stages fit
      int ctas = 2, warps = (int)std::min<size_t>(bwd ? 12 : 16, (113 * 1024 - weights) / per_warp);
      if (warps < 8) {
        ctas = 1;
        warps = (int)std::min<size_t>(bwd ? 12 : 16, (226 * 1024 - weights) / per_warp);
      }
      // at least six warps, and room for their dgamma / dbeta sums
      if (warps < 6 || (bwd && per_warp < 8u * C)) continue;
      // few rows: more, smaller CTAs finish sooner than few full ones
      const int blocks = div_up(rows, n.q.rows);
      n.q.warps = blocks < sms * warps ? div_up(blocks, sms) : warps;
      n.smem = weights + n.q.warps * per_warp;
      n.grid = std::min(sms * ctas, div_up(blocks, n.q.warps));
      return n;
    }
  }
  n.lanes = 0;
  // a warp, or above 1024 channels a CTA, per row: a few CTAs per SM
  const long long want = C > 1024 ? rows : div_up(rows, kLnWarps);
  n.grid = static_cast<int>(std::min<long long>(want, sms * (bwd ? 2 : 8)));
  return n;
}

template <typename T, int V, int NV, bool CTA>
int ln_launch_row(const LnParams& p, const LnPlan& n, bool bwd, cudaStream_t st) {
  if (!bwd) {
    TraceScope ts(K_LN_FWD, st);
    return launch(ln_row_fwd_kernel<T, V, NV, CTA>, dim3(n.grid), kLnThreads, 0, st, 1, p);
  }
  const size_t smem = CTA || !p.part ? 0 : (size_t)kLnWarps * 2 * p.C * 4;
  int rc = set_smem(ln_row_bwd_kernel<T, V, NV, CTA>, smem, kSmemBesideStatic);
  if (rc) return rc;
  TraceScope ts(K_LN_BWD, st);
  return launch(ln_row_bwd_kernel<T, V, NV, CTA>, dim3(n.grid), kLnThreads, smem, st, 1, p);
}

template <typename T, int V, int NV, int L>
int ln_launch_async(const LnParams& p, const LnPlan& n, bool bwd, cudaStream_t st) {
  auto kernel = bwd ? ln_async_kernel<T, V, NV, L, true> : ln_async_kernel<T, V, NV, L, false>;
  int rc = set_smem(kernel, n.smem, kSmemBesideStatic);
  if (rc) return rc;
  LnBlocks q = n.q;
  q.wait_limit_ns = g_wait_limit_ns;
  TraceScope ts(bwd ? K_LN_BWD : K_LN_FWD, st);
  return launch(kernel, dim3(n.grid), 32 * q.warps, n.smem, st, 1, p, q);
}

template <typename T>
int ln_dispatch(const LnParams& p, const LnPlan& n, bool bwd, cudaStream_t st) {
  constexpr int V = 16 / sizeof(T);
#define RIB_LN(V_, NV_, L_)                             \
  if (n.vec == V_ && n.nv == NV_ && n.lanes == L_) \
  return ln_launch_async<T, V_, NV_, L_>(p, n, bwd, st)
  RIB_LN(V, 1, 4);
  RIB_LN(V, 2, 4);
  RIB_LN(V, 3, 4);
  RIB_LN(V, 4, 4);
  RIB_LN(V, 3, 8);
  RIB_LN(V, 4, 8);
  RIB_LN(V, 3, 16);
  RIB_LN(V, 4, 16);
  RIB_LN(V, 3, 32);
  RIB_LN(V, 4, 32);
  if constexpr (V == 4) {
    RIB_LN(V, 8, 32);
  }
  RIB_LN(1, 2, 8);
  RIB_LN(1, 4, 8);
  RIB_LN(1, 4, 16);
  RIB_LN(1, 4, 32);
  RIB_LN(1, 6, 32);
  RIB_LN(1, 8, 32);
  RIB_LN(1, 12, 32);
  RIB_LN(1, 16, 32);
#undef RIB_LN
  const int C = p.C;
  if (n.vec == V && C > 1024)
    return C <= 256 * V * 2 ? ln_launch_row<T, V, 2, true>(p, n, bwd, st)
                            : ln_launch_row<T, V, 32 / V, true>(p, n, bwd, st);
  if (C <= 256) return ln_launch_row<T, 1, 8, false>(p, n, bwd, st);
  if (C <= 1024) return ln_launch_row<T, 1, 32, false>(p, n, bwd, st);
  if (C <= 2048) return ln_launch_row<T, 1, 8, true>(p, n, bwd, st);
  return ln_launch_row<T, 1, 32, true>(p, n, bwd, st);
}

int ln_check(int dtype, int rows, int C) {
  if (dtype != RIB_DTYPE_BF16 && dtype != RIB_DTYPE_F32) return RIB_ERR_ARG;
  if (rows < 0 || C <= 0) return RIB_ERR_ARG;
  if (C > kLnMaxC || rows > kMaxRows) return RIB_ERR_UNSUPPORTED;
  return RIB_OK;
}

bool aligned_to(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// ---------------------------------------------------------------- workspaces

int dz_row_splits(int rows, int N, int sms) {
  const int gx = div_up(N, 256);
  const int most = std::max(1, 6 * sms / gx);
  return std::min(div_up(rows, 32), most);
}

struct LinearBwdWs {
  size_t dz, part_sum, part_dw, part_db, total;
  DwPlan dw;
  int row_splits;
};

LinearBwdWs linear_bwd_ws(int rows, int K, int N, int act, int sms) {
  LinearBwdWs w{};
  w.dw = plan_dw(rows, N, K, sms);
  w.row_splits = dz_row_splits(rows, N, sms);
  size_t off = 0;
  w.dz = off;
  off = align256(off + (act == RIB_ACT_NONE ? 0 : (size_t)rows * N * 2));
  w.part_sum = off;
  off = align256(off + (size_t)w.row_splits * N * 4);
  w.part_dw = off;
  off += w.dw.part;
  w.part_db = off;
  off += w.dw.part_db;
  w.total = off;
  return w;
}

struct FfnBwdPlan {
  int m_tiles, n_tiles, splits, k_steps, stages, grid;
  bool resident;
  size_t smem;
};

FfnBwdPlan plan_ffn_bwd(int rows, int C, int H, int sms) {
  FfnBwdPlan f{};
  f.m_tiles = div_up(rows, 128);
  f.n_tiles = div_up(H, kFfnCols);
  f.k_steps = div_up(C, 64);
  f.splits = pick_splits(f.m_tiles, f.n_tiles, sms);
  f.grid = std::min(f.n_tiles * f.splits, sms);
  const size_t room = kSmemMax - ffn_bwd_smem_bytes(0, 0, false);
  const size_t b = (size_t)f.k_steps * kFfnB;
  f.resident = f.m_tiles >= 2 * f.splits && b + 3 * kFfnA <= room;
  f.stages = static_cast<int>((room - (f.resident ? b : 0)) / (kFfnA + (f.resident ? 0 : kFfnB)));
  f.stages = std::min(f.stages, kFfnMaxStages);
  f.smem = ffn_bwd_smem_bytes(f.stages, f.k_steps, f.resident);
  return f;
}

struct FfnBwdWs {
  size_t h, d, part_sum, part_dw, part_db, total;
  FfnBwdPlan f;
  DwPlan in, out;
};

FfnBwdWs ffn_bwd_ws(int rows, int C, int H, int sms) {
  FfnBwdWs w{};
  w.f = plan_ffn_bwd(rows, C, H, sms);
  w.in = plan_dw(rows, 2 * H, C, sms);
  w.out = plan_dw(rows, C, H, sms);
  size_t off = 0;
  w.h = off;
  off = align256(off + (size_t)rows * H * 2);
  w.d = off;
  off = align256(off + (size_t)rows * H * 4);
  w.part_sum = off;
  off = align256(off + (size_t)w.f.splits * 8 * H * 4);
  w.part_dw = off;   // shared by the two weight gradients, one after the other
  off += std::max(w.in.part, w.out.part);
  w.part_db = off;
  off += w.out.part_db;
  w.total = off;
  return w;
}

int check_ffn(int rows, int C, int H) {
  int rc = check_product(rows, C, H);
  if (rc) return rc;
  return 2 * H > kMaxChannels ? RIB_ERR_UNSUPPORTED : RIB_OK;
}

int check_workspace(const void* ws, size_t bytes, size_t need) {
  if (need == 0) return RIB_OK;
  if (!ws || bytes < need) return RIB_ERR_WORKSPACE;
  return aligned_to(ws, 256) ? RIB_OK : RIB_ERR_ALIGN;
}

int zero_async(void* p, size_t bytes, cudaStream_t st) {
  return !p || cudaMemsetAsync(p, 0, bytes, st) == cudaSuccess ? RIB_OK : RIB_ERR_CUDA;
}

size_t dtype_bytes(int dtype) { return dtype == RIB_DTYPE_F32 ? 4 : 2; }

template <int ACT>
int launch_dz(const DzParams& p, int row_splits, cudaStream_t st) {
  TraceScope ts(K_DZ, st);
  return launch(dz_kernel<ACT>, dim3(div_up(p.N, 256), row_splits), 256, 0, st, 1, p);
}

template <int ACT, bool CHUNKED>
int launch_ffn_bwd_as(const FfnBwdWs& w, const void* x, const void* dy, const void* w_in,
                   const void* w_out, const FfnBwdParams& p, uint8_t* ws, cudaStream_t st) {
  CUtensorMap tx, ty, ti, to, th, td;
  int rc = map_2d(&tx, x, p.M, p.C, 64, 128);
  if (!rc) rc = map_2d(&ty, dy, p.M, p.C, 64, 128);
  if (!rc) rc = map_2d(&ti, w_in, 2ull * p.H, p.C, 64, 64);
  if (!rc) rc = map_2d(&to, w_out, p.C, p.H, 64, 64);
  if (!rc) rc = map_2d(&th, ws + w.h, p.M, p.H, 16, 32, CU_TENSOR_MAP_SWIZZLE_32B);
  if (!rc) {
    const uint64_t dims[3] = {(uint64_t)p.H, 2, (uint64_t)p.M};
    const uint64_t strides[2] = {2ull * p.H, 4ull * p.H};
    const uint32_t box[3] = {16, 1, 32};
    rc = make_map(&td, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, ws + w.d, dims, strides, box,
                  CU_TENSOR_MAP_SWIZZLE_32B);
  }
  if (rc) return rc;
  if ((rc = set_smem(ffn_bwd_kernel<ACT, CHUNKED>, w.f.smem))) return rc;
  TraceScope ts(K_FFN_BWD, st);
  return launch(ffn_bwd_kernel<ACT, CHUNKED>, dim3(w.f.grid), kFfnThreads, w.f.smem, st, 1, tx, ty, ti, to,
                th, td, p);
}

template <int ACT>
int launch_ffn_bwd(const FfnBwdWs& w, const void* x, const void* dy, const void* w_in,
                   const void* w_out, FfnBwdParams p, uint8_t* ws, cudaStream_t st) {
  if (p.k_steps <= kFfnChain) return launch_ffn_bwd_as<ACT, false>(w, x, dy, w_in, w_out, p, ws, st);
  p.piece = div_up(p.k_steps, div_up(p.k_steps, kFfnPiece));   // pieces of about the same length
  return launch_ffn_bwd_as<ACT, true>(w, x, dy, w_in, w_out, p, ws, st);
}

// ---------------------------------------------------------------- fused feed-forward

// A pair takes the same time for a row tile however few tiles there are, and
// the two products spread few rows over more SMs: one kernel wins from a tile
// per pair on (147456 rows, silu, residual: 192 x 384 86 us for 93, 192 x 768
// 142 for 165, 96 x 384 63 for 91; 102400 x 256 x 1024 152 for 168), also where
// the last round of pairs is nearly empty (75 tiles on 74 pairs, 192 x 384 22.0
// for 25.3, 192 x 768 36.0 for 38.0, 256 x 1024 50.4 for 52.7; the one size found
// where it loses is 149 tiles of 192 x 768, 52.4 for 50.7); below that where a
// tile is short (4096 x 96 x 192 8.0 for 9.8; 9216 x 192 x 384 13.3 for 15.3; 8192 x
// 128 x 512 14.0 for 15.4; but 4096 x 128 x 512 13.8 for 13.0, 2304 x 192 x 384
// 12.9 for 11.4, 8192 x 256 x 1024 27.3 for 23.1).
bool fused_wins(int rows, int C, int hidden, int sms) {
  const int tiles = div_up(rows, 256);
  return C <= kFusedMaxC && (tiles >= sms / 2 || tiles >= 3 * div_up(hidden, 64));
}

// Bytes that the forward's h takes in HBM: fp32 for a few rows, bf16 between two
// products, none in one kernel.
size_t ffn_fwd_need(int rows, int C, int hidden) {
  int sms = 0;
  if (few_rows_win(rows, C, 2 * hidden)) return align256((size_t)rows * hidden * 4);
  if (device_sms(&sms) == RIB_OK && fused_wins(rows, C, hidden, sms)) return 0;
  return align256((size_t)rows * hidden * 2);
}

template <int ACT, bool RES>
int launch_fused_as(const void* x, const void* w_in, const float* b_in, const void* w_out,
                    const float* b_out, const void* residual, void* y, int rows, int C, int H,
                    int sms, cudaStream_t st) {
  CUtensorMap tx, ti, to, ty, tr;
  int rc = map_2d(&tx, x, rows, C, 64, 128);
  if (!rc) rc = map_2d(&ti, w_in, 2ull * H, C, 64, 64);
  if (!rc) rc = map_2d(&to, w_out, C, H, 64, fused_cols(C) / 2);
  if (!rc) rc = map_2d(&ty, y, rows, C, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B);
  if (!rc) rc = map_2d(&tr, RES ? residual : y, rows, C, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B);
  if (rc) return rc;
  FusedParams p{};
  p.b_in = b_in; p.b_out = b_out;
  p.M = rows; p.C = C; p.H = H;
  p.m_tiles = div_up(rows, 256);
  p.chunks = div_up(H, 64);
  p.k_steps = div_up(C, 64);
  p.ring = kFusedMaxRing;
  while (p.ring > 2 && fused_smem_bytes(C, p.ring) > kSmemMax) --p.ring;
  p.wait_limit_ns = g_wait_limit_ns;
  const size_t smem = fused_smem_bytes(C, p.ring);
  auto kernel = ffn_fused_kernel<ACT, RES>;
  if ((rc = set_smem(kernel, smem))) return rc;
  TraceScope ts(K_FFN_FUSED, st);
  return launch(kernel, dim3(2 * std::min(p.m_tiles, sms / 2)), kGemmThreads, smem, st, 2, tx, ti,
                to, ty, tr, p);
}

template <int ACT>
int launch_fused(const void* x, const void* w_in, const float* b_in, const void* w_out,
                 const float* b_out, const void* residual, void* y, int rows, int C, int H,
                 int sms, cudaStream_t st) {
  return residual ? launch_fused_as<ACT, true>(x, w_in, b_in, w_out, b_out, residual, y, rows, C,
                                               H, sms, st)
                  : launch_fused_as<ACT, false>(x, w_in, b_in, w_out, b_out, residual, y, rows, C,
                                                H, sms, st);
}

}  // namespace
}  // namespace rib

extern "C" {

int rib_layer_norm_fwd(const void* x, int dtype, int rows, int C, const float* gamma,
                       const float* beta, float eps, void* y, float* mean, float* rstd,
                       void* stream) {
  int rc = ln_check(dtype, rows, C);
  if (rc) return rc;
  if (!(eps >= 0.f)) return RIB_ERR_ARG;
  if (rows == 0) return RIB_OK;
  if (!x || !y) return RIB_ERR_ARG;
  const uintptr_t es = dtype_bytes(dtype);
  if (!aligned_to(x, es) || !aligned_to(y, es) || !aligned_to(gamma, 4) || !aligned_to(beta, 4) ||
      !aligned_to(mean, 4) || !aligned_to(rstd, 4))
    return RIB_ERR_ALIGN;
  const size_t map = es * rows * C, row = 4ull * rows, col = 4ull * C;
  if (clash_unless_same({y, map}, {{x, map}}) || clash({y, map}, {{gamma, col}, {beta, col}}) ||
      clash({mean, row}, {{x, map}, {y, map}, {gamma, col}, {beta, col}}) ||
      clash_unless_same({mean, row}, {{rstd, row}}) ||   // one scratch buffer for both will do
      clash({rstd, row}, {{x, map}, {y, map}, {gamma, col}, {beta, col}}))
    return RIB_ERR_ARG;
  int sms = 0;
  if ((rc = device_sms(&sms))) return rc;
  LnParams p{};
  p.x = x; p.out = y; p.gamma = gamma; p.beta = beta; p.mean = mean; p.rstd = rstd;
  p.rows = rows; p.C = C; p.eps = eps;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const LnPlan n = plan_ln(rows, C, (int)es, false, aligned16_all({x, y}), sms);
  return dtype == RIB_DTYPE_BF16 ? ln_dispatch<__nv_bfloat16>(p, n, false, st)
                                 : ln_dispatch<float>(p, n, false, st);
}

size_t rib_layer_norm_bwd_workspace(int rows, int C) {
  int sms = 0;
  if (ln_check(RIB_DTYPE_BF16, rows, C) || rows == 0 || device_sms(&sms)) return 0;
  // at most two CTAs per SM leave partials, however the call runs
  return align256((size_t)std::min(2 * sms, rows) * 2 * C * 4);
}

int rib_layer_norm_bwd(const void* x, const void* dy, int dtype, int rows, int C,
                       const float* mean, const float* rstd, const float* gamma, const void* dres,
                       void* dx, float* dgamma, float* dbeta, void* workspace,
                       size_t workspace_bytes, void* stream) {
  int rc = ln_check(dtype, rows, C);
  if (rc) return rc;
  if (!aligned_to(dgamma, 4) || !aligned_to(dbeta, 4)) return RIB_ERR_ALIGN;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (rows == 0) {   // empty sums
    if ((rc = zero_async(dgamma, (size_t)C * 4, st))) return rc;
    return zero_async(dbeta, (size_t)C * 4, st);
  }
  if (!x || !dy || !mean || !rstd || !dx) return RIB_ERR_ARG;
  const uintptr_t es = dtype_bytes(dtype);
  if (!aligned_to(x, es) || !aligned_to(dy, es) || !aligned_to(dx, es) || !aligned_to(dres, es) ||
      !aligned_to(mean, 4) || !aligned_to(rstd, 4) || !aligned_to(gamma, 4))
    return RIB_ERR_ALIGN;
  const bool sums = dgamma || dbeta;
  if (sums && (rc = check_workspace(workspace, workspace_bytes,
                                    rib_layer_norm_bwd_workspace(rows, C))))
    return rc;
  const size_t map = es * rows * C, row = 4ull * rows, col = 4ull * C;
  if (clash_unless_same({dx, map}, {{x, map}, {dy, map}, {dres, map}}) ||
      clash({dx, map}, {{mean, row}, {rstd, row}, {gamma, col}, {dgamma, col}, {dbeta, col}}) ||
      clash_unless_same({dgamma, col}, {{dbeta, col}}))
    return RIB_ERR_ARG;
  int sms = 0;
  if ((rc = device_sms(&sms))) return rc;
  LnParams p{};
  p.x = x; p.dy = dy; p.dres = dres; p.out = dx; p.gamma = gamma;
  p.mean = const_cast<float*>(mean);
  p.rstd = const_cast<float*>(rstd);
  p.part = sums ? static_cast<float*>(workspace) : nullptr;
  p.rows = rows; p.C = C;
  const LnPlan n = plan_ln(rows, C, (int)es, true, aligned16_all({x, dy, dres, dx}), sms);
  rc = dtype == RIB_DTYPE_BF16 ? ln_dispatch<__nv_bfloat16>(p, n, true, st)
                               : ln_dispatch<float>(p, n, true, st);
  if (rc || !sums) return rc;
  return launch_reduce_rows(p.part, n.grid, C, dgamma, C, dbeta, st);
}

int rib_linear_fwd(const void* x, int rows, int K, const void* w, int N, const float* bias,
                   int act, const void* residual, void* pre, void* y, void* stream) {
  int rc = check_product(rows, K, N);
  if (rc || (rc = check_act(act))) return rc;
  if (rows == 0) return RIB_OK;
  if (!x || !w || !y) return RIB_ERR_ARG;
  if (!aligned16_all({x, w, bias, residual, pre, y})) return RIB_ERR_ALIGN;
  // other tiles still read x and the weights, and the residual after pre is written
  const size_t in = 2ull * rows * K, out = 2ull * rows * N, wts = 2ull * N * K, col = 4ull * N;
  if (clash({y, out}, {{x, in}, {pre, out}}) || clash_unless_same({y, out}, {{residual, out}}) ||
      clash({pre, out}, {{x, in}, {residual, out}}))
    return RIB_ERR_ARG;
  int sms = 0;
  if ((rc = device_sms(&sms))) return rc;
  if (clash({y, out}, {{w, wts}, {bias, col}}) || clash({pre, out}, {{w, wts}, {bias, col}}))
    return RIB_ERR_ARG;
  if (few_rows_win(rows, K, N))
    return launch_few<false>(act, few_params(x, w, bias, residual, pre, y, rows, N, K),
                             static_cast<cudaStream_t>(stream));
  const GemmPlan g = plan_gemm(kLinear, rows, N, K, residual != nullptr, sms);
  return launch_gemm_act<kLinear>(act, K_LINEAR, g, x, w, bias, residual, pre, y, rows, N, K,
                                  static_cast<cudaStream_t>(stream));
}

size_t rib_linear_bwd_workspace(int rows, int K, int N, int act) {
  int sms = 0;
  if (check_product(rows, K, N) || check_act(act) || rows == 0 || device_sms(&sms)) return 0;
  return linear_bwd_ws(rows, K, N, act, sms).total;
}

int rib_linear_bwd(const void* x, int rows, int K, const void* w, int N, int act, const void* pre,
                   const void* dy, const void* dx_add, void* dx, void* dw, int dw_dtype, float* db,
                   void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_product(rows, K, N);
  if (rc || (rc = check_act(act))) return rc;
  if (dw_dtype != RIB_DTYPE_BF16 && dw_dtype != RIB_DTYPE_F32) return RIB_ERR_ARG;
  if (!aligned16_all({dw, db})) return RIB_ERR_ALIGN;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (rows == 0) {   // empty sums; the maps are not looked at
    if ((rc = zero_async(dw, (size_t)N * K * dtype_bytes(dw_dtype), st))) return rc;
    return zero_async(db, (size_t)N * 4, st);
  }
  if (!aligned16_all({x, w, pre, dy, dx_add, dx})) return RIB_ERR_ALIGN;
  if (!dy || (dx && !w) || (dw && !x) || (act != RIB_ACT_NONE && !pre)) return RIB_ERR_ARG;
  const size_t in = 2ull * rows * K, out = 2ull * rows * N, wts = 2ull * N * K,
               grad = dtype_bytes(dw_dtype) * N * K, col = 4ull * N;
  // x and dy are read after dx is written
  if (clash({dx, in}, {{dy, out}, {x, in}}) || clash_unless_same({dx, in}, {{dx_add, in}}))
    return RIB_ERR_ARG;
  int sms = 0;
  if ((rc = device_sms(&sms))) return rc;
  if (clash({dx, in}, {{w, wts}}) || clash({dw, grad}, {{x, in}, {dy, out}, {dx, in}}) ||
      clash({db, col}, {{x, in}, {dy, out}, {dx, in}, {dw, grad}, {w, wts}, {dx_add, in}}))
    return RIB_ERR_ARG;
  const LinearBwdWs L = linear_bwd_ws(rows, K, N, act, sms);
  if ((rc = check_workspace(workspace, workspace_bytes, L.total))) return rc;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const void* dz = dy;
  // db comes out of the dW product where dz is dy itself; an activation's dz
  // is summed in fp32 before its rounding, in the kernel that forms it
  const bool db_in_dw = act == RIB_ACT_NONE && dw;
  if (act != RIB_ACT_NONE || (db && !db_in_dw)) {
    DzParams p{};
    p.dy = static_cast<const __nv_bfloat16*>(dy);
    p.pre = static_cast<const __nv_bfloat16*>(pre);
    p.dz = reinterpret_cast<__nv_bfloat16*>(ws + L.dz);
    p.part = db ? reinterpret_cast<float*>(ws + L.part_sum) : nullptr;
    p.rows = rows; p.N = N;
    rc = act == RIB_ACT_GELU   ? launch_dz<kActGelu>(p, L.row_splits, st)
         : act == RIB_ACT_SILU ? launch_dz<kActSilu>(p, L.row_splits, st)
                               : launch_dz<kActNone>(p, L.row_splits, st);
    if (rc) return rc;
    if (act != RIB_ACT_NONE) dz = p.dz;
    if (db && !dw)   // with dW they are added in its reduction
      if ((rc = launch_dw_reduce(nullptr, 0, 0, p.part, L.row_splits, N / 4, nullptr, nullptr, db,
                                 st)))
        return rc;
  }
  if (dx) {
    const GemmPlan g = plan_gemm(kDx, rows, K, N, dx_add != nullptr, sms);
    rc = launch_gemm<kDx, kActNone>(K_LINEAR_DX, g, dz, w, nullptr, dx_add, nullptr, dx, rows, K,
                                    N, st);
    if (rc) return rc;
  }
  if (dw)
    rc = launch_dw(L.dw, dz, x, rows, N, K, dw, dw_dtype, db, ws + L.part_dw,
                   ws + (db_in_dw ? L.part_db : L.part_sum), db_in_dw ? 0 : L.row_splits, st);
  return rc;
}

size_t rib_gated_ffn_fwd_workspace(int rows, int C, int hidden) {
  if (check_ffn(rows, C, hidden)) return 0;
  size_t need = ffn_fwd_need(rows, C, hidden);
  // at least what fewer rows need with h in fp32: a workspace for some rows serves
  // the few that run without the tensor cores
  for (int r = std::min(rows, kFewRows); need && r > 0; --r)
    if (few_rows_win(r, C, 2 * hidden)) return std::max(need, align256((size_t)r * hidden * 4));
  return need;
}

int rib_gated_ffn_fwd(const void* x, int rows, int C, int hidden, const void* w_in,
                      const float* b_in, const void* w_out, const float* b_out, int act,
                      const void* residual, void* y, void* workspace, size_t workspace_bytes,
                      void* stream) {
  int rc = check_ffn(rows, C, hidden);
  if (rc || (rc = check_act(act))) return rc;
  if (rows == 0) return RIB_OK;
  if (!x || !w_in || !w_out || !y) return RIB_ERR_ARG;
  if (!aligned16_all({x, w_in, b_in, w_out, b_out, residual, y})) return RIB_ERR_ALIGN;
  if ((rc = check_workspace(workspace, workspace_bytes, ffn_fwd_need(rows, C, hidden)))) return rc;
  const size_t map = 2ull * rows * C, wts = 2ull * hidden * C, col = 4ull * hidden;
  if (clash_unless_same({y, map}, {{x, map}, {residual, map}})) return RIB_ERR_ARG;
  int sms = 0;
  if ((rc = device_sms(&sms))) return rc;
  if (clash({y, map}, {{w_in, 2 * wts}, {b_in, 2 * col}, {w_out, wts}, {b_out, 4ull * C}}))
    return RIB_ERR_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (few_rows_win(rows, C, 2 * hidden)) {
    if ((rc = launch_few<true>(
             act, few_params(x, w_in, b_in, nullptr, nullptr, workspace, rows, hidden, C), st)))
      return rc;
    return launch_few_as<kActNone, false, true>(
        few_params(workspace, w_out, b_out, residual, nullptr, y, rows, C, hidden), st);
  }
  if (fused_wins(rows, C, hidden, sms))
    return act == RIB_ACT_GELU   ? launch_fused<kActGelu>(x, w_in, b_in, w_out, b_out, residual, y,
                                                          rows, C, hidden, sms, st)
           : act == RIB_ACT_SILU ? launch_fused<kActSilu>(x, w_in, b_in, w_out, b_out, residual, y,
                                                          rows, C, hidden, sms, st)
                                 : launch_fused<kActNone>(x, w_in, b_in, w_out, b_out, residual, y,
                                                          rows, C, hidden, sms, st);
  const GemmPlan g = plan_gemm(kGated, rows, hidden, C, false, sms);
  rc = launch_gemm_act<kGated>(act, K_GATED, g, x, w_in, b_in, nullptr, nullptr, workspace, rows,
                               hidden, C, st);
  if (rc) return rc;
  const GemmPlan o = plan_gemm(kLinear, rows, C, hidden, residual != nullptr, sms);
  return launch_gemm<kLinear, kActNone>(K_LINEAR, o, workspace, w_out, b_out, residual, nullptr, y,
                                        rows, C, hidden, st);
}

size_t rib_gated_ffn_bwd_workspace(int rows, int C, int hidden) {
  int sms = 0;
  if (check_ffn(rows, C, hidden) || rows == 0 || device_sms(&sms)) return 0;
  return ffn_bwd_ws(rows, C, hidden, sms).total;
}

int rib_gated_ffn_bwd(const void* x, int rows, int C, int hidden, const void* w_in,
                      const float* b_in, const void* w_out, int act, const void* dy,
                      const void* dx_add, void* dx, void* dw_in, float* db_in, void* dw_out,
                      float* db_out, int dw_dtype, void* workspace, size_t workspace_bytes,
                      void* stream) {
  int rc = check_ffn(rows, C, hidden);
  if (rc || (rc = check_act(act))) return rc;
  if (dw_dtype != RIB_DTYPE_BF16 && dw_dtype != RIB_DTYPE_F32) return RIB_ERR_ARG;
  if (!dw_in || !dw_out) return RIB_ERR_ARG;
  if (!aligned16_all({dw_in, db_in, dw_out, db_out})) return RIB_ERR_ALIGN;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const size_t es = dtype_bytes(dw_dtype);
  if (rows == 0) {   // empty sums; the maps are not looked at
    if ((rc = zero_async(dw_in, 2 * es * hidden * C, st))) return rc;
    if ((rc = zero_async(db_in, (size_t)hidden * 8, st))) return rc;
    if ((rc = zero_async(dw_out, es * C * hidden, st))) return rc;
    return zero_async(db_out, (size_t)C * 4, st);
  }
  if (!aligned16_all({x, w_in, b_in, w_out, dy, dx_add, dx})) return RIB_ERR_ALIGN;
  if (!x || !w_in || !w_out || !dy || !dx) return RIB_ERR_ARG;
  const size_t map = 2ull * rows * C, wts = 2ull * hidden * C, grad = es * hidden * C,
               col = 4ull * hidden;
  // x and dy are read after dx is written
  if (clash({dx, map}, {{x, map}, {dy, map}}) || clash_unless_same({dx, map}, {{dx_add, map}}))
    return RIB_ERR_ARG;
  int sms = 0;
  if ((rc = device_sms(&sms))) return rc;
  const Span maps[3] = {{x, map}, {dy, map}, {dx, map}};
  const Span sums[4] = {{dw_in, 2 * grad}, {dw_out, grad}, {db_in, 2 * col}, {db_out, 4ull * C}};
  if (clash({dx, map}, {{w_in, 2 * wts}})) return RIB_ERR_ARG;
  for (int i = 0; i < 4; ++i) {
    if (clash(sums[i], {maps[0], maps[1], maps[2]})) return RIB_ERR_ARG;
    for (int k = 0; k < i; ++k)
      if (overlap(sums[i], sums[k])) return RIB_ERR_ARG;
  }
  const FfnBwdWs L = ffn_bwd_ws(rows, C, hidden, sms);
  if ((rc = check_workspace(workspace, workspace_bytes, L.total))) return rc;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  FfnBwdParams p{};
  p.b_in = b_in;
  p.part = db_in ? reinterpret_cast<float*>(ws + L.part_sum) : nullptr;
  p.M = rows; p.C = C; p.H = hidden;
  p.m_tiles = L.f.m_tiles; p.n_tiles = L.f.n_tiles; p.splits = L.f.splits;
  p.k_steps = L.f.k_steps; p.stages = L.f.stages; p.b_resident = L.f.resident;
  p.wait_limit_ns = g_wait_limit_ns;
  rc = act == RIB_ACT_GELU   ? launch_ffn_bwd<kActGelu>(L, x, dy, w_in, w_out, p, ws, st)
       : act == RIB_ACT_SILU ? launch_ffn_bwd<kActSilu>(L, x, dy, w_in, w_out, p, ws, st)
                             : launch_ffn_bwd<kActNone>(L, x, dy, w_in, w_out, p, ws, st);
  if (rc) return rc;
  const GemmPlan g = plan_gemm(kDx, rows, C, 2 * hidden, dx_add != nullptr, sms);
  rc = launch_gemm<kDx, kActNone>(K_LINEAR_DX, g, ws + L.d, w_in, nullptr, dx_add, nullptr, dx,
                                  rows, C, 2 * hidden, st);
  if (rc) return rc;
  if ((rc = launch_dw(L.in, ws + L.d, x, rows, 2 * hidden, C, dw_in, dw_dtype, db_in,
                      ws + L.part_dw, p.part, L.f.splits * 4, st)))
    return rc;
  return launch_dw(L.out, dy, ws + L.h, rows, C, hidden, dw_out, dw_dtype, db_out, ws + L.part_dw,
                   ws + L.part_db, 0, st);
}

}  // extern "C"
