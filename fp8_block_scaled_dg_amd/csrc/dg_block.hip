// dg_block.hip -- C ABI of the transformer block's further operators (declared in
// include/dg.h): layer norm with dropout and FP8 output, the gated feed-forward product,
// dropout, and their backward passes. Argument checks, choice of a kernel form, launches.
#include <hip/hip_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <cstring>

#include "../../include/dg.h"
#include "dropout.hpp"
#include "gated_kernel.hpp"
#include "gated_ring.hpp"
#include "host.hpp"
#include "layernorm_kernel.hpp"
#include "pipe_kernel.hpp"

namespace dg {
namespace {

// ---------------------------------------------------------------- dropout

// The device's form of (p, rng, subsequence).
dg_status drop_args(double p, const int64_t* rng, int64_t subsequence, DropArgs* d) {
  if (!(p >= 0 && p <= 1)) return fail(DG_ERR_BAD_SHAPE, "dropout_p=%g is not in [0, 1)", p);
  const uint32_t threshold = (uint32_t)(65536 * p + 0.5);
  if (threshold > 65535) return fail(DG_ERR_BAD_SHAPE, "dropout_p=%g would keep nothing", p);
  if (threshold && !rng) return fail(DG_ERR_NULL_POINTER, "NULL rng");
  if (!aligned(rng, 8)) return fail(DG_ERR_MISALIGNED, "rng must be 8-byte aligned");
  *d = DropArgs{threshold ? (const uint64_t*)rng : nullptr, (uint64_t)subsequence, threshold,
                (float)(65536.0 / (65536.0 - threshold))};
  return DG_OK;
}

// ---------------------------------------------------------------- column sums in one launch
//
// Up to these sizes the backward kernels sum columns in the same launch, in further workgroups, ahead
// of the others, that read the inputs a second time. Us in a graph, so many buffers in turn that they
// come from HBM, one launch against two:
//             layer norm bf16         gated (gelu)            dropout fp32
//    130 x 2048   4.8,  6.9             6.0,  7.4               3.3,  6.0
//    257 x 2048   6.2,  7.8             8.1,  8.0               4.9,  6.2
//    512 x 2048   8.1,  9.4            11.4,  9.2               5.9,  6.8
//    700 x 2048  10.2, 10.0            13.8, 10.7               7.9,  7.6
//    130 x 7168   6.3, 11.6             6.8,  9.2               4.6,  6.7
//    257 x 7168   8.7, 12.9            10.9, 11.4               5.8,  8.2
//    512 x 7168  12.1, 17.5            17.6, 14.6               8.4,  9.9
//    700 x 7168  15.6, 19.0            20.6, 19.3              11.1, 11.9
//   1000 x 7168  21.0, 21.9            27.9, 23.2              14.3, 14.1
//    130 x 16384 14.3, 16.5            11.8, 12.1               5.9,  8.5
//    200 x 16384 15.9, 22.4            16.1, 14.9               7.9, 10.0
//    512 x 16384 27.0, 27.9            33.5, 25.0              16.4, 15.8
// (The layer norm's two launches move 8 K bytes of partials for each workgroup, 256 of them from 256
// rows on.)
constexpr int64_t kLnDirectValues = 1 << 23, kGatedDirectRows = 256, kGatedDirectValues = 1 << 21;
constexpr int64_t kDropDirectRows = 640, kDropDirectValues = 3 << 21;
int64_t ln_direct_rows(int64_t K) { return 384 + K / 16; }

// R teams of a row's threads; LDS for their sums, or for the sums of workgroups that only sum.
template <bool BF16, bool WBF, int C>
dg_status launch_layernorm_backward(const LayerNormBwdArgs& a, unsigned grid, unsigned threads,
                                    hipStream_t st) {
  const auto kernel = layernorm_backward_kernel<BF16, WBF, C>;
  constexpr bool lds_dw = kLnLdsDw<BF16, C>;
  if (lds_dw) {  // up to 128 KB, an attribute of the kernel on each device
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    const uint64_t bit = (uint64_t)1 << (dev & 63);
    if (e == hipSuccess && (dev > 63 || !(done.load() & bit))) {
      e = hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize,
                              kNormMaxK * (int)sizeof(float));
      if (e == hipSuccess && dev <= 63) done.fetch_or(bit);
    }
    if (e != hipSuccess) return fail(DG_ERR_LAUNCH, "hipFuncSetAttribute: %s", take_error(e));
  }
  size_t bytes = (size_t)(lds_dw ? a.K : (a.teams - 1) * a.K) * sizeof(float);
  const size_t direct = (size_t)threads * 2 * Pieces<BF16>::P * sizeof(float);
  if (!a.part && direct > bytes) bytes = direct;
  return launch_kernel("layernorm_backward_kernel", kernel, dim3(grid), dim3(threads), bytes, st, a);
}

// ---------------------------------------------------------------- gated product

template <class Cfg>
dg_status launch_pipe_gated(const Problem& p0, const Epilogue& ep, hipStream_t stream) {
  PipeArgs a{};
  a.p = p0;
  a.ep = ep;
  a.p.tiles_m = (int32_t)((p0.M + Cfg::BM - 1) / Cfg::BM);
  a.p.tiles_n = (int32_t)(p0.N / 256);
  int64_t grid = (int64_t)a.p.tiles_m * a.p.tiles_n;
  if (grid > 0x7FFFFFFF) return fail(DG_ERR_UNSUPPORTED_SHAPE, "grid of %lld tiles", (long long)grid);
  a.full_tiles = (int32_t)grid;
  a.parts = 1;
  const TailSplit ts = pipe_tail_split(grid, p0.K / kKBlock);
  const StreamTurn turn(stream, ts.parts > 1);
  if (ts.parts > 1) {
    const int64_t split = grid - ts.full;
    const size_t bytes = (size_t)(split * ts.parts) * Cfg::BM * Cfg::BN * sizeof(float);
    const dg_status st = get_workspace(stream, bytes, (size_t)split, &a.ws, &a.counters);
    if (st != DG_OK) return st;
    a.full_tiles = (int32_t)ts.full;
    a.parts = (int32_t)ts.parts;
    grid = ts.full + split * ts.parts;
  }
  a.items = (int32_t)grid;
  const int64_t wgs = grid < kCUs ? grid : kCUs;  // persistent, one workgroup per CU
  return launch_kernel("pipe_kernel", pipe_kernel<Cfg, kDense, false, 0, kEpiGated>, dim3((unsigned)wgs),
                       dim3(Cfg::NT), 0, stream, a);
}

constexpr int64_t kLaunchThreads = (int64_t)1 << 32;  // a launch holds fewer

template <class Cfg>
dg_status launch_gated_ring_as(const Problem& p, int64_t S, const Epilogue& ep, hipStream_t stream) {
  GatedArgs a{};
  a.p = p;
  a.ep = ep;
  a.tiles_m = (int32_t)((p.M + Cfg::BM - 1) / Cfg::BM);
  const int64_t tiles = a.tiles_m * (p.N / 256), pairs = (p.K / kKBlock + 1) / 2;
  a.S = (int32_t)S;
  a.KS = (int32_t)(2 * ((pairs + S - 1) / S));
  const int64_t grid = tiles * S;
  if (grid >= kLaunchThreads / Cfg::NT)
    return fail(DG_ERR_UNSUPPORTED_SHAPE, "grid of %lld workgroups", (long long)grid);
  const StreamTurn turn(stream, S > 1);
  if (S > 1) {
    const size_t part = (size_t)grid * 2 * Cfg::BM * 128 * sizeof(float);
    const dg_status st = get_workspace(stream, part, (size_t)tiles, &a.ws, &a.counters);
    if (st != DG_OK) return st;
  }
  return launch_kernel("gated_ring_kernel", gated_ring_kernel<Cfg>, dim3((unsigned)grid), dim3(Cfg::NT), 0,
                       stream, a);
}

template <bool PACKED, bool STREAM_B>
dg_status launch_gated_ring(int bm, int64_t S, const Problem& p, const Epilogue& ep, hipStream_t st) {
  if (bm == 16) return launch_gated_ring_as<GatedCfg<1, 1, 1, PACKED, STREAM_B>>(p, S, ep, st);
  if (bm == 32) return launch_gated_ring_as<GatedCfg<2, 1, 2, PACKED, STREAM_B>>(p, S, ep, st);
  return launch_gated_ring_as<GatedCfg<2, 2, 2, PACKED, STREAM_B>>(p, S, ep, st);
}

// Estimated times in us, fitted to measurements on one MI355X: products of 1 to 2048 rows, 256 to
// 18432 columns of h, K = 512 to 18432, the kernels' every form that fits (bm rows, S splits). On
// 227 of them with so many weights in turn that each came from HBM the choice is within 0.6 % of the
// best form measured on average and within 10 % on all; on 86 with three weights in turn within 1.9 %,
// and within 10 % on all but three (32 x 14336 x 2048, 32 x 1024 x 1408, 96 x 18432 x 512: 17 - 18 %).
//   ring: launch, prologue and epilogue; the run's pairs; B's bytes; further rounds of tiles; for
//   S > 1 the partials' trip through memory and the last split's sum over them.
// us by S, weights from HBM, the form taken in brackets:
//                                              1     2     3     4     5     6     7    10    14  (tiles)
//    M = 1,  I = 2048, K = 7168, bm = 16     37.9  23.3  18.9  15.5  14.7  13.7 [12.8] 13.1  13.6   25.4
//    M = 16, I = 2048, K = 7168, bm = 16     39.4  24.4  19.7  16.3  15.4  14.4 [13.6] 13.6  14.0   26.9
//    M = 64, I = 2048, K = 7168, bm = 32     40.2  25.2  20.8  17.3  17.0  16.1 [15.6]              28.2
//                                bm = 64     46.3  29.4  24.6  21.2  21.0  19.8  19.5  21.4  23.8
//    M = 64, I = 8192, K = 8192, bm = 64     55.2  40.6  32.2 [31.7]                                48.4
//    M = 1000, I = 2048, K = 7168, bm = 64  [43.9]                                                  46.3
//    M = 2048, I = 2816, K = 4096, bm = 64   76.0                                                  [67.3]
struct GatedPlan {
  int bm;  // 0: the tile kernel
  int64_t S;
  double time;
};

GatedPlan gated_ring_plan(int bm, int64_t M, int64_t I, int64_t K) {
  const int k = bm == 16 ? 0 : bm == 32 ? 1 : 2;
  const double start[] = {3.7, 4.1, 5.8}, pair[] = {0.93, 1.0, 1.2}, each[] = {0.24, 0.38, 0.78};
  const int64_t pairs = (K / kKBlock + 1) / 2, tiles = (M + bm - 1) / bm * (I / 128);
  const int64_t rounds = (tiles + kCUs - 1) / kCUs;
  const double fixed = start[k] + (double)(2 * I) * (double)K / 11e6;
  GatedPlan best{bm, 1, fixed + (double)rounds * pair[k] * (double)pairs + 4.2 * (double)(rounds - 1)};
  for (int64_t S = 2; S <= 16 && S <= pairs && tiles * S <= kCUs; ++S) {
    const int64_t run = (pairs + S - 1) / S, used = (pairs + run - 1) / run;
    // of the partials' cost half goes by the rows that a tile has
    const double rows = M < bm ? 0.5 + 0.5 * (double)M / bm : 1.0;
    const double batch = bm == 16 && used > 8 ? 1.0 : 0.0;  // beyond the eight that are loaded at once
    const double t = fixed + pair[k] * (double)run + 2.0 + each[k] * rows * (double)used + batch;
    if (t < best.time) best = GatedPlan{bm, used, t};
  }
  return best;
}

double gated_pipe_time(int64_t M, int64_t I, int64_t K) {
  const int64_t KB = K / kKBlock, tiles = (M + 127) / 128 * (I / 128);
  const TailSplit ts = pipe_tail_split(tiles, KB);
  const double round = 0.83 * (double)KB + 8.6, fixed = (double)(2 * I) * (double)K / 14.9e6 - 1.0;
  if (ts.parts == 1) return fixed + (double)((tiles + kCUs - 1) / kCUs) * round;
  const double filled = (double)((tiles - ts.full) * ts.parts) / kCUs;  // of the last round
  return fixed + (double)(ts.full / kCUs) * round + 0.83 * (double)(KB / ts.parts) + 9.2 + (double)ts.parts +
         11.3 * filled;
}

// The tile kernel's 32-bit offsets reach from a gate row to its up row. Beyond that only the ring
// kernel is left, whose launches hold fewer than 2^23 workgroups of 512 threads.
bool gated_pipe_fits(int64_t I, int64_t K) { return (I + 256) * K < (int64_t)1 << 31; }

GatedPlan gated_plan(int64_t M, int64_t I, int64_t K) {
  const char* forced = getenv("DG_FORCE_CONFIG");
  if (forced && strcmp(forced, "pipe128x256") == 0 && gated_pipe_fits(I, K)) return GatedPlan{0, 1, 0};
  GatedPlan best{0, 1, gated_pipe_fits(I, K) ? gated_pipe_time(M, I, K) : 1e30};
  for (int bm : {16, 32, 64}) {
    const GatedPlan pl = gated_ring_plan(bm, M, I, K);
    char name[16];
    snprintf(name, sizeof name, "gated_m%d", bm);
    if (forced && strcmp(forced, name) == 0) return pl;
    if ((M + bm - 1) / bm * (I / 128) < kLaunchThreads / 512 && pl.time < best.time) best = pl;
  }
  return best;
}

// From this many bytes on B is streamed past the caches where one row tile reads it: by the ring
// kernel's rule and for its reason. us, streamed and not, with so many weights in turn that none
// stays in a cache: 64 x 18432 x 7168 56.8, 61.8; 1 x 18432 x 7168 48.1, 52.5; with a weight of
// 75 MB that stays (1 x 2048 x 18432) 23.7, 18.6.
constexpr int64_t kGatedStreamB = int64_t(96) << 20;

dg_status gated(const Problem& p, const Epilogue& ep, hipStream_t stream) {
  const int64_t I = p.N / 2;
  const GatedPlan pl = gated_plan(p.M, I, p.K);
  if (pl.bm == 0 && !gated_pipe_fits(I, p.K))
    return fail(DG_ERR_UNSUPPORTED_SHAPE,
                "(I + 256) * K beyond 2^31 with 2^23 tiles of 64 x 128 or more (M=%lld, I=%lld, K=%lld)",
                (long long)p.M, (long long)I, (long long)p.K);
  if (pl.bm == 0) {
    print_dense_choice(p.M, p.N, p.K, "pipe128x256", " (gated)");
    return p.K / kKBlock >= kLongKB ? launch_pipe_gated<PipeCfg<128, 256, 12>>(p, ep, stream)
                                    : launch_pipe_gated<PipeCfg<128, 256>>(p, ep, stream);
  }
  char note[32];
  snprintf(note, sizeof note, " (gated, %d K splits)", (int)pl.S);
  print_dense_choice(p.M, p.N, p.K, pl.bm == 16 ? "gated_m16" : pl.bm == 32 ? "gated_m32" : "gated_m64",
                     pl.S > 1 ? note : " (gated)");
  if (p.M <= pl.bm && p.N * p.K >= kGatedStreamB)
    return p.sfa_packed ? launch_gated_ring<true, true>(pl.bm, pl.S, p, ep, stream)
                        : launch_gated_ring<false, true>(pl.bm, pl.S, p, ep, stream);
  return p.sfa_packed ? launch_gated_ring<true, false>(pl.bm, pl.S, p, ep, stream)
                      : launch_gated_ring<false, false>(pl.bm, pl.S, p, ep, stream);
}

}  // namespace
}  // namespace dg

using namespace dg;

extern "C" {

dg_status dg_dropout_add(const void* x, const void* residual, int32_t x_dtype, double dropout_p,
                         const int64_t* rng, int64_t subsequence, void* out, int64_t n,
                         void* stream) {
  g_detail[0] = 0;
  if (!known_dtype(x_dtype))
    return fail(DG_ERR_BAD_SHAPE, "x_dtype=%d is neither DG_DTYPE_F32 nor DG_DTYPE_BF16", x_dtype);
  if (n < 0) return fail(DG_ERR_BAD_SHAPE, "negative size n=%lld", (long long)n);
  DropAddArgs a{x, residual, out, n, {}};
  const dg_status s = drop_args(dropout_p, rng, subsequence, &a.drop);
  if (s != DG_OK || n == 0) return s;
  if (n > (int64_t)1 << 40) return fail(DG_ERR_UNSUPPORTED_SHAPE, "n beyond 2^40");
  if (!x || !out) return fail(DG_ERR_NULL_POINTER, "NULL x or out");
  if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(out, 16))
    return fail(DG_ERR_MISALIGNED, "x, residual and out must be 16-byte aligned");
  const int64_t per_wg = kDropChunk * (kDropThreads / 64) * kDropUnroll;
  const dim3 grid((unsigned)even_grid((n + per_wg - 1) / per_wg, 8 * kCUs)), block(kDropThreads);
  return launch_kernel("dropout_add_kernel",
                       x_dtype == DG_DTYPE_BF16 ? dropout_add_kernel<true> : dropout_add_kernel<false>, grid,
                       block, 0, (hipStream_t)stream, a);
}

dg_status dg_dropout_backward_fp8(const void* dy, int32_t dy_dtype, double dropout_p,
                                  const int64_t* rng, int64_t subsequence, void* codes, void* sf,
                                  int32_t sf_packed, float* dbias, int64_t M, int64_t K,
                                  void* stream) {
  g_detail[0] = 0;
  if (!known_dtype(dy_dtype))
    return fail(DG_ERR_BAD_SHAPE, "dy_dtype=%d is neither DG_DTYPE_F32 nor DG_DTYPE_BF16", dy_dtype);
  dg_status s = check_rows(M, K, "K");
  if (s != DG_OK) return s;
  DropArgs drop;
  s = drop_args(dropout_p, rng, subsequence, &drop);
  if (s != DG_OK || K == 0) return s;
  if (K > (int64_t)1 << 30) return fail(DG_ERR_UNSUPPORTED_SHAPE, "K beyond 2^30");
  if (M > 0 && (!dy || !codes || !sf)) return fail(DG_ERR_NULL_POINTER, "NULL dy, codes or sf");
  if (!aligned(dy, 16) || !aligned(codes, 16) || !aligned(dbias, 16))
    return fail(DG_ERR_MISALIGNED, "dy, codes and dbias must be 16-byte aligned");
  if (!aligned(sf, 4)) return fail(DG_ERR_MISALIGNED, "sf must be 4-byte aligned");
  const hipStream_t st = (hipStream_t)stream;
  if (M == 0) return dbias ? launch_column_sum(nullptr, dbias, 0, K, st) : DG_OK;
  const StripPlan pl = strip_plan(M, K);
  const bool direct = dbias && M <= kDropDirectRows && M * K <= kDropDirectValues, sum = dbias && !direct;
  float* part = nullptr;
  const StreamTurn turn(st, sum);
  if (sum) {
    s = get_partials(st, pl.groups * K, &part);
    if (s != DG_OK) return s;
  }
  const DropBwdArgs a{dy, (uint8_t*)codes, ScaleOut{(uint8_t*)sf, sf_packed != 0, (int32_t)(K / 128)}, part,
                      dbias, M, pl.rows, (int32_t)K, (int32_t)pl.strips, (int32_t)pl.groups, drop};
  const dim3 grid((unsigned)(pl.strips * pl.groups + (direct ? K / kDropDirectCols : 0)));
  s = launch_kernel("dropout_backward_kernel",
                    dy_dtype == DG_DTYPE_BF16 ? dropout_backward_kernel<true> : dropout_backward_kernel<false>,
                    grid, dim3(256), 0, st, a);
  return s == DG_OK && sum ? launch_column_sum(part, dbias, pl.groups, K, st) : s;
}

dg_status dg_layernorm_fp8_1x128(const void* x, const void* residual, int32_t x_dtype,
                                 const void* weight, const void* bias, int32_t w_dtype, float eps,
                                 double dropout_p, const int64_t* rng, int64_t subsequence, void* h,
                                 float* mean, float* rstd, void* codes, void* sf, int32_t sf_packed,
                                 int64_t M, int64_t K, void* stream) {
  g_detail[0] = 0;
  dg_status s = check_norm(x_dtype, w_dtype, M, K);
  if (s != DG_OK) return s;
  if (!(eps > 0.f && eps < INFINITY)) return fail(DG_ERR_BAD_SHAPE, "eps=%g is not positive", (double)eps);
  LayerNormArgs a{x, residual, weight, bias, h, mean, rstd, (uint8_t*)codes,
                  ScaleOut{(uint8_t*)sf, sf_packed != 0, (int32_t)(K / 128)}, M, (int32_t)K, eps, {}};
  s = drop_args(dropout_p, rng, subsequence, &a.drop);
  if (s != DG_OK || M == 0 || K == 0) return s;
  if (!x || !weight || !codes || !sf) return fail(DG_ERR_NULL_POINTER, "NULL x, weight, codes or sf");
  if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(weight, 16) || !aligned(bias, 16) ||
      !aligned(h, 16) || !aligned(codes, 16))
    return fail(DG_ERR_MISALIGNED, "x, residual, weight, bias, h and codes must be 16-byte aligned");
  if (!aligned(mean, 4) || !aligned(rstd, 4) || !aligned(sf, 4))
    return fail(DG_ERR_MISALIGNED, "mean, rstd and sf must be 4-byte aligned");
  const int nt = norm_threads(K);
  const int resident = norm_chunks(K) == 1 ? 1024 / nt : 1;  // as for the RMS norm
  const dim3 grid((unsigned)even_grid(M, kCUs * resident)), block((unsigned)nt);
  norm_form(x_dtype == DG_DTYPE_BF16, w_dtype == DG_DTYPE_BF16, K, [&](auto xb, auto wb, auto c) {
    s = launch_kernel("layernorm_kernel",
                      a.drop.threshold ? layernorm_kernel<xb.value, wb.value, c.value, true>
                                       : layernorm_kernel<xb.value, wb.value, c.value, false>,
                      grid, block, 0, (hipStream_t)stream, a);
  });
  return s;
}

dg_status dg_layernorm_backward(const void* dy, const void* dh, const void* h, int32_t x_dtype,
                                const void* weight, int32_t w_dtype, const float* mean,
                                const float* rstd, void* dx, float* dweight, float* dbias, int64_t M,
                                int64_t K, void* stream) {
  g_detail[0] = 0;
  dg_status s = check_norm(x_dtype, w_dtype, M, K);
  if (s != DG_OK || K == 0) return s;
  if (!dweight || (M > 0 && (!dy || !h || !weight || !mean || !rstd || !dx)))
    return fail(DG_ERR_NULL_POINTER, "NULL dy, h, weight, mean, rstd, dx or dweight");
  if (!aligned(dy, 16) || !aligned(dh, 16) || !aligned(h, 16) || !aligned(weight, 16) ||
      !aligned(dx, 16) || !aligned(dweight, 16) || !aligned(dbias, 16))
    return fail(DG_ERR_MISALIGNED, "dy, dh, h, weight, dx, dweight and dbias must be 16-byte aligned");
  if (!aligned(mean, 4) || !aligned(rstd, 4))
    return fail(DG_ERR_MISALIGNED, "mean and rstd must be 4-byte aligned");
  const hipStream_t st = (hipStream_t)stream;
  if (M == 0) return launch_column_sum2(nullptr, dweight, dbias, 0, K, st);
  // workgroups and teams as for the RMS norm's backward
  const int nt = norm_threads(K);
  int64_t R = nt < 512 ? 512 / nt : 1;
  if (R > (M + kCUs - 1) / kCUs) R = (M + kCUs - 1) / kCUs;
  const int64_t G = even_grid((M + R - 1) / R, kCUs);
  // a dx in the place of dy or h would be written while the column sums read them
  const bool direct = M <= ln_direct_rows(K) && M * K <= kLnDirectValues && dx != dy && dx != h;
  float* part = nullptr;
  const StreamTurn turn(st, !direct);
  if (!direct) {
    s = get_partials(st, G * 2 * K, &part);
    if (s != DG_OK) return s;
  }
  const LayerNormBwdArgs a{dy, dh, h, weight, mean, rstd, dx, part, dweight, dbias, M, (int32_t)K,
                           (int32_t)R, (int32_t)G};
  const unsigned grid = (unsigned)(G + (direct ? K / kLnDirectCols : 0));
  norm_form(x_dtype == DG_DTYPE_BF16, w_dtype == DG_DTYPE_BF16, K, [&](auto xb, auto wb, auto c) {
    s = launch_layernorm_backward<xb.value, wb.value, c.value>(a, grid, (unsigned)(nt * R), st);
  });
  return s == DG_OK && !direct ? launch_column_sum2(part, dweight, dbias, G, K, st) : s;
}

dg_status dg_fp8_gemm_nt_gated_fp8(const void* A, const void* B, void* codes, void* sf,
                                   int32_t sf_packed, const void* sfA, int32_t sfA_packed,
                                   const float* sfB, const void* bias, int32_t bias_dtype,
                                   int32_t activation, void* pre, int64_t M, int64_t I, int64_t K,
                                   void* stream) {
  g_detail[0] = 0;
  if (M < 0 || I < 0) return fail(DG_ERR_BAD_SHAPE, "negative size (M=%lld, I=%lld)", (long long)M, (long long)I);
  if (!known_act(activation)) return fail(DG_ERR_BAD_SHAPE, "activation=%d is unknown", activation);
  if (bias && !known_dtype(bias_dtype))
    return fail(DG_ERR_BAD_SHAPE, "bias_dtype=%d is neither DG_DTYPE_F32 nor DG_DTYPE_BF16", bias_dtype);
  if (I % 128 != 0) return fail(DG_ERR_BAD_SHAPE, "I=%lld is not a multiple of 128", (long long)I);
  if (I > (int64_t)1 << 29 || M > (int64_t)1 << 30)
    return fail(DG_ERR_UNSUPPORTED_SHAPE, "I beyond 2^29 or M beyond 2^30");
  const dg_status s = check_common(A, B, codes, sfA, sfB, 2 * I, K, M > 0 && I > 0);
  if (s != DG_OK || M == 0 || I == 0) return s;
  if (!sf) return fail(DG_ERR_NULL_POINTER, "NULL sf");
  if (!aligned(sf, 4)) return fail(DG_ERR_MISALIGNED, "sf must be 4-byte aligned");
  if (!aligned(bias, 16) || !aligned(pre, 16))
    return fail(DG_ERR_MISALIGNED, "bias and pre must be 16-byte aligned");
  if (K / kKBlock > kPipeMaxKB || I / 128 * (K / kKBlock) >= (int64_t)1 << 28)
    return fail(DG_ERR_UNSUPPORTED_SHAPE, "K beyond 2^22, or I * K beyond 2^42");
  Problem p{};
  p.A = (const uint8_t*)A;
  p.B = (const uint8_t*)B;
  p.sfA = (const uint8_t*)sfA;
  p.sfa_packed = sfA_packed != 0;
  p.sfB = sfB;
  p.M = M;
  p.N = 2 * I;
  p.K = K;
  p.G = 1;
  Epilogue ep{};
  ep.bias = bias;
  ep.bias_bf16 = bias_dtype == DG_DTYPE_BF16;
  ep.act = activation;
  ep.pre = (uint16_t*)pre;
  ep.codes = (uint8_t*)codes;
  ep.so = ScaleOut{(uint8_t*)sf, sf_packed != 0, (int32_t)(I / 128)};
  return no_throw([&] { return gated(p, ep, (hipStream_t)stream); });
}

dg_status dg_gated_backward_fp8(const void* dh, const void* pre, int32_t activation, void* codes,
                                void* sf, int32_t sf_packed, float* dbias, int64_t M, int64_t I,
                                void* stream) {
  g_detail[0] = 0;
  if (!known_act(activation)) return fail(DG_ERR_BAD_SHAPE, "activation=%d is unknown", activation);
  dg_status s = check_rows(M, I, "I");
  if (s != DG_OK || I == 0) return s;
  if (I > (int64_t)1 << 29) return fail(DG_ERR_UNSUPPORTED_SHAPE, "I beyond 2^29");
  if (M > 0 && (!dh || !pre || !codes || !sf)) return fail(DG_ERR_NULL_POINTER, "NULL dh, pre, codes or sf");
  if (!aligned(dh, 16) || !aligned(pre, 16) || !aligned(codes, 16) || !aligned(dbias, 16))
    return fail(DG_ERR_MISALIGNED, "dh, pre, codes and dbias must be 16-byte aligned");
  if (!aligned(sf, 4)) return fail(DG_ERR_MISALIGNED, "sf must be 4-byte aligned");
  const hipStream_t st = (hipStream_t)stream;
  if (M == 0) return dbias ? launch_column_sum(nullptr, dbias, 0, 2 * I, st) : DG_OK;
  const StripPlan pl = strip_plan(M, I);
  const bool direct = dbias && M <= kGatedDirectRows && M * I <= kGatedDirectValues, sum = dbias && !direct;
  float* part = nullptr;
  const StreamTurn turn(st, sum);
  if (sum) {
    s = get_partials(st, pl.groups * 2 * I, &part);
    if (s != DG_OK) return s;
  }
  const GatedBwdArgs a{(const uint16_t*)dh, (const uint16_t*)pre, (uint8_t*)codes,
                       ScaleOut{(uint8_t*)sf, sf_packed != 0, (int32_t)(I / 64)}, part, dbias, M, pl.rows,
                       (int32_t)I, activation, (int32_t)pl.strips, (int32_t)pl.groups};
  s = launch_kernel("gated_backward_kernel", gated_backward_kernel,
                    dim3((unsigned)(pl.strips * pl.groups + (direct ? I / kGatedDirectCols : 0))), dim3(256), 0, st,
                    a);
  return s == DG_OK && sum ? launch_column_sum(part, dbias, pl.groups, 2 * I, st) : s;
}

}  // extern "C"
