// layernorm_kernel.hpp -- layer norm of residual + dropout(x) with an FP8 output with 1x128
// scales, and its backward pass, for gfx950. Bound by HBM like the RMS norm's kernels, whose
// lanes, chunks and teams (norm_kernel.hpp) they share: each value is read once (the backward
// kernel's of few rows twice) and written once, what lies between stays in registers, in fp32.
//
// Forward, row m of K values (K % 128 == 0):
//   s = dropout(x) + r (both optional; in fp32, not rounded);  h = s rounded to x's type
//   mean = sum(s) / K;  rstd = 1 / sqrt(sum((s - mean)^2) / K + eps)
//   y = (s - mean) rstd w + b (b optional);  codes, scale = y quantized per 1x128 block
// Backward, with xh = (h - mean) rstd and g = w dy:
//   dx = rstd (g - mean(g) - xh mean(g xh)) + dh (optional)
//   dweight = sum over rows of dy xh;  dbias = sum over rows of dy
//
// The variance is a sum of squared differences from a mean, never a difference of two large
// sums: each wave takes its own values' mean and squares about it, without a barrier, and the
// waves' triples (count, mean, squares) are joined behind the row's one barrier by
//   squares = sum over waves of squares_w + count_w (mean_w - mean)^2
// (Chan, Golub, LeVeque, "Updating formulae and a pairwise algorithm for computing sample
// variances", 1979).
//
// Measured: forward 4096 x 7168 bf16 with residual and dropout 37.5 us, 206 MB at 5.5 TB/s (a copy of
// 1 GiB: 5.1), one row 3.3 us from start to end, most of it dependent steps; backward 4096 x 7168
// bf16 with dh 45 us, 235 MB at 5.2 TB/s, and 4.8 for the column sums; 257 x 2048 fp32, one launch,
// 4.0 us.
#pragma once

#include "dropout.hpp"
#include "norm_kernel.hpp"

namespace dg {

// Sum of v over groups of 8 lanes and over the wave's 64, in each of them.
__device__ __forceinline__ float sum8(float v) {
  v += dppf<kDppXor1>(v);
  v += dppf<kDppXor2>(v);
  return v + dppf<kDppMirror8>(v);
}
__device__ __forceinline__ float wave_sum(float v) {
  v = sum8(v);
  v += dppf<kDppMirror16>(v);
  v += __shfl_xor(v, 16, 64);
  return v + __shfl_xor(v, 32, 64);
}

struct LayerNormArgs {
  const void* x;
  const void* r;  // NULL: no residual
  const void* w;
  const void* b;  // NULL: no bias
  void* h;        // NULL: the sum is not stored
  float* mean;    // NULL: not stored
  float* rstd;    // NULL: not stored
  uint8_t* codes;
  ScaleOut so;
  int64_t M;
  int32_t K;
  float eps;
  DropArgs drop;
};

// The rows and chunks of rmsnorm_kernel. KEEP: weights and bias stay in registers; otherwise
// (long rows) they are loaded where they are used. AHEAD: the next row is loaded before the
// barrier of this one, which only the longest fp32 rows leave no registers for (1000 x 32768 fp32:
// 86 us).
template <bool BF16, bool WBF, int C, bool DROP>
__global__ void __launch_bounds__(kNormThreads) layernorm_kernel(LayerNormArgs a) {
  constexpr bool KEEP = C <= (BF16 ? 2 : 1), AHEAD = BF16 || C <= 3;
  static_assert(kNormThreads / 64 == 8, "a row's waves fit 8 lanes");
  __shared__ float buf[2][2][8];  // means and squares of the waves; two in turn
  const int K = a.K, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  const float inv_k = 1.f / (float)K;
  const Drop drop(a.drop);
  int col[C];
  Weight16<BF16, WBF> w[KEEP ? C : 1], b[KEEP ? C : 1];
  Raw16<BF16> x[C], r[C];
  // values that the wave in question holds: this one, and wave i in lanes i, i + 8, ...
  auto count_of = [&](int v) {
    int n = 0;
#pragma unroll
    for (int c = 0; c < C; ++c) n += max(0, min(1024, K - 16 * (int)(c * blockDim.x + 64 * v)));
    return (float)n;
  };
  const float count = count_of(wave), peer = (int)(threadIdx.x & 7) < waves ? count_of(threadIdx.x & 7) : 0.f;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    col[c] = norm_col<BF16>(c, blockDim.x, threadIdx.x);
    if (KEEP && col[c] < K) {
      w[c].load(a.w, col[c]);
      if (a.b) b[c].load(a.b, col[c]);
    }
  }
  auto fetch = [&](int64_t m) {
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (col[c] < K) {
        x[c].load(a.x, m * K + col[c]);
        if (a.r) r[c].load(a.r, m * K + col[c]);
      }
  };
  int64_t m = blockIdx.x;
  if (AHEAD && m < a.M) fetch(m);
  for (int par = 0; m < a.M; m += gridDim.x, par ^= 1) {
    if (!AHEAD) fetch(m);
    float v[C][16];
    float sum = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if (col[c] >= K) continue;
#pragma unroll
      for (int i = 0; i < 16; ++i) v[c][i] = x[c][i];
      if (DROP) drop16<BF16>(drop, m * K + col[c], v[c]);
      if (a.r) {
#pragma unroll
        for (int i = 0; i < 16; ++i) v[c][i] += r[c][i];
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) sum += v[c][i];
    }
    if (AHEAD && m + gridDim.x < a.M) fetch(m + gridDim.x);
    const float own = wave_sum(sum) / count;
    float sq = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if (col[c] >= K) continue;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float d = v[c][i] - own;
        sq = __builtin_fmaf(d, d, sq);
      }
    }
    sq = wave_sum(sq);
    if ((threadIdx.x & 63) == 0) buf[par][0][wave] = own, buf[par][1][wave] = sq;
    lds_barrier();
    const float theirs = peer > 0.f ? buf[par][0][threadIdx.x & 7] : 0.f;
    const float squares = peer > 0.f ? buf[par][1][threadIdx.x & 7] : 0.f;
    const float mean = sum8(peer * theirs) * inv_k;
    const float var = sum8(__builtin_fmaf(peer * (theirs - mean), theirs - mean, squares)) * inv_k;
    const float rstd = 1.f / sqrtf(var + a.eps);
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[m] = mean;
      if (a.rstd) a.rstd[m] = rstd;
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if (col[c] >= K) continue;
      if (a.h) store16<BF16>(a.h, m * K + col[c], v[c]);
      const int k = KEEP ? c : 0;
      if (!KEEP) {
        w[0].load(a.w, col[c]);
        if (a.b) b[0].load(a.b, col[c]);
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) v[c][i] = (v[c][i] - mean) * rstd * w[k][i];
      if (a.b) {
#pragma unroll
        for (int i = 0; i < 16; ++i) v[c][i] += b[k][i];
      }
      quantize16<BF16>(v[c], threadIdx.x & 7, m, col[c] >> 7, a.codes, a.so);
    }
  }
}

constexpr int kLnDirectCols = 32;  // columns of a workgroup that only sums

struct LayerNormBwdArgs {
  const void* dy;
  const void* dh;  // NULL: nothing is added to dx
  const void* h;
  const void* w;
  const float* mean;
  const float* rstd;
  void* dx;
  float* part;     // [groups][2 K] partial dweight, dbias; NULL: further workgroups sum them
  float* dweight;  // part == NULL: the sums
  float* dbias;
  int64_t M;
  int32_t K;
  int32_t teams;   // rows that a workgroup works on side by side
  int32_t groups;  // workgroups that take rows
};

// Values added to a lane's 16 fp32 sums in LDS (its own, so nothing has to be waited for).
template <bool BF16>
__device__ __forceinline__ void lds_add16(float* sums, const float (&v)[16]) {
  constexpr int P = Pieces<BF16>::P;
#pragma unroll
  for (int i = 0; i < 16; i += 4) {
    nk_v4f* p = (nk_v4f*)(sums + i / P * 8 * P + i % P);
    const nk_v4f t = *p;
    *p = nk_v4f{t[0] + v[i], t[1] + v[i + 1], t[2] + v[i + 2], t[3] + v[i + 3]};
  }
}

// The teams and chunks of rmsnorm_backward_kernel, with two sums per row and two per column.
// LDS_DW: the sums of dweight lie in LDS, those of dbias in registers, which do not hold both
// beside the values of a row in several chunks (registers alone spill 77 to 169 of them from
// 16384 fp32 values on, 1000 x 18432: 121 us; 74 with LDS). AHEAD as there.
template <bool BF16, int C>
constexpr bool kLnLdsDw = C >= (BF16 ? 3 : 2);

template <bool BF16, bool WBF, int C>
__global__ void __launch_bounds__(kNormThreads) layernorm_backward_kernel(LayerNormBwdArgs a) {
  constexpr bool LDS_DW = kLnLdsDw<BF16, C>, AHEAD = C <= 2;
  __shared__ float buf[2][2][kNormThreads / 64];
  extern __shared__ float lds[];  // [teams - 1][K], LDS_DW: [K]; or the direct sums'
  const int K = a.K, R = a.teams, threads = blockDim.x / R;
  const float inv_k = 1.f / (float)K;
  const int index = sums_first(a.groups);
  if (index >= a.groups) {
    constexpr int P = Pieces<BF16>::P;
    struct Row {
      quant_v4u dy, h;
      float mean, rstd;
    };
    direct_sums<2, P, kLnDirectCols, true>(
        a.M, (index - a.groups) * kLnDirectCols, {a.dweight, a.dbias}, lds,
        [&](int64_t m, int c) {
          return Row{raw_piece<BF16>(a.dy, m * K + c), raw_piece<BF16>(a.h, m * K + c), a.mean[m], a.rstd[m]};
        },
        [&](const Row& row, int64_t, float (&v)[2][P]) {
          float d[P], x[P];
          unpack_piece<BF16>(row.dy, d);
          unpack_piece<BF16>(row.h, x);
#pragma unroll
          for (int i = 0; i < P; ++i) {
            v[0][i] = __builtin_fmaf(d[i], (x[i] - row.mean) * row.rstd, v[0][i]);
            v[1][i] += d[i];
          }
        });
    return;
  }
  const int team = threadIdx.x / threads, t = threadIdx.x - team * threads;
  const int wave = t >> 6, waves = threads >> 6;
  const bool peer = (int)(threadIdx.x & 7) < waves;
  int col[C];
  Weight16<BF16, WBF> w[AHEAD ? C : 1];
  float dw[LDS_DW ? 1 : C][16], db[C][16];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    col[c] = norm_col<BF16>(c, threads, t);
#pragma unroll
    for (int i = 0; i < 16; ++i) dw[LDS_DW ? 0 : c][i] = db[c][i] = 0.f;
    if (LDS_DW && col[c] < K) store_sums16<BF16>(lds + col[c], dw[0]);
    if (AHEAD && col[c] < K) w[c].load(a.w, col[c]);
  }
  Raw16<BF16> h[C], dy[C], dh[AHEAD ? C : 1];
  float mu = 0.f, rs = 0.f;
  auto fetch = [&](int64_t m) {
    mu = a.mean[m];
    rs = a.rstd[m];
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (col[c] < K) {
        h[c].load(a.h, m * K + col[c]);
        dy[c].load(a.dy, m * K + col[c]);
      }
  };
  auto fetch_dh = [&](int64_t m) {
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (AHEAD && col[c] < K && a.dh) dh[c].load(a.dh, m * K + col[c]);
  };
  const int64_t step = (int64_t)a.groups * R;
  int64_t m = (int64_t)index * R + team;
  if (AHEAD && m < a.M) {
    fetch(m);
    fetch_dh(m);
  }
  // every team passes every barrier: the loop runs while team 0 has a row
  for (int par = 0; m - team < a.M; m += step, par ^= 1) {
    const bool live = m < a.M;
    if (!AHEAD && live) fetch(m);
    const float mean = mu, rstd = rs;
    float xh[AHEAD ? C : 1][16], g[AHEAD ? C : 1][16];
    float sum = 0.f, dot = 0.f;
    if (live) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        if (col[c] >= K) continue;
        const int k = AHEAD ? c : 0;
        if (!AHEAD) w[0].load(a.w, col[c]);
        float p[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float d = dy[c][i];
          xh[k][i] = (h[c][i] - mean) * rstd;
          if (LDS_DW) p[i] = d * xh[k][i];
          else dw[LDS_DW ? 0 : c][i] = __builtin_fmaf(d, xh[k][i], dw[LDS_DW ? 0 : c][i]);
          db[c][i] += d;
          g[k][i] = d * w[k][i];
          sum += g[k][i];
          dot = __builtin_fmaf(g[k][i], xh[k][i], dot);
        }
        if (LDS_DW && a.part) lds_add16<BF16>(lds + col[c], p);
      }
    }
    if (AHEAD && m + step < a.M) fetch(m + step);
    sum = wave_sum(sum);
    dot = wave_sum(dot);
    if ((threadIdx.x & 63) == 0) {
      buf[par][0][team * waves + wave] = sum;
      buf[par][1][team * waves + wave] = dot;
    }
    lds_barrier();
    sum = sum8(peer ? buf[par][0][team * waves + (threadIdx.x & 7)] : 0.f) * inv_k;
    dot = sum8(peer ? buf[par][1][team * waves + (threadIdx.x & 7)] : 0.f) * inv_k;
    if (live) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        if (col[c] >= K) continue;
        const int k = AHEAD ? c : 0;
        if (!AHEAD) {
          if (a.dh) dh[0].load(a.dh, m * K + col[c]);
          w[0].load(a.w, col[c]);
#pragma unroll
          for (int i = 0; i < 16; ++i) xh[0][i] = (h[c][i] - mean) * rstd, g[0][i] = dy[c][i] * w[0][i];
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          g[k][i] = rstd * __builtin_fmaf(-xh[k][i], dot, g[k][i] - sum);
          if (a.dh) g[k][i] += dh[k][i];
        }
        store16<BF16>(a.dx, m * K + col[c], g[k]);
      }
    }
    if (AHEAD && m + step < a.M) fetch_dh(m + step);
  }
  if (!a.part) return;
  float* part = a.part + (int64_t)index * 2 * K;
  if constexpr (LDS_DW) {  // R = 1
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (col[c] < K) {
        float v[16] = {};
        add_sums16<BF16>(lds + col[c], v);
        store_sums16<BF16>(part + col[c], v);
        store_sums16<BF16>(part + K + col[c], db[c]);
      }
  } else {
    // one sum after the other through the same LDS; every team passes every barrier
#pragma unroll
    for (int k = 0; k < 2 && R > 1; ++k) {
      float(&own)[C][16] = k ? db : dw;
      if (k) __syncthreads();
#pragma unroll
      for (int c = 0; c < C; ++c)
        if (team > 0 && col[c] < K) store_sums16<BF16>(lds + (team - 1) * K + col[c], own[c]);
      __syncthreads();
      for (int q = 0; q < R - 1 && team == 0; ++q)
#pragma unroll
        for (int c = 0; c < C; ++c)
          if (col[c] < K) add_sums16<BF16>(lds + q * K + col[c], own[c]);
    }
    if (team > 0) return;
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (col[c] < K) {
        store_sums16<BF16>(part + col[c], dw[c]);
        store_sums16<BF16>(part + K + col[c], db[c]);
      }
  }
}

}  // namespace dg
