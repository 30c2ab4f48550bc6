// gated_kernel.hpp -- backward pass of the gated feed-forward product's epilogue, for gfx950:
//
//   z = [zg, zu] (pre, bf16);  h = act(zg) zu
//   dzg = dh zu act'(zg);  dzu = dh act(zg);  codes, scales = [dzg, dzu] quantized per 1x128 block
//   dbias = sum over rows of [dzg, dzu]
// Bound by HBM: 6 bytes read and 2 written per value of h, everything between in registers, in
// fp32. The column sums are those of the other backward kernels (norm_kernel.hpp). Measured: 4096 x
// 18432 (silu) 118 us, 605 MB at 5.1 TB/s, and 4.7 for the column sums; 130 x 2048 (gelu), one launch,
// 4.9 us, most of it the slopes of the columns that one wave per SIMD sums.
#pragma once

#include "norm_kernel.hpp"

namespace dg {

constexpr int kGatedDirectCols = 32;  // columns of a workgroup that only sums

struct GatedBwdArgs {
  const uint16_t* dh;
  const uint16_t* pre;
  uint8_t* codes;
  ScaleOut so;
  float* part;   // [row groups][2 I] partial dbias; NULL: none
  float* dbias;  // part == NULL: written by further workgroups, if any
  int64_t M;
  int64_t rows;  // rows per row group
  int32_t I;
  int32_t act;
  int32_t strips;  // strips of 1024 columns of h
  int32_t groups;  // row groups
};

// The layout of act_backward_kernel: a workgroup of four waves takes a strip of 1024 columns of
// h, and with it the same columns of both halves of pre, over a group of rows.
static __global__ void __launch_bounds__(256) gated_backward_kernel(GatedBwdArgs a) {
  __shared__ float sums[3][2][1024];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t I = a.I, N = 2 * I;
  const int work = a.strips * a.groups, index = sums_first(work);
  if (index >= work) {
    struct Row {
      quant_v4u d, g, u;
    };
    direct_sums<2, 8, kGatedDirectCols, false>(
        a.M, (index - work) * kGatedDirectCols, {a.dbias, a.dbias + I}, &sums[0][0][0],
        [&](int64_t m, int c) {
          return Row{raw_piece<true>(a.dh, m * I + c), raw_piece<true>(a.pre, m * N + c),
                     raw_piece<true>(a.pre, m * N + I + c)};
        },
        [&](const Row& row, int64_t, float (&v)[2][8]) {
          float d[8], g[8], x[8];
          unpack_piece<true>(row.d, d);
          unpack_piece<true>(row.g, g);
          unpack_piece<true>(row.u, x);
          gated_backward(d, g, x, a.act);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[0][i] += g[i], v[1][i] += x[i];
        });
    return;
  }
  const int strip = index % a.strips, group = index / a.strips;
  const int in_strip = (lane >> 3) * 128 + (lane & 7) * Pieces<true>::P;
  const int col = strip * 1024 + in_strip;
  const int64_t m1 = min(a.M, (group + 1) * a.rows);
  float sg[16], su[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) sg[i] = su[i] = 0.f;
  if (col < a.I) {
    Raw16<true> d, g, u;
    auto fetch = [&](int64_t m) {
      if (m >= m1) return;
      d.load(a.dh, m * I + col);
      g.load(a.pre, m * N + col);
      u.load(a.pre, m * N + I + col);
    };
    int64_t m = group * a.rows + wave;
    fetch(m);
    for (; m < m1; m += 4) {
      float p[16], zg[16], zu[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) p[i] = d[i], zg[i] = g[i], zu[i] = u[i];
      fetch(m + 4);
      gated_backward(p, zg, zu, a.act);
#pragma unroll
      for (int i = 0; i < 16; ++i) sg[i] += zg[i], su[i] += zu[i];
      quantize16<true>(zg, lane & 7, m, col >> 7, a.codes, a.so);
      quantize16<true>(zu, lane & 7, m, (int)((I + col) >> 7), a.codes, a.so);
    }
  }
  if (!a.part) return;
  if (wave > 0) {
    store_sums16<true>(sums[wave - 1][0] + in_strip, sg);
    store_sums16<true>(sums[wave - 1][1] + in_strip, su);
  }
  __syncthreads();
  if (wave > 0 || col >= a.I) return;
#pragma unroll
  for (int w = 0; w < 3; ++w) {
    add_sums16<true>(sums[w][0] + in_strip, sg);
    add_sums16<true>(sums[w][1] + in_strip, su);
  }
  store_sums16<true>(a.part + group * N + col, sg);
  store_sums16<true>(a.part + group * N + I + col, su);
}

}  // namespace dg
