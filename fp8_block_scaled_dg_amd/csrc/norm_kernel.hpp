// norm_kernel.hpp -- RMS norm with the residual's addition and an FP8 output with 1x128
// scales, its backward pass, and the backward pass of the GEMM's bias + activation epilogue
// with an FP8 output, for gfx950. All three are bound by HBM: each value is read once and
// written once, everything in between stays in registers, in fp32.
//
// Forward, row m of K values (K % 128 == 0):
//   s = x + r (r optional, the sum in fp32, not rounded);  h = s rounded to x's type
//   rstd = 1 / sqrt(mean(s^2) + eps);  y = s rstd w
//   codes, scale = y quantized per 1x128 block by the quantizer's rule (quant_kernel.hpp)
// Backward, with xh = h rstd and g = w dy:
//   dx = rstd (g - xh mean(g xh)) + dh (dh optional: the gradient that reaches h along the
//   residual stream);  dweight = sum over rows of dy xh
// Epilogue backward:  p = dc act'(pre);  codes, scale = p quantized per 1x128 block;
//   dbias = sum over rows of p
//
// Column sums (dweight, dbias): every workgroup sums its own rows in registers and writes
// one fp32 row of partials; column_sum_kernel adds the partials in a fixed order, so the
// results do not depend on scheduling.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "activation.hpp"
#include "quant_kernel.hpp"

namespace dg {

typedef float nk_v2f __attribute__((ext_vector_type(2)));
typedef float nk_v4f __attribute__((ext_vector_type(4)));
typedef __bf16 nk_v2bf __attribute__((ext_vector_type(2)));

// Two fp32 values rounded to bf16 (nearest even, NaN kept), low half first.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(nk_v2f{a, b}, nk_v2bf));
}

// 16 consecutive values to element idx of a bf16 or fp32 array.
template <bool BF16>
__device__ __forceinline__ void store16(void* dst, int64_t idx, const float (&v)[16]) {
  if constexpr (BF16) {
    quant_v4u* p = (quant_v4u*)((uint16_t*)dst + idx);
#pragma unroll
    for (int q = 0; q < 2; ++q)
      p[q] = quant_v4u{pack_bf16(v[8 * q], v[8 * q + 1]), pack_bf16(v[8 * q + 2], v[8 * q + 3]),
                       pack_bf16(v[8 * q + 4], v[8 * q + 5]), pack_bf16(v[8 * q + 6], v[8 * q + 7])};
  } else {
    nk_v4f* p = (nk_v4f*)((float*)dst + idx);
#pragma unroll
    for (int q = 0; q < 4; ++q) p[q] = nk_v4f{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
  }
}

// 16 consecutive weights (bf16 or fp32, chosen at run time), cached: every row reads them.
__device__ __forceinline__ void load_weight16(const void* w, int bf16, int64_t idx, float (&v)[16]) {
  if (bf16) {
    const quant_v4u* p = (const quant_v4u*)((const uint16_t*)w + idx);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const quant_v4u u = p[q];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[8 * q + 2 * j] = __uint_as_float(u[j] << 16);
        v[8 * q + 2 * j + 1] = __uint_as_float(u[j] & 0xFFFF0000u);
      }
    }
  } else {
    const nk_v4f* p = (const nk_v4f*)((const float*)w + idx);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const nk_v4f u = p[q];
#pragma unroll
      for (int j = 0; j < 4; ++j) v[4 * q + j] = u[j];
    }
  }
}

// Where scales go: fp32 [rows][KB], or (packed) rows of ceil(KB/4) words of UE8M0 bytes.
struct ScaleOut {
  uint8_t* sf;
  int32_t packed;
  int32_t KB;
};

// The scale 2^e of K-block kb in row m. The packed form holds exponents from -127 on; the
// row's last block zeroes the bytes that pad its last word.
__device__ __forceinline__ void store_scale(const ScaleOut& so, int64_t m, int kb, int e) {
  if (so.packed) {
    const int row_bytes = (so.KB + 3) / 4 * 4;
    uint8_t* row = so.sf + m * row_bytes;
    row[kb] = (uint8_t)(e + 127);
    if (kb == so.KB - 1)
      for (int j = kb + 1; j < row_bytes; ++j) row[j] = 0;
  } else {
    ((float*)so.sf)[m * so.KB + kb] = ldexpf(1.f, e);
  }
}

// The exponent of the block scale for a largest magnitude amax.
__device__ __forceinline__ int scale_exp(const ScaleOut& so, float amax) {
  const int e = quant_scale_exp(amax);
  return so.packed && e < -127 ? -127 : e;
}

// Quantizes 16 values of a 1x128 block that 8 neighbouring lanes hold (li = 0..7 of them),
// K-block kb of row m: 16 code bytes to codes, the scale by lane li = 0.
__device__ __forceinline__ void quantize16(const float (&y)[16], int li, int64_t m, int kb,
                                           uint8_t* codes, const ScaleOut& so) {
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(y[i]));
#pragma unroll
  for (int d = 1; d < 8; d <<= 1) amax = fmaxf(amax, __shfl_xor(amax, d, 8));
  const int e = scale_exp(so, amax);
  quant_v4u w;
#pragma unroll
  for (int q = 0; q < 4; ++q)
    w[q] = quant_e4m3fn_x4(ldexpf(y[4 * q], -e), ldexpf(y[4 * q + 1], -e),
                           ldexpf(y[4 * q + 2], -e), ldexpf(y[4 * q + 3], -e));
  *(quant_v4u*)(codes + (m * so.KB + kb) * 128 + li * 16) = w;
  if (li == 0) store_scale(so, m, kb, e);
}

// Sum of v over the workgroup, the same in every thread, added in a fixed order. buf: one
// float per wave, not written again before another barrier has passed (two buffers in turn).
__device__ __forceinline__ float block_sum(float v, float* buf) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d, 64);
  const int waves = blockDim.x >> 6;
  if ((threadIdx.x & 63) == 0) buf[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = 0.f;
  for (int i = 0; i < waves; ++i) s += buf[i];
  return s;
}

constexpr int kNormMaxK = 32768;    // two 16-value chunks in each of 1024 threads
constexpr int kNormMaxThreads = 1024;

struct NormArgs {
  const void* x;
  const void* r;  // NULL: no residual
  const void* w;
  void* h;        // NULL: the sum is not stored
  float* rstd;    // NULL: not stored
  uint8_t* codes;
  ScaleOut so;
  int64_t M;
  int32_t K;
  float eps;
  int32_t w_bf16;
};

// Workgroup b takes rows b, b + G, b + 2G, ... (G workgroups); thread t holds the 16 values
// from column (c * threads + t) * 16 in chunk c < C.
template <bool BF16, int C>
__global__ void __launch_bounds__(kNormMaxThreads) rmsnorm_kernel(NormArgs a) {
  __shared__ float buf[2][kNormMaxThreads / 64];
  const int K = a.K, NT = blockDim.x;
  int par = 0;
  for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x, par ^= 1) {
    float v[C][16];
    float ss = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int col = (c * NT + (int)threadIdx.x) * 16;
      if (col < K) {
        quant_load16<BF16>(a.x, m * K + col, v[c]);
        if (a.r) {
          float r[16];
          quant_load16<BF16>(a.r, m * K + col, r);
#pragma unroll
          for (int i = 0; i < 16; ++i) v[c][i] += r[i];
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) ss = __builtin_fmaf(v[c][i], v[c][i], ss);
      }
    }
    const float rstd = 1.f / sqrtf(block_sum(ss, buf[par]) / (float)K + a.eps);
    if (a.rstd && threadIdx.x == 0) a.rstd[m] = rstd;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int col = (c * NT + (int)threadIdx.x) * 16;
      if (col < K) {
        if (a.h) store16<BF16>(a.h, m * K + col, v[c]);
        float w[16];
        load_weight16(a.w, a.w_bf16, col, w);
#pragma unroll
        for (int i = 0; i < 16; ++i) v[c][i] = v[c][i] * rstd * w[i];
        quantize16(v[c], threadIdx.x & 7, m, col >> 7, a.codes, a.so);
      }
    }
  }
}

struct NormBwdArgs {
  const void* dy;
  const void* dh;  // NULL: nothing is added to dx
  const void* h;
  const void* w;
  const float* rstd;
  void* dx;
  float* part;     // [gridDim.x][K] partial dweight
  int64_t M;
  int32_t K;
  int32_t w_bf16;
};

// Workgroup b takes rows b, b + G, b + 2G, ... (G workgroups), its threads the columns of
// rmsnorm_kernel; the weights and the column sums of dweight stay in registers.
template <bool BF16, int C>
__global__ void __launch_bounds__(kNormMaxThreads) rmsnorm_backward_kernel(NormBwdArgs a) {
  __shared__ float buf[2][kNormMaxThreads / 64];
  const int K = a.K, NT = blockDim.x;
  float w[C][16], dw[C][16];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int col = (c * NT + (int)threadIdx.x) * 16;
#pragma unroll
    for (int i = 0; i < 16; ++i) dw[c][i] = 0.f, w[c][i] = 0.f;
    if (col < K) load_weight16(a.w, a.w_bf16, col, w[c]);
  }
  int par = 0;
  for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x, par ^= 1) {
    const float rstd = a.rstd[m];
    float xh[C][16], g[C][16];
    float dot = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int col = (c * NT + (int)threadIdx.x) * 16;
      if (col < K) {
        quant_load16<BF16>(a.h, m * K + col, xh[c]);
        quant_load16<BF16>(a.dy, m * K + col, g[c]);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          xh[c][i] *= rstd;
          dw[c][i] = __builtin_fmaf(g[c][i], xh[c][i], dw[c][i]);
          g[c][i] *= w[c][i];
          dot = __builtin_fmaf(g[c][i], xh[c][i], dot);
        }
      }
    }
    const float mean = block_sum(dot, buf[par]) / (float)K;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int col = (c * NT + (int)threadIdx.x) * 16;
      if (col < K) {
        float o[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i] = rstd * __builtin_fmaf(-xh[c][i], mean, g[c][i]);
        if (a.dh) {
          float d[16];
          quant_load16<BF16>(a.dh, m * K + col, d);
#pragma unroll
          for (int i = 0; i < 16; ++i) o[i] += d[i];
        }
        store16<BF16>(a.dx, m * K + col, o);
      }
    }
  }
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int col = (c * NT + (int)threadIdx.x) * 16;
    if (col < K) store16<false>(a.part, (int64_t)blockIdx.x * K + col, dw[c]);
  }
}

struct ActBwdArgs {
  const uint16_t* dc;
  const uint16_t* pre;  // unused with DG_ACT_NONE
  uint8_t* codes;
  ScaleOut so;
  float* part;          // [row groups][N] partial dbias; NULL: no dbias
  int64_t M;
  int64_t rows;         // rows per row group
  int32_t N;
  int32_t act;
  int32_t strips;       // column strips of 1024
};

// A workgroup of four waves takes a strip of 1024 columns (64 lanes of 16) over a group of
// rows, wave w rows w, w + 4, ... of the group; the waves' column sums meet in LDS.
__global__ void __launch_bounds__(256) act_backward_kernel(ActBwdArgs a) {
  __shared__ float sums[4][1024];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int strip = blockIdx.x % a.strips, group = blockIdx.x / a.strips;
  const int col = strip * 1024 + lane * 16;
  const int64_t m1 = min(a.M, (group + 1) * a.rows);
  float sum[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) sum[i] = 0.f;
  if (col < a.N) {
    for (int64_t m = group * a.rows + wave; m < m1; m += 4) {
      float d[16];
      quant_load16<true>(a.dc, m * a.N + col, d);
      if (a.act != DG_ACT_NONE) {
        float x[16];
        quant_load16<true>(a.pre, m * a.N + col, x);
        act_backward(d, x, a.act);
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) sum[i] += d[i];
      quantize16(d, lane & 7, m, col >> 7, a.codes, a.so);
    }
  }
  if (!a.part) return;
#pragma unroll
  for (int i = 0; i < 16; ++i) sums[wave][lane * 16 + i] = sum[i];
  __syncthreads();
  for (int i = threadIdx.x; i < 1024; i += 256)
    if (strip * 1024 + i < a.N)
      a.part[(int64_t)group * a.N + strip * 1024 + i] =
          (sums[0][i] + sums[1][i]) + (sums[2][i] + sums[3][i]);
}

// out[n] = sum of the R partial rows part[.][n], n < N (N % 16 == 0): 16 columns per
// workgroup, thread (q, r) adds rows r, r + 64, ... of columns 4q .. 4q+3, and the 64 row
// sums are added pairwise in LDS.
__global__ void __launch_bounds__(256) column_sum_kernel(const float* part, float* out, int R, int N) {
  __shared__ nk_v4f s[64][4];
  const int q = threadIdx.x & 3, r = threadIdx.x >> 2;
  const int col = blockIdx.x * 16 + q * 4;
  nk_v4f sum = {0.f, 0.f, 0.f, 0.f};
  for (int i = r; i < R; i += 64) {
    const nk_v4f v = *(const nk_v4f*)(part + (int64_t)i * N + col);
    for (int j = 0; j < 4; ++j) sum[j] += v[j];
  }
  s[r][q] = sum;
  for (int d = 32; d >= 1; d >>= 1) {
    __syncthreads();
    if (r < d) {
      for (int j = 0; j < 4; ++j) sum[j] += s[r + d][q][j];
      s[r][q] = sum;
    }
  }
  if (r == 0) *(nk_v4f*)(out + col) = sum;
}

}  // namespace dg
