// norm_kernel.hpp -- RMS norm with the residual's addition and an FP8 output with 1x128
// scales, its backward pass, and the backward pass of the GEMM's bias + activation epilogue
// with an FP8 output, for gfx950. All three are bound by HBM: each value is read once (the
// backward kernels' on few rows twice, see below) and written once, everything in between
// stays in registers, in fp32.
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
// results do not depend on scheduling. With few rows the second launch costs more than
// reading them twice: then the launch holds a second kind of workgroup, which sums 64 columns
// over all rows (direct_column_sums) and writes the result itself.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "activation.hpp"
#include "quant_kernel.hpp"

namespace dg {

typedef float nk_v2f __attribute__((ext_vector_type(2)));
typedef float nk_v4f __attribute__((ext_vector_type(4)));
typedef __bf16 nk_v2bf __attribute__((ext_vector_type(2)));

// Lanes and values. Eight neighbouring lanes own a block of 128 consecutive values, 16 each,
// as Q pieces of P values that one 16-byte access moves: piece q of lane li (0..7) starts at
// value 8 P q + P li of the block (bf16: P = 8, Q = 2; fp32: P = 4, Q = 4). Eight lanes'
// accesses then cover a whole 128-byte line. With 16 consecutive values per lane instead,
// an access touched every second (fp32: fourth) 16 bytes of twice (four times) the lines,
// and the streamed lines were fetched again for the next piece.
template <bool BF16>
struct Pieces {
  static constexpr int P = BF16 ? 8 : 4, Q = 16 / P;
};

// Two fp32 values rounded to bf16 (nearest even, NaN kept), low half first.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(nk_v2f{a, b}, nk_v2bf));
}

// A lane's 16 values as loaded, from element idx (its first piece) of an array that is read
// once; value i as fp32 with [i], i a compile-time constant.
template <bool BF16>
struct Raw16 {
  quant_v4u w[Pieces<BF16>::Q];
  __device__ __forceinline__ void load(const void* src, int64_t idx) {
    const quant_v4u* p = BF16 ? (const quant_v4u*)((const uint16_t*)src + idx)
                              : (const quant_v4u*)((const float*)src + idx);
#pragma unroll
    for (int q = 0; q < Pieces<BF16>::Q; ++q) w[q] = __builtin_nontemporal_load(p + 8 * q);
  }
  __device__ __forceinline__ float operator[](int i) const {
    if constexpr (BF16)
      return __uint_as_float(i & 1 ? w[i / 8][i / 2 % 4] & 0xFFFF0000u : w[i / 8][i / 2 % 4] << 16);
    else
      return __uint_as_float(w[i / 4][i % 4]);
  }
};

// A lane's 16 values to element idx (its first piece).
template <bool BF16>
__device__ __forceinline__ void store16(void* dst, int64_t idx, const float (&v)[16]) {
  if constexpr (BF16) {
    quant_v4u* p = (quant_v4u*)((uint16_t*)dst + idx);
#pragma unroll
    for (int q = 0; q < 2; ++q)
      __builtin_nontemporal_store(
          quant_v4u{pack_bf16(v[8 * q], v[8 * q + 1]), pack_bf16(v[8 * q + 2], v[8 * q + 3]),
                    pack_bf16(v[8 * q + 4], v[8 * q + 5]), pack_bf16(v[8 * q + 6], v[8 * q + 7])},
          p + 8 * q);
  } else {
    nk_v4f* p = (nk_v4f*)((float*)dst + idx);
#pragma unroll
    for (int q = 0; q < 4; ++q)
      __builtin_nontemporal_store(nk_v4f{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]},
                                  p + 8 * q);
  }
}

// A lane's 16 weights at the positions of its values of type BF16, kept as loaded (WBF: bf16
// weights, else fp32).
template <bool BF16, bool WBF>
struct Weight16 {
  uint32_t w[WBF ? 8 : 16];
  __device__ __forceinline__ void load(const void* src, int64_t idx) {
    constexpr int P = Pieces<BF16>::P, D = WBF ? P / 2 : P;  // dwords per piece
#pragma unroll
    for (int q = 0; q < Pieces<BF16>::Q; ++q) {
      const uint32_t* p = WBF ? (const uint32_t*)((const uint16_t*)src + idx + 8 * P * q)
                              : (const uint32_t*)((const float*)src + idx + 8 * P * q);
#pragma unroll
      for (int j = 0; j < D; ++j) w[D * q + j] = p[j];
    }
  }
  __device__ __forceinline__ float operator[](int i) const {
    if constexpr (WBF) return __uint_as_float(i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
    else return __uint_as_float(w[i]);
  }
};

// A lane's 16 fp32 column sums, at the positions of its values of type BF16.
template <bool BF16>
__device__ __forceinline__ void store_sums16(float* dst, const float (&v)[16]) {
  constexpr int P = Pieces<BF16>::P;
#pragma unroll
  for (int i = 0; i < 16; i += 4)
    *(nk_v4f*)(dst + i / P * 8 * P + i % P) = nk_v4f{v[i], v[i + 1], v[i + 2], v[i + 3]};
}

template <bool BF16>
__device__ __forceinline__ void add_sums16(const float* src, float (&v)[16]) {
  constexpr int P = Pieces<BF16>::P;
#pragma unroll
  for (int i = 0; i < 16; i += 4) {
    const nk_v4f u = *(const nk_v4f*)(src + i / P * 8 * P + i % P);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[i + j] += u[j];
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

// Data-parallel moves within a wave (v_mov_b32_dpp), without a trip through LDS.
constexpr int kDppXor1 = 0xB1, kDppXor2 = 0x4E;  // quad_perm [1,0,3,2], [2,3,0,1]
constexpr int kDppMirror8 = 0x141, kDppMirror16 = 0x140;  // lane i <- 7 - i, 15 - i
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t x) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, 0xF, 0xF, false);
}
template <int CTRL>
__device__ __forceinline__ float dppf(float x) {
  return __uint_as_float(dpp<CTRL>(__float_as_uint(x)));
}

// Largest v of 8 neighbouring lanes, in each of them (once the four lanes of a quad agree,
// the mirrored lane holds the other quad's value).
__device__ __forceinline__ float max8(float v) {
  v = fmaxf(v, dppf<kDppXor1>(v));
  v = fmaxf(v, dppf<kDppXor2>(v));
  return fmaxf(v, dppf<kDppMirror8>(v));
}

// Quantizes a lane's 16 values (type BF16's pieces) of the 1x128 block kb of row m. Each lane
// makes 4 or 8 consecutive codes per piece; neighbouring lanes trade them so that each
// stores 16 consecutive ones: lane pairs exchange halves (bf16), groups of four lanes
// transpose their 4x4 words (fp32). The scale is stored by lane li = 0.
template <bool BF16>
__device__ __forceinline__ void quantize16(const float (&y)[16], int li, int64_t m, int kb,
                                           uint8_t* codes, const ScaleOut& so) {
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(y[i]));
  const int e = scale_exp(so, max8(amax));
  uint32_t w[4];
#pragma unroll
  for (int q = 0; q < 4; ++q)
    w[q] = quant_e4m3fn_x4(ldexpf(y[4 * q], -e), ldexpf(y[4 * q + 1], -e),
                           ldexpf(y[4 * q + 2], -e), ldexpf(y[4 * q + 3], -e));
  const bool odd = li & 1;
  int off;
  quant_v4u out;
  if constexpr (BF16) {
    const uint32_t a = dpp<kDppXor1>(odd ? w[0] : w[2]), b = dpp<kDppXor1>(odd ? w[1] : w[3]);
    out = odd ? quant_v4u{a, b, w[2], w[3]} : quant_v4u{w[0], w[1], a, b};
    off = odd ? 64 + 8 * (li - 1) : 8 * li;
  } else {
    // 2x2 blocks of words, then the words inside them
    const bool hi = li & 2;
    const uint32_t a = dpp<kDppXor2>(hi ? w[0] : w[2]), b = dpp<kDppXor2>(hi ? w[1] : w[3]);
    const uint32_t t0 = hi ? a : w[0], t1 = hi ? b : w[1], t2 = hi ? w[2] : a, t3 = hi ? w[3] : b;
    const uint32_t c = dpp<kDppXor1>(odd ? t0 : t1), d = dpp<kDppXor1>(odd ? t2 : t3);
    out = odd ? quant_v4u{c, t1, d, t3} : quant_v4u{t0, c, t2, d};
    off = 32 * (li & 3) + 4 * (li & 4);
  }
  *(quant_v4u*)(codes + (m * so.KB + kb) * 128 + off) = out;
  if (li == 0) store_scale(so, m, kb, e);
}

// Workgroup barrier for LDS traffic only: global loads in flight stay in flight.
__device__ __forceinline__ void lds_barrier() {
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt 0
  __builtin_amdgcn_s_barrier();
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
}

// Sums 64 columns (from col0) over all rows, for workgroups of blockDim.x threads (a multiple
// of 64, at most NT): groups of 64 / P lanes of P values take rows r, r + groups, ...; add(m,
// col, v) adds row m's values at columns col .. col + P - 1 to v. The groups' sums are added
// in order through LDS.
template <int P, int NT, class F>
__device__ __forceinline__ void direct_column_sums(int64_t M, int col0, float* out, F add) {
  constexpr int L = 64 / P;
  __shared__ float sums[NT / L][64];
  const int groups = blockDim.x / L, r = threadIdx.x / L, c = (threadIdx.x % L) * P;
  float v[P];
#pragma unroll
  for (int i = 0; i < P; ++i) v[i] = 0.f;
  for (int64_t m = r; m < M; m += groups) add(m, col0 + c, v);
#pragma unroll
  for (int i = 0; i < P; ++i) sums[r][c + i] = v[i];
  __syncthreads();
  if (threadIdx.x < 64) {
    float s = 0.f;
    for (int i = 0; i < groups; ++i) s += sums[i][threadIdx.x];
    out[col0 + threadIdx.x] = s;
  }
}

// 16 bytes of a bf16 or fp32 array from element idx on, and their values.
template <bool BF16>
__device__ __forceinline__ quant_v4u raw_piece(const void* src, int64_t idx) {
  return *(BF16 ? (const quant_v4u*)((const uint16_t*)src + idx) : (const quant_v4u*)((const float*)src + idx));
}

template <bool BF16>
__device__ __forceinline__ void unpack_piece(const quant_v4u& u, float (&v)[Pieces<BF16>::P]) {
#pragma unroll
  for (int i = 0; i < Pieces<BF16>::P; ++i)
    v[i] = __uint_as_float(!BF16 ? u[i & 3] : i & 1 ? u[i / 2] & 0xFFFF0000u : u[i / 2] << 16);
}

// P consecutive values, bf16 (P = 8) or fp32 (P = 4).
template <bool BF16>
__device__ __forceinline__ void load_piece(const void* src, int64_t idx, float (&v)[Pieces<BF16>::P]) {
  unpack_piece<BF16>(raw_piece<BF16>(src, idx), v);
}

// Index of this workgroup among those with a part of the main work, of `work` in all; those that
// only sum columns, work and on, come first in the launch: they take longest.
__device__ __forceinline__ int sums_first(int work) {
  const int sums = (int)gridDim.x - work, b = blockIdx.x;
  return b < sums ? work + b : b - sums;
}

// direct_column_sums with NS sums of each of COLS columns, to out[0 .. NS - 1] (NULL: not stored), four
// rows' loads in flight: load(m, col) gives a row's values, add(row, m, v) adds them to
// v[0 .. NS - 1]. sums: LDS for NS * P floats of every thread. WHOLE: no test lies between the rows
// of a whole batch of four, so that their arithmetic overlaps; 512 x 2048 fp32 of dropout's gradient
// 5.9 us, 8.9 with a test at each row. Not for rows with much arithmetic, where waves with both
// whole batches and rests pay for both: 200 x 2048 of gelu's gated gradient 10.0 us, 6.8 row by row.
template <int NS, int P, int COLS, bool WHOLE, class Load, class Add>
__device__ __forceinline__ void direct_sums(int64_t M, int col0, float* const (&out)[NS], float* sums,
                                            Load load, Add add) {
  constexpr int L = COLS / P;  // lanes to a row
  static_assert(COLS % P == 0 && 64 % L == 0, "whole rows per wave");
  const int groups = blockDim.x / L, r = threadIdx.x / L, c = (threadIdx.x % L) * P;
  float v[NS][P];
#pragma unroll
  for (int k = 0; k < NS; ++k)
#pragma unroll
    for (int i = 0; i < P; ++i) v[k][i] = 0.f;
  int64_t m = r;
  decltype(load(m, col0)) row[4];
  for (; WHOLE && m + 3 * groups < M; m += 4 * groups) {
#pragma unroll
    for (int u = 0; u < 4; ++u) row[u] = load(m + u * groups, col0 + c);
#pragma unroll
    for (int u = 0; u < 4; ++u) add(row[u], m + u * groups, v);
  }
  for (; m < M; m += 4 * groups) {  // rows past the last: that one's values, not added
#pragma unroll
    for (int u = 0; u < 4; ++u) row[u] = load(min(m + u * groups, M - 1), col0 + c);
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (m + u * groups < M) add(row[u], m + u * groups, v);
  }
#pragma unroll
  for (int k = 0; k < NS; ++k)
#pragma unroll
    for (int i = 0; i < P; ++i) sums[(k * groups + r) * COLS + c + i] = v[k][i];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < NS; ++k)
    for (int n = threadIdx.x; n < COLS && out[k]; n += blockDim.x) {
      float s = 0.f;
      for (int i = 0; i < groups; ++i) s += sums[(k * groups + i) * COLS + n];
      out[k][col0 + n] = s;
    }
}

// Sum of v over a row's `waves` waves, of which `wave` is this one, the same in every
// thread, added in a fixed order. buf: one float per wave of the row, not written again
// before another barrier has passed (two buffers in turn).
__device__ __forceinline__ float row_sum(float v, float* buf, int wave, int waves) {
  v += dppf<kDppXor1>(v);
  v += dppf<kDppXor2>(v);
  v += dppf<kDppMirror8>(v);
  v += dppf<kDppMirror16>(v);
  v += __shfl_xor(v, 16, 64);
  v += __shfl_xor(v, 32, 64);
  if ((threadIdx.x & 63) == 0) buf[wave] = v;
  lds_barrier();
  float s = 0.f;
  for (int i = 0; i < waves; ++i) s += buf[i];
  return s;
}

constexpr int kNormThreads = 512;                // most threads of a workgroup
constexpr int kNormMaxK = 4 * 16 * kNormThreads;  // four 16-value chunks in each

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
};

// First value, in its row, of thread t's chunk c, `threads` threads to a row.
template <bool BF16>
__device__ __forceinline__ int norm_col(int c, int threads, int t) {
  return ((c * threads + t) >> 3) * 128 + (t & 7) * Pieces<BF16>::P;
}

// Workgroup b takes rows b, b + G, b + 2G, ... (G workgroups), its threads C chunks of 16
// values each. AHEAD: the weights stay in registers and the next row is loaded before the
// barrier of this one; otherwise (long rows, whose values fill the registers) both are loaded
// where they are used.
template <bool BF16, bool WBF, int C, bool AHEAD>
__global__ void __launch_bounds__(kNormThreads) rmsnorm_kernel(NormArgs a) {
  __shared__ float buf[2][kNormThreads / 64];
  const int K = a.K, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  int col[C];
  Weight16<BF16, WBF> w[C];
  Raw16<BF16> x[C], r[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    col[c] = norm_col<BF16>(c, blockDim.x, threadIdx.x);
    if (AHEAD && col[c] < K) w[c].load(a.w, col[c]);
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
    float ss = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if (col[c] >= K) continue;
#pragma unroll
      for (int i = 0; i < 16; ++i) v[c][i] = x[c][i];
      if (a.r) {
#pragma unroll
        for (int i = 0; i < 16; ++i) v[c][i] += r[c][i];
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) ss = __builtin_fmaf(v[c][i], v[c][i], ss);
    }
    if (AHEAD && m + gridDim.x < a.M) fetch(m + gridDim.x);
    const float rstd = 1.f / sqrtf(row_sum(ss, buf[par], wave, waves) / (float)K + a.eps);
    if (a.rstd && threadIdx.x == 0) a.rstd[m] = rstd;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if (col[c] >= K) continue;
      if (a.h) store16<BF16>(a.h, m * K + col[c], v[c]);
      if (!AHEAD) w[c].load(a.w, col[c]);
#pragma unroll
      for (int i = 0; i < 16; ++i) v[c][i] = v[c][i] * rstd * w[c][i];
      quantize16<BF16>(v[c], threadIdx.x & 7, m, col[c] >> 7, a.codes, a.so);
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
  float* part;     // [groups][K] partial dweight; NULL: workgroups from `groups` on sum it
  float* dweight;  // part == NULL: the sums
  int64_t M;
  int32_t K;
  int32_t teams;   // rows that a workgroup works on side by side
  int32_t groups;  // workgroups that take rows
};

// A workgroup is `teams` teams of threads, each on a row of its own (the columns of
// rmsnorm_kernel); team i of workgroup b takes rows b teams + i + j G teams, j = 0, 1, ...
// The weights and the column sums of dweight stay in registers; the teams' sums meet in LDS
// at the end, in team order, so that a workgroup leaves one row of partials. AHEAD: the next
// row's h and dy are loaded before the barrier of this one, and its dh behind it; otherwise
// (long rows) a row's values are kept as loaded, and the weights are read again where they
// are used.
template <bool BF16, bool WBF, int C, bool AHEAD>
__global__ void __launch_bounds__(kNormThreads) rmsnorm_backward_kernel(NormBwdArgs a) {
  __shared__ float buf[2][kNormThreads / 64];
  extern __shared__ float teams_dw[];
  const int K = a.K, R = a.teams, threads = blockDim.x / R;
  if ((int)blockIdx.x >= a.groups) {
    direct_column_sums<Pieces<BF16>::P, kNormThreads>(
        a.M, ((int)blockIdx.x - a.groups) * 64, a.dweight,
        [&](int64_t m, int c, float (&v)[Pieces<BF16>::P]) {
          float d[Pieces<BF16>::P], x[Pieces<BF16>::P];
          load_piece<BF16>(a.dy, m * K + c, d);
          load_piece<BF16>(a.h, m * K + c, x);
          const float rstd = a.rstd[m];
#pragma unroll
          for (int i = 0; i < Pieces<BF16>::P; ++i) v[i] = __builtin_fmaf(d[i], x[i] * rstd, v[i]);
        });
    return;
  }
  const int team = threadIdx.x / threads, t = threadIdx.x - team * threads;
  const int wave = t >> 6, waves = threads >> 6;
  int col[C];
  Weight16<BF16, WBF> w[C];
  float dw[C][16];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    col[c] = norm_col<BF16>(c, threads, t);
#pragma unroll
    for (int i = 0; i < 16; ++i) dw[c][i] = 0.f;
    if (AHEAD && col[c] < K) w[c].load(a.w, col[c]);
  }
  Raw16<BF16> h[C], dy[C], dh[C];
  float rs = 0.f;
  auto fetch = [&](int64_t m) {
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
      if (col[c] < K && a.dh) dh[c].load(a.dh, m * K + col[c]);
  };
  const int64_t step = (int64_t)a.groups * R;
  int64_t m = (int64_t)blockIdx.x * R + team;
  if (AHEAD && m < a.M) {
    fetch(m);
    fetch_dh(m);
  }
  // every team passes every barrier: the loop runs while team 0 has a row
  for (int par = 0; m - team < a.M; m += step, par ^= 1) {
    const bool live = m < a.M;
    if (!AHEAD && live) fetch(m);
    const float rstd = rs;
    float xh[AHEAD ? C : 1][16], g[AHEAD ? C : 1][16];
    float dot = 0.f;
    if (live) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        if (col[c] >= K) continue;
        if (!AHEAD) w[c].load(a.w, col[c]);
        const int k = AHEAD ? c : 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float d = dy[c][i];
          xh[k][i] = h[c][i] * rstd;
          dw[c][i] = __builtin_fmaf(d, xh[k][i], dw[c][i]);
          g[k][i] = d * w[c][i];
          dot = __builtin_fmaf(g[k][i], xh[k][i], dot);
        }
      }
    }
    if (AHEAD && m + step < a.M) fetch(m + step);
    const float mean = row_sum(dot, buf[par] + team * waves, wave, waves) / (float)K;
    if (live) {
      if (!AHEAD) fetch_dh(m);
#pragma unroll
      for (int c = 0; c < C; ++c) {
        if (col[c] >= K) continue;
        const int k = AHEAD ? c : 0;
        if (!AHEAD) {
          w[c].load(a.w, col[c]);
#pragma unroll
          for (int i = 0; i < 16; ++i) xh[k][i] = h[c][i] * rstd, g[k][i] = dy[c][i] * w[c][i];
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          g[k][i] = rstd * __builtin_fmaf(-xh[k][i], mean, g[k][i]);
          if (a.dh) g[k][i] += dh[c][i];
        }
        store16<BF16>(a.dx, m * K + col[c], g[k]);
      }
    }
    if (AHEAD && m + step < a.M) fetch_dh(m + step);
  }
  if (!a.part) return;
  if (R > 1) {
    if (team > 0) {
#pragma unroll
      for (int c = 0; c < C; ++c)
        if (col[c] < K) store_sums16<BF16>(teams_dw + (team - 1) * K + col[c], dw[c]);
    }
    __syncthreads();
    if (team > 0) return;
    for (int q = 0; q < R - 1; ++q)
#pragma unroll
      for (int c = 0; c < C; ++c)
        if (col[c] < K) add_sums16<BF16>(teams_dw + q * K + col[c], dw[c]);
  }
#pragma unroll
  for (int c = 0; c < C; ++c)
    if (col[c] < K) store_sums16<BF16>(a.part + (int64_t)blockIdx.x * K + col[c], dw[c]);
}

struct ActBwdArgs {
  const uint16_t* dc;
  const uint16_t* pre;  // unused with DG_ACT_NONE
  uint8_t* codes;
  ScaleOut so;
  float* part;          // [row groups][N] partial dbias; NULL: none
  float* dbias;         // part == NULL: written by workgroups from strips * groups on, if any
  int64_t M;
  int64_t rows;         // rows per row group
  int32_t N;
  int32_t act;
  int32_t strips;       // column strips of 1024
  int32_t groups;       // row groups
};

// A workgroup of four waves takes a strip of 1024 columns (8 blocks of 128, 8 lanes each)
// over a group of rows, wave w rows w, w + 4, ... of the group, the next row's loads in
// flight; the waves' column sums meet in LDS.
static __global__ void __launch_bounds__(256) act_backward_kernel(ActBwdArgs a) {
  __shared__ float sums[3][1024];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  if ((int)blockIdx.x >= a.strips * a.groups) {
    direct_column_sums<8, 256>(a.M, ((int)blockIdx.x - a.strips * a.groups) * 64, a.dbias,
                               [&](int64_t m, int c, float (&v)[8]) {
                                 float d[8], x[8];
                                 load_piece<true>(a.dc, m * a.N + c, d);
                                 if (a.act != DG_ACT_NONE) {
                                   load_piece<true>(a.pre, m * a.N + c, x);
                                   act_backward(d, x, a.act);
                                 }
#pragma unroll
                                 for (int i = 0; i < 8; ++i) v[i] += d[i];
                               });
    return;
  }
  const int strip = blockIdx.x % a.strips, group = blockIdx.x / a.strips;
  const int in_strip = (lane >> 3) * 128 + (lane & 7) * Pieces<true>::P;
  const int col = strip * 1024 + in_strip;
  const bool has_pre = a.act != DG_ACT_NONE;
  const int64_t m1 = min(a.M, (group + 1) * a.rows);
  float sum[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) sum[i] = 0.f;
  if (col < a.N) {
    Raw16<true> d, x;
    auto fetch = [&](int64_t m) {
      if (m >= m1) return;
      d.load(a.dc, m * a.N + col);
      if (has_pre) x.load(a.pre, m * a.N + col);
    };
    int64_t m = group * a.rows + wave;
    fetch(m);
    for (; m < m1; m += 4) {
      float p[16], z[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) p[i] = d[i], z[i] = has_pre ? x[i] : 0.f;
      fetch(m + 4);
      act_backward(p, z, a.act);
#pragma unroll
      for (int i = 0; i < 16; ++i) sum[i] += p[i];
      quantize16<true>(p, lane & 7, m, col >> 7, a.codes, a.so);
    }
  }
  if (!a.part) return;
  if (wave > 0) store_sums16<true>(sums[wave - 1] + in_strip, sum);
  __syncthreads();
  if (wave > 0 || col >= a.N) return;
#pragma unroll
  for (int w = 0; w < 3; ++w) add_sums16<true>(sums[w] + in_strip, sum);
  store_sums16<true>(a.part + (int64_t)group * a.N + col, sum);
}

// out[n] = sum of the R partial rows part[.][n], `pitch` values apart, and from column `split`
// on out2[n - split] (split % 32 == 0): a workgroup takes 32 columns (a 128-byte line of each
// row), thread (q, r) rows r, r + 32, ... of columns 4q .. 4q+3 with eight loads in flight (past
// the last row: the last row again, not added), and the 32 row sums are added pairwise in LDS.
static __global__ void __launch_bounds__(256) column_sum_kernel(const float* part, float* out, int R,
                                                                int pitch, float* out2, int split) {
  __shared__ nk_v4f s[32][8];
  constexpr int U = 8;
  const int q = threadIdx.x & 7, r = threadIdx.x >> 3;
  const int col = blockIdx.x * 32 + q * 4;
  nk_v4f sum = {0.f, 0.f, 0.f, 0.f};
  for (int i = r; i < R; i += 32 * U) {
    nk_v4f v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = *(const nk_v4f*)(part + (int64_t)min(i + 32 * u, R - 1) * pitch + col);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int j = 0; j < 4; ++j) sum[j] += i + 32 * u < R ? v[u][j] : 0.f;
  }
  s[r][q] = sum;
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) {
    __syncthreads();
    if (r < d) {
#pragma unroll
      for (int j = 0; j < 4; ++j) sum[j] += s[r + d][q][j];
      s[r][q] = sum;
    }
  }
  if (r == 0) *(nk_v4f*)(col < split ? out + col : out2 + (col - split)) = sum;
}

}  // namespace dg
