// epilogue.hpp -- what the dense GEMM can do to an fp32 output value before its one rounding:
//
//   z = acc + bias[n];  pre[m][n] = bf16(z) (optional)
//   kEpiBf16: C[m][n] = bf16(act(z) + residual[m][n])
//   kEpiFp8:  codes and scales of act(z), quantized per 1x128 block (quant_kernel.hpp)
//
// The GEMM kernels pass their fp32 tile through LDS and hand each lane eight consecutive
// columns of one row at a time, so that the bias is read once per lane and the residual,
// pre and C move in 16-byte pieces of whole row segments.
#pragma once

#include "gemm_kernel.hpp"
#include "norm_kernel.hpp"

namespace dg {

enum Epi : int { kEpiNone = 0, kEpiBf16 = 1, kEpiFp8 = 2 };

struct Epilogue {
  const void* bias;          // [N] bf16 or fp32; NULL: none
  const uint16_t* residual;  // [M][N] bf16; NULL: none (may be C itself)
  uint16_t* pre;             // [M][N] bf16; NULL: not stored
  uint8_t* codes;            // kEpiFp8: e4m3fn [M][N]
  ScaleOut so;               // kEpiFp8: scales, so.KB = N / 128
  int32_t bias_bf16;
  int32_t act;
};

// bias of columns col .. col + 7 (zero without one)
__device__ __forceinline__ void epi_bias8(const Epilogue& ep, int64_t col, float (&b)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) b[i] = 0.f;
  if (!ep.bias) return;
  if (ep.bias_bf16) {
    const v4u u = *(const v4u*)((const uint16_t*)ep.bias + col);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      b[2 * j] = __uint_as_float(u[j] << 16);
      b[2 * j + 1] = __uint_as_float(u[j] & 0xFFFF0000u);
    }
  } else {
    const v4f* p = (const v4f*)((const float*)ep.bias + col);
    const v4f x = p[0], y = p[1];
#pragma unroll
    for (int j = 0; j < 4; ++j) b[j] = x[j], b[4 + j] = y[j];
  }
}

__device__ __forceinline__ v4u epi_pack8(const float (&v)[8]) {
  return v4u{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
             pack_bf16(v[6], v[7])};
}

// v (products at row, col .. col + 7, element offset off = row * N + col) -> act(v + b),
// storing pre on the way
__device__ __forceinline__ void epi_act8(const Epilogue& ep, const float (&b)[8], int64_t off,
                                         float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] += b[i];
  if (ep.pre) __builtin_nontemporal_store(epi_pack8(v), (v4u*)(ep.pre + off));
  act_apply(v, ep.act);
}

// + residual, one rounding, store
__device__ __forceinline__ void epi_store8(v4u res, uint16_t* C, int64_t off, float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] += __uint_as_float(res[j] << 16);
    v[2 * j + 1] += __uint_as_float(res[j] & 0xFFFF0000u);
  }
  __builtin_nontemporal_store(epi_pack8(v), (v4u*)(C + off));
}

// Row pitch, in floats, of the fp32 tile that the ring kernel leaves in LDS: 4 floats
// past BN spread the rows over the banks.
template <int BN>
constexpr int kEpiPitch = BN + 4;

// Finishes ROWS rows of the fp32 tile of columns n0 .. n0 + BN - 1, held in
// out[ROWS][kEpiPitch<BN>]: 8 columns of a row per thread and step. load() fetches bias and
// residual, which needs nothing of the product and may be called long before finish().
// kEpiFp8: BN = 128, 16 neighbouring lanes hold a row's 1x128 block.
template <int BN, int NT, int EPI, int ROWS>
struct EpiTile {
  static_assert(EPI != kEpiFp8 || BN == 128, "a scale block per tile row");
  static constexpr int LPR = BN / 8;  // lanes per row
  static constexpr int STEPS = (ROWS * LPR + NT - 1) / NT;
  static_assert(64 % LPR == 0 && (ROWS * LPR) % 64 == 0 && NT % LPR == 0, "whole rows per wave");
  v4u res[EPI == kEpiBf16 ? STEPS : 1];
  v4u bias[2];  // as stored: unpacking it here would wait for it

  __device__ __forceinline__ void load(const Problem& p, int64_t n0, const Epilogue& ep, int row0) {
    const int64_t col = n0 + (int)(threadIdx.x % LPR) * 8;
    bias[0] = bias[1] = v4u{0, 0, 0, 0};
    if (ep.bias && col < p.N) {
      const v4u* src = ep.bias_bf16 ? (const v4u*)((const uint16_t*)ep.bias + col)
                                    : (const v4u*)((const float*)ep.bias + col);
      bias[0] = src[0];
      if (!ep.bias_bf16) bias[1] = src[1];
    }
    if (EPI != kEpiBf16) return;
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      const int rl = (threadIdx.x + i * NT) / LPR;
      res[i] = v4u{0, 0, 0, 0};
      if (ep.residual && rl < ROWS && row0 + rl < p.M && col < p.N)
        res[i] = __builtin_nontemporal_load((const v4u*)(ep.residual + (row0 + rl) * p.N + col));
    }
  }

  // all threads of the workgroup, after a barrier behind the writes of out
  __device__ __forceinline__ void finish(const Problem& p, int64_t n0, const float* out,
                                         const Epilogue& ep, int row0) {
    const int col0 = (int)(threadIdx.x % LPR) * 8;
    const int64_t col = n0 + col0;
    float b[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t u = bias[0][j / 2], half = j & 1 ? u & 0xFFFF0000u : u << 16;
      b[j] = __uint_as_float(ep.bias_bf16 ? half : bias[j / 4][j % 4]);
    }
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      const int rl = (threadIdx.x + i * NT) / LPR, row = row0 + rl;
      if (rl >= ROWS || row >= p.M || col >= p.N) continue;
      const int64_t off = row * p.N + col;
      float x[8];
      const v4f lo = *(const v4f*)(out + rl * kEpiPitch<BN> + col0);
      const v4f hi = *(const v4f*)(out + rl * kEpiPitch<BN> + col0 + 4);
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = lo[j], x[4 + j] = hi[j];
      epi_act8(ep, b, off, x);
      if (EPI == kEpiBf16) {
        epi_store8(res[i], p.C, off, x);
      } else {
        float m = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(x[j]));
        m = max8(m);
        const int e = scale_exp(ep.so, fmaxf(m, dppf<kDppMirror16>(m)));
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = ldexpf(x[j], -e);
        *(uint2*)(ep.codes + off) =
            make_uint2(quant_e4m3fn_x4(x[0], x[1], x[2], x[3]), quant_e4m3fn_x4(x[4], x[5], x[6], x[7]));
        if (col0 == 0) store_scale(ep.so, row, (int)(col >> 7), e);
      }
    }
  }
};

}  // namespace dg
