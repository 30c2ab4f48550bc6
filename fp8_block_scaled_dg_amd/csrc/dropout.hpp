// dropout.hpp -- dropout from a counter-based generator, for gfx950: the mask is a function of
// the element's index, a seed and an offset, so that the backward pass forms it again and
// nothing stores it.
//
//   threshold = round(65536 p);  r_i = 16 random bits of element i (row-major index)
//   dropout(x)_i = r_i >= threshold ? x_i 65536 / (65536 - threshold) : 0
// Bits: Philox 4x32 with 7 rounds (Salmon, Moraes, Dror, Shaw, "Parallel random numbers: as
// easy as 1, 2, 3", 2011, where 7 rounds are the fewest that pass BigCrush), one block of four
// words per eight elements: key = the seed's words, counter = the words of i / 8, then those of
// offset + subsequence; element i takes half i % 2 (low first) of word (i % 8) / 2. 16 bits an
// element, not 32: the two kinds of multiplication of a round run at a quarter of the rate of
// an addition and bound the generator, and p is still met to 2^-17. Seed and offset are read on
// the device, so that a captured graph draws new masks when its caller changes them.
#pragma once

#include "norm_kernel.hpp"

namespace dg {

struct DropArgs {
  const uint64_t* rng;  // seed, offset
  uint64_t subsequence;
  uint32_t threshold;  // 0 .. 65535; 0 keeps everything
  float scale;
};

// The generator of one call: scalars.
struct Drop {
  uint32_t k0, k1, o0, o1, threshold;
  float scale;
  __device__ __forceinline__ explicit Drop(const DropArgs& a)
      : k0(0), k1(0), o0(0), o1(0), threshold(a.threshold << 16), scale(a.scale) {
    if (!a.rng) return;
    const uint64_t seed = a.rng[0], offset = a.rng[1] + a.subsequence;
    k0 = __builtin_amdgcn_readfirstlane((uint32_t)seed);
    k1 = __builtin_amdgcn_readfirstlane((uint32_t)(seed >> 32));
    o0 = __builtin_amdgcn_readfirstlane((uint32_t)offset);
    o1 = __builtin_amdgcn_readfirstlane((uint32_t)(offset >> 32));
  }
  // the four words of elements 8 group .. 8 group + 7
  __device__ __forceinline__ quant_v4u words(int64_t group) const {
    uint32_t c0 = (uint32_t)group, c1 = (uint32_t)((uint64_t)group >> 32), c2 = o0, c3 = o1;
#pragma unroll
    for (int r = 0; r < 7; ++r) {
      const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
      c0 = (uint32_t)(b >> 32) ^ c1 ^ (k0 + (uint32_t)r * 0x9E3779B9u);
      c2 = (uint32_t)(a >> 32) ^ c3 ^ (k1 + (uint32_t)r * 0xBB67AE85u);
      c1 = (uint32_t)b;
      c3 = (uint32_t)a;
    }
    return quant_v4u{c0, c1, c2, c3};
  }
  // x, or 0 where the low (high) half of w says so
  __device__ __forceinline__ float low(float x, uint32_t w) const {
    return (w << 16) >= threshold ? x * scale : 0.f;
  }
  __device__ __forceinline__ float high(float x, uint32_t w) const {
    return w >= threshold ? x * scale : 0.f;
  }
};

// Neighbouring lanes with four values each share a group: the even lane gives words 2, 3 of its
// group a and takes words 0, 1 of the odd lane's group b, which takes the even one's in turn.
// mine: the two words of this lane's own group (a in even lanes, b in odd ones), other: those
// of the neighbour's.
__device__ __forceinline__ void trade_words(const quant_v4u& w, bool odd, uint32_t (&mine)[2],
                                            uint32_t (&other)[2]) {
  mine[0] = odd ? w[2] : w[0], mine[1] = odd ? w[3] : w[1];
  other[0] = dpp<kDppXor1>(odd ? w[0] : w[2]), other[1] = dpp<kDppXor1>(odd ? w[1] : w[3]);
}

// Dropout of a lane's 16 values of a 1x128 block (type BF16's pieces); idx: the index of the
// first. bf16: each piece is a group. fp32: a piece is half of one, so of the four groups that
// two neighbouring lanes share the even lane forms two and the odd lane the others.
template <bool BF16>
__device__ __forceinline__ void drop16(const Drop& d, int64_t idx, float (&v)[16]) {
  if constexpr (BF16) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const quant_v4u w = d.words((idx >> 3) + 8 * q);
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        v[8 * q + i] = d.low(v[8 * q + i], w[i / 2]);
        v[8 * q + i + 1] = d.high(v[8 * q + i + 1], w[i / 2]);
      }
    }
  } else {
    const bool odd = (idx >> 2) & 1;
    uint32_t w[4][2];  // pieces 0, 1: the even lane's groups, 2, 3: the odd lane's
    uint32_t mine[2][2], other[2][2];
#pragma unroll
    for (int q = 0; q < 2; ++q)
      trade_words(d.words((idx >> 3) + 4 * (2 * odd + q)), odd, mine[q], other[q]);
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        w[q][j] = odd ? other[q][j] : mine[q][j];
        w[2 + q][j] = odd ? mine[q][j] : other[q][j];
      }
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        v[4 * q + 2 * j] = d.low(v[4 * q + 2 * j], w[q][j]);
        v[4 * q + 2 * j + 1] = d.high(v[4 * q + 2 * j + 1], w[q][j]);
      }
  }
}

// P consecutive values of one piece (load_piece), idx a multiple of P.
template <bool BF16>
__device__ __forceinline__ void drop_piece(const Drop& d, int64_t idx, float (&v)[Pieces<BF16>::P]) {
  const quant_v4u w = d.words(idx >> 3);
  const bool odd = !BF16 && ((idx >> 2) & 1);
#pragma unroll
  for (int i = 0; i < Pieces<BF16>::P; i += 2) {
    const uint32_t u = BF16 ? w[i / 2] : odd ? w[(2 + i / 2) & 3] : w[i / 2];
    v[i] = d.low(v[i], u);
    v[i + 1] = d.high(v[i + 1], u);
  }
}

// ---------------------------------------------------------------- out = dropout(x) + residual

struct DropAddArgs {
  const void* x;
  const void* r;  // NULL: no residual
  void* out;
  int64_t n;
  DropArgs drop;
};

constexpr int kDropThreads = 256, kDropUnroll = 2;
constexpr int64_t kDropChunk = 512;  // values that a wave takes per step

// 16 bytes of type BF16 of fp32 values.
template <bool BF16>
__device__ __forceinline__ quant_v4u pack_piece(const float (&v)[Pieces<BF16>::P]) {
  if constexpr (BF16)
    return quant_v4u{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                     pack_bf16(v[6], v[7])};
  else
    return quant_v4u{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                     __float_as_uint(v[3])};
}

template <bool BF16>
__device__ __forceinline__ float load_one(const void* src, int64_t i) {
  if constexpr (BF16) return __uint_as_float((uint32_t)((const uint16_t*)src)[i] << 16);
  else return ((const float*)src)[i];
}

// A wave takes 512 values at a time, a lane one group of eight: bf16, 16 bytes; fp32, two
// pieces of 16 bytes, 256 values apart, so that a wave's accesses cover whole lines, each
// piece half of a group that the neighbouring lane shares. Two steps' loads are in flight
// before the first is worked on. Bound by HBM: 4096 x 7168 bf16 with residual 30.5 us, 176 MB at
// 5.8 TB/s.
template <bool BF16>
__global__ void __launch_bounds__(kDropThreads) dropout_add_kernel(DropAddArgs a) {
  constexpr int P = Pieces<BF16>::P, Q = 8 / P, U = kDropUnroll;
  const Drop d(a.drop);
  const int lane = threadIdx.x & 63;
  const bool odd = lane & 1;
  const int64_t step = (int64_t)gridDim.x * (kDropThreads / 64) * kDropChunk;
  int64_t base = ((int64_t)blockIdx.x * (kDropThreads / 64) + (threadIdx.x >> 6)) * kDropChunk;
  const uint32_t e = BF16 ? 2 : 4;
  for (; base < a.n; base += U * step) {
    quant_v4u x[U][Q], r[U][Q];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        const int64_t i = base + u * step + 64 * P * q + P * lane;
        x[u][q] = r[u][q] = quant_v4u{0, 0, 0, 0};
        if (i + P <= a.n) {
          x[u][q] = __builtin_nontemporal_load((const quant_v4u*)((const uint8_t*)a.x + i * e));
          if (a.r) r[u][q] = __builtin_nontemporal_load((const quant_v4u*)((const uint8_t*)a.r + i * e));
        }
      }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t b = base + u * step;
      if (b >= a.n) break;  // the same for the whole wave
      uint32_t w[Q][P / 2];
      if constexpr (BF16) {
        const quant_v4u t = d.words((b >> 3) + lane);
#pragma unroll
        for (int j = 0; j < 4; ++j) w[0][j] = t[j];
      } else {
        uint32_t mine[2], other[2];
        trade_words(d.words((b >> 3) + 32 * odd + (lane >> 1)), odd, mine, other);
#pragma unroll
        for (int j = 0; j < 2; ++j) w[0][j] = odd ? other[j] : mine[j], w[1][j] = odd ? mine[j] : other[j];
      }
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        const int64_t i = b + 64 * P * q + P * lane;
        float v[P], s[P];
        if (i + P <= a.n) {
          unpack_piece<BF16>(x[u][q], v);
          unpack_piece<BF16>(r[u][q], s);
#pragma unroll
          for (int k = 0; k < P; k += 2) {
            v[k] = d.low(v[k], w[q][k / 2]);
            v[k + 1] = d.high(v[k + 1], w[q][k / 2]);
          }
          if (a.r) {
#pragma unroll
            for (int k = 0; k < P; ++k) v[k] += s[k];
          }
          __builtin_nontemporal_store(pack_piece<BF16>(v), (quant_v4u*)((uint8_t*)a.out + i * e));
        } else if (i < a.n) {  // the last values of a tensor that does not end with a piece
#pragma unroll
          for (int k = 0; k < P; ++k) {
            if (i + k >= a.n) continue;
            const float y = load_one<BF16>(a.x, i + k);
            float t = k & 1 ? d.high(y, w[q][k / 2]) : d.low(y, w[q][k / 2]);
            if (a.r) t += load_one<BF16>(a.r, i + k);
            if constexpr (BF16) ((uint16_t*)a.out)[i + k] = (uint16_t)pack_bf16(t, 0.f);
            else ((float*)a.out)[i + k] = t;
          }
        }
      }
    }
  }
}

// ---------------------------------------------------------------- its gradient, FP8 output

constexpr int kDropDirectCols = 32;  // columns of a workgroup that only sums

struct DropBwdArgs {
  const void* dy;
  uint8_t* codes;
  ScaleOut so;
  float* part;   // [row groups][K] partial dbias; NULL: none
  float* dbias;  // part == NULL: written by further workgroups, if any
  int64_t M;
  int64_t rows;  // rows per row group
  int32_t K;
  int32_t strips;  // column strips of 1024
  int32_t groups;  // row groups
  DropArgs drop;
};

// p = dropout(dy): codes and scales of p, dbias = sum of p over rows. The layout of
// act_backward_kernel. Bound by HBM: 4096 x 7168 fp32 28.8 us, 147 MB at 5.1 TB/s, 33.5 with dbias and
// its second launch; 1000 x 2048 4.7 and 8.2.
template <bool BF16>
__global__ void __launch_bounds__(256) dropout_backward_kernel(DropBwdArgs a) {
  __shared__ float sums[3][1024];
  const Drop drop(a.drop);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int work = a.strips * a.groups, index = sums_first(work);
  if (index >= work) {
    constexpr int P = Pieces<BF16>::P;
    struct Row {
      quant_v4u dy;
      int c;
    };
    direct_sums<1, P, kDropDirectCols, true>(
        a.M, (index - work) * kDropDirectCols, {a.dbias}, &sums[0][0],
        [&](int64_t m, int c) {
          return Row{raw_piece<BF16>(a.dy, m * a.K + c), c};
        },
        [&](const Row& row, int64_t m, float (&v)[1][P]) {
          float d[P];
          unpack_piece<BF16>(row.dy, d);
          drop_piece<BF16>(drop, m * a.K + row.c, d);
#pragma unroll
          for (int i = 0; i < P; ++i) v[0][i] += d[i];
        });
    return;
  }
  const int strip = index % a.strips, group = index / a.strips;
  const int in_strip = (lane >> 3) * 128 + (lane & 7) * Pieces<BF16>::P;
  const int col = strip * 1024 + in_strip;
  const int64_t m1 = min(a.M, (group + 1) * a.rows);
  float sum[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) sum[i] = 0.f;
  if (col < a.K) {
    Raw16<BF16> d;
    auto fetch = [&](int64_t m) {
      if (m < m1) d.load(a.dy, m * a.K + col);
    };
    int64_t m = group * a.rows + wave;
    fetch(m);
    for (; m < m1; m += 4) {
      float p[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) p[i] = d[i];
      fetch(m + 4);
      drop16<BF16>(drop, m * a.K + col, p);
#pragma unroll
      for (int i = 0; i < 16; ++i) sum[i] += p[i];
      quantize16<BF16>(p, lane & 7, m, col >> 7, a.codes, a.so);
    }
  }
  if (!a.part) return;
  if (wave > 0) store_sums16<BF16>(sums[wave - 1] + in_strip, sum);
  __syncthreads();
  if (wave > 0 || col >= a.K) return;
#pragma unroll
  for (int w = 0; w < 3; ++w) add_sums16<BF16>(sums[w] + in_strip, sum);
  store_sums16<BF16>(a.part + (int64_t)group * a.K + col, sum);
}

}  // namespace dg
