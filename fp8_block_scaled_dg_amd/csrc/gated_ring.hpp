// gated_ring.hpp -- the gated feed-forward product for few rows or few tiles, gfx950: tiles of
// 16, 32 or 64 rows by 128 gate and the same 128 up columns, so that one workgroup holds whole
// 1x128 blocks of h.
//
// B's rows come by LDS DMA as in the ring kernel (ring_kernel.hpp): 256 contiguous bytes of
// every row at a time, a pair of K-blocks, which HBM serves faster than 128. A chunk is a pair
// of blocks of the tile's 128 gate or 128 up rows, 32 KB; gate and up chunks alternate through a
// ring of three. A's pair (16 KB at 64 rows) and the scales arrive with the gate chunk, once for
// both, in a ring of their own. 64 KB of B and A's part are in flight all the time.
//
// A wave owns the same rows and columns of gate and up, TM x TN tiles of 16x16 each. Fragments
// are read from LDS one block ahead of the MFMAs that use them: a chunk's second block while its
// first is multiplied, the next chunk's first block (and A's next pair, kept in registers for
// gate and up) behind the barrier while the second is. So a chunk costs one wait (vmcnt) and one
// barrier, in the middle of its MFMAs: every wave's DMAs of the next chunk have landed, and
// every wave has read this one, whose slot is refilled at once. Reads, MFMAs and promotion
// (two-level accumulation: DeepGEMM launch article, deepseek.csdn.net, section 1.2 "precision
// safeguards") then overlap within a wave as well as between the two waves of a SIMD.
//
// No branch lies between the steps of the loop. DMAs past the run's end take a resource
// without records: they write zeros, fetch nothing, and keep the counts of the waits the same.
// The second block of an odd run's last pair is zeroed the same way, A, B and scales, by offsets
// out of range in the lanes that would bring it.
//
// A chunk's DMAs are issued one or two at a time behind the MFMAs between two barriers; all at
// once behind the barrier, M = 1000, I = 2048, K = 7168 took 45.1 us instead of 44.1, 512 rows 31.0
// instead of 30.3 (one row the same). Times here are of launches in a graph, with so many weights in
// turn that each comes from HBM.
//
// What bounds it: with B beyond its L2, a CU takes in about 62 KB/us by LDS DMA, which is 64 KB
// in flight at 1.1 us, however deep the ring, in 128- or 256-byte pieces (that product, one tile per
// CU: 44 - 46 us, 36 - 40 with three weights in turn, in part from the caches; the DMAs alone, without
// reads and MFMAs, 43; with B's lines in L2 36), and HBM gives all CUs together 5.2 TB/s (64 x 18432 x
// 7168, 264 MB of B: 56 us; 1 x 18432 x 7168: 48). B in registers, 64 bytes of 16 rows per load, took
// 70 us for the first and 80 for the second; four waves of 64 x 64 of each half 52.7 and 58.5. A product
// of one row (1 x 2048 x 7168, 29 MB: 12.8 us at 5.7 for the bytes) waits for the launch, the first
// bytes and the splits' trip through memory.
//
// The FP8 MFMA sums its 128 products in fewer bits than fp32, as in every GEMM of the library: on normal
// operands 1.2 % of pre's bf16 values are the exact product's other neighbour (0.1 % where the sum is
// fp32) and 0.1 - 0.2 % of the codes differ by a step. K-blocks, splits, bias, activation and product
// are summed in fp32.
//
// S > 1 K splits: fp32 partials (rows below M only) and an arrival count per tile; the last
// split to arrive adds all of them in split order (splitk_arrive), so results are deterministic.
#pragma once

#include "epilogue.hpp"
#include "gemm_kernel.hpp"
#include "pipe_kernel.hpp"

namespace dg {

// Eight waves as WM x 8 / WM.
template <int WM_, int TM_, int TN_, bool PACKED_, bool STREAM_B_>
struct GatedCfg {
  static constexpr int W = 8, NT = 512, WM = WM_, WN = W / WM, TM = TM_, TN = TN_;
  static constexpr bool PACKED = PACKED_;      // sfA in the packed UE8M0 form
  static constexpr bool STREAM_B = STREAM_B_;  // B's lines leave room in the caches for A's
  static constexpr int BM = 16 * WM * TM;
  static constexpr int ROW = 2 * kKBlock;                   // bytes of a row per pair
  static constexpr int A_ROWS = BM < 4 * W ? 4 * W : BM;    // staged: whole DMAs for every wave
  static constexpr int A_DMA = A_ROWS / 4 / W, B_DMA = 4;  // 1 KB DMAs per wave
  static constexpr int OPS_UP = B_DMA, OPS_GATE = B_DMA + A_DMA + 1;
  static constexpr int OFF_S = A_ROWS * ROW;  // scales: four 16-row groups of A, then B's
  static constexpr int A_STAGE = OFF_S + 5 * 256;
  static_assert(WN * TN == 8 && BM <= 64, "128 columns of each half, four groups of rows");
};

struct GatedArgs {
  Problem p;           // N = 2 I
  float* ws;           // [tiles][S][2 BM 128] fp32 partials (S > 1)
  uint32_t* counters;  // [tiles], zero between calls
  int32_t S, KS;       // K splits, K-blocks per split (even; the last may have fewer)
  int32_t tiles_m;     // row tiles
  Epilogue ep;
};

constexpr int kGatedChunk = 128 * 2 * kKBlock;
template <int I>
__shared__ __align__(16) uint8_t gated_chunk[kGatedChunk];
template <int BYTES, int I>
__shared__ __align__(16) uint8_t gated_a[BYTES];

template <class Cfg>
struct GatedSrc {
  const uint8_t *a, *gate, *up, *s;             // first byte of the run, of the scales
  uint32_t a_bytes, b_bytes, s_bytes;           // records behind them
  uint32_t a_off[Cfg::A_DMA], b_off[Cfg::B_DMA], s_off;
  // 2^31, out of every range, in the lanes that bring the second block of a pair: of rows with
  // r % 16 < 8 (the other rows' chunks are swapped), and of the scales
  uint32_t second, s_second;
  int s_shift;      // the scales' scalar offset is (kb >> s_shift) * 4
  int wave, kb0, pairs;  // kb0 is even
  bool odd;         // the last pair has one block
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t gated_rsrc(const uint8_t* p, uint32_t bytes, bool live) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p), 0, live ? (int)bytes : 0, 0x00020000);
}

// DMAs [LO, HI) of the chunk of pair t, into slot I: the gate rows' (UP false: the scales first,
// then A's pair into slot T of its ring, then B) or the up rows'.
template <class Cfg, bool UP, int I, int T, int LO, int HI>
__device__ __forceinline__ void gated_issue(const GatedSrc<Cfg>& src, int t) {
#if defined(__HIP_DEVICE_COMPILE__)
  typedef __attribute__((address_space(3))) void* lds_ptr;
  constexpr int kPolicyB = Cfg::STREAM_B ? 2 : 0;  // 2: non-temporal
  constexpr int B0 = UP ? 0 : 1 + Cfg::A_DMA;      // first DMA of B
  t = __builtin_amdgcn_readfirstlane(t);
  const bool live = t < src.pairs, half = src.odd && t == src.pairs - 1;
  const uint32_t skip[2] = {half ? src.second : 0, half ? src.second ^ 0x80000000u : 0};
  uint8_t* st = gated_a<Cfg::A_STAGE, T>;
  const __amdgpu_buffer_rsrc_t ra = gated_rsrc(src.a, src.a_bytes, live);
  const __amdgpu_buffer_rsrc_t rb = gated_rsrc(UP ? src.up : src.gate, src.b_bytes, live);
#pragma unroll
  for (int op = LO; op < HI; ++op) {
    if (!UP && op == 0) {
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          gated_rsrc(src.s, src.s_bytes, live),
          (lds_ptr)(st + Cfg::OFF_S + (src.wave < 4 ? src.wave : 4) * 256), 4,
          src.s_off | (half ? src.s_second : 0), ((src.kb0 + 2 * t) >> src.s_shift) << 2, 0, 0);
    } else if (op < B0) {
      const int q = op - 1;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_ptr)(st + (src.wave * Cfg::A_DMA + q) * 1024), 16,
                                               src.a_off[q] | skip[((src.wave * Cfg::A_DMA + q) >> 1) & 1],
                                               t * Cfg::ROW, 0, 0);
    } else {
      const int q = op - B0;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (lds_ptr)(gated_chunk<I> + (src.wave * Cfg::B_DMA + q) * 1024),
                                               16, src.b_off[q] | skip[(q >> 1) & 1], t * Cfg::ROW, 0, kPolicyB);
    }
  }
#endif
}

// 128 bytes (block h of the pair) of row `row`: lane group g holds k in [16g, 16g + 16) and
// [64 + 16g, 80 + 16g), for both operands. 16-byte chunk c of row r sits at c ^ (r % 16).
__device__ __forceinline__ v8i gated_frag(const uint8_t* tile, int row, int h, int g) {
  const uint8_t* p = tile + row * 2 * kKBlock;
  const v4u lo = *(const v4u*)(p + (((8 * h + g) ^ (row & 15)) << 4));
  const v4u hi = *(const v4u*)(p + (((8 * h + g + 4) ^ (row & 15)) << 4));
  return v8i{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3],
             (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
}

// A's fragments and scales of a pair.
template <class Cfg>
struct GatedA {
  v8i f[2][Cfg::TM];
  float s[2][Cfg::TM];
  template <int T>
  __device__ __forceinline__ void read(const GatedSrc<Cfg>& src, int t, int g, int l16) {
    const uint8_t* st = gated_a<Cfg::A_STAGE, T>;
    const int wm = src.wave / Cfg::WN;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < Cfg::TM; ++i) {
        const int tile = wm * Cfg::TM + i;
        f[h][i] = gated_frag(st, tile * 16 + l16, h, g);
        const uint32_t w = *(const uint32_t*)(st + Cfg::OFF_S + tile * 256 + (16 * h + l16) * 4);
        // packed: kb0 + 2 t is even, so both blocks lie in one word
        const int shift = Cfg::PACKED ? ((src.kb0 + 2 * t + h) & 3) * 8 : 0;
        s[h][i] = Cfg::PACKED ? ue8m0_value((w >> shift) & 0xFFu) : __uint_as_float(w);
        // the byte behind an odd run's last one may be anything
        if (Cfg::PACKED && h == 1 && src.odd && t == src.pairs - 1) s[h][i] = 0.f;
      }
  }
};

template <class Cfg, int I>
__device__ __forceinline__ void gated_read_b(v8i (&f)[Cfg::TN], int wave, int h, int g, int l16) {
  const int wn = wave % Cfg::WN;
#pragma unroll
  for (int j = 0; j < Cfg::TN; ++j) f[j] = gated_frag(gated_chunk<I>, (wn * Cfg::TN + j) * 16 + l16, h, g);
}

// acc += a b sa sb for one block, with the DMAs of issue.template op<n>() behind MFMA n, and a tile's
// promotion behind the next tile's.
template <class Cfg, int N, class Issue>
__device__ __forceinline__ void gated_mma_from(v4f (&acc)[Cfg::TM][Cfg::TN], const v8i (&a)[Cfg::TM],
                                               const v8i (&b)[Cfg::TN], const float (&s)[Cfg::TM], v4f before,
                                               const Issue& issue) {
  constexpr int TN = Cfg::TN, TILES = Cfg::TM * TN;
  v4f part = before;
  if constexpr (N < TILES) {
    part = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b[N % TN], a[N / TN], v4f{0.f, 0.f, 0.f, 0.f}, 0, 0, 0,
                                                            0, 0, 0);
    issue.template op<N>();
  }
  if constexpr (N > 0) {
    constexpr int I = (N - 1) / TN, J = (N - 1) % TN;
#pragma unroll
    for (int q = 0; q < 4; ++q) acc[I][J][q] = __builtin_fmaf(before[q], s[I], acc[I][J][q]);
    // the promotion stays in the MFMAs' basic block (ring_block says why)
    asm volatile("" : "+v"(acc[I][J]));
  }
  __builtin_amdgcn_sched_barrier(0);
  if constexpr (N < TILES) gated_mma_from<Cfg, N + 1>(acc, a, b, s, part, issue);
}

template <class Cfg, class Issue>
__device__ __forceinline__ void gated_mma(v4f (&acc)[Cfg::TM][Cfg::TN], const v8i (&a)[Cfg::TM],
                                          const v8i (&b)[Cfg::TN], const float (&sa)[Cfg::TM], float sb,
                                          const Issue& issue) {
  float s[Cfg::TM];
#pragma unroll
  for (int i = 0; i < Cfg::TM; ++i) s[i] = sa[i] * sb;
  gated_mma_from<Cfg, 0>(acc, a, b, s, v4f{0.f, 0.f, 0.f, 0.f}, issue);
}

// The DMAs of a chunk over the MFMAs of two blocks (HALF 0, 1), between one barrier and the next.
template <class Cfg, bool UP, int I, int T, int HALF>
struct GatedIssue {
  const GatedSrc<Cfg>& src;
  int t;
  template <int N>
  __device__ __forceinline__ void op() const {
    constexpr int TILES = Cfg::TM * Cfg::TN, OPS = UP ? Cfg::OPS_UP : Cfg::OPS_GATE;
    gated_issue<Cfg, UP, I, T, (HALF * TILES + N) * OPS / (2 * TILES), (HALF * TILES + N + 1) * OPS / (2 * TILES)>(
        src, t);
  }
};

// Wait until at most N of this wave's DMAs are in flight and its LDS reads are done, then the
// workgroup's barrier.
template <int N>
__device__ __forceinline__ void gated_sync() {
  __builtin_amdgcn_sched_barrier(0);
  wait_vm_lgkm0<N>();
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
}

// Pair t, T = t % 3: chunks 2 t and 2 t + 1 in slots 2 T % 3 and (2 T + 1) % 3, A in slot T. `a`
// holds the pair's A and `b0` the gate chunk's first block on entry, the next pair's on exit. The
// gate chunk of pair t + 1 is half issued on entry, that of pair t + 2 on exit.
template <class Cfg, int T>
__device__ __forceinline__ void gated_pair(v4f (&gate)[Cfg::TM][Cfg::TN], v4f (&up)[Cfg::TM][Cfg::TN],
                                           GatedA<Cfg>& a, v8i (&b0)[Cfg::TN], const GatedSrc<Cfg>& src,
                                           int t, int g, int l16) {
  constexpr int G = 2 * T % 3, U = (2 * T + 1) % 3, NEXT = (2 * T + 2) % 3;
  const float* sb = (const float*)(gated_a<Cfg::A_STAGE, T> + Cfg::OFF_S + 1024);
  const float g0 = sb[0], g1 = sb[1], u0 = sb[2], u1 = sb[3];
  v8i b1[Cfg::TN];
  gated_read_b<Cfg, G>(b1, src.wave, 1, g, l16);
  __builtin_amdgcn_sched_barrier(0);
  gated_mma<Cfg>(gate, a.f[0], b0, a.s[0], g0, GatedIssue<Cfg, false, NEXT, (T + 1) % 3, 1>{src, t + 1});
  gated_sync<Cfg::OPS_GATE>();
  gated_read_b<Cfg, U>(b0, src.wave, 0, g, l16);
  __builtin_amdgcn_sched_barrier(0);
  gated_mma<Cfg>(gate, a.f[1], b1, a.s[1], g1, GatedIssue<Cfg, true, G, 0, 0>{src, t + 1});
  gated_read_b<Cfg, U>(b1, src.wave, 1, g, l16);
  __builtin_amdgcn_sched_barrier(0);
  gated_mma<Cfg>(up, a.f[0], b0, a.s[0], u0, GatedIssue<Cfg, true, G, 0, 1>{src, t + 1});
  gated_sync<Cfg::OPS_UP>();
  GatedA<Cfg> next;
  next.template read<(T + 1) % 3>(src, t + 1, g, l16);
  gated_read_b<Cfg, NEXT>(b0, src.wave, 0, g, l16);
  __builtin_amdgcn_sched_barrier(0);
  gated_mma<Cfg>(up, a.f[1], b1, a.s[1], u1, GatedIssue<Cfg, false, U, (T + 2) % 3, 0>{src, t + 2});
  a = next;
}

template <class Cfg>
__global__ void __launch_bounds__(512) gated_ring_kernel(GatedArgs args) {
  constexpr int TM = Cfg::TM, TN = Cfg::TN;
  const Problem& p = args.p;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int g = lane >> 4, l16 = lane & 15;
  const int64_t I = p.N / 2, K = p.K;
  const int KB = (int)(K / kKBlock), S = args.S;
  // units in the order column tile, split, row tile (fastest); each XCD takes a contiguous
  // range of it, so that the row tiles that read the same part of B share its L2
  // (the quotients come from vector instructions: readfirstlane makes them scalars again, or
  // every DMA below would loop over the values that its resource might have)
  const int unit = xcd_tile_order(blockIdx.x, gridDim.x);
  const int rest = __builtin_amdgcn_readfirstlane(unit / args.tiles_m), mt = unit - rest * args.tiles_m;
  const int nt = __builtin_amdgcn_readfirstlane(rest / S), split = rest - nt * S;
  const int tile = nt * args.tiles_m + mt;
  const int64_t n0 = (int64_t)nt * 128, m0 = (int64_t)mt * Cfg::BM;
  const int M = (int)(p.M - m0 < Cfg::BM ? p.M - m0 : Cfg::BM);  // rows of this tile
  const int kb0 = split * args.KS;
  const int ks = min(args.KS, KB - kb0);  // >= 1 (host guarantees)

  GatedSrc<Cfg> src;
  src.wave = wave;
  src.kb0 = kb0;
  src.pairs = (ks + 1) >> 1;
  src.odd = ks & 1;
  {
    const int64_t rb = sfa_row_bytes(KB, Cfg::PACKED), skip = (int64_t)kb0 * kKBlock;
    src.a = p.A + m0 * K + skip;
    src.a_bytes = (uint32_t)(M * K - skip);
    src.gate = p.B + n0 * K + skip;
    src.up = p.B + (I + n0) * K + skip;
    src.b_bytes = (uint32_t)(128 * K - skip);
    if (wave < 4) {  // lane (h, row): block h of the pair (the packed form: the word both lie in)
      src.s = p.sfA + m0 * rb;
      src.s_bytes = (uint32_t)(M * rb);
      src.s_off = (uint32_t)(wave * 16 + l16) * (uint32_t)rb + (Cfg::PACKED ? 0 : 4 * (g & 1));
      src.s_shift = Cfg::PACKED ? 2 : 0;
      src.s_second = !Cfg::PACKED && (g & 1) ? 0x80000000u : 0;
    } else {  // lanes 0..3: gate, gate of the second block, up, up of the second block
      src.s = (const uint8_t*)(p.sfB + n0 / 128 * KB);
      src.s_bytes = (uint32_t)((I / 128 + 1) * KB * 4);
      src.s_off = (uint32_t)((lane >> 1) & 1) * (uint32_t)(I / 128 * KB * 4) + 4 * (lane & 1);
      src.s_shift = 0;
      src.s_second = lane & 1 ? 0x80000000u : 0;
    }
    src.s_bytes = __builtin_amdgcn_readfirstlane(src.s_bytes);
    src.s_shift = __builtin_amdgcn_readfirstlane(src.s_shift);
#pragma unroll
    for (int q = 0; q < Cfg::A_DMA; ++q) {
      const int r = (wave * Cfg::A_DMA + q) * 4 + (lane >> 4);
      src.a_off[q] = (uint32_t)r * (uint32_t)K + (uint32_t)((l16 ^ (r & 15)) << 4);
    }
#pragma unroll
    for (int q = 0; q < Cfg::B_DMA; ++q) {
      const int r = (wave * Cfg::B_DMA + q) * 4 + (lane >> 4);
      src.b_off[q] = (uint32_t)r * (uint32_t)K + (uint32_t)((l16 ^ (r & 15)) << 4);
    }
  }
  src.second = l16 & 8 ? 0x80000000u : 0;

  v4f gate[TM][TN], up[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) gate[i][j] = up[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
  gated_issue<Cfg, false, 0, 0, 0, Cfg::OPS_GATE>(src, 0);
  gated_issue<Cfg, true, 1, 0, 0, Cfg::OPS_UP>(src, 0);
  gated_issue<Cfg, false, 2, 1, 0, Cfg::OPS_GATE / 2>(src, 1);  // as a pair's last block leaves it
  gated_sync<Cfg::OPS_UP + Cfg::OPS_GATE / 2>();
  GatedA<Cfg> a;
  v8i b0[TN];
  a.template read<0>(src, 0, g, l16);
  gated_read_b<Cfg, 0>(b0, wave, 0, g, l16);
  // One exit from the loop: where several met, the compiler also joined the steps' states of the
  // DMAs, and waited for all of them in the first step of every three.
  int t = 0;
  for (; t + 3 <= src.pairs; t += 3) {
    gated_pair<Cfg, 0>(gate, up, a, b0, src, t, g, l16);
    gated_pair<Cfg, 1>(gate, up, a, b0, src, t + 1, g, l16);
    gated_pair<Cfg, 2>(gate, up, a, b0, src, t + 2, g, l16);
  }
  if (t < src.pairs) {
    gated_pair<Cfg, 0>(gate, up, a, b0, src, t, g, l16);
    if (t + 1 < src.pairs) gated_pair<Cfg, 1>(gate, up, a, b0, src, t + 1, g, l16);
  }

  // biases as stored: unpacking them here would wait for them (loaded ahead of the product, they
  // would cost registers that 64 rows do not have)
  const int c8 = (lane & 15) * 8;  // this lane's columns in the epilogue
  v4u bias[2][2] = {};
  if (args.ep.bias) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int64_t col = k * I + n0 + c8;
      const v4u* b = args.ep.bias_bf16 ? (const v4u*)((const uint16_t*)args.ep.bias + col)
                                       : (const v4u*)((const float*)args.ep.bias + col);
      bias[k][0] = b[0];
      if (!args.ep.bias_bf16) bias[k][1] = b[1];
    }
  }

  const int wm = wave / Cfg::WN, wn = wave % Cfg::WN;
  if (S > 1) {
    constexpr int per_split = 2 * Cfg::BM * 128 * 4;
    const __amdgpu_buffer_rsrc_t ws = __builtin_amdgcn_make_buffer_rsrc(
        args.ws + (int64_t)tile * S * (2 * Cfg::BM * 128), 0, 0x7FFFFFFF, 0x00020000);
    constexpr int kSc1 = 16;  // cache policy: device scope
    auto off = [&](int sp, int k, int i, int j) {
      return sp * per_split + ((((wave * 2 + k) * TM + i) * TN + j) * 64 + lane) * 16;
    };
#pragma unroll
    for (int i = 0; i < TM; ++i)
      if ((wm * TM + i) * 16 + l16 < M) {
#pragma unroll
        for (int j = 0; j < TN; ++j) {
          __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(v4u, gate[i][j]), ws, off(split, 0, i, j), 0, kSc1);
          __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(v4u, up[i][j]), ws, off(split, 1, i, j), 0, kSc1);
        }
      }
    if (!splitk_arrive(&args.counters[tile], (uint32_t)S)) return;
    v4f sum[2][TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) sum[0][i][j] = sum[1][i][j] = v4f{0.f, 0.f, 0.f, 0.f};
    // eight or four splits' partials in flight at a time, 64 or 128 registers (this split's own are
    // there already); with four, a product of one row took 0.7 us longer
    constexpr int F = TM * TN == 1 ? 8 : 4;
    for (int s0 = 0; s0 < S; s0 += F) {
      v4u part[F][2][TM][TN];
#pragma unroll
      for (int f = 0; f < F; ++f)
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
          for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              part[f][k][i][j] = v4u{0, 0, 0, 0};
              if (s0 + f < S && s0 + f != split && (wm * TM + i) * 16 + l16 < M)
                part[f][k][i][j] = __builtin_amdgcn_raw_buffer_load_b128(ws, off(s0 + f, k, i, j), 0, kSc1);
            }
#pragma unroll
      for (int f = 0; f < F; ++f)
        if (s0 + f < S) {
#pragma unroll
          for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const v4f own = k ? up[i][j] : gate[i][j];
                const v4f x = s0 + f == split ? own : __builtin_bit_cast(v4f, part[f][k][i][j]);
#pragma unroll
                for (int q = 0; q < 4; ++q) sum[k][i][j][q] += x[q];
              }
        }
    }
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) gate[i][j] = sum[0][i][j], up[i][j] = sum[1][i][j];
    if (tid == 0)
      __hip_atomic_store(&args.counters[tile], 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }

  // The fp32 tile through LDS, 32 rows of 1 KB in each of two chunks (every DMA has to have
  // landed, and every wave to have read its last fragments), back with 16 lanes to a row, 8 gate
  // and 8 up columns each; the layout and its swizzle are pipe_store_gated's.
  gated_sync<0>();
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const int row = (wm * TM + i) * 16 + l16;
    uint8_t* dst = (row < 32 ? gated_chunk<0> : gated_chunk<1>) + (row & 31) * 1024;
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      const int c = 4 * (wn * TN + j) + g, pos = ((c >> 1) + 16 * (c & 1)) ^ (row & 31);
      *(v4f*)(dst + pos * 16) = gate[i][j];
      *(v4f*)(dst + 512 + pos * 16) = up[i][j];
    }
  }
  lds_barrier();
  float bg[8], bu[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t vg = bias[0][0][j / 2], vu = bias[1][0][j / 2];
    bg[j] = __uint_as_float(args.ep.bias_bf16 ? (j & 1 ? vg & 0xFFFF0000u : vg << 16) : bias[0][j / 4][j % 4]);
    bu[j] = __uint_as_float(args.ep.bias_bf16 ? (j & 1 ? vu & 0xFFFF0000u : vu << 16) : bias[1][j / 4][j % 4]);
  }
#pragma unroll
  for (int r0 = 0; r0 < Cfg::BM; r0 += 32) {  // four rows of each wave at a time
    const int row = r0 + wave * 4 + (lane >> 4);
    if (row >= M) break;  // 16 lanes to a row; later rows lie further on
    const uint8_t* st = (row < 32 ? gated_chunk<0> : gated_chunk<1>) + (row & 31) * 1024;
    const int p0 = l16 ^ (row & 31), p1 = (16 + l16) ^ (row & 31);
    const v4f g0 = *(const v4f*)(st + p0 * 16), g1 = *(const v4f*)(st + p1 * 16);
    const v4f u0 = *(const v4f*)(st + 512 + p0 * 16), u1 = *(const v4f*)(st + 512 + p1 * 16);
    float vg[8], vu[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) vg[i] = g0[i], vg[4 + i] = g1[i], vu[i] = u0[i], vu[4 + i] = u1[i];
    epi_gated8(args.ep, bg, bu, m0 + row, I, nt, c8, vg, vu);
  }
}

}  // namespace dg
