// ring_kernel.hpp -- block-scaled FP8 GEMM with a fused epilogue for few rows or few tiles,
// gfx950: tiles of up to 64 x 64 or 128, or of 128 x 128: an eighth, a quarter or half of the
// tile kernel's, so that products of a few hundred rows still give every CU a tile without
// splitting K, or with partial tiles of 4 to 64 KB instead of 128.
//
// Memory-bound: with up to 64 rows every byte of B meets few rows of A, so the kernel has to
// keep enough bytes of B in flight on every CU, and to ask for them in the right pieces. A
// workgroup (4 or 8 waves) takes a tile and a run of consecutive K-blocks. It moves A and B by LDS DMA,
// two K-blocks at a time: 256 contiguous bytes of every row. (Reading B [18432][7168] alone,
// 128 bytes of each of 128 rows per step, took 41 us; 256 bytes, 26 us, and the rate that one
// CU reaches grew with it: 32 workgroups on [4096][7168], 24.7 against 14.0 us.) D stages of
// a pair of blocks keep 2 (D - 1) blocks in flight whatever the registers hold: 96 KB per CU
// at D = 3, BN = 128.
// What bounds it: one CU takes in about 42 KB/us (64 x 18432 x 7168, FP8 output: 144 tiles on as
// many CUs, 28 KB/us of B and 14 of A each, 37.7 us), HBM gives 20 KB/us of B to each of 256
// (64 x 32768 x 7168: 43.9 us). Splitting K pays while it brings idle CUs in (64 x 16384 x 7168
// in two halves: 28.5 us).
// Per pair: wait for this wave's DMAs of it (vmcnt), one barrier (every wave's DMAs of the
// pair have landed and every wave is done with the previous pair), refill the previous
// pair's stage, then per block and 16x16 tile one v_mfma_f32_16x16x128_f8f6f4 and the
// promotion into fp32 accumulators with sfA[m][kb] * sfB[n/128][kb]: the two-level
// accumulation of the DeepGEMM launch article (deepseek.csdn.net), section 1.2 "precision
// safeguards".
//
// LDS rows are 256 bytes; 16-byte chunk c of row r sits at c ^ (r & 15), so that 16 lanes
// reading one chunk of 16 rows hit disjoint banks. Each stage is its own __shared__ array, so
// that the compiler can tell a DMA into one from a read of another; the loop is unrolled by
// D. Runs are aligned at their end: the first group of D steps skips the pairs before the
// run, so that the last group, whose waits count down as nothing more is issued, is always
// the same code. The steps between hold no branch: with branches inside, the compiler lost
// track of which stage a read comes from and drained every DMA before it. A run of odd
// length reads 128 bytes per row past its end (the next row's, or zeros past the last) and
// does not compute them.
//
// sfA: each wave brings 16 rows' values of both blocks by one 4-byte DMA per lane (waves past
// the tile's rows repeat others'). Rows past M and N read as zero (the buffer resources end
// there) and are never stored.
//
// S > 1 K splits: fp32 partials and an arrival count per column tile, the last split to
// arrive adds all of them in split order (see splitk_arrive), so results are deterministic.
#pragma once

#include "epilogue.hpp"
#include "gemm_kernel.hpp"
#include "pipe_kernel.hpp"

namespace dg {

// W waves as WM x W/WM; a wave owns TM x TN 16x16 tiles.
template <int W_, int WM_, int TM_, int TN_, int D_, bool PACKED_, bool STREAM_B_>
struct RingCfg {
  static constexpr int W = W_, WM = WM_, WN = W / WM, TM = TM_, TN = TN_, D = D_, NT = W * 64;
  static constexpr bool PACKED = PACKED_;      // sfA in the packed UE8M0 form
  static constexpr bool STREAM_B = STREAM_B_;  // B's lines leave room in the caches for A's
  static constexpr int BM = 16 * WM * TM, BN = 16 * WN * TN;
  static constexpr int ROW = 2 * kKBlock;                // bytes of a row per step
  static constexpr int A_ROWS = BM < 4 * W ? 4 * W : BM;  // staged: whole DMAs for every wave
  static constexpr int A_DMA = A_ROWS / 4 / W, B_DMA = BN / 4 / W;  // 1 KB DMAs per wave and step
  static constexpr int OPS = 1 + A_DMA + B_DMA;
  static constexpr int OFF_B = A_ROWS * ROW, OFF_S = OFF_B + BN * ROW;
  static constexpr int SROWS = BM <= 64 ? 4 : 8;  // 16-row groups whose scales are staged
  static constexpr int STAGE = OFF_S + SROWS * 256;
  static constexpr int SMAX = TM * TN <= 4 ? 8 : 2;  // splits whose partials fit the registers
  static constexpr int ROWS = BM < 64 ? BM : 64;  // rows per pass of the epilogue
  static_assert(SROWS <= W && BM <= 16 * SROWS, "scale rows");
  static_assert(BM <= 128 && B_DMA >= 1 && W % 4 == 0, "DMA split");
  static_assert(ROWS * kEpiPitch<BN> * 4 <= OFF_S, "a pass of the fp32 tile fits a stage");
  static_assert((D - 1) * OPS < 64, "vmcnt range");
};

struct RingArgs {
  Problem p;
  float* ws;           // [tiles][S][BM * BN] fp32 partials (S > 1)
  uint32_t* counters;  // [tiles], zero between calls
  int32_t S, KS;       // K splits, K-blocks per split (even; the last may have fewer)
  int32_t tiles_m;     // row tiles
  Epilogue ep;
};

template <int BYTES, int I>
__shared__ __align__(16) uint8_t ring_stage[BYTES];

// Values that the kernel only reads, as scalar loads.
typedef const float __attribute__((address_space(4)))* ring_const;

template <class Cfg>
struct RingSrc {
  __amdgpu_buffer_rsrc_t a, b, s;
  uint32_t a_off[Cfg::A_DMA], b_off[Cfg::B_DMA], s_off;
  int wave, kb0;   // kb0 is even
  ring_const sfb;         // this column block's sfB, at kb0
};

// The DMAs of pair t of the run (blocks 2t, 2t + 1) into stage T.
template <class Cfg, int T>
__device__ __forceinline__ void ring_issue(const RingSrc<Cfg>& src, int t) {
#if defined(__HIP_DEVICE_COMPILE__)
  typedef __attribute__((address_space(3))) void* lds_ptr;
  constexpr int kPolicyB = Cfg::STREAM_B ? 2 : 0;  // 2: non-temporal
  uint8_t* st = ring_stage<Cfg::STAGE, T>;
  const int kb = src.kb0 + 2 * t;  // even: in the packed form both blocks lie in one word
  __builtin_amdgcn_raw_ptr_buffer_load_lds(src.s, (lds_ptr)(st + Cfg::OFF_S + (src.wave & (Cfg::SROWS - 1)) * 256), 4, src.s_off,
                                           Cfg::PACKED ? kb & ~3 : kb * 4, 0, 0);
#pragma unroll
  for (int q = 0; q < Cfg::A_DMA; ++q)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(src.a, (lds_ptr)(st + (src.wave * Cfg::A_DMA + q) * 1024),
                                             16, src.a_off[q], t * Cfg::ROW, 0, 0);
#pragma unroll
  for (int q = 0; q < Cfg::B_DMA; ++q)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        src.b, (lds_ptr)(st + Cfg::OFF_B + (src.wave * Cfg::B_DMA + q) * 1024), 16, src.b_off[q],
        t * Cfg::ROW, 0, kPolicyB);
#endif
}

template <class Cfg, int T>
__device__ __forceinline__ void ring_prologue(const RingSrc<Cfg>& src, int t) {
  if constexpr (T < Cfg::D - 1) {
    if (t + T >= 0) ring_issue<Cfg, T>(src, t + T);
    ring_prologue<Cfg, T + 1>(src, t);
  }
}

// 128 bytes (block h of the pair) of row `row`: lane group g holds k in [16g, 16g + 16) and
// [64 + 16g, 80 + 16g), for both operands.
__device__ __forceinline__ v8i ring_frag(const uint8_t* tile, int row, int h, int g) {
  const uint8_t* p = tile + row * 2 * kKBlock;
  const v4u lo = *(const v4u*)(p + (((8 * h + g) ^ (row & 15)) << 4));
  const v4u hi = *(const v4u*)(p + (((8 * h + g + 4) ^ (row & 15)) << 4));
  return v8i{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3],
             (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
}

// Block h of pair t, held in stage T.
template <class Cfg, int T>
__device__ __forceinline__ void ring_block(v4f (&acc)[Cfg::TM][Cfg::TN], const RingSrc<Cfg>& src,
                                           int t, int h, float sb, int g, int l16) {
  constexpr int TM = Cfg::TM, TN = Cfg::TN;
  const int wm = src.wave / Cfg::WN, wn = src.wave % Cfg::WN;
  const uint8_t* st = ring_stage<Cfg::STAGE, T>;
  const int shift = Cfg::PACKED ? ((src.kb0 + 2 * t + h) & 3) * 8 : 0;
  v8i bf[TN], af[TM];
  float s[TM];
#pragma unroll
  for (int j = 0; j < TN; ++j) bf[j] = ring_frag(st + Cfg::OFF_B, (wn * TN + j) * 16 + l16, h, g);
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const int tile = wm * TM + i;
    af[i] = ring_frag(st, tile * 16 + l16, h, g);
    const uint32_t w = *(const uint32_t*)(st + Cfg::OFF_S + tile * 256 + (16 * h + l16) * 4);
    s[i] = sb * (Cfg::PACKED ? ue8m0_value((w >> shift) & 0xFFu) : __uint_as_float(w));
  }
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      const v4f part = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
          bf[j], af[i], v4f{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
#pragma unroll
      for (int q = 0; q < 4; ++q) acc[i][j][q] = __builtin_fmaf(part[q], s[i], acc[i][j][q]);
    }
  // The promotion stays in the MFMAs' basic block: moved past a branch, it ended up 5 wait
  // states behind its MFMA on one of the two paths, 12 being needed (the compiler counted
  // the other path's undefined registers as instructions), and read the register's old value.
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) asm volatile("" : "+v"(acc[i][j]));
}

// Steps T .. D-1 of a group that starts at pair t (pair t + T in stage T). FIRST: pairs
// before the run (negative) pass without work. LAST: the group that ends the run.
template <class Cfg, int T, bool FIRST, bool LAST>
__device__ __forceinline__ void ring_steps(v4f (&acc)[Cfg::TM][Cfg::TN], const RingSrc<Cfg>& src,
                                           int t, int ks, int g, int l16) {
  if constexpr (T < Cfg::D) {
    constexpr int D = Cfg::D;
    constexpr int left = (LAST && T > 0 ? D - 1 - T : D - 2) * Cfg::OPS;  // later DMAs in flight
    const int tc = t + T;
    if (!FIRST || tc >= 0) {
      constexpr bool END = LAST && T == D - 1;
      const bool two = !END || 2 * tc + 1 < ks;
      const float sb0 = src.sfb[2 * tc], sb1 = src.sfb[two ? 2 * tc + 1 : 2 * tc];
      __builtin_amdgcn_s_waitcnt((left & 15) | ((left >> 4) << 14) | (7 << 4));  // lgkmcnt 0
      __builtin_amdgcn_s_barrier();
      __builtin_amdgcn_sched_barrier(0);
      if (!LAST || T == 0) ring_issue<Cfg, (T + D - 1) % D>(src, tc + D - 1);
      __builtin_amdgcn_sched_barrier(0);
      ring_block<Cfg, T>(acc, src, tc, 0, sb0, g, l16);
      if (two) ring_block<Cfg, T>(acc, src, tc, 1, sb1, g, l16);
    } else if (!LAST || T == 0) {
      ring_issue<Cfg, (T + D - 1) % D>(src, tc + D - 1);
    }
    ring_steps<Cfg, T + 1, FIRST, LAST>(acc, src, t, ks, g, l16);
  }
}

template <class Cfg, int EPI>
__global__ void __launch_bounds__(Cfg::NT) ring_kernel(RingArgs args) {
  constexpr int TM = Cfg::TM, TN = Cfg::TN, BN = Cfg::BN, D = Cfg::D;
  const Problem& p = args.p;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int g = lane >> 4, l16 = lane & 15;
  const int64_t N = p.N, K = p.K;
  const int KB = (int)(K / kKBlock), S = args.S;
  // units in the order column tile, split, row tile (fastest); each XCD takes a contiguous
  // range of it, so that the row tiles that read the same part of B share its L2
  const int unit = xcd_tile_order(blockIdx.x, gridDim.x);
  const int mt = unit % args.tiles_m, rest = unit / args.tiles_m;
  const int split = rest % S, nt = rest / S, tile = nt * args.tiles_m + mt;
  const int64_t n0 = (int64_t)nt * BN, m0 = (int64_t)mt * Cfg::BM;
  const int M = (int)(p.M - m0 < Cfg::BM ? p.M - m0 : Cfg::BM);  // rows of this tile
  const int kb0 = split * args.KS;
  const int ks = min(args.KS, KB - kb0);  // >= 1 (host guarantees)

  RingSrc<Cfg> src;
  src.wave = wave;
  src.kb0 = kb0;
  {
    const int64_t rb = sfa_row_bytes(KB, Cfg::PACKED);
    const int64_t b_rows = N - n0 < BN ? N - n0 : BN, skip = (int64_t)kb0 * kKBlock;
    src.a = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p.A + m0 * K + skip), 0,
                                              (int)(M * K - skip), 0x00020000);
    src.b = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p.B + n0 * K + skip), 0,
                                              (int)(b_rows * K - skip), 0x00020000);
    src.s = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p.sfA + m0 * rb), 0, (int)(M * rb),
                                              0x00020000);
    // lane (h, row): block h of the pair (the packed form: the word both lie in)
    src.s_off = (uint32_t)((wave & (Cfg::SROWS - 1)) * 16 + l16) * (uint32_t)rb + (Cfg::PACKED ? 0 : 4 * (g & 1));
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
  src.sfb = (ring_const)(uintptr_t)(p.sfB + (n0 / kKBlock) * KB + kb0);

  constexpr int ROWS = Cfg::ROWS;
  EpiTile<BN, Cfg::NT, EPI, ROWS> epi;
  epi.load(p, n0, args.ep, (int)m0);

  v4f acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
  const int pairs = (ks + 1) >> 1;
  int t = -((D - pairs % D) % D);  // the run ends at the end of a group
  ring_prologue<Cfg, 0>(src, t);
  if (t + D >= pairs) {
    ring_steps<Cfg, 0, true, true>(acc, src, t, ks, g, l16);
  } else {
    ring_steps<Cfg, 0, true, false>(acc, src, t, ks, g, l16);
    for (t += D; t + D < pairs; t += D) ring_steps<Cfg, 0, false, false>(acc, src, t, ks, g, l16);
    ring_steps<Cfg, 0, false, true>(acc, src, t, ks, g, l16);
  }

  if (S > 1) {
    constexpr int per_split = Cfg::BM * BN * 4;
    const __amdgpu_buffer_rsrc_t ws = __builtin_amdgcn_make_buffer_rsrc(
        args.ws + (int64_t)tile * S * (Cfg::BM * BN), 0, 0x7FFFFFFF, 0x00020000);
    constexpr int kSc1 = 16;  // cache policy: device scope
    auto off = [&](int sp, int i, int j) {
      return sp * per_split + (((wave * TM + i) * TN + j) * 64 + lane) * 16;
    };
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j)
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(v4u, acc[i][j]), ws, off(split, i, j), 0, kSc1);
    if (!splitk_arrive(&args.counters[tile], (uint32_t)S)) return;
    // all of the other splits' partials in flight at once (this split's is in registers)
    v4u part[Cfg::SMAX][TM][TN];
#pragma unroll
    for (int sp = 0; sp < Cfg::SMAX; ++sp)
      if (sp < S && sp != split) {
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
          for (int j = 0; j < TN; ++j)
            part[sp][i][j] = __builtin_amdgcn_raw_buffer_load_b128(ws, off(sp, i, j), 0, kSc1);
      }
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        v4f sum = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int sp = 0; sp < Cfg::SMAX; ++sp)
          if (sp < S) {
            const v4f x = sp == split ? acc[i][j] : __builtin_bit_cast(v4f, part[sp][i][j]);
#pragma unroll
            for (int q = 0; q < 4; ++q) sum[q] += x[q];
          }
        acc[i][j] = sum;
      }
    if (tid == 0)
      __hip_atomic_store(&args.counters[tile], 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }

  // the fp32 tile through LDS, ROWS rows at a time. Every DMA has landed: the last step
  // waited for all of them.
  const int wm = wave / Cfg::WN, wn = wave % Cfg::WN;
  float* out = (float*)ring_stage<Cfg::STAGE, 0>;
#pragma unroll
  for (int h = 0; h < Cfg::BM / ROWS; ++h) {
    if (ROWS * h >= M) break;
    lds_barrier();
    if (h > 0) epi.load(p, n0, args.ep, (int)m0 + ROWS * h);
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      const int row = (wm * TM + i) * 16 - ROWS * h;  // of the pass
      if (row < 0 || row >= ROWS) continue;
#pragma unroll
      for (int j = 0; j < TN; ++j)
        *(v4f*)(out + (row + l16) * kEpiPitch<BN> + (wn * TN + j) * 16 + 4 * g) = acc[i][j];
    }
    lds_barrier();
    epi.finish(p, n0, out, args.ep, (int)m0 + ROWS * h);
  }
}

}  // namespace dg
