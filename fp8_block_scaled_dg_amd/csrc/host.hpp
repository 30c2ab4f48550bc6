// host.hpp -- host code that the library's translation units share: error reporting, the
// per-(device, stream) workspace, argument checks, and the launch shapes of the row kernels.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <exception>
#include <mutex>
#include <tuple>
#include <type_traits>
#include <utility>

#include "../../include/dg.h"
#include "gemm_kernel.hpp"

namespace dg {

constexpr int64_t kCUs = 256;  // MI355X compute units (8 XCDs x 32)

// Defined in dg_api.hip.
extern thread_local char g_detail[512];
dg_status fail(dg_status s, const char* fmt, ...);
dg_status get_workspace(hipStream_t stream, size_t partial_bytes, size_t counters,
                        float** partials, uint32_t** counter_ptr);
dg_status check_common(const void* A, const void* B, const void* C, const void* sfA,
                       const float* sfB, int64_t N, int64_t K, bool any_output);
dg_status check_rows(int64_t M, int64_t K, const char* k);
void print_dense_choice(int64_t M, int64_t N, int64_t K, const char* config, const char* note);
dg_status check_norm(int32_t x_dtype, int32_t w_dtype, int64_t M, int64_t K);
dg_status get_partials(hipStream_t st, int64_t count, float** part);
dg_status launch_column_sum(const float* part, float* out, int64_t R, int64_t N, hipStream_t st);
dg_status launch_column_sum2(const float* part, float* out, float* out2, int64_t R, int64_t N,
                             hipStream_t st);

// The text of a failed runtime call's error. HIP keeps the error for whoever asks the thread for its
// last one; it is reported here, so it is taken off, and no later call of anyone is blamed for it.
inline const char* take_error(hipError_t e) {
  (void)hipGetLastError();
  return hipGetErrorString(e);
}

inline bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

inline bool known_dtype(int32_t t) { return t == DG_DTYPE_F32 || t == DG_DTYPE_BF16; }
inline bool known_act(int32_t a) { return a >= DG_ACT_NONE && a <= DG_ACT_GELU_TANH; }

// Held from where a call takes its stream's buffers to its last launch that uses them, so that
// calls of several threads on one stream do not launch in between (a backward call's partial sums
// and their sum are two launches, and the partials of any K split lie in the same buffer). A mutex
// for every 64th of the streams; recursive, since a call on transposed copies makes another.
class StreamTurn {
 public:
  explicit StreamTurn(hipStream_t stream, bool needed = true) : mu_(needed ? &slot(stream) : nullptr) {
    if (mu_) mu_->lock();
  }
  ~StreamTurn() {
    if (mu_) mu_->unlock();
  }
  StreamTurn(const StreamTurn&) = delete;
  StreamTurn& operator=(const StreamTurn&) = delete;

 private:
  static std::recursive_mutex& slot(hipStream_t stream) {
    static std::recursive_mutex slots[64];
    return slots[((uintptr_t)stream >> 6) & 63];
  }
  std::recursive_mutex* mu_;
};

// f(), a C++ exception of the host code (std::bad_alloc of the workspace tables) turned into
// a status: none leaves a C entry.
template <class F>
dg_status no_throw(F f) noexcept {
  try {
    return f();
  } catch (const std::exception& e) {
    return fail(DG_ERR_LAUNCH, "host code: %s", e.what());
  } catch (...) {
    return fail(DG_ERR_LAUNCH, "host code: an unknown exception");
  }
}

// Launches kernel(args...) and reports what this launch returned. hipGetLastError would also report
// an error that some earlier call left in the thread, of a launch that then runs all the same.
template <class... P, class... A>
dg_status launch_kernel(const char* what, void (*kernel)(P...), dim3 grid, dim3 block, size_t lds,
                        hipStream_t stream, A&&... args) {
  std::tuple<P...> values(std::forward<A>(args)...);
  const hipError_t e = std::apply(
      [&](P&... v) {
        void* ptrs[] = {(void*)&v...};
        return hipLaunchKernel((const void*)kernel, grid, block, ptrs, lds, stream);
      },
      values);
  return e == hipSuccess ? DG_OK : fail(DG_ERR_LAUNCH, "%s: %s", what, take_error(e));
}

// The pipelined kernel addresses a tile's rows with 32-bit offsets below 256 * K
// bytes; this bound keeps them under 2^31.
constexpr int kPipeMaxKB = (1 << 22) / kKBlock;

constexpr int kLongKB = 32;                  // K-blocks from which the 128x256 tiles use it

// Dense tail balancing: with T tiles on kCUs CUs (one workgroup each), the last
// r = T mod kCUs tiles would run in a partial round. Each of them is split into
// `parts` K ranges (at least 8 K-blocks each) so that the last round fills the GPU.
struct TailSplit {
  int64_t full, parts;
};

inline TailSplit pipe_tail_split(int64_t tiles, int64_t KB) {
  TailSplit t{tiles, 1};
  const int64_t r = tiles % kCUs;
  if (r == 0) return t;
  int64_t parts = kCUs / r;
  if (parts > 8) parts = 8;
  if (parts > KB / 8) parts = KB / 8;
  if (parts < 2) return t;
  t.full = tiles - r;
  t.parts = parts;
  return t;
}

// A row's threads, at most 512, hold 16 values each in one to four chunks. (4096 x 18432,
// three chunks against two of up to 1024 threads: backward bf16 144 and 160 us, fp32 186 and
// 262; forward bf16 100 and 90, fp32 92 and 102.)
inline int norm_chunks(int64_t K) { return (int)((K + 8191) / 8192); }
inline int norm_threads(int64_t K) {
  const int64_t t = (K / 16 + norm_chunks(K) - 1) / norm_chunks(K);
  return (int)((t + 63) / 64 * 64);
}

// Up to this many rows the backward kernels sum columns in the same launch, reading their
// inputs a second time; for the activation's, whose values are also computed twice, up to
// this many values. Us, one launch against two, back to back calls (3 us of host time for each
// launch) and in a graph:
//   norm bf16   64 x  7168   7.7, 10.3    4.5,  7.3     gelu  64 x 18432   7.0, 9.7   5.7, 7.8
//              256 x  7168   7.6, 11.4    6.9, 11.7          130 x 18432  11.3, 9.7  11.7, 9.6
//              512 x  7168  11.7, 13.4   12.0, 13.7          256 x  2048   7.1, 9.9   7.4, 6.5
//              256 x   768   7.8, 10.8    8.0,  6.2          256 x   512   7.2, 9.9   7.4, 6.3
//       fp32  256 x  2048   7.2,  9.9    7.0,  7.0          512 x   512  12.1, 9.8  12.5, 6.3
//             512 x  2048  10.0,  9.8   10.5,  7.9
// The bounds follow the calls. They give away 1 to 2 us in a graph at 256 rows of few columns,
// and as much of either at 512 rows of many.
constexpr int64_t kDirectRows = 256, kDirectActValues = 3 << 19;

// Workgroups for `rows` steps of work, at most `most`, evened out so that every workgroup
// takes the same number of steps or one fewer (bf16 4096 x 7168 on 512 workgroups, 8 rows
// each: 34.5 us; on 768, 5 or 6 each: 39.1).
inline int64_t even_grid(int64_t rows, int64_t most) {
  const int64_t each = (rows + most - 1) / most;
  return (rows + each - 1) / each;
}

// Work of the kernels that take strips of 1024 columns over groups of rows, a row per wave and
// step. Row groups: about 8 workgroups per CU (gelu with its column sums, 4096 x 18432: 78.8 us,
// with 16 80.1), of at least 8 rows, two per wave, or 4 where 8 would leave CUs idle (at least
// 4 / 8 / 16: 4096 x 2048 19.9 / 16.9 / 16.2 us, 1000 x 512 6.7 / 7.8 / 10.1).
struct StripPlan {
  int64_t strips, rows, groups;
};

inline StripPlan strip_plan(int64_t M, int64_t N) {
  const int64_t strips = (N + 1023) / 1024, least = (M + 7) / 8 * strips < kCUs ? 4 : 8;
  int64_t groups = (8 * kCUs + strips - 1) / strips;
  if (groups > (M + least - 1) / least) groups = (M + least - 1) / least;
  const int64_t rows = ((M + groups - 1) / groups + 3) / 4 * 4;
  return StripPlan{strips, rows, (M + rows - 1) / rows};
}

// Calls f with the compile-time form of a norm kernel for these types and K:
// f(bf16 x?, bf16 weights?, chunks).
template <class F>
void norm_form(bool x_bf16, bool w_bf16, int64_t K, F f) {
  auto by_k = [&](auto xb, auto wb) {
    using std::integral_constant;
    switch (norm_chunks(K)) {
      case 1: f(xb, wb, integral_constant<int, 1>{}); break;
      case 2: f(xb, wb, integral_constant<int, 2>{}); break;
      case 3: f(xb, wb, integral_constant<int, 3>{}); break;
      default: f(xb, wb, integral_constant<int, 4>{}); break;
    }
  };
  auto by_w = [&](auto xb) {
    if (w_bf16) by_k(xb, std::true_type{});
    else by_k(xb, std::false_type{});
  };
  if (x_bf16) by_w(std::true_type{});
  else by_w(std::false_type{});
}

}  // namespace dg
