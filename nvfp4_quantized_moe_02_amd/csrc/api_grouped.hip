// The C ABI (include/nvfp4moe.h) of the products with 8- and 16-bit weights and of the
// combine: argument validation and launches. Every entry point validates all of its
// arguments before enqueueing anything.
#include "../../include/nvfp4moe.h"
#include "grouped.h"

using namespace nvfp4;

namespace {

constexpr int32_t kMaxExpertsGrouped = 8192;
constexpr int32_t kMaxWidth = 1 << 20;           // N and K
constexpr int64_t kMaxRows = (int64_t)1 << 30;   // sorted rows
// largest K with an int32 sum of K products of two int8 values: 2^14 K < 2^31
constexpr int32_t kMaxKI8 = (1 << 17) - 16;

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline hipStream_t as_stream(void* s) { return reinterpret_cast<hipStream_t>(s); }
inline int hip_status(hipError_t e) { return e == hipSuccess ? NVFP4_OK : NVFP4_EHIP; }
inline bool dtype_ok(int32_t d) { return d >= NVFP4_F32 && d <= NVFP4_F16; }

// What the grouped calls share. srows: the rows that sorted_pairs index (x), or -1 when the
// call takes no list. kmul: K and (16-bit) N must be multiples of it.
int check_grouped(const int32_t* offsets, int32_t E, const int32_t* pairs, int32_t topk, int32_t x_rows,
                  int32_t rows, int32_t N, int32_t K, int32_t out_dtype, const void* out) {
  if (!offsets || E < 1 || rows < 0 || N < 1 || K < 1 || !dtype_ok(out_dtype)) return NVFP4_EINVAL;
  if (pairs != nullptr) {
    if (topk < 1 || x_rows < 0 || (int64_t)x_rows * topk != rows) return NVFP4_EINVAL;
  } else if (x_rows != rows) {
    return NVFP4_EINVAL;
  }
  if (!aligned(offsets, 4) || !aligned(pairs, 4) || !aligned(out, 16)) return NVFP4_EINVAL;
  if (E > kMaxExpertsGrouped || N > kMaxWidth || K > kMaxWidth || rows > kMaxRows) return NVFP4_EUNSUPPORTED;
  return NVFP4_OK;
}

// Grids are counted in 32 bits. The smallest tile is 16 rows by 16 columns (forward), and
// 128 by 256 in the gradients.
bool grid_ok(int64_t rows, int64_t E, int64_t cols) {
  const int64_t e = E < rows ? E : rows;
  return (rows / 16 + e) * ((cols + 15) / 16) < ((int64_t)1 << 31) - 8;
}

int type_of(int32_t dtype) { return dtype == NVFP4_BF16 ? 0 : 1; }

}  // namespace

extern "C" {

int nvfp4_linear_i8(const int8_t* x, const float* x_scale, int32_t T, const int8_t* w, const float* w_scale,
                    int32_t N, int32_t K, void* out, int32_t out_dtype, void* stream) {
  if (T < 0 || N < 1 || K < 1 || !dtype_ok(out_dtype) || !w || !w_scale) return NVFP4_EINVAL;
  if (T > 0 && (!x || !x_scale || !out)) return NVFP4_EINVAL;
  if (!aligned(x, 16) || !aligned(w, 16) || !aligned(out, 16) || !aligned(x_scale, 4) || !aligned(w_scale, 4))
    return NVFP4_EINVAL;
  if (K % 16 != 0 || K > kMaxKI8 || N > kMaxWidth || T > kMaxRows || !grid_ok(T, 1, N)) return NVFP4_EUNSUPPORTED;
  if (T == 0) return NVFP4_OK;
  (void)hipGetLastError();
  const GroupedArgs g{x, w, x_scale, w_scale, nullptr, nullptr, 1, T, 1, T, N, K, out, out_dtype};
  return hip_status(launch_grouped_fwd(2, g, as_stream(stream)));
}

int nvfp4_grouped_linear_i8(const int8_t* x, const float* x_scale, int32_t x_rows, const int8_t* w,
                            const float* w_scale, const int32_t* expert_offsets, int32_t E,
                            const int32_t* sorted_pairs, int32_t topk, int32_t rows, int32_t N, int32_t K, void* out,
                            int32_t out_dtype, void* stream) {
  const int st = check_grouped(expert_offsets, E, sorted_pairs, topk, x_rows, rows, N, K, out_dtype, out);
  if (st == NVFP4_EINVAL || !w || !w_scale || (rows > 0 && (!x || !x_scale || !out))) return NVFP4_EINVAL;
  if (!aligned(x, 16) || !aligned(w, 16) || !aligned(x_scale, 4) || !aligned(w_scale, 4)) return NVFP4_EINVAL;
  if (st != NVFP4_OK || K % 16 != 0 || K > kMaxKI8 || !grid_ok(rows, E, N)) return NVFP4_EUNSUPPORTED;
  if (rows == 0) return NVFP4_OK;
  (void)hipGetLastError();
  const GroupedArgs g{x, w, x_scale, w_scale, expert_offsets, sorted_pairs, sorted_pairs ? topk : 1, x_rows, E, rows,
                      N, K, out, out_dtype};
  return hip_status(launch_grouped_fwd(2, g, as_stream(stream)));
}

int nvfp4_grouped_linear(const void* x, int32_t x_rows, const void* w, int32_t dtype, const int32_t* expert_offsets,
                         int32_t E, const int32_t* sorted_pairs, int32_t topk, int32_t rows, int32_t N, int32_t K,
                         void* out, int32_t out_dtype, void* stream) {
  const int st = check_grouped(expert_offsets, E, sorted_pairs, topk, x_rows, rows, N, K, out_dtype, out);
  if (st == NVFP4_EINVAL || !dtype_ok(dtype) || !w || (rows > 0 && (!x || !out))) return NVFP4_EINVAL;
  if (!aligned(x, 16) || !aligned(w, 16)) return NVFP4_EINVAL;
  if (st != NVFP4_OK || dtype == NVFP4_F32 || N % 8 != 0 || K % 8 != 0 || !grid_ok(rows, E, N))
    return NVFP4_EUNSUPPORTED;
  if (rows == 0) return NVFP4_OK;
  (void)hipGetLastError();
  const GroupedArgs g{x, w, nullptr, nullptr, expert_offsets, sorted_pairs, sorted_pairs ? topk : 1, x_rows, E, rows,
                      N, K, out, out_dtype};
  return hip_status(launch_grouped_fwd(type_of(dtype), g, as_stream(stream)));
}

int nvfp4_grouped_linear_dx(const void* dy, const void* w, int32_t dtype, const int32_t* expert_offsets, int32_t E,
                            int32_t rows, int32_t N, int32_t K, void* dx, int32_t out_dtype, void* stream) {
  const int st = check_grouped(expert_offsets, E, nullptr, 1, rows, rows, N, K, out_dtype, dx);
  if (st == NVFP4_EINVAL || !dtype_ok(dtype) || !w || (rows > 0 && (!dy || !dx))) return NVFP4_EINVAL;
  if (!aligned(dy, 16) || !aligned(w, 16)) return NVFP4_EINVAL;
  if (st != NVFP4_OK || dtype == NVFP4_F32 || N % 8 != 0 || K % 8 != 0 || !grid_ok(rows, E, K))
    return NVFP4_EUNSUPPORTED;
  if (rows == 0) return NVFP4_OK;
  (void)hipGetLastError();
  const GroupedArgs g{dy, w, nullptr, nullptr, expert_offsets, nullptr, 1, rows, E, rows, N, K, dx, out_dtype};
  return hip_status(launch_grouped_dx(type_of(dtype), g, as_stream(stream)));
}

int nvfp4_grouped_linear_dw(const void* dy, const void* x, int32_t x_rows, int32_t dtype,
                            const int32_t* expert_offsets, int32_t E, const int32_t* sorted_pairs, int32_t topk,
                            int32_t rows, int32_t N, int32_t K, void* dw, int32_t out_dtype, void* stream) {
  const int st = check_grouped(expert_offsets, E, sorted_pairs, topk, x_rows, rows, N, K, out_dtype, dw);
  if (st == NVFP4_EINVAL || !dtype_ok(dtype) || !dw || (rows > 0 && (!dy || !x))) return NVFP4_EINVAL;
  if (!aligned(dy, 16) || !aligned(x, 16)) return NVFP4_EINVAL;
  const int64_t tiles = (int64_t)E * ((N + 63) / 64) * ((K + 63) / 64);
  if (st != NVFP4_OK || dtype == NVFP4_F32 || N % 8 != 0 || K % 8 != 0 || tiles >= ((int64_t)1 << 31) - 8)
    return NVFP4_EUNSUPPORTED;
  (void)hipGetLastError();
  const GroupedArgs g{dy, x, nullptr, nullptr, expert_offsets, sorted_pairs, sorted_pairs ? topk : 1, x_rows, E, rows,
                      N, K, dw, out_dtype};
  return hip_status(launch_grouped_dw(type_of(dtype), g, as_stream(stream)));
}

size_t nvfp4_moe_combine_workspace_size(int32_t T, int32_t topk) {
  if (T < 0 || topk < 1) return 0;
  const int64_t P = (int64_t)T * topk;
  return P <= kSmallPairs ? 0 : ((size_t)P * 4 + 255) / 256 * 256;
}

static int check_combine(const int32_t* pairs, const float* w, int32_t T, int32_t topk, int32_t H, const void* ws,
                         size_t ws_bytes) {
  const size_t need = nvfp4_moe_combine_workspace_size(T, topk);
  if (T < 0 || topk < 1 || H < 1 || (need > 0 && !ws) || (T > 0 && !pairs)) return NVFP4_EINVAL;
  if (!aligned(pairs, 4) || !aligned(w, 4) || !aligned(ws, 16)) return NVFP4_EINVAL;
  if ((int64_t)T * topk > kMaxRows || H > kMaxWidth || (int64_t)T * H >= (int64_t)1 << 38) return NVFP4_EUNSUPPORTED;
  if (ws_bytes < need) return NVFP4_EWORKSPACE;
  return NVFP4_OK;
}

int nvfp4_moe_combine(const void* y, int32_t y_dtype, const int32_t* sorted_pairs, const float* topk_weights,
                      int32_t T, int32_t topk, int32_t H, void* out, int32_t out_dtype, void* ws, size_t ws_bytes,
                      void* stream) {
  if (!dtype_ok(y_dtype) || !dtype_ok(out_dtype) || (T > 0 && (!y || !out))) return NVFP4_EINVAL;
  if (!aligned(y, 16) || !aligned(out, 16)) return NVFP4_EINVAL;
  const int st = check_combine(sorted_pairs, topk_weights, T, topk, H, ws, ws_bytes);
  if (st != NVFP4_OK || T == 0) return st;
  (void)hipGetLastError();
  const CombineArgs c{sorted_pairs, topk_weights, reinterpret_cast<int32_t*>(ws), T, topk, H};
  return hip_status(launch_combine_rows(c, y, y_dtype, out, out_dtype, as_stream(stream)));
}

int nvfp4_moe_combine_grad(const void* dout, const void* y, int32_t dtype, const int32_t* sorted_pairs,
                           const float* topk_weights, int32_t T, int32_t topk, int32_t H, void* dy, float* dweights,
                           void* ws, size_t ws_bytes, void* stream) {
  if (!dtype_ok(dtype) || (T > 0 && (!dout || !dy || (dweights && !y)))) return NVFP4_EINVAL;
  if (!aligned(dout, 16) || !aligned(y, 16) || !aligned(dy, 16) || !aligned(dweights, 4)) return NVFP4_EINVAL;
  const int st = check_combine(sorted_pairs, topk_weights, T, topk, H, ws, ws_bytes);
  if (st != NVFP4_OK || T == 0) return st;
  (void)hipGetLastError();
  const CombineArgs c{sorted_pairs, topk_weights, reinterpret_cast<int32_t*>(ws), T, topk, H};
  return hip_status(launch_combine_grad(c, dout, y, dtype, dy, dweights, as_stream(stream)));
}

}  // extern "C"
