// Combine of the rows of routed pairs, which lie in expert order, into their tokens, and its
// gradient. Both are bound by memory: every row of y is read (and in the gradient a row
// written) once, so all of a token's rows are in flight together.
//
// A pair's position in the sorted order comes from one scatter of the sorted list into the
// workspace, inv[pair] = position. Dropped pairs are not in the list, so their entries keep
// whatever the workspace held: an entry counts only if the list has that pair there, which
// needs no cleared workspace. Up to kSmallPairs pairs each block inverts the list in LDS
// instead: one launch, and the list is at most 4 KB.
#include "grouped.h"

namespace nvfp4 {

constexpr int kSmallPairs = 1024;
constexpr int kSlots = 8;  // rows of a token in flight together

__global__ __launch_bounds__(256) void invert_kernel(const int32_t* __restrict__ pairs, int P,
                                                     int32_t* __restrict__ inv) {
  const int r = blockIdx.x * 256 + threadIdx.x;
  if (r >= P) return;
  const int p = pairs[r];
  if ((unsigned)p < (unsigned)P) inv[p] = r;
}

template <int T>
__device__ __forceinline__ float to_f32(uint32_t bits16) {
  if constexpr (T == 1) return __uint_as_float(bits16 << 16);
  return (float)__builtin_bit_cast(_Float16, (uint16_t)bits16);
}

// V consecutive values at element `at` (V = 8: 16-byte loads; V = 1: any alignment)
template <int T, int V>
__device__ __forceinline__ void load_v(const void* src, size_t at, float* v) {
  if constexpr (T == 0) {
    const float* p = reinterpret_cast<const float*>(src) + at;
    if constexpr (V == 8) {
      const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
      v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
      v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
      v[0] = p[0];
    }
  } else {
    const uint16_t* p = reinterpret_cast<const uint16_t*>(src) + at;
    if constexpr (V == 8) {
      const uint4 a = *reinterpret_cast<const uint4*>(p);
      const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[2 * j] = to_f32<T>(u[j] & 0xFFFFu);
        v[2 * j + 1] = to_f32<T>(u[j] >> 16);
      }
    } else {
      v[0] = to_f32<T>(p[0]);
    }
  }
}

template <int V>
__device__ __forceinline__ void store_v(void* dst, int dtype, size_t at, const float* v) {
  if (dtype == 0) {
    float* p = reinterpret_cast<float*>(dst) + at;
    if constexpr (V == 8) {
      reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
      reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      p[0] = v[0];
    }
  } else {
    uint32_t h[V];
#pragma unroll
    for (int j = 0; j < V; ++j) h[j] = dtype == 1 ? f32_to_bf16_bits(v[j]) : f32_to_f16_bits(v[j]);
    uint16_t* p = reinterpret_cast<uint16_t*>(dst) + at;
    if constexpr (V == 8)
      *reinterpret_cast<uint4*>(p) =
          make_uint4(h[0] | (h[1] << 16), h[2] | (h[3] << 16), h[4] | (h[5] << 16), h[6] | (h[7] << 16));
    else
      p[0] = (uint16_t)h[0];
  }
}

// Fills the block's LDS copy of the inverse (small lists). Callers pass the result of
// pos_of as a row index only when it is >= 0.
__device__ __forceinline__ void invert_lds(const CombineArgs& c, int P, int32_t* s_inv) {
  for (int p = threadIdx.x; p < P; p += blockDim.x) s_inv[p] = -1;
  __syncthreads();
  for (int r = threadIdx.x; r < P; r += blockDim.x) {
    const int p = c.pairs[r];
    if ((unsigned)p < (unsigned)P) s_inv[p] = r;
  }
  __syncthreads();
}
template <bool SMALL>
__device__ __forceinline__ int pos_of(const CombineArgs& c, int P, const int32_t* s_inv, int p) {
  if constexpr (SMALL) return s_inv[p];
  const int r = c.inv[p];
  return (unsigned)r < (unsigned)P && c.pairs[r] == p ? r : -1;
}

// One thread per (token, V columns): the token's rows, kSlots at a time, added in slot order.
template <int T, int V, bool SMALL>
__global__ __launch_bounds__(256) void combine_rows_kernel(CombineArgs c, const void* __restrict__ y,
                                                           void* __restrict__ out, int out_dtype) {
  __shared__ int32_t s_inv[SMALL ? kSmallPairs : 1];
  const int P = c.T * c.topk;
  if constexpr (SMALL) invert_lds(c, P, s_inv);
  const int per = c.H / V;
  const int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (u >= (int64_t)c.T * per) return;
  const int t = (int)(u / per);
  const size_t col = (size_t)(u - (int64_t)t * per) * V;
  float acc[V];
#pragma unroll
  for (int j = 0; j < V; ++j) acc[j] = 0.f;
  for (int j0 = 0; j0 < c.topk; j0 += kSlots) {
    int pos[kSlots];
    float v[kSlots][V];
#pragma unroll
    for (int s = 0; s < kSlots; ++s)
      pos[s] = j0 + s < c.topk ? pos_of<SMALL>(c, P, s_inv, t * c.topk + j0 + s) : -1;
#pragma unroll
    for (int s = 0; s < kSlots; ++s)
      if (pos[s] >= 0) load_v<T, V>(y, (size_t)pos[s] * c.H + col, v[s]);
#pragma unroll
    for (int s = 0; s < kSlots; ++s)
      if (pos[s] >= 0) {
        const float w = c.w != nullptr ? c.w[t * c.topk + j0 + s] : 1.f;
#pragma unroll
        for (int j = 0; j < V; ++j) acc[j] = fmaf(w, v[s][j], acc[j]);
      }
  }
  store_v<V>(out, out_dtype, (size_t)t * c.H + col, acc);
}

// G waves per token: each lane takes V columns at a time of dout once per kSlots slots,
// writes the scaled row of every slot and sums the slot's dot product; the partial sums
// are added over the lanes and then over the G waves, in a fixed order.
template <int T, int V, int G, bool SMALL, bool DW>
__global__ __launch_bounds__(256) void combine_grad_kernel(CombineArgs c, const void* __restrict__ dout,
                                                           const void* __restrict__ y, void* __restrict__ dy,
                                                           float* __restrict__ dw) {
  __shared__ int32_t s_inv[SMALL ? kSmallPairs : 1];
  __shared__ float s_dot[4][kSlots];
  const int P = c.T * c.topk;
  if constexpr (SMALL) invert_lds(c, P, s_inv);
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int t = blockIdx.x * (4 / G) + wave / G, sub = wave % G;
  const bool live = t < c.T;
  for (int j0 = 0; j0 < c.topk; j0 += kSlots) {
    int pos[kSlots];
    float w[kSlots], dot[kSlots];
#pragma unroll
    for (int s = 0; s < kSlots; ++s) {
      const bool in = live && j0 + s < c.topk;
      pos[s] = in ? pos_of<SMALL>(c, P, s_inv, t * c.topk + j0 + s) : -1;
      w[s] = in && c.w != nullptr ? c.w[t * c.topk + j0 + s] : 1.f;
      dot[s] = 0.f;
    }
    if (live)
      for (int col = (sub * 64 + lane) * V; col < c.H; col += G * 64 * V) {
        float d[V], v[kSlots][V], o[V];
        load_v<T, V>(dout, (size_t)t * c.H + col, d);
        if constexpr (DW) {
#pragma unroll
          for (int s = 0; s < kSlots; ++s)
            if (pos[s] >= 0) load_v<T, V>(y, (size_t)pos[s] * c.H + col, v[s]);
        }
#pragma unroll
        for (int s = 0; s < kSlots; ++s)
          if (pos[s] >= 0) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
              o[j] = w[s] * d[j];
              if constexpr (DW) dot[s] = fmaf(d[j], v[s][j], dot[s]);
            }
            store_v<V>(dy, T, (size_t)pos[s] * c.H + col, o);
          }
      }
    if constexpr (DW) {
#pragma unroll
      for (int s = 0; s < kSlots; ++s) {
        float v = sum16(dot[s]);
        v += __shfl_xor(v, 16);
        v += __shfl_xor(v, 32);
        if (lane == 0) s_dot[wave][s] = v;
      }
      __syncthreads();
      if (live && sub == 0 && lane < kSlots && j0 + lane < c.topk) {
        float v = s_dot[wave][lane];
#pragma unroll
        for (int q = 1; q < G; ++q) v += s_dot[wave + q][lane];
        dw[(size_t)t * c.topk + j0 + lane] = v;
      }
      __syncthreads();
    }
  }
}

static hipError_t invert(const CombineArgs& c, hipStream_t st) {
  const int P = c.T * c.topk;
  if (P > kSmallPairs) invert_kernel<<<(P + 255) / 256, 256, 0, st>>>(c.pairs, P, c.inv);
  return hipGetLastError();
}

template <int T, int V>
static void combine_rows(const CombineArgs& c, const void* y, void* out, int out_dtype, hipStream_t st) {
  const int64_t units = (int64_t)c.T * (c.H / V);
  const unsigned grid = (unsigned)((units + 255) / 256);
  if (c.T * c.topk <= kSmallPairs)
    combine_rows_kernel<T, V, true><<<grid, 256, 0, st>>>(c, y, out, out_dtype);
  else
    combine_rows_kernel<T, V, false><<<grid, 256, 0, st>>>(c, y, out, out_dtype);
}

hipError_t launch_combine_rows(const CombineArgs& c, const void* y, int y_dtype, void* out, int out_dtype,
                               hipStream_t st) {
  if (c.T == 0) return hipSuccess;
  const hipError_t e = invert(c, st);
  if (e != hipSuccess) return e;
  const bool vec = c.H % 8 == 0;
#define NVFP4_COMBINE(T)                           \
  if (vec)                                         \
    combine_rows<T, 8>(c, y, out, out_dtype, st);  \
  else                                             \
    combine_rows<T, 1>(c, y, out, out_dtype, st)
  if (y_dtype == 0) {
    NVFP4_COMBINE(0);
  } else if (y_dtype == 1) {
    NVFP4_COMBINE(1);
  } else {
    NVFP4_COMBINE(2);
  }
#undef NVFP4_COMBINE
  return hipGetLastError();
}

template <int T, int V, int G, bool DW>
static void combine_grad_g(const CombineArgs& c, const void* dout, const void* y, void* dy, float* dw,
                           hipStream_t st) {
  const unsigned grid = (unsigned)((c.T + 4 / G - 1) / (4 / G));
  if (c.T * c.topk <= kSmallPairs)
    combine_grad_kernel<T, V, G, true, DW><<<grid, 256, 0, st>>>(c, dout, y, dy, dw);
  else
    combine_grad_kernel<T, V, G, false, DW><<<grid, 256, 0, st>>>(c, dout, y, dy, dw);
}

// Waves per token: one per 512 columns (64 lanes x 8), at most 4.
template <int T, int V>
static void combine_grad_t(const CombineArgs& c, const void* dout, const void* y, void* dy, float* dw,
                           hipStream_t st) {
  const int G = c.H <= 64 * V ? 1 : c.H <= 128 * V ? 2 : 4;
#define NVFP4_GRAD(D)                                     \
  if (G == 1)                                             \
    combine_grad_g<T, V, 1, D>(c, dout, y, dy, dw, st);   \
  else if (G == 2)                                        \
    combine_grad_g<T, V, 2, D>(c, dout, y, dy, dw, st);   \
  else                                                    \
    combine_grad_g<T, V, 4, D>(c, dout, y, dy, dw, st)
  if (dw != nullptr) {
    NVFP4_GRAD(true);
  } else {
    NVFP4_GRAD(false);
  }
#undef NVFP4_GRAD
}

hipError_t launch_combine_grad(const CombineArgs& c, const void* dout, const void* y, int dtype, void* dy, float* dw,
                               hipStream_t st) {
  if (c.T == 0) return hipSuccess;
  const hipError_t e = invert(c, st);
  if (e != hipSuccess) return e;
  const bool vec = c.H % 8 == 0;
  if (dtype == 0)
    vec ? combine_grad_t<0, 8>(c, dout, y, dy, dw, st) : combine_grad_t<0, 1>(c, dout, y, dy, dw, st);
  else if (dtype == 1)
    vec ? combine_grad_t<1, 8>(c, dout, y, dy, dw, st) : combine_grad_t<1, 1>(c, dout, y, dy, dw, st);
  else
    vec ? combine_grad_t<2, 8>(c, dout, y, dy, dw, st) : combine_grad_t<2, 1>(c, dout, y, dy, dw, st);
  return hipGetLastError();
}

}  // namespace nvfp4
