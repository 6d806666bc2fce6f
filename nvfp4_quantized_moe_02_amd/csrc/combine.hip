// Combine of the rows of routed pairs, which lie in expert order, into their tokens, and its
// gradient. Both are bound by memory: every row of y is read (and in the gradient a row
// written) once, so all of a token's rows are in flight together.
//
// A pair's position in the sorted order comes from one scatter of the sorted list into the
// workspace, inv[pair] = position. Dropped pairs are not in the list, so their entries keep
// whatever the workspace held: an entry counts only if the list has that pair there, which
// needs no cleared workspace. Up to kSmallPairs pairs each block inverts the list in LDS
// instead: one launch, and the list is at most 4 KB.
//
// A wave works on one token, so its positions are scalars and its row loads are issued
// together without lane-dependent branches. Measured, 8192 tokens of 8 slots, 2048 columns of
// bf16: forward 60 us, gradient 115 us (5.0 TB/s of what has to move in both; the gradient 94
// when its output buffer stays in the cache from the call before); with one thread per 8
// columns of a token, each looking up its own positions, 104 and 194 us; without the
// non-temporal loads 68 and 124 us. Non-temporal stores gain the forward 3 us, but then its
// output, which the next operator reads, is not in the cache.
#include "grouped.h"

namespace nvfp4 {

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

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

// V consecutive values as loaded (V = 8: 16-byte loads; V = 1: any alignment) and as fp32
template <int T, int V>
struct Raw {
  static constexpr int NW = V == 1 ? 1 : T == 0 ? 8 : 4;
  uint32_t w[NW];
  __device__ __forceinline__ void load(const void* src, size_t at) {
    if constexpr (V == 1) {
      w[0] = T == 0 ? reinterpret_cast<const uint32_t*>(src)[at] : reinterpret_cast<const uint16_t*>(src)[at];
    } else {
      const u32x4_t* p = reinterpret_cast<const u32x4_t*>(reinterpret_cast<const char*>(src) + at * (T == 0 ? 4 : 2));
#pragma unroll
      for (int i = 0; i < NW / 4; ++i) {
        const u32x4_t a = __builtin_nontemporal_load(p + i);  // rows are read once
        w[4 * i] = a.x;
        w[4 * i + 1] = a.y;
        w[4 * i + 2] = a.z;
        w[4 * i + 3] = a.w;
      }
    }
  }
  __device__ __forceinline__ float get(int j) const {
    if constexpr (T == 0) return __uint_as_float(w[j]);
    return to_f32<T>((j & 1) ? w[j / 2] >> 16 : w[j / 2] & 0xFFFFu);
  }
};

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

// Fills the block's LDS copy of the inverse (small lists).
__device__ __forceinline__ void invert_lds(const CombineArgs& c, int P, int32_t* s_inv) {
  for (int p = threadIdx.x; p < P; p += blockDim.x) s_inv[p] = -1;
  __syncthreads();
  for (int r = threadIdx.x; r < P; r += blockDim.x) {
    const int p = c.pairs[r];
    if ((unsigned)p < (unsigned)P) s_inv[p] = r;
  }
  __syncthreads();
}

// Lane s < kSlots looks up slot j0 + s of token t; the wave takes the results as scalars:
// positions (-1: no row) and weights.
template <bool SMALL>
__device__ __forceinline__ void slots(const CombineArgs& c, int P, const int32_t* s_inv, int t, int j0, int* pos,
                                      float* w) {
  const int lane = threadIdx.x & 63;
  int r = -1;
  float wt = 1.f;
  if (lane < kSlots && j0 + lane < c.topk) {
    const int p = t * c.topk + j0 + lane;
    if constexpr (SMALL) {
      r = s_inv[p];
    } else {
      r = c.inv[p];
      if ((unsigned)r >= (unsigned)P || c.pairs[r] != p) r = -1;
    }
    if (c.w != nullptr) wt = c.w[p];
  }
#pragma unroll
  for (int s = 0; s < kSlots; ++s) {
    pos[s] = __builtin_amdgcn_readlane(r, s);
    w[s] = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, wt), s));
  }
}

// G waves per token, V columns per lane at a time: the token's rows, kSlots in flight
// together, added in slot order. The sum stays in registers over all slots, so the loop over
// the columns is the outer one, and more than kSlots slots are looked up once per column step.
template <int T, int V, int G, bool SMALL>
__global__ __launch_bounds__(256) void combine_rows_kernel(CombineArgs c, const void* __restrict__ y,
                                                           void* __restrict__ out, int out_dtype) {
  __shared__ int32_t s_inv[SMALL ? kSmallPairs : 1];
  const int P = c.T * c.topk;
  if constexpr (SMALL) invert_lds(c, P, s_inv);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int t = blockIdx.x * (4 / G) + wave / G, sub = wave % G;
  if (t >= c.T) return;
  int pos[kSlots];
  float w[kSlots];
  slots<SMALL>(c, P, s_inv, t, 0, pos, w);
  for (int c0 = sub * 64 * V; c0 < c.H; c0 += G * 64 * V) {
    const int col = c0 + lane * V;
    const bool in = col < c.H;
    float acc[V];
#pragma unroll
    for (int j = 0; j < V; ++j) acc[j] = 0.f;
    for (int j0 = 0; j0 < c.topk; j0 += kSlots) {
      if (c.topk > kSlots) slots<SMALL>(c, P, s_inv, t, j0, pos, w);
      Raw<T, V> v[kSlots];
      if (in) {
#pragma unroll
        for (int s = 0; s < kSlots; ++s)
          if (pos[s] >= 0) v[s].load(y, (size_t)pos[s] * c.H + col);
#pragma unroll
        for (int s = 0; s < kSlots; ++s)
          if (pos[s] >= 0) {
#pragma unroll
            for (int j = 0; j < V; ++j) acc[j] = fmaf(w[s], v[s].get(j), acc[j]);
          }
      }
    }
    if (in) store_v<V>(out, out_dtype, (size_t)t * c.H + col, acc);
  }
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
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int t = blockIdx.x * (4 / G) + wave / G, sub = wave % G;
  const bool live = t < c.T;
  for (int j0 = 0; j0 < c.topk; j0 += kSlots) {
    int pos[kSlots];
    float w[kSlots], dot[kSlots];
#pragma unroll
    for (int s = 0; s < kSlots; ++s) dot[s] = 0.f;
    if (live) {
      slots<SMALL>(c, P, s_inv, t, j0, pos, w);
      for (int col = (sub * 64 + lane) * V; col < c.H; col += G * 64 * V) {
        Raw<T, V> d, v[kSlots];
        d.load(dout, (size_t)t * c.H + col);
        if constexpr (DW) {
#pragma unroll
          for (int s = 0; s < kSlots; ++s)
            if (pos[s] >= 0) v[s].load(y, (size_t)pos[s] * c.H + col);
        }
#pragma unroll
        for (int s = 0; s < kSlots; ++s)
          if (pos[s] >= 0) {
            float o[V];
#pragma unroll
            for (int j = 0; j < V; ++j) {
              o[j] = w[s] * d.get(j);
              if constexpr (DW) dot[s] = fmaf(d.get(j), v[s].get(j), dot[s]);
            }
            store_v<V>(dy, T, (size_t)pos[s] * c.H + col, o);
          }
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

// Waves per token: one per 64 V columns, at most 4.
static int waves_per_token(int H, int V) { return H <= 64 * V ? 1 : H <= 128 * V ? 2 : 4; }

template <int T, int V, int G>
static void combine_rows_g(const CombineArgs& c, const void* y, void* out, int out_dtype, hipStream_t st) {
  const unsigned grid = (unsigned)((c.T + 4 / G - 1) / (4 / G));
  if (c.T * c.topk <= kSmallPairs)
    combine_rows_kernel<T, V, G, true><<<grid, 256, 0, st>>>(c, y, out, out_dtype);
  else
    combine_rows_kernel<T, V, G, false><<<grid, 256, 0, st>>>(c, y, out, out_dtype);
}

template <int T, int V>
static void combine_rows(const CombineArgs& c, const void* y, void* out, int out_dtype, hipStream_t st) {
  const int G = waves_per_token(c.H, V);
  if (G == 1)
    combine_rows_g<T, V, 1>(c, y, out, out_dtype, st);
  else if (G == 2)
    combine_rows_g<T, V, 2>(c, y, out, out_dtype, st);
  else
    combine_rows_g<T, V, 4>(c, y, out, out_dtype, st);
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

template <int T, int V>
static void combine_grad_t(const CombineArgs& c, const void* dout, const void* y, void* dy, float* dw,
                           hipStream_t st) {
  const int G = waves_per_token(c.H, V);
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
