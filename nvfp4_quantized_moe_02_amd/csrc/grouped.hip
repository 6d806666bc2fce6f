// Matrix products grouped by expert over rows sorted by expert (the order of
// nvfp4_moe_route), with bf16 / fp16 weights and their two gradients, and with int8
// operands that carry a scale per row and per channel; the dense int8 product is the same
// with one expert.
//
//   forward  out[r][n]   = sum_k x[src r][k] w_e[n][k]
//   dx       dx[r][k]    = sum_n dy[r][n] w_e[n][k]
//   dw       dw_e[n][k]  = sum_{r of e} dy[r][n] x[src r][k]
//
// All three are C[m][c] = sum_j A[m][j] B[c][j]. An operand whose contraction index j is
// contiguous in memory (x and w forward, dy in dx) is staged as LDS rows of JB bytes of j;
// the others (w in dx, both in dw) as JB / 2 rows of j, each a run of m or c, and read
// through the LDS transpose load. 64 bytes are 32 sixteen-bit or 64 eight-bit values: two
// matrix instructions of 32 x 32 outputs either way, with the same 16 bytes per lane.
#include <type_traits>

#include "grouped.h"

namespace nvfp4 {

typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef short s16x8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));

constexpr int kFwd = 0, kDx = 1, kDw = 2;
constexpr int kBf16 = 0, kF16 = 1, kI8 = 2;
constexpr int kIdxTile = 1024;  // rows of the gather table of dw

typedef __attribute__((address_space(3))) char* lds_char_t;

// 16 bytes per lane from src to the wave's LDS window at dst (wave-uniform) + 16 * lane.
// In asm because the compiler waits for every outstanding load before any LDS read that
// might alias the builtin's LDS write; the waits are wait_barrier's. The instruction
// writes no register. The address is a scalar base (one per K-block) and a 32-bit offset per lane; gathered rows
// take a whole address per lane.
__device__ __forceinline__ void dma16(const char* base, uint32_t off, uint32_t dst) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(base), "s"(dst)
               : "memory", "m0");
}
__device__ __forceinline__ void dma16(const char* addr, uint32_t dst) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(addr), "s"(dst)
               : "memory", "m0");
}
__device__ __forceinline__ uint32_t lds_addr(const char* p) {
  return __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds_char_t)p);
}
// a value that is the same in every lane, for the scalar unit
__device__ __forceinline__ int uni(int v) { return __builtin_amdgcn_readfirstlane(v); }

// At most N vector loads of this wave outstanding, its LDS reads done, then the barrier.
template <int N>
__device__ __forceinline__ void wait_barrier() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Nothing is scheduled across: the loads and fragment reads stay where they are written.
__device__ __forceinline__ void hold_order() { __builtin_amdgcn_sched_barrier(0); }

__device__ __forceinline__ int clampi(int v, int lo, int hi) { return v < lo ? lo : v > hi ? hi : v; }

// Row of x that sorted row r reads. A pair outside the tokens reads row 0 (in bounds).
__device__ __forceinline__ int src_row(const GroupedArgs& g, int r) {
  if (g.pairs == nullptr) return r;
  const int t = g.pairs[r] / g.topk;
  return (unsigned)t < (unsigned)g.xrows ? t : 0;
}

struct Tile {
  int e, rows, base, nb;  // the tile's rows are base .. base + rows - 1
};

// Row tiles are counted in expert order (an expert with n rows has ceil(n / bm)), and every row
// tile has NB column blocks, one after the other. Each XCD (blockIdx % 8) takes a contiguous
// range of these blocks, so that those that share rows of x and those that share weights meet
// in one L2. Offsets are clamped to [0, P].
//
// Every block finds its tile from the offsets itself (one round trip and one block scan), so
// that no launch and no workspace comes before this one; a launch that lists the tiles gained
// 1 to 4% where there are 1000 tiles. Ranges even in cost rather than in blocks (a first row
// tile, which brings an expert's weights from memory, counted twice) lost 5%. Returns false
// for a block without a tile.
template <int THREADS>
__device__ __forceinline__ bool find_tile(const GroupedArgs& g, int bm, int NB, Tile& t) {
  __shared__ int s_tot[THREADS / 64];
  __shared__ int s_tile[3];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int xcd = blockIdx.x & 7, jj = blockIdx.x >> 3;
  if (g.offsets == nullptr) {
    const long long total = (long long)((g.P + bm - 1) / bm) * NB, per = (total + 7) >> 3;
    const long long L = xcd * per + jj;
    if (jj >= per || L >= total) return false;
    const int mt = (int)(L / NB);
    t = Tile{0, g.P - mt * bm < bm ? g.P - mt * bm : bm, mt * bm, (int)(L - (long long)mt * NB)};
    return true;
  }
  const int per_t = (g.E + THREADS - 1) / THREADS;
  const int e0 = tid * per_t < g.E ? tid * per_t : g.E, e1 = e0 + per_t < g.E ? e0 + per_t : g.E;
  int cnt = 0;
  int lo = clampi(g.offsets[e0], 0, g.P);
  for (int e = e0; e < e1; ++e) {
    const int hi = clampi(g.offsets[e + 1], lo, g.P);
    cnt += (hi - lo + bm - 1) / bm;
    lo = hi;
  }
  int inc = cnt;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int v = __shfl_up(inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 63) s_tot[wave] = inc;
  if (tid == 0) s_tile[2] = 0;
  __syncthreads();
  int before = 0, tiles = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 64; ++w) {
    if (w < wave) before += s_tot[w];
    tiles += s_tot[w];
  }
  const long long total = (long long)tiles * NB, per = (total + 7) >> 3;
  const long long L = xcd * per + jj;
  if (jj >= per || L >= total) return false;
  const int mt = (int)(L / NB);
  int excl = before + inc - cnt;
  if (mt >= excl && mt < excl + cnt) {
    lo = clampi(g.offsets[e0], 0, g.P);
    for (int e = e0; e < e1; ++e) {
      const int hi = clampi(g.offsets[e + 1], lo, g.P);
      const int n = (hi - lo + bm - 1) / bm;
      if (mt < excl + n) {
        const int m0 = (mt - excl) * bm;
        s_tile[0] = e;
        s_tile[1] = lo + m0;
        s_tile[2] = hi - lo - m0 < bm ? hi - lo - m0 : bm;
        break;
      }
      excl += n;
      lo = hi;
    }
  }
  __syncthreads();
  t.e = uni(s_tile[0]);
  t.base = uni(s_tile[1]);
  t.rows = uni(s_tile[2]);
  t.nb = uni((int)(L - (long long)mt * NB));
  return t.rows > 0;  // 0: offsets that do not ascend, whose counts disagree
}

// The slot-th expert of the order in which those with at least the average number of rows come
// first (each half in expert order). A gradient tile takes as long as its expert has rows, so
// the long ones must not come last.
template <int THREADS>
__device__ __forceinline__ int busy_first(const GroupedArgs& g, int slot) {
  __shared__ int s_tot[THREADS / 64];
  __shared__ int s_e;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int per_t = (g.E + THREADS - 1) / THREADS;
  const int e0 = tid * per_t < g.E ? tid * per_t : g.E, e1 = e0 + per_t < g.E ? e0 + per_t : g.E;
  auto busy = [&](int e) {
    const int lo = clampi(g.offsets[e], 0, g.P);
    return (long long)(clampi(g.offsets[e + 1], lo, g.P) - lo) * g.E >= g.P;
  };
  int cnt = 0;
  for (int e = e0; e < e1; ++e) cnt += busy(e);
  int inc = cnt;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int v = __shfl_up(inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 63) s_tot[wave] = inc;
  __syncthreads();
  int before = inc - cnt, all = 0;  // busy experts before e0, and in all
#pragma unroll
  for (int w = 0; w < THREADS / 64; ++w) {
    if (w < wave) before += s_tot[w];
    all += s_tot[w];
  }
  for (int e = e0; e < e1; ++e) {
    const bool b = busy(e);
    if ((b ? before : all + e - before) == slot) s_e = e;
    before += b;
  }
  __syncthreads();
  return uni(s_e);
}

template <int T>
struct Acc {
  typedef f32x16_t v32;
  typedef f32x4_t v16;
};
template <>
struct Acc<kI8> {
  typedef i32x16_t v32;
  typedef i32x4_t v16;
};

template <int T>
__device__ __forceinline__ typename Acc<T>::v32 mma(i32x4_t a, i32x4_t b, typename Acc<T>::v32 c) {
  if constexpr (T == kBf16)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c,
                                                   0, 0, 0);
  else if constexpr (T == kF16)
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b), c, 0,
                                                  0, 0);
  else
    return __builtin_amdgcn_mfma_i32_32x32x32_i8(a, b, c, 0, 0, 0);
}
template <int T>
__device__ __forceinline__ typename Acc<T>::v16 mma(i32x4_t a, i32x4_t b, typename Acc<T>::v16 c) {
  if constexpr (T == kBf16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c,
                                                   0, 0, 0);
  else if constexpr (T == kF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b), c, 0,
                                                  0, 0);
  else
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
}

// ------------------------------------------------------------------ LDS images of a K-block
// Straight operand: rows of JB bytes, 16-byte chunk c of row r in slot c ^ key(r): the 16
// rows that an LDS read cycle serves then cover all 64 banks once (measured: no conflicts).
template <int JB>
struct Straight {
  static constexpr int CPR = JB / 16;
  __device__ static int key(int row) { return JB == 64 ? (row >> 2) & 3 : (row >> 1) & 7; }
  __device__ static int at(int row, int chunk) { return row * JB + ((chunk ^ key(row)) << 4); }
};

// Transposed operand: JB / 2 contraction rows of W elements (2 W bytes). A transpose load
// takes 4 rows x 64 bytes per 32 lanes; the 64-byte blocks of a row are permuted by the
// row so that those four rows fall on different banks.
template <int W>
struct Trans {
  static constexpr int RBY = W * 2;
  static constexpr int PER = RBY >= 256 ? 1 : 256 / RBY;
  static constexpr int MASK = (RBY / 64 < 4 ? RBY / 64 : 4) - 1;
  static constexpr int CPR = RBY / 16;
  __device__ static int key(int row) { return (row / PER) & MASK; }
};

template <int OP, int T, int WM, int WN, int RB, int CB, int MT, int JB, int ST>
struct Cfg {
  static constexpr int BM = WM * RB * 32, BN = WN * CB * 32, THREADS = WM * WN * 64;
  static constexpr bool ATR = OP == kDw, BTR = OP != kFwd;
  static constexpr int ABYTES = BM * JB, BBYTES = BN * JB, STAGE = ABYTES + BBYTES;
  static constexpr int NLA = ABYTES / 16 / THREADS, NLB = BBYTES / 16 / THREADS;
  static_assert(ST * STAGE / (WM * WN) >= 32 * (CB * 128 + 16), "room for the epilogue");
  // The tiles of large products store past the L2, which their outputs would only sweep: dw of 512
  // experts 1201 -> 1073 us, int8 down 285 -> 276, dense int8 122 -> 116, dx of 64 experts 449 ->
  // 440. The small tiles leave theirs in the cache for the next operator.
  static constexpr bool NT = BM * BN >= 128 * 256;
  static_assert(MT == 32 || OP == kFwd, "transposed operands are read for 32 x 32");
  static_assert(JB >= 128 || MT == 32, "two steps per K-block at least");
  static_assert(ABYTES / 16 % THREADS == 0 && BBYTES / 16 % THREADS == 0, "whole loads per thread");
};

// Stores a wave's NRB x CB blocks of 32 x 32 outputs of OS bytes each, one row block at a
// time through `buf` (wave-private LDS). value(rb, cb, i, scale) is accumulator element i;
// rows first .. of the tile below mlim exist, as do columns below nout. NT: non-temporal stores.
template <int OS, int MT, int CB, int NRB, bool ALIGNED, bool NT, class V, class S>
__device__ __forceinline__ void store_rows(const GroupedArgs& g, char* buf, V value, S scale, int first, int mlim,
                                           size_t out0, int col0, int nout) {
  const int lane = threadIdx.x & 63, part = lane / MT, lm = lane % MT;
  constexpr int U = 32 / MT, Q = MT == 32 ? 4 : 1;  // blocks per 32, runs of 4 columns per block and lane
  constexpr int PITCH = CB * 32 * OS + 16;
  constexpr int CPR = CB * 32 * OS / 16;  // 16-byte chunks per row
  constexpr int E = 16 / OS;              // outputs per chunk
  char* out = reinterpret_cast<char*>(g.out);
  const bool vec = ALIGNED || nout % E == 0;
  const int ch = lane % CPR, r0 = lane / CPR;
  const int col = col0 + ch * E;
#pragma unroll
  for (int rb = 0; rb < NRB; ++rb) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float rs = scale(rb * U + u);
#pragma unroll
      for (int cb = 0; cb < CB * U; ++cb)
#pragma unroll
        for (int q = 0; q < Q; ++q) {
          float v[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) v[j] = value(rb * U + u, cb, 4 * q + j, rs);
          char* p = buf + (u * MT + lm) * PITCH + (cb * MT + 8 * q + 4 * part) * OS;
          if constexpr (OS == 4) {
            *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
          } else {
            uint32_t h[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) h[j] = g.out_dtype == 1 ? f32_to_bf16_bits(v[j]) : f32_to_f16_bits(v[j]);
            *reinterpret_cast<uint2*>(p) = make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
          }
        }
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the other lanes' rows are in LDS
#pragma unroll
    for (int i = 0; i < CPR / 2; ++i) {
      const int r = r0 + i * (64 / CPR), row = first + rb * 32 + r;
      const uint4 v = *reinterpret_cast<const uint4*>(buf + r * PITCH + ch * 16);
      if (row < mlim && col < nout) {
        char* p = out + ((out0 + row) * nout + col) * OS;
        if (vec) {
          const i32x4_t o = {(int)v.x, (int)v.y, (int)v.z, (int)v.w};
          if constexpr (NT)
            __builtin_nontemporal_store(o, reinterpret_cast<i32x4_t*>(p));
          else
            *reinterpret_cast<i32x4_t*>(p) = o;
        } else {
          const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int j = 0; j < E; ++j)
            if (col + j < nout) {
              if constexpr (OS == 4)
                reinterpret_cast<uint32_t*>(p)[j] = u[j];
              else
                reinterpret_cast<uint16_t*>(p)[j] = (uint16_t)(u[j / 2] >> (16 * (j & 1)));
            }
        }
      }
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // read before the next row block overwrites
  }
}

// The tile's K loop and epilogue for NRB occupied row blocks of this wave (0 .. RB).
//
// Every K-block is KS steps of 32 bytes of the contraction (64 for 16 x 16 matrix
// instructions, MT 16). A step's fragments are read while
// the step before multiplies. The last step of a K-block starts with the one barrier: by
// then every wave holds that K-block's last fragments, so its stage may be refilled, and the
// next K-block's loads have arrived, so its first fragments are read under the last step's
// matrix instructions. The refill's loads are issued one at a time between them: in one burst
// they queue in the address unit ahead of the wave's next instructions.
//
// Bound by the matrix cores where experts have many rows (dense bf16 8192 x 4096 x 4096, 275
// GFLOP: 228 us, 1.2 PFLOP/s; int8 117 us, 2.35 POP/s), by the weights' bytes where they have
// few (512 experts of 8 rows, 3.2 GB: 547 us, 5.9 TB/s).
template <int OP, int T, int WM, int WN, int RB, int CB, int MT, int JB, int ST, int NRB>
__device__ __forceinline__ void tile_product(const GroupedArgs& g, int e, int base, int mrows, int m0, int c0, int C,
                                             char* lds, int* s_src) {
  typedef Cfg<OP, T, WM, WN, RB, CB, MT, JB, ST> F;
  constexpr int ES = T == kI8 ? 1 : 2;
  constexpr int THREADS = F::THREADS;
  // loads of A: only the occupied row blocks when one row of waves covers the straight tile
  constexpr int NA = F::ATR || WM > 1 ? F::NLA : (NRB * 32 * (JB / 16) + THREADS - 1) / THREADS;
  constexpr int NBL = F::NLB;
  constexpr int LPS = NA + NBL;  // loads per stage and thread
  const int tid = threadIdx.x, lane = tid & 63, wave = uni(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int part = lane / MT, lm = lane % MT;
  const int nout = OP == kFwd ? g.N : g.K;  // columns of C
  const int mlim = OP == kDw ? g.N - m0 : mrows;  // rows of C from the tile's first
  constexpr int JE = JB / ES;               // contraction elements per K-block
  constexpr int JR = JB / 2;                // contraction rows per K-block of a transposed operand
  constexpr int SB = MT == 32 ? 32 : 64;    // bytes of the contraction per matrix instruction
  constexpr int KS = JB / SB;               // matrix-instruction steps per K-block
  typedef Straight<JB> SX;
  const int nk = (C + JE - 1) / JE;
  const int tail = C - (nk - 1) * JE;       // elements of the last K-block

  // ---- where this thread's chunks come from: scalar bases that move with the K-blocks and
  // offsets from them (below 2^32: a tile is at most 256 rows of 2^20 values); rows of x that
  // may be gathered (forward A, dw's B) have 64-bit addresses
  constexpr bool AG = OP == kFwd;
  const char* abase = reinterpret_cast<const char*>(g.a);
  const char* bbase = reinterpret_cast<const char*>(g.b);
  uint32_t ao[NA], bo[NBL];
  const char* ap[NA];
  int arow[NA], brow[NBL], ach[NA], bch[NBL];
  const size_t astep = F::ATR ? (size_t)JR * g.N * 2 : JB, bstep = F::BTR ? (size_t)JR * g.K * 2 : JB;
  if constexpr (F::ATR)
    abase += ((size_t)base * g.N + m0) * 2;
  else if constexpr (OP == kDx)
    abase += (size_t)base * g.N * ES;
  if constexpr (OP == kFwd)
    bbase += ((size_t)e * g.N + c0) * g.K * ES;
  else if constexpr (OP == kDx)
    bbase += ((size_t)e * g.N * g.K + c0) * 2;
  else
    bbase += (size_t)c0 * 2;
#pragma unroll
  for (int i = 0; i < NA; ++i) {
    const int ci = i * THREADS + tid;
    if constexpr (!F::ATR) {
      arow[i] = ci / SX::CPR;
      ach[i] = (ci % SX::CPR) ^ SX::key(arow[i]);
      const int r = arow[i] < mrows ? arow[i] : mrows - 1;
      if constexpr (AG)
        ap[i] = abase + (size_t)s_src[r] * g.K * ES + ach[i] * 16;
      else
        ao[i] = r * (uint32_t)(g.N * ES) + ach[i] * 16;
    } else {
      typedef Trans<F::BM> X;
      arow[i] = ci / X::CPR;
      const int s = ci % X::CPR;
      const int ch = (((s >> 2) ^ X::key(arow[i])) << 2) | (s & 3);
      ach[i] = 0;
      ao[i] = (arow[i] * (uint32_t)g.N + (m0 + ch * 8 < g.N ? ch * 8 : 0)) * 2;
    }
  }
#pragma unroll
  for (int i = 0; i < NBL; ++i) {
    const int ci = i * THREADS + tid;
    if constexpr (!F::BTR) {
      brow[i] = ci / SX::CPR;
      bch[i] = (ci % SX::CPR) ^ SX::key(brow[i]);
      const int n = c0 + brow[i] < g.N ? brow[i] : g.N - 1 - c0;
      bo[i] = n * (uint32_t)(g.K * ES) + bch[i] * 16;
    } else {
      typedef Trans<F::BN> X;
      brow[i] = ci / X::CPR;
      const int s = ci % X::CPR;
      const int ch = (((s >> 2) ^ X::key(brow[i])) << 2) | (s & 3);
      bch[i] = 0;
      // dw: the row comes from the table; bo is the column only
      bo[i] = ((OP == kDx ? brow[i] * (uint32_t)g.K : 0) + (c0 + ch * 8 < g.K ? ch * 8 : 0)) * 2;
    }
  }
  // Before the loads of K-block kb: in the last one, chunks and rows past the contraction's
  // end read something in bounds (zero_tail clears them in LDS); dw's table of source rows
  // is refilled every kIdxTile rows (a barrier: kb is the same in every wave, and every
  // wave has passed a barrier since its last look at the table).
  auto prepare = [&](int kb) {
    if (kb == nk - 1 && tail < JE) {
#pragma unroll
      for (int i = 0; i < NA; ++i) {
        if constexpr (F::ATR)
          ao[i] -= arow[i] >= tail ? (arow[i] - (tail - 1)) * (uint32_t)g.N * 2 : 0;
        else if constexpr (AG)
          ap[i] -= ach[i] * (16 / ES) >= tail ? ach[i] * 16 : 0;
        else
          ao[i] -= ach[i] * (16 / ES) >= tail ? ach[i] * 16 : 0;
      }
      if constexpr (OP != kDw) {
#pragma unroll
        for (int i = 0; i < NBL; ++i) {
          if constexpr (F::BTR)
            bo[i] -= brow[i] >= tail ? (brow[i] - (tail - 1)) * (uint32_t)g.K * 2 : 0;
          else
            bo[i] -= bch[i] * (16 / ES) >= tail ? bch[i] * 16 : 0;
        }
      }
    }
    if constexpr (OP == kDw) {
      if (kb % (kIdxTile / JR) == 0) {
        for (int r = tid; r < kIdxTile; r += THREADS) {
          const int j = kb * JR + r;
          s_src[r] = src_row(g, base + (j < C ? j : C - 1));
        }
        lds_barrier();
      }
    }
  };
  const uint32_t lds0 = lds_addr(lds) + wave * 1024;
  // load i of K-block kb into stage s (in order; prepare(kb) first)
  auto issue = [&](int kb, int s, int i) {
    const uint32_t dst = lds0 + s * F::STAGE + i * THREADS * 16;
    if (i < NA) {
      if constexpr (AG) {
        dma16(ap[i], dst);
        ap[i] += JB;
      } else {
        dma16(abase + kb * astep, ao[i], dst);
      }
    } else {
      const int b = i - NA;
      const uint32_t d = dst + (F::NLA - NA) * THREADS * 16;
      if constexpr (OP == kDw)
        dma16(bbase + (size_t)s_src[(kb * JR + brow[b]) % kIdxTile] * (g.K * 2) + bo[b], d);
      else
        dma16(bbase + kb * bstep, bo[b], d);
    }
  };
  auto zero_tail = [&](int s) {
    char* As = lds + s * F::STAGE;
    char* Bs = As + F::ABYTES;
    const uint4 z = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < NA; ++i)
      if (F::ATR ? arow[i] >= tail : ach[i] * (16 / ES) >= tail)
        *reinterpret_cast<uint4*>(As + (i * THREADS + tid) * 16) = z;
#pragma unroll
    for (int i = 0; i < NBL; ++i)
      if (F::BTR ? brow[i] >= tail : bch[i] * (16 / ES) >= tail)
        *reinterpret_cast<uint4*>(Bs + (i * THREADS + tid) * 16) = z;
    lds_barrier();
  };
  // fragment of operand block `blk` (MT rows of m or c), step ks: lane (part, lm) has 16 bytes of
  // row lm
  auto frag_straight = [&](const char* S, int blk, int ks) -> i32x4_t {
    return *reinterpret_cast<const i32x4_t*>(S + SX::at(blk * MT + lm, ks * (SB / 16) + part));
  };
  const int tr_row = 8 * part + ((lane & 15) >> 2);
  const int tr_in = (16 * ((lane >> 4) & 1) + 4 * (lane & 3)) * 2;
  auto frag_trans = [&](const char* S, auto x, int blk, int ks) -> i32x4_t {
    typedef decltype(x) X;
    s16x4_t q[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int row = ks * 16 + tr_row + 4 * h;
      const char* p = S + row * X::RBY + ((blk ^ X::key(row)) << 6) + tr_in;
      q[h] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          reinterpret_cast<__attribute__((address_space(3))) s16x4_t*>((lds_char_t)p));
    }
    return __builtin_bit_cast(i32x4_t, __builtin_shufflevector(q[0], q[1], 0, 1, 2, 3, 4, 5, 6, 7));
  };

  constexpr int U = 32 / MT;           // instructions' blocks per 32 rows or columns
  constexpr int RM = NRB * U, CM = CB * U;
  constexpr int R = RM > 0 ? RM : 1;
  constexpr int AV = MT == 32 ? 16 : 4;  // accumulator elements per lane and block
  typedef typename std::conditional<MT == 32, typename Acc<T>::v32, typename Acc<T>::v16>::type AccV;
  AccV acc[R][CM];
#pragma unroll
  for (int rb = 0; rb < R; ++rb)
#pragma unroll
    for (int cb = 0; cb < CM; ++cb)
#pragma unroll
      for (int i = 0; i < AV; ++i) acc[rb][cb][i] = 0;
  i32x4_t fa[2][R], fb[2][CM];
  // fragment f of step ks of stage s into set q: the CM of B, then the RM of A
  auto read_frag = [&](int s, int ks, int q, int f) {
    const char* As = lds + s * F::STAGE;
    const char* Bs = As + F::ABYTES;
    if (f < CM) {
      if constexpr (F::BTR)
        fb[q][f] = frag_trans(Bs, Trans<F::BN>{}, wn * CM + f, ks);
      else
        fb[q][f] = frag_straight(Bs, wn * CM + f, ks);
    } else {
      if constexpr (F::ATR)
        fa[q][f - CM] = frag_trans(As, Trans<F::BM>{}, wm * RB * U + f - CM, ks);
      else
        fa[q][f - CM] = frag_straight(As, wm * RB * U + f - CM, ks);
    }
  };
  constexpr int NF = NRB > 0 ? CM + RM : 0;
  auto read_frags = [&](int s, int ks, int q) {
#pragma unroll
    for (int f = 0; f < NF; ++f) read_frag(s, ks, q, f);
  };
  // step ks's matrix instructions, with share `slot` of the loads of K-block `fill` between
  constexpr int PER = (LPS + KS - 1) / KS;
  auto multiply = [&](int ks, auto filling, int slot, int fill, int fstage) {
#pragma unroll
    for (int rb = 0; rb < R; ++rb) {
      if constexpr (NRB > 0) {
#pragma unroll
        for (int cb = 0; cb < CM; ++cb) {
          acc[rb][cb] = mma<T>(fb[ks & 1][cb], fa[ks & 1][rb], acc[rb][cb]);
        }
      }
      if constexpr (decltype(filling)::value) {
#pragma unroll
        for (int i = 0; i < PER; ++i)
          if (i * R / PER == rb && slot * PER + i < LPS) {
            issue(fill, fstage, slot * PER + i);
            hold_order();
          }
      }
    }
  };

  // The same with one fragment of the next step (rs, rks) read before each matrix instruction
  // instead of all of them ahead of the step (16 x 16 instructions, of which a step has 2 to 3
  // times as many as fragments).
  auto interleaved = [&](int ks, int rs, int rks, int slot, int fill, int fstage) {
    constexpr int NM = RM * CM, SL = NM > 0 ? NM : 1;
    constexpr int RPS = (NF + SL - 1) / SL;
#pragma unroll
    for (int rb = 0; rb < R; ++rb)
#pragma unroll
      for (int cb = 0; cb < CM; ++cb) {
        const int i = rb * CM + cb;
        if constexpr (NRB > 0) {
#pragma unroll
          for (int f = 0; f < RPS; ++f)
            if (i * RPS + f < NF) read_frag(rs, rks, (ks & 1) ^ 1, i * RPS + f);
          acc[rb][cb] = mma<T>(fb[ks & 1][cb], fa[ks & 1][rb], acc[rb][cb]);
        }
#pragma unroll
        for (int l = 0; l < PER; ++l)
          if ((2 * l + 1) * SL / (2 * PER) == (NRB > 0 ? i : 0) && (NRB > 0 || cb == 0) && slot * PER + l < LPS)
            issue(fill, fstage, slot * PER + l);
      }
  };

  if (nk > 0) {
#pragma unroll
    for (int s = 0; s < ST; ++s)
      if (s < nk) {
        prepare(s);
#pragma unroll
        for (int i = 0; i < LPS; ++i) issue(s, s, i);
      }
    if (nk >= ST)
      wait_barrier<LPS*(ST - 1)>();
    else
      wait_barrier<0>();
    if (nk == 1 && tail < JE) zero_tail(0);
    read_frags(0, 0, 0);
#pragma unroll
    for (int ks = 0; ks + 1 < KS; ++ks) {
      read_frags(0, ks + 1, (ks + 1) & 1);
      multiply(ks, std::false_type{}, 0, 0, 0);
    }
  }
  int cur = 0, kb = 0;
  // the last step of K-block kb, the others of kb + 1, and the loads of kb + ST
  for (; kb + ST < nk; ++kb) {
    const int nxt = cur + 1 == ST ? 0 : cur + 1;
    wait_barrier<LPS*(ST - 2)>();
    if constexpr (MT == 16) {
      prepare(kb + ST);
      interleaved(KS - 1, nxt, 0, 0, kb + ST, cur);
#pragma unroll
      for (int ks = 0; ks + 1 < KS; ++ks) interleaved(ks, nxt, ks + 1, ks + 1, kb + ST, cur);
    } else {
      read_frags(nxt, 0, 0);
      prepare(kb + ST);
      hold_order();
      multiply(KS - 1, std::true_type{}, 0, kb + ST, cur);
#pragma unroll
      for (int ks = 0; ks + 1 < KS; ++ks) {
        read_frags(nxt, ks + 1, (ks + 1) & 1);
        hold_order();
        multiply(ks, std::true_type{}, ks + 1, kb + ST, cur);
      }
    }
    cur = nxt;
  }
  for (; kb < nk; ++kb) {
    const int nxt = cur + 1 == ST ? 0 : cur + 1;
    const int later = nk - 2 - kb;  // K-blocks behind the next one, all being loaded
    if (later >= 0) {
      if (ST > 3 && later >= 2)
        wait_barrier<LPS*(ST > 3 ? 2 : 0)>();
      else if (ST > 2 && later == 1)
        wait_barrier<LPS*(ST > 2 ? 1 : 0)>();
      else
        wait_barrier<0>();
      if (later == 0 && tail < JE) zero_tail(nxt);
      read_frags(nxt, 0, 0);
    }
    multiply(KS - 1, std::false_type{}, 0, 0, 0);
    if (later >= 0) {
#pragma unroll
      for (int ks = 0; ks + 1 < KS; ++ks) {
        read_frags(nxt, ks + 1, (ks + 1) & 1);
        multiply(ks, std::false_type{}, 0, 0, 0);
      }
    }
    cur = nxt;
  }

  // Accumulator element i of lane (part, lm): row lm of the row block, column
  // 8 (i / 4) + 4 part + i % 4 of the column block. Each wave passes a row block through
  // its part of the stages, so that it stores whole runs of a row (128 bytes of 16-bit outputs)
  // instead of 8 bytes per row.
  lds_barrier();
  if constexpr (NRB > 0) {
    char* mine = lds + wave * (ST * F::STAGE / (WM * WN));
    const int col0 = c0 + wn * CB * 32;
    float bs[CM][AV];
    if constexpr (T == kI8) {
#pragma unroll
      for (int cb = 0; cb < CM; ++cb)
#pragma unroll
        for (int i = 0; i < AV; ++i) {
          const int col = col0 + cb * MT + 8 * (i >> 2) + 4 * part + (i & 3);
          bs[cb][i] = g.b_scale[(size_t)e * g.N + (col < g.N ? col : g.N - 1)];
        }
    }
    const size_t out0 = OP == kDw ? (size_t)e * g.N + m0 : (size_t)base;
    auto value = [&](int rb, int cb, int i, float rs) -> float {
      float v = (float)acc[rb][cb][i];
      if constexpr (T == kI8) {
        v = v * rs * bs[cb][i];
        // the output is this fp32 value rounded again: kept apart from the narrowing, which the
        // backend would fold into one mixed-precision multiply
        asm volatile("" : "+v"(v));
      }
      return v;
    };
    auto scale = [&](int rb) { return T == kI8 ? g.a_scale[s_src[wm * RB * 32 + rb * MT + lm]] : 1.f; };
    if (g.out_dtype == 0)
      store_rows<4, MT, CB, NRB, OP != kFwd || T != kI8, F::NT>(g, mine, value, scale, wm * RB * 32, mlim, out0, col0, nout);
    else
      store_rows<2, MT, CB, NRB, OP != kFwd || T != kI8, F::NT>(g, mine, value, scale, wm * RB * 32, mlim, out0, col0, nout);
  }
}

template <int OP, int T, int WM, int WN, int RB, int CB, int MT, int JB, int ST>
__global__ __launch_bounds__(WM* WN * 64, 2) void grouped_kernel(GroupedArgs g, int NB, bool ordered) {
  typedef Cfg<OP, T, WM, WN, RB, CB, MT, JB, ST> F;
  __shared__ __attribute__((aligned(256))) char lds[ST * F::STAGE];
  __shared__ int s_src[OP == kDw ? kIdxTile : F::BM];
  if constexpr (OP == kDw) {
    // Every XCD takes an eighth of each expert's tiles (BM rows n, BN columns k), so experts
    // with many rows do not gather on one; which eighth turns with the expert.
    const int tiles = (g.N + F::BM - 1) / F::BM * NB, per = (tiles + 7) >> 3;
    const int j = blockIdx.x >> 3;
    const int slot = j / per, tile = ((blockIdx.x + slot) & 7) * per + (j - slot * per);
    if (tile >= tiles) return;
    const int e = ordered ? busy_first<F::THREADS>(g, slot) : slot;
    const int mb = tile / NB, nb = tile - mb * NB;
    const int lo = uni(clampi(g.offsets[e], 0, g.P)), hi = uni(clampi(g.offsets[e + 1], lo, g.P));
    // an expert without rows has a zero gradient: no K-block, the cleared accumulator is stored
    tile_product<OP, T, WM, WN, RB, CB, MT, JB, ST, RB>(g, e, lo, 0, mb * F::BM, nb * F::BN, hi - lo, lds, s_src);
  } else {
    Tile t;
    if (!find_tile<F::THREADS>(g, F::BM, NB, t)) return;
    const int base = t.base;
    if constexpr (OP == kFwd) {
      for (int r = threadIdx.x; r < F::BM; r += F::THREADS)
        s_src[r] = src_row(g, base + (r < t.rows ? r : t.rows - 1));
      __syncthreads();
    }
    const int c0 = t.nb * F::BN, C = OP == kFwd ? g.K : g.N;
    // occupied row blocks of this wave's row of waves (the same in all its lanes)
    const int nrb = uni(clampi(((t.rows + 31) >> 5) - (int)(threadIdx.x >> 6) / WN * RB, 0, RB));
#define NVFP4_TILE(NRB) tile_product<OP, T, WM, WN, RB, CB, MT, JB, ST, NRB>(g, t.e, base, t.rows, 0, c0, C, lds, s_src)
    if (nrb == RB)
      NVFP4_TILE(RB);
    else if (RB > 3 && nrb == 3)
      NVFP4_TILE((RB > 3 ? 3 : RB));
    else if (RB > 2 && nrb == 2)
      NVFP4_TILE((RB > 2 ? 2 : RB));
    else if (WM > 1 && nrb == 0)
      NVFP4_TILE((WM > 1 ? 0 : RB));
    else
      NVFP4_TILE(1);
#undef NVFP4_TILE
  }
}

// ------------------------------------------------------------------ few rows
// Four adjacent outputs of one row, rounded once to the output type. n: columns left in
// the row (fewer than 4 only in the last group); vec: the row's groups of 4 are aligned.
__device__ __forceinline__ void store4(void* out, int dtype, size_t at, const float* v, int n, bool vec) {
  if (n <= 0) return;
  if (dtype == 0) {
    float* o = reinterpret_cast<float*>(out) + at;
    if (vec && n >= 4)
      *reinterpret_cast<float4*>(o) = make_float4(v[0], v[1], v[2], v[3]);
    else
      for (int j = 0; j < 4; ++j)
        if (j < n) o[j] = v[j];
  } else {
    uint16_t* o = reinterpret_cast<uint16_t*>(out) + at;
    uint32_t h[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) h[j] = dtype == 1 ? f32_to_bf16_bits(v[j]) : f32_to_f16_bits(v[j]);
    if (vec && n >= 4)
      *reinterpret_cast<uint2*>(o) = make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
    else
      for (int j = 0; j < 4; ++j)
        if (j < n) o[j] = (uint16_t)h[j];
  }
}

// Forward product of up to 16 RB rows: bound by reading the weights once. A block takes 16 NW
// weight rows of one expert; its four waves split the contraction, each reading U
// consecutive 64-byte steps of its rows straight into registers (U (NW + RB) loads of 16
// bytes per lane in flight) and multiplying them on 16 x 16 matrix instructions, the weights as
// the first operand. The four partial results are added in wave order through LDS. Measured: one
// token over 8 of 512 experts, 50 MB of bf16 weights, 12.4 us (4.1 TB/s); one row of dense int8
// 2048 x 2048 4.0 us, of which an empty launch is 1.6.
template <int T, int RB, int U, int NW>
__global__ __launch_bounds__(256) void stream_kernel(GroupedArgs g, int NB) {
  constexpr int ES = T == kI8 ? 1 : 2;
  typedef typename Acc<T>::v16 V;
  __shared__ V s_part[4][NW * RB][64];
  Tile t;
  if (!find_tile<256>(g, 16 * RB, NB, t)) return;
  const int lane = threadIdx.x & 63, wave = uni(threadIdx.x >> 6);
  const int l16 = lane & 15, ch = lane >> 4;
  const int base = t.base;
  const int n0 = t.nb * 16 * NW;
  const int kb = g.K * ES;  // bytes of a row
  const char* wp[NW];
  const char* xp[RB];
  int src[RB];
#pragma unroll
  for (int q = 0; q < NW; ++q) {
    const int n = n0 + q * 16 + l16 < g.N ? n0 + q * 16 + l16 : g.N - 1;
    wp[q] = reinterpret_cast<const char*>(g.b) + ((size_t)t.e * g.N + n) * kb + ch * 16;
  }
#pragma unroll
  for (int rb = 0; rb < RB; ++rb) {
    const int r = rb * 16 + l16;
    src[rb] = src_row(g, base + (r < t.rows ? r : t.rows - 1));
    xp[rb] = reinterpret_cast<const char*>(g.a) + (size_t)src[rb] * kb + ch * 16;
  }
  V acc[NW][RB];
#pragma unroll
  for (int q = 0; q < NW; ++q)
#pragma unroll
    for (int rb = 0; rb < RB; ++rb)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[q][rb][i] = 0;
  for (int s0 = wave * U; s0 * 64 < kb; s0 += 4 * U) {
    i32x4_t w[NW][U], x[RB][U];
    const int at = s0 * 64;
    if (at + U * 64 <= kb) {
#pragma unroll
      for (int q = 0; q < NW; ++q)
#pragma unroll
        for (int u = 0; u < U; ++u) w[q][u] = *reinterpret_cast<const i32x4_t*>(wp[q] + at + u * 64);
#pragma unroll
      for (int rb = 0; rb < RB; ++rb)
#pragma unroll
        for (int u = 0; u < U; ++u) x[rb][u] = *reinterpret_cast<const i32x4_t*>(xp[rb] + at + u * 64);
    } else {
      // the row's end: chunks past it are zero in both operands
      const i32x4_t z = {0, 0, 0, 0};
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const bool in = at + u * 64 + ch * 16 < kb;
#pragma unroll
        for (int q = 0; q < NW; ++q) w[q][u] = in ? *reinterpret_cast<const i32x4_t*>(wp[q] + at + u * 64) : z;
#pragma unroll
        for (int rb = 0; rb < RB; ++rb) x[rb][u] = in ? *reinterpret_cast<const i32x4_t*>(xp[rb] + at + u * 64) : z;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int q = 0; q < NW; ++q)
#pragma unroll
        for (int rb = 0; rb < RB; ++rb) acc[q][rb] = mma<T>(w[q][u], x[rb][u], acc[q][rb]);
  }
#pragma unroll
  for (int q = 0; q < NW; ++q)
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) s_part[wave][q * RB + rb][lane] = acc[q][rb];
  __syncthreads();
  // wave w finishes block w of the NW x RB: lane (ch, l16) has row l16 and columns 4 ch ..
#pragma unroll
  for (int q = 0; q < NW; ++q)
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
      if (q * RB + rb != wave) continue;
      const int r = rb * 16 + l16;
      if (r >= t.rows) continue;
      V sum = s_part[0][q * RB + rb][lane];
#pragma unroll
      for (int w = 1; w < 4; ++w) sum += s_part[w][q * RB + rb][lane];
      const int col = n0 + q * 16 + 4 * ch;
      float v[4];
      float rs = 1.f;
      if constexpr (T == kI8) rs = g.a_scale[src[rb]];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[j] = (float)sum[j];
        if constexpr (T == kI8) {
          v[j] = v[j] * rs * g.b_scale[(size_t)t.e * g.N + (col + j < g.N ? col + j : g.N - 1)];
          asm volatile("" : "+v"(v[j]));  // rounded to fp32 before the output type, as in tile_product
        }
      }
      store4(g.out, g.out_dtype, (size_t)(base + r) * g.N + col, v, g.N - col, (g.N & 3) == 0);
    }
}

// The most row tiles that P rows in E experts can make.
static long long most_tiles(int P, int E, int bm) { return P / bm + (E < P ? E : P); }

// Blocks of a grid whose blocks find their tiles.
static unsigned grid_rows(const GroupedArgs& g, int bm, int NB) {
  const long long tiles = g.offsets == nullptr ? ((long long)g.P + bm - 1) / bm : most_tiles(g.P, g.E, bm);
  return (unsigned)((tiles * NB + 7) / 8 * 8);
}

template <int OP, int T, int WM, int WN, int RB, int CB, int MT, int JB, int ST>
static hipError_t launch_cfg(const GroupedArgs& g, hipStream_t st) {
  typedef Cfg<OP, T, WM, WN, RB, CB, MT, JB, ST> F;
  const int nout = OP == kFwd ? g.N : g.K;
  const int NB = (nout + F::BN - 1) / F::BN;
  // dw: the search costs a block about a microsecond. 64 experts of 1024 rows on average under Zipf
  // routing 470 -> 448 us, 8 of 2048 131 -> 118; 64 of 128 rows 156 -> 162, 512 of 32 807 -> 830.
  const bool ordered = OP == kDw && g.E > 1 && g.P / g.E >= 256;
  unsigned grid;
  if (OP == kDw)
    grid = (unsigned)((long long)g.E * (((g.N + F::BM - 1) / F::BM * NB + 7) / 8) * 8);
  else
    grid = grid_rows(g, F::BM, NB);
  grouped_kernel<OP, T, WM, WN, RB, CB, MT, JB, ST><<<grid, F::THREADS, 0, st>>>(g, NB, ordered);
  return hipGetLastError();
}

template <int T, int RB, int U, int NW>
static hipError_t launch_stream(const GroupedArgs& g, hipStream_t st) {
  static_assert(NW * RB <= 4, "one wave finishes each block");
  const int NB = (g.N + 16 * NW - 1) / (16 * NW);
  stream_kernel<T, RB, U, NW><<<grid_rows(g, 16 * RB, NB), 256, 0, st>>>(g, NB);
  return hipGetLastError();
}

// Rows of an expert when all experts that can have rows have the same, and the row tiles of bm
// rows that this makes.
struct Load {
  int64_t experts, rows;
  explicit Load(const GroupedArgs& g) {
    experts = g.offsets == nullptr ? 1 : (g.E < g.P ? g.E : g.P);
    rows = (g.P + experts - 1) / experts;
  }
  int64_t tiles(int bm) const { return experts * ((rows + bm - 1) / bm); }
};
static int64_t blocks(int64_t n, int b) { return (n + b - 1) / b; }

// The largest tile that still fills the device, because a larger tile reads less per product:
//   256 x 256, 8 waves, one block per CU: forward two 128-byte stages and 16 x 16 matrix
//     instructions, the gradients four 64-byte stages and 32 x 32
//   128 x 256, 4 waves, two blocks per CU, three stages: less of a tile is empty at the end
//     of an expert, and one block's stores overlap the other's products
//   64 x 128, 4 waves, two blocks per CU, three 128-byte stages
//   64 x 64, 4 waves, four 128-byte stages
// Measured, us (top 8, 2048 -> 1536 in bf16 unless said): 64 experts, 8192 tokens, forward
// 256 x 256 406 (as the gradients' 419), 128 x 256 472, 64 x 128 600; dx 440 (as the forward's
// 475) / 435 / 670; dense int8 8192 x 4096 x 4096 117 (133); 8 experts, forward 113 / 132 /
// 155; 512 experts, uniform, 32 rows each: 128 x 256 595, 64 x 128 588; 64 rows each 648 / 714;
// dx of 8 rows each 459 / 479. Dense int8 2048 x 4096 x 4096 (256 tiles of 128 x 256): 45,
// 64 x 128 72; 1024 rows (128 tiles): 38 / 36, 64 x 64 42; 512 rows 34 / 24 / 23; 128 rows
// 33 / 15 / 11.
template <int OP, int T>
static hipError_t launch_tiles(const GroupedArgs& g, const Load& l, hipStream_t st) {
  const int nout = OP == kFwd ? g.N : g.K;
  const int64_t t128 = l.tiles(128) * blocks(nout, 256);
  if (l.rows >= (OP == kFwd ? 512 : 1024) && l.tiles(256) * blocks(nout, 256) >= 256)
    return launch_cfg<OP, T, 2, 4, 4, 2, OP == kFwd ? 16 : 32, OP == kFwd ? 128 : 64, OP == kFwd ? 2 : 4>(g, st);
  if (t128 >= 192 && (OP == kDx || l.rows >= 48)) return launch_cfg<OP, T, 1, 4, 4, 2, 32, 64, 3>(g, st);
  if (l.tiles(64) * blocks(nout, 128) >= 300) return launch_cfg<OP, T, 1, 4, 2, 1, 32, 128, 3>(g, st);
  return launch_cfg<OP, T, 2, 2, 1, 1, 32, 128, 4>(g, st);
}

template <int T>
static hipError_t forward(const GroupedArgs& g, hipStream_t st) {
  const Load l(g);
  const int64_t n16 = blocks(g.N, 16), row_kb = (int64_t)g.K * (T == kI8 ? 1 : 2);
  // Few rows: the weights stream. Dense int8 4096 x 4096, 1 row: 6.7 us, 64 x 64 tile 10.1; 512
  // experts in bf16, 8 rows: 13.3 / 12.8, 16 rows: two groups of weight rows 21.9, one 23.8, tile
  // 24.2; 64 rows 53.6 / 56.0 / 58.7. Past 16 rows each row tile reads the weights again, which
  // pays while that is little: dense int8 1001 x 1040, 128 rows: 4.8, tile 7.7; 2048 x 2048, 64
  // rows 6.7 / 7.8, 128 rows 9.5 / 8.1.
  if (l.rows <= 16 && g.P <= 64)
    return l.tiles(16) * n16 >= 1536 ? launch_stream<T, 1, 8, 2>(g, st) : launch_stream<T, 1, 8, 1>(g, st);
  if (l.tiles(32) * n16 * row_kb <= 640 * 1024) return launch_stream<T, 2, 4, 1>(g, st);
  return launch_tiles<kFwd, T>(g, l, st);
}

hipError_t launch_grouped_fwd(int type, const GroupedArgs& g, hipStream_t st) {
  if (g.P == 0) return hipSuccess;
  if (type == kBf16) return forward<kBf16>(g, st);
  if (type == kF16) return forward<kF16>(g, st);
  return forward<kI8>(g, st);
}

hipError_t launch_grouped_dx(int type, const GroupedArgs& g, hipStream_t st) {
  if (g.P == 0) return hipSuccess;
  if (type == kBf16) return launch_tiles<kDx, kBf16>(g, Load(g), st);
  return launch_tiles<kDx, kF16>(g, Load(g), st);
}

template <int T>
static hipError_t weight_gradient(const GroupedArgs& g, hipStream_t st) {
  // 256 x 256 while that fills the device: 64 experts of 1536 x 2048, 8192 tokens 472 us, 128 x 128
  // 526. Else 64 x 64, whose smaller tiles spread further (3 experts of 2048 x 256, 2667 rows each:
  // 31.4 us, 128 x 128 45.4; 13 of 520 x 392, 256 rows 12.4 / 14.0), unless 128 x 128 makes enough
  // tiles of many rows for its fewer reads to count (one of 1536 x 2048, 8192 rows 103 / 121).
  if (g.E * blocks(g.N, 256) * blocks(g.K, 256) >= 256) return launch_cfg<kDw, T, 2, 4, 4, 2, 32, 64, 4>(g, st);
  if (g.E * blocks(g.N, 128) * blocks(g.K, 128) >= 128 && g.P / g.E >= 1024)
    return launch_cfg<kDw, T, 2, 2, 2, 2, 32, 64, 3>(g, st);
  return launch_cfg<kDw, T, 2, 2, 1, 1, 32, 64, 4>(g, st);
}

hipError_t launch_grouped_dw(int type, const GroupedArgs& g, hipStream_t st) {
  return type == kBf16 ? weight_gradient<kBf16>(g, st) : weight_gradient<kF16>(g, st);
}

}  // namespace nvfp4
