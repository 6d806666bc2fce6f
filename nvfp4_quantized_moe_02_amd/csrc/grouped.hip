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
// contiguous in memory (x and w forward, dy in dx) is staged as LDS rows of 64 bytes of j;
// the others (w in dx, both in dw) as 32 rows of j, each a run of m or c, and read
// through the LDS transpose load. 64 bytes are 32 sixteen-bit or 64 eight-bit values: two
// matrix instructions of 32 x 32 outputs either way, with the same 16 bytes per lane.
#include "grouped.h"

namespace nvfp4 {

typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef short s16x8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));

constexpr int kFwd = 0, kDx = 1, kDw = 2;
constexpr int kBf16 = 0, kF16 = 1, kI8 = 2;
constexpr int JB = 64;        // bytes of the contraction dimension per K-block
constexpr int JR = 32;        // contraction rows per K-block of a transposed operand
constexpr int kIdxTile = 1024;  // rows of the gather table of dw

typedef __attribute__((address_space(3))) char* lds_char_t;

// 16 bytes per lane from src to the wave's LDS window at dst (wave-uniform) + 16 * lane.
// In asm because the compiler waits for every outstanding load before any LDS read that
// might alias the builtin's LDS write; the waits are wait_barrier's. The instruction
// writes no register.
__device__ __forceinline__ void dma16(const void* src, const char* dst) {
  const uint32_t m = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds_char_t)dst);
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(src), "s"(m) : "memory", "m0");
}

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

__device__ __forceinline__ int clampi(int v, int lo, int hi) { return v < lo ? lo : v > hi ? hi : v; }

// Row of x that sorted row r reads. A pair outside the tokens reads row 0 (in bounds).
__device__ __forceinline__ int src_row(const GroupedArgs& g, int r) {
  if (g.pairs == nullptr) return r;
  const int t = g.pairs[r] / g.topk;
  return (unsigned)t < (unsigned)g.xrows ? t : 0;
}

struct Tile {
  int e, m0, rows, base, nb;
};

// The expert and row tile of this block: row tiles of bm rows in expert order, the NB
// column blocks of a row tile one after the other. Each XCD (blockIdx % 8) takes a
// contiguous range, so the column blocks that share rows of x and the row tiles that share
// weights meet in one L2. Every block sums the tile counts itself from the offsets (one
// round trip and one block scan), so no launch before this one has to build a list.
// Offsets are clamped to [0, P]. Returns false for a block without a tile.
template <int THREADS>
__device__ __forceinline__ bool find_tile(const GroupedArgs& g, int bm, int NB, Tile& t) {
  __shared__ int s_tot[THREADS / 64];
  __shared__ int s_tile[3];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int bid = blockIdx.x;
  const int xcd = bid & 7, jj = bid >> 3;
  int mt;
  if (g.offsets == nullptr) {
    const int total = ((g.P + bm - 1) / bm) * NB, per = (total + 7) >> 3;
    const int L = xcd * per + jj;
    if (jj >= per || L >= total) return false;
    mt = L / NB;
    t = Tile{0, mt * bm, g.P - mt * bm < bm ? g.P - mt * bm : bm, 0, L - mt * NB};
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
  mt = (int)(L / NB);
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
  t.e = s_tile[0];
  t.base = s_tile[1];
  t.m0 = 0;
  t.rows = s_tile[2];
  t.nb = (int)(L - (long long)mt * NB);
  return t.rows > 0;  // 0: offsets that do not ascend, whose counts disagree
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
__device__ __forceinline__ typename Acc<T>::v32 mma32(i32x4_t a, i32x4_t b, typename Acc<T>::v32 c) {
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
__device__ __forceinline__ typename Acc<T>::v16 mma16(i32x4_t a, i32x4_t b, typename Acc<T>::v16 c) {
  if constexpr (T == kBf16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c,
                                                   0, 0, 0);
  else if constexpr (T == kF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b), c, 0,
                                                  0, 0);
  else
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
}

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

// ------------------------------------------------------------------ LDS images of a K-block
// Straight operand: rows of 64 bytes, 16-byte chunk c of row r in slot c ^ ((r >> 2) & 3):
// the 16 rows that an LDS read cycle serves then cover all 64 banks once.
__device__ __forceinline__ int straight_at(int row, int chunk) { return row * JB + ((chunk ^ ((row >> 2) & 3)) << 4); }

// Transposed operand: 32 contraction rows of W elements (2 W bytes). A transpose load
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

template <int OP, int T, int WM, int WN, int RB, int CB, int ST>
struct Cfg {
  static constexpr int BM = WM * RB * 32, BN = WN * CB * 32, THREADS = WM * WN * 64;
  static constexpr bool ATR = OP == kDw, BTR = OP != kFwd;
  static constexpr int ABYTES = BM * JB, BBYTES = BN * JB, STAGE = ABYTES + BBYTES;
  static constexpr int NLA = BM * 4 / THREADS, NLB = BN * 4 / THREADS;
  static_assert(BM * 4 % THREADS == 0 && BN * 4 % THREADS == 0, "whole loads per thread");
};

// The tile's K loop and epilogue for NRB occupied row blocks per wave (NRB < RB only when
// one wave row covers the tile).
template <int OP, int T, int WM, int WN, int RB, int CB, int ST, int NRB>
__device__ __forceinline__ void tile_product(const GroupedArgs& g, int e, int base, int mrows, int m0, int c0, int C,
                                             char* lds, int* s_src) {
  typedef Cfg<OP, T, WM, WN, RB, CB, ST> F;
  constexpr int ES = T == kI8 ? 1 : 2;
  constexpr int THREADS = F::THREADS;
  // loads of A: only the occupied row blocks when the rows are straight
  constexpr int NA = F::ATR ? F::NLA : (WM * NRB * 32 * 4 + THREADS - 1) / THREADS;
  constexpr int NBL = F::NLB;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave / WN, wn = wave % WN;
  const int half = lane >> 5, l32 = lane & 31;
  const int nout = OP == kFwd ? g.N : g.K;  // columns of C
  const int mlim = OP == kDw ? g.N : mrows;  // rows of C in this tile's range
  constexpr int JE = JB / ES;               // contraction elements per K-block
  const int nk = (C + JE - 1) / JE;
  const int tail = C - (nk - 1) * JE;       // elements of the last K-block

  // ---- where this thread's chunks come from
  const char* ap[NA];
  const char* bp[NBL];
  int arow[NA], brow[NBL], ach[NA], bch[NBL];
#pragma unroll
  for (int i = 0; i < NA; ++i) {
    const int ci = i * THREADS + tid;
    if constexpr (!F::ATR) {
      arow[i] = ci >> 2;
      ach[i] = ((ci & 3) ^ ((arow[i] >> 2) & 3));
      const int lda = OP == kFwd ? g.K : g.N;
      const int r = arow[i] < mrows ? arow[i] : mrows - 1;
      const size_t sr = OP == kFwd ? (size_t)s_src[r] : (size_t)(base + r);
      ap[i] = reinterpret_cast<const char*>(g.a) + sr * lda * ES;
    } else {
      typedef Trans<F::BM> X;
      arow[i] = ci / X::CPR;
      const int s = ci % X::CPR;
      const int ch = (((s >> 2) ^ X::key(arow[i])) << 2) | (s & 3);
      const int col = m0 + ch * 8 < g.N ? m0 + ch * 8 : 0;
      ach[i] = 0;
      ap[i] = reinterpret_cast<const char*>(g.a) + (size_t)col * 2;
    }
  }
#pragma unroll
  for (int i = 0; i < NBL; ++i) {
    const int ci = i * THREADS + tid;
    if constexpr (!F::BTR) {
      brow[i] = ci >> 2;
      bch[i] = ((ci & 3) ^ ((brow[i] >> 2) & 3));
      const int n = c0 + brow[i] < g.N ? c0 + brow[i] : g.N - 1;
      bp[i] = reinterpret_cast<const char*>(g.b) + ((size_t)e * g.N + n) * g.K * ES;
    } else {
      typedef Trans<F::BN> X;
      brow[i] = ci / X::CPR;
      const int s = ci % X::CPR;
      const int ch = (((s >> 2) ^ X::key(brow[i])) << 2) | (s & 3);
      const int col = c0 + ch * 8 < g.K ? c0 + ch * 8 : 0;
      bch[i] = 0;
      const size_t first = OP == kDx ? (size_t)e * g.N * g.K : 0;
      bp[i] = reinterpret_cast<const char*>(g.b) + (first + col) * 2;
    }
  }
  // K-block kb into stage s. Chunks and rows past the contraction's end read something in
  // bounds; zero_tail clears them in LDS.
  auto issue = [&](int kb, int s) {
    char* As = lds + s * F::STAGE;
    char* Bs = As + F::ABYTES;
    const bool last = kb == nk - 1;
    if (OP == kDw && g.pairs != nullptr && (kb % (kIdxTile / JR)) == 0) {
      // the next kIdxTile rows' source rows (kb is the same in every wave)
      lds_barrier();
      for (int r = tid; r < kIdxTile; r += THREADS) {
        const int j = kb * JR + r;
        s_src[r] = j < C ? src_row(g, base + j) : 0;
      }
      lds_barrier();
    }
#pragma unroll
    for (int i = 0; i < NA; ++i) {
      const char* p;
      if constexpr (!F::ATR) {
        const int off = kb * JB + ach[i] * 16;
        p = ap[i] + (last && off >= C * ES ? 0 : off);
      } else {
        const int j = kb * JR + arow[i];
        p = ap[i] + (size_t)(base + (j < C ? j : C - 1)) * g.N * 2;
      }
      dma16(p, As + (i * THREADS + wave * 64) * 16);
    }
#pragma unroll
    for (int i = 0; i < NBL; ++i) {
      const char* p;
      if constexpr (!F::BTR) {
        const int off = kb * JB + bch[i] * 16;
        p = bp[i] + (last && off >= C * ES ? 0 : off);
      } else {
        int j = kb * JR + brow[i];
        j = j < C ? j : C - 1;
        size_t r = j;
        if (OP == kDw) r = g.pairs != nullptr ? s_src[j % kIdxTile] : base + j;
        p = bp[i] + r * g.K * 2;
      }
      dma16(p, Bs + (i * THREADS + wave * 64) * 16);
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
  };
  // fragment of operand block `blk` (32 rows of m or c), K-step ks
  auto frag_straight = [&](const char* S, int row, int ks) -> i32x4_t {
    return *reinterpret_cast<const i32x4_t*>(S + straight_at(row, 2 * ks + half));
  };
  const int tr_row = 8 * half + ((lane & 15) >> 2);
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

  typename Acc<T>::v32 acc[NRB][CB];
#pragma unroll
  for (int rb = 0; rb < NRB; ++rb)
#pragma unroll
    for (int cb = 0; cb < CB; ++cb)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[rb][cb][i] = 0;

  constexpr int LPS = NA + NBL;  // loads per stage and thread
#pragma unroll
  for (int s = 0; s < ST - 1; ++s)
    if (s < nk) issue(s, s);
  int cur = 0;
  for (int kb = 0; kb < nk; ++kb) {
    // stage kb has arrived when at most the later stages' loads are outstanding
    if (kb + ST - 2 < nk)
      wait_barrier<LPS*(ST - 2)>();
    else
      wait_barrier<0>();
    const int nxt = cur == 0 ? ST - 1 : cur - 1;  // (kb + ST - 1) % ST
    if (kb + ST - 1 < nk) issue(kb + ST - 1, nxt);
    if (kb == nk - 1 && tail < JE) {
      zero_tail(cur);
      lds_barrier();
    }
    const char* As = lds + cur * F::STAGE;
    const char* Bs = As + F::ABYTES;
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      i32x4_t bf[CB];
#pragma unroll
      for (int cb = 0; cb < CB; ++cb) {
        if constexpr (F::BTR)
          bf[cb] = frag_trans(Bs, Trans<F::BN>{}, wn * CB + cb, ks);
        else
          bf[cb] = frag_straight(Bs, (wn * CB + cb) * 32 + l32, ks);
      }
#pragma unroll
      for (int rb = 0; rb < NRB; ++rb) {
        i32x4_t af;
        if constexpr (F::ATR)
          af = frag_trans(As, Trans<F::BM>{}, wm * RB + rb, ks);
        else
          af = frag_straight(As, (wm * RB + rb) * 32 + l32, ks);
        // columns first: a lane ends with 4 x 4 adjacent columns of one row
#pragma unroll
        for (int cb = 0; cb < CB; ++cb) acc[rb][cb] = mma32<T>(bf[cb], af, acc[rb][cb]);
      }
    }
    cur = cur + 1 == ST ? 0 : cur + 1;
  }

  // Accumulator element i of lane (half, l32): row l32 of the row block, column
  // 8 (i / 4) + 4 half + i % 4 of the column block.
  const bool vec = (nout & 3) == 0;
#pragma unroll
  for (int rb = 0; rb < NRB; ++rb) {
    const int m = (wm * RB + rb) * 32 + l32;
    const int row = OP == kDw ? m0 + m : m;
    if (row >= mlim) continue;
    const size_t at = (OP == kDw ? (size_t)e * g.N + row : (size_t)(base + row)) * nout;
    float rs = 1.f;
    if constexpr (T == kI8) rs = g.a_scale[s_src[row]];
#pragma unroll
    for (int cb = 0; cb < CB; ++cb)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int col = c0 + (wn * CB + cb) * 32 + 8 * q + 4 * half;
        float v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v[j] = (float)acc[rb][cb][4 * q + j];
          if constexpr (T == kI8) v[j] = v[j] * rs * (col + j < nout ? g.b_scale[(size_t)e * g.N + col + j] : 0.f);
        }
        store4(g.out, g.out_dtype, at + col, v, nout - col, vec);
      }
  }
}

template <int OP, int T, int WM, int WN, int RB, int CB, int ST>
__global__ __launch_bounds__(WM* WN * 64, 2) void grouped_kernel(GroupedArgs g, int NB) {
  typedef Cfg<OP, T, WM, WN, RB, CB, ST> F;
  __shared__ __attribute__((aligned(256))) char lds[ST * F::STAGE];
  __shared__ int s_src[OP == kDw ? kIdxTile : F::BM];
  if constexpr (OP == kDw) {
    // blocks of (expert, BM rows n, BN columns k); an XCD takes a contiguous range
    const int NM = (g.N + F::BM - 1) / F::BM;
    const long long total = (long long)g.E * NM * NB, per = (total + 7) >> 3;
    const long long L = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
    if ((long long)(blockIdx.x >> 3) >= per || L >= total) return;
    const int e = (int)(L / (NM * NB)), rest = (int)(L - (long long)e * NM * NB);
    const int mb = rest / NB, nb = rest - mb * NB;
    const int lo = clampi(g.offsets[e], 0, g.P), hi = clampi(g.offsets[e + 1], lo, g.P);
    // an expert without rows has a zero gradient: no K-block, the cleared accumulator is stored
    tile_product<OP, T, WM, WN, RB, CB, ST, RB>(g, e, lo, 0, mb * F::BM, nb * F::BN, hi - lo, lds, s_src);
  } else {
    Tile t;
    if (!find_tile<F::THREADS>(g, F::BM, NB, t)) return;
    const int base = t.base + t.m0;
    if constexpr (OP == kFwd) {
      for (int r = threadIdx.x; r < F::BM; r += F::THREADS)
        s_src[r] = src_row(g, base + (r < t.rows ? r : t.rows - 1));
      __syncthreads();
    }
    const int c0 = t.nb * F::BN, C = OP == kFwd ? g.K : g.N;
    if constexpr (WM == 1 && RB == 4) {
      const int nrb = (t.rows + 31) >> 5;
      if (nrb == 4)
        tile_product<OP, T, WM, WN, RB, CB, ST, 4>(g, t.e, base, t.rows, 0, c0, C, lds, s_src);
      else if (nrb == 3)
        tile_product<OP, T, WM, WN, RB, CB, ST, 3>(g, t.e, base, t.rows, 0, c0, C, lds, s_src);
      else if (nrb == 2)
        tile_product<OP, T, WM, WN, RB, CB, ST, 2>(g, t.e, base, t.rows, 0, c0, C, lds, s_src);
      else
        tile_product<OP, T, WM, WN, RB, CB, ST, 1>(g, t.e, base, t.rows, 0, c0, C, lds, s_src);
    } else {
      tile_product<OP, T, WM, WN, RB, CB, ST, RB>(g, t.e, base, t.rows, 0, c0, C, lds, s_src);
    }
  }
}

// Blocks for the most row tiles that P rows in E experts can make.
static unsigned grid_rows(const GroupedArgs& g, int bm, int NB) {
  const long long e = g.offsets == nullptr ? 1 : (g.E < g.P ? g.E : g.P);
  const long long tiles = g.offsets == nullptr ? ((long long)g.P + bm - 1) / bm : g.P / bm + e;
  return (unsigned)((tiles * NB + 7) / 8 * 8);
}

template <int OP, int T, int WM, int WN, int RB, int CB, int ST>
static hipError_t launch_cfg(const GroupedArgs& g, hipStream_t st) {
  typedef Cfg<OP, T, WM, WN, RB, CB, ST> F;
  const int nout = OP == kFwd ? g.N : g.K;
  const int NB = (nout + F::BN - 1) / F::BN;
  unsigned grid;
  if (OP == kDw)
    grid = (unsigned)(((long long)g.E * ((g.N + F::BM - 1) / F::BM) * NB + 7) / 8 * 8);
  else
    grid = grid_rows(g, F::BM, NB);
  grouped_kernel<OP, T, WM, WN, RB, CB, ST><<<grid, F::THREADS, 0, st>>>(g, NB);
  return hipGetLastError();
}

hipError_t launch_grouped_fwd(int type, const GroupedArgs& g, hipStream_t st) {
  if (g.P == 0) return hipSuccess;
  if (type == kBf16) return launch_cfg<kFwd, kBf16, 1, 4, 4, 2, 3>(g, st);
  if (type == kF16) return launch_cfg<kFwd, kF16, 1, 4, 4, 2, 3>(g, st);
  return launch_cfg<kFwd, kI8, 1, 4, 4, 2, 3>(g, st);
}

hipError_t launch_grouped_dx(int type, const GroupedArgs& g, hipStream_t st) {
  if (g.P == 0) return hipSuccess;
  if (type == kBf16) return launch_cfg<kDx, kBf16, 1, 4, 4, 2, 3>(g, st);
  return launch_cfg<kDx, kF16, 1, 4, 4, 2, 3>(g, st);
}

hipError_t launch_grouped_dw(int type, const GroupedArgs& g, hipStream_t st) {
  if (type == kBf16) return launch_cfg<kDw, kBf16, 1, 4, 4, 2, 3>(g, st);
  return launch_cfg<kDw, kF16, 1, 4, 4, 2, 3>(g, st);
}

}  // namespace nvfp4
