// qb_gemm16.hpp -- the tiled product of 16-bit operands with sums in 32 bits:
//
//   out[m][n] = sum_k A(m, k) B(n, k)
//
// Each operand lies with its summed index contiguous (KC: A[m][k]) or strided
// (KS: A[k][m]), so that the forward product, the rows' gradient and the
// matrices' gradient of an expert read the same arrays and nothing is
// transposed in memory.  A stage is 64 of K: 128 bytes of each row of a KC
// operand, 64 rows of a KS one, brought to an LDS ring by loads that go there
// directly.  Lanes of the matrix instruction (v_mfma_f32_16x16x32) hold 8
// consecutive K of row l % 16; a KC operand gives them as 16 bytes, a KS one
// as two transposing reads (ds_read_b64_tr_b16: 16 lanes read 4 rows of 16
// columns and each gets a column).
//
// LDS banks.  A KC row's 128 bytes are 8 slots of 16, XORed with a number of
// the row's, so that the 16 rows that a quarter wave reads in one slot lie in
// all banks once.  A KS row is slots of 32 bytes (16 columns), XORed with a
// number made of the bits of k in which the 8 rows that half a wave reads
// differ (0..3 and 8..11): those 8 slots lie in all banks once.
//
// What lies outside an operand (K past its end, columns past a KS operand's,
// rows that were routed nowhere) is read from 16 bytes of zeros, both
// operands' alike, so nothing that a caller keeps behind its rows is
// multiplied.
#pragma once

#include <algorithm>
#include <type_traits>

#include "qb_tiles.hpp"

namespace qbk {

typedef short v4s __attribute__((ext_vector_type(4)));
typedef short v8s __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) v4s* lds_v4s;

static __device__ const uint4 kZero16 = {0, 0, 0, 0};

// What is computed:
//   kRows   out bf16 [M][N]: an expert's rows (off) times its matrix; A's rows by number (src)
//   kGrad   out float [G][M][N]: K runs over an expert's rows (off, src: B's rows by number)
//   kSym    S = A A^T, kSqr  P = b S + c S S, kStep  X' = a X + P X: the steps of qb_orthogonalize (batches of G)
enum GemmKind { kRows, kGrad, kSym, kSqr, kStep };

struct Gemm16 {
  const uint16_t *A, *B;
  int64_t lda, ldb;          // values between rows
  int64_t mat_a, mat_b;      // values between the matrices of a batch (kRows: between B's)
  int M, N, K;               // rows and columns of a result, summed length (kGrad: all rows)
  const int32_t* src;        // nullable
  int Mx;                    // rows of the operand that src numbers
  const int32_t* off;        // nullable: one matrix
  int G;
  int tiles, splits;         // kGrad: each expert's K in so many parts
  void* out;
  // the orthogonalising steps: two 16-bit parts of a value, `part` values apart
  int64_t part_a, part_b, mat_out, ldo, part_out;
  const uint16_t* add;       // what the result is added to (kSqr: S, kStep: X), in out's layout
  float by_sum, by_add;      // out = by_sum * sum + by_add * add
  // 4-bit operands: exponent bytes, 8 for each 128 bytes of a row (mat_bs: between B's matrices)
  const uint8_t *As, *Bs;
  int64_t sld, mat_bs;
  uint16_t* last;            // kStep: the final result, bf16 [G][M][N], instead of out
  float by_last;
};

// 4-bit values (e2m1), two a byte, with a power of two for each 32 of them:
// qb_fp4.hip.  A row's 128 bytes a stage are 256 values and 8 exponents.
struct Fp4 {};

template <class T>
__device__ __forceinline__ v4f mma16(v8s a, v8s b, v4f c) {
  if constexpr (std::is_same_v<T, _Float16>)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0,
                                                   0);
}

// The 128 4-bit products of a pair of rows, each lane's 32 with the exponents in
// byte `half` of its words.  Sums are held in 32 bits: measured with single
// values in all four lanes of a row, nothing within 2^-23 of the largest is lost.
__device__ __forceinline__ v4f mma4(v8s a, v8s b, v4f c, int as, int bs, int half) {
  const v4i x = __builtin_bit_cast(v4i, a), y = __builtin_bit_cast(v4i, b);
  const v8i u = __builtin_shufflevector(x, x, 0, 1, 2, 3, -1, -1, -1, -1);
  const v8i v = __builtin_shufflevector(y, y, 0, 1, 2, 3, -1, -1, -1, -1);
  return half == 0 ? __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(u, v, c, 4, 4, 0, as, 0, bs)
                   : __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(u, v, c, 4, 4, 1, as, 1, bs);
}

// A value in two fp16 parts: the nearest, and the nearest to what is left.
__device__ __forceinline__ void split16(float v, uint16_t& hi, uint16_t& lo) {
  const _Float16 h = _Float16(v);
  hi = __builtin_bit_cast(uint16_t, h);
  lo = __builtin_bit_cast(uint16_t, _Float16(v - float(h)));
}
__device__ __forceinline__ float joined16(uint16_t hi, uint16_t lo) {
  return float(__builtin_bit_cast(_Float16, hi)) + float(__builtin_bit_cast(_Float16, lo));
}

// 8 values from p of which n lie inside the operand, the others zero.
__device__ __forceinline__ uint4 ld_inside(const uint16_t* p, int n) {
  if (n >= 8) {
    typedef uint32_t half8 __attribute__((ext_vector_type(4), aligned(2)));
    const half8 t = *reinterpret_cast<const half8*>(p);
    return make_uint4(t[0], t[1], t[2], t[3]);
  }
  uint32_t v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = 2 * i < n ? p[2 * i] : 0, hi = 2 * i + 1 < n ? p[2 * i + 1] : 0;
    v[i] = lo | (hi << 16);
  }
  return make_uint4(v[0], v[1], v[2], v[3]);
}

// 16 bytes a lane from memory to the 1 KiB of LDS at `to` (the wave's).  The
// compiler waits for every load that it knows to go to LDS before it reads
// LDS by a transposing read, whatever the addresses; of these it does not know,
// and the kernel's own waits order them (an operand lands a stage before it is
// read).  There is no result register, so nothing is reused too early, and m0
// has no other use in a kernel that calls this.
__device__ __forceinline__ void load_to_lds(const void* from, uint8_t* to) {
  const uint32_t at = uint32_t(uintptr_t((__attribute__((address_space(3))) uint8_t*)to));
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(at), "v"(from) : "memory");
}

// BM x BN tiles, waves WM x WN, a ring of S stages.  DIRECT: rows are multiples
// of 16 bytes, and the loads go to LDS; else they pass through registers, 2
// bytes being the only alignment asked for.  PA, PB: which part of each operand
// each of PARTS passes over K multiplies, a bit a pass.
template <class T, int KIND, bool A_KS, bool B_KS, int BM, int BN, int WM, int WN, int S, bool DIRECT, int PARTS = 1,
          int PA = 0, int PB = 0>
__global__ __launch_bounds__(WM* WN* kWave, 2) void k_gemm16(const Gemm16 g) {
  constexpr int W = WM * WN, TM = BM / WM / 16, TN = BN / WN / 16;
  constexpr int KT = 64;  // of K a stage
  constexpr int A_BYTES = BM * KT * 2, B_BYTES = BN * KT * 2;
  constexpr int A_PW = A_BYTES / 1024 / W, B_PW = B_BYTES / 1024 / W;  // 1 KiB loads a wave and stage
  constexpr bool FOUR = std::is_same_v<T, Fp4>;
  constexpr int ROWS = BM + BN, S_PW = FOUR ? (ROWS / 32 + W - 1) / W : 0;  // loads of 32 rows' 8 exponents a wave
  constexpr int S_BYTES = FOUR ? ROWS * 8 : 0;
  constexpr bool RAGGED = KIND == kRows || KIND == kGrad, SYM = KIND == kSym || KIND == kSqr;
  constexpr bool WIDE = KIND == kRows && !B_KS;
  constexpr int JT = TN < 4 ? TN : 4;  // WIDE: column tiles that share a stretch of 16 JT columns
  static_assert(A_PW * W * 1024 == A_BYTES && B_PW * W * 1024 == B_BYTES, "tile split");
  static_assert(TN % JT == 0 && JT >= 2 && (!SYM || BM == BN) && (KIND != kGrad || BM == BN), "tile shape");
  // a row's number in the swizzle of its slots
  auto key_a = [](int row) { return (row >> 1) & 7; };
  auto key_b = [](int row) { return WIDE ? ((row >> 1) & 1) | ((row >> (JT == 4 ? 3 : 2)) & 6) : (row >> 1) & 7; };
  auto key_k = [](int k, int bx) {
    return bx >= 128 ? (k & 3) | ((k >> 1) & 4) : ((k >> 1) & 1) | ((k >> 2) & 2);
  };
  __shared__ __align__(1024) uint8_t lds[S * (A_BYTES + B_BYTES + S_BYTES) + (RAGGED ? 1024 * 3 + 16 : 16)];
  uint8_t* const lds_b = lds + S * A_BYTES;
  uint8_t* const lds_s = lds + S * (A_BYTES + B_BYTES);
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int tn_all = (g.N + BN - 1) / BN, tm_all = (g.M + BM - 1) / BM;
  int tiles = g.tiles;

  // the experts' first and last rows and their tiles of rows before each
  int* const first_of = reinterpret_cast<int*>(lds + S * (A_BYTES + B_BYTES + S_BYTES));
  int *const end_of = first_of + 256, *const before_of = end_of + 256;  // 256, 256 and 257 of them
  if (RAGGED && g.off) {
    if (wave == 0) {
      int lo[4], hi[4], n[4], before;
      const int total = group_tiles(g.off, g.G, KIND == kGrad ? g.K : g.M, BM, lane, lo, hi, n, before);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        first_of[4 * lane + j] = lo[j];
        end_of[4 * lane + j] = hi[j];
        before_of[4 * lane + j] = before;
        before += n[j];
      }
      if (lane == 0) before_of[256] = total;
    }
    __syncthreads();
    // (offsets out of order could make more than there are)
    if constexpr (KIND == kRows) tiles = (before_of[256] < tiles / tn_all ? before_of[256] : tiles / tn_all) * tn_all;
  }

  // A tile: rows m0 .. m_end - 1 and columns from n0 of a result; K from k0 to
  // k1; e: its matrix, and for kGrad the part of K.
  struct Place {
    int m0, m_end, n0, k0, k1, e, part;
  };
  auto place = [&](int t) {
    Place p{0, g.M, 0, 0, g.K, 0, 0};
    int tm, tn;
    if constexpr (KIND == kGrad) {
      const int per = tm_all * tn_all;
      p.part = t / (per * g.G);
      t -= p.part * per * g.G;
      p.e = t / per;
      tile_order(t % per, tm_all, tn_all, 8, tm, tn);
      if (g.off) {
        p.k0 = __builtin_amdgcn_readfirstlane(first_of[p.e]);
        p.k1 = __builtin_amdgcn_readfirstlane(end_of[p.e]);
      }
      if (g.splits > 1) {
        const int stages = (p.k1 - p.k0 + KT - 1) / KT, each = (stages + g.splits - 1) / g.splits;
        p.k0 += std::min(p.part * each, stages) * KT;
        p.k1 = std::min(p.k1, p.k0 + each * KT);
      }
      p.m0 = tm * BM;
    } else if constexpr (KIND == kRows) {
      if (g.off) {
        tile_order(t, tiles / tn_all, tn_all, 8, tm, tn);
        // the expert whose tiles hold tm: the last of those that begin at or before it
        int begun = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) begun += __popcll(__ballot(before_of[4 * lane + j] <= tm));
        p.e = begun > 0 ? begun - 1 : 0;
        p.m0 = __builtin_amdgcn_readfirstlane(first_of[p.e] + (tm - before_of[p.e]) * BM);
        p.m_end = __builtin_amdgcn_readfirstlane(end_of[p.e]);
      } else {
        tile_order(t, tm_all, tn_all, 8, tm, tn);
        p.m0 = tm * BM;
      }
    } else if constexpr (SYM) {
      // tiles on and below the diagonal, row by row
      const int per = tm_all * (tm_all + 1) / 2;
      p.e = t / per;
      t %= per;
      tm = int((__builtin_sqrtf(8.f * float(t) + 1.f) - 1.f) * 0.5f);
      while ((tm + 1) * (tm + 2) / 2 <= t) ++tm;
      while (tm * (tm + 1) / 2 > t) --tm;
      tn = t - tm * (tm + 1) / 2;
      p.m0 = tm * BM;
    } else {
      const int per = tm_all * tn_all;
      p.e = t / per;
      tile_order(t % per, tm_all, tn_all, 8, tm, tn);
      p.m0 = tm * BM;
    }
    p.n0 = tn * BN;
    return p;
  };
  auto stages_of = [&](const Place& p) {
    return KIND == kGrad ? (p.k1 - p.k0 + KT - 1) / KT : (g.K + KT - 1) / KT * PARTS;
  };

  // The tile whose loads are issued next, the stage of it, and the numbers of
  // the rows that this lane loads for it.
  Place lp{};
  int ls = 0, ln = 0, lat = int(blockIdx.x);
  bool more = false;
  constexpr int A_ROWS = A_KS ? 1 : A_PW;
  int a_row[A_ROWS], k_row[B_PW];
  // lane's part in load u: of a KC operand row r and slot q, of a KS one row k and 8 columns from c
  auto kc_r = [&](int u, int pw) { return ((wave * pw + u) * kWave + lane) >> 3; };
  auto ks_k = [&](int u, int pw, int bx) { return ((wave * pw + u) * kWave + lane) / (bx / 8); };
  auto ks_c = [&](int u, int pw, int bx) {
    const int s = ((wave * pw + u) * kWave + lane) % (bx / 8);
    return (((s >> 1) ^ key_k(ks_k(u, pw, bx), bx)) * 2 + (s & 1)) * 8;
  };
  auto load_rows = [&]() {  // of stage ls
    if constexpr (!A_KS) {
      if (ls == 0) {
#pragma unroll
        for (int u = 0; u < A_PW; ++u) {
          const int r = kc_r(u, A_PW), row = lp.m0 + r < lp.m_end ? lp.m0 + r : lp.m_end - 1;
          a_row[u] = row;
        }
        if (KIND == kRows && !FOUR && g.src) {
#pragma unroll
          for (int u = 0; u < A_PW; ++u) a_row[u] = g.src[a_row[u]];
          // waited for here, once a tile, and not before the loads of every stage
#pragma unroll
          for (int u = 0; u < A_PW; ++u) asm volatile("" : "+v"(a_row[u]));
        }
      }
    }
    if constexpr (KIND == kGrad) {
#pragma unroll
      for (int u = 0; u < B_PW; ++u) {
        const int row = lp.k0 + ls * KT + ks_k(u, B_PW, BN);
        k_row[u] = row < lp.k1 ? row : lp.k1 - 1;
      }
      if (g.src) {
#pragma unroll
        for (int u = 0; u < B_PW; ++u) k_row[u] = g.src[k_row[u]];
      }
    }
  };
  // The next tile that has something to multiply; of the others (experts
  // without rows) the gradient is written as zeros.
  auto advance = [&]() {
    more = false;
    for (; lat < tiles; lat += int(gridDim.x)) {
      const bool in_turn = KIND == kGrad && gridDim.x % 8 == 0;
      lp = place(in_turn ? tile_in_turn<BM == 256 ? 16 : 8>(lat, tiles) : tile_at(lat, int(gridDim.x), tiles));
      ln = stages_of(lp);
      if (ln > 0) {
        more = true;
        lat += int(gridDim.x);
        break;
      }
      if constexpr (KIND == kGrad)
        zero_tile<BM, BN, W>(static_cast<float*>(g.out), (int64_t(lp.part) * g.G + lp.e) * g.M, lp.m0, g.M, lp.n0, g.N,
                             tid);
    }
    ls = 0;
    if (more) load_rows();
  };

  // Where load u of the stage lies, and how many of its 8 values are inside.
  auto a_at = [&](int u, int& n) -> const uint16_t* {
    const uint16_t* base = g.A;
    if constexpr (!RAGGED) base += int64_t(lp.e) * g.mat_a;
    int k = ls * KT;
    if constexpr (PARTS > 1) {
      const int each = (g.K + KT - 1) / KT, p = ls / each;
      k = (ls - p * each) * KT;
      base += ((PA >> p) & 1) * g.part_a;
    }
    if constexpr (A_KS) {
      const int kr = ks_k(u, A_PW, BM), c = lp.m0 + ks_c(u, A_PW, BM);
      const int row = KIND == kGrad ? lp.k0 + k + kr : k + kr;
      bool in = row < (KIND == kGrad ? lp.k1 : g.K);
      if constexpr (KIND == kGrad) in = in && (!g.src || uint32_t(k_row[u < B_PW ? u : 0]) < uint32_t(g.Mx));
      n = in ? g.M - c : 0;
      return base + int64_t(uint64_t(uint32_t(row)) * uint32_t(g.lda)) + c;
    } else {
      const int r = kc_r(u, A_PW), q = (lane & 7) ^ key_a(r), row = a_row[u < A_ROWS ? u : 0];
      const bool in = KIND != kRows || FOUR || !g.src || uint32_t(row) < uint32_t(g.Mx);
      k += q * 8;
      n = in ? g.K - k : 0;
      return base + int64_t(uint64_t(uint32_t(row)) * uint32_t(g.lda)) + k;
    }
  };
  auto b_at = [&](int u, int& n) -> const uint16_t* {
    const uint16_t* base = g.B;
    if constexpr (KIND != kGrad) base += int64_t(lp.e) * g.mat_b;
    int k = ls * KT;
    if constexpr (PARTS > 1) {
      const int each = (g.K + KT - 1) / KT, p = ls / each;
      k = (ls - p * each) * KT;
      base += ((PB >> p) & 1) * g.part_b;
    }
    if constexpr (B_KS) {
      const int kr = ks_k(u, B_PW, BN), c = lp.n0 + ks_c(u, B_PW, BN);
      const int row = KIND == kGrad ? k_row[u] : k + kr;
      const bool in = KIND == kGrad ? lp.k0 + k + kr < lp.k1 && (!g.src || uint32_t(row) < uint32_t(g.Mx)) : row < g.K;
      n = in ? g.N - c : 0;
      return base + int64_t(uint64_t(uint32_t(row)) * uint32_t(g.ldb)) + c;
    } else {
      const int r = kc_r(u, B_PW), q = (lane & 7) ^ key_b(r);
      const int row = lp.n0 + r < g.N ? lp.n0 + r : g.N - 1;
      k += q * 8;
      n = g.K - k;
      return base + int64_t(uint64_t(uint32_t(row)) * uint32_t(g.ldb)) + k;
    }
  };
  constexpr int LOADS = A_PW + B_PW;
  auto at = [&](int u, int& n) { return u < A_PW ? a_at(u < A_PW ? u : 0, n) : b_at(u < A_PW ? 0 : u - A_PW, n); };
  auto slot = [&](int u, int st) {
    return u < A_PW ? lds + st * A_BYTES + (wave * A_PW + u) * 1024 : lds_b + st * B_BYTES + (wave * B_PW + u - A_PW) * 1024;
  };
  uint4 held[DIRECT ? 1 : LOADS];
  auto next_stage = [&]() {
    if (++ls < ln)
      load_rows();
    else
      advance();
  };
  auto issue = [&](int st) {
#pragma unroll
    for (int u = 0; u < LOADS; ++u) {
      int n;
      const uint16_t* p = at(u, n);
      if constexpr (DIRECT) {
        const uint8_t* q = n > 0 ? reinterpret_cast<const uint8_t*>(p) : reinterpret_cast<const uint8_t*>(&kZero16);
        if constexpr (A_KS || B_KS)
          load_to_lds(q, slot(u, st));
        else
          __builtin_amdgcn_global_load_lds((glb_vptr)q, (lds_vptr)slot(u, st), 16, 0, 0);
      } else {
        held[u] = ld_inside(p, n);
      }
    }
    if constexpr (FOUR) {
#pragma unroll
      for (int j = 0; j < S_PW; ++j) {
        const int first = (wave * S_PW + j) % (ROWS / 32) * 32, r = first + (lane >> 1);
        const uint8_t* p;
        if (first < BM) {
          const int row = lp.m0 + r < lp.m_end ? lp.m0 + r : lp.m_end - 1;
          p = g.As + int64_t(row) * g.sld;
        } else {
          const int row = lp.n0 + r - BM < g.N ? lp.n0 + r - BM : g.N - 1;
          p = g.Bs + int64_t(lp.e) * g.mat_bs + int64_t(row) * g.sld;
        }
        __builtin_amdgcn_global_load_lds((glb_vptr)(p + ls * 8 + (lane & 1) * 4),
                                         (lds_vptr)(lds_s + st * S_BYTES + first * 8), 4, 0, 0);
      }
    }
    next_stage();
  };
  auto put = [&](int st) {  // !DIRECT: what issue() read
    if constexpr (!DIRECT) {
#pragma unroll
      for (int u = 0; u < LOADS; ++u) *reinterpret_cast<uint4*>(slot(u, st) + lane * 16) = held[u];
    }
  };

  v4f acc[TM][TN];
  const int r = lane & 15, g4 = lane >> 4;
  // (4 bits: a lane's two halves are side by side, so that their exponents are)
  constexpr int HALF = FOUR ? 16 : 64;
  const int s4 = FOUR ? 2 * g4 : g4;
  const int frag_a = A_KS ? (8 * g4 + (r >> 2)) * (BM * 2) + (((wm * TM) ^ key_k(8 * g4 + (r >> 2), BM)) * 32) + (r & 3) * 8
                          : (wm * TM * 16 + r) * 128 + ((s4 ^ key_a(r)) * 16);
  const int br = WIDE ? (r >> 2) * (4 * JT) + (r & 3) : r;  // KC: its row of column tile 0, and what tile j adds
  auto b_row = [](int j) { return WIDE ? j / JT * (16 * JT) + j % JT * 4 : j * 16; };
  auto frag_b = [&](int j) {
    if constexpr (B_KS) {
      return ((8 * g4 + (r >> 2)) * (BN * 2) + (((wn * TN) ^ key_k(8 * g4 + (r >> 2), BN)) * 32) + (r & 3) * 8) ^ (j * 32);
    } else {
      const int row = br + b_row(j);
      return (wn * TN * 16 + row) * 128 + ((s4 ^ key_b(row)) * 16);
    }
  };
  // half h of the stage's K: 8 values of the lane's row or column
  auto read_ks = [&](const uint8_t* p, int pitch, int h) {
    const auto q = (__attribute__((address_space(3))) uint8_t*)p;
    const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s)(q + (32 * h) * pitch));
    const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s)(q + (32 * h + 4) * pitch));
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  };
  auto read_a = [&](int st, int i, int h) -> v8s {
    const uint8_t* p = lds + st * A_BYTES;
    if constexpr (A_KS)
      return read_ks(p + (frag_a ^ (i * 32)), BM * 2, h);
    else
      return *reinterpret_cast<const v8s*>(p + i * 16 * 128 + (frag_a ^ (h * HALF)));
  };
  auto read_b = [&](int st, int j, int h) -> v8s {
    const uint8_t* p = lds_b + st * B_BYTES;
    if constexpr (B_KS)
      return read_ks(p + frag_b(j), BN * 2, h);
    else
      return *reinterpret_cast<const v8s*>(p + (frag_b(j) ^ (h * HALF)));
  };
  // stage st's products, while the next loads go to stage `into` after the first row tile's
  auto multiply = [&](int st, bool load, int into) {
    int as[FOUR ? TM : 1], bs[FOUR ? TN : 1];  // two exponents each, one a half
    if constexpr (FOUR) {
      const uint8_t* ss = lds_s + st * S_BYTES + g4 * 2;
#pragma unroll
      for (int i = 0; i < TM; ++i) as[i] = *reinterpret_cast<const uint16_t*>(ss + ((wm * TM + i) * 16 + r) * 8);
#pragma unroll
      for (int j = 0; j < TN; ++j)
        bs[j] = *reinterpret_cast<const uint16_t*>(ss + (BM + wn * TN * 16 + br + b_row(j)) * 8);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      v8s b[TN], a[2];
#pragma unroll
      for (int j = 0; j < TN; ++j) b[j] = read_b(st, j, h);
      a[0] = read_a(st, 0, h);
#pragma unroll
      for (int i = 0; i < TM; ++i) {
        if (i + 1 < TM) a[(i + 1) & 1] = read_a(st, i + 1, h);
#pragma unroll
        for (int j = 0; j < TN; ++j) {
          if constexpr (FOUR)
            acc[i][j] = mma4(b[j], a[i & 1], acc[i][j], bs[j], as[i], h);
          else
            acc[i][j] = mma16<T>(b[j], a[i & 1], acc[i][j]);
        }
        if (h == 0 && i == 0 && load) issue(into);
      }
    }
  };

  // element c of acc[i][j]: row 16 i + r, column 16 j + 4 g4 + c (WIDE: 4 JT g4 + 4 j + c of its JT column tiles)
  constexpr int STORES = TM * (WIDE ? TN / 2 : TN);
  auto store_some = [&](const Place& p, auto whole) {
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      const int row = p.m0 + (wm * TM + i) * 16 + r;
      if constexpr (KIND == kGrad) {
        if (!whole() && row >= p.m_end) continue;
        float* o = static_cast<float*>(g.out) + ((int64_t(p.part) * g.G + p.e) * g.M + row) * g.N;
#pragma unroll
        for (int j = 0; j < TN; ++j) {
          const int col = p.n0 + (wn * TN + j) * 16 + g4 * 4;
          const v4f v = acc[i][j];
          if (whole() || col + 3 < g.N) {
            Float4 t;
#pragma unroll
            for (int c = 0; c < 4; ++c) t.v[c] = v[c];
            *reinterpret_cast<Float4*>(o + col) = t;
          } else {
#pragma unroll
            for (int c = 0; c < 4; ++c)
              if (col + c < g.N) o[col + c] = v[c];
          }
        }
      } else if constexpr (KIND == kRows) {
        if (!whole() && row >= p.m_end) continue;
        uint16_t* o = static_cast<uint16_t*>(g.out) + int64_t(row) * g.N;
        if constexpr (WIDE) {
#pragma unroll
          for (int h = 0; h < TN / 2; ++h) {  // 8 columns each
            const int col = p.n0 + (wn * TN + 2 * h / JT * JT) * 16 + g4 * (4 * JT) + 8 * (h % (JT / 2));
            Half8 t;
#pragma unroll
            for (int k = 0; k < 4; ++k)
              t.v[k] = bf16x2_rne(acc[i][2 * h + k / 2][2 * (k & 1)], acc[i][2 * h + k / 2][2 * (k & 1) + 1]);
            if (whole() || col + 7 < g.N) {
              *reinterpret_cast<Half8*>(o + col) = t;
            } else {
#pragma unroll
              for (int c = 0; c < 8; ++c)
                if (col + c < g.N) o[col + c] = uint16_t(t.v[c >> 1] >> (16 * (c & 1)));
            }
          }
        } else {
#pragma unroll
          for (int j = 0; j < TN; ++j) {
            const int col = p.n0 + (wn * TN + j) * 16 + g4 * 4;
            Half4 t;
            t.v[0] = bf16x2_rne(acc[i][j][0], acc[i][j][1]);
            t.v[1] = bf16x2_rne(acc[i][j][2], acc[i][j][3]);
            if (whole() || col + 3 < g.N) {
              *reinterpret_cast<Half4*>(o + col) = t;
            } else {
#pragma unroll
              for (int c = 0; c < 4; ++c)
                if (col + c < g.N) o[col + c] = uint16_t(t.v[c >> 1] >> (16 * (c & 1)));
            }
          }
        }
      } else {
        // rows of ldo values, a multiple of 8, of which those past N are kept zero
#pragma unroll
        for (int j = 0; j < TN; ++j) {
          const int col = p.n0 + (wn * TN + j) * 16 + g4 * 4;
          const int64_t at0 = int64_t(p.e) * g.mat_out + int64_t(row) * g.ldo + col;
          const bool here = row < g.M && col < g.ldo;
          float v[4];
          uint16_t hi[4], lo[4];
          uint2 ah = make_uint2(0, 0), al = make_uint2(0, 0);
          if (KIND != kSym && here) {
            ah = *reinterpret_cast<const uint2*>(g.add + at0);
            al = *reinterpret_cast<const uint2*>(g.add + at0 + g.part_out);
          }
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const uint32_t h2 = c < 2 ? ah.x : ah.y, l2 = c < 2 ? al.x : al.y;
            v[c] = g.by_sum * acc[i][j][c];
            if constexpr (KIND != kSym)
              v[c] += g.by_add * joined16(uint16_t(h2 >> (16 * (c & 1))), uint16_t(l2 >> (16 * (c & 1))));
            v[c] = row < g.M && col + c < g.N ? v[c] : 0.f;
            split16(v[c], hi[c], lo[c]);
          }
          if (KIND == kStep && g.last) {
            if (here) {
              uint16_t* o = g.last + (int64_t(p.e) * g.M + row) * g.N + col;
              const uint32_t x0 = bf16x2_rne(v[0] * g.by_last, v[1] * g.by_last),
                             x1 = bf16x2_rne(v[2] * g.by_last, v[3] * g.by_last);
              if (col + 3 < g.N) {
                Half4 t;
                t.v[0] = x0;
                t.v[1] = x1;
                *reinterpret_cast<Half4*>(o) = t;
              } else {
                for (int c = 0; c < 4; ++c)
                  if (col + c < g.N) o[c] = uint16_t((c < 2 ? x0 : x1) >> (16 * (c & 1)));
              }
            }
          } else {
            uint16_t* o = static_cast<uint16_t*>(g.out);
            if (here) {
              *reinterpret_cast<uint2*>(o + at0) = make_uint2(hi[0] | uint32_t(hi[1]) << 16, hi[2] | uint32_t(hi[3]) << 16);
              *reinterpret_cast<uint2*>(o + at0 + g.part_out) =
                  make_uint2(lo[0] | uint32_t(lo[1]) << 16, lo[2] | uint32_t(lo[3]) << 16);
            }
            if (SYM && p.m0 != p.n0 && row < g.ldo) {
              // the same value across the diagonal
#pragma unroll
              for (int c = 0; c < 4; ++c)
                if (col + c < g.N) {
                  const int64_t at1 = int64_t(p.e) * g.mat_out + int64_t(col + c) * g.ldo + row;
                  o[at1] = hi[c];
                  o[at1 + g.part_out] = lo[c];
                }
            }
          }
        }
      }
    }
  };
  auto store = [&](const Place& p) {
    const bool whole = p.m0 + BM <= p.m_end && p.n0 + BN <= g.N;
    if constexpr (RAGGED) {
      if (whole)
        store_some(p, std::true_type{});
      else
        store_some(p, std::false_type{});
      return whole;
    } else {
      store_some(p, std::false_type{});
      return false;
    }
  };

  // D stages ahead of the products; the loads of a wave are waited for in the
  // order of their issue, and a barrier publishes every wave's.
  constexpr int D = DIRECT ? S - 1 : 1;
  // (kGrad's numbers of rows are loads too)
  constexpr int PER = LOADS + S_PW, PER_SRC = LOADS + (KIND == kGrad ? B_PW : 0);
  advance();
  int ist = 0, ahead = 0;
  // the multiplying cursor walks the same tiles as the loading one
  Place now{};
  int cs = 0, cn = 0, cat = int(blockIdx.x);
  auto begin = [&]() {
    for (; cat < tiles; cat += int(gridDim.x)) {
      const bool in_turn = KIND == kGrad && gridDim.x % 8 == 0;
      now = place(in_turn ? tile_in_turn<BM == 256 ? 16 : 8>(cat, tiles) : tile_at(cat, int(gridDim.x), tiles));
      cn = stages_of(now);
      if (cn > 0) {
        cat += int(gridDim.x);
        cs = 0;
        return true;
      }
    }
    return false;
  };
#pragma unroll
  for (int d = 0; d < D; ++d) {
    if (more) {
      issue(ist);
      put(ist);
      ist = ist + 1 < S ? ist + 1 : 0;
      ++ahead;
    }
  }
  int st = 0;
  bool behind = false;  // the last tile's stores are younger than the loads that are waited for
  while (begin()) {
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) acc[i][j] = (v4f){0.f, 0.f, 0.f, 0.f};
    for (; cs < cn; ++cs) {
      if constexpr (DIRECT && D > 1) {
        if (ahead < D)
          __builtin_amdgcn_s_waitcnt(vm_count(0));
        else if (KIND == kGrad && g.src)
          __builtin_amdgcn_s_waitcnt(vm_count(std::min(63, (D - 1) * PER_SRC)));
        else
          __builtin_amdgcn_s_waitcnt(vm_count(std::min(63, (D - 1) * PER)));
      } else if (DIRECT && behind) {
        __builtin_amdgcn_s_waitcnt(vm_count(std::min(63, STORES)));
      } else if (DIRECT) {
        __builtin_amdgcn_s_waitcnt(vm_count(0));
      } else {
        __builtin_amdgcn_s_waitcnt(0xC07F);  // LDS alone: the loads went through registers
      }
      behind = false;
      asm volatile("" ::: "memory");
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
      if constexpr (KIND == kGrad && D == 1) {
        // the numbers of rows that the next loads go by arrived with this stage: the compiler's wait for them belongs here
#pragma unroll
        for (int u = 0; u < B_PW; ++u) asm volatile("" : "+v"(k_row[u]));
      }
      const bool load = more;
      multiply(st, load, ist);
      if (load) {
        put(ist);
        ist = ist + 1 < S ? ist + 1 : 0;
      } else {
        --ahead;
      }
      st = st + 1 < S ? st + 1 : 0;
    }
    behind = store(now);
  }
  __builtin_amdgcn_s_waitcnt(vm_count(0));  // no load may land after the LDS has changed hands
}

}  // namespace qbk
