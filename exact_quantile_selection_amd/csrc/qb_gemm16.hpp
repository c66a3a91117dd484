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
// bf16, 8192 x 8192 x 4096: 432 us KC x KC (1.27 PFLOP/s; the vendor library's
// product 350 on the same card), 430 KC x KS, 489 KS x KS, whose transposing reads
// get half the LDS bandwidth.  The matrix units are busy 64% of the CUs' cycles, at
// the 1.87 GHz that this leaves.  With experts' short sums a tile's results leave
// beside too few products: 131,072 rows over 64 experts of 1024 x 2048 take 520,
// 588 and 711, the matrix units busy 50% in the first.
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
  int out_parts;             // parts of a value that are written: 1 or 2 (both are added)
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
// its words' lowest bytes.  Sums are held in 32 bits: measured with single
// values in all four lanes of a row, nothing within 2^-23 of the largest is lost.
__device__ __forceinline__ v4f mma4(v8s a, v8s b, v4f c, int as, int bs) {
  const v4i x = __builtin_bit_cast(v4i, a), y = __builtin_bit_cast(v4i, b);
  const v8i u = __builtin_shufflevector(x, x, 0, 1, 2, 3, -1, -1, -1, -1);
  const v8i v = __builtin_shufflevector(y, y, 0, 1, 2, 3, -1, -1, -1, -1);
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(u, v, c, 4, 4, 0, as, 0, bs);
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

// The 8 values from `at` of a row of `length` (8 at least), zeros past its end,
// in two parts so that nothing waits between them: one load of 16 bytes, which
// begins earlier where fewer than 8 values are left, and the shift that puts
// those in their place, `missing` of them.
__device__ __forceinline__ int missing(int at, int length) {
  const int n = at + 8 - length;
  return n < 0 ? 0 : n > 8 ? 8 : n;
}
__device__ __forceinline__ uint4 ld_half8(const void* p) {
  typedef uint32_t half8 __attribute__((ext_vector_type(4), aligned(2)));
  const half8 t = *(const __attribute__((address_space(1))) half8*)p;
  return make_uint4(t[0], t[1], t[2], t[3]);
}
__device__ __forceinline__ uint4 ld_inside(const uint16_t* row, int at, int length) {
  return ld_half8(row + (at < length - 8 ? at : length - 8));
}
__device__ __forceinline__ uint4 in_place(uint4 v, int missing) {
  if (missing & 8) v = make_uint4(0, 0, 0, 0);
  if (missing & 4) v = make_uint4(v.z, v.w, 0, 0);
  if (missing & 2) v = make_uint4(v.y, v.z, v.w, 0);
  if (missing & 1) v = make_uint4(v.x >> 16 | v.y << 16, v.y >> 16 | v.z << 16, v.z >> 16 | v.w << 16, v.w >> 16);
  return v;
}
// The same value by value, for rows of fewer than 8.
__device__ __forceinline__ uint4 ld_short(const uint16_t* from, int at, int length) {
  const auto row = (const __attribute__((address_space(1))) uint16_t*)from;
  auto two = [&](int i) {
    const uint32_t lo = at + i < length ? row[at + i] : 0, hi = at + i + 1 < length ? row[at + i + 1] : 0;
    return lo | hi << 16;
  };
  return make_uint4(two(0), two(2), two(4), two(6));
}

// 16 or 4 bytes a lane from memory to the LDS at `to` (the wave's), lane by
// lane.  The compiler waits for every load that it knows to go to LDS before it
// reads LDS by a transposing read, whatever the addresses; of these it does not
// know, and the kernel's own waits order them (an operand lands a stage before
// it is read).  There is no result register, so nothing is reused too early,
// and m0 has no other use in a kernel that calls this.
template <int BYTES>
__device__ __forceinline__ void load_to_lds(const void* from, uint8_t* to) {
  const uint32_t at = uint32_t(uintptr_t((__attribute__((address_space(3))) uint8_t*)to));
  if constexpr (BYTES == 16)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(at), "v"(from) : "memory");
  else
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(at), "v"(from) : "memory");
}
// The same from a base that the wave shares and an offset of the lane's.
template <int BYTES>
__device__ __forceinline__ void load_to_lds(const void* base, uint32_t off, uint8_t* to) {
  const uint32_t at = uint32_t(uintptr_t((__attribute__((address_space(3))) uint8_t*)to));
  if constexpr (BYTES == 16)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(at), "v"(off), "s"(base) : "memory");
  else
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, %2" ::"s"(at), "v"(off), "s"(base) : "memory");
}

// A pointer that all lanes hold, told to the compiler: it then lies in scalar registers.
__device__ __forceinline__ const uint8_t* same_for_all(const void* p) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane(uint32_t(v)), hi = __builtin_amdgcn_readfirstlane(uint32_t(v >> 32));
  return reinterpret_cast<const uint8_t*>(uint64_t(hi) << 32 | lo);
}

// Waits until at most k (of up to K) stages of PER loads, and EXTRA stores, are
// outstanding, and every LDS read is back.
template <int K, int PER, int EXTRA>
__device__ __forceinline__ void wait_stages(int k) {
  if constexpr (K > 0) {
    if (k < K) return wait_stages<K - 1, PER, EXTRA>(k);
  }
  __builtin_amdgcn_s_waitcnt(vm_count(K * PER + EXTRA < 63 ? K * PER + EXTRA : 63));
}

// Whether 256 x 256 tiles (t256 of them) or 128 x 128 (t128).  It is a matter of whole rounds over the chip, one large
// tile a CU or two small ones: a round of large tiles takes 1.65 times as long as one of small ones and does twice the
// work.  Measured, us in 128 x 128 and 256 x 256:
//   two rounds against one: bf16 4096 x 4096 x 1024 40 and 36, 4 bits 4096 x 4096 x 4096 52 and 42, three-pass fp16 (24
//   updates of 1024 x 1024) 2212 and 2042;
//   five against three: bf16 5120 x 8192 x 2048 172 and 159, 4 bits 68.5 and 65, fp16 (64 updates of 1024 x 2048) 9847 and
//   8559;
//   one against one: bf16 2048 x 4096 x 1024 23.5 and 30, 4 bits 12.7 and 16.4, fp16 (12 of 1024 x 1024) 1118 and 1253.
// Ragged experts fill a part of their last tiles and are of unequal length: `uneven` of a round, by which they take the
// small tiles near an even choice.  Rows' products, 0.1: it decides five rounds against three, where either may be ahead
// (bf16, 16,384 rows over 16 experts of 2048 x 512 57 and 63; 40,000 over 64 of 1024 x 1024 126 and 111, over experts of
// weights e^2n, n normal, 126 and 134; 4 bits, 16,384 over 16 of 2048 x 2048 61 and 65).  Gradients, 0.25: it decides two
// against one, where unequal experts lose more than equal ones win (4096 rows over 8 of 2048 x 1024 41 and 34 if equal, 51
// and 71 with weights e^n).
inline bool in_large_tiles(int64_t t256, int64_t t128, double uneven) {
  const int64_t cu = device_cu_count();
  const double rounds256 = double((t256 + cu - 1) / cu), rounds128 = double((t128 + 2 * cu - 1) / (2 * cu));
  return t256 > 0 && 3.3 * (rounds256 + uneven) < 2 * rounds128;
}

#define QB_INLINE __attribute__((always_inline))

// B x B tiles by 2 x 4 waves (2 x 2 for the smaller ones), a ring of S stages.  DIRECT: rows are multiples
// of 16 bytes, and the loads go to LDS; else they pass through registers, 2
// bytes being the only alignment asked for.  PA, PB: which part of each operand
// each of PARTS passes over K multiplies, a bit a pass.
//
// A stage is two steps of 32 of K.  While a wave multiplies a step, whose
// operands are in registers, it reads the next one's, A's row tile by row tile
// into the registers that are done with; early in a stage's second step it waits
// at a barrier for the next stage's loads, and every wave has read all of this
// one, whose place in the ring takes new loads in the shadow of the products
// that are left.  The loads run on over the end of a tile.
template <class T, int KIND, bool A_KS, bool B_KS, int B, int S, bool DIRECT, int PARTS = 1, int PA = 0, int PB = 0>
__global__ __launch_bounds__(B == 256 ? 512 : 256, B == 64 && !DIRECT ? 4 : 2) void k_gemm16(const Gemm16 g) {
  constexpr int WN = B == 256 ? 4 : 2, W = 2 * WN, TM = B / 32, TN = B / WN / 16;
  constexpr int KT = 64;  // of K a stage: 128 bytes of a KC row
  constexpr int BYTES = B * KT * 2, PW = BYTES / 1024 / W;  // of an operand's stage; its 1 KiB loads a wave
  constexpr bool FOUR = std::is_same_v<T, Fp4>;
  constexpr int S_PW = FOUR ? 2 * B / 32 / W : 0;  // loads of 32 rows' 8 exponents a wave
  constexpr int S_BYTES = FOUR ? 2 * B * 8 : 0;
  constexpr bool RAGGED = KIND == kRows || KIND == kGrad, SYM = KIND == kSym || KIND == kSqr;
  constexpr bool BY_ROW = KIND == kRows && !FOUR;  // A's rows may be numbered by src
  // a row's number in the swizzle of its slots
  auto key_r = [](int row) { return (row >> 1) & 7; };
  auto key_k = [](int k) { return B >= 128 ? (k & 3) | ((k >> 1) & 4) : ((k >> 1) & 1) | ((k >> 2) & 2); };
  constexpr int RING = S * (2 * BYTES + S_BYTES);
  constexpr int SRC_BYTES = BY_ROW ? 8 * B * 4 : 0;  // numbers of the last 8 tiles' rows
  __shared__ __align__(1024) uint8_t lds[RING + SRC_BYTES + W * 256 + (RAGGED ? 1024 * 3 + 16 : 0) +
                                         (SYM ? W * (TN < 4 ? 1024 : 2048) : 0)];
  uint8_t* const lds_b = lds + S * BYTES;
  uint8_t* const lds_s = lds + S * 2 * BYTES;
  int* const src_of = reinterpret_cast<int*>(lds + RING);
  uint8_t* const turned = lds + RING + SRC_BYTES + W * 256;  // SYM: 16 rows of a wave's results
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  int* const kept_of = reinterpret_cast<int*>(lds + RING + SRC_BYTES) + wave * 64;  // the last 8 tiles' places, a copy a wave
  const int tn_all = (g.N + B - 1) / B, tm_all = (g.M + B - 1) / B;
  int tiles = g.tiles;

  // the experts' first and last rows and their tiles of rows before each
  int* const first_of = reinterpret_cast<int*>(lds + RING + SRC_BYTES + W * 256);
  int *const end_of = first_of + 256, *const before_of = end_of + 256;  // 256, 256 and 257 of them
  if (RAGGED && g.off) {
    if (wave == 0) {
      int lo[4], hi[4], n[4], before;
      const int total = group_tiles(g.off, g.G, KIND == kGrad ? g.K : g.M, B, lane, lo, hi, n, before);
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
    if constexpr (KIND == kRows)
      tiles = std::min(__builtin_amdgcn_readfirstlane(before_of[256]), tiles / tn_all) * tn_all;
  }

  // A tile: rows m0 .. m_end - 1 and columns from n0 of a result; K from k0 to
  // k1; e: its matrix, and for kGrad the part of K.
  struct Place {
    int m0, m_end, n0, k0, k1, e, part;
  };
  auto place = [&](int t) QB_INLINE {
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
      p.m0 = tm * B;
    } else if constexpr (KIND == kRows) {
      if (g.off) {
        tile_order(t, tiles / tn_all, tn_all, 8, tm, tn);
        // the expert whose tiles hold tm: the last of those that begin at or before it
        int begun = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) begun += __popcll(__ballot(before_of[4 * lane + j] <= tm));
        p.e = begun > 0 ? begun - 1 : 0;
        p.m0 = __builtin_amdgcn_readfirstlane(first_of[p.e] + (tm - before_of[p.e]) * B);
        p.m_end = __builtin_amdgcn_readfirstlane(end_of[p.e]);
      } else {
        tile_order(t, tm_all, tn_all, 8, tm, tn);
        p.m0 = tm * B;
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
      p.m0 = tm * B;
    } else {
      const int per = tm_all * tn_all;
      p.e = t / per;
      tile_order(t % per, tm_all, tn_all, 8, tm, tn);
      p.m0 = tm * B;
    }
    p.n0 = tn * B;
    return p;
  };
  // stages of one pass over K
  auto pass_of = [&](const Place& p) QB_INLINE {
    return KIND == kGrad ? (p.k1 - p.k0 + KT - 1) / KT : (g.K + KT - 1) / KT;
  };
  auto order = [&](int t) QB_INLINE {
    const bool in_turn = KIND == kGrad && gridDim.x % 8 == 0;
    return in_turn ? tile_in_turn<B == 256 ? 16 : 8>(t, tiles) : tile_at(t, int(gridDim.x), tiles);
  };

  // --- the loads ---
  // The tile whose loads are issued next; its stages: ls of ln in this pass over
  // K, lpass of PARTS.
  Place lp{}, np{};
  int ls = 0, ln = 0, lpass = 0, lat = int(blockIdx.x), ltile = 0;
  bool more = false;
  int ctile = -1;  // the number of the tile that is multiplied, as ltile - 1 is of the one that is loaded
  // lane's part in load u: of a KC operand row r, 8 values from q; of a KS one row k, 8 columns from c
  auto kc_r = [&](int u) QB_INLINE { return ((wave * PW + u) * kWave + lane) >> 3; };
  auto kc_q = [&](int u) QB_INLINE { return ((lane & 7) ^ key_r(kc_r(u))) * 8; };
  auto ks_k = [&](int u) QB_INLINE { return ((wave * PW + u) * kWave + lane) / (B / 8); };
  auto ks_c = [&](int u) QB_INLINE {
    const int s = ((wave * PW + u) * kWave + lane) % (B / 8);
    return (((s >> 1) ^ key_k(ks_k(u))) * 2 + (s & 1)) * 8;
  };
  auto times = [](int row, int64_t ld) QB_INLINE { return int64_t(uint64_t(uint32_t(row)) * uint32_t(ld)); };
  // Each lane's offsets in bytes from the stage's bases.
  const uint8_t *a_base = nullptr, *b_base = nullptr;
  uint32_t a_off[PW], b_off[PW];
  const uint8_t* s_base = nullptr;  // 4 bits: the exponents' of the operand whose this wave loads
  uint32_t s_off[FOUR ? S_PW : 1];
  int a_row[BY_ROW && !DIRECT ? PW : 1];    // !DIRECT: A's rows, which may lie beyond 32 bits of their base
  uint32_t off_end = 0;                     // !DIRECT: how many of a load's columns lie past their rows' end, 4 bits each
  int k_row[KIND == kGrad ? PW : 1];
  uint32_t k_off[KIND == kGrad ? PW : 1];  // kGrad with src: B's offsets of this stage's rows
  bool some_out = false;                            // and whether one of the wave's rows was routed nowhere
  auto wait_all = [&]() QB_INLINE {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(vm_count(0));
    asm volatile("" ::: "memory");
  };
  // kRows: the numbers of tile p's rows, each wave those that it loads.
  constexpr int RPW = B / W;
  auto fetch_rows = [&](const Place& p, int tile) QB_INLINE {
    const int row = p.m0 + wave * RPW + lane;
    if (lane < RPW)
      load_to_lds<4>(g.src + (row < p.m_end ? row : p.m_end - 1),
                     reinterpret_cast<uint8_t*>(src_of + (tile & 7) * B + wave * RPW));
  };
  // kGrad: a stage's rows, of which each wave loads KPW that follow one another, and each of its loads RPL of them;
  // their numbers are read into scalar registers (by a counter of their own: they keep no vector load waiting).
  constexpr int KPW = KT / W, RPL = KPW / PW;
  int rows[KIND == kGrad ? KPW : 1];
  // Where the first stage of a pass lies.
  auto set_bases = [&]() QB_INLINE {
    const uint16_t *a = g.A, *b = g.B;
    if constexpr (!RAGGED) a += int64_t(lp.e) * g.mat_a;
    if constexpr (KIND != kGrad) b += int64_t(lp.e) * g.mat_b;
    if constexpr (PARTS > 1) {
      a += ((PA >> lpass) & 1) * g.part_a;
      b += ((PB >> lpass) & 1) * g.part_b;
    }
    if constexpr (A_KS)
      a += times(lp.k0, g.lda);
    else if (!BY_ROW || !g.src)
      a += times(lp.m0, g.lda);
    if constexpr (!B_KS)
      b += times(lp.n0, g.ldb);
    else if (KIND != kGrad || !g.src)
      b += times(lp.k0, g.ldb);
    a_base = same_for_all(a);
    b_base = same_for_all(b);
    if constexpr (FOUR)
      s_base = same_for_all(wave < W / 2 ? g.As + times(lp.m0, g.sld)
                                         : g.Bs + int64_t(lp.e) * g.mat_bs + times(lp.n0, g.sld));
  };
  // Rows and columns past a tile's end are the last ones again, for results
  // that are not kept; rows that src routes nowhere are row 0, and their results
  // are written as zeros.
  auto set_offsets = [&]() QB_INLINE {
    off_end = 0;
#pragma unroll
    for (int u = 0; u < PW; ++u) {
      // a column, the last 8 of a row at most (DIRECT: rows are multiples of 8)
      auto column = [&](int c, int length, int load) QB_INLINE {
        const int most = DIRECT ? (length - 1) & ~7 : length < 8 ? 0 : length - 8;
        if (!DIRECT) off_end |= uint32_t(missing(c, length)) << (4 * load);
        return c < most ? c : most;
      };
      if constexpr (A_KS) {
        a_off[u] = 2 * (uint32_t(ks_k(u)) * uint32_t(g.lda) + column(lp.m0 + ks_c(u), g.M, u));
      } else {
        const int r = kc_r(u);
        int row = lp.m0 + r < lp.m_end ? r : lp.m_end - 1 - lp.m0;
        if (BY_ROW && g.src) {
          row = src_of[(((ltile - 1) & 7) * B + r) & (8 * B - 1)];
          row = uint32_t(row) < uint32_t(g.Mx) ? row : 0;
        }
        if constexpr (BY_ROW && !DIRECT) a_row[u] = row;
        a_off[u] = 2 * ((BY_ROW && !DIRECT ? 0 : uint32_t(row) * uint32_t(g.lda)) + kc_q(u));
      }
      if constexpr (B_KS) {
        b_off[u] = 2 * ((KIND == kGrad && g.src ? 0 : uint32_t(ks_k(u)) * uint32_t(g.ldb)) +
                        column(lp.n0 + ks_c(u), g.N, PW + u));
      } else {
        const int r = kc_r(u), row = lp.n0 + r < g.N ? r : g.N - 1 - lp.n0;
        b_off[u] = 2 * (uint32_t(row) * uint32_t(g.ldb) + kc_q(u));
      }
    }
  };
  auto set_scales = [&]() QB_INLINE {
    if constexpr (FOUR) {
#pragma unroll
      for (int j = 0; j < S_PW; ++j) {
        int r = (wave * S_PW + j) * 32 % B + (lane >> 1);
        const int most = (wave < W / 2 ? lp.m_end - lp.m0 : g.N - lp.n0) - 1;
        r = r < most ? r : most;
        s_off[j] = uint32_t(r) * uint32_t(g.sld) + (lane & 1) * 4;
      }
    }
  };
  // The numbers of the rows that stage ls reads.
  auto stage_rows = [&]() QB_INLINE {
    if constexpr (KIND == kGrad) {
      if (g.src) {
        const auto src = (const __attribute__((address_space(4))) int32_t*)g.src;
        const int k = __builtin_amdgcn_readfirstlane(lp.k0 + ls * KT + wave * KPW);
        if (k + KPW <= lp.k1) {
#pragma unroll
          for (int i = 0; i < KPW; ++i) rows[i] = src[k + i];
        } else {
#pragma unroll
          for (int i = 0; i < KPW; ++i) rows[i] = src[std::min(k + i, lp.k1 - 1)];
        }
      }
    }
  };
  // and, once those reads are back, where the rows lie
  auto take_rows = [&]() QB_INLINE {
    if constexpr (KIND == kGrad) {
      if (g.src) {
        bool out = false;
#pragma unroll
        for (int u = 0; u < PW; ++u) {
          k_row[u] = rows[u * RPL];
#pragma unroll
          for (int i = 1; i < RPL; ++i) k_row[u] = lane / (kWave / RPL) == i ? rows[u * RPL + i] : k_row[u];
          out = out || uint32_t(k_row[u]) >= uint32_t(g.Mx);
          k_off[u] = uint32_t(k_row[u]) * uint32_t(2 * g.ldb) + b_off[u];
        }
        some_out = __ballot(out) != 0;
      }
    }
  };
  // The next tile that has something to multiply; of the others (experts
  // without rows) the gradient is written as zeros.
  auto advance = [&]() QB_INLINE {
    more = false;
    for (; lat < tiles; lat += int(gridDim.x)) {
      lp = BY_ROW && ltile > 0 && g.src ? np : place(order(lat));
      ln = pass_of(lp);
      if (ln > 0) {
        more = true;
        lat += int(gridDim.x);
        break;
      }
      if constexpr (KIND == kGrad)
        zero_tile<B, B, W>(static_cast<float*>(g.out), (int64_t(lp.part) * g.G + lp.e) * g.M, lp.m0, g.M, lp.n0, g.N,
                           tid);
    }
    ls = lpass = 0;
    if (!more) return;
    if constexpr (BY_ROW) {
      if (g.src) {
        // the first tile's numbers are waited for; another's were fetched with the tile before it, and have landed
        // with what that multiplied already unless it had less than a ring of stages
        if (ltile == 0) fetch_rows(lp, 0);
        if (ltile == 0 || ln < S + 1) wait_all();
      }
    }
    ++ltile;
    if (lane == 0) {
      int* kept = kept_of + ((ltile - 1) & 7) * 8;
      kept[0] = lp.m0, kept[1] = lp.m_end, kept[2] = lp.n0, kept[3] = lp.e, kept[4] = lp.part, kept[5] = ln * PARTS;
    }
    set_bases();
    set_offsets();
    set_scales();
    stage_rows();
    if constexpr (BY_ROW) {
      if (g.src && lat < tiles) {
        np = place(order(lat));
        fetch_rows(np, ltile);
      }
    }
  };
  auto next_stage = [&]() QB_INLINE {
    if (++ls < ln) {
      a_base += A_KS ? KT * 2 * g.lda : KT * 2;
      b_base += B_KS ? (KIND == kGrad && g.src ? 0 : KT * 2 * g.ldb) : KT * 2;
      if constexpr (FOUR) s_base += 8;
      stage_rows();
    } else if (lpass + 1 < PARTS) {
      ls = 0;
      ++lpass;
      set_bases();
    } else {
      advance();
    }
  };

  auto slot_a = [&](int u, int st) QB_INLINE { return lds + st * BYTES + (wave * PW + u) * 1024; };
  auto slot_b = [&](int u, int st) QB_INLINE { return lds_b + st * BYTES + (wave * PW + u) * 1024; };
  auto left_of_k = [&]() QB_INLINE { return (KIND == kGrad ? lp.k1 - lp.k0 : g.K) - ls * KT; };
  // Whether stage ls is whole and (kGrad) all its rows are there.
  auto plain = [&]() QB_INLINE {
    return more && left_of_k() >= KT && !(KIND == kGrad && some_out) && (DIRECT || (g.lda >= 8 && g.ldb >= 8));
  };
  // !DIRECT: what a stage's loads read, and how many values of each are missing, 4 bits each
  uint4 held[DIRECT ? 1 : 2 * PW];
  uint32_t held_missing = 0;
  int held_for = -1;  // the place in the ring that they are for
  auto a_row_at = [&](int u) QB_INLINE { return BY_ROW && !DIRECT ? 2 * times(a_row[BY_ROW && !DIRECT ? u : 0], g.lda) : 0; };
  auto b_row_at = [&](int u) QB_INLINE {
    return KIND == kGrad && g.src ? 2 * times(k_row[KIND == kGrad ? u : 0], g.ldb) : 0;
  };
  // one of a whole stage's loads, A's and B's in turn
  auto issue_plain = [&](int v, int st) QB_INLINE {
    const int u = v >> 1;
    if constexpr (DIRECT) {
      if (v & 1)
        load_to_lds<16>(b_base, KIND == kGrad && g.src ? k_off[KIND == kGrad ? u : 0] : b_off[u], slot_b(u, st));
      else
        load_to_lds<16>(a_base, a_off[u], slot_a(u, st));
    } else {
      if (v & 1)
        held[PW + u] = ld_half8(b_base + b_row_at(u) + b_off[u]);
      else
        held[u] = ld_half8(a_base + a_row_at(u) + a_off[u]);
      held_missing = off_end;
      held_for = st;
    }
  };
  auto issue_scales = [&](int st) QB_INLINE {
    if constexpr (FOUR) {
#pragma unroll
      for (int j = 0; j < S_PW; ++j)
        load_to_lds<4>(s_base, s_off[j], lds_s + st * S_BYTES + (wave * S_PW + j) * 256);
    }
  };
  // Stage ls of the loading tile to place st of the ring, whatever it is: zeros past the end of K, and for kGrad in both
  // operands' rows that src routes nowhere.
  auto issue = [&](int st) QB_INLINE {
    const int left = left_of_k();
    held_missing = off_end;
    held_for = st;
#pragma unroll
    for (int u = 0; u < PW; ++u) {
      const bool out = KIND == kGrad && g.src && uint32_t(k_row[KIND == kGrad ? u : 0]) >= uint32_t(g.Mx);
      const uint8_t *pa = a_base + a_row_at(u) + a_off[u], *pb = b_base + (out ? 0 : b_row_at(u)) + b_off[u];
      if constexpr (DIRECT) {
        const uint8_t* const zero = reinterpret_cast<const uint8_t*>(&kZero16);
        load_to_lds<16>((A_KS ? ks_k(u) : kc_q(u)) < left && !out ? pa : zero, slot_a(u, st));
        load_to_lds<16>((B_KS ? ks_k(u) : kc_q(u)) < left && !out ? pb : zero, slot_b(u, st));
      } else {
        // a KS operand's row, or the last there is (by_src: its own); a KC operand's values, or the row's last 8
        auto hold = [&](bool ks, const uint8_t* p, int64_t ld, int length, int col, int i, bool by_src) QB_INLINE {
          const int over = ks ? ks_k(u) - left + 1 : kc_q(u) + 8 - left;
          if (ks && over > 0 && !by_src) p -= 2 * times(over, ld);
          if (length < 8) {
            // (rows of fewer than 8 values: p is a KS operand's row, or q values on in a KC one's)
            const uint16_t* row = reinterpret_cast<const uint16_t*>(p) - (ks ? 0 : kc_q(u));
            held[i] = ld_short(row, ks ? col : kc_q(u), out || (ks && over > 0) ? 0 : ks ? length : left);
            held_missing &= ~(15u << (4 * i));
            return;
          }
          if (!ks && over > 0) p -= 2 * over;
          held[i] = ld_half8(p);
          const int none = out || (ks && over > 0) ? 8 : ks || over <= 0 ? 0 : over < 8 ? over : 8;
          if (none) held_missing = (held_missing & ~(15u << (4 * i))) | uint32_t(none) << (4 * i);
        };
        hold(A_KS, pa, g.lda, A_KS ? g.M : g.K, lp.m0 + ks_c(u), u, false);
        hold(B_KS, pb, g.ldb, B_KS ? g.N : g.K, lp.n0 + ks_c(u), PW + u, KIND == kGrad && g.src);
      }
    }
    issue_scales(st);
  };
  auto put = [&]() QB_INLINE {  // !DIRECT: what issue() read
    if constexpr (!DIRECT) {
      if (held_for >= 0) {
        if (__ballot(held_missing != 0) != 0)
#pragma unroll
          for (int i = 0; i < 2 * PW; ++i) held[i] = in_place(held[i], held_missing >> (4 * i) & 15);
        held_missing = 0;
#pragma unroll
        for (int u = 0; u < PW; ++u) {
          *reinterpret_cast<uint4*>(slot_a(u, held_for) + lane * 16) = held[u];
          *reinterpret_cast<uint4*>(slot_b(u, held_for) + lane * 16) = held[PW + u];
        }
      }
      held_for = -1;
    }
  };

  // --- the products ---
  v4f acc[TM][TN];
  const int r = lane & 15, g4 = lane >> 4;
  // The lane's 16 bytes of step 0 of row tile 0; step 1's lie 4 slots on.
  const int frag_a = A_KS ? (8 * g4 + (r >> 2)) * (B * 2) + (((wm * TM) ^ key_k(8 * g4 + (r >> 2))) * 32) + (r & 3) * 8
                          : (wm * TM * 16 + r) * 128 + ((g4 ^ key_r(r)) * 16);
  const int frag_b = B_KS ? (8 * g4 + (r >> 2)) * (B * 2) + (((wn * TN) ^ key_k(8 * g4 + (r >> 2))) * 32) + (r & 3) * 8
                          : (wn * TN * 16 + r) * 128 + ((g4 ^ key_r(r)) * 16);
  auto read_ks = [&](const uint8_t* p, int h) QB_INLINE {
    const auto q = (__attribute__((address_space(3))) uint8_t*)p;
    const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s)(q + 32 * h * (B * 2)));
    const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s)(q + (32 * h + 4) * (B * 2)));
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  };
  // a step's operands, and B's of two steps; their exponents
  v8s a[TM], b[2][TN];
  int as[FOUR ? TM : 1], bs[2][FOUR ? TN : 1];
  // step h's part of column tile j, or of row tile i, of the stage in place st of the ring
  auto read_b = [&](int j, int st, auto h) QB_INLINE {
    constexpr int H = decltype(h)::value;
    const uint8_t* p = lds_b + st * BYTES;
    if constexpr (B_KS)
      b[H][j] = read_ks(p + (frag_b ^ (j * 32)), H);
    else
      b[H][j] = *reinterpret_cast<const v8s*>(p + j * 16 * 128 + (frag_b ^ (H * 64)));
    if constexpr (FOUR) bs[H][j] = lds_s[st * S_BYTES + (B + (wn * TN + j) * 16 + r) * 8 + g4 + 4 * H];
  };
  auto read_a = [&](int i, int st, auto h) QB_INLINE {
    constexpr int H = decltype(h)::value;
    const uint8_t* p = lds + st * BYTES;
    if constexpr (A_KS)
      a[i] = read_ks(p + (frag_a ^ (i * 32)), H);
    else
      a[i] = *reinterpret_cast<const v8s*>(p + i * 16 * 128 + (frag_a ^ (H * 64)));
    if constexpr (FOUR) as[i] = lds_s[st * S_BYTES + ((wm * TM + i) * 16 + r) * 8 + g4 + 4 * H];
  };
  auto multiply = [&](int i, auto h) QB_INLINE {
    constexpr int H = decltype(h)::value;
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      if constexpr (FOUR)
        acc[i][j] = mma4(b[H][j], a[i], acc[i][j], bs[H][j], as[i]);
      else
        acc[i][j] = mma16<T>(b[H][j], a[i], acc[i][j]);
    }
    if constexpr (FOUR) {
      // the products stay here: the compiler would gather a stage's behind its reads, out of registers
#pragma unroll
      for (int j = 0; j < TN; ++j) asm volatile("" : "+v"(acc[i][j]));
    }
  };
  constexpr std::integral_constant<int, 0> first{};
  constexpr std::integral_constant<int, 1> second{};

  // Element c of acc[i][j] is row 16 i + r, column 16 j + 4 g4 + c.  For 16-bit results the four lanes of a row
  // exchange what they hold of JT column tiles, so that each has 4 JT columns side by side: of tile g4 (JT = 4), or half
  // of tile g4 & 1 (JT = 2).
  constexpr int JT = TN < 4 ? TN : 4;
  auto exchange = [&](uint32_t(&w)[JT]) QB_INLINE {
    auto swap32 = [](uint32_t& x, uint32_t& y) {
      const auto t = __builtin_amdgcn_permlane32_swap(x, y, false, false);
      x = t[0], y = t[1];
    };
    auto swap16 = [](uint32_t& x, uint32_t& y) {
      const auto t = __builtin_amdgcn_permlane16_swap(x, y, false, false);
      x = t[0], y = t[1];
    };
    if constexpr (JT == 4) {
      swap32(w[0], w[2]);
      swap32(w[1], w[3]);
      swap16(w[0], w[1]);
      swap16(w[2], w[3]);
    } else {
      swap16(w[0], w[1]);
    }
  };
  // where the lane's stretch of 4 JT columns of column tiles from j begins
  auto stretch = [&](const Place& p, int j) QB_INLINE {
    return p.n0 + (wn * TN + j) * 16 + (JT == 4 ? g4 * 16 : (g4 & 1) * 16 + (g4 >> 1) * 8);
  };
  constexpr int STORES = KIND == kGrad ? TM * TN : TM * TN / 2;
  // kSqr, kStep: the addends of the lane's part of row tile i and the JT column tiles from j0, which are read two such
  // parts ahead of the one that is written
  constexpr bool SQUARE = SYM || KIND == kStep, ADDS = KIND == kSqr || KIND == kStep;
  constexpr int STRIPS = TN / JT;
  uint4 addend[ADDS ? 3 : 1][JT / 2][2];
  // A strip's place in out's layout, the same for all lanes, and the lane's in bytes from there.  Made anew for each
  // tile: the compiler would keep a register for each strip through the products.
  uint32_t lane_at = 0;
  auto strip_at = [&](const uint16_t* array, const Place& p, int strip) QB_INLINE {
    const int64_t row = p.m0 + (wm * TM + strip / STRIPS) * 16, col = p.n0 + (wn * TN + strip % STRIPS * JT) * 16;
    return same_for_all(array + int64_t(p.e) * g.mat_out + row * g.ldo + col);
  };
  auto ld_16_of = [](const uint8_t* base, uint32_t off) QB_INLINE {
    typedef uint32_t w4 __attribute__((ext_vector_type(4)));
    const w4 t = *(const __attribute__((address_space(1))) w4*)((const __attribute__((address_space(1))) uint8_t*)base + off);
    return make_uint4(t[0], t[1], t[2], t[3]);
  };
  auto st_16_of = [](uint8_t* base, uint32_t off, uint4 v) QB_INLINE {
    typedef uint32_t w4 __attribute__((ext_vector_type(4)));
    *(__attribute__((address_space(1))) w4*)((__attribute__((address_space(1))) uint8_t*)base + off) = (w4){v.x, v.y, v.z, v.w};
  };
  auto read_addends = [&](const Place& p, int strip, auto whole) QB_INLINE {
    if constexpr (ADDS) {
      const int row = p.m0 + (wm * TM + strip / STRIPS) * 16 + r, col0 = stretch(p, strip % STRIPS * JT);
      const uint8_t* const from = strip_at(g.add, p, strip);
#pragma unroll
      for (int h = 0; h < JT / 2; ++h) {
        const int col = col0 + 8 * h;
        uint4(&v)[2] = addend[strip % 3][h];
        v[0] = v[1] = make_uint4(0, 0, 0, 0);
        if (whole() || (row < g.M && col < g.ldo)) {
          v[0] = ld_16_of(from, lane_at + 16 * h);
          v[1] = ld_16_of(from + 2 * g.part_out, lane_at + 16 * h);
        }
      }
    }
  };
  auto store_some = [&](const Place& p, auto whole) QB_INLINE {
    if constexpr (SQUARE) {
      lane_at = 2 * (uint32_t(r) * uint32_t(g.ldo) + (JT == 4 ? g4 * 16 : (g4 & 1) * 16 + (g4 >> 1) * 8));
      asm volatile("" : "+v"(lane_at));
    }
    if constexpr (ADDS) {
      read_addends(p, 0, whole);
      if (TM * STRIPS > 1) read_addends(p, 1, whole);
    }
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
        const bool dead = BY_ROW && g.src &&
                          uint32_t(src_of[((ctile & 7) * B + (wm * TM + i) * 16 + r) & (8 * B - 1)]) >= uint32_t(g.Mx);
        uint16_t* o = static_cast<uint16_t*>(g.out) + int64_t(row) * g.N;
#pragma unroll
        for (int j0 = 0; j0 < TN; j0 += JT) {
          uint32_t w[2][JT];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
#pragma unroll
            for (int j = 0; j < JT; ++j) w[k][j] = bf16x2_rne(acc[i][j0 + j][2 * k], acc[i][j0 + j][2 * k + 1]);
            exchange(w[k]);
          }
          if (!whole() && row >= p.m_end) continue;
          const int col0 = stretch(p, j0);
#pragma unroll
          for (int h = 0; h < JT / 2; ++h) {  // 8 columns each
            const int col = col0 + 8 * h;
            Half8 t;
#pragma unroll
            for (int k = 0; k < 4; ++k) t.v[k] = dead ? 0 : w[k & 1][2 * h + (k >> 1)];
            if (whole() || col + 7 < g.N) {
              *reinterpret_cast<Half8*>(o + col) = t;
            } else {
#pragma unroll
              for (int c = 0; c < 8; ++c)
                if (col + c < g.N) o[col + c] = uint16_t(t.v[c >> 1] >> (16 * (c & 1)));
            }
          }
        }
      } else {
        // rows of ldo values, a multiple of 8, of which those past N are kept zero
#pragma unroll
        for (int j0 = 0; j0 < TN; j0 += JT) {
          const int strip = i * STRIPS + j0 / JT;
          if (strip + 2 < TM * STRIPS) read_addends(p, strip + 2, whole);
          uint32_t w[4][JT];  // the lane's columns: w[c][x] is column 4 x + c of its stretch
#pragma unroll
          for (int c = 0; c < 4; ++c) {
#pragma unroll
            for (int j = 0; j < JT; ++j) {
              const float e = acc[i][j0 + j][c];  // (a bit cast of the element itself would take the vector's first)
              w[c][j] = __builtin_bit_cast(uint32_t, e);
            }
            exchange(w[c]);
          }
          const int col0 = stretch(p, j0);
          uint4 parts[2][JT / 2];
#pragma unroll
          for (int h = 0; h < JT / 2; ++h) {  // 8 columns each
            const int col = col0 + 8 * h;
            const uint4 ah = addend[ADDS ? strip % 3 : 0][h][0], al = addend[ADDS ? strip % 3 : 0][h][1];
            const uint32_t h4[4] = {ah.x, ah.y, ah.z, ah.w}, l4[4] = {al.x, al.y, al.z, al.w};
            float v[8];
            uint16_t hi[8], lo[8];
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              v[c] = g.by_sum * __builtin_bit_cast(float, w[c & 3][2 * h + (c >> 2)]);
              if constexpr (ADDS)
                v[c] += g.by_add * joined16(uint16_t(h4[c >> 1] >> (16 * (c & 1))), uint16_t(l4[c >> 1] >> (16 * (c & 1))));
              if (!whole()) v[c] = row < g.M && col + c < g.N ? v[c] : 0.f;
              split16(v[c], hi[c], lo[c]);
            }
            auto two = [](const uint16_t(&x)[8], int k) { return x[2 * k] | uint32_t(x[2 * k + 1]) << 16; };
            parts[0][h] = make_uint4(two(hi, 0), two(hi, 1), two(hi, 2), two(hi, 3));
            parts[1][h] = make_uint4(two(lo, 0), two(lo, 1), two(lo, 2), two(lo, 3));
            const bool here = whole() || (row < g.M && col < g.ldo);
            if (KIND == kStep && g.last) {
              if (here) {
                uint16_t* o = g.last + (int64_t(p.e) * g.M + row) * g.N + col;
                Half8 t;
#pragma unroll
                for (int k = 0; k < 4; ++k) t.v[k] = bf16x2_rne(v[2 * k] * g.by_last, v[2 * k + 1] * g.by_last);
                if (whole() || col + 7 < g.N) {
                  *reinterpret_cast<Half8*>(o) = t;
                } else {
#pragma unroll
                  for (int c = 0; c < 8; ++c)
                    if (col + c < g.N) o[c] = uint16_t(t.v[c >> 1] >> (16 * (c & 1)));
                }
              }
            } else if (here) {
              uint8_t* const to = const_cast<uint8_t*>(strip_at(static_cast<const uint16_t*>(g.out), p, strip));
              st_16_of(to, lane_at + 16 * h, parts[0][h]);
              if (g.out_parts > 1) st_16_of(to + 2 * g.part_out, lane_at + 16 * h, parts[1][h]);
            }
          }
          if (SYM && p.m0 != p.n0) {
            // The same values across the diagonal: 16 rows of 16 JT columns pass through LDS, 16-byte slots XORed with
            // the row, and come back as 8 rows of a column.
            constexpr int ROW = JT * 32, SLOTS = ROW / 16;
            uint8_t* const turn = turned + wave * (16 * ROW);
#pragma unroll
            for (int part = 0; part < 2; ++part) {
              if (part == 1 && g.out_parts == 1) break;
#pragma unroll
              for (int h = 0; h < JT / 2; ++h)
                *reinterpret_cast<uint4*>(turn + r * ROW + ((((col0 - p.n0 - (wn * TN + j0) * 16) / 8 + h) ^ r) % SLOTS) * 16) =
                    parts[part][h];
#pragma unroll
              for (int q = 0; q < JT / 2; ++q) {  // the lane's column of tile jt, 8 rows from 8 half
                const int jt = JT == 4 ? g4 : g4 & 1, half = JT == 4 ? q : g4 >> 1;
                v4s t[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                  const int from = 8 * half + 4 * k + (r >> 2);
                  const auto at = (__attribute__((address_space(3))) uint8_t*)(turn + from * ROW +
                                                                               ((2 * jt + (r >> 1 & 1)) ^ from) % SLOTS * 16 +
                                                                               (r & 1) * 8);
                  t[k] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s)at);
                }
                const int col = p.n0 + (wn * TN + j0 + jt) * 16 + r, row8 = p.m0 + (wm * TM + i) * 16 + 8 * half;
                if (whole() || (col < g.N && row8 < g.ldo))
                  *reinterpret_cast<v8s*>(static_cast<uint16_t*>(g.out) + int64_t(p.e) * g.mat_out + part * g.part_out +
                                          int64_t(col) * g.ldo + row8) =
                      __builtin_shufflevector(t[0], t[1], 0, 1, 2, 3, 4, 5, 6, 7);
              }
            }
          }
        }
      }
    }
  };
  auto store = [&](const Place& p) QB_INLINE {
    const bool whole = p.m0 + B <= p.m_end && p.n0 + B <= g.N;
    if (whole)
      store_some(p, std::true_type{});
    else
      store_some(p, std::false_type{});
    return RAGGED && whole;
  };

  // The loads of a wave are waited for in the order of their issue, and a
  // barrier publishes every wave's.  `ahead`: stages issued and not multiplied yet,
  // the current one among them; `behind`: that many stages more have loads that
  // are older than the last tile's stores.
  constexpr int PER = 2 * PW + S_PW;
  int ahead = 0, behind = 0;
  // the tile that is multiplied: what was kept of it when its loads began
  Place now{};
  auto begin = [&]() QB_INLINE {
    if (++ctile == ltile) return 0;
    const int* kept = kept_of + (ctile & 7) * 8;
    auto at = [&](int i) QB_INLINE { return __builtin_amdgcn_readfirstlane(kept[i]); };
    now = Place{at(0), at(1), at(2), 0, 0, at(3), at(4)};
    return at(5);
  };
  auto clear = [&]() QB_INLINE {
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) acc[i][j] = (v4f){0.f, 0.f, 0.f, 0.f};
  };
  advance();
#pragma unroll 1
  for (int d = 0; d < S; ++d) {
    if (!more) break;
    take_rows();
    issue(d);
    put();
    next_stage();
    ++ahead;
  }
  int left = begin(), st = 0;
  if (left > 0) {
    asm volatile("" ::: "memory");
    if constexpr (DIRECT)
      wait_stages<S - 1, PER, 0>(ahead - 1);
    else
      __builtin_amdgcn_s_waitcnt(0xC07F);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
#pragma unroll
    for (int j = 0; j < TN; ++j) read_b(j, 0, first);
#pragma unroll
    for (int i = 0; i < TM; ++i) read_a(i, 0, first);
    clear();
  }
  // the second step's products but for the first row's, the next stage's first reads and, if `load`, a stage's loads
  auto second_step = [&](int next, bool load) QB_INLINE {
    read_a(0, next, first);
#pragma unroll
    for (int i = 1; i < TM; ++i) {
      if (load) {
#pragma unroll
        for (int v = (i - 1) * 2 * PW / (TM - 1); v < i * 2 * PW / (TM - 1); ++v) issue_plain(v, st);
      }
#pragma unroll
      for (int j = (i - 1) * TN / (TM - 1); j < i * TN / (TM - 1); ++j) read_b(j, next, first);
      multiply(i, second);
      read_a(i, next, first);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  while (left > 0) {
#pragma unroll
    for (int i = 0; i < TM; ++i) {
#pragma unroll
      for (int j = i * TN / TM; j < (i + 1) * TN / TM; ++j) read_b(j, st, second);
      multiply(i, first);
      read_a(i, st, second);
      __builtin_amdgcn_sched_barrier(0);
    }
    multiply(0, second);
    put();  // (the place was read before the last barrier)
    // this wave's reads of this stage, its loads of the next
    asm volatile("" ::: "memory");
    if constexpr (!DIRECT)
      __builtin_amdgcn_s_waitcnt(0xC07F);
    else if (behind > 0)
      wait_stages<S - 2, PER, STORES>(ahead - 2);
    else
      wait_stages<S - 2, PER, 0>(ahead - 2);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    behind -= behind > 0;
    take_rows();
    // (behind the last stage the reads find an old one, which nothing multiplies)
    const int next = st + 1 < S ? st + 1 : 0;
    const bool load = plain();
    if (!load && more) issue(st);
    second_step(next, load);
    if (load) issue_scales(st);
    if (more)
      next_stage();
    else
      --ahead;
    st = next;
    if (--left == 0) {
      behind = store(now) ? S - 1 : 0;
      left = begin();
      if constexpr (SQUARE) {
        // What was read of the next tile is read again (an old stage, behind the last one): kept, it would not leave
        // the registers that the addends need.
#pragma unroll
        for (int j = 0; j < TN; ++j) read_b(j, st, first);
#pragma unroll
        for (int i = 0; i < TM; ++i) read_a(i, st, first);
      }
      clear();
    }
  }
  __builtin_amdgcn_s_waitcnt(vm_count(0));  // no load may land after the LDS has changed hands
}

}  // namespace qbk
