// qb_bf16.hip -- the experts' products in bfloat16: forward, the gradient of
// the rows and that of the matrices, over ragged stretches of rows.
//
//   y[m][n]    = sum_c x[src m][c] w_e[n][c]      (e: m's expert)
//   dx[m][c]   = sum_n dy[m][n] w_e[n][c]         (the same w, read across its rows)
//   dw_e[n][c] = sum_{m of e} dy[m][n] x[src m][c]
//
// Products of two bf16 values are exact in 32 bits and every sum is held there,
// rounded once on the way out (y, dx) or not at all (dw).
#include "qb_gemm16.hpp"

namespace qbk {

// ---------------------------------------------------------------------------
// the product of few rows

// 16 of a row's K values from `at`, in two parts (see ld_inside).
template <bool SHORT, bool WHOLE>
__device__ __forceinline__ void ld_16(const uint16_t* row, int at, int K, uint4 (&v)[2]) {
#pragma unroll
  for (int h = 0; h < 2; ++h)
    v[h] = SHORT ? ld_short(row, at + 8 * h, K) : WHOLE ? ld_half8(row + at + 8 * h) : ld_inside(row, at + 8 * h, K);
}
template <bool SHORT>
__device__ __forceinline__ v8s part_of(const uint4 (&v)[2], int h, int at, int K) {
  return __builtin_bit_cast(v8s, SHORT ? v[h] : in_place(v[h], missing(at + 8 * h, K)));
}

// Bound by the weight's bytes: a workgroup of 8 waves takes 16 MT rows and
// 16 * 8 / KW columns; KW waves share a column tile's K, 64 at a time, so that
// the whole weight is in flight at once, and join their sums through LDS in
// order.  Both operands go from memory to registers: lane l takes 32
// contiguous bytes of row l % 16, four lanes a line.  128 rows over 256 experts
// of 1024 x 2048: 81 us, 5.1 TB/s; 8 rows over 64 of 256 x 512: 5.5 us, a launch
// and one chain of waits.
template <int MT, int KW, bool SHORT>
__global__ __launch_bounds__(512) void k_bf16_thin(const uint16_t* __restrict__ A, int Mx,
                                                   const int32_t* __restrict__ src, const uint16_t* __restrict__ Bm,
                                                   int64_t M, int N, int K, const int32_t* __restrict__ off, int G,
                                                   uint16_t* __restrict__ out) {
  constexpr int NW = 8 / KW, BM = 16 * MT, BN = 16 * NW, U = MT >= 2 ? 2 : 4;
  __shared__ __align__(16) float red[KW > 1 ? 8 : 1][MT][kWave][4];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = wave / KW, wk = wave % KW;
  const int tn_all = (N + BN - 1) / BN;
  int64_t m0, m_end;
  int n0;
  if (off) {
    const int tm = int(blockIdx.x) / tn_all;
    n0 = (int(blockIdx.x) % tn_all) * BN;
    int lo[4], hi[4], n[4], before;
    group_tiles(off, G, M, BM, lane, lo, hi, n, before);
    const Tile g = group_find(tm, lane, lo, hi, n, before);
    if (g.e < 0) return;
    m0 = g.lo + int64_t(g.at) * BM;
    m_end = g.hi;
    Bm += int64_t(g.e) * N * K;
  } else {
    m0 = int64_t(int(blockIdx.x) / tn_all) * BM;
    n0 = (int(blockIdx.x) % tn_all) * BN;
    m_end = M;
  }
  const int r = lane & 15, g4 = lane >> 4;
  const int KB = (K + 63) / 64;
  const int ncol = n0 + wn * 16;
  const int brow = ncol + r < N ? ncol + r : N - 1;
  const uint16_t* bp = Bm + int64_t(brow) * K;
  const uint16_t* ap[MT];
  bool live[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    int64_t row = m0 + 16 * i + r;
    row = row < m_end ? row : m_end - 1;
    if (src) row = src[row];
    live[i] = !src || (row >= 0 && row < Mx);
    ap[i] = A + (live[i] ? row : 0) * K;
  }
  v4f acc[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) acc[i] = (v4f){0.f, 0.f, 0.f, 0.f};
  auto step = [&](int kb, auto whole) {
    constexpr bool WHOLE = decltype(whole)::value;
    uint4 b[U][2], a[U][MT][2];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int at = (kb + u * KW) * 64 + g4 * 16;
      ld_16<SHORT, WHOLE>(bp, at, K, b[u]);
#pragma unroll
      for (int i = 0; i < MT; ++i) ld_16<SHORT, WHOLE>(ap[i], at, K, a[u][i]);
    }
    __builtin_amdgcn_sched_barrier(0);  // (all of them before the first product)
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int at = (kb + u * KW) * 64 + g4 * 16;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < MT; ++i)
          acc[i] = mma16<__bf16>(part_of<SHORT || WHOLE>(b[u], h, at, K), part_of<SHORT || WHOLE>(a[u][i], h, at, K), acc[i]);
    }
  };
  int kb = wk;
  for (; (kb + (U - 1) * KW) * 64 + 64 <= K; kb += KW * U) step(kb, std::true_type{});
  for (; kb < KB; kb += KW * U) step(kb, std::false_type{});  // (past the end: zeros)
  if constexpr (KW > 1) {
#pragma unroll
    for (int i = 0; i < MT; ++i) *reinterpret_cast<v4f*>(&red[wave][i][lane][0]) = acc[i];
    __syncthreads();
    if (wk != 0) return;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int k = 1; k < KW; ++k) acc[i] += *reinterpret_cast<const v4f*>(&red[wave + k][i][lane][0]);
  }
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int64_t row = m0 + 16 * i + r;
    const int col = ncol + g4 * 4;
    if (row >= m_end) continue;
    uint16_t* o = out + row * N + col;
    Half4 t;  // (a row that was routed nowhere was multiplied as row 0)
    t.v[0] = live[i] ? bf16x2_rne(acc[i][0], acc[i][1]) : 0;
    t.v[1] = live[i] ? bf16x2_rne(acc[i][2], acc[i][3]) : 0;
    if (col + 3 < N) {
      *reinterpret_cast<Half4*>(o) = t;
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (col + c < N) o[c] = uint16_t(t.v[c >> 1] >> (16 * (c & 1)));
    }
  }
}

// The parts of a gradient whose sum over rows was split, added in order: bound
// by their bytes, 32 MiB at most.
__global__ __launch_bounds__(256) void k_bf16_join(const float* __restrict__ part, int64_t n, int splits,
                                                   float* __restrict__ out) {
  const int64_t i = (int64_t(blockIdx.x) * 256 + threadIdx.x) * 4;
  if (i >= n) return;
  if (i + 3 < n) {
    Float4 a = *reinterpret_cast<const Float4*>(part + i);
    for (int s = 1; s < splits; ++s) {
      const Float4 b = *reinterpret_cast<const Float4*>(part + s * n + i);
#pragma unroll
      for (int c = 0; c < 4; ++c) a.v[c] += b.v[c];
    }
    *reinterpret_cast<Float4*>(out + i) = a;
  } else {
    for (int64_t j = i; j < n; ++j) {
      float a = part[j];
      for (int s = 1; s < splits; ++s) a += part[s * n + j];
      out[j] = a;
    }
  }
}

// ---------------------------------------------------------------------------

template <int KIND, bool A_KS, bool B_KS, int B, int S, bool DIRECT>
static int tiled(Gemm16 g, hipStream_t st) {
  const int64_t tn = (g.N + B - 1) / B;
  int64_t tm = (g.M + B - 1) / B;
  if (KIND == kRows && g.off) tm = g.M / B + std::min(g.G, g.M);
  const int64_t tiles = KIND == kGrad ? tm * tn * g.G * g.splits : tm * tn;
  if (tiles > INT32_MAX / 2) return int(hipErrorInvalidValue);  // (a tile's number plus a grid's size is an int)
  g.tiles = int(tiles);
  // as many workgroups as run at once (a 256 x 256 tile's ring fills a CU's LDS, the others' half of it)
  const int64_t most = int64_t(device_cu_count()) * (B == 256 ? 1 : B == 64 && !DIRECT ? 4 : 2);
  hipLaunchKernelGGL((k_gemm16<__bf16, KIND, A_KS, B_KS, B, S, DIRECT>), dim3(unsigned(std::min(tiles, most))),
                     dim3(B == 256 ? 512 : 256), 0, st, g);
  return int(hipGetLastError());
}

// Which tile.  The smallest while its tiles all run at once: 776 x 2008 x 1000 takes 13.5 us with them, 15.6 with 128 x
// 128 and 28.8 with 256 x 256; 2048 x 4096 x 1024, of four times as many, 41, 23.6 and 31.  By registers (!DIRECT) one
// stage is in flight whatever the ring, so that four groups with two stages each share a CU there and the bound is twice
// as high (1999 rows over 16 experts of 730 x 1163, rows' gradient: 25 us against 34 with 128 x 128 in two rounds).  256 x
// 256 against 128 x 128: in_large_tiles.
template <int KIND, bool A_KS, bool B_KS>
static int gemm(const Gemm16& g, int64_t t256, int64_t t128, int64_t t64, double uneven, bool direct, hipStream_t st) {
  const int64_t cu = device_cu_count();
  if (t64 <= (direct ? 2 : 4) * cu)
    return direct ? tiled<KIND, A_KS, B_KS, 64, 4, true>(g, st) : tiled<KIND, A_KS, B_KS, 64, 2, false>(g, st);
  if (direct && in_large_tiles(t256, t128, uneven)) return tiled<KIND, A_KS, B_KS, 256, 2, true>(g, st);
  return direct ? tiled<KIND, A_KS, B_KS, 128, 2, true>(g, st) : tiled<KIND, A_KS, B_KS, 128, 2, false>(g, st);
}

template <int MT, int KW>
static int thin(const Gemm16& g, int64_t row_tiles, hipStream_t st) {
  constexpr int BN = 16 * (8 / KW);
  const int64_t blocks = row_tiles * ((g.N + BN - 1) / BN);
  if (blocks > INT32_MAX) return int(hipErrorInvalidValue);
  if (g.K >= 8)
    hipLaunchKernelGGL((k_bf16_thin<MT, KW, false>), dim3(unsigned(blocks)), dim3(512), 0, st, g.A, g.Mx, g.src, g.B, g.M,
                       g.N, g.K, g.off, g.G, static_cast<uint16_t*>(g.out));
  else
    hipLaunchKernelGGL((k_bf16_thin<MT, KW, true>), dim3(unsigned(blocks)), dim3(512), 0, st, g.A, g.Mx, g.src, g.B, g.M,
                       g.N, g.K, g.off, g.G, static_cast<uint16_t*>(g.out));
  return int(hipGetLastError());
}

template <int MT>
static int few(const Gemm16& g, hipStream_t st) {
  const int64_t rt = g.off ? g.M / (16 * MT) + std::min(g.G, g.M) : (g.M + 16 * MT - 1) / (16 * MT);
  const int64_t waves = rt * ((g.N + 15) / 16);
  // (32 rows come here with two waves a CU at most)
  int kw = MT == 2 ? 4 : g.K >= 8 * 64 ? 2 : 1;
  while (kw < 8 && waves * kw < 8 * int64_t(device_cu_count())) kw *= 2;
  if constexpr (MT == 1) {
    if (kw == 1) return thin<MT, 1>(g, rt, st);
    if (kw == 2) return thin<MT, 2>(g, rt, st);
  }
  return kw == 4 ? thin<MT, 4>(g, rt, st) : thin<MT, 8>(g, rt, st);
}

// Rows of 16-byte multiples at 16-byte addresses, within 32-bit offsets of their array's start where they are taken by
// number.
static bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
static bool by_offset(const int32_t* src, int64_t Mx, int64_t C) { return !src || (Mx > 0 && Mx * C * 2 <= (int64_t(1) << 32)); }

int launch_bf16_product(const uint16_t* x, int Mx, const int32_t* src, int M, const uint16_t* w, int N, int C,
                        const int32_t* off, int G, bool transposed, uint16_t* y, hipStream_t st) {
  Gemm16 g{};
  // (x without a row: every row is zeros, and something that may be read stands for them)
  g.A = Mx > 0 ? x : w;
  g.B = w;
  g.lda = C;
  g.ldb = transposed ? N : C;
  g.mat_b = int64_t(N) * C;
  g.M = M;
  g.N = N;
  g.K = C;
  g.src = src;
  g.Mx = Mx;
  g.off = off;
  g.G = G;
  g.splits = 1;
  g.out = y;
  const int rows = off ? (M + G - 1) / G : M;  // rows of an expert, on average
  auto tiles = [&](int b) {
    return (off ? int64_t(M / b) + std::min(G, M) : int64_t(M + b - 1) / b) * ((N + b - 1) / b);
  };
  const bool direct = C % 8 == 0 && (!transposed || N % 8 == 0) && aligned16(x) && aligned16(w) && by_offset(src, Mx, C);
  // The kernel of few rows: while a workgroup for each 16 columns, two a CU, shares out K (64 x 1024 x 4096: 13 us against
  // 28 in tiles of 64 x 64, 64 x 4096 x 4096 24 against 29, 128 x 4096 x 4096 44 against 29), and for very few rows, whose
  // tiles would multiply little else than padding (1 x 16,384 x 4096 27 against 32; 512 rows over 256 experts of 1024 x
  // 2048 167 against 179; 8 rows each of 64 experts 53 against 43), unless experts' rows begin anywhere (256 rows over 64
  // experts of 730 x 1163 60 against 30).  The other order has no such kernel: its few rows run in tiles, K by one workgroup
  // (the gradient of 1 or 16 rows of 4096 x 4096 28 us where the forward product takes 8 and 10, of 4096 x 16,384 103).
  const int few_rows = rows <= 16 ? 16 : 32;
  const int64_t strips =
      (off ? int64_t(M / few_rows) + std::min(G, M) : int64_t(M + few_rows - 1) / few_rows) * ((N + 15) / 16);
  if (!transposed && (strips <= 2 * device_cu_count() || (rows <= 4 && (direct || !off))))
    return rows <= 16 ? few<1>(g, st) : few<2>(g, st);
  // Experts of so few rows fill half of a large tile at most (5120 rows over 40 experts of 1024 x 2048 57 us in 128 x 128,
  // 67 in 256 x 256; 5000 over 40 of 1000 x 2048 57 and 65).
  const int64_t t256 = rows <= 128 && off ? 0 : tiles(256);
  // Of ragged experts' tiles of 64 rows a third is taken to be missing or nearly empty (2000 rows over 16 experts of 700 x
  // 1160 17 us in 64 x 64, 23 in 128 x 128; of 1400 x 1024 22 and 18; near the border the other is up to 14% faster: of
  // 1024 x 1024 19 and 16.6, 1500 over 64 of 768 x 1024 22.4 and 25.6).
  const int64_t t64 = !off ? tiles(64) : tiles(64) * 2 / 3;
  const double uneven = off ? 0.1 : 0.0;
  return transposed ? gemm<kRows, false, true>(g, t256, tiles(128), t64, uneven, direct, st)
                    : gemm<kRows, false, false>(g, t256, tiles(128), t64, uneven, direct, st);
}

int launch_bf16_weight_grad(const uint16_t* dy, const uint16_t* x, int Mx, const int32_t* src, int M, int N, int C,
                            const int32_t* off, int G, float* dw, float* ws, hipStream_t st) {
  Gemm16 g{};
  g.A = dy;
  g.B = Mx > 0 ? x : reinterpret_cast<const uint16_t*>(dw);
  g.lda = N;
  g.ldb = C;
  g.M = N;
  g.N = C;
  g.K = M;
  g.src = src;
  g.Mx = Mx;
  g.off = off;
  g.G = G;
  g.splits = ws ? bf16_grad_splits(M, N, C, G) : 1;
  g.out = g.splits > 1 ? ws : dw;
  auto tiles = [&](int b) { return int64_t(G) * g.splits * ((N + b - 1) / b) * ((C + b - 1) / b); };
  const bool direct = N % 8 == 0 && C % 8 == 0 && aligned16(dy) && aligned16(x) && by_offset(src, Mx, C);
  if (int rc = gemm<kGrad, true, true>(g, tiles(256), tiles(128), tiles(64), off ? 0.25 : 0.0, direct, st)) return rc;
  if (g.splits > 1) {
    const int64_t n = int64_t(G) * N * C;
    hipLaunchKernelGGL(k_bf16_join, dim3(unsigned((n + 1023) / 1024)), dim3(256), 0, st, ws, n, g.splits, dw);
  }
  return int(hipGetLastError());
}

}  // namespace qbk
