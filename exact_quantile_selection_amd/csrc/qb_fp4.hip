// qb_fp4.hip -- matrix products in 4-bit floating point (e2m1: 0, 0.5, 1, 1.5,
// 2, 3, 4, 6 and their negatives) with a power-of-two scale for each block of
// 32, for one weight matrix and for one matrix per expert.
//
// Quantising a row: for each 32 consecutive values the least whole e >= -126
// with max|x| <= 6 * 2^e, stored as e + 127 in 8 bits; the values are x 2^-e
// rounded to nearest even, which the conversion instruction does (checked on
// the GPU against every bf16 pattern).  A block that holds a NaN or an infinity
// has the scale 255, with which every product of it is NaN.
//
// Product: y[m][n] = sum_c x[m][c] w_e[n][c] on v_mfma_scale_f32_16x16x128_f8f6f4,
// four times bf16's rate, whose scale operands are these bytes, one for each 32
// values a lane supplies.  All products of a block are multiples of a quarter
// below 2^6, and sums are held in 32 bits, across blocks too, unlike with 8-bit
// operands; so there is one way to multiply, and it is exact to 32 bits.
#include "qb_gemm16.hpp"

namespace qbk {

// ---------------------------------------------------------------------------
// quantising

// The exponent byte of a block whose largest |x| has the float pattern `top`
// (sign cleared), 255 if that is no finite number.
__device__ __forceinline__ int scale_byte4(uint32_t top) {
  // 6 = 1.5 * 2^2: one more power when the fraction is above 0.5
  const int e = int(top >> 23) - 127 - 2 + ((top & 0x7FFFFFu) > 0x400000u ? 1 : 0);
  return top >= 0x7F800000u ? 255 : (e < -126 ? -126 : e) + 127;
}
// 2^e of such a byte (255: any).
__device__ __forceinline__ float scale_of(int byte) { return __builtin_bit_cast(float, uint32_t(byte == 255 ? 254 : byte) << 23); }

// Four values' codes in 16 bits, the first lowest.
__device__ __forceinline__ uint32_t to_e2m1x4(float a, float b, float c, float d, float scale) {
  uint32_t r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, a, b, scale, 0);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, c, d, scale, 1) & 0xFFFFu;
}

// A wave takes 512 columns of U rows, 4 lanes a block.  Bound by its 2 bytes in
// and 17/32 out a value: 131,072 rows of 2048 by number of 16,384 98 us (what is
// read comes from the last cache), 65,536 in order 74 us, 4.6 TB/s.
template <int U, bool SHORT>
__global__ __launch_bounds__(256) void k_fp4_quantize(const uint16_t* __restrict__ x, int64_t Mx,
                                                      const int32_t* __restrict__ row_src, int64_t M, int C, int64_t ld,
                                                      int64_t sld, uint8_t* __restrict__ xq, uint8_t* __restrict__ xs) {
  const int lane = threadIdx.x & 63;
  const int64_t r0 = (int64_t(blockIdx.x) * 4 + (threadIdx.x >> 6)) * U;
  const int c0 = int(blockIdx.y) * 512 + lane * 8;
  uint4 v[U];
  bool out[U];  // a row of zeros
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t r = r0 + u;
    int64_t src = r < M ? r : -1;
    if (row_src && src >= 0) {
      src = row_src[r];
      if (src >= Mx) src = -1;
    }
    const uint16_t* row = x + (src >= 0 ? src : 0) * C;
    v[u] = SHORT ? ld_short(row, c0, src >= 0 ? C : 0) : ld_inside(row, c0, C);
    out[u] = src < 0;
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t r = r0 + u;
    if (!SHORT && (out[u] || c0 + 8 > C)) v[u] = in_place(v[u], out[u] ? 8 : missing(c0, C));
    const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = w[i] & 0x7FFFu, hi = (w[i] >> 16) & 0x7FFFu;
      top = top > lo ? top : lo;
      top = top > hi ? top : hi;
    }
    auto join = [&](int o) { top = top > uint32_t(o) ? top : uint32_t(o); };
    join(__builtin_amdgcn_mov_dpp(int(top), kQuadXor1, 0xF, 0xF, true));
    join(__builtin_amdgcn_mov_dpp(int(top), kQuadXor2, 0xF, 0xF, true));
    const int byte = scale_byte4(top << 16);
    const float f = scale_of(byte);
    if (r < M && c0 < 2 * ld) {
      auto lo = [&](int i) { return __builtin_bit_cast(float, w[i] << 16); };
      auto hi = [&](int i) { return __builtin_bit_cast(float, w[i] & 0xFFFF0000u); };
      const uint32_t o = to_e2m1x4(lo(0), hi(0), lo(1), hi(1), f) | to_e2m1x4(lo(2), hi(2), lo(3), hi(3), f) << 16;
      *reinterpret_cast<uint32_t*>(xq + r * ld + c0 / 2) = o;
      if ((lane & 3) == 0) xs[r * sld + c0 / 32] = uint8_t(byte);
    }
  }
}

int launch_fp4_quantize(const uint16_t* x, int64_t Mx, const int32_t* row_src, int64_t M, int C, uint8_t* xq,
                        uint8_t* xs, hipStream_t st) {
  const unsigned chunks = unsigned((C + 511) / 512);
  // Four rows a wave once that still gives every CU its waves: rows by number wait twice, for their numbers and for
  // themselves (131,072 of 2048 values 91 us against 107 with one, as they were timed together; in order 74 against 70).
  const bool four = M * chunks >= 16 * 1024;
  const dim3 grid{unsigned(four ? (M + 15) / 16 : (M + 3) / 4), chunks, 1u};
  if (C < 8 || Mx == 0)
    hipLaunchKernelGGL((k_fp4_quantize<1, true>), dim3(unsigned((M + 3) / 4), chunks), dim3(256), 0, st, x, Mx, row_src, M,
                       C, fp4_ld(C), fp4_sld(C), xq, xs);
  else if (four)
    hipLaunchKernelGGL((k_fp4_quantize<4, false>), grid, dim3(256), 0, st, x, Mx, row_src, M, C, fp4_ld(C), fp4_sld(C), xq,
                       xs);
  else
    hipLaunchKernelGGL((k_fp4_quantize<1, false>), grid, dim3(256), 0, st, x, Mx, row_src, M, C, fp4_ld(C), fp4_sld(C), xq,
                       xs);
  return int(hipGetLastError());
}

// A weight stack in one order or both: a workgroup takes 64 rows x 128 columns
// of one matrix, so that four of them share a CU.  Along the rows a thread holds
// 4 columns of 8 rows, 8 lanes a block; for the other order the values cross
// through LDS (rows of 129 words), and a thread takes 32 rows of a column.
// Bound by the 4 bytes in: 64 matrices of 1024 x 2048 in both orders 164 us, 4.1
// TB/s; with 128 x 128 a workgroup, two to a CU, 236.
template <bool BOTH>
__global__ __launch_bounds__(256) void k_fp4_quantize_weight(const float* __restrict__ w, int N, int C, int64_t ldc,
                                                             int64_t sldc, int64_t ldn, int64_t sldn,
                                                             uint8_t* __restrict__ wq, uint8_t* __restrict__ ws,
                                                             uint8_t* __restrict__ wt, uint8_t* __restrict__ wts) {
  constexpr int ROWS = 64;
  __shared__ float vals[BOTH ? ROWS * 129 : 1];
  const int tid = threadIdx.x, cg = tid & 31, rg = tid >> 5;
  const int across = int(ldc / 64), bx = int(blockIdx.x % unsigned(across)), by = int(blockIdx.x / unsigned(across));
  const int c0 = bx * 128 + cg * 4, n0 = by * ROWS;
  const int64_t g = blockIdx.y;
#pragma unroll
  for (int u = 0; u < ROWS / 8; ++u) {
    const int row = rg + 8 * u, n = n0 + row;
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    if (n < N) {
      const float* p = w + (g * N + n) * C + c0;
      if (c0 + 3 < C) {
        const Float4 t = *reinterpret_cast<const Float4*>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = t.v[i];
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = c0 + i < C ? p[i] : 0.f;
      }
    }
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t a = __builtin_bit_cast(uint32_t, v[i]) & 0x7FFFFFFFu;
      top = top > a ? top : a;
      if constexpr (BOTH) vals[row * 129 + cg * 4 + i] = v[i];
    }
    auto join = [&](int o) { top = top > uint32_t(o) ? top : uint32_t(o); };
    join(__builtin_amdgcn_mov_dpp(int(top), kQuadXor1, 0xF, 0xF, true));
    join(__builtin_amdgcn_mov_dpp(int(top), kQuadXor2, 0xF, 0xF, true));
    join(__builtin_amdgcn_mov_dpp(int(top), kHalfMirror, 0xF, 0xF, true));
    const int byte = scale_byte4(top);
    if (n < N && c0 < 2 * ldc) {
      *reinterpret_cast<uint16_t*>(wq + (g * N + n) * ldc + c0 / 2) =
          uint16_t(to_e2m1x4(v[0], v[1], v[2], v[3], scale_of(byte)));
      if ((cg & 7) == 0) ws[(g * N + n) * sldc + c0 / 32] = uint8_t(byte);
    }
  }
  if constexpr (BOTH) {
    __syncthreads();
    {
      const int col = tid & 127, blk = tid >> 7, c = bx * 128 + col;
      float v[32];
      uint32_t top = 0;
#pragma unroll
      for (int k = 0; k < 32; ++k) {
        v[k] = vals[(blk * 32 + k) * 129 + col];
        const uint32_t a = __builtin_bit_cast(uint32_t, v[k]) & 0x7FFFFFFFu;
        top = top > a ? top : a;
      }
      const int byte = scale_byte4(top);
      const float f = scale_of(byte);
      uint32_t o[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        o[k] = to_e2m1x4(v[8 * k], v[8 * k + 1], v[8 * k + 2], v[8 * k + 3], f) |
               to_e2m1x4(v[8 * k + 4], v[8 * k + 5], v[8 * k + 6], v[8 * k + 7], f) << 16;
      const int n = n0 + blk * 32;
      if (c < C && n < 2 * ldn) {
        *reinterpret_cast<uint4*>(wt + (g * C + c) * ldn + n / 2) = make_uint4(o[0], o[1], o[2], o[3]);
        wts[(g * C + c) * sldn + n / 32] = uint8_t(byte);
      }
    }
  }
}

int launch_fp4_quantize_weight(const float* w, int G, int N, int C, uint8_t* wq, uint8_t* ws, uint8_t* wt,
                               uint8_t* wts, hipStream_t st) {
  // rows of 256 values, and columns of them in the other order: both whole
  const int64_t blocks = fp4_ld(C) / 64 * (wt ? fp4_ld(N) / 32 : (N + 63) / 64);
  if (blocks > INT32_MAX / 256) return int(hipErrorInvalidValue);
  const dim3 grid{unsigned(blocks), unsigned(G)};
  if (wt)
    hipLaunchKernelGGL(k_fp4_quantize_weight<true>, grid, dim3(256), 0, st, w, N, C, fp4_ld(C), fp4_sld(C), fp4_ld(N),
                       fp4_sld(N), wq, ws, wt, wts);
  else
    hipLaunchKernelGGL(k_fp4_quantize_weight<false>, grid, dim3(256), 0, st, w, N, C, fp4_ld(C), fp4_sld(C), fp4_ld(N),
                       fp4_sld(N), wq, ws, wt, wts);
  return int(hipGetLastError());
}

// ---------------------------------------------------------------------------
// the product of few rows

// Bound by the weight's bytes, or for the smallest calls by the chain of their
// waits: a workgroup of 8 waves takes 16 MT rows and 16 * 8 / KW columns; KW
// waves share a column tile's K, 256 values at a time, and join their sums
// through LDS in order.  Lane l takes 32 contiguous bytes of row l % 16, two
// blocks of 32 and their two exponents.  1 x 4096 x 4096: 6.2 us.
template <int MT, int KW>
__global__ __launch_bounds__(512) void k_fp4_thin(const uint8_t* __restrict__ A, const uint8_t* __restrict__ As,
                                                  const uint8_t* __restrict__ Bm, const uint8_t* __restrict__ Bs,
                                                  int64_t M, int N, int64_t ld, int64_t sld,
                                                  const int32_t* __restrict__ off, int G, uint16_t* __restrict__ out) {
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
    Bm += int64_t(g.e) * N * ld;
    Bs += int64_t(g.e) * N * sld;
  } else {
    m0 = int64_t(int(blockIdx.x) / tn_all) * BM;
    n0 = (int(blockIdx.x) % tn_all) * BN;
    m_end = M;
  }
  const int r = lane & 15, g4 = lane >> 4;
  const int KB = int(ld / 128);
  const int ncol = n0 + wn * 16;
  const int64_t brow = ncol + r < N ? ncol + r : N - 1;
  const uint8_t *bp = Bm + brow * ld + g4 * 32, *bsp = Bs + brow * sld + g4 * 2;
  const uint8_t *ap[MT], *asp[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    int64_t row = m0 + 16 * i + r;
    row = row < m_end ? row : m_end - 1;
    ap[i] = A + row * ld + g4 * 32;
    asp[i] = As + row * sld + g4 * 2;
  }
  v4f acc[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) acc[i] = (v4f){0.f, 0.f, 0.f, 0.f};
  for (int kb = wk; kb < KB; kb += KW * U) {
    v8s b[U][2], a[U][MT][2];
    int bs[U], as[U][MT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = kb + u * KW, kc = k < KB ? k : kb;  // past the end: re-read, and not used
#pragma unroll
      for (int h = 0; h < 2; ++h) b[u][h] = *reinterpret_cast<const v8s*>(bp + int64_t(kc) * 128 + h * 16);
      bs[u] = *reinterpret_cast<const uint16_t*>(bsp + int64_t(kc) * 8);
#pragma unroll
      for (int i = 0; i < MT; ++i) {
#pragma unroll
        for (int h = 0; h < 2; ++h) a[u][i][h] = *reinterpret_cast<const v8s*>(ap[i] + int64_t(kc) * 128 + h * 16);
        as[u][i] = *reinterpret_cast<const uint16_t*>(asp[i] + int64_t(kc) * 8);
      }
    }
    __builtin_amdgcn_sched_barrier(0);  // (all of them before the first product)
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (kb + u * KW < KB) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < MT; ++i) acc[i] = mma4(b[u][h], a[u][i][h], acc[i], bs[u] >> (8 * h), as[u][i] >> (8 * h));
      }
  }
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
    Half4 t;
    t.v[0] = bf16x2_rne(acc[i][0], acc[i][1]);
    t.v[1] = bf16x2_rne(acc[i][2], acc[i][3]);
    if (col + 3 < N) {
      *reinterpret_cast<Half4*>(o) = t;
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (col + c < N) o[c] = uint16_t(t.v[c >> 1] >> (16 * (c & 1)));
    }
  }
}

// ---------------------------------------------------------------------------

static int64_t row_tiles(const Gemm16& g, int BM) {
  return g.off ? g.M / BM + std::min(g.G, g.M) : (g.M + BM - 1) / BM;
}

// 8192 x 8192 x 4096: 151 us, 3.6 PFLOP/s, the matrix units busy 39% of the CUs' cycles (bf16: 64%): a stage has as many
// products as in bf16, each as long, and twelve reads of exponents a step more, and a tile a fourth of the stages beside
// which its results leave.  131,072 rows over 64 experts of 1024 x 2048 232 us, 2.4 PFLOP/s, busy 31%: 8 stages a tile
// (in 128 x 128, two to a CU, 262; 65,536 rows of 2048 x 1024 150 against 170).
template <int B, int S>
static int tiled(Gemm16 g, hipStream_t st) {
  const int64_t tiles = row_tiles(g, B) * ((g.N + B - 1) / B);
  if (tiles > INT32_MAX / 2) return int(hipErrorInvalidValue);
  g.tiles = int(tiles);
  const int64_t most = int64_t(device_cu_count()) * (B == 256 ? 1 : 2);
  hipLaunchKernelGGL((k_gemm16<Fp4, kRows, false, false, B, S, true>), dim3(unsigned(std::min(tiles, most))),
                     dim3(B == 256 ? 512 : 256), 0, st, g);
  return int(hipGetLastError());
}

template <int MT, int KW>
static int thin(const Gemm16& g, hipStream_t st) {
  constexpr int BN = 16 * (8 / KW);
  const int64_t blocks = row_tiles(g, 16 * MT) * ((g.N + BN - 1) / BN);
  if (blocks > INT32_MAX) return int(hipErrorInvalidValue);
  hipLaunchKernelGGL((k_fp4_thin<MT, KW>), dim3(unsigned(blocks)), dim3(512), 0, st,
                     reinterpret_cast<const uint8_t*>(g.A), g.As, reinterpret_cast<const uint8_t*>(g.B), g.Bs, g.M, g.N,
                     2 * g.lda, g.sld, g.off, g.G, static_cast<uint16_t*>(g.out));
  return int(hipGetLastError());
}

template <int MT>
static int few(const Gemm16& g, hipStream_t st) {
  const int64_t waves = row_tiles(g, 16 * MT) * ((g.N + 15) / 16);
  // (32 rows come here with two waves a CU at most)
  int kw = MT == 2 ? 4 : g.K >= 8 * 64 ? 2 : 1;
  while (kw < 8 && waves * kw < 8 * int64_t(device_cu_count())) kw *= 2;
  if constexpr (MT == 1) {
    if (kw == 1) return thin<MT, 1>(g, st);
    if (kw == 2) return thin<MT, 2>(g, st);
  }
  return kw == 4 ? thin<MT, 4>(g, st) : thin<MT, 8>(g, st);
}

int launch_fp4_product(const uint8_t* xq, const uint8_t* xs, const uint8_t* w, const uint8_t* ws, int M, int N, int C,
                       const int32_t* off, int G, uint16_t* y, hipStream_t st) {
  Gemm16 g{};
  g.A = reinterpret_cast<const uint16_t*>(xq);
  g.B = reinterpret_cast<const uint16_t*>(w);
  g.As = xs;
  g.Bs = ws;
  g.lda = g.ldb = fp4_ld(C) / 2;  // in 16-bit words, of which K has so many: whole stages
  g.K = int(fp4_ld(C) / 2);
  g.sld = fp4_sld(C);
  g.mat_b = int64_t(N) * g.ldb;
  g.mat_bs = int64_t(N) * g.sld;
  g.M = M;
  g.N = N;
  g.off = off;
  g.G = G;
  g.splits = 1;
  g.out = y;
  const int rows = off ? (M + G - 1) / G : M;  // rows of an expert, on average
  auto tiles = [&](int b) { return row_tiles(g, b) * ((N + b - 1) / b); };
  const int64_t cu = device_cu_count();
  // The kernel of few rows while a workgroup for each 16 columns, two a CU, shares out K (64 x 1024 x 4096: 6.5 us against
  // 11 in tiles of 64 x 64, 128 x 4096 x 4096 18 against 11.5; 128 rows over 256 experts of 1024 x 2048 34 against 27), and
  // for very few rows of one matrix (1 x 16,384 x 4096 8.9 against 11.4).
  if (row_tiles(g, rows <= 16 ? 16 : 32) * ((N + 15) / 16) <= 2 * cu || (!off && rows <= 4))
    return rows <= 16 ? few<1>(g, st) : few<2>(g, st);
  // As the bf16 products: experts of so few rows fill half of a large tile at most (5120 rows over 40 experts of 1024 x
  // 2048 18.6 us in 128 x 128, 23 in 256 x 256), and a third of ragged experts' tiles of 64 rows is taken to be missing
  // (2000 rows over 16 experts of 700 x 1160 8.9 us in 64 x 64, 10.9 in 128 x 128; of 1400 x 1024 12.1 and 10.8).
  const int64_t t256 = rows <= 128 && off ? 0 : tiles(256);
  if ((off ? tiles(64) * 2 / 3 : tiles(64)) <= 2 * cu) return tiled<64, 4>(g, st);
  if (in_large_tiles(t256, tiles(128), off ? 0.1 : 0.0)) return tiled<256, 2>(g, st);
  return tiled<128, 2>(g, st);
}

}  // namespace qbk
