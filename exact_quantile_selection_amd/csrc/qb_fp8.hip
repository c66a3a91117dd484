// qb_fp8.hip -- matrix products in 8-bit floating point (e4m3) with a
// power-of-two scale for each block of 128, for one weight matrix and for one
// matrix per expert.
//
// Quantising a row: for each 128 consecutive values the least whole e >= -126
// with max|x| <= 448 * 2^e, stored as e + 127 in 8 bits; the values are
// x 2^-e (exact) rounded to nearest even.  2^e is the matrix instruction's
// own scale operand (v_mfma_scale_f32_16x16x128_f8f6f4 multiplies 32 values
// of each operand's row by one such byte), so a scale costs no arithmetic:
// one instruction's 128 values of K are one block, and all four lanes of a
// row hold its byte.  Sums are held in 32 bits and rounded once on the way
// out.
//
//   product:      y[m][n]  = sum_c x[m][c] w_e[n][c]          (e: m's expert)
//   weight grad:  dw_e[n][c] = sum_{m of e} dy[m][n] x[m][c]
// both as out[a][b] = sum_k A[a][k] B[b][k] of two K-contiguous operands (the
// gradient's operands are quantised along the rows, so that their blocks lie
// along its sum).
//
// Operand layout of the instruction (checked on the GPU): lane l supplies 32
// of the 128 values of row l % 16 of either operand, the same ones of both;
// which 32 is free as long as A and B agree.  Result element i of lane l is
// C[row 4 (l / 16) + i of the first operand][row l % 16 of the second].
//
// How exactly it adds (measured with single values, on the GPU): the eight
// products of a group are aligned to the largest of them and what lies more
// than 2^-13 below it is dropped; groups, and the running sum, are added in 32
// bits.  All 8-bit matrix instructions of this GPU do so, the 16-bit ones do
// not.  So there are two ways to multiply, with the same tiles:
//   * EXACT: both operands widened in registers to bf16 (e4m3 times its
//     scale is exact there from 2^-133 up and below 2^128), whose instruction
//     adds products in full: every sum in 32 bits, half the peak rate.  What a call does unless told
//     otherwise; the weight gradient, whose result keeps 32 bits, and the
//     products of few rows, where the weight's bytes cost more than either
//     instruction, know no other way.
//   * the 8-bit instruction, where the caller allows it: up to 2^-10 of sum
//     |a b| is lost, unseen beside a bf16 result's own 2^-8 unless the sum
//     cancels (256 and -256 among each eight products, the others 2^-9: not
//     one bit of a result is right).
// Large products are bound by the matrix units as the loop feeds them, at the
// clock that the card holds under them: 8192 x 8192 x 4096 takes 412 to 448 us
// (1.2 to 1.3 PFLOP/s; the vendor library's bf16 product 433), its weight
// gradient 405 to 431, and with the 8-bit instruction 231 to 272 (2.0 to 2.4;
// the vendor's plain e4m3 product 227).  What the last spent 229 us on, by
// leaving work out: without the loads 216, without seven eighths of the LDS
// reads of A too 200, with a quarter of the products 165: the products and the
// operands' way overlap to within 15%.
#include <algorithm>
#include <type_traits>

#include "qb_device.hpp"
#include "qb_internal.hpp"

namespace qbk {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef int v4i __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void* lds_vptr;
typedef __attribute__((address_space(1))) void* glb_vptr;

struct __attribute__((packed, aligned(2))) Half8 {
  uint32_t v[4];
};
struct __attribute__((packed, aligned(2))) Half4 {
  uint32_t v[2];
};
struct __attribute__((packed, aligned(4))) Float4 {
  float v[4];
};

// ---------------------------------------------------------------------------
// quantising

// 8 bf16 of a row from p, of which n lie inside it; the others are zero.
// NT: past the caches.
template <bool NT>
__device__ __forceinline__ void ld_half8(const uint16_t* p, int n, uint32_t (&v)[4]) {
  if (n >= 8) {
    typedef uint32_t half8 __attribute__((ext_vector_type(4), aligned(2)));
    const half8* q = reinterpret_cast<const half8*>(p);
    const half8 t = NT ? __builtin_nontemporal_load(q) : *q;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = t[i];
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = 2 * i < n ? p[2 * i] : 0, hi = 2 * i + 1 < n ? p[2 * i + 1] : 0;
      v[i] = lo | (hi << 16);
    }
  }
}

// The exponent byte of a block whose largest |x| has the bf16 pattern `top`
// (sign cleared; patterns order as values do, NaN above infinity).
__device__ __forceinline__ int scale_byte(uint32_t top) {
  // 448 = 1.75 * 2^8: one more power when the fraction is above 0.75
  const int e = int(top >> 7) - 127 - 8 + ((top & 0x7Fu) > 0x60u ? 1 : 0);
  return (e < -126 ? -126 : e) + 127;
}
// 2^-e of such a byte; e <= 120 for finite blocks, so it is a normal float.
__device__ __forceinline__ float scale_down(int byte) {
  return __builtin_bit_cast(float, uint32_t(254 - byte) << 23);
}
__device__ __forceinline__ float half_lo(uint32_t p) { return __builtin_bit_cast(float, p << 16); }
__device__ __forceinline__ float half_hi(uint32_t p) { return __builtin_bit_cast(float, p & 0xFFFF0000u); }

// Four values to e4m3 bytes (nearest even).  bad: the block holds a NaN or an
// infinity; those values become NaN, as a cast of them does.
__device__ __forceinline__ uint32_t to_e4m3x4(float a, float b, float c, float d, bool bad) {
  int r = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  r = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, r, true);
  if (bad) {
    uint32_t u = uint32_t(r);
    const float inf = __builtin_inff();
    if (!(fabsf(a) < inf)) u = (u & ~0xFFu) | 0x7Fu;
    if (!(fabsf(b) < inf)) u = (u & ~0xFF00u) | 0x7F00u;
    if (!(fabsf(c) < inf)) u = (u & ~0xFF0000u) | 0x7F0000u;
    if (!(fabsf(d) < inf)) u = (u & ~0xFF000000u) | 0x7F000000u;
    return u;
  }
  return uint32_t(r);
}

__device__ __forceinline__ uint32_t abs_max2(uint32_t m, uint32_t p) {
  const uint32_t lo = p & 0x7FFFu, hi = (p >> 16) & 0x7FFFu;
  m = m > lo ? m : lo;
  return m > hi ? m : hi;
}

// Along the rows: a wave takes 512 columns (one word of four scales) of U
// rows, 16 lanes a block.  Bound by its 2 bytes in, 1 byte out a value:
// 135,000 x 2048 take 146 us, 5.7 TB/s (a copy reaches 5.1 in cached accesses).
// Taken by row_src from 16,384 rows, 139,000 of them take 102.
template <int U, bool NT>
__global__ __launch_bounds__(256) void k_fp8_quantize(const uint16_t* __restrict__ x, int64_t Mx,
                                                      const int32_t* __restrict__ row_src, int64_t M, int C,
                                                      uint8_t* __restrict__ xq, uint8_t* __restrict__ xs) {
  const int lane = threadIdx.x & 63;
  const int chunks = int(gridDim.y);
  const int64_t r0 = (int64_t(blockIdx.x) * 4 + (threadIdx.x >> 6)) * U;
  const int c0 = int(blockIdx.y) * 512 + lane * 8;
  const int64_t ld = (int64_t(C) + kQBlock - 1) / kQBlock * kQBlock;
  uint32_t v[U][4];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t r = r0 + u;
    int64_t src = r < M ? r : -1;
    if (row_src && src >= 0) {
      src = row_src[r];
      if (src >= Mx) src = -1;
    }
    if (src >= 0 && c0 < C) {
      ld_half8<NT>(x + src * C + c0, C - c0, v[u]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[u][i] = 0;
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t r = r0 + u;
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) top = abs_max2(top, v[u][i]);
    auto join = [&](int o) { top = top > uint32_t(o) ? top : uint32_t(o); };
    join(__builtin_amdgcn_mov_dpp(int(top), kQuadXor1, 0xF, 0xF, true));
    join(__builtin_amdgcn_mov_dpp(int(top), kQuadXor2, 0xF, 0xF, true));
    join(__builtin_amdgcn_mov_dpp(int(top), kHalfMirror, 0xF, 0xF, true));
    join(__builtin_amdgcn_mov_dpp(int(top), 0x140, 0xF, 0xF, true));  // row_mirror: lane i of 16 reads lane 15 - i
    const int byte = scale_byte(top);
    const float f = scale_down(byte);
    const bool bad = top >= 0x7F80u;
    if (r < M) {
      if (c0 < ld) {
        uint2 o;
        o.x = to_e4m3x4(half_lo(v[u][0]) * f, half_hi(v[u][0]) * f, half_lo(v[u][1]) * f, half_hi(v[u][1]) * f, bad);
        o.y = to_e4m3x4(half_lo(v[u][2]) * f, half_hi(v[u][2]) * f, half_lo(v[u][3]) * f, half_hi(v[u][3]) * f, bad);
        *reinterpret_cast<uint2*>(xq + r * ld + c0) = o;
      }
      if ((lane & 15) == 0) xs[r * (int64_t(chunks) * 4) + int(blockIdx.y) * 4 + (lane >> 4)] = uint8_t(byte);
    }
  }
}

// Lane l ^ D's word, D 16 or 32 (the instruction exchanges the D-lane halves of
// two registers: one result is the own word, the other the partner's).
template <int D>
__device__ __forceinline__ uint32_t swapped(uint32_t a) {
  uint32_t b = a;
  asm volatile("" : "+v"(b));  // two registers: with one and the same operand the compiler takes the results as equal
  const auto h = D == 16 ? __builtin_amdgcn_permlane16_swap(a, b, false, false)
                         : __builtin_amdgcn_permlane32_swap(a, b, false, false);
  return threadIdx.x & D ? h[0] : h[1];
}

// Along the columns: a workgroup takes 128 rows (one block) of 64 columns and
// writes them transposed, 128 contiguous bytes a column.  A thread holds 8
// columns of 4 consecutive rows, so that a column's 4 bytes are one word; the
// words cross to the columns' order through LDS (33 words a column: the 64
// lanes of a store lie in 64 banks).  Bound like the one along the rows: 156 us
// for the same matrix, 125 gathered.
template <bool NT>
__global__ __launch_bounds__(256) void k_fp8_quantize_cols(const uint16_t* __restrict__ x, int64_t Mx,
                                                           const int32_t* __restrict__ row_src, int64_t M, int C,
                                                           int64_t ld, int64_t sld, uint8_t* __restrict__ xt,
                                                           uint8_t* __restrict__ xts) {
  __shared__ uint32_t tops[4][64];
  __shared__ uint32_t words[64 * 33];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int cg = tid & 7, rg = tid >> 3;
  const int64_t blk = int64_t(blockIdx.y);
  const int64_t r0 = blk * kQBlock + rg * 4;
  const int cbase = int(blockIdx.x) * 64, c0 = cbase + cg * 8;
  uint32_t v[4][4];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int64_t r = r0 + u;
    int64_t src = r < M ? r : -1;
    if (row_src && src >= 0) {
      src = row_src[r];
      if (src >= Mx) src = -1;
    }
    if (src >= 0 && c0 < C) {
      ld_half8<NT>(x + src * C + c0, C - c0, v[u]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[u][i] = 0;
    }
  }
  uint32_t top[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    top[2 * i] = top[2 * i + 1] = 0;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint32_t lo = v[u][i] & 0x7FFFu, hi = (v[u][i] >> 16) & 0x7FFFu;
      top[2 * i] = top[2 * i] > lo ? top[2 * i] : lo;
      top[2 * i + 1] = top[2 * i + 1] > hi ? top[2 * i + 1] : hi;
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    auto join = [&](uint32_t o) { top[j] = top[j] > o ? top[j] : o; };
    join(uint32_t(__builtin_amdgcn_mov_dpp(int(top[j]), 0x128, 0xF, 0xF, true)));  // row_ror:8
    join(swapped<16>(top[j]));
    join(swapped<32>(top[j]));
    if (lane < 8) tops[wave][cg * 8 + j] = top[j];
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    uint32_t t = tops[0][cg * 8 + j];
#pragma unroll
    for (int w = 1; w < 4; ++w) t = t > tops[w][cg * 8 + j] ? t : tops[w][cg * 8 + j];
    const int byte = scale_byte(t);
    const float f = scale_down(byte);
    float a[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) a[u] = ((j & 1) ? half_hi(v[u][j >> 1]) : half_lo(v[u][j >> 1])) * f;
    words[(cg * 8 + j) * 33 + rg] = to_e4m3x4(a[0], a[1], a[2], a[3], t >= 0x7F80u);
    if (rg == 0 && c0 + j < C) xts[(c0 + j) * sld + blk] = uint8_t(byte);
  }
  __syncthreads();
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int i = h * 256 + tid, col = i >> 3, part = i & 7;
    if (cbase + col < C) {
      uint4 o;
      const uint32_t* src = words + col * 33 + part * 4;
      o.x = src[0], o.y = src[1], o.z = src[2], o.w = src[3];
      *reinterpret_cast<uint4*>(xt + int64_t(cbase + col) * ld + blk * kQBlock + part * 16) = o;
    }
  }
}

// An input of half the last cache (256 MiB) or more, which the results push
// out of it, passes it by (135,000 rows of 2048: along the rows 169 -> 145 us,
// along the columns 177 -> 157; 8192 of 8192: 53 -> 50 and 50 -> 47; 8192 of
// 4096: 25 -> 23 but 23 -> 25).  Unless its rows are read again: taken by
// row_src for 2 experts each and more, the caches serve them better at every
// size (past them -> through them: 16,384 rows of 2048 for 8 experts each 140 ->
// 117 and 163 -> 138; 32,768 for 8 355 -> 234 and 352 -> 298; 131,072 for 2 391
// -> 304 and 361 -> 335; but 262,144 of 1024 for one 132 -> 161, 164 -> 185).
static bool past_caches(int64_t Mx, int64_t M, int C) { return M < 2 * Mx && Mx * C * 2 >= (int64_t(128) << 20); }

int launch_fp8_quantize(const uint16_t* x, int64_t Mx, const int32_t* row_src, int64_t M, int C, uint8_t* xq,
                        uint8_t* xs, hipStream_t st) {
  const unsigned chunks = unsigned(fp8_sld(C) / 4);
  // four rows a wave once that still gives every CU its waves
  const bool four = M * chunks >= 16 * 1024;
  const dim3 grid{unsigned(four ? (M + 15) / 16 : (M + 3) / 4), chunks, 1u};
  if (four && past_caches(Mx, M, C))
    hipLaunchKernelGGL((k_fp8_quantize<4, true>), grid, dim3(256), 0, st, x, Mx, row_src, M, C, xq, xs);
  else if (four)
    hipLaunchKernelGGL((k_fp8_quantize<4, false>), grid, dim3(256), 0, st, x, Mx, row_src, M, C, xq, xs);
  else
    hipLaunchKernelGGL((k_fp8_quantize<1, false>), grid, dim3(256), 0, st, x, Mx, row_src, M, C, xq, xs);
  return int(hipGetLastError());
}

int launch_fp8_quantize_cols(const uint16_t* x, int64_t Mx, const int32_t* row_src, int64_t M, int C, uint8_t* xt,
                             uint8_t* xts, hipStream_t st) {
  const int64_t ld = fp8_ld(M);
  const dim3 grid{unsigned((C + 63) / 64), unsigned(ld / kQBlock), 1u};
  if (past_caches(Mx, M, C))
    hipLaunchKernelGGL(k_fp8_quantize_cols<true>, grid, dim3(256), 0, st, x, Mx, row_src, M, C, ld, fp8_sld(M), xt, xts);
  else
    hipLaunchKernelGGL(k_fp8_quantize_cols<false>, grid, dim3(256), 0, st, x, Mx, row_src, M, C, ld, fp8_sld(M), xt,
                       xts);
  return int(hipGetLastError());
}

// A weight stack: a workgroup takes one 128 x 128 block of one matrix, in both
// orders.  A thread holds 16 rows of 4 columns; both layouts leave through the
// same LDS bytes (rows of 132, so that the reads of a column spread over the
// banks).  64 matrices of 1024 x 2048 take 203 us (805 MB, 4.0 TB/s): the 4-byte
// loads of a row that may have any alignment, and the transpose's reads of
// single bytes, stand between it and HBM.
__global__ __launch_bounds__(256) void k_fp8_quantize_weight(const float* __restrict__ w, int N, int C,
                                                             uint8_t* __restrict__ wq, uint8_t* __restrict__ ws,
                                                             uint8_t* __restrict__ wt, uint8_t* __restrict__ wts) {
  __shared__ uint32_t tops[4];
  __shared__ uint32_t words[kQBlock * 33];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int cb = int(blockIdx.x), nb = int(blockIdx.y);
  const int64_t g = blockIdx.z;
  const int64_t ldc = (int64_t(C) + kQBlock - 1) / kQBlock * kQBlock, ldn = (int64_t(N) + kQBlock - 1) / kQBlock * kQBlock;
  const int64_t sldc = (ldc / kQBlock + 3) / 4 * 4, sldn = (ldn / kQBlock + 3) / 4 * 4;
  const int cg = tid & 31, rg = tid >> 5;  // 4 columns from 4 cg, rows rg + 8 u
  const int c0 = cb * kQBlock + cg * 4;
  float v[16][4];
  uint32_t top = 0;
#pragma unroll
  for (int u = 0; u < 16; ++u) {
    const int n = nb * kQBlock + rg + 8 * u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[u][i] = n < N && c0 + i < C ? w[(g * N + n) * C + c0 + i] : 0.f;
      const uint32_t a = __builtin_bit_cast(uint32_t, v[u][i]) & 0x7FFFFFFFu;
      top = top > a ? top : a;
    }
  }
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) {
    const uint32_t o = __shfl_xor(top, d);
    top = top > o ? top : o;
  }
  if (lane == 0) tops[wave] = top;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 4; ++k) top = top > tops[k] ? top : tops[k];
  // 448 = 1.75 * 2^8: one more power when the fraction is above 0.75
  int e = int(top >> 23) - 127 - 8 + ((top & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  e = e < -126 ? -126 : e;
  const float f = scale_down(e + 127);
  const bool bad = top >= 0x7F800000u;
#pragma unroll
  for (int u = 0; u < 16; ++u) {
    const int row = rg + 8 * u;
    words[row * 33 + cg] = to_e4m3x4(v[u][0] * f, v[u][1] * f, v[u][2] * f, v[u][3] * f, bad);
  }
  __syncthreads();
  // 128 rows of eight 16-byte parts
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    const int i = h * 256 + tid, row = i >> 3, part = i & 7, n = nb * kQBlock + row;
    if (n < N) {
      const uint32_t* src = words + row * 33 + part * 4;
      uint4 o;
      o.x = src[0], o.y = src[1], o.z = src[2], o.w = src[3];
      *reinterpret_cast<uint4*>(wq + (g * N + n) * ldc + cb * kQBlock + part * 16) = o;
    }
  }
  if (tid == 0) ws[(g * (ldn / kQBlock) + nb) * sldc + cb] = uint8_t(e + 127);
  if (wt) {
    const uint8_t* bytes = reinterpret_cast<const uint8_t*>(words);
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      const int i = h * 256 + tid, col = i & 127, part = i >> 7, c = cb * kQBlock + col;
      if (c < C) {
        uint32_t o[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          o[k] = 0;
#pragma unroll
          for (int j = 0; j < 4; ++j) o[k] |= uint32_t(bytes[(part * 16 + k * 4 + j) * 132 + col]) << (8 * j);
        }
        *reinterpret_cast<uint4*>(wt + (g * C + c) * ldn + nb * kQBlock + part * 16) = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
    if (tid == 0) wts[(g * (ldc / kQBlock) + cb) * sldn + nb] = uint8_t(e + 127);
  }
}

int launch_fp8_quantize_weight(const float* w, int G, int N, int C, uint8_t* wq, uint8_t* ws, uint8_t* wt,
                               uint8_t* wts, hipStream_t st) {
  const dim3 grid{unsigned(fp8_ld(C) / kQBlock), unsigned(fp8_ld(N) / kQBlock), unsigned(G)};
  hipLaunchKernelGGL(k_fp8_quantize_weight, grid, dim3(256), 0, st, w, N, C, wq, ws, wt, wts);
  return int(hipGetLastError());
}

// Eight e4m3 bytes times a scale as bf16, exactly.
__device__ __forceinline__ bf16x8 widen(int lo, int hi, float scale) {
  const auto a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false);
  const auto b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true);
  const auto c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false);
  const auto d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true);
  return (bf16x8){a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}
// 2^(byte - 127) of a scale byte.
__device__ __forceinline__ float scale_value(int byte) { return __builtin_bit_cast(float, uint32_t(byte) << 23); }

// ---------------------------------------------------------------------------
// which expert a tile of rows belongs to

struct Tile {
  int e;            // expert, -1: none
  int64_t lo, hi;   // its rows
  int at;           // the tile's number inside it
};

// The wave finds tile t of the list of all experts' tiles of BM rows (four
// experts a lane); total: the list's length.  Offsets outside [0, M] or out
// of order are clamped, so any `off` stays inside the arrays.
__device__ __forceinline__ int group_tiles(const int32_t* off, int G, int64_t M, int BM, int lane, int (&lo)[4],
                                           int (&hi)[4], int (&n)[4], int& before) {
  int sum = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int e = 4 * lane + j;
    int a = e < G ? off[e] : 0, b = e < G ? off[e + 1] : 0;
    a = a < 0 ? 0 : (a > M ? int(M) : a);
    b = b < a ? a : (b > M ? int(M) : b);
    lo[j] = a;
    hi[j] = b;
    n[j] = (b - a + BM - 1) / BM;
    sum += n[j];
  }
  int run = sum;
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) {
    const int o = __shfl_up(run, d);
    run += lane >= d ? o : 0;
  }
  before = run - sum;
  return __shfl(run, kWave - 1);
}
__device__ __forceinline__ Tile group_find(int t, int lane, const int (&lo)[4], const int (&hi)[4], const int (&n)[4],
                                           int before) {
  int e = -1, at = 0, a = 0, b = 0, run = before;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (t >= run && t < run + n[j]) {
      e = 4 * lane + j;
      at = t - run;
      a = lo[j];
      b = hi[j];
    }
    run += n[j];
  }
  const uint64_t m = __ballot(e >= 0);
  Tile r;
  if (m == 0) {
    r.e = -1;
    r.lo = r.hi = 0;
    r.at = 0;
    return r;
  }
  const int from = __builtin_ctzll(m);
  r.e = __builtin_amdgcn_readlane(e, from);
  r.at = __builtin_amdgcn_readlane(at, from);
  r.lo = __builtin_amdgcn_readlane(a, from);
  r.hi = __builtin_amdgcn_readlane(b, from);
  return r;
}

// Workgroups are dealt out to the 8 XCDs in turn, and each takes every
// grid'th number; each XCD takes a consecutive stretch of the tiles, so the
// tiles in flight on one L2 share rows.  A permutation of [0, n).
__device__ __forceinline__ int tile_at(int i, int grid, int n) {
  // numbers of XCD x: those i < n with (i mod grid) mod 8 = x
  const int x = (i % grid) % 8, full = n / grid, rest = n % grid;
  auto of = [&](int y) { return full * ((grid + 7 - y) / 8) + (rest + 7 - y) / 8; };
  int first = 0;
#pragma unroll
  for (int y = 0; y < 8; ++y) first += y < x ? of(y) : 0;
  return first + (i / grid) * ((grid + 7 - x) / 8) + (i % grid) / 8;
}

// The same for experts whose sums are of unequal length: the XCDs take turns
// at chunks of C tiles, so that a long expert's do not all fall to one of them
// (one of 16 experts with all of 2048 rows, 768 x 1152: 59 us with stretches).
template <int C>
__device__ __forceinline__ int tile_in_turn(int i, int n) {
  const int s = i / 8;
  return i < n / (8 * C) * (8 * C) ? ((s / C) * 8 + i % 8) * C + s % C : i;
}

// s_waitcnt's immediate: at most n vector memory operations outstanding, and
// every LDS read back.
constexpr int vm_count(int n) { return 0x0070 | (n & 15) | ((n >> 4) << 14); }

// Zeros in rows m0 .. (below M) and columns n0 .. (below N) of a tile.
template <int BM, int BN, int W>
__device__ __forceinline__ void zero_tile(float* out, int64_t out_row, int64_t m0, int64_t M, int n0, int N, int tid) {
  const Float4 zero = {};
  for (int i = tid; i < BM * BN / 4; i += W * kWave) {
    const int64_t row = m0 + i / (BN / 4);
    const int col = n0 + i % (BN / 4) * 4;
    if (row >= M) break;
    float* o = out + (out_row + row) * N + col;
    if (col + 3 < N) {
      *reinterpret_cast<Float4*>(o) = zero;
    } else {
      for (int c = 0; col + c < N; ++c) o[c] = 0.f;
    }
  }
}

// Tiles in groups of GM rows of tiles, column by column inside a group.
__device__ __forceinline__ void tile_order(int t, int tm_all, int tn_all, int GM, int& tm, int& tn) {
  const int g = t / (GM * tn_all), r = t % (GM * tn_all);
  const int rows = tm_all - g * GM < GM ? tm_all - g * GM : GM;
  tm = g * GM + r % rows;
  tn = r / rows;
}

// ---------------------------------------------------------------------------
// the tiled product

// A workgroup computes BM x BN tiles of the result from an LDS ring of S
// stages of 128 bytes of K, filled by loads that go to LDS directly; the waves
// tile it WM x WN.  It takes one tile after another (XCD by XCD, see
// tile_at), and the loads run ahead of the products over the end of a tile,
// so that only the first tile of a workgroup waits for its operands and its
// results leave beside the next one's.  GRAD: the weight gradient (float out,
// K = an expert's rows, every expert's output is written); else the product
// (bf16 out, an expert's rows tiled).
//
// A row's 128 bytes are 8 slots of 16, XORed with a number of the row's, so
// that the 16 rows that the lanes of a quarter wave read in one slot lie in
// all banks once (two rows fill them).  For float results a wave's column
// tile j holds columns 16 j .. 16 j + 15: lane groups g of 16 lanes write 16
// bytes side by side.  For bf16 results column tile j takes columns 16 g + 4
// j + c instead, so that a lane ends up with 16 columns side by side, 32
// bytes, and four lanes with a row's 128.
//
// S = 2, where every CU has tiles enough: four blocks' scales are one word a
// row and loaded every fourth stage.  S = 4, for the smallest tiles, one or
// two workgroups a CU: a block's loads are three steps ahead, and each stage
// loads its scales' word so that the number of loads in flight is known.
template <int BM, int BN, int WM, int WN, int S, bool GRAD, bool EXACT>
__global__ __launch_bounds__(WM* WN* kWave, 2) void k_fp8_gemm(const uint8_t* __restrict__ A,
                                                            const uint8_t* __restrict__ As,
                                                            const uint8_t* __restrict__ Bm,
                                                            const uint8_t* __restrict__ Bs, int64_t M, int N,
                                                            int64_t ldk, int64_t sld, const int32_t* __restrict__ off,
                                                            int G, int tiles, void* __restrict__ outp) {
  constexpr int W = WM * WN, TM = BM / WM / 16, TN = BN / WN / 16;
  constexpr int A_BYTES = BM * kQBlock, B_BYTES = BN * kQBlock;
  constexpr int A_PW = A_BYTES / 1024 / W, B_PW = B_BYTES / 1024 / W;  // 1 KiB loads per wave and stage
  constexpr int ROWS = BM + BN;
  constexpr int S_PW = (ROWS / kWave + W - 1) / W;  // loads of 64 rows' scale words per wave
  constexpr bool WIDE = !GRAD;
  constexpr int JT = TN < 4 ? TN : 4;  // column tiles that share a stretch of 16 JT columns
  static_assert(A_PW * W * 1024 == A_BYTES && B_PW * W * 1024 == B_BYTES && ROWS % kWave == 0, "tile split");
  static_assert(TN % JT == 0 && JT >= 2, "a bf16 result's columns");
  // a row's number in the swizzle of its slots
  auto key_a = [](int row) { return (row >> 1) & 7; };
  auto key_b = [](int row) { return WIDE ? ((row >> 1) & 1) | ((row >> (JT == 4 ? 3 : 2)) & 6) : (row >> 1) & 7; };
  // one array: with several, the compiler waits for the loads to LDS before it reads any of them
  __shared__ __align__(1024) uint8_t lds[S * (A_BYTES + B_BYTES) + S * ROWS * 4 + 1024 * 3 + 16];
  uint8_t* const lds_b = lds + S * A_BYTES;
  uint8_t* const lds_s = lds + S * (A_BYTES + B_BYTES);
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int tn_all = (N + BN - 1) / BN, kb_all = int(ldk / kQBlock);

  // the experts' first and last rows (GRAD: blocks of rows) and their tiles of rows before each, kept in LDS: a
  // tile's expert is found while the last tile's products wait for it
  int* const first_of = reinterpret_cast<int*>(lds_s + S * ROWS * 4);
  int *const end_of = first_of + 256, *const before_of = end_of + 256;  // 256, 256 and 257 of them
  if (off) {
    int total = 0;
    if constexpr (GRAD) {
      for (int e = tid; e < G; e += W * kWave) {
        int a = off[e] / kQBlock, b = off[e + 1] / kQBlock;
        a = a < 0 ? 0 : (a > kb_all ? kb_all : a);
        b = b < a ? a : (b > kb_all ? kb_all : b);
        first_of[e] = a;
        end_of[e] = b;
      }
    } else if (wave == 0) {
      int lo[4], hi[4], n[4], before;
      total = group_tiles(off, G, M, BM, lane, lo, hi, n, before);
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
    if constexpr (!GRAD) tiles = (before_of[256] < tiles / tn_all ? before_of[256] : tiles / tn_all) * tn_all;
  }

  // What a tile's results need: rows m0 .. m_end - 1 and columns n0 ... of
  // the result, whose rows are counted from out_row; blocks k0 .. k1 - 1.
  struct Place {
    int m0, m_end, out_row, n0, k0, k1;
  };
  // and what its loads need
  const uint8_t *a_base, *b_base, *s_src[S_PW];
  uint32_t a_off[A_PW], b_off[B_PW];
  auto place = [&](int t) {
    Place p{0, int(M), 0, 0, 0, kb_all};
    const uint8_t *bm = Bm, *bsc = Bs;
    int tm, tn;
    if constexpr (GRAD) {
      const int tm_all = int((M + BM - 1) / BM), per = tm_all * tn_all, e = t / per;
      tile_order(t % per, tm_all, tn_all, 8, tm, tn);
      if (off) {
        p.k0 = __builtin_amdgcn_readfirstlane(first_of[e]);
        p.k1 = __builtin_amdgcn_readfirstlane(end_of[e]);
      }
      p.m0 = tm * BM;
      p.out_row = e * int(M);
    } else if (off) {
      tile_order(t, tiles / tn_all, tn_all, 8, tm, tn);
      // the expert whose tiles hold tm: the one before the first that begins past it
      int begun = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) begun += __popcll(__ballot(before_of[4 * lane + j] <= tm));
      const int e = begun > 0 ? begun - 1 : 0;  // the last of those that begin at tm: the ones before it have no tile
      p.m0 = __builtin_amdgcn_readfirstlane(first_of[e] + (tm - before_of[e]) * BM);
      p.m_end = __builtin_amdgcn_readfirstlane(end_of[e]);
      bm += int64_t(e) * N * ldk;
      bsc += int64_t(e) * ((N + kQBlock - 1) / kQBlock) * sld;
    } else {
      tile_order(t, int((M + BM - 1) / BM), tn_all, 8, tm, tn);
      p.m0 = tm * BM;
    }
    p.n0 = tn * BN;
    // per-lane sources: rows past the end re-read the last one
    a_base = A + int64_t(p.m0) * ldk;
    b_base = bm + int64_t(p.n0) * ldk;
#pragma unroll
    for (int j = 0; j < A_PW; ++j) {
      const int at = (wave * A_PW + j) * kWave + lane, r = at >> 3, q = (at & 7) ^ key_a(r);
      const int row = p.m0 + r < p.m_end ? r : p.m_end - 1 - p.m0;
      a_off[j] = uint32_t(row) * uint32_t(ldk) + q * 16;
    }
#pragma unroll
    for (int j = 0; j < B_PW; ++j) {
      const int at = (wave * B_PW + j) * kWave + lane, r = at >> 3, q = (at & 7) ^ key_b(r);
      const int row = p.n0 + r < N ? r : N - 1 - p.n0;
      b_off[j] = uint32_t(row) * uint32_t(ldk) + q * 16;
    }
#pragma unroll
    for (int j = 0; j < S_PW; ++j) {
      const int i = (wave * S_PW + j) % (ROWS / kWave) * kWave + lane;  // (with fewer than waves, some load them twice)
      if (i < BM) {
        const int row = p.m0 + i < p.m_end ? p.m0 + i : p.m_end - 1;
        s_src[j] = As + int64_t(row) * sld;
      } else {
        int row = p.n0 + (i - BM);
        row = row < N ? row : N - 1;
        s_src[j] = bsc + int64_t(GRAD ? row : row / kQBlock) * sld;
      }
    }
    return p;
  };
  // Load u of a stage's tiles.
  constexpr int LOADS = A_PW + B_PW;
  auto issue = [&](int u, int64_t ko, int st) {
    if (u < A_PW)
      __builtin_amdgcn_global_load_lds((glb_vptr)(a_base + ko + a_off[u < A_PW ? u : 0]),
                                       (lds_vptr)(lds + st * A_BYTES + (wave * A_PW + u) * 1024), 16, 0, 0);
    else
      __builtin_amdgcn_global_load_lds((glb_vptr)(b_base + ko + b_off[u < A_PW ? 0 : u - A_PW]),
                                       (lds_vptr)(lds_b + st * B_BYTES + (wave * B_PW + u - A_PW) * 1024), 16, 0, 0);
  };
  auto issue_scales = [&](int kb, int slot) {
#pragma unroll
    for (int j = 0; j < S_PW; ++j)
      __builtin_amdgcn_global_load_lds((glb_vptr)(s_src[j] + (kb & ~3)),
                                       (lds_vptr)(lds_s + slot * (ROWS * 4) + (wave * S_PW + j) % (ROWS / kWave) * 256), 4, 0,
                                       0);
  };
  auto issue_all = [&](int kb, int st, int slot) {
#pragma unroll
    for (int u = 0; u < LOADS; ++u) issue(u, int64_t(kb) * kQBlock, st);
    issue_scales(kb, slot);
  };

  v4f acc[TM][TN];
  const int r = lane & 15, g4 = lane >> 4;
  // this lane's slots g4 and g4 + 4 of its row
  const int frag_a = r * kQBlock + ((g4 ^ key_a(r)) * 16);
  const int br = WIDE ? (r >> 2) * (4 * JT) + (r & 3) : r;  // its row of column tile 0, and what tile j adds
  auto b_row = [](int j) { return WIDE ? j / JT * (16 * JT) + j % JT * 4 : j * 16; };
  auto frag_b = [&](int j) {
    const int row = br + b_row(j);
    return row * kQBlock + ((g4 ^ key_b(row)) * 16);
  };
  // block kb's products out of stage st, its scales out of `slot`, while block
  // `load`'s tiles go to stage `into`: after the first row tile's products
  // (8192 x 8192 x 4096: 249 us; before them all 261, spread over the rows 265)
  auto multiply = [&](int kb, int st, int slot, int load, int into) {
    const int64_t ko = int64_t(load) * kQBlock;
    const uint8_t* sa = lds + st * A_BYTES + wm * (TM * 16) * kQBlock;
    const uint8_t* sb = lds_b + st * B_BYTES + wn * (TN * 16) * kQBlock;
    const uint8_t* ss = lds_s + slot * (ROWS * 4) + (kb & 3);
    const uint8_t *ssa = ss + (wm * TM * 16 + r) * 4, *ssb = ss + (BM + wn * TN * 16 + br) * 4;
    if constexpr (!EXACT) {
      v8i b[TN];
      int bs[TN];
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        const v4i lo4 = *reinterpret_cast<const v4i*>(sb + frag_b(j));
        const v4i hi4 = *reinterpret_cast<const v4i*>(sb + (frag_b(j) ^ 64));
        b[j] = __builtin_shufflevector(lo4, hi4, 0, 1, 2, 3, 4, 5, 6, 7);
        bs[j] = ssb[b_row(j) * 4];
      }
      // row tile i + 1 is read while i's products run
      v8i a[2];
      int as[2];
      auto read = [&](int i) {
        const v4i lo4 = *reinterpret_cast<const v4i*>(sa + i * 16 * kQBlock + frag_a);
        const v4i hi4 = *reinterpret_cast<const v4i*>(sa + i * 16 * kQBlock + (frag_a ^ 64));
        a[i & 1] = __builtin_shufflevector(lo4, hi4, 0, 1, 2, 3, 4, 5, 6, 7);
        as[i & 1] = ssa[i * 64];
      };
      read(0);
#pragma unroll
      for (int i = 0; i < TM; ++i) {
        if (i + 1 < TM) read(i + 1);
#pragma unroll
        for (int j = 0; j < TN; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b[j], a[i & 1], acc[i][j], 0, 0, 0, bs[j], 0,
                                                                      as[i & 1]);
        if (i == 0)
#pragma unroll
          for (int u = 0; u < LOADS; ++u) issue(u, ko, into);
      }
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        bf16x8 b[TN][2];
#pragma unroll
        for (int j = 0; j < TN; ++j) {
          const v4i t = *reinterpret_cast<const v4i*>(sb + (frag_b(j) ^ (h * 64)));
          const float f = scale_value(ssb[b_row(j) * 4]);
          b[j][0] = widen(t[0], t[1], f);
          b[j][1] = widen(t[2], t[3], f);
        }
        v4i a[2];
        int as[2];
        auto read = [&](int i) {
          a[i & 1] = *reinterpret_cast<const v4i*>(sa + i * 16 * kQBlock + (frag_a ^ (h * 64)));
          as[i & 1] = ssa[i * 64];
        };
        read(0);
#pragma unroll
        for (int i = 0; i < TM; ++i) {
          if (i + 1 < TM) read(i + 1);
          const v4i t = a[i & 1];
          const float f = scale_value(as[i & 1]);
          const bf16x8 a0 = widen(t[0], t[1], f), a1 = widen(t[2], t[3], f);
#pragma unroll
          for (int j = 0; j < TN; ++j) {
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[j][0], a0, acc[i][j], 0, 0, 0);
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[j][1], a1, acc[i][j], 0, 0, 0);
          }
          if (h == 0 && i == 0)
#pragma unroll
            for (int u = 0; u < LOADS; ++u) issue(u, ko, into);
        }
      }
    }
  };

  // element c of acc[i][j]: row 16 i + r, column 16 j + 4 g4 + c (WIDE: 4 JT g4 + 4 j + c of its JT column tiles);
  // returns whether every store of the tile was issued
  constexpr int STORES = TM * (WIDE ? TN / 2 : TN);
  auto store_some = [&](const Place& p, auto whole) {
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      const int row = p.m0 + (wm * TM + i) * 16 + r;
      if (!whole() && row >= p.m_end) continue;
      if constexpr (GRAD) {
        float* o = static_cast<float*>(outp) + int64_t(p.out_row + row) * N;
#pragma unroll
        for (int j = 0; j < TN; ++j) {
          const int col = p.n0 + (wn * TN + j) * 16 + g4 * 4;
          const v4f v = acc[i][j];
          if (whole() || col + 3 < N) {
            Float4 t;
#pragma unroll
            for (int c = 0; c < 4; ++c) t.v[c] = v[c];
            *reinterpret_cast<Float4*>(o + col) = t;
          } else {
#pragma unroll
            for (int c = 0; c < 4; ++c)
              if (col + c < N) o[col + c] = v[c];
          }
        }
      } else {
        uint16_t* o = static_cast<uint16_t*>(outp) + int64_t(row) * N;
#pragma unroll
        for (int h = 0; h < TN / 2; ++h) {  // 8 columns each
          const int col = p.n0 + (wn * TN + 2 * h / JT * JT) * 16 + g4 * (4 * JT) + 8 * (h % (JT / 2));
          Half8 t;
#pragma unroll
          for (int k = 0; k < 4; ++k)
            t.v[k] = bf16x2_rne(acc[i][2 * h + k / 2][2 * (k & 1)], acc[i][2 * h + k / 2][2 * (k & 1) + 1]);
          if (whole() || col + 7 < N) {
            *reinterpret_cast<Half8*>(o + col) = t;
          } else {
#pragma unroll
            for (int c = 0; c < 8; ++c)
              if (col + c < N) o[col + c] = uint16_t(t.v[c >> 1] >> (16 * (c & 1)));
          }
        }
      }
    }
  };
  auto store = [&](const Place& p) {
    const bool whole = p.m0 + BM <= p.m_end && p.n0 + BN <= N;
    if (whole)
      store_some(p, std::true_type{});
    else
      store_some(p, std::false_type{});
    return whole;
  };
  auto clear = [&]() {
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) acc[i][j] = (v4f){0.f, 0.f, 0.f, 0.f};
  };

  int at = int(blockIdx.x);
  Place now{};
  // the next tile that has a product to compute; those without (an expert without rows) are written as zeros
  auto advance = [&](bool& found) {
    found = false;
    for (; at < tiles; at += int(gridDim.x)) {
      const bool in_turn = GRAD && off && gridDim.x % 8 == 0;
      const Place p = place(in_turn ? tile_in_turn<BM == 256 ? 16 : 8>(at, tiles) : tile_at(at, int(gridDim.x), tiles));
      if (p.k0 < p.k1) {
        found = true;
        at += int(gridDim.x);
        return p;
      }
      if constexpr (GRAD) zero_tile<BM, BN, W>(static_cast<float*>(outp), p.out_row, p.m0, M, p.n0, N, tid);
    }
    return Place{};
  };
  bool more;
  now = advance(more);
  if constexpr (S == 2) {
    int put = 0, get = 1, st = 0;  // the halves of the scales' ring that was filled last and that is read
    if (more) issue_all(now.k0, 0, 0);
    bool behind = false;  // the last tile's stores are younger than the loads that are waited for
    while (more) {
      clear();
      Place then{};
      bool next = false;
      for (int kb = now.k0; kb < now.k1; ++kb) {
        // this wave's loads of the stage; the barrier publishes every wave's
        // and retires all reads of the stage that is filled next
        if (behind && kb == now.k0)
          __builtin_amdgcn_s_waitcnt(vm_count(STORES));
        else
          __builtin_amdgcn_s_waitcnt(vm_count(0));
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        if (kb == now.k0 || (kb & 3) == 0) get ^= 1;
        // the next block: of this tile, of the next one, or (no more tiles) this one again, which nothing reads
        int load = kb + 1;
        bool scales = (load & 3) == 0;
        if (load == now.k1) {
          then = advance(next);
          scales = next;
          load = next ? then.k0 : kb;
        }
        if (scales) {
          put ^= 1;
          issue_scales(load, put);
        }
        multiply(kb, st, get, load, st ^ 1);
        st ^= 1;
      }
      behind = store(now);
      now = then;
      more = next;
    }
    __builtin_amdgcn_s_waitcnt(vm_count(0));  // no load may land after the LDS has changed hands
  } else {
    constexpr int PER = LOADS + S_PW;
    while (more) {
      clear();
#pragma unroll
      for (int u = 0; u < S - 1; ++u) {
        const int kb = now.k0 + u < now.k1 ? now.k0 + u : now.k1 - 1;
        issue_all(kb, u, u);
      }
      int st = 0;
      for (int kb = now.k0; kb < now.k1; ++kb) {
        __builtin_amdgcn_s_waitcnt(vm_count((S - 2) * PER));
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        // past the tile's end the last block again, which nothing reads
        const int load = kb + S - 1 < now.k1 ? kb + S - 1 : now.k1 - 1, into = st == 0 ? S - 1 : st - 1;
        issue_scales(load, into);
        multiply(kb, st, st, load, into);
        st = st + 1 < S ? st + 1 : 0;
      }
      store(now);
      __builtin_amdgcn_s_waitcnt(vm_count(0));
      now = advance(more);
      if (more) __syncthreads();  // all have read the ring
    }
  }
}

// ---------------------------------------------------------------------------
// the product of few rows

// Bound by the weight's bytes: a workgroup of 8 waves takes 16 MT rows and
// 16 * 8 / KW columns; KW waves share a column tile's K, block by block, so
// that the whole weight is in flight at once, and join their sums through
// LDS in order.  Both operands go from memory to registers: lane l takes 32
// contiguous bytes of row l % 16, four lanes a line.
template <int MT, int KW>
__global__ __launch_bounds__(512) void k_fp8_thin(const uint8_t* __restrict__ A, const uint8_t* __restrict__ As,
                                                  const uint8_t* __restrict__ Bm, const uint8_t* __restrict__ Bs,
                                                  int64_t M, int N, int64_t ldk, int64_t sld,
                                                  const int32_t* __restrict__ off, int G,
                                                  uint16_t* __restrict__ out) {
  constexpr int NW = 8 / KW, BM = 16 * MT, BN = 16 * NW, U = MT >= 4 ? 2 : 4;
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
    Bm += int64_t(g.e) * N * ldk;
    Bs += int64_t(g.e) * ((N + kQBlock - 1) / kQBlock) * sld;
  } else {
    m0 = int64_t(int(blockIdx.x) / tn_all) * BM;
    n0 = (int(blockIdx.x) % tn_all) * BN;
    m_end = M;
  }
  const int r = lane & 15, g4 = lane >> 4;
  const int KB = int(ldk / kQBlock);
  const int ncol = n0 + wn * 16;
  const int brow = ncol + r < N ? ncol + r : N - 1;
  const uint8_t* bp = Bm + int64_t(brow) * ldk + g4 * 32;
  const uint8_t* bsp = Bs + int64_t(brow / kQBlock) * sld;
  const uint8_t* ap[MT];
  const uint8_t* asp[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    int64_t row = m0 + 16 * i + r;
    row = row < m_end ? row : m_end - 1;
    ap[i] = A + row * ldk + g4 * 32;
    asp[i] = As + row * sld;
  }
  v4f acc[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) acc[i] = (v4f){0.f, 0.f, 0.f, 0.f};
  for (int kb = wk; kb < KB; kb += KW * U) {
    v8i b[U], a[U][MT];
    int bs[U], as[U][MT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = kb + u * KW;
      const int kc = k < KB ? k : kb;  // past the end: re-read, and not used
      b[u] = *reinterpret_cast<const v8i*>(bp + int64_t(kc) * kQBlock);
      bs[u] = bsp[kc];
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        a[u][i] = *reinterpret_cast<const v8i*>(ap[i] + int64_t(kc) * kQBlock);
        as[u][i] = asp[i][kc];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (kb + u * KW < KB) {
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          const bf16x8 bw = widen(b[u][2 * h], b[u][2 * h + 1], scale_value(bs[u]));
#pragma unroll
          for (int i = 0; i < MT; ++i)
            acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                bw, widen(a[u][i][2 * h], a[u][i][2 * h + 1], scale_value(as[u][i])), acc[i], 0, 0, 0);
        }
      }
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

struct Gemm {
  const uint8_t *A, *As, *B, *Bs;
  int64_t M;
  int N;
  int64_t ldk, sld;
  const int32_t* off;
  int G;
  void* out;
};

// Tiles of BM rows that G experts' M rows make at most.
static int64_t row_tiles(const Gemm& g, int BM) {
  if (!g.off) return (g.M + BM - 1) / BM;
  return g.M / BM + std::min<int64_t>(g.G, g.M);
}

template <int BM, int BN, int WM, int WN, int S, bool GRAD, bool EXACT>
static int gemm_tiled(const Gemm& g, hipStream_t st) {
  const int64_t tn = (g.N + BN - 1) / BN;
  const int64_t tiles = GRAD ? int64_t(g.G) * ((g.M + BM - 1) / BM) * tn : row_tiles(g, BM) * tn;
  if (tiles > INT32_MAX) return int(hipErrorInvalidValue);
  // as many workgroups as run at once (a 256 x 256 tile's ring fills a CU's LDS, a 128 x 128 tile's half of it)
  const int64_t most = int64_t(device_cu_count()) * (S * (BM + BN) > 512 ? 1 : 2);
  hipLaunchKernelGGL((k_fp8_gemm<BM, BN, WM, WN, S, GRAD, EXACT>), dim3(unsigned(std::min(tiles, most))),
                     dim3(WM * WN * kWave), 0, st, g.A, g.As, g.B, g.Bs, g.M, g.N, g.ldk, g.sld, g.off, g.G, int(tiles),
                     g.out);
  return int(hipGetLastError());
}

// Which tiles: 64 x 64 while two workgroups a CU take them all at once (768 x
// 2048 x 1024: 10.0 us, 128 x 128 tiles 12.9; 2048 x 2048 x 2048: 29.6 and
// 24.8).  Above that 128 x 128, two at a time on a CU, or 256 x 256, which read
// half the operands' bytes per product and cost 3.3 small ones' time where two
// small ones at a time cost 2 (8192 x 8192 x 4096: 412 us, 459; 4096 x 4096 x
// 4096: 110 and 123), whichever has the cheaper number of rounds over the CUs.
// The 8-bit instruction has the same order at each of these sizes (7.4 and
// 9.2; 19.0 and 17.0; 229 and 278; 60 and 72).  `uneven`: the part of a round
// that large tiles lose where experts of unequal length leave some CUs waiting.
template <bool GRAD, bool EXACT>
static int gemm(const Gemm& g, int64_t t256, int64_t t128, int64_t t64, double uneven, hipStream_t st) {
  const int64_t cu = device_cu_count();
  if (t64 <= 2 * cu) return gemm_tiled<64, 64, 2, 2, 4, GRAD, EXACT>(g, st);
  const double rounds256 = double((t256 + cu - 1) / cu), rounds128 = double((t128 + 2 * cu - 1) / (2 * cu));
  if (t256 > 0 && 3.3 * (rounds256 + uneven) < 2 * rounds128) return gemm_tiled<256, 256, 2, 4, 2, GRAD, EXACT>(g, st);
  return gemm_tiled<128, 128, 2, 2, 2, GRAD, EXACT>(g, st);
}

template <int MT, int KW>
static int gemm_thin(const Gemm& g, hipStream_t st) {
  constexpr int BN = 16 * (8 / KW);
  const int64_t blocks = row_tiles(g, 16 * MT) * ((g.N + BN - 1) / BN);
  if (blocks > INT32_MAX) return int(hipErrorInvalidValue);
  hipLaunchKernelGGL((k_fp8_thin<MT, KW>), dim3(unsigned(blocks)), dim3(512), 0, st, g.A, g.As, g.B, g.Bs, g.M, g.N,
                     g.ldk, g.sld, g.off, g.G, static_cast<uint16_t*>(g.out));
  return int(hipGetLastError());
}

// How many waves share a column tile's K: as many as give every CU a
// workgroup, and two where a wave's part is then still four blocks long (one
// token through 4096 x 4096: 20.5, 11.6, 7.4, 5.2 us with 1, 2, 4, 8; 128 rows
// over 256 experts of 1024 x 2048: 47, 44, 50, 90, since each workgroup of
// eight has so little of the weight that finding its tile counts; 64 x 64
// tiles take 45, 34 with the 8-bit instruction).
template <int MT>
static int gemm_few(const Gemm& g, hipStream_t st) {
  const int64_t waves = row_tiles(g, 16 * MT) * ((g.N + 15) / 16);
  int kw = g.ldk >= 8 * kQBlock ? 2 : 1;
  while (kw < 8 && waves * kw < 8 * int64_t(device_cu_count())) kw *= 2;
  switch (kw) {
    case 1: return gemm_thin<MT, 1>(g, st);
    case 2: return gemm_thin<MT, 2>(g, st);
    case 4: return gemm_thin<MT, 4>(g, st);
    default: return gemm_thin<MT, 8>(g, st);
  }
}

int launch_fp8_product(const uint8_t* xq, const uint8_t* xs, const uint8_t* w, const uint8_t* ws, int64_t M, int N,
                       int64_t ldk, const int32_t* off, int G, bool exact, uint16_t* y, hipStream_t st) {
  const Gemm g{xq, xs, w, ws, M, N, ldk, fp8_sld(ldk), off, G, y};
  const int64_t rows = off ? (M + G - 1) / G : M;  // rows of an expert, on average
  auto tiles = [&](int b) { return row_tiles(g, b) * ((N + b - 1) / b); };
  const int64_t cu = device_cu_count();
  // few rows and no tile for every CU: 16 columns of the weight a wave (32 rows, 4096 x 4096: 10.4 us, tiles 17.5, with
  // the 8-bit instruction 11.3; 16 rows 7.5, 17.4 and 11.2; 64 rows 17.6, 17.5 and 11.4)
  if (rows <= 32 && tiles(64) <= cu) return rows <= 16 ? gemm_few<1>(g, st) : gemm_few<2>(g, st);
  // an expert of up to 128 rows fills no more than half of a 256 x 256 tile, and one of up to 16 a quarter of a 64 x
  // 64 one; of the tiles that experts' rows make at most, some are not there
  const int64_t t256 = rows <= 128 && off ? 0 : tiles(256);
  const int64_t t64 = !off ? tiles(64) : (rows <= 16 ? 0 : tiles(64) * 2 / 3);
  const double uneven = off ? 0.1 : 0.0;
  return exact ? gemm<false, true>(g, t256, tiles(128), t64, uneven, st)
               : gemm<false, false>(g, t256, tiles(128), t64, uneven, st);
}

int launch_fp8_weight_grad(const uint8_t* dyt, const uint8_t* dyts, const uint8_t* xt, const uint8_t* xts, int N,
                           int C, int64_t ldm, const int32_t* off, int G, float* dw, hipStream_t st) {
  const Gemm g{dyt, dyts, xt, xts, N, C, ldm, fp8_sld(ldm), off, G, dw};
  auto tiles = [&](int b) { return int64_t(G) * ((N + b - 1) / b) * ((C + b - 1) / b); };
  return gemm<true, true>(g, tiles(256), tiles(128), tiles(64), off ? 0.25 : 0.0, st);
}

}  // namespace qbk
