// qb_ortho.hip -- the orthogonalised update of a stack of matrices, by
// Newton-Schulz steps of an odd polynomial of fifth degree:
//
//   x <- x / |x|_F;   `steps` times   x <- a x + (b S + c S S) x,   S = x x^T
//
// which takes every singular value s to a s + b s^3 + c s^5 and leaves the
// singular vectors; for a matrix with more rows than columns S = x^T x on the
// other side, the same result from the smaller square.
//
// A step is three products, S, P = b S + c S S and a x + P x.  S and P are
// symmetric: the tiles on and below the diagonal are computed and written to
// both places.  64 matrices of 1024 x 2048: S 544 us (0.95 PFLOP/s of what is
// computed, 10 tiles of 16 a matrix), P 326 (0.79), the sum 800 (1.03), the matrix
// units busy 57, 47 and 52% of the CUs' cycles: the 640 tiles of S and P take three
// rounds for two and a half, and the sum's 1.5 GB of addends and results, 290 us by
// themselves, overlap its products in part.  The coarse form: S 227, P 172 in one
// pass, the sum 453 in one pass and 634 in two.  Small matrices are bound by
// launches of 6 to 11 us, three a step.
//
// Roundings.  Values are held as fp16 in two parts, the nearest and the nearest
// to the rest (22 bits), times 2^12 for x and 2^8 for S and P (entries of x
// below 16 and of S and P below 256 fit; with the usual polynomials they stay
// below 1.3 and 3), and every sum in 32 bits.  A product takes both parts of
// both operands in three passes, without that of the low parts, below 2^-22: the
// result before its rounding to bf16 is 3e-7 to 8e-7 of |result| off (simulated,
// 16 x 16 to 1024 x 1024, five steps), where values held in 32 bits are 6e-7 to
// 2e-6 off.
//
// exact = false takes fewer passes.  What a product reads was chosen by what it
// costs the result (simulated; relative to |result|, random 512 x 1024, five
// steps; the result's own rounding to bf16 is 1.7e-3): x in one part for S
// 4.6e-4, S in one part for S S 2.3e-3, P in one part 1.0e-3, x in one part for P
// x 9e-4, x in one part where it is added 1.4e-3.  What the last two steps round
// weighs most (the ones before are 6e-4 off with all of that but the last in one
// part).  So the sum takes both parts of x, S and P x one part of x; S S both
// parts of both and P x both of P, but for the first three steps of matrices of
// 256 rows and more (roundings of smaller ones add up less evenly: 2e-3 and more
// so), unless they are among the last two, which take one: 1.1e-3 in all.  bf16
// in one part, as such steps are often run, is 2.1e-2 off.
#include "qb_gemm16.hpp"

namespace qbk {

constexpr float kScaleX = 4096.f, kScaleS = 256.f;

// Sums of squares in 64 bits, one for each of `gridDim.x` stretches of a matrix: bound by the 4 bytes a value (64 matrices
// of 1024 x 2048: 105 us, 5.1 TB/s).
__global__ __launch_bounds__(256) void k_ortho_sums(const float* __restrict__ x, int64_t n, double* __restrict__ sums) {
  __shared__ double part[4];
  const float* p = x + int64_t(blockIdx.y) * n;
  const int64_t each = ((n + gridDim.x - 1) / gridDim.x + 3) / 4 * 4, first = each * blockIdx.x;
  const int64_t last = first + each < n ? first + each : n;
  double t = 0;
  constexpr int U = 4;
  int64_t i = first + threadIdx.x * 4;
  for (; i + (U - 1) * 1024 + 3 < last; i += U * 1024) {
    Float4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = *reinterpret_cast<const Float4*>(p + i + u * 1024);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int c = 0; c < 4; ++c) t += double(v[u].v[c]) * double(v[u].v[c]);
  }
  for (; i < last; i += 1024)
    for (int64_t k = i; k < i + 4 && k < last; ++k) t += double(p[k]) * double(p[k]);
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) t += __shfl_xor(t, d);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = t;
  __syncthreads();
  if (threadIdx.x == 0) sums[int64_t(blockIdx.y) * kOrthoSums + blockIdx.x] = (part[0] + part[1]) + (part[2] + part[3]);
}

// x / |x| in two parts, zeros in what rounds a row up: 4 bytes in and 4 out a value (the same matrices: 255 us, 4.2 TB/s).
__global__ __launch_bounds__(256) void k_ortho_scale(const float* __restrict__ x, int N, int C, int64_t ld, int parts,
                                                     const double* __restrict__ sums, int64_t part,
                                                     uint16_t* __restrict__ out) {
  const int64_t g = blockIdx.y;
  double t = 0;
  for (int i = 0; i < parts; ++i) t += sums[g * kOrthoSums + i];
  // (a zero matrix stays zero; one with a NaN or an infinity becomes NaN)
  const double f = t > 0 ? double(kScaleX) / __builtin_sqrt(t) : t;
  const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;  // 8 values each
  const int64_t per = ld / 8;
  if (i >= N * per) return;
  const int64_t row = i / per;
  const int col = int(i % per) * 8;
  const float* p = x + (g * N + row) * C + col;
  float v[8];
  if (col + 7 < C) {
    const Float4 v0 = *reinterpret_cast<const Float4*>(p), v1 = *reinterpret_cast<const Float4*>(p + 4);
#pragma unroll
    for (int c = 0; c < 4; ++c) v[c] = v0.v[c], v[4 + c] = v1.v[c];
  } else {
#pragma unroll
    for (int c = 0; c < 8; ++c) v[c] = col + c < C ? p[c] : 0.f;
  }
  uint32_t hi[4], lo[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint16_t h[2], l[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) split16(col + 2 * k + c < C ? float(double(v[2 * k + c]) * f) : 0.f, h[c], l[c]);
    hi[k] = h[0] | uint32_t(h[1]) << 16;
    lo[k] = l[0] | uint32_t(l[1]) << 16;
  }
  uint16_t* o = out + (g * N + row) * ld + col;
  *reinterpret_cast<uint4*>(o) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
  *reinterpret_cast<uint4*>(o + part) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
}

// ---------------------------------------------------------------------------

template <int KIND, bool A_KS, bool B_KS, int PARTS, int PA, int PB, int B, int S>
static int tiled(Gemm16 g, int64_t tiles, hipStream_t st) {
  if (tiles > INT32_MAX / 2) return int(hipErrorInvalidValue);
  g.tiles = int(tiles);
  const int64_t most = int64_t(device_cu_count()) * (B == 256 ? 1 : 2);
  hipLaunchKernelGGL((k_gemm16<_Float16, KIND, A_KS, B_KS, B, S, true, PARTS, PA, PB>),
                     dim3(unsigned(std::min(tiles, most))), dim3(B == 256 ? 512 : 256), 0, st, g);
  return int(hipGetLastError());
}

// The smallest tiles while they all run at once (five steps of 2 matrices of 1024 x 1024 409 us, 572 in 128 x 128; of 20
// of 512 x 512, which are too many for that, 452 and 433), then by whole rounds: in_large_tiles.
template <int KIND, bool A_KS, bool B_KS, int PARTS, int PA, int PB>
static int product(const Gemm16& g, hipStream_t st) {
  const int64_t cu = device_cu_count();
  auto tiles = [&](int b) -> int64_t {
    const int64_t tm = (g.M + b - 1) / b, tn = (g.N + b - 1) / b;
    return g.G * (KIND == kStep ? tm * tn : tm * (tm + 1) / 2);
  };
  const int64_t t256 = tiles(256), t128 = tiles(128), t64 = tiles(64);
  if (t64 <= 2 * cu) return tiled<KIND, A_KS, B_KS, PARTS, PA, PB, 64, 4>(g, t64, st);
  if (in_large_tiles(t256, t128, 0.0)) return tiled<KIND, A_KS, B_KS, PARTS, PA, PB, 256, 2>(g, t256, st);
  return tiled<KIND, A_KS, B_KS, PARTS, PA, PB, 128, 2>(g, t128, st);
}

int launch_orthogonalize(const float* x, int G, int N, int C, int steps, float a, float b, float c, bool exact,
                         uint16_t* o, uint8_t* ws, hipStream_t st) {
  const OrthoWs w = ortho_ws_layout(G, N, C);
  double* sums = reinterpret_cast<double*>(ws);
  uint16_t* xs[2] = {reinterpret_cast<uint16_t*>(ws + w.x0), reinterpret_cast<uint16_t*>(ws + w.x1)};
  uint16_t *s = reinterpret_cast<uint16_t*>(ws + w.s), *p = reinterpret_cast<uint16_t*>(ws + w.p);
  const int64_t n = int64_t(N) * C, mat_x = N * w.ldx, mat_s = w.R * w.ldr;
  const int64_t part_x = G * mat_x, part_s = G * mat_s;
  // a workgroup for 4096 values, as many as a matrix has room for
  const int sums_of = int(std::max<int64_t>(1, std::min<int64_t>(kOrthoSums, n / 4096)));
  hipLaunchKernelGGL(k_ortho_sums, dim3(unsigned(sums_of), unsigned(G)), dim3(256), 0, st, x, n, sums);
  hipLaunchKernelGGL(k_ortho_scale, dim3(unsigned((N * (w.ldx / 8) + 255) / 256), unsigned(G)), dim3(256), 0, st, x, N, C,
                     w.ldx, sums_of, sums, part_x, xs[0]);
  if (int rc = int(hipGetLastError())) return rc;
  for (int i = 0; i < steps; ++i) {
    const uint16_t* now = xs[i & 1];
    Gemm16 g{};
    g.G = G;
    g.splits = 1;
    g.out_parts = 2;
    // S
    g.A = g.B = now;
    g.lda = g.ldb = w.ldx;
    g.mat_a = g.mat_b = mat_x;
    g.part_a = g.part_b = part_x;
    g.M = g.N = int(w.R);
    g.K = w.tall ? N : C;
    g.out = s;
    g.ldo = w.ldr;
    g.mat_out = mat_s;
    g.part_out = part_s;
    g.by_sum = kScaleS / (kScaleX * kScaleX);
    int rc;
    if (exact)
      rc = w.tall ? product<kSym, true, true, 3, 0b100, 0b010>(g, st) : product<kSym, false, false, 3, 0b100, 0b010>(g, st);
    else
      rc = w.tall ? product<kSym, true, true, 1, 0, 0>(g, st) : product<kSym, false, false, 1, 0, 0>(g, st);
    if (rc) return rc;
    // P
    g.A = g.B = s;
    g.lda = g.ldb = w.ldr;
    g.mat_a = g.mat_b = mat_s;
    g.part_a = g.part_b = part_s;
    g.K = int(w.R);
    g.add = s;
    g.out = p;
    g.by_sum = c / kScaleS;
    g.by_add = b;
    // (8 matrices of 512 x 1024 coarsely: 226 us, 262 without it)
    const bool rough = !exact && w.R >= 256 && i < 3 && i + 2 < steps;
    g.out_parts = rough ? 1 : 2;
    rc = rough ? product<kSqr, false, false, 1, 0, 0>(g, st) : product<kSqr, false, false, 3, 0b100, 0b010>(g, st);
    if (rc) return rc;
    // a x + P x, or a x + x P
    g.M = N;
    g.N = C;
    g.K = int(w.R);
    g.add = now;
    g.out = xs[1 - (i & 1)];
    g.ldo = w.ldx;
    g.mat_out = mat_x;
    g.part_out = part_x;
    g.by_sum = 1.f / kScaleS;
    g.by_add = a;
    g.out_parts = 2;
    g.last = i + 1 == steps ? o : nullptr;
    g.by_last = 1.f / kScaleX;
    if (w.tall) {
      g.A = now;
      g.lda = w.ldx;
      g.mat_a = mat_x;
      g.part_a = part_x;
      g.B = p;
      g.ldb = w.ldr;
      g.mat_b = mat_s;
      g.part_b = part_s;
      rc = exact   ? product<kStep, false, false, 3, 0b100, 0b010>(g, st)
           : rough ? product<kStep, false, false, 1, 0, 0>(g, st)
                   : product<kStep, false, false, 2, 0, 0b10>(g, st);
    } else {
      g.A = p;
      g.B = now;
      g.ldb = w.ldx;
      g.mat_b = mat_x;
      g.part_b = part_x;
      rc = exact   ? product<kStep, false, true, 3, 0b100, 0b010>(g, st)
           : rough ? product<kStep, false, true, 1, 0, 0>(g, st)
                   : product<kStep, false, true, 2, 0b10, 0>(g, st);
    }
    if (rc) return rc;
  }
  return 0;
}

}  // namespace qbk
