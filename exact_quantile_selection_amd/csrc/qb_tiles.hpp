// qb_tiles.hpp -- what the tiled matrix products share: register types, the
// order of the tiles over the XCDs, and the search for the expert that a tile
// of rows belongs to.
#pragma once

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

}  // namespace qbk
