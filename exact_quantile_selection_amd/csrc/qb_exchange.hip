// qb_exchange.hip -- the exchange between tokens and experts: the order that
// puts each expert's (token, choice) pairs side by side, the gate-weighted
// sum of what the experts return, and its gradients.
//
// dispatch, with pair i = t K + k and e = topk[i] (outside [0, E): unrouted):
//   count_e = |{i : topk[i] = e}|,  off_0 = 0,  off_{e+1} = off_e + count_e
//             rounded up to a multiple of `align`
//   pos[i] = off_e + |{j < i : topk[j] = e}|  (-1 if unrouted),
//   row_src[pos[i]] = t, and -1 for every other row
// so the order inside an expert is that of the pairs (a stable counting
// sort: the same on every run).  A block of pairs is counted with 64-lane
// ballots (the lanes that share an expert, from its 8 bits), which gives each
// pair its rank among its wave's pairs without atomics.  Up to 8192 pairs one
// workgroup does everything in one launch; above, one launch counts blocks of
// pairs and a second ranks them, each workgroup adding up the counts of the
// blocks before its own (from L2); only where those are many does a launch
// between add them up once for all.
//
// combine:           out_t   = sum_k gate_tk rows[pos_tk]
// combine backward:  dgate_tk = <dout_t, rows[pos_tk]>,  drows[pos_tk] = gate_tk dout_t,
//                    0 in rows that no pair fills
// Both are streams of rows bound by HBM: a token is owned by up to 256 lanes
// with 8 columns each per step, so a row of `dout` is read once for its K
// rows and every access is 16 bytes a lane; sums are held in 32 bits and
// rounded once.  32,768 tokens x 8 x 2048: the sum 203 us (5.9 TB/s), the
// gradients 446 (5.4; a copy of 1 GiB reaches 5.1, a fill 6.9).
#include <algorithm>
#include <type_traits>

#include "qb_device.hpp"
#include "qb_internal.hpp"

namespace qbk {

constexpr int kDispThreads = 1024;
constexpr int kDispWaves = kDispThreads / kWave;
constexpr int kDispSteps = 8;                           // 64-pair steps per wave held in registers
constexpr int kDispMost = kDispThreads * kDispSteps;    // pairs of one workgroup at most

// Pairs per workgroup: at most 128 workgroups' counts to add up until that
// takes more than kDispMost pairs each.
static int64_t dispatch_block(int64_t pairs) {
  if (pairs <= kDispMost) return kDispMost;
  const int64_t want = (pairs + 127) / 128;
  const int64_t b = (want + kDispThreads - 1) / kDispThreads * kDispThreads;
  return std::min<int64_t>(b, kDispMost);
}
static int64_t dispatch_blocks(int64_t pairs) {
  const int64_t b = dispatch_block(pairs);
  return std::max<int64_t>(1, (pairs + b - 1) / b);
}
static int table_row(int E) { return (E + 3) / 4 * 4; }
// Above this many blocks a launch between turns the counts into sums (8 of 256
// experts each: 2^18 tokens, 256 blocks, 28 us either way; 2^20 tokens 102 us
// without it and 68 with it, 2^24 11.1 ms and 1.04).
constexpr int64_t kDispScan = 256;

int64_t dispatch_ws_bytes(int64_t pairs, int E) {
  const int64_t n = dispatch_blocks(pairs);
  return n <= 1 ? 0 : (n + (n > kDispScan)) * table_row(E) * 4;
}

__global__ __launch_bounds__(kDispThreads) void k_dispatch_count(const int32_t* __restrict__ topk, int64_t pairs,
                                                                 int64_t per, int E, int ER,
                                                                 int32_t* __restrict__ table) {
  __shared__ int cnt[256];
  const int tid = threadIdx.x;
  if (tid < 256) cnt[tid] = 0;
  __syncthreads();
  const int64_t i0 = int64_t(blockIdx.x) * per;
  const int64_t i1 = i0 + per < pairs ? i0 + per : pairs;
  for (int64_t i = i0 + tid; i < i1; i += kDispThreads) {
    const int e = topk[i];
    if (unsigned(e) < unsigned(E)) atomicAdd(&cnt[e], 1);
  }
  __syncthreads();
  if (tid < ER) table[int64_t(blockIdx.x) * ER + tid] = cnt[tid];
}

// The table's counts become those of the blocks before each; a last row has
// all blocks'.  A workgroup takes 4 experts, a thread a run of blocks.
__global__ __launch_bounds__(kDispThreads) void k_dispatch_scan(int32_t* __restrict__ table, int n, int ER) {
  __shared__ int part[kDispWaves][4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int each = (n + kDispThreads - 1) / kDispThreads;
  const int j0 = tid * each < n ? tid * each : n, j1 = j0 + each < n ? j0 + each : n;
  int32_t* const col = table + 4 * blockIdx.x;
  int sum[4] = {0, 0, 0, 0}, run[4];
  for (int j = j0; j < j1; ++j) {
    const int4 v = *reinterpret_cast<const int4*>(col + int64_t(j) * ER);
    sum[0] += v.x, sum[1] += v.y, sum[2] += v.z, sum[3] += v.w;
  }
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    run[c] = sum[c];
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
      const int o = __shfl_up(run[c], d);
      run[c] += lane >= d ? o : 0;
    }
    if (lane == kWave - 1) part[wave][c] = run[c];
    run[c] -= sum[c];
  }
  __syncthreads();
#pragma unroll
  for (int c = 0; c < 4; ++c)
    for (int w = 0; w < wave; ++w) run[c] += part[w][c];
  for (int j = j0; j < j1; ++j) {
    int4* const at = reinterpret_cast<int4*>(col + int64_t(j) * ER);
    const int4 v = *at;
    *at = make_int4(run[0], run[1], run[2], run[3]);
    run[0] += v.x, run[1] += v.y, run[2] += v.z, run[3] += v.w;
  }
  if (tid == kDispThreads - 1)
    *reinterpret_cast<int4*>(col + int64_t(n) * ER) = make_int4(run[0], run[1], run[2], run[3]);
}

__global__ __launch_bounds__(kDispThreads) void k_dispatch(const int32_t* __restrict__ topk, int64_t pairs,
                                                           int64_t per, int K, int E, int ER, int align,
                                                           const int32_t* __restrict__ table, bool scanned,
                                                           int32_t* __restrict__ off, int64_t R,
                                                           int32_t* __restrict__ row_src,
                                                           int32_t* __restrict__ pos) {
  __shared__ int wcnt[kDispWaves][256];   // counts, then first rows, per wave and expert
  __shared__ __align__(16) int before[256], total[256];
  __shared__ int start[257], used[256];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int nblk = int(gridDim.x), blk = int(blockIdx.x);
  for (int j = tid; j < kDispWaves * 256; j += kDispThreads) (&wcnt[0][0])[j] = 0;
  if (tid < 256) before[tid] = total[tid] = 0;
  __syncthreads();

  // this wave's pairs, in order, and their ranks among the wave's pairs
  const int64_t i0 = int64_t(blk) * per;
  const int64_t i1 = i0 + per < pairs ? i0 + per : pairs;
  const int steps = int((per + kDispThreads - 1) / kDispThreads);
  const int64_t w0 = i0 + int64_t(wave) * steps * kWave;
  int ex[kDispSteps], rank[kDispSteps];
#pragma unroll
  for (int u = 0; u < kDispSteps; ++u) {
    const int64_t i = w0 + u * kWave + lane;
    int e = u < steps && i < i1 ? topk[i] : -1;
    ex[u] = unsigned(e) < unsigned(E) ? e : -1;
  }
#pragma unroll
  for (int u = 0; u < kDispSteps; ++u) {
    if (u < steps) {
      const int e = ex[u];
      uint64_t same = __ballot(e >= 0);
      if (same != 0) {
#pragma unroll
        for (int bit = 0; bit < 8; ++bit) {
          const uint64_t m = __ballot((e >> bit) & 1);
          same &= ((e >> bit) & 1) ? m : ~m;
        }
        const uint64_t below = same & ((1ull << lane) - 1ull);
        const int old = e >= 0 ? wcnt[wave][e] : 0;
        rank[u] = old + __popcll(below);
        __builtin_amdgcn_wave_barrier();
        asm volatile("" ::: "memory");
        if (e >= 0 && below == 0) wcnt[wave][e] = old + __popcll(same);
        asm volatile("" ::: "memory");
        __builtin_amdgcn_wave_barrier();
      }
    }
  }
  // the counts of the blocks before this one, and of all
  if (scanned) {
    if (tid < ER) {
      before[tid] = table[int64_t(blk) * ER + tid];
      total[tid] = table[int64_t(nblk) * ER + tid];
    }
  } else if (nblk > 1) {
    const int quads = ER / 4;              // 64 threads or fewer take one row of the table, 4 experts each
    const int qd = tid & 63, slice = tid >> 6;
    if (qd < quads) {
      int4 bsum = make_int4(0, 0, 0, 0), tsum = make_int4(0, 0, 0, 0);
      for (int j = slice; j < nblk; j += kDispWaves) {
        const int4 v = *reinterpret_cast<const int4*>(table + int64_t(j) * ER + 4 * qd);
        tsum.x += v.x, tsum.y += v.y, tsum.z += v.z, tsum.w += v.w;
        if (j < blk) bsum.x += v.x, bsum.y += v.y, bsum.z += v.z, bsum.w += v.w;
      }
      atomicAdd(&before[4 * qd], bsum.x), atomicAdd(&before[4 * qd + 1], bsum.y);
      atomicAdd(&before[4 * qd + 2], bsum.z), atomicAdd(&before[4 * qd + 3], bsum.w);
      atomicAdd(&total[4 * qd], tsum.x), atomicAdd(&total[4 * qd + 1], tsum.y);
      atomicAdd(&total[4 * qd + 2], tsum.z), atomicAdd(&total[4 * qd + 3], tsum.w);
    }
  }
  __syncthreads();
  // per expert: running sum over the waves
  if (tid < 256) {
    int run = before[tid];
#pragma unroll
    for (int w = 0; w < kDispWaves; ++w) {
      const int c = wcnt[w][tid];
      wcnt[w][tid] = run;
      run += c;
    }
    if (nblk == 1) total[tid] = run;
  }
  __syncthreads();
  // the experts' first rows: 4 experts a lane of wave 0
  if (wave == 0) {
    int c[4], sum = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int t = total[4 * lane + j];
      used[4 * lane + j] = t;
      // (t + align - 1 may pass 2^31 though the rows do not)
      c[j] = int((unsigned(t) + unsigned(align) - 1u) / unsigned(align) * unsigned(align));
      sum += c[j];
    }
    int run = sum;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
      const int o = __shfl_up(run, d);
      run += lane >= d ? o : 0;
    }
    int at = run - sum;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      start[4 * lane + j] = at;
      at += c[j];
    }
    if (lane == kWave - 1) start[256] = at;
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < kDispSteps; ++u) {
    if (u < steps) {
      const int64_t i = w0 + u * kWave + lane;
      if (i < i1) {
        const int e = ex[u];
        int row = -1;
        if (e >= 0) {
          row = start[e] + wcnt[wave][e] + rank[u];
          row = row < R ? row : -1;
          if (row >= 0) row_src[row] = int(i / K);
        }
        pos[i] = row;
      }
    }
  }
  // off, the rows between an expert's last pair and the next expert, and the
  // rows past the last expert
  if (blk == 0)
    for (int j = tid; j <= E; j += kDispThreads) off[j] = start[j];
  if (align > 1)  // (else there are none of the former: 16 tokens of 256 experts 4.9 -> 3.8 us)
    for (int e = blk + nblk * wave; e < E; e += nblk * kDispWaves)
      for (int64_t r = int64_t(start[e]) + used[e] + lane; r < start[e + 1] && r < R; r += kWave) row_src[r] = -1;
  for (int64_t r = int64_t(start[E]) + int64_t(blk) * kDispThreads + tid; r < R; r += int64_t(nblk) * kDispThreads)
    row_src[r] = -1;
}

int launch_dispatch(const Dispatch& a, hipStream_t st) {
  const int64_t per = dispatch_block(a.pairs), n = dispatch_blocks(a.pairs);
  const int ER = table_row(a.E);
  if (n > 1) {
    hipLaunchKernelGGL(k_dispatch_count, dim3(unsigned(n)), dim3(kDispThreads), 0, st, a.topk, a.pairs, per, a.E, ER,
                       a.ws);
    int rc = int(hipGetLastError());
    if (rc != int(hipSuccess)) return rc;
    if (n > kDispScan) {
      hipLaunchKernelGGL(k_dispatch_scan, dim3(unsigned(ER / 4)), dim3(kDispThreads), 0, st, a.ws, int(n), ER);
      rc = int(hipGetLastError());
      if (rc != int(hipSuccess)) return rc;
    }
  }
  // one workgroup takes only as many steps as its pairs need
  const int64_t mine = n > 1 ? per : std::max<int64_t>(1, (a.pairs + kDispThreads - 1) / kDispThreads) * kDispThreads;
  hipLaunchKernelGGL(k_dispatch, dim3(unsigned(n)), dim3(kDispThreads), 0, st, a.topk, a.pairs, mine, a.K, a.E, ER,
                     a.align, a.ws, n > kDispScan, a.off, a.R, a.row_src, a.pos);
  return int(hipGetLastError());
}

// ---------------------------------------------------------------------------

// 8 bf16 of a row (the address needs only the element's alignment); NT: past
// the caches, for what no cache holds long enough to be read again.
typedef uint32_t bf8 __attribute__((ext_vector_type(4), aligned(2)));

__device__ __forceinline__ float bf_lo(uint32_t p) { return __builtin_bit_cast(float, p << 16); }
__device__ __forceinline__ float bf_hi(uint32_t p) { return __builtin_bit_cast(float, p & 0xFFFF0000u); }

// A lane's 8 columns, h0 on.  Near a row's end they begin earlier, at H - 8,
// so that every access is whole: the columns that the lane before has too are
// computed and written twice, to the same values.  Rows of fewer than 8
// columns (SHORT: kernels of their own, as the branches would cost every
// other row more than its loads) go element by element.
template <bool NT, bool SHORT>
__device__ __forceinline__ bf8 ld_bf8(const uint16_t* p, int H) {
  if constexpr (SHORT) {
    bf8 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = 2 * i < H ? p[2 * i] : 0, hi = 2 * i + 1 < H ? p[2 * i + 1] : 0;
      v[i] = lo | (hi << 16);
    }
    return v;
  } else if constexpr (NT) {
    return __builtin_nontemporal_load(reinterpret_cast<const bf8*>(p));
  } else {
    return *reinterpret_cast<const bf8*>(p);
  }
}
template <bool NT, bool SHORT>
__device__ __forceinline__ void st_bf8(uint16_t* p, int H, bf8 v) {
  if constexpr (SHORT) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (2 * i < H) p[2 * i] = uint16_t(v[i]);
      if (2 * i + 1 < H) p[2 * i + 1] = uint16_t(v[i] >> 16);
    }
  } else if constexpr (NT) {
    __builtin_nontemporal_store(v, reinterpret_cast<bf8*>(p));
  } else {
    *reinterpret_cast<bf8*>(p) = v;
  }
}
// A value that all lanes of a token hold: one for the wave where the token has all of it.
template <int LT, class V>
__device__ __forceinline__ V of_token(V x) {
  if constexpr (LT >= kWave) return __builtin_bit_cast(V, __builtin_amdgcn_readfirstlane(__builtin_bit_cast(int, x)));
  return x;
}
__device__ __forceinline__ int bf8_column(int h0, int H) { return H < 8 ? 0 : (h0 < H - 8 ? h0 : H - 8); }

// LT lanes own a token: as many as its row has 8 columns for, 256 at most, so
// that a row's 4 KiB are read by one workgroup at once.
template <int LT, bool NT, bool SHORT = false>
__global__ __launch_bounds__(256) void k_combine(const uint16_t* __restrict__ rows, int64_t R,
                                                 const int32_t* __restrict__ pos, const float* __restrict__ gate,
                                                 int64_t N, int K, int H, uint16_t* __restrict__ out) {
  const int tl = threadIdx.x % LT;
  const int64_t t = int64_t(blockIdx.x) * (256 / LT) + threadIdx.x / LT;
  if (t >= N) return;
  const int h0 = (int(blockIdx.y) * LT + tl) * 8;
  if (h0 >= H) return;
  const int at = bf8_column(h0, H);
  float acc[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.f;
  for (int k0 = 0; k0 < K; k0 += 8) {
    bf8 v[8];
    float g[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int k = k0 + u;
      const int p = of_token<LT>(k < K ? pos[t * K + k] : -1);
      const bool on = p >= 0 && p < R;
      g[u] = on ? (gate ? gate[t * K + k] : 1.0f) : 0.f;
      v[u] = on ? ld_bf8<NT, SHORT>(rows + int64_t(p) * H + at, H) : (bf8){0, 0, 0, 0};
    }
#pragma unroll
    for (int u = 0; u < 8; ++u)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[2 * i] = fmaf(g[u], bf_lo(v[u][i]), acc[2 * i]);
        acc[2 * i + 1] = fmaf(g[u], bf_hi(v[u][i]), acc[2 * i + 1]);
      }
  }
  bf8 o;
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = bf16x2_rne(acc[2 * i], acc[2 * i + 1]);
  st_bf8<NT, SHORT>(out + t * H + at, H, o);
}

// The sums of eight values over L lanes (64 at most), value (lane >> 3) & 7
// of them in every lane for L = 64: each exchange halves how many a lane
// carries, so that they cost 10 shuffles together and not 48.
template <int L>
__device__ __forceinline__ void sum8(float (&v)[8], int lane) {
  int have = 8;
#pragma unroll
  for (int d = L / 2; d >= 1; d >>= 1) {
    if (have > 1) {
      const bool up = lane & d;
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (u < have / 2) {
          const float keep = up ? v[u + have / 2] : v[u], give = up ? v[u] : v[u + have / 2];
          v[u] = keep + __shfl_xor(give, d);
        }
      have /= 2;
    } else {
      v[0] += __shfl_xor(v[0], d);
    }
  }
}

template <int LT, bool DG, bool NT, bool SHORT = false>
__global__ __launch_bounds__(256) void k_combine_bwd(const uint16_t* __restrict__ dout,
                                                     const uint16_t* __restrict__ rows, int64_t R,
                                                     const int32_t* __restrict__ pos,
                                                     const int32_t* __restrict__ row_src,
                                                     const float* __restrict__ gate, int64_t N, int K, int H,
                                                     int64_t row_blocks, uint16_t* __restrict__ drows,
                                                     float* __restrict__ dgate) {
  constexpr int L = LT < kWave ? LT : kWave;  // of one wave
  __shared__ float part[4][8];
  const int lane = threadIdx.x & 63;
  if (blockIdx.x < row_blocks) {
    // rows that no pair fills: 16 rows a wave, zeroed by all its lanes (they come first, so that they fill the gaps
    // between the tokens' work rather than follow it)
    for (int64_t r0 = (int64_t(blockIdx.x) * 4 + (threadIdx.x >> 6)) * 16; r0 < R; r0 += row_blocks * 64) {
      const bool empty = lane < 16 && r0 + lane < R && row_src[r0 + lane] < 0;
      uint64_t m = __ballot(empty);
      while (m) {
        const int j = __builtin_ctzll(m);
        m &= m - 1;
        uint16_t* dst = drows + (r0 + j) * H;
        for (int h = lane * 8; h < H; h += kWave * 8) st_bf8<NT, SHORT>(dst + bf8_column(h, H), H, (bf8){0, 0, 0, 0});
      }
    }
    return;
  }
  const int tl = threadIdx.x % LT;
  const int64_t t = (int64_t(blockIdx.x) - row_blocks) * (256 / LT) + threadIdx.x / LT;
  const bool live = t < N;
  for (int k0 = 0; k0 < K; k0 += 8) {
    int p[8];
    float g[8], dot[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int k = k0 + u;
      const int q = live && k < K ? pos[t * K + k] : -1;
      p[u] = of_token<LT>(q < R ? q : -1);
      g[u] = of_token<LT>(p[u] >= 0 ? (gate ? gate[t * K + k] : 1.0f) : 0.f);
      dot[u] = 0.f;
    }
    if (live) {
      for (int h0 = tl * 8; h0 < H; h0 += LT * 8) {
        const int at = bf8_column(h0, H);
        const bf8 d = ld_bf8<false, SHORT>(dout + t * H + at, H);
        bf8 v[DG ? 8 : 1];
        if constexpr (DG) {
#pragma unroll
          for (int u = 0; u < 8; ++u)
            if (p[u] >= 0) v[u] = ld_bf8<NT, SHORT>(rows + int64_t(p[u]) * H + at, H);
        }
        float df[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) df[2 * i] = bf_lo(d[i]), df[2 * i + 1] = bf_hi(d[i]);
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          if (p[u] < 0) continue;
          bf8 o;
#pragma unroll
          for (int i = 0; i < 4; ++i) o[i] = bf16x2_rne(g[u] * df[2 * i], g[u] * df[2 * i + 1]);
          st_bf8<NT, SHORT>(drows + int64_t(p[u]) * H + at, H, o);
        }
        if constexpr (DG) {
          const int seen = h0 - at;  // columns that the lane before counts
          auto add = [&](auto all) {
#pragma unroll
            for (int u = 0; u < 8; ++u) {
              if (p[u] < 0) continue;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                if (all() || 2 * i >= seen) dot[u] = fmaf(df[2 * i], bf_lo(v[u][i]), dot[u]);
                if (all() || 2 * i + 1 >= seen) dot[u] = fmaf(df[2 * i + 1], bf_hi(v[u][i]), dot[u]);
              }
            }
          };
          if (seen == 0)
            add(std::true_type{});
          else
            add(std::false_type{});
        }
      }
    }
    if constexpr (DG) {
      sum8<L>(dot, lane);
      // bits of the lane, from the highest that sum8 exchanged, number the value
      constexpr int TOP = L >= 8 ? L / 8 : 1;  // lanes that end up with the same value
      const int u = (tl % L) / TOP;
      if constexpr (LT > kWave) {
        __syncthreads();
        if (lane % TOP == 0) part[threadIdx.x >> 6][lane / TOP] = dot[0];
        __syncthreads();
        constexpr int WT = LT / kWave;  // waves of a token
        if (tl < 8 && live && k0 + tl < K) {
          float sum = 0.f;
#pragma unroll
          for (int w = 0; w < WT; ++w) sum += part[(threadIdx.x >> 6) + w][tl];
          dgate[t * K + k0 + tl] = sum;
        }
      } else if (live && tl % TOP == 0 && k0 + u < K) {
        dgate[t * K + k0 + u] = dot[0];
      }
    }
  }
}

// A launch takes fewer than 2^32 threads along an axis: above 2^23 tokens one
// has 128 lanes at most, and the rows that no pair fills are gone through by
// kZeroBlocks workgroups at most, 64 rows each at a time.
constexpr int64_t kZeroBlocks = int64_t(1) << 17;

// Lanes that own a token, and whether its rows are too many bytes for any
// cache (256 MiB, the last one's size): then they pass it by (262,144 rows of
// 2048: 239 -> 195 us, the backward 495 -> 451).
static int lanes_per_token(int64_t N, int H) {
  if (H > 1024 && N <= (int64_t(1) << 23)) return 256;
  return H <= 64 ? 8 : (H <= 128 ? 16 : (H <= 256 ? 32 : (H <= 512 ? 64 : 128)));
}
static bool past_caches(int64_t R, int H) { return R * H * 2 > (int64_t(256) << 20); }

template <int LT>
static int combine_lt(const uint16_t* rows, int64_t R, const int32_t* pos, const float* gate, int64_t N, int K, int H,
                      uint16_t* out, hipStream_t st) {
  const dim3 grid{unsigned((N * LT + 255) / 256), unsigned((H + LT * 8 - 1) / (LT * 8)), 1u}, block{256u, 1u, 1u};
  if (LT == 8 && H < 8)
    hipLaunchKernelGGL((k_combine<8, false, true>), grid, block, 0, st, rows, R, pos, gate, N, K, H, out);
  else if (past_caches(R, H))
    hipLaunchKernelGGL((k_combine<LT, true>), grid, block, 0, st, rows, R, pos, gate, N, K, H, out);
  else
    hipLaunchKernelGGL((k_combine<LT, false>), grid, block, 0, st, rows, R, pos, gate, N, K, H, out);
  return int(hipGetLastError());
}

int launch_combine(const uint16_t* rows, int64_t R, const int32_t* pos, const float* gate, int64_t N, int K, int H,
                   uint16_t* out, hipStream_t st) {
  switch (lanes_per_token(N, H)) {
    case 8: return combine_lt<8>(rows, R, pos, gate, N, K, H, out, st);
    case 16: return combine_lt<16>(rows, R, pos, gate, N, K, H, out, st);
    case 32: return combine_lt<32>(rows, R, pos, gate, N, K, H, out, st);
    case 64: return combine_lt<64>(rows, R, pos, gate, N, K, H, out, st);
    case 128: return combine_lt<128>(rows, R, pos, gate, N, K, H, out, st);
    default: return combine_lt<256>(rows, R, pos, gate, N, K, H, out, st);
  }
}

template <int LT>
static int bwd_lt(const uint16_t* dout, const uint16_t* rows, int64_t R, const int32_t* pos, const int32_t* row_src,
                  const float* gate, int64_t N, int K, int H, uint16_t* drows, float* dgate, hipStream_t st) {
  const int64_t tb = (N * LT + 255) / 256, rb = std::min((R + 63) / 64, kZeroBlocks);
  const dim3 grid{unsigned(tb + rb), 1u, 1u}, block{256u, 1u, 1u};
#define QB_BWD(LANES, DG, NT, SHORT)                                                                                \
  hipLaunchKernelGGL((k_combine_bwd<LANES, DG, NT, SHORT>), grid, block, 0, st, dout, rows, R, pos, row_src, gate, N, \
                     K, H, rb, drows, dgate)
  if (LT == 8 && H < 8) {
    if (dgate) QB_BWD(8, true, false, true); else QB_BWD(8, false, false, true);
  } else if (past_caches(R, H)) {
    if (dgate) QB_BWD(LT, true, true, false); else QB_BWD(LT, false, true, false);
  } else {
    if (dgate) QB_BWD(LT, true, false, false); else QB_BWD(LT, false, false, false);
  }
#undef QB_BWD
  return int(hipGetLastError());
}

int launch_combine_bwd(const uint16_t* dout, const uint16_t* rows, int64_t R, const int32_t* pos,
                       const int32_t* row_src, const float* gate, int64_t N, int K, int H, uint16_t* drows,
                       float* dgate, hipStream_t st) {
  // 64 lanes a token while its rows stay in the caches: more need a barrier for the sums over their waves (3001 tokens
  // of 1101: 31 us, 36 with 256 lanes; 32,768 of 2048: 471 and 451)
  switch (past_caches(R, H) ? lanes_per_token(N, H) : std::min(lanes_per_token(N, H), 64)) {
    case 8: return bwd_lt<8>(dout, rows, R, pos, row_src, gate, N, K, H, drows, dgate, st);
    case 16: return bwd_lt<16>(dout, rows, R, pos, row_src, gate, N, K, H, drows, dgate, st);
    case 32: return bwd_lt<32>(dout, rows, R, pos, row_src, gate, N, K, H, drows, dgate, st);
    case 64: return bwd_lt<64>(dout, rows, R, pos, row_src, gate, N, K, H, drows, dgate, st);
    case 128: return bwd_lt<128>(dout, rows, R, pos, row_src, gate, N, K, H, drows, dgate, st);
    default: return bwd_lt<256>(dout, rows, R, pos, row_src, gate, N, K, H, drows, dgate, st);
  }
}

}  // namespace qbk
