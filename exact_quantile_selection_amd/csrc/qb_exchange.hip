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
// blocks before its own (from L2; no scan launch between).
//
// combine:           out_t   = sum_k gate_tk rows[pos_tk]
// combine backward:  dgate_tk = <dout_t, rows[pos_tk]>,  drows[pos_tk] = gate_tk dout_t,
//                    0 in rows that no pair fills
// Both are streams of rows bound by HBM: a token is owned by up to 64 lanes
// with 8 columns each per step, so a row of `dout` is read once for its K
// rows and every access is 16 bytes a lane; sums are held in 32 bits and
// rounded once.
#include <algorithm>

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

int64_t dispatch_ws_bytes(int64_t pairs, int E) {
  const int64_t n = dispatch_blocks(pairs);
  return n <= 1 ? 0 : n * table_row(E) * 4;
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

__global__ __launch_bounds__(kDispThreads) void k_dispatch(const int32_t* __restrict__ topk, int64_t pairs,
                                                           int64_t per, int K, int E, int ER, int align,
                                                           const int32_t* __restrict__ table,
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
  if (nblk > 1) {
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
      c[j] = (t + align - 1) / align * align;
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
    const int rc = int(hipGetLastError());
    if (rc != int(hipSuccess)) return rc;
  }
  // one workgroup takes only as many steps as its pairs need
  const int64_t mine = n > 1 ? per : std::max<int64_t>(1, (a.pairs + kDispThreads - 1) / kDispThreads) * kDispThreads;
  hipLaunchKernelGGL(k_dispatch, dim3(unsigned(n)), dim3(kDispThreads), 0, st, a.topk, a.pairs, mine, a.K, a.E, ER,
                     a.align, a.ws, a.off, a.R, a.row_src, a.pos);
  return int(hipGetLastError());
}

// ---------------------------------------------------------------------------

// 8 bf16 of a row from element `at`; VEC: all 8 lie inside the row (the
// address needs only the element's alignment), else those below `n`.
struct __attribute__((packed, aligned(2))) Bf8 {
  uint32_t v[4];
};

__device__ __forceinline__ float bf_lo(uint32_t p) { return __builtin_bit_cast(float, p << 16); }
__device__ __forceinline__ float bf_hi(uint32_t p) { return __builtin_bit_cast(float, p & 0xFFFF0000u); }

__device__ __forceinline__ void ld_bf8(const uint16_t* p, int n, uint32_t (&v)[4]) {
  if (n >= 8) {
    const Bf8 t = *reinterpret_cast<const Bf8*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = t.v[i];
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t lo = 2 * i < n ? p[2 * i] : 0, hi = 2 * i + 1 < n ? p[2 * i + 1] : 0;
      v[i] = lo | (hi << 16);
    }
  }
}
__device__ __forceinline__ void st_bf8(uint16_t* p, int n, const uint32_t (&v)[4]) {
  if (n >= 8) {
    Bf8 t;
#pragma unroll
    for (int i = 0; i < 4; ++i) t.v[i] = v[i];
    *reinterpret_cast<Bf8*>(p) = t;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (2 * i < n) p[2 * i] = uint16_t(v[i]);
      if (2 * i + 1 < n) p[2 * i + 1] = uint16_t(v[i] >> 16);
    }
  }
}

// Lanes that own a token: enough for one 8-column step over the row, 64 at most.
template <int LT>
__global__ __launch_bounds__(256) void k_combine(const uint16_t* __restrict__ rows, int64_t R,
                                                 const int32_t* __restrict__ pos, const float* __restrict__ gate,
                                                 int64_t N, int K, int H, uint16_t* __restrict__ out) {
  const int tl = threadIdx.x % LT;
  const int64_t t = int64_t(blockIdx.x) * (256 / LT) + threadIdx.x / LT;
  if (t >= N) return;
  const int h0 = (int(blockIdx.y) * LT + tl) * 8;
  if (h0 >= H) return;
  const int n = H - h0;
  float acc[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.f;
  for (int k0 = 0; k0 < K; k0 += 8) {
    uint32_t v[8][4];
    float g[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int k = k0 + u;
      const int p = k < K ? pos[t * K + k] : -1;
      const bool on = p >= 0 && p < R;
      g[u] = on ? (gate ? gate[t * K + k] : 1.0f) : 0.f;
      if (on) {
        ld_bf8(rows + int64_t(p) * H + h0, n, v[u]);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[u][i] = 0;
      }
    }
#pragma unroll
    for (int u = 0; u < 8; ++u)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[2 * i] = fmaf(g[u], bf_lo(v[u][i]), acc[2 * i]);
        acc[2 * i + 1] = fmaf(g[u], bf_hi(v[u][i]), acc[2 * i + 1]);
      }
  }
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = bf16x2_rne(acc[2 * i], acc[2 * i + 1]);
  st_bf8(out + t * H + h0, n, o);
}

template <int LT, bool DG>
__global__ __launch_bounds__(256) void k_combine_bwd(const uint16_t* __restrict__ dout,
                                                     const uint16_t* __restrict__ rows, int64_t R,
                                                     const int32_t* __restrict__ pos,
                                                     const int32_t* __restrict__ row_src,
                                                     const float* __restrict__ gate, int64_t N, int K, int H,
                                                     int64_t token_blocks, uint16_t* __restrict__ drows,
                                                     float* __restrict__ dgate) {
  const int lane = threadIdx.x & 63;
  if (blockIdx.x >= token_blocks) {
    // rows that no pair fills: 64 rows a wave, zeroed by all its lanes
    const int64_t r0 = ((int64_t(blockIdx.x) - token_blocks) * 4 + (threadIdx.x >> 6)) * kWave;
    const bool empty = r0 + lane < R && row_src[r0 + lane] < 0;
    uint64_t m = __ballot(empty);
    const uint32_t zero[4] = {0, 0, 0, 0};
    while (m) {
      const int j = __builtin_ctzll(m);
      m &= m - 1;
      uint16_t* dst = drows + (r0 + j) * H;
      for (int h = lane * 8; h < H; h += kWave * 8) st_bf8(dst + h, H - h, zero);
    }
    return;
  }
  const int tl = threadIdx.x % LT;
  const int64_t t = int64_t(blockIdx.x) * (256 / LT) + threadIdx.x / LT;
  const bool live = t < N;
  for (int k0 = 0; k0 < K; k0 += 8) {
    int p[8];
    float g[8], dot[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int k = k0 + u;
      int q = live && k < K ? pos[t * K + k] : -1;
      p[u] = q < R ? q : -1;
      g[u] = p[u] >= 0 ? (gate ? gate[t * K + k] : 1.0f) : 0.f;
      dot[u] = 0.f;
    }
    if (live) {
      for (int h0 = tl * 8; h0 < H; h0 += LT * 8) {
        const int n = H - h0;
        uint32_t d[4], v[DG ? 8 : 1][4];
        ld_bf8(dout + t * H + h0, n, d);
        if constexpr (DG) {
#pragma unroll
          for (int u = 0; u < 8; ++u)
            if (p[u] >= 0) ld_bf8(rows + int64_t(p[u]) * H + h0, n, v[u]);
        }
        float df[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) df[2 * i] = bf_lo(d[i]), df[2 * i + 1] = bf_hi(d[i]);
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          if (p[u] < 0) continue;
          if constexpr (DG) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              dot[u] = fmaf(df[2 * i], bf_lo(v[u][i]), dot[u]);
              dot[u] = fmaf(df[2 * i + 1], bf_hi(v[u][i]), dot[u]);
            }
          }
          uint32_t o[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) o[i] = bf16x2_rne(g[u] * df[2 * i], g[u] * df[2 * i + 1]);
          st_bf8(drows + int64_t(p[u]) * H + h0, n, o);
        }
      }
    }
    if constexpr (DG) {
#pragma unroll
      for (int u = 0; u < 8; ++u) {
#pragma unroll
        for (int s = LT / 2; s >= 1; s >>= 1) dot[u] += __shfl_xor(dot[u], s);
        const int k = k0 + u;
        if (live && k < K && tl == (u % LT)) dgate[t * K + k] = dot[u];
      }
    }
  }
}

static int lanes_per_token(int H) { return H <= 64 ? 8 : (H <= 128 ? 16 : (H <= 256 ? 32 : 64)); }

int launch_combine(const uint16_t* rows, int64_t R, const int32_t* pos, const float* gate, int64_t N, int K, int H,
                   uint16_t* out, hipStream_t st) {
  const int LT = lanes_per_token(H);
  const dim3 grid{unsigned((N * LT + 255) / 256), unsigned((H + LT * 8 - 1) / (LT * 8)), 1u}, block{256u, 1u, 1u};
#define QB_COMBINE(L) hipLaunchKernelGGL((k_combine<L>), grid, block, 0, st, rows, R, pos, gate, N, K, H, out)
  switch (LT) {
    case 8: QB_COMBINE(8); break;
    case 16: QB_COMBINE(16); break;
    case 32: QB_COMBINE(32); break;
    default: QB_COMBINE(64); break;
  }
#undef QB_COMBINE
  return int(hipGetLastError());
}

template <int LT>
static int bwd_lt(const uint16_t* dout, const uint16_t* rows, int64_t R, const int32_t* pos, const int32_t* row_src,
                  const float* gate, int64_t N, int K, int H, uint16_t* drows, float* dgate, hipStream_t st) {
  const int64_t tb = (N * LT + 255) / 256, rb = (R + 255) / 256;
  const dim3 grid{unsigned(tb + rb), 1u, 1u}, block{256u, 1u, 1u};
  if (dgate)
    hipLaunchKernelGGL((k_combine_bwd<LT, true>), grid, block, 0, st, dout, rows, R, pos, row_src, gate, N, K, H, tb,
                       drows, dgate);
  else
    hipLaunchKernelGGL((k_combine_bwd<LT, false>), grid, block, 0, st, dout, rows, R, pos, row_src, gate, N, K, H, tb,
                       drows, dgate);
  return int(hipGetLastError());
}

int launch_combine_bwd(const uint16_t* dout, const uint16_t* rows, int64_t R, const int32_t* pos,
                       const int32_t* row_src, const float* gate, int64_t N, int K, int H, uint16_t* drows,
                       float* dgate, hipStream_t st) {
  switch (lanes_per_token(H)) {
    case 8: return bwd_lt<8>(dout, rows, R, pos, row_src, gate, N, K, H, drows, dgate, st);
    case 16: return bwd_lt<16>(dout, rows, R, pos, row_src, gate, N, K, H, drows, dgate, st);
    case 32: return bwd_lt<32>(dout, rows, R, pos, row_src, gate, N, K, H, drows, dgate, st);
    default: return bwd_lt<64>(dout, rows, R, pos, row_src, gate, N, K, H, drows, dgate, st);
  }
}

}  // namespace qbk
