// qb_balance.hip -- routing with a sequence-wise balance loss: the K experts
// of every token by biased score, their normalised gates, the per-expert
// counts of every sequence, the loss, and the gradient of gates and loss
// through the sigmoid.
//
// For token i of sequence q (T_q live tokens, B sequences, n of them with a
// live token), scores s, bias b:
//   topk[i]  = the K largest of fl32(s_i + b), larger first, equal values by
//              lower expert index;  gate_ik = s_ik / sum_k s_ik
//   z_i = sum_e s_ie,  p_ie = s_ie / z_i          (0 where z_i = 0)
//   c_qe = number of live tokens of q that chose e,  f_qe = c_qe E / (K T_q)
//   loss = (coef / n) sum_q sum_e f_qe (1 / T_q) sum_{i in q} p_ie
// f is held constant in the gradient.  With g the gradient of the gates:
//   dloss/ds_ie = (w_qe - sum_e' w_qe' p_ie') / z_i,  w_qe = coef (f_qe - 1) / (n T_q)
//   (sum_e p = 1, so subtracting 1 from every f changes nothing and keeps the
//   small differences that carry the signal in 32 bits)
//   dgate/ds_ik = (g_ik - sum_k' g_ik' gate_ik') / sum_k s_ik
//   dlogit = ds s (1 - s).
//
// Both passes read the scores once from HBM.  131,072 x 256 with K = 6: the
// forward takes 32.7 us (4.1 TB/s), bound by its vector instructions (745 for 8
// rows, 81% of the busy CUs' issue slots; the K largest cost 7 of them a score),
// the sums 9.0 us, bound by waiting, the gradient 43.8 us (6.1 TB/s), bound by
// HBM.  The K largest are
// kept as biased scores whose low bits are the expert's number: a list's entry
// is then one register, insertion one median, and no second look for the
// chosen ones is needed (with a mask of them: 41 us); rows where the K-th and
// the next share the upper bits are settled by the whole values.
//
// A row is held by LPR lanes in registers (V = E / LPR scores a lane), so
// column sums of p stay in a lane's registers from row to row and only the
// end of a sequence's stretch of rows reduces them across lanes.  A workgroup
// takes a chunk of T consecutive rows and leaves one partial row (E counts,
// E sums) for every sequence that meets its chunk, at slot chunk + sequence
// (both only grow along the rows, so no two stretches share a slot), summed
// over at most 128 rows in 32 bits, a quarter or an eighth of them to a lane.  A
// second kernel adds each sequence's slots in order in 64 bits: the same
// result on every run, no atomics on floating-point numbers.
#include <algorithm>

#include "qb_device.hpp"
#include "qb_internal.hpp"

namespace qbk {

typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kBalThreads = 256;
constexpr int kBalWaves = kBalThreads / kWave;

template <int E>
struct BalShape {
  static constexpr int LPR = E >= 256 ? 8 : 4;   // lanes per row
  static constexpr int V = E / LPR;              // scores per lane and row
  static constexpr int F4 = V / 4;
  static constexpr int RPW = kWave / LPR;        // rows per wave and step
  static constexpr int R = RPW * kBalWaves;      // rows per workgroup and step
  static_assert(V >= 4 && V <= 32, "scores per lane");
};

template <int LPR>
__device__ __forceinline__ float bal_row_sum(float x) {
  x += quad_mov<kQuadXor1>(x);
  x += quad_mov<kQuadXor2>(x);
  if constexpr (LPR >= 8) x += quad_mov<kHalfMirror>(x);
  return x;
}
template <int LPR>
__device__ __forceinline__ int bal_row_sum_i(int x) {
  x += quad_mov_i<kQuadXor1>(x);
  x += quad_mov_i<kQuadXor2>(x);
  if constexpr (LPR >= 8) x += quad_mov_i<kHalfMirror>(x);
  return x;
}

// Lane l ^ D's value, D 16 or 32 (the instruction exchanges the D-lane halves
// of two registers, so one of the two results is the own value and the other
// is the partner's).
template <int D>
__device__ __forceinline__ float bal_swapped(float x) {
  unsigned a = __builtin_bit_cast(unsigned, x), b = a;
  asm volatile("" : "+v"(b));  // two registers: with one and the same operand the compiler takes the results as equal
  const auto h = D == 16 ? __builtin_amdgcn_permlane16_swap(a, b, false, false)
                         : __builtin_amdgcn_permlane32_swap(a, b, false, false);
  return __builtin_bit_cast(float, threadIdx.x & D ? h[0] : h[1]);
}

// The sum over the lanes that hold the same columns (l, l + LPR, ...), in all
// of them: within 16 lanes by rotation, then by exchanging halves.
template <int LPR>
__device__ __forceinline__ float bal_col_sum(float x) {
  if constexpr (LPR <= 4) x += quad_mov<0x124>(x);  // row_ror:4
  x += quad_mov<0x128>(x);                          // row_ror:8
  x += bal_swapped<16>(x);
  return x + bal_swapped<32>(x);
}

// The larger and the smaller of two packed scores.  As medians with the type's
// ends: fmaxf would first quiet each operand, which comes from an integer and
// might be a signalling NaN for all the compiler knows (90 of the 810
// instructions of a wave's step).
constexpr float kBalMost = 3.4028234663852886e38f;
__device__ __forceinline__ float bal_max(float a, float b) { return __builtin_amdgcn_fmed3f(a, b, kBalMost); }
__device__ __forceinline__ float bal_min(float a, float b) { return __builtin_amdgcn_fmed3f(a, b, -kBalMost); }

// v into a descending list (its least entry leaves).
template <int P>
__device__ __forceinline__ void bal_insert(float (&t)[P], float v) {
#pragma unroll
  for (int k = P - 1; k > 0; --k) t[k] = __builtin_amdgcn_fmed3f(v, t[k - 1], t[k]);
  t[0] = bal_max(v, t[0]);
}

// One stage at distance D of a bitonic merge of the last P of W entries, the
// others counting as infinite.
template <int P, int W, int D>
__device__ __forceinline__ void bal_stage(float (&c)[P]) {
  if constexpr (D >= 1) {
#pragma unroll
    for (int i = W - P; i < W; ++i)
      if ((i & D) == 0) {
        float &a = c[i - (W - P)], &b = c[i + D - (W - P)];
        const float hi = bal_max(a, b);
        b = bal_min(a, b);
        a = hi;
      }
    bal_stage<P, W, D / 2>(c);
  }
}

// This lane's list and the partner's into the P largest of both: the larger
// of entry k here and entry P - 1 - k there are those, first falling, then
// rising.
template <int P, int CTRL>
__device__ __forceinline__ void bal_merge(float (&t)[P]) {
  constexpr int W = P <= 4 ? 4 : (P <= 8 ? 8 : 16);
  float c[P];
#pragma unroll
  for (int k = 0; k < P; ++k) c[k] = bal_max(t[k], quad_mov<CTRL>(t[P - 1 - k]));
  bal_stage<P, W, W / 2>(c);
#pragma unroll
  for (int k = 0; k < P; ++k) t[k] = c[k];
}

// What a row is multiplied by before it is divided by this sum of its scores:
// a sum below 2^-100 (all of them far down the sigmoid) may have no inverse in
// 32 bits.  1 - s is 1 in such a row.
__device__ __forceinline__ float bal_up(float sum) { return sum < 0x1p-100f ? 0x1p100f : 1.0f; }

// The sequence that row r belongs to: the number of ends off[1..B] at or
// below r (B: past the last sequence).  off need not be sorted for this to
// stay within [0, B].
__device__ __forceinline__ int bal_find(const int32_t* off, int B, int r) {
  int lo = 0, hi = B;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (off[mid + 1] <= r)
      lo = mid + 1;
    else
      hi = mid;
  }
  return lo;
}

// The same for one row of the whole wave: 64 ends a trip, so that B <= 64
// sequences take one load's latency (a binary search of 41 took six: 4 us of
// the 14 that a batch of 5003 tokens spent here).
__device__ __forceinline__ int bal_find_wave(const int32_t* off, int B, int r, int lane) {
  int lo = 0, hi = B;
  while (lo < hi) {
    const int step = (hi - lo + kWave - 1) / kWave;
    const int j = lo + (lane + 1) * step - 1;
    const int below = __popcll(__ballot(j < hi && off[j + 1] <= r));
    lo += below * step;
    hi = hi < lo + step - 1 ? hi : lo + step - 1;
  }
  return lo;
}

// Rows per chunk: short chunks keep all CUs busy on few tokens, longer ones
// keep the partial rows small beside the scores (128 rows of 256 experts:
// 2 KiB of partials for 128 KiB of scores).
int balance_chunk_rows(int64_t N) { return N <= 32768 ? 32 : 128; }

// Threads of the second kernel: 16 for each of up to 64 experts.
constexpr int kBalFinWays = 16;
constexpr int kBalFinCols = 64;
// Its workgroups at most, one a CU: each counts the sequences and arrives at
// one word (8192 sequences of 16 tokens, 256 experts: the forward takes 344
// us, 354 with 512, 372 with 1024, 953 with one for each 64 experts of a
// sequence; 131,072 of one token 5.1 and 105 ms).
constexpr int kBalFinMost = 256;
static int bal_fin_cols(int E) { return E < kBalFinCols ? E : kBalFinCols; }

BalWs balance_ws_layout(int64_t N, int E, int B) {
  BalWs w;
  w.T = balance_chunk_rows(N);
  w.chunks = (N + w.T - 1) / w.T;
  w.slots = w.chunks + B;
  w.groups = std::min<int64_t>(int64_t(B) * (E / bal_fin_cols(E)), kBalFinMost);
  w.part = 16;  // the arrival counter comes first
  w.psum = w.part + (w.groups * 8 + 15) / 16 * 16;
  w.cnt = w.psum + w.slots * E * 4;
  w.live = w.cnt + w.slots * E * 4;
  w.bytes = w.live + (w.slots * 4 + 15) / 16 * 16;
  return w;
}

// Entries m .. K - 1 of a row's list, where the K-th and the next share their
// upper bits (`edge`): the largest whole values among those that do, equal
// ones by lower expert.  It reads the row from LDS again rather than hold
// registers in every row's way; a row needs it once in some 300 (scores as of
// a router of 256 experts), and then mostly for one entry.
template <int E>
__device__ __forceinline__ void bal_edge(const float* src, const float* lds_b, int ql, int m, int K, uint32_t edge,
                                         uint2* stage) {
  using S = BalShape<E>;
  constexpr int LPR = S::LPR;
  constexpr int STEP = S::F4 < 4 ? S::F4 : 4;
  uint32_t rem = ~0u;
  for (int k = m; k < K; ++k) {
    float best = 0.f;
    int at = E;
#pragma unroll 1
    for (int t0 = 0; t0 < S::F4; t0 += STEP) {
      f32x4 v[STEP];
#pragma unroll
      for (int t = 0; t < STEP; ++t) v[t] = *reinterpret_cast<const f32x4*>(src + 4 * (LPR * (t0 + t) + ql));
#pragma unroll
      for (int t = 0; t < STEP; ++t) {
        const f32x4 bb = *reinterpret_cast<const f32x4*>(lds_b + 4 * (LPR * (t0 + t) + ql));
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float w = v[t][c] + bb[c];
          const bool take = (__builtin_bit_cast(uint32_t, w) ^ edge) < uint32_t(E) &&
                            ((rem >> (4 * (t0 + t) + c)) & 1u) && (at == E || w > best);
          best = take ? w : best;
          at = take ? 4 * (LPR * (t0 + t) + ql) + c : at;
        }
      }
    }
    auto join = [&](float ov, int oa) {
      const bool take = oa < E && (at == E || ov > best || (ov == best && oa < at));
      best = take ? ov : best;
      at = take ? oa : at;
    };
    join(quad_mov<kQuadXor1>(best), quad_mov_i<kQuadXor1>(at));
    join(quad_mov<kQuadXor2>(best), quad_mov_i<kQuadXor2>(at));
    if constexpr (LPR >= 8) join(quad_mov<kHalfMirror>(best), quad_mov_i<kHalfMirror>(at));
    if (at < E && (at >> 2) % LPR == ql) {
      rem &= ~(1u << (4 * ((at >> 2) / LPR) + (at & 3)));
      stage[k] = make_uint2(__builtin_bit_cast(uint32_t, best), uint32_t(at));
    }
  }
}

template <int E, int P, bool STATS>
__global__ __launch_bounds__(kBalThreads, P <= 9 ? 4 : 3) void k_balance_fwd(
    const float* __restrict__ s, const float* __restrict__ b, int N, int K, const int32_t* __restrict__ seq_off, int B,
    const uint8_t* __restrict__ valid, int T, int32_t* __restrict__ topk, float* __restrict__ gate,
    float* __restrict__ psum, int32_t* __restrict__ cnt, int32_t* __restrict__ live, uint32_t* __restrict__ arrivals) {
  using S = BalShape<E>;
  constexpr int LPR = S::LPR, F4 = S::F4, RPW = S::RPW, R = S::R, KU = (P - 1 + LPR - 1) / LPR;
  __shared__ __align__(16) float lds_b[E];
  __shared__ uint2 stage[kBalWaves][RPW][P - 1];  // a row's chosen biased scores and experts
  // the step's rows: a chosen score is read from here by its expert's number (from memory it is a trip to L2 more)
  __shared__ __align__(16) float lds_x[kBalWaves][RPW][E];
  __shared__ int lds_cnt[STATS ? E : 1];
  __shared__ __align__(16) float lds_p[kBalWaves][STATS ? E : 4];
  int* const lds_live = reinterpret_cast<int*>(&lds_p[0][0]);  // the two are never in use together

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int rho = lane / LPR, ql = lane % LPR;
  const int r0 = int(blockIdx.x) * T;
  const int r1 = N - r0 < T ? N : r0 + T;
  for (int j = tid; j < E; j += kBalThreads) {
    lds_b[j] = fminf(fmaxf(b[j], -kBalMost), kBalMost);  // an infinite sum, with an expert in its low bits, is no number
    if constexpr (STATS) lds_cnt[j] = 0;
  }
  if constexpr (STATS)
    if (blockIdx.x == 0 && tid == 0) *arrivals = 0;
  __syncthreads();

  // The sequence whose rows come next.  A chunk's rows are taken step by step
  // whatever sequences they belong to, so that short sequences share a step's
  // reading and sorting; q's sums are written once its end is passed.
  const int first = seq_off ? seq_off[0] : 0, last = seq_off ? seq_off[B] : N;
  struct Run {
    int q, begin, end;  // begin: its first row in this chunk
  };
  auto end_of = [&](int i) { return seq_off && i < B ? seq_off[i + 1] : N; };
  const int q0 = seq_off ? bal_find_wave(seq_off, B, r0, lane) : 0;
  Run now{q0, r0, end_of(q0)};
  f32x4 acc[STATS ? F4 : 1];
  int n_live = 0;
  if constexpr (STATS)
#pragma unroll
    for (int t = 0; t < F4; ++t) acc[t] = (f32x4){0.f, 0.f, 0.f, 0.f};
  // this chunk's sum of p of sequence i: the lanes of one wave that hold the same columns, then the waves
  auto write_p = [&](int i) {
#pragma unroll
    for (int t = 0; t < F4; ++t) {
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[t][c] = bal_col_sum<LPR>(acc[t][c]);
      if (rho == 0) *reinterpret_cast<f32x4*>(&lds_p[wave][4 * (LPR * t + ql)]) = acc[t];
      acc[t] = (f32x4){0.f, 0.f, 0.f, 0.f};
    }
    __syncthreads();
    const int64_t slot = int64_t(blockIdx.x) + i;
    for (int j = tid; j < E; j += kBalThreads)
      psum[slot * E + j] = (lds_p[0][j] + lds_p[1][j]) + (lds_p[2][j] + lds_p[3][j]);
    __syncthreads();
  };
  auto write_count = [&](int i) {
    if (lane == 0) lds_live[wave] = n_live;
    n_live = 0;
    __syncthreads();
    const int64_t slot = int64_t(blockIdx.x) + i;
    for (int j = tid; j < E; j += kBalThreads) {
      cnt[slot * E + j] = lds_cnt[j];
      lds_cnt[j] = 0;
    }
    if (tid == 0) live[slot] = (lds_live[0] + lds_live[1]) + (lds_live[2] + lds_live[3]);
    __syncthreads();
  };
  for (int rb = r0; rb < r1; rb += R) {
    const int step_end = rb + R < r1 ? rb + R : r1;
    const bool busy = rb + wave * RPW < step_end;
    const int row = rb + wave * RPW + rho;
    const bool here = row < step_end;
    const int64_t ld_row = here ? row : r1 - 1;
    const float* src = s + ld_row * E;
    const bool lv = here && row >= first && row < last && (!valid || valid[ld_row] != 0);
    const bool whole = now.end >= step_end;  // the step's rows are all of one sequence
    Run now_p = now;
    float* xrow = lds_x[wave][rho];
    float top[P], inv = 0.f, up = 1.0f;
    if (busy) {
      f32x4 x[F4];
#pragma unroll
      for (int t = 0; t < F4; ++t) x[t] = *reinterpret_cast<const f32x4*>(src + 4 * (LPR * t + ql));
#pragma unroll
      for (int t = 0; t < F4; ++t) *reinterpret_cast<f32x4*>(xrow + 4 * (LPR * t + ql)) = x[t];
      // the P largest biased scores, each with its expert in the low bits
#pragma unroll
      for (int k = 0; k < P; ++k) top[k] = __builtin_bit_cast(float, 0xFF7FFFFFu & ~uint32_t(E - 1));
      float z = 0.f;
#pragma unroll
      for (int t = 0; t < F4; ++t) {
        const float4 bb = *reinterpret_cast<const float4*>(lds_b + 4 * (LPR * t + ql));
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint32_t v = __builtin_bit_cast(uint32_t, x[t][c] + comp(bb, c));
          bal_insert<P>(top, __builtin_bit_cast(float, (v & ~uint32_t(E - 1)) | uint32_t(4 * t + c)));
        }
        if constexpr (STATS) z += (x[t].x + x[t].y) + (x[t].z + x[t].w);
      }
#pragma unroll
      for (int k = 0; k < P; ++k)
        top[k] = __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, top[k]) | uint32_t(ql * S::V));
      bal_merge<P, kQuadXor1>(top);
      bal_merge<P, kQuadXor2>(top);
      if constexpr (LPR >= 8) bal_merge<P, kHalfMirror>(top);
      if constexpr (STATS) {
        z = bal_row_sum<LPR>(z);
        up = bal_up(z);
        inv = z > 0.f ? 1.0f / (z * up) : 0.f;
        if (up != 1.0f)
#pragma unroll
          for (int t = 0; t < F4; ++t) x[t] *= up;
        if (whole && lv)  // a dead row's scores may be anything
#pragma unroll
          for (int t = 0; t < F4; ++t)
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[t][c] = fmaf(x[t][c], inv, acc[t][c]);
      }
    }
    // The step's rows to their sequences: `add` takes those of i, `write` what
    // the chunk held of i, once its end or the chunk's is passed.
    auto deal = [&](auto&& add, auto&& write, Run& g) {
      for (int from = rb;;) {
        add(row >= from && row < g.end);
        if (g.end >= step_end && step_end < r1) break;
        if (g.q < B && (g.end < r1 ? g.end : r1) > g.begin) write(g.q);
        if (g.end >= step_end) break;
        from = g.end > from ? g.end : from;
        g = {g.q + 1, from, end_of(g.q + 1)};
      }
    };
    if constexpr (STATS)
      deal(
          [&](bool mine) {
            if (!whole && busy && mine && lv)  // the rows are read again: kept, they would cost the sorting its registers
#pragma unroll
              for (int t = 0; t < F4; ++t) {
                const f32x4 x = *reinterpret_cast<const f32x4*>(xrow + 4 * (LPR * t + ql));
#pragma unroll
                for (int c = 0; c < 4; ++c) acc[t][c] = fmaf(x[c] * up, inv, acc[t][c]);
              }
          },
          write_p, now_p);
    int id[KU];
    if (busy) {
      // the set of the K is certain unless the next one differs in the bits below only
      uint32_t edge = 0;
      bool tie = false;
#pragma unroll
      for (int k = 1; k < P; ++k) {
        const uint32_t above = __builtin_bit_cast(uint32_t, top[k - 1]);
        edge = k == K ? above : edge;
        tie = k == K ? (__builtin_bit_cast(uint32_t, top[k]) ^ above) < uint32_t(E) : tie;
      }
      // lane ql holds the list's entries ql, ql + LPR, ...
      uint2* mine = stage[wave][rho];
      float sv[KU], v[KU], total = 0.f;
      int rank[KU];
#pragma unroll
      for (int u = 0; u < KU; ++u) {
        uint32_t m = __builtin_bit_cast(uint32_t, top[u * LPR < P ? u * LPR : 0]);
#pragma unroll
        for (int j = 1; j < LPR; ++j)
          if (u * LPR + j < P) m = ql == j ? __builtin_bit_cast(uint32_t, top[u * LPR + j]) : m;
        const int k = ql + u * LPR, n = int(m & uint32_t(S::V - 1)), from = int(m & uint32_t(E - 1)) / S::V;
        id[u] = 4 * (LPR * (n >> 2) + from) + (n & 3);
        sv[u] = xrow[id[u]];
        v[u] = sv[u] + lds_b[id[u]];
        if (k < K) mine[k] = make_uint2(__builtin_bit_cast(uint32_t, v[u]), uint32_t(id[u]));
      }
      if (__ballot(tie) != 0) {
        if (tie) {
          int m = 0;
#pragma unroll
          for (int k = 0; k < P - 1; ++k) m += k < K && (__builtin_bit_cast(uint32_t, top[k]) ^ edge) >= uint32_t(E) ? 1 : 0;
          bal_edge<E>(xrow, lds_b, ql, m, K, edge, mine);
        }
        __builtin_amdgcn_wave_barrier();
        asm volatile("" ::: "memory");
#pragma unroll
        for (int u = 0; u < KU; ++u) {
          const int k = ql + u * LPR;
          id[u] = k < K ? int(mine[k].y & uint32_t(E - 1)) : 0;
          sv[u] = xrow[id[u]];
          v[u] = sv[u] + lds_b[id[u]];
        }
      }
      __builtin_amdgcn_wave_barrier();
      asm volatile("" ::: "memory");
      // their order is that of the whole values, equal ones by their expert
#pragma unroll
      for (int u = 0; u < KU; ++u) {
        rank[u] = 0;
        sv[u] = ql + u * LPR < K ? sv[u] : 0.f;
        total += sv[u];
      }
#pragma unroll
      for (int j = 0; j < P - 1; ++j) {
        if (j < K) {
          const uint2 o = mine[j];
          const float ov = __builtin_bit_cast(float, o.x);
#pragma unroll
          for (int u = 0; u < KU; ++u) rank[u] += ov > v[u] || (ov == v[u] && int(o.y) < id[u]) ? 1 : 0;
        }
      }
      total = bal_row_sum<LPR>(total);
      const float c = bal_up(total), per = total > 0.f ? 1.0f / (total * c) : 0.f;
#pragma unroll
      for (int u = 0; u < KU; ++u) {
        if (here && ql + u * LPR < K) {
          const int64_t o = int64_t(row) * K + (lv ? rank[u] : ql + u * LPR);  // a dead row may hold NaN
          topk[o] = lv ? id[u] : -1;
          if (gate) gate[o] = lv ? sv[u] * c * per : 0.f;
        }
      }
      asm volatile("" ::: "memory");
      __builtin_amdgcn_wave_barrier();
    }
    if constexpr (STATS) {
      deal(
          [&](bool mine) {
            const bool on = mine && lv;
            n_live += __popcll(__ballot(on)) / LPR;
            if (busy && on)
#pragma unroll
              for (int u = 0; u < KU; ++u)
                if (ql + u * LPR < K) atomicAdd(&lds_cnt[id[u]], 1);
          },
          write_count, now);
    }
  }
}

// ---------------------------------------------------------------------------
// The sums of each sequence's slots, its weights and its share of the loss:
// one workgroup for up to 64 experts of one sequence at a time, 16 threads an
// expert.
// Every workgroup counts the sequences that have a live token itself (a scan
// of a few live words); the last one to arrive adds the shares of the loss in
// a fixed order.  All of it is waiting (each load is of memory that another
// XCD wrote, and arrivals at one word pass one by one), so the loads of a
// stage are issued together and the workgroups are few: 32 sequences of
// 131,072 x 256 take 12 us with 512 workgroups of 16 experts.
__device__ __forceinline__ void bal_slots(const int32_t* seq_off, int N, int T, int q, int64_t& s0, int64_t& s1) {
  int lo = 0, hi = N;
  if (seq_off) {
    lo = seq_off[q];
    lo = lo < 0 ? 0 : (lo > N ? N : lo);
    hi = seq_off[q + 1];
    hi = hi < lo ? lo : (hi > N ? N : hi);
  }
  s0 = int64_t(lo / T) + q;
  s1 = hi > lo ? int64_t((hi - 1) / T) + q + 1 : s0;
}

__global__ __launch_bounds__(kBalFinWays* kBalFinCols) void k_balance_fin(
    const int32_t* __restrict__ seq_off, int B, int N, int E, int K, int T, float coef, const float* __restrict__ psum,
    const int32_t* __restrict__ cnt, const int32_t* __restrict__ live, double* __restrict__ part,
    uint32_t* __restrict__ arrivals, int32_t* __restrict__ count, float* __restrict__ weight,
    float* __restrict__ loss) {
  __shared__ double sh_p[kBalFinWays * kBalFinCols];
  __shared__ int sh_c[kBalFinWays * kBalFinCols];
  __shared__ int sh_filled, sh_tok;
  __shared__ bool sh_last;
  const int threads = int(blockDim.x), cols = threads / kBalFinWays;
  const int tid = threadIdx.x, col = tid % cols, way = tid / cols;
  const int eg = E / cols;
  if (tid == 0) {
    sh_filled = 0;
    sh_tok = 0;
  }
  int64_t a0 = 0, a1 = 0;
  if (tid < B) bal_slots(seq_off, N, T, tid, a0, a1);
  double share = 0.0;
  for (int g = int(blockIdx.x);;) {
    const int q = g / eg, e = (g % eg) * cols + col;
    int64_t s0, s1;
    bal_slots(seq_off, N, T, q, s0, s1);
    // eight slots a thread, the sequence's live words and another's first one are on their way at once
    const bool first = g == int(blockIdx.x);
    bool any = first && a0 < a1 && live[a0] != 0;
    double p = 0.0;
    int c = 0, tok = 0;
    for (int64_t t = s0; t < s1; t += 8 * kBalFinWays) {
      float pv[8];
      int cv[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int64_t at = t + u * kBalFinWays + way, from = at < s1 ? at : s1 - 1;
        pv[u] = psum[from * E + e];
        cv[u] = cnt[from * E + e];
      }
      const int64_t mine = t + tid;
      if (tid < 8 * kBalFinWays && mine < s1) tok += live[mine];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const bool on = t + u * kBalFinWays + way < s1;
        p += on ? double(pv[u]) : 0.0;
        c += on ? cv[u] : 0;
      }
    }
    sh_p[tid] = p;
    sh_c[tid] = c;
    __syncthreads();
    if (tok) atomicAdd(&sh_tok, tok);
    if (first) {
      int filled = 0;
      for (int j = tid; j < B;) {
        for (++a0; a0 < a1 && !any; ++a0) any = live[a0] != 0;
        filled += any ? 1 : 0;
        j += threads;
        if (j < B) {
          bal_slots(seq_off, N, T, j, a0, a1);
          any = a0 < a1 && live[a0] != 0;
        }
      }
      if (filled) atomicAdd(&sh_filled, filled);
    }
    __syncthreads();
    if (tid < cols) {
#pragma unroll
      for (int w = 1; w < kBalFinWays; ++w) {
        p += sh_p[w * cols + col];
        c += sh_c[w * cols + col];
      }
      const double toks = double(sh_tok);
      const double per = sh_tok > 0 ? 1.0 / toks : 0.0;
      const double scale = double(coef) / double(sh_filled > 0 ? sh_filled : 1);
      const double f = double(c) * per * (double(E) / double(K));
      if (count) count[int64_t(q) * E + e] = c;
      if (weight) weight[int64_t(q) * E + e] = float(scale * (f - 1.0) * per);
      share += scale * f * p * per;
    }
    g += int(gridDim.x);
    if (g >= B * eg) break;
    __syncthreads();
    if (tid == 0) sh_tok = 0;
  }
  if (!loss) return;
  if (tid < kWave) {
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) share += __shfl_xor(share, d);
    if (tid == 0) {
      // The share and the counter are the only words that cross workgroups,
      // and both are atomics of the whole GPU, which no cache holds back;
      // that the share is there before the count is this wait.  (A release
      // would write back the XCD's whole L2.)
      __hip_atomic_store(reinterpret_cast<unsigned long long*>(part + blockIdx.x),
                         __builtin_bit_cast(unsigned long long, share), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      sh_last = __hip_atomic_fetch_add(arrivals, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == gridDim.x - 1;
    }
  }
  __syncthreads();
  if (!sh_last) return;
  double sum = 0.0;
  for (int i = tid; i < int(gridDim.x); i += threads)
    sum += __builtin_bit_cast(double, __hip_atomic_load(reinterpret_cast<unsigned long long*>(part + i),
                                                        __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) sum += __shfl_xor(sum, d);
  if ((tid & 63) == 0) sh_p[tid >> 6] = sum;
  __syncthreads();
  if (tid == 0) {
    double all = 0.0;
    for (int w = 0; w < threads / kWave; ++w) all += sh_p[w];
    *loss = float(all);
  }
}

// ---------------------------------------------------------------------------
// Backward: one read of the scores, one write of the gradient.  The K gate
// terms of a row go through a small LDS table (E floats a row, zero between
// rows) that the row's lanes read in their own layout.
template <int E, bool NT>
__global__ __launch_bounds__(kBalThreads) void k_balance_bwd(
    const float* __restrict__ s, const int32_t* __restrict__ topk, int N, int K, const int32_t* __restrict__ seq_off,
    int B, const uint8_t* __restrict__ valid, const float* __restrict__ weight, const float* __restrict__ dloss,
    const float* __restrict__ dgate, float* __restrict__ dlogits) {
  using S = BalShape<E>;
  constexpr int LPR = S::LPR, F4 = S::F4, RPW = S::RPW, R = S::R, KU = 16 / LPR;
  __shared__ __align__(16) float add[kBalWaves][RPW][E];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int rho = lane / LPR, ql = lane % LPR;
  float* mine = add[wave][rho];
#pragma unroll
  for (int t = 0; t < F4; ++t)
    *reinterpret_cast<float4*>(mine + 4 * (LPR * t + ql)) = make_float4(0.f, 0.f, 0.f, 0.f);
  const float dl = weight ? (dloss ? *dloss : 1.0f) : 0.f;
  for (int64_t rb = int64_t(blockIdx.x) * R; rb < N; rb += int64_t(gridDim.x) * R) {
    if (rb + wave * RPW >= N) break;
    const int64_t row = rb + wave * RPW + rho;
    const bool here = row < N;
    const int64_t lr = here ? row : N - 1;
    const float* src = s + lr * E;
    f32x4 x[F4];
#pragma unroll
    for (int t = 0; t < F4; ++t) x[t] = *reinterpret_cast<const f32x4*>(src + 4 * (LPR * t + ql));
    bool lv = !valid || valid[lr] != 0;
    int q = 0;
    if (seq_off) {
      // nearly always one sequence holds all of the wave's rows
      const int64_t w0 = rb + wave * RPW, w1 = (w0 + RPW < N ? w0 + RPW : int64_t(N)) - 1;
      q = bal_find_wave(seq_off, B, int(w0), lane);
      if (q < B && seq_off[q + 1] <= w1) q = bal_find(seq_off, B, int(lr));
      lv = lv && q < B && lr >= seq_off[0];
      q = q < B ? q : B - 1;
    }
    int id[KU];
    if (dgate) {
      float sv[KU], dg[KU], total = 0.f, inner = 0.f;
#pragma unroll
      for (int u = 0; u < KU; ++u) {
        const int k = ql + u * LPR;
        id[u] = k < K ? topk[lr * K + k] : -1;
        const bool on = lv && unsigned(id[u]) < unsigned(E);
        id[u] = on ? id[u] : -1;
        sv[u] = on ? src[id[u]] : 0.f;
        dg[u] = on ? dgate[lr * K + k] : 0.f;
        total += sv[u];
      }
      total = bal_row_sum<LPR>(total);
      const float c = bal_up(total), per = total > 0.f ? 1.0f / (total * c) : 0.f;
#pragma unroll
      for (int u = 0; u < KU; ++u) {
        sv[u] *= c * per;  // the gate
        inner = fmaf(dg[u], sv[u], inner);
      }
      inner = bal_row_sum<LPR>(inner);
#pragma unroll
      for (int u = 0; u < KU; ++u)
        if (id[u] >= 0) mine[id[u]] = (dg[u] - inner) * sv[u];
    }
    __builtin_amdgcn_wave_barrier();
    asm volatile("" ::: "memory");
    float z = 0.f, dot = 0.f;
    f32x4 w[F4];
    if (weight) {
      const float* wr = weight + int64_t(q) * E;
#pragma unroll
      for (int t = 0; t < F4; ++t) {
        w[t] = *reinterpret_cast<const f32x4*>(wr + 4 * (LPR * t + ql));
        z += (x[t].x + x[t].y) + (x[t].z + x[t].w);
        dot = fmaf(w[t].x, x[t].x, dot);
        dot = fmaf(w[t].y, x[t].y, dot);
        dot = fmaf(w[t].z, x[t].z, dot);
        dot = fmaf(w[t].w, x[t].w, dot);
      }
      z = bal_row_sum<LPR>(z);
      dot = bal_row_sum<LPR>(dot);
    } else {
#pragma unroll
      for (int t = 0; t < F4; ++t) w[t] = (f32x4){0.f, 0.f, 0.f, 0.f};
    }
    const float up = weight ? bal_up(z) : 1.0f;
    if (up != 1.0f) {
      dot = 0.f;
#pragma unroll
      for (int t = 0; t < F4; ++t)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          x[t][c] *= up;
          dot = fmaf(w[t][c], x[t][c], dot);
        }
      dot = bal_row_sum<LPR>(dot);
    }
    const float inv = lv && z > 0.f ? 1.0f / (z * up) : 0.f;
    const float mean = dot * inv, scale = dl * inv;
#pragma unroll
    for (int t = 0; t < F4; ++t) {
      f32x4 g = (f32x4){0.f, 0.f, 0.f, 0.f}, o;
      if (dgate) g = *reinterpret_cast<const f32x4*>(mine + 4 * (LPR * t + ql));
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float rest = up != 1.0f ? 1.0f : 1.0f - x[t][c];
        o[c] = fmaf((w[t][c] - mean) * scale, x[t][c] * rest, g[c] * rest);
      }
      if (!lv) o = (f32x4){0.f, 0.f, 0.f, 0.f};
      f32x4* dst = reinterpret_cast<f32x4*>(dlogits + row * E + 4 * (LPR * t + ql));
      if (here) {
        if constexpr (NT)
          __builtin_nontemporal_store(o, dst);
        else
          *dst = o;
      }
    }
    asm volatile("" ::: "memory");
    __builtin_amdgcn_wave_barrier();
    if (dgate) {
#pragma unroll
      for (int u = 0; u < KU; ++u)
        if (id[u] >= 0) mine[id[u]] = 0.f;
    }
  }
}

// ---------------------------------------------------------------------------

template <int E, int P>
static int fwd_ep(const BalFwd& a, const BalWs& w, hipStream_t st) {
  const dim3 grid{unsigned(w.chunks), 1u, 1u}, block{unsigned(kBalThreads), 1u, 1u};
  uint8_t* ws = a.ws;
  if (ws)
    hipLaunchKernelGGL((k_balance_fwd<E, P, true>), grid, block, 0, st, a.s, a.b, int(a.N), a.K, a.seq_off, a.B,
                       a.valid, w.T, a.topk, a.gate, reinterpret_cast<float*>(ws + w.psum),
                       reinterpret_cast<int32_t*>(ws + w.cnt), reinterpret_cast<int32_t*>(ws + w.live),
                       reinterpret_cast<uint32_t*>(ws));
  else
    hipLaunchKernelGGL((k_balance_fwd<E, P, false>), grid, block, 0, st, a.s, a.b, int(a.N), a.K, a.seq_off, a.B,
                       a.valid, w.T, a.topk, a.gate, nullptr, nullptr, nullptr, nullptr);
  return int(hipGetLastError());
}

template <int E>
static int fwd_e(const BalFwd& a, const BalWs& w, hipStream_t st) {
  // lists of the next of 4, 7, 9 and 16 entries above K
  if (a.K <= 3) return fwd_ep<E, 4>(a, w, st);
  if (a.K <= 6) return fwd_ep<E, 7>(a, w, st);
  if (a.K <= 8) return fwd_ep<E, 9>(a, w, st);
  return fwd_ep<E, 16>(a, w, st);
}

int launch_balance_fwd(const BalFwd& a, hipStream_t st) {
  const BalWs w = balance_ws_layout(a.N, a.E, a.B);
  int rc = int(hipErrorInvalidValue);
  switch (a.E) {
    case 16: rc = fwd_e<16>(a, w, st); break;
    case 32: rc = fwd_e<32>(a, w, st); break;
    case 64: rc = fwd_e<64>(a, w, st); break;
    case 128: rc = fwd_e<128>(a, w, st); break;
    case 256: rc = fwd_e<256>(a, w, st); break;
  }
  if (rc != int(hipSuccess) || !a.ws) return rc;
  uint8_t* ws = a.ws;
  hipLaunchKernelGGL(k_balance_fin, dim3(unsigned(w.groups)), dim3(kBalFinWays * bal_fin_cols(a.E)), 0,
                     st, a.seq_off, a.B, int(a.N),
                     a.E, a.K, w.T, a.coef, reinterpret_cast<const float*>(ws + w.psum),
                     reinterpret_cast<const int32_t*>(ws + w.cnt), reinterpret_cast<const int32_t*>(ws + w.live),
                     reinterpret_cast<double*>(ws + w.part), reinterpret_cast<uint32_t*>(ws), a.count, a.weight,
                     a.loss);
  return int(hipGetLastError());
}

template <int E>
static int bwd_e(const BalBwd& a, hipStream_t st) {
  constexpr int R = BalShape<E>::R;
  const int64_t steps = (a.N + R - 1) / R;
  const int64_t most = int64_t(device_cu_count()) * 4;  // workgroups that run at once; more rows are further trips
  const dim3 grid{unsigned(std::min(steps, most)), 1u, 1u}, block{unsigned(kBalThreads), 1u, 1u};
  // Where scores and gradient together exceed the last cache (256 MiB), the
  // gradient passes it by and leaves it the scores that the forward has read
  // (131,072 x 256 with other scores each time: 104.8 -> 100.0 us a pass).
  if (2 * 4 * a.N * E >= (int64_t(256) << 20))
    hipLaunchKernelGGL((k_balance_bwd<E, true>), grid, block, 0, st, a.s, a.topk, int(a.N), a.K, a.seq_off, a.B,
                       a.valid, a.weight, a.dloss, a.dgate, a.dlogits);
  else
    hipLaunchKernelGGL((k_balance_bwd<E, false>), grid, block, 0, st, a.s, a.topk, int(a.N), a.K, a.seq_off, a.B,
                       a.valid, a.weight, a.dloss, a.dgate, a.dlogits);
  return int(hipGetLastError());
}

int launch_balance_bwd(const BalBwd& a, hipStream_t st) {
  switch (a.E) {
    case 16: return bwd_e<16>(a, st);
    case 32: return bwd_e<32>(a, st);
    case 64: return bwd_e<64>(a, st);
    case 128: return bwd_e<128>(a, st);
    case 256: return bwd_e<256>(a, st);
  }
  return int(hipErrorInvalidValue);
}

// ---------------------------------------------------------------------------
// The bias update of a batch with padding.  Its first pass counts every row's
// margins in a histogram, whose totals give the rank, and its second reads
// that pass's alpha.  So rows that were routed nowhere leave it in two steps:
// their scores, which may be anything, become zeros before the first pass,
// which makes their margins all one value (the (K+1)-th largest bias); that
// many counts are taken out of its bin again, and their alpha becomes infinity,
// whose key lies above every finite margin's.  Two launches that read one word
// of topk a row: an update of 131,072 x 256, a tenth of it padding, takes 80 us
// with them and 73 over all rows.

constexpr int kUnrThreads = 256;

__device__ __forceinline__ bool unrouted(const int32_t* topk, int64_t row, int64_t N, int K, int E) {
  return row < N && unsigned(topk[row * K]) >= unsigned(E);
}

__global__ __launch_bounds__(kUnrThreads) void k_unrouted_clear(const int32_t* __restrict__ topk, int64_t N, int K,
                                                                int E, float* __restrict__ s) {
  const int lane = threadIdx.x & 63;
  const int64_t r0 = int64_t(blockIdx.x) * kUnrThreads + (threadIdx.x - lane);
  uint64_t m = __ballot(unrouted(topk, r0 + lane, N, K, E));
  while (m) {
    float* row = s + (r0 + __builtin_ctzll(m)) * E;
    m &= m - 1;
    for (int c = 4 * lane; c < E; c += 4 * kWave) *reinterpret_cast<f32x4*>(row + c) = (f32x4){0.f, 0.f, 0.f, 0.f};
  }
}

__global__ __launch_bounds__(kUnrThreads) void k_unrouted_uncount(const int32_t* __restrict__ topk, int64_t N, int K,
                                                                  int E, float* __restrict__ alpha,
                                                                  int32_t* __restrict__ hist_hi) {
  __shared__ int n;
  __shared__ float a;
  const int tid = threadIdx.x;
  if (tid == 0) n = 0;
  __syncthreads();
  int mine = 0;
  for (int64_t row = int64_t(blockIdx.x) * kUnrThreads + tid; row < N; row += int64_t(gridDim.x) * kUnrThreads)
    if (unrouted(topk, row, N, K, E)) {
      a = alpha[row];  // the same value for all of them
      alpha[row] = __builtin_inff();
      ++mine;
    }
  if (mine) atomicAdd(&n, mine);
  __syncthreads();
  if (n == 0) return;
  const uint32_t key = key2(bf16x2_rne(a, a)) & 0xFFFFu;
  for (int e = tid; e < E; e += kUnrThreads) atomicSub(hist_hi + e * 256 + (key >> 8), n);
}

int launch_unrouted_clear(const int32_t* topk, int64_t N, int K, int E, float* s, hipStream_t st) {
  hipLaunchKernelGGL(k_unrouted_clear, dim3(unsigned((N + kUnrThreads - 1) / kUnrThreads)), dim3(kUnrThreads), 0, st,
                     topk, N, K, E, s);
  return int(hipGetLastError());
}

int launch_unrouted_uncount(const int32_t* topk, int64_t N, int K, int E, float* alpha, int32_t* hist_hi,
                            hipStream_t st) {
  const int64_t most = device_cu_count();  // each subtracts its rows from every expert's bin
  hipLaunchKernelGGL(k_unrouted_uncount, dim3(unsigned(std::min((N + kUnrThreads - 1) / kUnrThreads, most))),
                     dim3(kUnrThreads), 0, st, topk, N, K, E, alpha, hist_hi);
  return int(hipGetLastError());
}

}  // namespace qbk
