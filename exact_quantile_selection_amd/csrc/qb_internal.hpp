// qb_internal.hpp -- launch plumbing shared by the libqb translation units.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace qbk {

// Block-cyclic work split of a pass over rows.  A workgroup "trip" is
// `step` consecutive rows; trip t of a layer goes to workgroup t % G, so the
// workgroups in flight at any moment read neighbouring blocks (all HBM
// channels busy) instead of each streaming its own distant chunk.  G is
// chosen so that L * G is a multiple of the CU count where possible, and
// large enough that no workgroup sees more than `max_rows` rows (the packed
// 16-bit LDS counters hold < 65536 per flush).
struct RowSplit {
  int64_t trips;     // trips per layer = ceil(N / step)
  int wg_per_layer;  // G
  int64_t blocks;    // L * G
};
RowSplit split_rows(int L, int64_t N, int step, int64_t max_rows);

int device_cu_count();

// A pass over this many bytes of scores per launch (at least three times the
// MI355X's 256 MiB Infinity Cache) reads them with non-temporal loads: the
// cache cannot hand much of such a layer from one pass to the next, and the
// non-temporal stream is faster (the stream probe reads 1 GiB at 7.0 TB/s
// with them against 6.3 without).  Smaller layers keep the cached loads, so
// that the next pass finds the rows the last one read.
#ifndef QB_STREAM_BYTES
#define QB_STREAM_BYTES (768LL << 20)
#endif
inline bool stream_pass(int L, int64_t N, int E) { return int64_t(L) * N * E * 4 >= QB_STREAM_BYTES; }

// Launchers (return hipError_t as int).  Shapes were validated by the caller.
// bdiv: that many consecutive layers share one bias row (1: one row per
// layer; C: layers are the C microbatches of one layer).
// load_mb (nullable, needs load): also count each token's top-K experts
// into load_mb[l][row / n_mb][e] with device atomics.
int launch_margins_topk(const float* s, const float* b, int L, int64_t N, int E, int K,
                        float* alpha, int32_t* load, int32_t* hist_hi, hipStream_t st, int bdiv = 1,
                        int32_t* load_mb = nullptr, int64_t n_mb = 1);
int radix_wg_per_layer(int L, int64_t N, int E);

// Workspace of the low-byte pass: one partial histogram row per (layer,
// expert, workgroup), row r = (layer * E + j) * G + g.  A row whose 256
// counts are all <= 255 is stored as bytes (p8: uint8 [rows][256]); any
// other as uint16 (p16: uint16 [rows][256]); flag[r] (uint8) says which.
// Every row's flag is written on every pass, so the contents on entry do
// not matter.
struct LoWs {
  int64_t flag;   // byte offset of the flags
  int64_t p16;    // byte offset of the uint16 rows (16-byte aligned)
  int64_t bytes;  // total
};
inline LoWs lo_ws_layout(int L, int E, int G) {
  const int64_t rows = int64_t(L) * E * G;
  LoWs w;
  w.flag = rows * 256;
  w.p16 = (w.flag + rows + 15) / 16 * 16;
  w.bytes = w.p16 + rows * 512;
  return w;
}
int launch_radix_hist_lo_ws(const float* s, const float* alpha, int L, int64_t N, int E,
                            const int32_t* sel_hi, uint8_t* ws, hipStream_t st);
int launch_radix_hist_lo_ws_loads(const float* s, const float* alpha, int L, int64_t N, int E,
                                  const int32_t* sel_hi, uint8_t* ws, const float* b, int K, int32_t* load,
                                  int64_t n_mb, int32_t* load_mb, hipStream_t st);
int radix_lo_trip_rows(int E);
int launch_select_lo_ws(int L, int E, int G, const uint8_t* ws, const int32_t* sel_hi, const int32_t* rank_lo,
                        int32_t* hist_lo, uint16_t* key_out, float* q_out, float* b, float* bounds,
                        int32_t* hist_hi, int32_t* err, hipStream_t st);
int launch_lei_bwd(const float* g, const float* s, const int32_t* load_mb, int64_t N, int E, int K,
                   int64_t n_mb, float eta, int bounded, float* g_out, float* dlogits, hipStream_t st);
int launch_allreduce_sum(int32_t* buf, int R, int64_t M, hipStream_t st);
int launch_rank_average(const float* q, int R, int E, float* b, float* bounds, hipStream_t st);
int launch_maxvio(const int32_t* load, int L, int C, int E, int K, int64_t n_tok, float* v,
                  float* summary, float* worst, hipStream_t st);
int launch_radix_hist(bool lo, const float* s, const float* alpha, int L, int64_t N, int E,
                      const int32_t* sel_hi, int32_t* hist, hipStream_t st);
int launch_margin_keys(const float* s, const float* alpha, int L, int64_t N, int E, uint16_t* keys,
                       hipStream_t st);
int launch_select(int phase, int L, int E, int K, const int32_t* hist, int n_bins,
                  int32_t* sel_hi, int32_t* rank_lo, uint16_t* key_out, float* q_out, float* b,
                  float* bounds, int32_t* err, hipStream_t st);
// Workspace of the K3 binning pass: one partial row of n_bins counts per
// (layer, expert j, workgroup g of j's slice), row r = (layer * E + j) * G +
// g, G = uniform_hist_groups(...).  A row whose counts are all <= 255 is
// stored as bytes (p8: rows of b8 bytes), any other as uint16 (p16: rows of
// b16 bytes); flag[r] says which.  Every row's flag is written on every
// pass, so the contents on entry do not matter.
struct UhWs {
  int64_t rows, b8, b16;  // row count, byte stride of the byte / uint16 rows
  int64_t flag, p8, p16;  // byte offsets (256-aligned)
  int64_t bytes;          // total
};
inline UhWs uh_ws_layout(int L, int E, int64_t G, int n_bins) {
  UhWs w;
  w.rows = int64_t(L) * E * G;
  w.b8 = (int64_t(n_bins) + 15) / 16 * 16;
  w.b16 = (2 * int64_t(n_bins) + 15) / 16 * 16;
  w.flag = 0;
  w.p8 = (w.rows + 255) / 256 * 256;
  w.p16 = w.p8 + (w.rows * w.b8 + 255) / 256 * 256;
  w.bytes = w.p16 + w.rows * w.b16;
  return w;
}
int64_t uniform_hist_groups(int L, int64_t N, int E, int n_bins);
int launch_uniform_hist_ws(const float* s, const float* alpha, int L, int64_t N, int E, const float* bounds,
                           int n_bins, uint8_t* ws, hipStream_t st);
int launch_select_uniform_ws(int L, int64_t N, int E, int K, int n_bins, int64_t G, const uint8_t* ws,
                             int32_t* hist_u, float* q_out, float* b, float* bounds, int32_t* err, hipStream_t st);
int launch_uniform_hist(const float* s, const float* alpha, int L, int64_t N, int E,
                        const float* bounds, int n_bins, int32_t* hist_u, hipStream_t st);
int launch_bias_bounds(const float* b, int L, int E, float* bounds, hipStream_t st);
int launch_fill_i32(int32_t* dst, int64_t count, int32_t value, hipStream_t st);
int launch_router_gemm(const uint16_t* hidden, const uint16_t* w, int64_t N, int H, int E,
                       float* s_out, float* logits_out, hipStream_t st);
int launch_router_fused(const uint16_t* hidden, const uint16_t* w, int64_t N, int H, int E, float* s_out,
                        float* logits_out, const float* b, int K, float* alpha, int32_t* load, int32_t* hist_hi,
                        hipStream_t st);
int launch_lei(float* g, const int32_t* load, int64_t N, int E, int K, float eta,
               hipStream_t st);

bool supported_E(int E);

// Routing with a balance loss.  Workspace: an arrival counter, one float64
// share of the loss for each workgroup of the sums (`groups` of them: one for
// up to 64 experts of every sequence, 256 at most), then for each slot (chunk
// of T rows + sequence) E sums, E counts and the live tokens.
// Every word that is read was written by the same call.
struct BalWs {
  int T;                                        // rows per chunk
  int64_t chunks, slots, groups;
  int64_t part, psum, cnt, live, bytes;         // byte offsets (16-byte aligned), total
};
BalWs balance_ws_layout(int64_t N, int E, int B);
struct BalFwd {
  const float *s, *b;
  int64_t N;
  int E, K;
  const int32_t* seq_off;  // nullable: one sequence of all rows
  int B;
  const uint8_t* valid;    // nullable
  float coef;
  int32_t* topk;
  float* gate;             // nullable
  int32_t* count;          // nullable
  float *weight, *loss;    // nullable
  uint8_t* ws;             // null: experts and gates alone
};
struct BalBwd {
  const float* s;
  const int32_t* topk;
  int64_t N;
  int E, K;
  const int32_t* seq_off;
  int B;
  const uint8_t* valid;
  const float *weight, *dloss, *dgate;  // each nullable
  float* dlogits;
};
int launch_balance_fwd(const BalFwd& a, hipStream_t st);
int launch_balance_bwd(const BalBwd& a, hipStream_t st);
int launch_unrouted_clear(const int32_t* topk, int64_t N, int K, int E, float* s, hipStream_t st);
int launch_unrouted_uncount(const int32_t* topk, int64_t N, int K, int E, float* alpha, int32_t* hist_hi,
                            hipStream_t st);

// The exchange between tokens and experts.
struct Dispatch {
  const int32_t* topk;
  int64_t pairs;  // N * K
  int K, E, align;
  int32_t* off;
  int64_t R;
  int32_t *row_src, *pos, *ws;
};
int64_t dispatch_ws_bytes(int64_t pairs, int E);
int launch_dispatch(const Dispatch& a, hipStream_t st);
int launch_combine(const uint16_t* rows, int64_t R, const int32_t* pos, const float* gate, int64_t N, int K, int H,
                   uint16_t* out, hipStream_t st);
int launch_combine_bwd(const uint16_t* dout, const uint16_t* rows, int64_t R, const int32_t* pos,
                       const int32_t* row_src, const float* gate, int64_t N, int K, int H, uint16_t* drows,
                       float* dgate, hipStream_t st);

// 8-bit products with a power-of-two scale for each block of 128.
constexpr int kQBlock = 128;
inline int64_t fp8_ld(int64_t n) { return (n + kQBlock - 1) / kQBlock * kQBlock; }
inline int64_t fp8_sld(int64_t n) { return (n + 4 * kQBlock - 1) / (4 * kQBlock) * 4; }
int launch_fp8_quantize(const uint16_t* x, int64_t Mx, const int32_t* row_src, int64_t M, int C, uint8_t* xq,
                        uint8_t* xs, hipStream_t st);
int launch_fp8_quantize_cols(const uint16_t* x, int64_t Mx, const int32_t* row_src, int64_t M, int C, uint8_t* xt,
                             uint8_t* xts, hipStream_t st);
int launch_fp8_quantize_weight(const float* w, int G, int N, int C, uint8_t* wq, uint8_t* ws, uint8_t* wt,
                               uint8_t* wts, hipStream_t st);
int launch_fp8_product(const uint8_t* xq, const uint8_t* xs, const uint8_t* w, const uint8_t* ws, int64_t M, int N,
                       int64_t ldk, const int32_t* off, int G, bool exact, uint16_t* y, hipStream_t st);
int launch_fp8_weight_grad(const uint8_t* dyt, const uint8_t* dyts, const uint8_t* xt, const uint8_t* xts, int N,
                           int C, int64_t ldm, const int32_t* off, int G, float* dw, hipStream_t st);

// bf16 products.  A gradient of few tiles is split along its rows into at most
// 16 parts and 512 parts of tiles of 128 x 128 in all (32 MiB of partial sums),
// as many as leave an expert of average length 256 rows a part: offsets lie on
// the device, so a longer expert has longer parts, and a shorter one parts that
// are empty.
inline int bf16_grad_splits(int64_t M, int64_t N, int64_t C, int G) {
  const int64_t tiles = G * ((N + 127) / 128) * ((C + 127) / 128);
  int64_t s = tiles > 0 && tiles < 256 ? 512 / tiles : 1;
  s = s < 16 ? s : 16;
  const int64_t rows = M / G / 256;
  s = s < rows ? s : rows;
  return s > 1 ? int(s) : 1;
}
int launch_bf16_product(const uint16_t* x, int Mx, const int32_t* src, int M, const uint16_t* w, int N, int C,
                        const int32_t* off, int G, bool transposed, uint16_t* y, hipStream_t st);
int launch_bf16_weight_grad(const uint16_t* dy, const uint16_t* x, int Mx, const int32_t* src, int M, int N, int C,
                            const int32_t* off, int G, float* dw, float* ws, hipStream_t st);

// 4-bit products with a power-of-two scale for each block of 32: bytes of a row of n values, and of its scales.
inline int64_t fp4_ld(int64_t n) { return (n + 255) / 256 * 128; }
inline int64_t fp4_sld(int64_t n) { return (n + 255) / 256 * 8; }
int launch_fp4_quantize(const uint16_t* x, int64_t Mx, const int32_t* row_src, int64_t M, int C, uint8_t* xq,
                        uint8_t* xs, hipStream_t st);
int launch_fp4_quantize_weight(const float* w, int G, int N, int C, uint8_t* wq, uint8_t* ws, uint8_t* wt,
                               uint8_t* wts, hipStream_t st);
int launch_fp4_product(const uint8_t* xq, const uint8_t* xs, const uint8_t* w, const uint8_t* ws, int M, int N, int C,
                       const int32_t* off, int G, uint16_t* y, hipStream_t st);

// The orthogonalised update.  Workspace (byte offsets, 256-aligned): partial
// sums of squares, x twice (this step's and the next's), S = x x^T or x^T x and
// P = b S + c S S, each value in two 16-bit parts, rows rounded up to 8 values.
constexpr int kOrthoSums = 64;  // partial sums of a matrix at most
struct OrthoWs {
  bool tall;
  int64_t R, ldx, ldr;           // rows of S; values between rows of x and of S
  int64_t x0, x1, s, p, bytes;
};
inline OrthoWs ortho_ws_layout(int64_t G, int64_t N, int64_t C) {
  OrthoWs w;
  auto up = [](int64_t n, int64_t a) { return (n + a - 1) / a * a; };
  w.tall = N > C;
  w.R = w.tall ? C : N;
  w.ldx = up(C, 8);
  w.ldr = up(w.R, 8);
  const int64_t x = up(G * N * w.ldx * 4, 256), s = up(G * w.R * w.ldr * 4, 256);
  w.x0 = up(G * kOrthoSums * 8, 256);
  w.x1 = w.x0 + x;
  w.s = w.x1 + x;
  w.p = w.s + s;
  w.bytes = w.p + s;
  return w;
}
int launch_orthogonalize(const float* x, int G, int N, int C, int steps, float a, float b, float c, bool exact,
                         uint16_t* o, uint8_t* ws, hipStream_t st);

}  // namespace qbk
