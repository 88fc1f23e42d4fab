// block.cuh -- parameters of the kernels around the experts' step: norms with
// a block's gate and residual, products with an epilogue, log probabilities.
#pragma once

#include <cuda.h>

#include <cstdint>

#include "common.cuh"

namespace moe {

// ---- norms (norm.cu)
enum { kNormOutF32 = 0, kNormOutBf16 = 1, kNormOutE4m3 = 2, kNormOutNone = 3 };
struct NormP {
  int t, h;
  float eps, inv_h;  // inv_h = 1 / h
  const void *y;  // [t][h]: what is normalised, or the block's output
  int64_t ldy;
  int y_bf16;
  // the end of a block (res != nullptr)
  int post, gate_bf16, gate_sigmoid, gate_cols;  // gate_cols: 1 or h
  float scale, res_scale;
  const float *wp;   // [h] or nullptr
  const void *gate;  // or nullptr; rows ldg apart, 0: one row for all
  int64_t ldg;
  const void *res;
  int64_t ldr;
  void *ro;
  int64_t ldro;
  int res_bf16, ro_bf16;
  // the norm's output
  int out_kind;
  const float *w;  // [h] or nullptr
  void *out;
  int64_t ldo;
  uint8_t *s;  // e4m3: a scale byte per 128 of a row
  int64_t lds;
  int T;    // threads of a row
  int ld8;  // rows that start anywhere, but alike: all strides' remainder by 8
};
constexpr int kNormMaxCols = 32768;
cudaError_t launch_norm(NormP p, int n_sms, cudaStream_t st);

// ---- log probabilities (logprobs.cu)
struct LogprobsP {
  const void *x;  // [t][v]
  int64_t ld;
  int bf16, t, v;
  float scale;
  const int32_t *tokens;  // [t][m]
  int m;
  float *logp;     // [t][m]
  float *entropy;  // [t] or nullptr
  uint32_t *top_idx;  // [t][k]
  float *top_logp;
  int k;
  int S, seg;  // blocks of a row, values of a block
  int ahead, fetch;  // rows at once; bytes of the row that far ahead to bring to L2 meanwhile
};
cudaError_t launch_logprobs(LogprobsP p, int n_sms, cudaStream_t st);

// ---- products with an epilogue (mm16.cu)
enum { kActNone = 0, kActSilu = 1, kActGelu = 2, kActGeluTanh = 3, kActRelu = 4, kActSigmoid = 5 };
struct Mm16Args {
  const uint16_t *a, *b;  // bf16 [t][k]; [n][k], gated [2n][k]
  int64_t lda, ldb;
  int t, n, k, gated, act;
  const float *bias;       // [n] (gated [2n]) or nullptr
  const float *row_scale;  // [t] or nullptr
  const void *res;         // [t][n] or nullptr
  int64_t ldr;
  int res_bf16, out_bf16;
  void *out;
  int64_t ldo;
  int wide;   // four neighbouring values of out (and residual) are one access
  int wide8;  // their rows start on 32 bytes
  int withhold;
  int *status;
  unsigned long long timeout_ns;
  // tensor cores: N side of a tile, k blocks, M and N tiles, CTAs that split
  // k, ring
  int w, nk, nmt, ntt, split, stage, stages;
  int two;    // k in two halves, each with an accumulator
  int chunk;  // k blocks of one sum of the tensor cores at most
};
struct Mm16P : Mm16Args {
  CUtensorMap tm_a, tm_b, tm_r;
};
// Whether the few-row kernel takes the rows.  us a call, few-row /
// tensor-core, in a graph of calls on weights that are not in L2 (fp32 out):
//   n x k             1 row        8 rows       16 rows
//   512 x 2048        5.4 / 7.5    5.2 / 7.7    6.2 / 8.0
//   2048 x 512        2.6 / 6.9    2.8 / 7.1    3.0 / 7.4
//   2048 x 2048       5.7 / 8.9    5.7 / 9.0    6.9 / 9.2
//   2048 x 8192      11.4 / 15.1  11.4 / 15.3  13.6 / 15.5
//   4096 x 2048       6.7 / 9.0    6.9 / 9.2   11.9 / 9.4
//   8192 x 2048       9.1 / 11.2   9.3 / 11.2  16.2 / 11.3
//   131072 x 2048    83.0 / 85.0  85.0 / 86.0   155 / 88.1
// (of 16 rows one thread block an SM fits: good as long as each tile has an SM)
bool mm16_few(const Mm16Args &p, int n_sms);
cudaError_t launch_mm16_few(const Mm16Args &p, int n_sms, cudaStream_t st);
cudaError_t launch_mm16_tc(Mm16P p, int n_sms, cudaStream_t st);

#ifdef __CUDACC__

// two values to bf16 (nearest, ties to even), lo in the lower half
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// 1 / (1 + exp(-x)) of a number, small values to their last bits.  exp(-|x|)
// is 2^t, t = -|x| log2(e) carried in two terms, so that its relative error
// does not grow with |x|; the quotient's by an approximate reciprocal of 1 ..
// 2: 2^-22 in all.  (With expf and a division the epilogue of 8192 x 8192 x
// 2048 took 250 us instead of the product's 151.)
__device__ __forceinline__ float logistic(float x) {
  constexpr float kHi = 1.44269502f, kLo = 1.9259629e-8f;  // log2(e)
  const float y = fmaxf(-fabsf(x), -150.f), t = y * kHi, r = fmaf(y, kLo, fmaf(y, kHi, -t));
  float e, q;
  asm("ex2.approx.f32 %0, %1;" : "=f"(e) : "f"(t));
  e = fmaf(e * r, 0.693147181f, e);
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(q) : "f"(1.f + e));
  return (x < 0.f ? e : 1.f) * q;
}

#endif

}  // namespace moe
