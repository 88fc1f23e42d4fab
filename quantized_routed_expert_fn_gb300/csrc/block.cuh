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
  float eps;
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
  int T;  // threads of a row
};
constexpr int kNormMaxCols = 32768;
cudaError_t launch_norm(const NormP &p, int n_sms, cudaStream_t st);

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
  int wide;  // four neighbouring values of out (and residual) are one access
  int withhold;
  int *status;
  unsigned long long timeout_ns;
  // tensor cores: tokens of a tile, k blocks, weight and token tiles, CTAs
  // that split k, ring
  int w, nk, nmt, ntt, split, stage, stages;
};
struct Mm16P : Mm16Args {
  CUtensorMap tm_a, tm_b;
};
// Whether the few-row kernel takes t rows.
inline bool mm16_few(int64_t t, int64_t, int64_t) { return t <= 8; }
cudaError_t launch_mm16_few(const Mm16Args &p, cudaStream_t st);
cudaError_t launch_mm16_tc(Mm16P p, int n_sms, cudaStream_t st);

}  // namespace moe
