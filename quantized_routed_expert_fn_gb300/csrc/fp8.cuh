// fp8.cuh -- parameters and helpers of the 8-bit expert kernels: routing from
// given logits, quantisation to e4m3 with E8M0 block scales, the
// block-scaled products and the routed experts' step.
#pragma once

#include <cuda.h>

#include <cstdint>

#include "common.cuh"

namespace moe {

// ---- routing (gate.cu)
struct GateP {
  const void *logits;
  int bf16;
  int64_t ld;
  const float *bias;  // [E] or nullptr
  int t, E, K;
  int sigmoid, renorm;
  int ng, gs, top_groups, group_top;  // ng 1: no groups; gs = E / ng
  float scale;
  uint32_t *idx;
  float *w;
};
cudaError_t launch_gate(const GateP &p, int n_sms, cudaStream_t st);

// ---- quantisation (quant8.cu)
struct Quant8P {
  const void *x;
  int bf16;
  int64_t ldx;
  int rows, cols;
  uint8_t *q;
  int64_t ldq;
  uint8_t *s;
  int64_t lds;
};
cudaError_t launch_quant8_rows(const Quant8P &p, int n_sms, cudaStream_t st);
cudaError_t launch_quant8_blocks(const Quant8P &p, cudaStream_t st);

// ---- products (mm8.cu)
struct Mm8Args {
  const uint8_t *a, *sa, *b, *sb;
  int64_t lda, lds;
  int t, n, k, nk, nb;  // nk = ceil(k / 128), nb = ceil(n / 128)
  int G;                // 0: one weight matrix for every row
  const int *offs;      // [G + 1] or nullptr
  void *out;            // [t][n], or h8 [t][n / 2] (silu)
  int64_t ldo;
  uint8_t *hs;          // silu: scales of h8
  int64_t ldhs;
  int wmax;             // token rows of a tile at most
  int wide;             // rows of out start on 16 bytes
  int tok, stage, stages;  // ring: token bytes a k block, bytes a stage, stages
  int withhold;
  int zero_status;      // the kernel zeroes *status first
  int *status;
  unsigned long long timeout_ns;
};
struct Mm8P : Mm8Args {
  // tokens: boxes of 1, 2, ... times 16 (or 32) rows; weights [G * n][k]:
  // boxes of 128 rows; 128 bytes of k a block, 128B swizzle
  CUtensorMap tm_a[7], tm_b;
};
enum { kOutF32 = 0, kOutBf16 = 1, kOutSilu8 = 2 };
// Whether the few-row kernel (weights streamed once into mma.sync) takes t
// rows.  The tensor-core kernel starts slower and takes k in series over n /
// 256 CTA pairs, whatever t; the few-row kernel shares k out over a CTA's
// warps, starts a CTA for every 16 of n, and takes longer with every group of
// eight rows.  us a call, few-row / tensor-core, in a graph of calls on
// weights that are not in L2 (bf16 out):
//   n x k          1 row        8 rows       16 rows      32 rows
//   2048 x 2048     2.9 / 6.4    3.2 / 6.4    3.9 / 6.4    5.7 / 6.5
//   4096 x 2048     4.2 / 6.5    4.4 / 6.6    5.3 / 6.6    7.5 / 6.6
//   8192 x 1024     4.1 / 5.5    4.6 / 5.6    6.1 / 5.6    8.6 / 5.6
//   4096 x 4096     6.4 / 9.2    6.9 / 9.3    8.8 / 9.3   12.8 / 9.4
//   8192 x 2048     6.1 / 7.3    6.7 / 7.4    9.0 / 7.4   13.5 / 7.4
//   8192 x 4096    10.4 / 11.0  11.3 / 11.0  15.9 / 11.0  23.7 / 11.1
//   4096 x 8192    11.0 / 14.4  11.5 / 14.4  15.1 / 14.4  23.1 / 14.6
//   8192 x 8192    19.0 / 17.8  19.8 / 17.8  27.9 / 17.8  42.8 / 17.8
//   16384 x 4096   16.6 / 15.2  17.7 / 15.3  26.6 / 15.3  42.6 / 15.2
//   4096 x 16384   19.7 / 24.6  20.6 / 24.7  27.6 / 24.7  47.3 / 24.7
//   16384 x 16384  55.9 / 47.2  57.8 / 47.3   100 / 47.5   169 / 47.4
inline bool mm8_small(int64_t t, int64_t n, int64_t k) {
  if (t <= 8) return n <= 4096 || n * k <= 1 << 25;
  if (t <= 16) return n * k < 1 << 23 || (n <= 4096 && n * k <= 1 << 24);
  return t <= 32 && n * k <= 1 << 22;
}
cudaError_t launch_mm8_small(const Mm8Args &p, int out_kind, cudaStream_t st);
cudaError_t launch_mm8_tc(const Mm8P &p, int out_kind, int n_sms, cudaStream_t st);

#ifdef __CUDACC__

// Programmatic dependent launch: the kernel may start while the one before it
// in the stream ends, and touches memory behind pdl_wait_prev only.  What a
// kernel does before that wait holds as long as the one before it lets it
// start (pdl_launch_next) behind its own.
__device__ __forceinline__ void pdl_launch_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void pdl_wait_prev() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
template <class F, class P>
cudaError_t launch_pdl(F f, dim3 grid, unsigned block, size_t smem, cudaStream_t st, const P &p) {
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, f, p);
}

// e8m0 byte -> the power of two it stands for
__device__ __forceinline__ float e8m0_f(uint32_t e) {
  return __uint_as_float(e == 0 ? 0x00400000u : (e == 255u ? 0x7fc00000u : e << 23));
}

// Two scales a and b of a product d (powers of two) are multiplied first, as
// scales far from 1 may cancel.  Where that is infinite or below the normal
// numbers, both are above 1 or both below: then d * a * b, one after the
// other, leaves the 32-bit range only where the result does, and zeros stay
// zeros (by_scales).  scales_hold: none of the N products is of that kind.
template <int N>
__device__ __forceinline__ bool scales_hold(const float (&p)[N]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < N; i++) m = max(m, __float_as_uint(p[i]) - 0x00800000u);
  return m < 0x7f000000u;
}
__device__ __forceinline__ float by_scales(float d, float a, float b) {
  const float p[1] = {a * b};
  return scales_hold(p) ? d * p[0] : d * a * b;
}

// Scale byte of a block whose largest finite magnitude has the bits `a`:
// the least e with |x| <= 448 * 2^(e - 127) = 1.75 * 2^(e - 119); 127 for a
// block of zeros, 0 at least.
__device__ __forceinline__ uint32_t e8m0_of_amax(uint32_t a) {
  if (a == 0) return 127u;
  int ex = (int)(a >> 23);           // a = m * 2^(ex - 127)
  const uint32_t m = a & 0x7fffffu;
  if (ex == 0) return 0u;            // below 2^-126: e would be below 0
  ex = ex - 8 + (m > 0x600000u);     // m > 1.75
  return ex > 0 ? (uint32_t)ex : 0u;
}
// 2^(127 - e): what a value is multiplied with before it is rounded
__device__ __forceinline__ float e8m0_inv(uint32_t e) {
  return e >= 254u ? __uint_as_float(0x00400000u) : __uint_as_float((254u - e) << 23);
}

// magnitude bits that count for the block's scale: finite values only
__device__ __forceinline__ uint32_t mag_bits(float v) {
  const uint32_t u = __float_as_uint(v) & 0x7fffffffu;
  return u < 0x7f800000u ? u : 0u;
}

// two values, scaled, to two e4m3 bytes (nearest, ties to even); SAFE:
// infinities become NaN (an infinity times 0 is the NaN the conversion keeps)
template <bool SAFE>
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  const float l = SAFE ? lo + 0.f * lo : lo, h = SAFE ? hi + 0.f * hi : hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(h), "f"(l));
  return r;
}
template <bool SAFE>
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  return e4m3x2<SAFE>(a, b) | e4m3x2<SAFE>(c, d) << 16;
}

// Warp: the 128 values of a scale block, N in each of 128 / N neighbouring
// lanes, to e4m3 words; e: the scale byte.  Values that are not finite are
// rare: a maximum that says one is there makes the warp do it with care.
template <int N>
__device__ __forceinline__ void quant_block(const float (&v)[N], uint32_t (&w)[N / 4], uint32_t &e) {
  uint32_t a = 0;
#pragma unroll
  for (int j = 0; j < N; j++) a = max(a, __float_as_uint(v[j]) & 0x7fffffffu);
#pragma unroll
  for (int o = 64 / N; o; o >>= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, o));
  if (__any_sync(0xffffffffu, a >= 0x7f800000u)) {
    a = 0;
#pragma unroll
    for (int j = 0; j < N; j++) a = max(a, mag_bits(v[j]));
#pragma unroll
    for (int o = 64 / N; o; o >>= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, o));
    e = e8m0_of_amax(a);
    const float f = e8m0_inv(e);
#pragma unroll
    for (int j = 0; j < N / 4; j++) w[j] = e4m3x4<true>(v[4 * j] * f, v[4 * j + 1] * f, v[4 * j + 2] * f, v[4 * j + 3] * f);
    return;
  }
  e = e8m0_of_amax(a);
  const float f = e8m0_inv(e);
#pragma unroll
  for (int j = 0; j < N / 4; j++) w[j] = e4m3x4<false>(v[4 * j] * f, v[4 * j + 1] * f, v[4 * j + 2] * f, v[4 * j + 3] * f);
}

// D(16x8 f32) += A(16x32 e4m3, row) * B(32x8 e4m3, col)
__device__ __forceinline__ void mma_e4m3(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

#endif

}  // namespace moe

namespace moe {

// ---- the routed experts' step (experts8.cu)
// shared-memory layouts of the few-row kernels, made on the host
struct GuLay {
  // bytes of a stage (8 rows), stages, teams.  An item is two stages; the
  // items' places in the ring are a multiple of the teams, so that a place is
  // one team's and that team waits for every phase of its barriers (one that
  // skipped a phase could not tell it from the phase before the last)
  int stage, ns, teams;
  size_t xs, sx, red, un, total;
};
struct DnLay {
  // bytes of a stage (16 rows), stages, warps at work: a divisor of the items
  // of a round of the ring, so that a stage's items are always the same warps'
  int stage, ns, warps;
  size_t hs, sh, sd, un, red, total;
};
struct Ex8P {
  GuLay gl;
  DnLay dl;
  unsigned long long timeout_ns;
  int H, E, I, t, K;
  const uint8_t *gu, *gus, *dn, *dns;
  const void *x;
  int x_bf16, out_bf16;
  const uint32_t *idx;  // [t][K]
  const float *w;       // [t][K]
  void *out;            // [t][H]
  int *status;
  // workspace
  float *h32;           // few rows: [t * K][I]
  uint8_t *h8, *h8s;    // [t * K][I] e4m3 and [t * K][ldi] scales
  int ldi, ldh;         // scale bytes of a row of h8 / x8
  uint8_t *x8, *x8s;    // many rows: [t * K][H] grouped rows, [t * K][ldh]
  int *counts;          // [E] entries per expert, then one ticket
  int *offs;            // [E + 1]
  int *place;           // [t * K] place of an entry within its expert, -1: none
  float *y;             // [t * K][H] the entries' outputs, not weighted yet
};
struct Ex8Sizes {
  size_t h32, h8, h8s, x8, x8s, counts, offs, place, y, total;
};
constexpr int kEx8SmallRows = 8;  // rows of the few-row path: one column each of an m16n8 tile
bool ex8_small(int H, int I, int t, int K);
Ex8Sizes ex8_sizes(int H, int E, int I, int t, int K);
cudaError_t launch_ex8_small(Ex8P &p, int n_sms, cudaStream_t st);
cudaError_t launch_ex8_group(const Ex8P &p, cudaStream_t st);
cudaError_t launch_ex8_combine(const Ex8P &p, int n_sms, cudaStream_t st);

}  // namespace moe
