// mm16.cu -- bf16 matrix products with what follows them in their epilogue:
//   z = a b^T + bias;  h = act(z), or gated act(z[:, :n]) * z[:, n:]
//   out = row_scale[r] * h + residual
//
// Two kernels:
//   few   up to 16 rows, by mm16_few: the weights are streamed once from HBM
//         straight into the fragments of mma.sync, a CTA takes 16 weight rows
//         and splits k over its warps.
//   tc    any number of rows: tcgen05 (kind::f16, fp32 accumulators in TMEM)
//         fed by TMA, in three forms.  Weights on the M side, tokens on the N
//         side, as the 8-bit products have them: M stays full whatever the
//         number of rows.  The same where there are too few tiles for the SMs,
//         a cluster of S CTAs a tile that split k and add their accumulators
//         in a fixed order.  Tokens on the M side: a lane has a token's
//         outputs one after another, and nothing is exchanged for them.  The
//         first and the last are persistent, over CTA pairs (256 x up to 256)
//         where the M side has two tiles.
#include <cuda_runtime.h>

#include <type_traits>

#include "block.cuh"
#include "fp8.cuh"
#include "tc05.cuh"
#include "tmap.cuh"

namespace moe {
namespace {

constexpr unsigned FULLM = 0xffffffffu;

// z times the normal distribution's function P(z).  P(-a) = exp(-a^2 / 2) q(u),
// u = 1 / (1 + 0.23 a), q a polynomial fitted to erfcx(a / sqrt 2) / 2 over 0
// <= a <= 14.5 (least relative error, by reweighted least squares: 5e-8); the
// square and its multiple of log2(e) are carried in two terms.
__device__ __forceinline__ float gelu(float z) {
  const float a = fminf(fabsf(z), 15.f);
  float u, e;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(u) : "f"(fmaf(0.23f, a, 1.f)));
  float q = -7.84846712e-02f;
  q = fmaf(q, u, 2.90501394e-01f), q = fmaf(q, u, -2.78316041e-01f), q = fmaf(q, u, 3.01701127e-01f);
  q = fmaf(q, u, -3.30880031e-02f), q = fmaf(q, u, 1.19590782e-01f), q = fmaf(q, u, 8.57416379e-02f);
  q = fmaf(q, u, 9.23817254e-02f), q = fmaf(q, u, -2.79751048e-05f);
  constexpr float kHi = 0.72134751f, kLo = 9.6298150e-9f;  // log2(e) / 2
  const float s = a * a, t = s * kHi, r = fmaf(s, kLo, fmaf(fmaf(a, a, -s), kHi, fmaf(s, kHi, -t)));
  asm("ex2.approx.f32 %0, %1;" : "=f"(e) : "f"(-t));
  const float below = q * fmaf(-e * r, 0.693147181f, e);
  return z * (z < 0.f ? below : 1.f - below);
}
__device__ __forceinline__ float activate(float z, int act) {
  switch (act) {
    case kActSilu: return z * logistic(z);
    case kActGelu: return gelu(z);
    case kActGeluTanh:  // (1 + tanh u) / 2 = 1 / (1 + exp(-2 u))
      return z * logistic(z * fmaf(z * z, 0.07135481627f, 1.5957691216f));
    case kActRelu: return z < 0.f ? 0.f : z;  // NaN stays
    case kActSigmoid: return z == z ? logistic(z) : z;
    default: return z;
  }
}

// the same of N values: one look at what is asked for
template <int N>
__device__ __forceinline__ void activate_all(float (&z)[N], int act) {
  auto all = [&](auto f) {
#pragma unroll
    for (int i = 0; i < N; i++) z[i] = f(z[i]);
  };
  switch (act) {
    case kActSilu: return all([](float x) { return activate(x, kActSilu); });
    case kActGelu: return all([](float x) { return activate(x, kActGelu); });
    case kActGeluTanh: return all([](float x) { return activate(x, kActGeluTanh); });
    case kActRelu: return all([](float x) { return activate(x, kActRelu); });
    case kActSigmoid: return all([](float x) { return activate(x, kActSigmoid); });
    default: return;
  }
}

__device__ __forceinline__ uint16_t bf16_of(float v) {
  uint16_t h;
  asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(h) : "f"(v));
  return h;
}

// One output: row r, column j, from h = the activated product.
__device__ __forceinline__ uint32_t residual1(const Mm16Args &P, int64_t r, int j) {
  const int64_t i = r * P.ldr + j;
  return P.res_bf16 ? (uint32_t)static_cast<const uint16_t *>(P.res)[i] << 16 : static_cast<const uint32_t *>(P.res)[i];
}
__device__ __forceinline__ void store1(const Mm16Args &P, int64_t r, int j, float v) {
  const int64_t o = r * P.ldo + j;
  if (P.out_bf16) static_cast<uint16_t *>(P.out)[o] = bf16_of(v);
  else static_cast<float *>(P.out)[o] = v;
}
__device__ __forceinline__ void finish1(const Mm16Args &P, int64_t r, int j, float h, float rs) {
  const float v = h * rs;
  store1(P, r, j, P.res ? v + __uint_as_float(residual1(P, r, j)) : v);
}
// Four neighbouring ones, in rows that allow whole accesses (P.wide); the
// residual's come first, so that they are on their way meanwhile.
__device__ __forceinline__ uint4 residual4(const Mm16Args &P, int64_t r, int j) {
  const int64_t i = r * P.ldr + j;
  if (!P.res_bf16) return *reinterpret_cast<const uint4 *>(static_cast<const float *>(P.res) + i);
  const uint2 u = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(P.res) + i);
  return make_uint4(u.x, u.y, 0u, 0u);
}
__device__ __forceinline__ void finish4(const Mm16Args &P, int64_t r, int j, const float *h, float rs, const uint4 &u) {
  float4 v = make_float4(h[0] * rs, h[1] * rs, h[2] * rs, h[3] * rs);
  if (P.res) {
    if (P.res_bf16) v.x += bf16lo(u.x), v.y += bf16hi(u.x), v.z += bf16lo(u.y), v.w += bf16hi(u.y);
    else
      v.x += __uint_as_float(u.x), v.y += __uint_as_float(u.y), v.z += __uint_as_float(u.z), v.w += __uint_as_float(u.w);
  }
  const int64_t o = r * P.ldo + j;
  if (P.out_bf16)
    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(P.out) + o) = make_uint2(bf16x2(v.x, v.y), bf16x2(v.z, v.w));
  else
    *reinterpret_cast<float4 *>(static_cast<float *>(P.out) + o) = v;
}

// ------------------------------------------------------------ few rows

constexpr int kFewWarps = 8;
// The tensor cores cut off what lies below 2^-23 of a sum at every step of 16
// of k, towards zero.  The k blocks of 64 that are summed so at most; longer
// sums are added up from these in 32 bits, rounded to nearest.  Terms of one
// sign then lose 2^-15 of the sum at most whatever k (measured: 1.0e-5; of
// 65536 in two sums 1.7e-4, of 2^19 in one 0.28 %), of bf16 outputs, whose
// rounding is 2^-8, 2^-12.
constexpr int kSumBlocks = 64, kSumBlocksBf16 = 512;

// A tile: 16 weight rows (gated: 8 gate rows and the 8 up rows of the same
// outputs) by 8 * NT token rows.  Lane (g, q) = (lane / 4, lane % 4) loads 16
// bytes of weight rows g and g + 8 at k = 8q and 32 + 8q of a block of 64: the
// four words of a piece serve as the k halves of two MMAs, and the same
// pieces of the token rows as B, so the order of k is permuted alike on both
// sides.  Warp w takes the blocks w, w + 8, ...; the warps' sums meet in
// shared memory in a fixed order.  A CTA walks the tiles i, i + grid, ...,
// the next D blocks' weights always on their way, across the tiles' ends.
// LONG: a warp's sums go to shared memory every kSumBlocks blocks.
template <int NT, int D, bool LONG>
__global__ void __launch_bounds__(32 * kFewWarps) mm16_few_rows(const __grid_constant__ Mm16Args P) {
  __shared__ float red[2][kFewWarps][16][8 * NT + 1];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q = lane & 3;
  pdl_wait_prev();
  pdl_launch_next();
  if (blockIdx.x == 0 && tid == 0) *P.status = 0;
  const int per = P.gated ? 8 : 16, nb = (P.k + 63) / 64, tiles = (P.n + per - 1) / per;
  const int mine = (nb - warp + kFewWarps - 1) / kFewWarps, rounds = (mine + D - 1) / D * D;  // blocks a tile
  const uint4 zero = make_uint4(0, 0, 0, 0);
  // 8 values from k on; the last ones of a row may be fewer
  auto piece = [&](const uint16_t *row, int k, bool ok, bool stream) {
    if (!ok || k >= P.k) return zero;
    if (k + 8 <= P.k) return stream ? ldg_stream4(row + k) : *reinterpret_cast<const uint4 *>(row + k);
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; j++) {
      const uint32_t lo = k + 2 * j < P.k ? row[k + 2 * j] : 0, hi = k + 2 * j + 1 < P.k ? row[k + 2 * j + 1] : 0;
      w[j] = lo | hi << 16;
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  };
  // the weights' place: block `at` (of the warp's) of tile `pt`
  int pt = blockIdx.x, at = 0;
  const uint16_t *w0, *w1;
  bool ok0, ok1;
  auto place = [&] {
    const int r0 = pt * per + g, r1 = P.gated ? P.n + r0 : r0 + 8;
    ok0 = pt < tiles && r0 < P.n, ok1 = P.gated ? ok0 : pt < tiles && r1 < P.n;
    w0 = P.b + (int64_t)r0 * P.ldb, w1 = P.b + (int64_t)r1 * P.ldb;
  };
  place();
  uint4 a[D][2][2], b[D][NT][2];  // [block][piece][row], [block][token rows][piece]
  auto load = [&](uint4 (&x)[2][2], uint4 (&y)[NT][2]) {
    const int k0 = (warp + at * kFewWarps) * 64 + q * 8;  // blocks beyond the warp's last are beyond k
#pragma unroll
    for (int p = 0; p < 2; p++) x[p][0] = piece(w0, k0 + 32 * p, ok0, true), x[p][1] = piece(w1, k0 + 32 * p, ok1, true);
#pragma unroll
    for (int j = 0; j < NT; j++)
#pragma unroll
      for (int p = 0; p < 2; p++) y[j][p] = piece(P.a + (int64_t)(8 * j + g) * P.lda, k0 + 32 * p, 8 * j + g < P.t, false);
    if (++at == rounds) at = 0, pt += gridDim.x, place();
  };
  if (mine > 0)
#pragma unroll
    for (int i = 0; i < D; i++) load(a[i], b[i]);
  int buf = 0;
  for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x, buf ^= 1) {
    float acc[NT][4];
#pragma unroll
    for (int j = 0; j < NT; j++)
#pragma unroll
      for (int i = 0; i < 4; i++) acc[j][i] = 0.f;
    // onto what lies at this lane's places
    auto add_up = [&](bool first) {
#pragma unroll
      for (int j = 0; j < NT; j++)
#pragma unroll
        for (int i = 0; i < 4; i++) {
          float &to = red[buf][warp][g + 8 * (i >> 1)][8 * j + 2 * q + (i & 1)];
          to = first ? acc[j][i] : to + acc[j][i];
          acc[j][i] = 0.f;
        }
    };
    for (int i0 = 0; i0 < rounds; i0 += D) {
#pragma unroll
      for (int d = 0; d < D; d++) {
        if (i0 + d < mine) {
#pragma unroll
          for (int j = 0; j < NT; j++)
#pragma unroll
            for (int p = 0; p < 2; p++) {
              mma_bf16_16816(acc[j], a[d][p][0].x, a[d][p][1].x, a[d][p][0].y, a[d][p][1].y, b[d][j][p].x, b[d][j][p].y);
              mma_bf16_16816(acc[j], a[d][p][0].z, a[d][p][1].z, a[d][p][0].w, a[d][p][1].w, b[d][j][p].z, b[d][j][p].w);
            }
        }
        load(a[d], b[d]);
      }
      if (LONG && (i0 + D) % kSumBlocks == 0) add_up(i0 + D == kSumBlocks);
    }
    if constexpr (LONG) {
      add_up(rounds < kSumBlocks);
    } else {
#pragma unroll
      for (int j = 0; j < NT; j++) {
        const int c = 8 * j + 2 * q;
        red[buf][warp][g][c] = acc[j][0], red[buf][warp][g][c + 1] = acc[j][1];
        red[buf][warp][g + 8][c] = acc[j][2], red[buf][warp][g + 8][c + 1] = acc[j][3];
      }
    }
    __syncthreads();  // the other buffer is read: every thread is past the tile before
    auto sum = [&](int row, int c) {
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kFewWarps; w++) v += red[buf][w][row][c];
      return v;
    };
    const int n0 = tile * per;
    for (int i = tid; i < per * 8 * NT; i += 32 * kFewWarps) {
      const int j = i & (per - 1), c = i / per;
      if (c < P.t && n0 + j < P.n) {
        float z = sum(j, c);
        if (P.bias) z += P.bias[n0 + j];
        z = activate(z, P.act);
        if (P.gated) {
          float u = sum(j + 8, c);
          if (P.bias) u += P.bias[P.n + n0 + j];
          z *= u;
        }
        finish1(P, c, n0 + j, z, P.row_scale ? P.row_scale[c] : 1.f);
      }
    }
  }
}

// ------------------------------------------------------------ tensor cores
//
//   warps 0-15 epilogue, in four groups
//   warp 16   (even CTA) issues a stage's MMAs once its operands are there
//   warp 17   TMA
// gated: a tile's 128 weight rows are 64 gate rows and the 64 up rows of the
// same outputs, so that both meet in the piece in shared memory.
// The full and acc_empty barriers of a pair are the even CTA's; the others are
// each CTA's own, committed to both.
constexpr int kEpi = 16;  // epilogue warps, in groups of four (one for each 32 lanes of TMEM)
constexpr int kTcThreads = 32 * (kEpi + 3);
constexpr int kResBufs = 2;  // pieces of residuals on their way
constexpr int kMaxStages = 10;
constexpr int kPiece = 16 * 128 * 4;  // bytes of 16 tokens x 128 rows

struct Bars {
  uint64_t full[kMaxStages], empty[kMaxStages], acc_full[2], acc_empty[2], res_full[kResBufs], res_empty[kResBufs], drain;
  uint32_t tmem;
};
constexpr int kResPiece = 128 * 128;      // bytes of 128 tokens' residuals: 64 columns of bf16, 32 of fp32
static_assert(kResBufs * kResPiece <= kEpi / 4 * kPiece, "they lie where the other forms have their pieces");
constexpr int kOffBars = kEpi / 4 * kPiece;
constexpr int kOffRing = (kOffBars + (int)sizeof(Bars) + 1023) / 1024 * 1024;
constexpr int kRoom = 226 * 1024 - kOffRing;

template <bool CL>
__device__ bool tc_wait(uint64_t *bar, uint32_t par, const Mm16Args &P) {
  // asleep on the barrier meanwhile: polling takes issue slots and power
  auto done = [&] { return CL ? tc05::mbar_sleep_wait_cluster(bar, par) : tc05::mbar_sleep_wait(bar, par); };
  if (done()) return true;
  const uint64_t t0 = globaltimer();
  while (!done()) {
    if (globaltimer() - t0 > P.timeout_ns) {
      atomicCAS(P.status, 0, kStatusTimeout);
      return false;
    }
  }
  return true;
}
template <bool CL>
__device__ __forceinline__ bool tc_warp_wait(uint64_t *bar, uint32_t par, const Mm16Args &P) {
  bool ok = true;
  if ((threadIdx.x & 31) == 0) ok = tc_wait<CL>(bar, par, P);
  return __shfl_sync(FULLM, ok ? 1 : 0, 0) != 0;
}

// 16 neighbouring values of SIZE bytes, 32 bytes an access
template <int SIZE>
__device__ __forceinline__ void store_run(void *p, const uint32_t *v) {
#pragma unroll
  for (int i = 0; i < SIZE / 2; i++)
    asm volatile("st.global.v8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"r"(v[8 * i]), "r"(v[8 * i + 1]),
                 "r"(v[8 * i + 2]), "r"(v[8 * i + 3]), "r"(v[8 * i + 4]), "r"(v[8 * i + 5]), "r"(v[8 * i + 6]),
                 "r"(v[8 * i + 7]), "l"(static_cast<uint8_t *>(p) + 32 * i)
                 : "memory");
}
// the same n values for every lane
__device__ __forceinline__ void load_bias(float (&v)[16], const float *bias, int n) {
  if (n == 16 && ((uintptr_t)bias & 15u) == 0) {
#pragma unroll
    for (int j = 0; j < 16; j += 4) {
      const float4 b = *reinterpret_cast<const float4 *>(bias + j);
      v[j] = b.x, v[j + 1] = b.y, v[j + 2] = b.z, v[j + 3] = b.w;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 16; j++) v[j] = j < n ? bias[j] : 0.f;
  }
}

// Warp: outputs of the tokens of a piece, which lie as z [token][128] in
// shared memory (plain: 128 outputs a token; gated: 64, from the values i and
// 64 + i).  In whole rows (four values a lane, a token's row by one warp, or
// half a warp where it is gated) fetch() asks for the residuals and row
// scales of NP such rows, before the piece is there; else of values one by
// one, neighbouring lanes on neighbouring columns.
template <int NP>
struct Outputs {
  uint4 res[NP];
  float rs[NP];
  // row i of this lane: its token among the piece's `j0 + i * step`
  __device__ __forceinline__ static int token(const Mm16Args &P, int i, int j0, int step) {
    return P.gated ? j0 + step * (2 * i + ((threadIdx.x & 31) >> 4)) : j0 + step * i;
  }
  // whole: rows of whole accesses
  __device__ __forceinline__ void fetch(const Mm16Args &P, int64_t r0, int n, int nbase, int j0, int step, bool whole) {
    const int lane = threadIdx.x & 31;
    if (whole) {
      const int col = nbase + 4 * (P.gated ? lane & 15 : lane), rows = P.gated ? NP / 2 : NP;
#pragma unroll
      for (int i = 0; i < NP; i++) {
        const int j = token(P, i, j0, step);
        if (i < rows && j < n) {
          if (P.res) res[i] = residual4(P, r0 + j, col);
          rs[i] = P.row_scale ? P.row_scale[r0 + j] : 1.f;
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < NP; i++) {
        const int j = j0 + step * i;
        if (j < n) {
          if (P.res) {
            uint32_t x[4];
#pragma unroll
            for (int e = 0; e < 4; e++) {
              const int c = nbase + lane + 32 * e;
              x[e] = c < P.n && (e < 2 || !P.gated) ? residual1(P, r0 + j, c) : 0u;
            }
            res[i] = make_uint4(x[0], x[1], x[2], x[3]);
          }
          rs[i] = P.row_scale ? P.row_scale[r0 + j] : 1.f;
        }
      }
    }
  }
  __device__ __forceinline__ void write(const Mm16Args &P, int64_t r0, int n, int nbase, const float *z, int j0, int step,
                                        bool whole) const {
    if (whole) write4(P, r0, n, nbase, z, j0, step);
    else write1(P, r0, n, nbase, z, j0, step);
  }
  __device__ __forceinline__ void write4(const Mm16Args &P, int64_t r0, int n, int nbase, const float *z, int j0, int step) const {
    const int lane = threadIdx.x & 31;
    if (!P.gated) {
#pragma unroll
      for (int i0 = 0; i0 < NP; i0 += 4) {
        float h[16];
#pragma unroll
        for (int i = 0; i < 4; i++) {
          const int j = j0 + step * (i0 + i);
          const float4 v = j < n ? *reinterpret_cast<const float4 *>(z + j * 128 + 4 * lane) : make_float4(0.f, 0.f, 0.f, 0.f);
          h[4 * i] = v.x, h[4 * i + 1] = v.y, h[4 * i + 2] = v.z, h[4 * i + 3] = v.w;
        }
        activate_all(h, P.act);
#pragma unroll
        for (int i = 0; i < 4; i++) {
          const int j = j0 + step * (i0 + i);
          if (j < n) finish4(P, r0 + j, nbase + 4 * lane, h + 4 * i, rs[i0 + i], res[i0 + i]);
        }
      }
    } else {
      const int l = lane & 15;
#pragma unroll
      for (int i0 = 0; i0 < NP / 2; i0 += 2) {
        float h[8], u[8];
#pragma unroll
        for (int i = 0; i < 2; i++) {
          const int j = token(P, i0 + i, j0, step);
          const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
          const float4 v = j < n ? *reinterpret_cast<const float4 *>(z + j * 128 + 4 * l) : zero;
          const float4 x = j < n ? *reinterpret_cast<const float4 *>(z + j * 128 + 64 + 4 * l) : zero;
          h[4 * i] = v.x, h[4 * i + 1] = v.y, h[4 * i + 2] = v.z, h[4 * i + 3] = v.w;
          u[4 * i] = x.x, u[4 * i + 1] = x.y, u[4 * i + 2] = x.z, u[4 * i + 3] = x.w;
        }
        activate_all(h, P.act);
#pragma unroll
        for (int i = 0; i < 8; i++) h[i] *= u[i];
#pragma unroll
        for (int i = 0; i < 2; i++) {
          const int j = token(P, i0 + i, j0, step);
          if (j < n) finish4(P, r0 + j, nbase + 4 * l, h + 4 * i, rs[i0 + i], res[i0 + i]);
        }
      }
    }
  }
  __device__ __forceinline__ void write1(const Mm16Args &P, int64_t r0, int n, int nbase, const float *z, int j0, int step) const {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < NP; i++) {
      const int j = j0 + step * i;
      if (j < n) {
        const float *x = z + j * 128 + lane;
        float h[4] = {x[0], x[32], P.gated ? 0.f : x[64], P.gated ? 0.f : x[96]};
        activate_all(h, P.act);
        if (P.gated) h[0] *= x[64], h[1] *= x[96];
        const uint32_t u[4] = {res[i].x, res[i].y, res[i].z, res[i].w};
#pragma unroll
        for (int e = 0; e < 4; e++) {
          const int c = nbase + lane + 32 * e;
          const float v = h[e] * rs[i];
          if (c < P.n && (e < 2 || !P.gated)) store1(P, r0 + j, c, P.res ? v + __uint_as_float(u[e]) : v);
        }
      }
    }
  }
};

enum { kWeights = 0, kSplit = 1, kTokens = 2 };  // what is on the M side; kSplit: weights, k split over a cluster

// 16 columns of an accumulator, with what lies in the other half of tensor memory
__device__ __forceinline__ void read_sums(uint32_t at, bool both, float (&x)[16]) {
  tc05::ld16(at, x);
  if (both) {
    float y[16];
    tc05::ld16(at + 256, y);
#pragma unroll
    for (int j = 0; j < 16; j++) x[j] += y[j];
  }
}
// Warp: an accumulator is read, and the MMAs may fill it again.
template <int CG>
__device__ __forceinline__ void release_acc(uint64_t *bar) {
  tc05::fence_before();
  __syncwarp();
  if ((threadIdx.x & 31) == 0) {
    if constexpr (CG == 1) tc05::mbar_arrive(bar);
    else tc05::mbar_arrive_cluster(tc05::map_rank(bar, 0));
  }
}

// LONG: a tile's k is summed P.chunk blocks at a time in the first half of tensor
// memory, and added up in the second.  A kernel of its own, as its loops cost
// the others 1 to 4 %.  One accumulator at a time: tiles of 160 columns, of
// which two and the sum so far fit, took 501 us instead of 340 at 2048 x 2048 x
// 65536, fp32.
template <int CG, int FORM, bool LONG>
__global__ void __launch_bounds__(kTcThreads, 1) mm16_tc(const __grid_constant__ Mm16P P) {
  constexpr bool CL = CG == 2, SPLIT = FORM == kSplit, TOK = FORM == kTokens;
  static_assert(!SPLIT || CG == 1, "a split tile is one CTA's rows");
  pdl_launch_next();
  extern __shared__ __align__(1024) uint8_t smraw[];
  // the same offset in all CTAs of a cluster: dynamic shared memory starts alike
  uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smraw) + 1023) & ~(uintptr_t)1023);
  uint8_t *ring = sm + kOffRing;
  Bars &B = *reinterpret_cast<Bars *>(sm + kOffBars);
  const int S = P.stages;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = CG == 2 || SPLIT ? (int)tc05::cluster_rank() : 0;

  if (tid == 0) {
    for (int s = 0; s < S; s++) mbar_init(&B.full[s], 1), mbar_init(&B.empty[s], 1);
    for (int b = 0; b < 2; b++) mbar_init(&B.acc_full[b], 1), mbar_init(&B.acc_empty[b], kEpi * CG);
    for (int b = 0; b < kResBufs; b++) mbar_init(&B.res_full[b], 1), mbar_init(&B.res_empty[b], kEpi);
    mbar_init(&B.drain, 1);
    fence_mbar_init();
  }
  if (warp == kEpi) {
    if constexpr (CG == 1) tc05::alloc(&B.tmem, 512);
    else tc05::alloc_pair(&B.tmem, 512);
  }
  pdl_wait_prev();  // the operands may be the previous kernel's
  // the status of the call: a wait gives up long after
  if (tid == 0 && blockIdx.x == 0) *P.status = 0;
  tc05::fence_before();
  if constexpr (CG == 1 && !SPLIT) __syncthreads();
  else tc05::cluster_sync();
  tc05::fence_after();
  const uint32_t tmem = B.tmem;

  const int w = P.w, mrank = CG == 2 ? rank : 0;
  const int rows = P.gated ? 64 : 128;         // weights on the M side: outputs of a CTA's tile
  const int cols = P.gated ? w / 2 : w;        // tokens on it: outputs of a tile
  const int nmp = (P.nmt + CG - 1) / CG;       // M tiles, CG at a time
  const int ntiles = P.ntt * nmp;
  const int width = CG == 2 ? 2 : (SPLIT ? P.split : 1);  // CTAs of a tile
  const int cl = (int)blockIdx.x / width, ncl = (int)gridDim.x / width;
  const int my_tiles = cl < ntiles ? (ntiles - 1 - cl) / ncl + 1 : 0;
  int kb0 = 0, kb1 = P.nk;
  if constexpr (SPLIT) kb0 = (int)((int64_t)P.nk * rank / P.split), kb1 = (int)((int64_t)P.nk * (rank + 1) / P.split);
  const int parts = LONG ? (kb1 - kb0 + P.chunk - 1) / P.chunk : 1;  // sums of a tile
  // whether there is one accumulator, the other half of tensor memory taken (read
  // again each time: a flag kept costs registers that the epilogue spills)
  auto single = [&] { return LONG || P.two; };
  // tile i: the M tiles of an N tile follow one another
  int tt = cl / nmp, mp = cl - tt * nmp;
  const int step_t = ncl / nmp, step_m = ncl - step_t * nmp;
  struct Tile {
    int mt, n0, nlen;  // M tile; N side: first token and their number, or first output column
  };
  auto next_tile = [&] {
    Tile T;
    T.mt = mp * CG + mrank;
    T.n0 = tt * (TOK ? cols : w);
    T.nlen = min(w, P.t - T.n0);
    tt += step_t, mp += step_m;
    if (mp >= nmp) mp -= nmp, tt++;
    return T;
  };

  if (warp == kEpi) {
    // ---------------------------------------------------------------- MMA issue
    if (mrank == 0 && tc05::elect_one()) {
      int s = 0;
      uint32_t ph = 0;
      bool ok = true;
      const uint32_t base = smem_u32(ring), idesc = tc05::idesc_f16(128 * CG, w);
      for (int lt = 0; lt < my_tiles && ok; lt++) {
        for (int p = 0; p < parts && ok; p++) {
          const int b = single() ? 0 : lt & 1, use = single() ? lt * parts + p : lt >> 1;
          if (!tc_wait<CL>(&B.acc_empty[b], (uint32_t)((use & 1) ^ 1), P)) {
            ok = false;
            break;
          }
          tc05::fence_after();
          uint32_t d = tmem + (uint32_t)(b * 256);
          int start = LONG ? kb0 + p * P.chunk : kb0;
          const int end = LONG ? min(kb1, start + P.chunk) : kb1;
          for (int kb = start; kb < end; kb++) {
            if (!LONG && P.two && kb == P.nk / 2) d += 256, start = kb;
            if (!tc_wait<CL>(&B.full[s], ph, P)) {
              ok = false;
              break;
            }
            tc05::fence_after();
            const uint32_t st = base + (uint32_t)(s * P.stage);
            const uint64_t ad = tc05::sdesc(st), bd = tc05::sdesc(st + 16384);
#pragma unroll
            for (int j = 0; j < 4; j++) tc05::mma_f16<CG>(d, ad + 2 * j, bd + 2 * j, idesc, kb != start || j != 0);
            if constexpr (CG == 1) tc05::commit(&B.empty[s]);
            else tc05::commit_pair(&B.empty[s]);
            if (++s == S) s = 0, ph ^= 1;
          }
          if (ok) {
            if constexpr (CG == 1) tc05::commit(&B.acc_full[b]);
            else tc05::commit_pair(&B.acc_full[b]);
          }
        }
      }
      // every MMA issued here has completed before TMEM is released
      if constexpr (CG == 1) tc05::commit(&B.drain);
      else tc05::commit_pair(&B.drain);
      tc_wait<CL>(&B.drain, 0, P);
    }
    __syncwarp();
  } else if (warp == kEpi + 1) {
    // ---------------------------------------------------------------- TMA
    int f = 0, s = 0;
    uint32_t ph = 0;
    bool ok = true;
    const int tok = w / CG;
    const uint32_t bytes = (uint32_t)(16384 + tok * 128) * CG;
    for (int lt = 0; lt < my_tiles && ok; lt++) {
      const Tile T = next_tile();
      const int wr = T.mt * rows;
      for (int kb = kb0; kb < kb1; kb++, f++) {
        // (failure-detection test: CTA 0 never expects its first stage's
        // copies, so the MMA warp's bounded wait runs out)
        if (!tc_warp_wait<CL>(&B.empty[s], ph ^ 1, P) || (P.withhold && blockIdx.x == 0 && f == 0)) {
          ok = false;
          break;
        }
        if (tc05::elect_one()) {
          uint8_t *st = ring + s * P.stage;
          if (mrank == 0) mbar_expect_tx(&B.full[s], bytes);
          const uint32_t bar = CG == 1 ? smem_u32(&B.full[s]) : tc05::map_rank(&B.full[s], 0);
          if constexpr (!TOK) {
            tc05::tma_load_xy<CG>(st, &P.tm_b, kb * 64, wr, bar);
            if (P.gated) tc05::tma_load_xy<CG>(st + 8192, &P.tm_b, kb * 64, P.n + wr, bar);
            tc05::tma_load_xy<CG>(st + 16384, &P.tm_a, kb * 64, T.n0 + mrank * tok, bar);
          } else {
            tc05::tma_load_xy<CG>(st, &P.tm_a, kb * 64, T.mt * 128, bar);
            // columns: gated, the gates and then the up rows, of a pair one each
            const int first = P.gated ? T.n0 + mrank * P.n : T.n0 + mrank * tok;
            tc05::tma_load_xy<CG>(st + 16384, &P.tm_b, kb * 64, first, bar);
            if (CG == 1 && P.gated) tc05::tma_load_xy<CG>(st + 16384 + tok * 64, &P.tm_b, kb * 64, P.n + first, bar);
          }
        }
        __syncwarp();
        if (++s == S) s = 0, ph ^= 1;
      }
    }
    // copies still in flight land before the CTA (the pair) ends
    if (lane == 0 && mrank == 0)
      for (int g = f > S ? f - S : 0; g < f; g++) tc_wait<CL>(&B.full[g % S], (uint32_t)((g / S) & 1), P);
    __syncwarp();
  } else if (warp == kEpi + 2) {
    // ---------------------------------------------------------------- residuals
    // (tokens on the M side) this CTA's 128 tokens' of a tile, a piece of
    // columns after the other (what the last piece holds beyond the tile's
    // columns is used by none)
    if (TOK && P.res) {
      int f = 0;
      bool ok = true;
      const int step = P.res_bf16 ? 64 : 32;
      for (int lt = 0; lt < my_tiles && ok; lt++) {
        const Tile T = next_tile();
        const int end = min(cols, P.n - T.n0);
        for (int c = 0; c < end; c += step, f++) {
          const int b = f % kResBufs;
          if (!tc_warp_wait<false>(&B.res_empty[b], (uint32_t)(((f / kResBufs) & 1) ^ 1), P)) {
            ok = false;
            break;
          }
          if (tc05::elect_one()) {
            mbar_expect_tx(&B.res_full[b], kResPiece);
            tc05::tma_load_xy<1>(sm + b * kResPiece, &P.tm_r, T.n0 + c, T.mt * 128, smem_u32(&B.res_full[b]));
          }
          __syncwarp();
        }
      }
      if (lane == 0)
        for (int g = f > kResBufs ? f - kResBufs : 0; g < f; g++)
          tc_wait<false>(&B.res_full[g % kResBufs], (uint32_t)((g / kResBufs) & 1), P);
      __syncwarp();
    }
  } else {
    // ---------------------------------------------------------------- epilogue
    const int q = warp & 3, grp = warp >> 2;  // TMEM lane quadrant; group: pieces grp, grp + 4, ...
    const int row = 32 * q + lane;            // the tile's weight row of this thread
    float *stg = reinterpret_cast<float *>(sm + grp * kPiece);
    bool fine = true, res_ok = true;
    int res_at = 0;  // pieces of residuals before the tile
    for (int lt = 0; lt < my_tiles; lt++) {
      const Tile T = next_tile();
      const int b = single() ? 0 : lt & 1, use = single() ? lt * parts + parts - 1 : lt >> 1, nbase = T.mt * rows;
      if constexpr (LONG) {
        const uint32_t tl = tmem + ((uint32_t)(32 * q) << 16);
        for (int p = 0; p < parts - 1; p++) {
          fine = tc05::named_and(5, 32 * kEpi, res_ok && (warp != 0 || tc_warp_wait<CL>(&B.acc_full[0], (uint32_t)((lt * parts + p) & 1), P)));
          if (!fine) break;
          tc05::fence_after();
#pragma unroll 1
          for (int c0 = 16 * grp; c0 < w; c0 += 4 * kEpi) {
            float v[16];
            read_sums(tl + c0, p > 0, v);
            tc05::st16(tl + 256 + c0, v);
          }
          tc05::wait_st();
          release_acc<CG>(&B.acc_empty[0]);
        }
        if (!fine) break;
      }
      const bool rows4 = P.wide && nbase + rows <= P.n;
      Outputs<FORM == kWeights ? 4 : 2> O;  // the first piece's residuals, and later the next one's
      if (FORM == kWeights && T.mt < P.nmt && 16 * grp < T.nlen) O.fetch(P, T.n0 + 16 * grp, min(16, T.nlen - 16 * grp), nbase, q, 4, rows4);
      // the warps stop together (they share named barriers)
      // (one waits for the MMAs, the others for it)
      fine = tc05::named_and(5, 32 * kEpi, res_ok && (warp != 0 || tc_warp_wait<CL>(&B.acc_full[b], (uint32_t)(use & 1), P)));
      if (!fine) break;
      tc05::fence_after();
      const uint32_t tl = tmem + (uint32_t)(b * 256) + ((uint32_t)(32 * q) << 16);
      auto read = [&](int at, float (&x)[16]) { read_sums(tl + at, LONG ? parts > 1 : !SPLIT && P.two, x); };
      const int o = nbase + (P.gated ? row & 63 : row);
      const int brow = P.gated && row >= 64 ? P.n + o : o;
      auto release = [&] { release_acc<CG>(&B.acc_empty[b]); };
      if constexpr (TOK) {
        // a lane has a token, and its columns one after another: no exchange
        // (through shared memory, which copies and MMAs keep busy, the
        // product with silu took 208 us at 8192 x 8192 x 2048)
        const int r = T.mt * 128 + row;
        const bool live = r < P.t;
        const float rs = live && P.row_scale ? P.row_scale[r] : 1.f;
        const int end = min(cols, P.n - T.n0), last = (end + 15) / 16;
        const int pieces = P.res ? (P.res_bf16 ? (end + 63) / 64 : (end + 31) / 32) : 0;
        if (grp >= last) release();
#pragma unroll 1
        for (int i = 0; i < 4; i++) {
          const int c0 = 16 * (grp + 4 * i), col = T.n0 + c0, n = min(16, P.n - col);
          const bool here = c0 < end;
          // the residuals' pieces in turn, those of other groups too: a warp
          // that skips a phase of a barrier cannot tell the next from the one
          // before the last
          uint32_t res[16];
          for (int p = P.res_bf16 ? i : 2 * i; p < pieces && p <= (P.res_bf16 ? i : 2 * i + 1); p++) {
            const int s = res_at + p, rb = s % kResBufs;
            if (res_ok) res_ok = tc_warp_wait<false>(&B.res_full[rb], (uint32_t)((s / kResBufs) & 1), P);
            if (here && (P.res_bf16 || p == 2 * i + (grp >> 1))) {
              const uint8_t *line = sm + rb * kResPiece + row * 128;
              const int first = P.res_bf16 ? 2 * grp : 4 * (grp & 1);  // 16-byte chunk, at its place ^ (row & 7)
#pragma unroll
              for (int j = 0; j < 4; j++)
                if (j < 2 || !P.res_bf16) {
                  const uint4 x = *reinterpret_cast<const uint4 *>(line + (((first + j) ^ (row & 7)) << 4));
                  res[4 * j] = x.x, res[4 * j + 1] = x.y, res[4 * j + 2] = x.z, res[4 * j + 3] = x.w;
                }
            }
            __syncwarp();
            if (lane == 0) tc05::mbar_arrive(&B.res_empty[rb]);
          }
          float v[16], u[16], bias[16];
          if (P.bias && here) load_bias(bias, P.bias + col, n);
          if (here) {
            read(c0, v);
            if (P.gated) read(cols + c0, u);
            if (grp + 4 * (i + 1) >= last) release();
          }
          if (here && live) {
            if (P.bias) {
#pragma unroll
              for (int j = 0; j < 16; j++) v[j] += bias[j];
              if (P.gated) load_bias(bias, P.bias + P.n + col, n);
            }
            activate_all(v, P.act);
            if (P.gated) {
              if (P.bias) {
#pragma unroll
                for (int j = 0; j < 16; j++) u[j] += bias[j];
              }
#pragma unroll
              for (int j = 0; j < 16; j++) v[j] *= u[j];
            }
#pragma unroll
            for (int j = 0; j < 16; j++) v[j] *= rs;
            if (P.res) {
#pragma unroll
              for (int j = 0; j < 16; j++)
                v[j] += P.res_bf16 ? ((j & 1) ? bf16hi(res[j / 2]) : bf16lo(res[j / 2])) : __uint_as_float(res[j]);
            }
            if (n == 16) {
              uint32_t o[16];
              if (P.out_bf16) {
#pragma unroll
                for (int j = 0; j < 8; j++) o[j] = bf16x2(v[2 * j], v[2 * j + 1]);
                store_run<2>(static_cast<uint16_t *>(P.out) + (int64_t)r * P.ldo + col, o);
              } else {
#pragma unroll
                for (int j = 0; j < 16; j++) o[j] = __float_as_uint(v[j]);
                store_run<4>(static_cast<float *>(P.out) + (int64_t)r * P.ldo + col, o);
              }
            } else {
#pragma unroll
              for (int j = 0; j < 16; j++)
                if (j < n) store1(P, r, col + j, v[j]);
            }
          }
          __syncwarp();
        }
        res_at += pieces;
      } else if constexpr (SPLIT) {
        // all of the accumulator to this CTA's shared memory, [token][128]
        // (the ring: every copy has landed and every MMA has read its operands)
        float *z = reinterpret_cast<float *>(ring);
        for (int c0 = 16 * grp; c0 < w; c0 += 4 * kEpi) {
          float v[16];
          read(c0, v);
#pragma unroll
          for (int j = 0; j < 16; j++) z[(c0 + j) * 128 + row] = v[j];
        }
      } else {
        const int last = (T.mt < P.nmt ? (T.nlen + 15) / 16 : 0);  // pieces with a token
        const float bias = P.bias && o < P.n ? P.bias[brow] : 0.f;
        if (grp >= last) release();
        for (int c = grp; c < last; c += kEpi / 4) {
          const int c0 = 16 * c, n = min(16, T.nlen - c0), c1 = c0 + 4 * kEpi;
          float v[16];
          read(c0, v);
          if (c + kEpi / 4 >= last) release();
#pragma unroll
          for (int j = 0; j < 16; j++) stg[j * 128 + row] = v[j] + bias;
          tc05::named_sync(1 + grp, 128);
          O.write(P, T.n0 + c0, n, nbase, stg, q, 4, rows4);
          if (c1 < T.nlen) O.fetch(P, T.n0 + c1, min(16, T.nlen - c1), nbase, q, 4, rows4);
          tc05::named_sync(1 + grp, 128);  // the piece is free again
        }
      }
    }
    if constexpr (SPLIT) {
      // every CTA's sums are there; this one finishes the tokens rank, rank + split, ...
      tc05::fence_before();
      __syncwarp();
      tc05::cluster_sync();
      if (fine && my_tiles > 0) {
        const int t0 = cl / nmp, m0 = cl - t0 * nmp, nbase = m0 * rows, n0 = t0 * w, nlen = min(w, P.t - n0);
        const bool rows4 = P.wide && nbase + rows <= P.n;
        float bias[4];
#pragma unroll
        for (int e = 0; e < 4; e++) {
          const int x = 4 * lane + e, c = nbase + (P.gated ? x & 63 : x);
          bias[e] = P.bias && c < P.n ? P.bias[P.gated && x >= 64 ? P.n + c : c] : 0.f;
        }
        // four tokens at a time: the CTAs' sums of them, added in the order
        // of k, then as a piece of four of the warp's own
        float *mine = reinterpret_cast<float *>(sm) + warp * 4 * 128;
        for (int j = rank * 4 + P.split * 4 * warp; j < nlen; j += P.split * 4 * kEpi) {
          const int n = min(4, nlen - j);
          Outputs<4> O;
          O.fetch(P, n0 + j, n, nbase, 0, 1, rows4);
          float4 v[4];
#pragma unroll
          for (int i = 0; i < 4; i++) v[i] = make_float4(bias[0], bias[1], bias[2], bias[3]);
#pragma unroll 4
          for (int r = 0; r < P.split; r++) {
            const uint32_t at = tc05::map_rank(ring + (size_t)(j * 128 + 4 * lane) * 4, r);
            float4 u[4];
#pragma unroll
            for (int i = 0; i < 4; i++) u[i] = tc05::ld_cluster4(at + (i < n ? i * 512 : 0));
#pragma unroll
            for (int i = 0; i < 4; i++) v[i].x += u[i].x, v[i].y += u[i].y, v[i].z += u[i].z, v[i].w += u[i].w;
          }
#pragma unroll
          for (int i = 0; i < 4; i++) *reinterpret_cast<float4 *>(mine + i * 128 + 4 * lane) = v[i];
          __syncwarp();
          O.write(P, n0 + j, n, nbase, mine, 0, 1, rows4);
          __syncwarp();
        }
      }
      __syncwarp();
    }
  }
  if constexpr (SPLIT) {
    if (warp >= kEpi) tc05::cluster_sync();  // the first of the two that the epilogue warps wait at
  }

  tc05::fence_before();
  if constexpr (CG == 1 && !SPLIT) __syncthreads();
  else tc05::cluster_sync();
  if (warp == kEpi) {
    if constexpr (CG == 1) tc05::dealloc(tmem, 512);
    else tc05::dealloc_pair(tmem, 512);
  }
}

// rows of k values (bf16 or fp32), ld apart: boxes of 128 bytes x box_rows, 128B swizzle, zeros outside
bool make_map16(CUtensorMap *m, const void *base, uint64_t k, uint64_t rows, uint64_t ld, uint32_t box_rows, bool f32 = false) {
  const cuuint64_t dims[2] = {k, rows}, strides[1] = {ld * (f32 ? 4 : 2)};
  const cuuint32_t box[2] = {f32 ? 32u : 64u, box_rows}, estr[2] = {1, 1};
  return encode_fn()(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base), dims, strides, box, estr,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int CG, int FORM, bool LONG>
cudaError_t launch_form(Mm16P &p, int n_sms, cudaStream_t st) {
  constexpr bool SPLIT = FORM == kSplit;
  const int nrows = p.w / CG;  // rows of the N side that a CTA loads
  p.stage = 16384 + nrows * 128;
  p.stages = kRoom / p.stage < kMaxStages ? kRoom / p.stage : kMaxStages;
  // (a split tile's sums, [w][128] with w up to 128, lie in two of the stages)
  // the most any launch asks for: another host thread's launch of the same
  // kernel may stand between this and the launch below.  Before the tensor
  // maps: it makes the device's context this thread's, which they need
  cudaError_t e = cudaFuncSetAttribute(mm16_tc<CG, FORM, LONG>, cudaFuncAttributeMaxDynamicSharedMemorySize, kOffRing + kRoom + 1024);
  if (e != cudaSuccess) return e;
  const int box_a = FORM == kTokens ? 128 : nrows, box_b = FORM == kTokens ? (p.gated ? p.w / 2 : nrows) : (p.gated ? 64 : 128);
  if (encode_fn() == nullptr || !make_map16(&p.tm_b, p.b, p.k, (uint64_t)p.n * (p.gated ? 2 : 1), p.ldb, (uint32_t)box_b) ||
      !make_map16(&p.tm_a, p.a, p.k, p.t, p.lda, (uint32_t)box_a) ||
      (FORM == kTokens && p.res && !make_map16(&p.tm_r, p.res, p.n, p.t, p.ldr, 128, !p.res_bf16)))
    return cudaErrorNotSupported;
  const int smem = kOffRing + p.stages * p.stage + 1024;
  const int64_t tiles = (int64_t)p.ntt * ((p.nmt + CG - 1) / CG);
  const int cluster = SPLIT ? p.split : CG;
  const int64_t most = n_sms / cluster;
  const int64_t grid = (SPLIT || tiles < most ? tiles : most) * cluster;
  cudaLaunchAttribute at[2];
  int n = 0;
  if (cluster > 1) {
    at[n].id = cudaLaunchAttributeClusterDimension;
    at[n].val.clusterDim.x = (unsigned)cluster, at[n].val.clusterDim.y = 1, at[n].val.clusterDim.z = 1;
    n++;
  }
  at[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[n].val.programmaticStreamSerializationAllowed = 1;
  n++;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kTcThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = (unsigned)n;
  return cudaLaunchKernelEx(&cfg, mm16_tc<CG, FORM, LONG>, p);
}
template <int CG, int FORM>
cudaError_t launch_tc(Mm16P &p, int n_sms, cudaStream_t st) {
  const bool several = !p.two && (p.nk + p.split - 1) / p.split > p.chunk;
  return several ? launch_form<CG, FORM, true>(p, n_sms, st) : launch_form<CG, FORM, false>(p, n_sms, st);
}

}  // namespace

template <int NT>
cudaError_t launch_few(const Mm16Args &p, int n_sms, cudaStream_t st) {
  const int per = p.gated ? 8 : 16, tiles = (p.n + per - 1) / per, blocks = ((p.k + 63) / 64 + kFewWarps - 1) / kFewWarps;
  // as many of a warp's blocks in flight as it has in a tile, four at the
  // most; two (three) thread blocks an SM fit
  const int most = n_sms * (blocks > 2 ? 2 : 3);
  const dim3 grid((unsigned)(tiles < most ? tiles : most));
  auto f = blocks > kSumBlocks ? mm16_few_rows<NT, 4, true> : (blocks > 2 ? mm16_few_rows<NT, 4, false> :
           (blocks > 1 ? mm16_few_rows<NT, 2, false> : mm16_few_rows<NT, 1, false>));
  return launch_pdl(f, grid, 32 * kFewWarps, 0, st, p);
}

bool mm16_few(const Mm16Args &p, int n_sms) {
  const int per = p.gated ? 8 : 16;
  return p.t <= 8 || (p.t <= 16 && (p.n + per - 1) / per <= n_sms);
}

cudaError_t launch_mm16_few(const Mm16Args &p, int n_sms, cudaStream_t st) {
  return p.t <= 8 ? launch_few<1>(p, n_sms, st) : launch_few<2>(p, n_sms, st);
}

cudaError_t launch_mm16_tc(Mm16P p, int n_sms, cudaStream_t st) {
  const int rows = p.gated ? 64 : 128;
  p.nmt = (p.n + rows - 1) / rows, p.nk = (p.k + 63) / 64;
  p.chunk = p.out_bf16 ? kSumBlocksBf16 : kSumBlocks;
  // Too few tiles for the SMs: k is split over a cluster.  Clusters of 4 and 8
  // CTAs of this size do not fill every SM (36 and 15 fit at once).  Then as
  // narrow tiles as still fit: less to add up and to write for each CTA (128 x
  // 512 x 2048: 10.7 -> 8.7 us, 333 x 1001 x 2008 14.2 -> 13.4).
  {
    int w = p.t <= 128 ? (p.t + 15) / 16 * 16 : 128, s = 1;
    auto tiles = [&](int width) { return (int64_t)((p.t + width - 1) / width) * p.nmt; };
    int64_t most = 0;
    auto may = [&](int split, int64_t fit) {
      if (p.nk >= 2 * split && tiles(w) <= fit) s = split, most = fit;
    };
    may(2, n_sms / 2), may(4, n_sms / 4 - 2), may(8, n_sms / 8 - 4);
    while (s > 1 && w > 16 && tiles(w - 16) <= most) w -= 16;
    if (s > 1) {
      p.w = w, p.ntt = (p.t + w - 1) / w, p.split = s;
      return launch_tc<1, kSplit>(p, n_sms, st);
    }
  }
  // fp32 results up to twice as long: the two halves of k in an accumulator each
  p.split = 1;
  p.two = !p.out_bf16 && p.k > 64 * p.chunk && p.nk <= 2 * p.chunk;
  // The tile width with the least (rounds of tiles) x (width + what a tile
  // costs whatever its width), with the weights or the tokens on the M side.
  int64_t best = INT64_MAX;
  bool tokens = false;
  int cg = 1;
  auto look = [&](bool tok, int nmt, int other, int per) {  // other: what the N side holds, per / 2 of a column
    const int c = nmt > 1 ? 2 : 1, nmp = (nmt + c - 1) / c;
    // (a tile's columns are whole pieces of 16: the epilogue writes no fewer)
    const int step = 32 / per > 16 * c ? 32 / per : 16 * c;
    for (int w = 256; w >= 32 * c; w -= step) {
      const int cols = w * per / 2;
      const int64_t rounds = ((int64_t)((other + cols - 1) / cols) * nmp + n_sms / c - 1) / (n_sms / c), cost = rounds * (w + 48);
      if (cost < best) best = cost, p.w = w, tokens = tok, cg = c;
    }
  };
  const int tok_tiles = (p.t + 127) / 128;
  const bool can = p.wide8;
  if (can) look(true, tok_tiles, p.n, p.gated ? 1 : 2);
  look(false, p.nmt, p.t, 2);
  if (tokens) {
    const int cols = p.gated ? p.w / 2 : p.w;
    p.nmt = tok_tiles, p.ntt = (p.n + cols - 1) / cols;
    return cg == 2 ? launch_tc<2, kTokens>(p, n_sms, st) : launch_tc<1, kTokens>(p, n_sms, st);
  }
  p.ntt = (p.t + p.w - 1) / p.w;
  return cg == 2 ? launch_tc<2, kWeights>(p, n_sms, st) : launch_tc<1, kWeights>(p, n_sms, st);
}

}  // namespace moe
