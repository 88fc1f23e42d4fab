// mm16.cu -- bf16 matrix products with what follows them in their epilogue:
//   z = a b^T + bias;  h = act(z), or gated act(z[:, :n]) * z[:, n:]
//   out = row_scale[r] * h + residual
//
// Two kernels:
//   few   up to 32 rows, by mm16_few: the weights are streamed once from HBM
//         straight into the fragments of mma.sync, a CTA takes 16 weight rows
//         and splits k over its warps.
//   tc    any number of rows: tcgen05 (kind::f16, fp32 accumulators in TMEM)
//         fed by TMA.  Weights on the M side, tokens on the N side, as the
//         8-bit products have them: M stays full whatever the number of rows.
//         Persistent over CTA pairs (256 weight rows x up to 256 tokens), or,
//         where there are too few tiles for the SMs, a cluster of S CTAs a
//         tile that split k and add their accumulators in a fixed order.
#include <cuda_runtime.h>

#include <type_traits>

#include "block.cuh"
#include "fp8.cuh"
#include "tc05.cuh"

namespace moe {
namespace {

constexpr unsigned FULLM = 0xffffffffu;

// 1 / (1 + exp(-x)), small values to their last bits
__device__ __forceinline__ float logistic(float x) {
  const float e = expf(-fabsf(x));
  return (x < 0.f ? e : 1.f) / (1.f + e);
}
__device__ __forceinline__ float activate(float z, int act) {
  switch (act) {
    case kActSilu: return z * logistic(z);
    case kActGelu: return 0.5f * z * erfcf(z * -0.70710678118654752f);
    case kActGeluTanh:  // (1 + tanh u) / 2 = 1 / (1 + exp(-2 u))
      return z * logistic(z * fmaf(z * z, 0.07135481627f, 1.5957691216f));
    case kActRelu: return z < 0.f ? 0.f : z;  // NaN stays
    case kActSigmoid: return logistic(z);
    default: return z;
  }
}

__device__ __forceinline__ uint16_t bf16_of(float v) {
  uint16_t h;
  asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(h) : "f"(v));
  return h;
}
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// One output: row r, column j, from h = the activated product.
__device__ __forceinline__ void finish1(const Mm16Args &P, int64_t r, int j, float h, float rs) {
  h *= rs;
  if (P.res) {
    const int64_t i = r * P.ldr + j;
    h += P.res_bf16 ? __uint_as_float((uint32_t)static_cast<const uint16_t *>(P.res)[i] << 16)
                    : static_cast<const float *>(P.res)[i];
  }
  const int64_t o = r * P.ldo + j;
  if (P.out_bf16) static_cast<uint16_t *>(P.out)[o] = bf16_of(h);
  else static_cast<float *>(P.out)[o] = h;
}
// Four neighbouring ones, in rows that allow whole accesses (P.wide).
__device__ __forceinline__ void finish4(const Mm16Args &P, int64_t r, int j, float4 h, float rs) {
  h.x *= rs, h.y *= rs, h.z *= rs, h.w *= rs;
  if (P.res) {
    const int64_t i = r * P.ldr + j;
    if (P.res_bf16) {
      const uint2 u = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(P.res) + i);
      h.x += bf16lo(u.x), h.y += bf16hi(u.x), h.z += bf16lo(u.y), h.w += bf16hi(u.y);
    } else {
      const float4 u = *reinterpret_cast<const float4 *>(static_cast<const float *>(P.res) + i);
      h.x += u.x, h.y += u.y, h.z += u.z, h.w += u.w;
    }
  }
  const int64_t o = r * P.ldo + j;
  if (P.out_bf16)
    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(P.out) + o) = make_uint2(bf16x2(h.x, h.y), bf16x2(h.z, h.w));
  else
    *reinterpret_cast<float4 *>(static_cast<float *>(P.out) + o) = h;
}

// ------------------------------------------------------------ few rows

constexpr int kFewWarps = 8;
constexpr int kFewDepth = 4;  // blocks of 64 k whose weights a warp has in flight

// One CTA: 16 weight rows (gated: 8 gate rows and the 8 up rows of the same
// outputs), 8 * NT token rows.  Lane (g, q) = (lane / 4, lane % 4) loads 16
// bytes of weight rows g and g + 8 at k = 8q and 32 + 8q of a block: the four
// words of a piece serve as the k halves of two MMAs, and the same pieces of
// the token rows as B, so the order of k is permuted alike on both sides.
// Warp w takes the blocks w, w + 8, ...; the warps' sums meet in shared
// memory in a fixed order.
template <int NT>
__global__ void __launch_bounds__(32 * kFewWarps) mm16_few_rows(const __grid_constant__ Mm16Args P) {
  __shared__ float red[kFewWarps][16][8 * NT + 1];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q = lane & 3;
  pdl_wait_prev();
  pdl_launch_next();
  if (blockIdx.x == 0 && tid == 0) *P.status = 0;
  const int per = P.gated ? 8 : 16, n0 = blockIdx.x * per, nb = (P.k + 63) / 64;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  const int r0 = n0 + g, r1 = P.gated ? P.n + n0 + g : n0 + g + 8;
  const bool ok0 = r0 < P.n, ok1 = P.gated ? ok0 : r1 < P.n;
  const uint16_t *w0 = P.b + (int64_t)r0 * P.ldb, *w1 = P.b + (int64_t)r1 * P.ldb;
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
  float acc[NT][4];
#pragma unroll
  for (int j = 0; j < NT; j++)
#pragma unroll
    for (int i = 0; i < 4; i++) acc[j][i] = 0.f;
  uint4 a[kFewDepth][2][2];  // [block][piece][row]
  auto load = [&](uint4 (&x)[2][2], int kb) {
    const int k0 = kb * 64 + q * 8;
#pragma unroll
    for (int p = 0; p < 2; p++) x[p][0] = piece(w0, k0 + 32 * p, ok0, true), x[p][1] = piece(w1, k0 + 32 * p, ok1, true);
  };
  auto step = [&](const uint4 (&x)[2][2], int kb) {
    const int k0 = kb * 64 + q * 8;
#pragma unroll
    for (int j = 0; j < NT; j++) {
      const int r = 8 * j + g;
      const uint16_t *xr = P.a + (int64_t)r * P.lda;
#pragma unroll
      for (int p = 0; p < 2; p++) {
        const uint4 b = piece(xr, k0 + 32 * p, r < P.t, false);
        mma_bf16_16816(acc[j], x[p][0].x, x[p][1].x, x[p][0].y, x[p][1].y, b.x, b.y);
        mma_bf16_16816(acc[j], x[p][0].z, x[p][1].z, x[p][0].w, x[p][1].w, b.z, b.w);
      }
    }
  };
#pragma unroll
  for (int i = 0; i < kFewDepth; i++) load(a[i], warp + i * kFewWarps);
  for (int kb = warp; kb < nb; kb += kFewDepth * kFewWarps) {
#pragma unroll
    for (int i = 0; i < kFewDepth; i++) {
      const int k1 = kb + i * kFewWarps;
      if (k1 < nb) {
        step(a[i], k1);
        load(a[i], k1 + kFewDepth * kFewWarps);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < NT; j++) {
    const int c = 8 * j + 2 * q;
    red[warp][g][c] = acc[j][0], red[warp][g][c + 1] = acc[j][1];
    red[warp][g + 8][c] = acc[j][2], red[warp][g + 8][c + 1] = acc[j][3];
  }
  __syncthreads();
  auto sum = [&](int row, int c) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kFewWarps; w++) v += red[w][row][c];
    return v;
  };
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

// ------------------------------------------------------------ tensor cores
//
//   warps 0-7 epilogue, four for the even and four for the odd pieces of 32
//             tokens: TMEM -> registers -> shared memory [token][128 rows] ->
//             whole runs of a token's outputs, from one of two accumulators
//             while the MMAs fill the other
//   warp 8    (even CTA) issues a stage's MMAs once its operands are there
//   warp 9    TMA: 128 weight rows x 64 k a stage, the CTA's share of the tokens
// gated: a tile's 128 weight rows are 64 gate rows and the 64 up rows of the
// same outputs, so that both meet in the piece in shared memory.
// The full and acc_empty barriers of a pair are the even CTA's; the others are
// each CTA's own, committed to both.
constexpr int kTcThreads = 320;
constexpr int kMaxStages = 10;
constexpr int kPiece = 32 * 128 * 4;  // bytes of 32 tokens x 128 rows

struct Bars {
  uint64_t full[kMaxStages], empty[kMaxStages], acc_full[2], acc_empty[2], drain;
  uint32_t tmem;
};
constexpr int kOffBars = 2 * kPiece;
constexpr int kOffRing = (kOffBars + (int)sizeof(Bars) + 1023) / 1024 * 1024;
constexpr int kRoom = 226 * 1024 - kOffRing;

template <bool CL>
__device__ bool tc_wait(uint64_t *bar, uint32_t par, const Mm16Args &P) {
  auto done = [&] { return CL ? tc05::mbar_try_wait_cluster(bar, par) : mbar_try_wait(bar, par); };
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

// Warp: the outputs of one token of a tile (row r of out) from its 128 values
// z, which get(i) reads for i % 4 == 0 four at a time, get1(i) one.  Gated:
// 64 outputs, from values i and 64 + i.
template <class G4, class G1>
__device__ __forceinline__ void token_out(const Mm16Args &P, int64_t r, int nbase, G4 get4, G1 get1) {
  const int lane = threadIdx.x & 31;
  const float rs = P.row_scale ? P.row_scale[r] : 1.f;
  if (!P.gated) {
    if (P.wide && nbase + 128 <= P.n) {
      float4 z = get4(4 * lane);
      z.x = activate(z.x, P.act), z.y = activate(z.y, P.act), z.z = activate(z.z, P.act), z.w = activate(z.w, P.act);
      finish4(P, r, nbase + 4 * lane, z, rs);
    } else {
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const int j = lane + 32 * i;
        if (nbase + j < P.n) finish1(P, r, nbase + j, activate(get1(j), P.act), rs);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2; i++) {
      const int j = lane + 32 * i;
      if (nbase + j < P.n) finish1(P, r, nbase + j, activate(get1(j), P.act) * get1(64 + j), rs);
    }
  }
}

template <int CG, bool SPLIT>
__global__ void __launch_bounds__(kTcThreads, 1) mm16_tc(const __grid_constant__ Mm16P P) {
  static_assert(!SPLIT || CG == 1, "a split tile is one CTA's rows");
  constexpr bool CL = CG == 2;
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
    for (int b = 0; b < 2; b++) mbar_init(&B.acc_full[b], 1), mbar_init(&B.acc_empty[b], 8 * CG);
    mbar_init(&B.drain, 1);
    fence_mbar_init();
  }
  if (warp == 8) {
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
  const int rows = P.gated ? 64 : 128;         // outputs of a CTA's tile
  const int nmp = (P.nmt + CG - 1) / CG;       // weight tiles, CG at a time
  const int ntiles = P.ntt * nmp;
  const int width = CG == 2 ? 2 : (SPLIT ? P.split : 1);  // CTAs of a tile
  const int cl = (int)blockIdx.x / width, ncl = (int)gridDim.x / width;
  const int my_tiles = cl < ntiles ? (ntiles - 1 - cl) / ncl + 1 : 0;
  int kb0 = 0, kb1 = P.nk;
  if constexpr (SPLIT) kb0 = (int)((int64_t)P.nk * rank / P.split), kb1 = (int)((int64_t)P.nk * (rank + 1) / P.split);
  // tile i: the weight tiles of a token tile follow one another
  int tt = cl / nmp, mp = cl - tt * nmp;
  const int step_t = ncl / nmp, step_m = ncl - step_t * nmp;
  struct Tile {
    int mt, n0, nlen;
  };
  auto next_tile = [&] {
    Tile T;
    T.mt = mp * CG + mrank;
    T.n0 = tt * w;
    T.nlen = min(w, P.t - T.n0);
    tt += step_t, mp += step_m;
    if (mp >= nmp) mp -= nmp, tt++;
    return T;
  };

  if (warp == 8) {
    // ---------------------------------------------------------------- MMA issue
    if (mrank == 0 && tc05::elect_one()) {
      int s = 0;
      uint32_t ph = 0;
      bool ok = true;
      const uint32_t base = smem_u32(ring), idesc = tc05::idesc_f16(128 * CG, w);
      for (int lt = 0; lt < my_tiles && ok; lt++) {
        const int b = lt & 1;
        if (!tc_wait<CL>(&B.acc_empty[b], (uint32_t)(((lt >> 1) & 1) ^ 1), P)) break;
        tc05::fence_after();
        const uint32_t d = tmem + (uint32_t)(b * 256);
        for (int kb = kb0; kb < kb1; kb++) {
          if (!tc_wait<CL>(&B.full[s], ph, P)) {
            ok = false;
            break;
          }
          tc05::fence_after();
          const uint32_t st = base + (uint32_t)(s * P.stage);
          const uint64_t ad = tc05::sdesc(st), bd = tc05::sdesc(st + 16384);
#pragma unroll
          for (int j = 0; j < 4; j++) tc05::mma_f16<CG>(d, ad + 2 * j, bd + 2 * j, idesc, kb != kb0 || j != 0);
          if constexpr (CG == 1) tc05::commit(&B.empty[s]);
          else tc05::commit_pair(&B.empty[s]);
          if (++s == S) s = 0, ph ^= 1;
        }
        if (ok) {
          if constexpr (CG == 1) tc05::commit(&B.acc_full[b]);
          else tc05::commit_pair(&B.acc_full[b]);
        }
      }
      // every MMA issued here has completed before TMEM is released
      if constexpr (CG == 1) tc05::commit(&B.drain);
      else tc05::commit_pair(&B.drain);
      tc_wait<CL>(&B.drain, 0, P);
    }
    __syncwarp();
  } else if (warp == 9) {
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
          tc05::tma_load_xy<CG>(st, &P.tm_b, kb * 64, wr, bar);
          if (P.gated) tc05::tma_load_xy<CG>(st + 8192, &P.tm_b, kb * 64, P.n + wr, bar);
          tc05::tma_load_xy<CG>(st + 16384, &P.tm_a, kb * 64, T.n0 + mrank * tok, bar);
        }
        __syncwarp();
        if (++s == S) s = 0, ph ^= 1;
      }
    }
    // copies still in flight land before the CTA (the pair) ends
    if (lane == 0 && mrank == 0)
      for (int g = f > S ? f - S : 0; g < f; g++) tc_wait<CL>(&B.full[g % S], (uint32_t)((g / S) & 1), P);
    __syncwarp();
  } else {
    // ---------------------------------------------------------------- epilogue
    const int q = warp & 3, grp = warp >> 2;  // TMEM lane quadrant; even or odd pieces
    const int row = 32 * q + lane;            // the tile's weight row of this thread
    float *stg = reinterpret_cast<float *>(sm + grp * kPiece);
    bool fine = true;
    for (int lt = 0; lt < my_tiles; lt++) {
      const Tile T = next_tile();
      const int b = lt & 1;
      // the warps stop together (they share named barriers)
      fine = tc05::named_and(3, 256, tc_warp_wait<CL>(&B.acc_full[b], (uint32_t)((lt >> 1) & 1), P));
      if (!fine) break;
      tc05::fence_after();
      const uint32_t tl = tmem + (uint32_t)(b * 256) + ((uint32_t)(32 * q) << 16);
      const int nbase = T.mt * rows, o = nbase + (P.gated ? row & 63 : row);
      const int brow = P.gated && row >= 64 ? P.n + o : o;
      if constexpr (SPLIT) {
        // all of the accumulator to this CTA's shared memory, [token][128]
        // (the ring: every copy has landed and every MMA has read its operands)
        float *z = reinterpret_cast<float *>(ring);
        for (int c0 = 32 * grp; c0 < w; c0 += 64) {
          float v[32];
          const bool whole = c0 + 32 <= w;
          if (whole) tc05::ld32(tl + c0, v);
          else tc05::ld16(tl + c0, v);
#pragma unroll
          for (int j = 0; j < 32; j++)
            if (whole || j < 16) z[(c0 + j) * 128 + row] = v[j];
        }
      } else {
        auto release = [&] {  // the accumulator is read: the MMAs may fill it again
          tc05::fence_before();
          __syncwarp();
          if (lane == 0) {
            if constexpr (CG == 1) tc05::mbar_arrive(&B.acc_empty[b]);
            else tc05::mbar_arrive_cluster(tc05::map_rank(&B.acc_empty[b], 0));
          }
        };
        const int last = (T.mt < P.nmt ? (T.nlen + 31) / 32 : 0);  // pieces with a token
        const float bias = P.bias && o < P.n ? P.bias[brow] : 0.f;
        if (grp >= last) release();
        for (int c = grp; c < last; c += 2) {
          float v[32];
          const int c0 = 32 * c;
          const bool whole = c0 + 32 <= w;
          if (whole) tc05::ld32(tl + c0, v);
          else tc05::ld16(tl + c0, v);
          if (c + 2 >= last) release();
#pragma unroll
          for (int j = 0; j < 32; j++)
            if (whole || j < 16) stg[j * 128 + row] = v[j] + bias;
          tc05::named_sync(1 + grp, 128);
#pragma unroll 1
          for (int i = 0; i < 8; i++) {
            const int j = 4 * i + q;
            if (c0 + j < T.nlen) {
              const float *z = stg + j * 128;
              token_out(P, T.n0 + c0 + j, nbase, [&](int x) { return *reinterpret_cast<const float4 *>(z + x); },
                        [&](int x) { return z[x]; });
            }
          }
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
        for (int j = rank + P.split * warp; j < nlen; j += P.split * 8) {
          auto bias_at = [&](int x) {
            const int c = nbase + (P.gated ? x & 63 : x);
            return P.bias && c < P.n ? P.bias[P.gated && x >= 64 ? P.n + c : c] : 0.f;
          };
          auto get4 = [&](int x) {
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int r = 0; r < P.split; r++) {
              const float4 u = tc05::ld_cluster4(tc05::map_rank(ring + (size_t)(j * 128 + x) * 4, r));
              v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
            }
            v.x += bias_at(x), v.y += bias_at(x + 1), v.z += bias_at(x + 2), v.w += bias_at(x + 3);
            return v;
          };
          auto get1 = [&](int x) {
            float v = 0.f;
            for (int r = 0; r < P.split; r++) v += tc05::ld_cluster(tc05::map_rank(ring + (size_t)(j * 128 + x) * 4, r));
            return v + bias_at(x);
          };
          token_out(P, n0 + j, nbase, get4, get1);
        }
      }
      __syncwarp();
    }
  }
  if constexpr (SPLIT) {
    if (warp >= 8) tc05::cluster_sync();  // the first of the two that the epilogue warps wait at
  }

  tc05::fence_before();
  if constexpr (CG == 1 && !SPLIT) __syncthreads();
  else tc05::cluster_sync();
  if (warp == 8) {
    if constexpr (CG == 1) tc05::dealloc(tmem, 512);
    else tc05::dealloc_pair(tmem, 512);
  }
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = [] {
    void *f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return (EncodeTiledFn) nullptr;
    return reinterpret_cast<EncodeTiledFn>(f);
  }();
  return fn;
}

// bf16 rows of k values, ld apart: boxes of 64 values x box_rows, 128B swizzle, zeros outside
bool make_map16(CUtensorMap *m, const void *base, uint64_t k, uint64_t rows, uint64_t ld, uint32_t box_rows) {
  const cuuint64_t dims[2] = {k, rows}, strides[1] = {ld * 2};
  const cuuint32_t box[2] = {64, box_rows}, estr[2] = {1, 1};
  return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base), dims, strides, box, estr,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int CG, bool SPLIT>
cudaError_t launch_tc(Mm16P &p, int n_sms, cudaStream_t st) {
  const int tok = p.w / CG;
  p.stage = 16384 + tok * 128;
  p.stages = kRoom / p.stage < kMaxStages ? kRoom / p.stage : kMaxStages;
  // the most any launch asks for: another host thread's launch of the same
  // kernel may stand between this and the launch below.  Before the tensor
  // maps: it makes the device's context this thread's, which they need
  cudaError_t e = cudaFuncSetAttribute(mm16_tc<CG, SPLIT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kOffRing + kRoom + 1024);
  if (e != cudaSuccess) return e;
  if (encode_fn() == nullptr ||
      !make_map16(&p.tm_b, p.b, p.k, (uint64_t)p.n * (p.gated ? 2 : 1), p.ldb, p.gated ? 64 : 128) ||
      !make_map16(&p.tm_a, p.a, p.k, p.t, p.lda, (uint32_t)tok))
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
  return cudaLaunchKernelEx(&cfg, mm16_tc<CG, SPLIT>, p);
}

}  // namespace

cudaError_t launch_mm16_few(const Mm16Args &p, cudaStream_t st) {
  const int per = p.gated ? 8 : 16, nt = (p.t + 7) / 8;
  auto f = nt <= 1 ? mm16_few_rows<1> : (nt <= 2 ? mm16_few_rows<2> : mm16_few_rows<4>);
  return launch_pdl(f, dim3((unsigned)((p.n + per - 1) / per)), 32 * kFewWarps, 0, st, p);
}

cudaError_t launch_mm16_tc(Mm16P p, int n_sms, cudaStream_t st) {
  const int rows = p.gated ? 64 : 128;
  p.nmt = (p.n + rows - 1) / rows, p.nk = (p.k + 63) / 64;
  // too few tiles for the SMs: k is split over a cluster
  {
    const int w = p.t <= 128 ? (p.t + 15) / 16 * 16 : 128;
    const int64_t tiles = (int64_t)((p.t + w - 1) / w) * p.nmt;
    int s = 1;
    while (s < 8 && tiles * s * 2 <= n_sms && p.nk / (s * 2) >= 2) s *= 2;
    if (s > 1) {
      p.w = w, p.ntt = (p.t + w - 1) / w, p.split = s;
      return launch_tc<1, true>(p, n_sms, st);
    }
  }
  const int cg = p.nmt > 1 ? 2 : 1, nmp = (p.nmt + cg - 1) / cg;
  // the tile width with the least (rounds of tiles) x (width + what a tile
  // costs whatever its width)
  int64_t best = INT64_MAX;
  for (int w = 256; w >= 16 * cg; w -= 16 * cg) {
    const int64_t rounds = ((int64_t)(p.t + w - 1) / w * nmp + n_sms / cg - 1) / (n_sms / cg), cost = rounds * (w + 48);
    if (cost < best) best = cost, p.w = w;
  }
  p.ntt = (p.t + p.w - 1) / p.w;
  return cg == 2 ? launch_tc<2, false>(p, n_sms, st) : launch_tc<1, false>(p, n_sms, st);
}

}  // namespace moe
