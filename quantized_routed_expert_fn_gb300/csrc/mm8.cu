// mm8.cu -- block-scaled 8-bit matrix products: out[r][j] = sum over blocks
// kb of 128 k of 2^(sa[r][kb] + sb[j / 128][kb] - 254) * (a[r] . b[j] in kb).
//
// Two kernels:
//   small  up to kMm8SmallRows rows: the weights are streamed once from HBM
//          straight into the fragments of mma.sync (no shared memory), the
//          few rows come from L1; a CTA takes 16 weight rows and splits k
//          over its warps.
//   tc     any number of rows, dense or grouped: persistent, warp
//          specialised, tcgen05 with the tensor cores' own block scaling
//          (kind::mxf8f6f4), accumulating all of k in TMEM.
#include <cuda_runtime.h>

#include <type_traits>

#include "fp8.cuh"
#include "tc05.cuh"

namespace moe {
namespace {

constexpr unsigned FULLM = 0xffffffffu;

__device__ __forceinline__ void pdl_launch_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void pdl_wait_prev() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <class T>
__device__ __forceinline__ void store_out(T *p, float v);
template <>
__device__ __forceinline__ void store_out<float>(float *p, float v) {
  *p = v;
}
template <>
__device__ __forceinline__ void store_out<uint16_t>(uint16_t *p, float v) {
  uint16_t h;
  asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(h) : "f"(v));
  *p = h;
}

// ------------------------------------------------------------ few rows

__device__ __forceinline__ void mma_e4m3(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

constexpr int kSmWarps = 8;

// One CTA: 16 weight rows, 8 * NT token columns.  Lane (g, q) = (lane / 4,
// lane % 4) loads 16 consecutive bytes of rows g and g + 8 at k = 16q and
// 64 + 16q of a block; the four words of a 16-byte piece serve as the k
// quarters of two MMAs.  The same pieces of the token rows serve as B, so
// the order of k inside a block is permuted alike on both sides.  Warp w
// takes the blocks w, w + 8, ...; the warps' sums meet in shared memory, in
// a fixed order.
template <int NT, class T>
__global__ void __launch_bounds__(32 * kSmWarps) mm8_small(const __grid_constant__ Mm8P P) {
  __shared__ float red[kSmWarps][16][8 * NT + 1];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q = lane & 3;
  if (blockIdx.x == 0 && tid == 0) *P.status = 0;
  const int n0 = blockIdx.x * 16;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  const uint8_t *w0 = P.b + (size_t)(n0 + g) * P.k, *w1 = w0 + (size_t)8 * P.k;
  const bool ok0 = n0 + g < P.n, ok1 = n0 + g + 8 < P.n;
  const uint8_t *sb = P.sb + (size_t)(n0 >> 7) * P.nk;
  float acc[NT][4];
#pragma unroll
  for (int j = 0; j < NT; j++)
#pragma unroll
    for (int i = 0; i < 4; i++) acc[j][i] = 0.f;
  for (int kb = warp; kb < P.nk; kb += kSmWarps) {
    const int k0 = kb * 128 + q * 16, k1 = k0 + 64;
    uint4 a[2][2];  // [piece][row g, g + 8]
    a[0][0] = ok0 && k0 < P.k ? ldg_stream4(w0 + k0) : zero;
    a[0][1] = ok1 && k0 < P.k ? ldg_stream4(w1 + k0) : zero;
    a[1][0] = ok0 && k1 < P.k ? ldg_stream4(w0 + k1) : zero;
    a[1][1] = ok1 && k1 < P.k ? ldg_stream4(w1 + k1) : zero;
    const float fb = e8m0_f(sb[kb]);
#pragma unroll
    for (int j = 0; j < NT; j++) {
      const int r = 8 * j + g;
      const uint8_t *x = P.a + (size_t)r * P.lda;
      const uint4 b0 = r < P.t && k0 < P.k ? *reinterpret_cast<const uint4 *>(x + k0) : zero;
      const uint4 b1 = r < P.t && k1 < P.k ? *reinterpret_cast<const uint4 *>(x + k1) : zero;
      float d[4] = {0.f, 0.f, 0.f, 0.f};
      mma_e4m3(d, a[0][0].x, a[0][1].x, a[0][0].y, a[0][1].y, b0.x, b0.y);
      mma_e4m3(d, a[0][0].z, a[0][1].z, a[0][0].w, a[0][1].w, b0.z, b0.w);
      mma_e4m3(d, a[1][0].x, a[1][1].x, a[1][0].y, a[1][1].y, b1.x, b1.y);
      mma_e4m3(d, a[1][0].z, a[1][1].z, a[1][0].w, a[1][1].w, b1.z, b1.w);
      const int c = 8 * j + 2 * q;
      const float s0 = c < P.t ? e8m0_f(P.sa[(size_t)c * P.lds + kb]) : 0.f;
      const float s1 = c + 1 < P.t ? e8m0_f(P.sa[(size_t)(c + 1) * P.lds + kb]) : 0.f;
      acc[j][0] += d[0] * s0 * fb;
      acc[j][1] += d[1] * s1 * fb;
      acc[j][2] += d[2] * s0 * fb;
      acc[j][3] += d[3] * s1 * fb;
    }
  }
#pragma unroll
  for (int j = 0; j < NT; j++) {
    const int c = 8 * j + 2 * q;
    red[warp][g][c] = acc[j][0], red[warp][g][c + 1] = acc[j][1];
    red[warp][g + 8][c] = acc[j][2], red[warp][g + 8][c + 1] = acc[j][3];
  }
  __syncthreads();
  for (int i = tid; i < 16 * 8 * NT; i += 32 * kSmWarps) {
    const int row = i & 15, c = i >> 4;
    if (c < P.t && n0 + row < P.n) {
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kSmWarps; w++) v += red[w][row][c];
      store_out(static_cast<T *>(P.out) + (size_t)c * P.ldo + n0 + row, v);
    }
  }
}

// ------------------------------------------------------------ tensor cores
//
// One CTA per SM walks the tiles blockIdx.x, + gridDim.x, ...  A tile is
// MB blocks of 128 weight rows (the M side: one TMEM lane a weight row) by
// up to kTcN / MB token rows of one group (the N side).  Weights on the M
// side keep M full whatever the group's size; N follows it in steps of 16.
// MB = 2 (silu): 128 gate rows and the 128 up rows of the same channels
// share the token tile, and the epilogue has a whole 128-channel scale block
// of h in its four warps.
//   warp 0    issues the scale copies and MMAs of a stage, commits them
//   warp 1    TMA: 128 weight rows x 128 k a block, the tile's token rows
//   warp 2    scale words of the token rows -> shared memory
//   warp 3    scale words of the weight blocks -> shared memory
//   warps 4-7 epilogue: TMEM -> registers -> global, from one of two
//             accumulators while the MMAs fill the other
// A stage is one k block: 16 KB of weights per M block, up to 28 KB (14 KB)
// of tokens, their scale words.  Its scale copies go to TMEM columns of the
// stage's own, so a copy never overwrites scales an MMA in flight reads
// (the stage's barriers order both).
constexpr int kTcThreads = 256;
constexpr int kTcStages = 4;
constexpr int kTcN = 224;              // accumulator columns of a buffer: two buffers and the scales fill 512
constexpr int kTcScaleCol = 2 * kTcN;  // first scale column; 16 a stage
static_assert(kTcScaleCol + 16 * kTcStages <= 512, "tensor memory");
constexpr int kMaxGroups = 1024;

struct TcBars {
  uint64_t full[kTcStages], empty[kTcStages], acc_full[2], acc_empty[2], drain;
  uint32_t tmem;
  int bad;
};

template <int MB>
struct TcLay {
  static constexpr int N = kTcN / MB;                         // token columns of a tile
  static constexpr int tok = (N + 31) / 32 * 4096;            // bytes of tokens a stage: whole 32-row boxes
  static constexpr int offW = tok;                            // weights: MB x 16 KB
  static constexpr int offS = offW + MB * 16384;              // scale words: tokens 2 x 512, weights MB x 512
  static constexpr int stage = offS + 2048;
  static constexpr int offEpi = kTcStages * stage;            // silu: h bytes [N][128], maxima [4][N]
  static constexpr int epi = MB == 2 ? N * 128 + 4 * N * 4 + N * 4 : 0;
  static constexpr int offTab = (offEpi + epi + 15) & ~15;    // int [G + 1] first row, [G + 1] first token tile
  static constexpr int offBars = offTab + (2 * (kMaxGroups + 1) + 2) * 4 + 8;
  static constexpr int smem = ((offBars + 7) & ~7) + (int)sizeof(TcBars) + 1024;
  static_assert(tok % 1024 == 0 && stage % 1024 == 0, "swizzled stages");
  static_assert(smem <= 227 * 1024, "shared memory");
};

struct Tile {
  int g, mt, n0, nlen, N;
};

__device__ bool tc_wait(uint64_t *bar, uint32_t par, const Mm8P &P) {
  if (mbar_try_wait(bar, par)) return true;
  const uint64_t t0 = globaltimer();
  while (!mbar_try_wait(bar, par)) {
    if (globaltimer() - t0 > P.timeout_ns) {
      atomicCAS(P.status, 0, kStatusTimeout);
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ bool tc_warp_wait(uint64_t *bar, uint32_t par, const Mm8P &P) {
  bool ok = true;
  if ((threadIdx.x & 31) == 0) ok = tc_wait(bar, par, P);
  return __shfl_sync(FULLM, ok ? 1 : 0, 0) != 0;
}

template <int MB, int KIND>
__global__ void __launch_bounds__(kTcThreads, 1) mm8_tc(const __grid_constant__ Mm8P P) {
  pdl_launch_next();
  extern __shared__ __align__(1024) uint8_t smraw[];
  uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smraw) + 1023) & ~(uintptr_t)1023);
  using LY = TcLay<MB>;
  TcBars &B = *reinterpret_cast<TcBars *>(sm + ((LY::offBars + 7) & ~7));
  int *s_off = reinterpret_cast<int *>(sm + LY::offTab), *s_tile = s_off + kMaxGroups + 1;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = P.G > 0 ? P.G : 1, nk = P.nk;
  const int nmt = MB == 2 ? P.n / 256 : P.nb;  // weight tiles a group

  if (tid == 0) {
    for (int s = 0; s < kTcStages; s++) {
      mbar_init(&B.full[s], 3);
      mbar_init(&B.empty[s], 1);
    }
    for (int b = 0; b < 2; b++) {
      mbar_init(&B.acc_full[b], 1);
      mbar_init(&B.acc_empty[b], 4);
    }
    mbar_init(&B.drain, 1);
    fence_mbar_init();
    B.bad = 0;
  }
  if (warp == 0) tc05::alloc(&B.tmem, 512);
  pdl_wait_prev();  // the offsets and the operands may be the previous kernel's
  tc05::fence_before();
  __syncthreads();
  tc05::fence_after();
  const uint32_t tmem = B.tmem;
  // group table: first row and first token tile of every group
  if (P.offs) {
    for (int g = tid; g <= G; g += kTcThreads) s_off[g] = P.offs[g];
    __syncthreads();
    for (int g = tid; g < G; g += kTcThreads)
      if (s_off[g] < 0 || s_off[g] > s_off[g + 1] || s_off[g + 1] > P.t) B.bad = 1;
    __syncthreads();
    if (B.bad) {
      if (tid == 0) atomicCAS(P.status, 0, kStatusDevice);
      if (warp == 0) tc05::dealloc(tmem, 512);
      return;
    }
    if (warp == 0) {
      int base = 0;
      for (int g0 = 0; g0 < G; g0 += 32) {
        const int g = g0 + lane;
        const int c = g < G ? (s_off[g + 1] - s_off[g] + LY::N - 1) / LY::N : 0;
        int x = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(FULLM, x, o);
          if (lane >= o) x += y;
        }
        if (g < G) s_tile[g] = base + x - c;
        base += __shfl_sync(FULLM, x, 31);
      }
      if (lane == 0) s_tile[G] = base;
    }
  } else if (tid == 0) {
    s_off[0] = 0, s_off[1] = P.t;
    s_tile[0] = 0, s_tile[1] = (P.t + LY::N - 1) / LY::N;
  }
  __syncthreads();
  const int ntiles = s_tile[G] * nmt;
  const int my_tiles = (int)blockIdx.x < ntiles ? (ntiles - 1 - (int)blockIdx.x) / (int)gridDim.x + 1 : 0;
  // tile i: the weight tiles of a token tile follow one another (their token
  // rows stay in L2); the rows of a group are cut into equal tiles
  auto tile_of = [&](int lt) {
    const int i = (int)blockIdx.x + lt * (int)gridDim.x, tt = i / nmt;
    int lo = 0, hi = G;  // the last group whose first token tile is <= tt
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s_tile[mid] <= tt) lo = mid; else hi = mid;
    }
    const int m = s_off[lo + 1] - s_off[lo], c = s_tile[lo + 1] - s_tile[lo];
    const int w = ((m + c - 1) / c + 15) & ~15, r0 = (tt - s_tile[lo]) * w;
    Tile T;
    T.g = lo, T.mt = i - tt * nmt;
    T.n0 = s_off[lo] + r0;
    T.nlen = max(0, min(w, m - r0));
    T.N = max(16, (T.nlen + 15) & ~15);
    return T;
  };

  if (warp == 0) {
    // ---------------------------------------------------------------- MMA issue
    int s = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (int lt = 0; lt < my_tiles && ok; lt++) {
      const Tile T = tile_of(lt);
      const int b = lt & 1;
      if (!tc_warp_wait(&B.acc_empty[b], (uint32_t)(((lt >> 1) & 1) ^ 1), P)) break;
      tc05::fence_after();
      const uint32_t d = tmem + (uint32_t)(b * kTcN), idesc = tc05::idesc_mx_e4m3(T.N);
      for (int kb = 0; kb < nk; kb++) {
        if (!tc_warp_wait(&B.full[s], ph, P)) {
          ok = false;
          break;
        }
        tc05::fence_after();
        if (tc05::elect_one()) {
          const uint32_t st = smem_u32(sm) + (uint32_t)(s * LY::stage), sc = st + LY::offS;
          const uint32_t sfb = tmem + (uint32_t)(kTcScaleCol + 16 * s), sfa = sfb + 8;
          tc05::cp_scales(sfb, tc05::sdesc_scales(sc));
          if (T.N > 128) tc05::cp_scales(sfb + 4, tc05::sdesc_scales(sc + 512));
#pragma unroll
          for (int m = 0; m < MB; m++) tc05::cp_scales(sfa + 4 * m, tc05::sdesc_scales(sc + 1024 + 512 * m));
          const uint64_t bd = tc05::sdesc(st);
#pragma unroll
          for (int m = 0; m < MB; m++) {
            const uint64_t ad = tc05::sdesc(st + LY::offW + 16384 * m);
#pragma unroll
            for (int j = 0; j < 4; j++)
              tc05::mma_mx(d + (uint32_t)(m * LY::N), ad + 2 * j, bd + 2 * j, idesc, sfa + 4 * m, sfb, (kb | j) != 0);
          }
          tc05::commit(&B.empty[s]);
        }
        __syncwarp();
        if (++s == kTcStages) s = 0, ph ^= 1;
      }
      if (ok) {
        if (tc05::elect_one()) tc05::commit(&B.acc_full[b]);
        __syncwarp();
      }
    }
    // every MMA issued here has completed before TMEM is released
    if (tc05::elect_one()) tc05::commit(&B.drain);
    __syncwarp();
    tc_warp_wait(&B.drain, 0, P);
  } else if (warp == 1) {
    // ---------------------------------------------------------------- TMA
    int f = 0;
    bool ok = true;
    for (int lt = 0; lt < my_tiles && ok; lt++) {
      const Tile T = tile_of(lt);
      const int n128 = T.N >> 7, n32 = ((T.N & 127) + 31) >> 5, ntok = n128 + n32;
      const uint32_t bytes = (uint32_t)((n128 * 128 + n32 * 32) * 128 + MB * 16384);
      for (int kb = 0; kb < nk; kb++, f++) {
        const int s = f % kTcStages;
        if (!tc_warp_wait(&B.empty[s], (uint32_t)(((f / kTcStages) & 1) ^ 1), P)) {
          ok = false;
          break;
        }
        uint8_t *st = sm + s * LY::stage;
        // (failure-detection test: CTA 0 never expects its first stage's
        // copies, so the MMA warp's bounded wait runs out)
        const bool withheld = P.withhold && blockIdx.x == 0 && f == 0;
        if (withheld) {
          ok = false;
          break;
        }
        if (lane == 0) mbar_expect_tx(&B.full[s], bytes);
        __syncwarp();
        if (lane < ntok) {
          const int r0 = lane < n128 ? 128 * lane : 128 * n128 + 32 * (lane - n128);
          tc05::tma_load_2d(st + r0 * 128, lane < n128 ? &P.tm_a128 : &P.tm_a32, kb * 128, T.n0 + r0, &B.full[s]);
        } else if (lane < ntok + MB) {
          const int m = lane - ntok;
          const int row = T.g * P.n + (MB == 2 ? m * (P.n / 2) : 0) + T.mt * 128;
          tc05::tma_load_2d(st + LY::offW + 16384 * m, &P.tm_b, kb * 128, row, &B.full[s]);
        }
      }
    }
    // copies still in flight land before the CTA ends
    if (lane == 0)
      for (int g = f > kTcStages ? f - kTcStages : 0; g < f; g++)
        tc_wait(&B.full[g % kTcStages], (uint32_t)((g / kTcStages) & 1), P);
    __syncwarp();
  } else if (warp == 2) {
    // ---------------------------------------------------------------- token scales
    // lane l: rows l, l + 32, ... of the tile; four blocks' bytes a load
    int f = 0;
    bool ok = true;
    for (int lt = 0; lt < my_tiles && ok; lt++) {
      const Tile T = tile_of(lt);
      uint32_t cur[7], nxt[7];
      auto fetch = [&](int kb, uint32_t (&v)[7]) {
#pragma unroll
        for (int i = 0; i < 7; i++) {
          const int r = T.n0 + lane + 32 * i;
          v[i] = 32 * i < T.N && r < P.t && kb < nk
                     ? *reinterpret_cast<const uint32_t *>(P.sa + (size_t)r * P.lds + kb) : 0x7f7f7f7fu;
        }
      };
      fetch(0, nxt);
      for (int kb = 0; kb < nk; kb++, f++) {
        if ((kb & 3) == 0) {
#pragma unroll
          for (int i = 0; i < 7; i++) cur[i] = nxt[i];
          fetch(kb + 4, nxt);
        }
        const int s = f % kTcStages;
        if (!tc_warp_wait(&B.empty[s], (uint32_t)(((f / kTcStages) & 1) ^ 1), P)) {
          ok = false;
          break;
        }
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; i++) w[i] = i < 7 ? ((cur[i < 7 ? i : 0] >> (8 * (kb & 3))) & 0xffu) * 0x01010101u : 0x7f7f7f7fu;
        uint4 *dst = reinterpret_cast<uint4 *>(sm + s * LY::stage + LY::offS) + lane;
        dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
        if (T.N > 128) dst[32] = make_uint4(w[4], w[5], w[6], w[7]);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) tc05::mbar_arrive(&B.full[s]);
      }
    }
  } else if (warp == 3) {
    // ---------------------------------------------------------------- weight scales
    int f = 0;
    bool ok = true;
    for (int lt = 0; lt < my_tiles && ok; lt++) {
      const Tile T = tile_of(lt);
      const uint8_t *sb[MB];
      uint32_t v[MB];
#pragma unroll
      for (int m = 0; m < MB; m++)
        sb[m] = P.sb + ((size_t)T.g * P.nb + (MB == 2 ? m * (P.nb / 2) : 0) + T.mt) * nk;
      for (int kb = 0; kb < nk; kb++, f++) {
        if ((kb & 31) == 0)
#pragma unroll
          for (int m = 0; m < MB; m++) v[m] = kb + lane < nk ? sb[m][kb + lane] : 127u;
        const int s = f % kTcStages;
        if (!tc_warp_wait(&B.empty[s], (uint32_t)(((f / kTcStages) & 1) ^ 1), P)) {
          ok = false;
          break;
        }
        uint4 *dst = reinterpret_cast<uint4 *>(sm + s * LY::stage + LY::offS + 1024) + lane;
#pragma unroll
        for (int m = 0; m < MB; m++) {
          const uint32_t w = __shfl_sync(FULLM, v[m], kb & 31) * 0x01010101u;
          dst[32 * m] = make_uint4(w, w, w, w);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) tc05::mbar_arrive(&B.full[s]);
      }
    }
  } else {
    // ---------------------------------------------------------------- epilogue
    const int q = warp & 3;    // TMEM lane quadrant this warp may read
    const int et = tid - 128;  // 0..127 over the epilogue warps: the tile's weight row (channel)
    for (int lt = 0; lt < my_tiles; lt++) {
      const Tile T = tile_of(lt);
      const int b = lt & 1;
      // the four epilogue warps stop together (they share named barriers)
      if (!tc05::named_and(2, 128, tc_warp_wait(&B.acc_full[b], (uint32_t)((lt >> 1) & 1), P))) break;
      tc05::fence_after();
      const uint32_t tl = tmem + (uint32_t)(b * kTcN) + ((uint32_t)(32 * q) << 16);
      if constexpr (KIND == kOutSilu8) {
        uint8_t *hb = sm + LY::offEpi;                                     // [N][128] h in e4m3
        uint32_t *mx = reinterpret_cast<uint32_t *>(hb + LY::N * 128);     // [4][N] warp maxima
        // channel scale blocks are whole: 128 channels = this tile's rows
        for (int c0 = 0; c0 < T.N; c0 += 16) {
          float gt[16], up[16], h[16];
          tc05::ld16(tl + c0, gt);
          tc05::ld16(tl + LY::N + c0, up);
          uint32_t m = 0;
#pragma unroll
          for (int j = 0; j < 16; j++) {
            h[j] = gt[j] / (1.f + expf(-gt[j])) * up[j];
            const uint32_t wm = __reduce_max_sync(FULLM, mag_bits(h[j]));
            if (lane == j) m = wm;
          }
          if (lane < 16) mx[q * LY::N + c0 + lane] = m;
          tc05::named_sync(1, 128);
          const uint32_t *mc = mx + c0 + (lane & 15);
          const uint32_t mm = max(max(mc[0], mc[LY::N]), max(mc[2 * LY::N], mc[3 * LY::N]));
          const uint32_t e = e8m0_of_amax(mm);
          const float fe = e8m0_inv(e);
          if (et < 16 && c0 + et < T.nlen) P.hs[(size_t)(T.n0 + c0 + et) * P.ldhs + T.mt] = (uint8_t)e;
#pragma unroll
          for (int j = 0; j < 16; j++) {
            const float v = h[j] * __shfl_sync(FULLM, fe, j);
            hb[(c0 + j) * 128 + et] = (uint8_t)e4m3x2(v, 0.f);
          }
        }
        // the accumulator is read: the next tile's MMAs may fill it
        tc05::fence_before();
        __syncwarp();
        if (lane == 0) tc05::mbar_arrive(&B.acc_empty[b]);
        tc05::named_sync(1, 128);
        for (int i = et; i < T.nlen * 8; i += 128)
          *reinterpret_cast<uint4 *>(static_cast<uint8_t *>(P.out) + (size_t)(T.n0 + (i >> 3)) * P.ldo + T.mt * 128 +
                                     (i & 7) * 16) = *reinterpret_cast<const uint4 *>(hb + i * 16);
        tc05::named_sync(1, 128);  // hb and the maxima are free again
      } else {
        using O = typename std::conditional<KIND == kOutF32, float, uint16_t>::type;
        const int row = T.mt * 128 + et;
        O *o = static_cast<O *>(P.out) + (size_t)T.n0 * P.ldo + row;
        for (int c0 = 0; c0 < T.N; c0 += 16) {
          float v[16];
          tc05::ld16(tl + c0, v);
          if (row < P.n) {
#pragma unroll
            for (int j = 0; j < 16; j++)
              if (c0 + j < T.nlen) store_out(o + (int64_t)(c0 + j) * P.ldo, v[j]);
          }
        }
        tc05::fence_before();
        __syncwarp();
        if (lane == 0) tc05::mbar_arrive(&B.acc_empty[b]);
      }
    }
  }

  tc05::fence_before();
  __syncthreads();
  if (warp == 0) tc05::dealloc(tmem, 512);
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = [] {
    void *f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) !=
            cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return (EncodeTiledFn) nullptr;
    return reinterpret_cast<EncodeTiledFn>(f);
  }();
  return fn;
}

// bytes [rows] x cols, rows ld apart, box 128 bytes x box_rows, 128B swizzle, zeros outside
bool make_map8(CUtensorMap *m, const void *base, uint64_t cols, uint64_t rows, uint64_t ld, uint32_t box_rows) {
  const cuuint64_t dims[2] = {cols, rows};
  const cuuint64_t strides[1] = {ld};
  const cuuint32_t box[2] = {128, box_rows};
  const cuuint32_t estr[2] = {1, 1};
  return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, box, estr,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int MB, int KIND>
cudaError_t launch_tc(const Mm8P &p, int grid, bool pdl, cudaStream_t st) {
  cudaError_t e = cudaFuncSetAttribute(mm8_tc<MB, KIND>, cudaFuncAttributeMaxDynamicSharedMemorySize, TcLay<MB>::smem);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kTcThreads);
  cfg.dynamicSmemBytes = TcLay<MB>::smem;
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, mm8_tc<MB, KIND>, p);
}

}  // namespace

int mm8_tensor_maps(Mm8P &p, const char **why) {
  if (!encode_fn()) {
    *why = "cuTensorMapEncodeTiled is not available from the driver";
    return -1;
  }
  const uint64_t rows_b = (uint64_t)(p.G > 0 ? p.G : 1) * p.n;
  if (!make_map8(&p.tm_a128, p.a, p.k, p.t, p.lda, 128) || !make_map8(&p.tm_a32, p.a, p.k, p.t, p.lda, 32) ||
      !make_map8(&p.tm_b, p.b, p.k, rows_b, p.k, 128)) {
    *why = "cuTensorMapEncodeTiled rejected a tensor map";
    return -1;
  }
  return 0;
}

cudaError_t launch_mm8_small(const Mm8P &p, int out_kind, cudaStream_t st) {
  const unsigned grid = (unsigned)((p.n + 15) / 16);
  const int nt = (p.t + 7) / 8;
#define MOE_SMALL(NT)                                                          \
  if (out_kind == kOutF32) mm8_small<NT, float><<<grid, 32 * kSmWarps, 0, st>>>(p); \
  else mm8_small<NT, uint16_t><<<grid, 32 * kSmWarps, 0, st>>>(p);
  if (nt <= 1) { MOE_SMALL(1) }
  else if (nt <= 2) { MOE_SMALL(2) }
  else { MOE_SMALL(4) }
#undef MOE_SMALL
  return cudaGetLastError();
}

cudaError_t launch_mm8_tc(const Mm8P &p, int out_kind, int n_sms, bool pdl, cudaStream_t st) {
  // no more CTAs than tiles (grouped: the bound of one partial tile a group)
  const int64_t nmax = kTcN / (out_kind == kOutSilu8 ? 2 : 1);
  const int64_t tt = (p.t + nmax - 1) / nmax + (p.offs ? p.G : 0);
  const int64_t tiles = tt * (out_kind == kOutSilu8 ? p.n / 256 : p.nb);
  const int grid = (int)(tiles < n_sms ? tiles : n_sms);
  if (out_kind == kOutF32) return launch_tc<1, kOutF32>(p, grid, pdl, st);
  if (out_kind == kOutBf16) return launch_tc<1, kOutBf16>(p, grid, pdl, st);
  return launch_tc<2, kOutSilu8>(p, grid, pdl, st);
}

}  // namespace moe
