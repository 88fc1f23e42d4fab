// mm8.cu -- block-scaled 8-bit matrix products: out[r][j] = sum over blocks
// kb of 128 k of 2^(sa[r][kb] + sb[j / 128][kb] - 254) * (a[r] . b[j] in kb).
//
// Two kernels:
//   small  up to 32 rows, by mm8_small: the weights are streamed once from HBM
//          straight into the fragments of mma.sync (no shared memory), the
//          few rows come from L1; a CTA takes 16 weight rows and splits k
//          over its warps.
//          1 x 2048 x 2048: 2.9 us a call in a graph of calls on weights
//          from HBM, of which the 4.2 MB are 0.6: launch and one HBM latency
//          bound it.  8 x 8192 x 4096: 11.3, the bytes 5.0.
//   tc     any number of rows, dense or grouped: persistent, warp
//          specialised, tcgen05 with the tensor cores' own block scaling
//          (kind::mxf8f6f4), accumulating all of k in TMEM.
//          8192 x 8192 x 2048: 94 to 98 us, 2.8 to 2.9 PFLOP/s; bound by what
//          the SMs take in from L2 (14.5 TB/s of requests there).  128 uneven
//          groups, 32668 rows x 1536 x 2048: 117 us, 470 MB read, 16 TB/s at
//          L2.
#include <cuda_runtime.h>

#include <type_traits>

#include "fp8.cuh"
#include "tc05.cuh"
#include "tmap.cuh"

namespace moe {
namespace {

constexpr unsigned FULLM = 0xffffffffu;

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

constexpr int kSmWarps = 8;

// One CTA: 16 weight rows, 8 * NT token columns.  Lane (g, q) = (lane / 4,
// lane % 4) loads 16 consecutive bytes of rows g and g + 8 at k = 16q and
// 64 + 16q of a block; the four words of a 16-byte piece serve as the k
// quarters of two MMAs.  The same pieces of the token rows serve as B, so
// the order of k inside a block is permuted alike on both sides.  Warp w
// takes the blocks w, w + 8, ...; the warps' sums meet in shared memory, in
// a fixed order.
template <int NT, class T>
__global__ void __launch_bounds__(32 * kSmWarps) mm8_few_rows(const __grid_constant__ Mm8Args P) {
  __shared__ float red[kSmWarps][16][8 * NT + 1];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q = lane & 3;
  pdl_wait_prev();
  pdl_launch_next();
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
  // two blocks' weights in flight: of k = 2048 all that the warp takes
  uint4 a[2][2][2];  // [block][piece][row g, g + 8]
  auto load = [&](uint4 (&x)[2][2], int kb) {
    const int k0 = kb * 128 + q * 16, k1 = k0 + 64;
    x[0][0] = ok0 && k0 < P.k ? ldg_stream4(w0 + k0) : zero;
    x[0][1] = ok1 && k0 < P.k ? ldg_stream4(w1 + k0) : zero;
    x[1][0] = ok0 && k1 < P.k ? ldg_stream4(w0 + k1) : zero;
    x[1][1] = ok1 && k1 < P.k ? ldg_stream4(w1 + k1) : zero;
  };
  auto step = [&](const uint4 (&x)[2][2], int kb) {
    const int k0 = kb * 128 + q * 16, k1 = k0 + 64;
    const float fb = e8m0_f(sb[kb]);
#pragma unroll
    for (int j = 0; j < NT; j++) {
      const int r = 8 * j + g;
      const uint8_t *xr = P.a + (size_t)r * P.lda;
      const uint4 b0 = r < P.t && k0 < P.k ? *reinterpret_cast<const uint4 *>(xr + k0) : zero;
      const uint4 b1 = r < P.t && k1 < P.k ? *reinterpret_cast<const uint4 *>(xr + k1) : zero;
      const int c = 8 * j + 2 * q;
      const float s0 = c < P.t ? e8m0_f(P.sa[(size_t)c * P.lds + kb]) : 1.f;
      const float s1 = c + 1 < P.t ? e8m0_f(P.sa[(size_t)(c + 1) * P.lds + kb]) : 1.f;
      float d[4] = {0.f, 0.f, 0.f, 0.f};
      mma_e4m3(d, x[0][0].x, x[0][1].x, x[0][0].y, x[0][1].y, b0.x, b0.y);
      mma_e4m3(d, x[0][0].z, x[0][1].z, x[0][0].w, x[0][1].w, b0.z, b0.w);
      mma_e4m3(d, x[1][0].x, x[1][1].x, x[1][0].y, x[1][1].y, b1.x, b1.y);
      mma_e4m3(d, x[1][0].z, x[1][1].z, x[1][0].w, x[1][1].w, b1.z, b1.w);
      const float p[2] = {s0 * fb, s1 * fb};
      if (scales_hold(p)) {
        acc[j][0] += d[0] * p[0], acc[j][1] += d[1] * p[1];
        acc[j][2] += d[2] * p[0], acc[j][3] += d[3] * p[1];
      } else {
        acc[j][0] += by_scales(d[0], s0, fb), acc[j][1] += by_scales(d[1], s1, fb);
        acc[j][2] += by_scales(d[2], s0, fb), acc[j][3] += by_scales(d[3], s1, fb);
      }
    }
  };
#pragma unroll
  for (int i = 0; i < 2; i++)
    if (warp + i * kSmWarps < P.nk) load(a[i], warp + i * kSmWarps);
  for (int kb = warp; kb < P.nk; kb += 2 * kSmWarps) {
#pragma unroll
    for (int i = 0; i < 2; i++) {
      const int k1 = kb + i * kSmWarps, k2 = k1 + 2 * kSmWarps;
      if (k1 < P.nk) {
        step(a[i], k1);
        if (k2 < P.nk) load(a[i], k2);
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
// Persistent: CTA (or CTA pair) i walks the tiles i, i + grid, ...  A tile is
// MB blocks of 128 weight rows (the M side: one TMEM lane a weight row) by up
// to N token rows of one group (the N side).  Weights on the M side keep M
// full whatever the group's size; N follows it in steps of 16 (32).
// CG = 2 (the usual form): a cluster of two CTAs takes two neighbouring
// weight tiles and shares the token rows, each CTA holding half of them
// (cta_group::2, M = 256).  A CTA then reads 30 KB a k block instead of 44 for
// the same products: the one-CTA form moved 14 TB/s from L2 to the SMs and
// was bound by that (8192 x 8192 x 2048 without its MMAs: 120 of 130 us).
// MB = 2 (silu): 128 gate rows and the 128 up rows of the same channels
// share the token tile, and the epilogue has a whole 128-channel scale block
// of h in its four warps.
//   warps 0-3 scales: E8M0 bytes -> words in TMEM, each warp its own 32 lanes
//             (the tensor cores read a row's scale from every quadrant)
//   warps 4-7 epilogue: TMEM -> registers -> global, from one of two
//             accumulators while the MMAs fill the other
//   warp 8    (even CTA) issues a stage's MMAs once its operands are there
//   warp 9    TMA: 128 weight rows x 128 k a block, the CTA's share of the token rows
// A stage is KB k blocks (one, or two where k allows: half as many copies,
// twice as long), as many stages as fit for the launch's tile width.  A scale
// word holds the bytes of four consecutive
// blocks, as they stand in memory; the MMAs of block kb name byte kb % 4, so
// scales are written once in four blocks, into one of four slots of TMEM
// columns with barriers of their own.  The full, scale and acc_empty
// barriers of a pair are the even CTA's, and the odd CTA's warps
// arrive on them: what those arrivals order is TMEM accesses (tcgen05
// fences), no shared memory.  (Scales passed through shared memory needed a
// release across the cluster every stage, 0.7 us each: 190 us at 8192 x 8192
// x 2048.)  The others are each CTA's own, committed to both.
constexpr int kTcThreads = 320;
constexpr int kMaxGroups = 1024;
constexpr int kMaxStages = 12;

struct TcBars {
  uint64_t full[kMaxStages], empty[kMaxStages], sc_full[4], sc_empty[4], acc_full[2], acc_empty[2], drain;
  uint32_t tmem;
  int bad;
};

template <int MB, int CG>
struct TcLay {
  static constexpr int step = 16 * CG;                           // tile widths
  static constexpr int N = MB == 1 ? 224 : (CG == 1 ? 112 : 96); // token columns of a tile
  static constexpr int accCols = MB * N;                         // of each of two buffers
  static constexpr int scaleCol = 2 * accCols;                   // then four slots of 12 scale columns
  static_assert(scaleCol + 12 * 4 <= 512, "tensor memory");
  static constexpr int unit = 16 * CG == 32 ? 16 : 32;           // token boxes: multiples of this many rows
  // front: silu: h bytes [N][128], maxima [4][N]; else 32 x 32 values a warp
  static constexpr int epi = MB == 2 ? N * 128 + 4 * N * 4 : 4 * 4096;
  static constexpr int offTab = (epi + 15) & ~15;                // int [G + 1] first row, first token tile, [G] tile width
  static constexpr int offBars = (offTab + 3 * (kMaxGroups + 1) * 4 + 15) & ~15;
  static constexpr int offRing = (offBars + (int)sizeof(TcBars) + 1023) / 1024 * 1024;
  static constexpr int room = 226 * 1024 - offRing;              // for the ring, the base rounded up
};

struct Tile {
  int g, mt, n0, nlen, N;
};

template <int CG>
__device__ bool tc_wait(uint64_t *bar, uint32_t par, const Mm8P &P) {
  auto done = [&] { return CG == 1 ? mbar_try_wait(bar, par) : tc05::mbar_try_wait_cluster(bar, par); };
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
template <int CG>
__device__ __forceinline__ bool tc_warp_wait(uint64_t *bar, uint32_t par, const Mm8P &P) {
  bool ok = true;
  if ((threadIdx.x & 31) == 0) ok = tc_wait<CG>(bar, par, P);
  return __shfl_sync(FULLM, ok ? 1 : 0, 0) != 0;
}

template <int MB, int KIND, int CG, int KB>
__global__ void __launch_bounds__(kTcThreads, 1) mm8_tc(const __grid_constant__ Mm8P P) {
  pdl_launch_next();
  extern __shared__ __align__(1024) uint8_t smraw[];
  // the same offset in both CTAs of a pair: dynamic shared memory starts alike
  uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smraw) + 1023) & ~(uintptr_t)1023);
  using LY = TcLay<MB, CG>;
  const int S = P.stages;
  uint8_t *ring = sm + LY::offRing;
  TcBars &B = *reinterpret_cast<TcBars *>(sm + LY::offBars);
  int *s_off = reinterpret_cast<int *>(sm + LY::offTab), *s_tile = s_off + kMaxGroups + 1, *s_w = s_tile + kMaxGroups + 1;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = CG == 1 ? 0 : (int)tc05::cluster_rank();
  const int G = P.G > 0 ? P.G : 1, nk = P.nk;
  const int nmt = MB == 2 ? P.n / 256 : P.nb;   // weight tiles a group
  const int nmp = (nmt + CG - 1) / CG;          // taken CG at a time

  if (tid == 0) {
    for (int s = 0; s < S; s++) {
      mbar_init(&B.full[s], 1);
      mbar_init(&B.empty[s], 1);
    }
    for (int s = 0; s < 4; s++) {
      mbar_init(&B.sc_full[s], 4 * CG);
      mbar_init(&B.sc_empty[s], 1);
    }
    for (int b = 0; b < 2; b++) {
      mbar_init(&B.acc_full[b], 1);
      mbar_init(&B.acc_empty[b], 4 * CG);
    }
    mbar_init(&B.drain, 1);
    fence_mbar_init();
    B.bad = 0;
  }
  if (warp == 8) {
    if constexpr (CG == 1) tc05::alloc(&B.tmem, 512);
    else tc05::alloc_pair(&B.tmem, 512);
  }
  pdl_wait_prev();  // the offsets and the operands may be the previous kernel's
  tc05::fence_before();
  if constexpr (CG == 1) __syncthreads();
  else tc05::cluster_sync();
  tc05::fence_after();
  const uint32_t tmem = B.tmem;
  // group table: first row, first token tile and tile width (the rows of a
  // group are cut into equal tiles) of every group
  auto width = [](int m, int c) { return ((m + c - 1) / c + LY::step - 1) / LY::step * LY::step; };
  if (P.offs) {
    for (int g = tid; g <= G; g += kTcThreads) s_off[g] = P.offs[g];
    __syncthreads();
    for (int g = tid; g < G; g += kTcThreads)
      if (s_off[g] < 0 || s_off[g] > s_off[g + 1] || s_off[g + 1] > P.t) B.bad = 1;
    __syncthreads();
    for (int g = tid; g < G; g += kTcThreads) {
      const int m = s_off[g + 1] - s_off[g], c = B.bad ? 0 : (m + P.wmax - 1) / P.wmax;
      s_tile[g] = c, s_w[g] = c ? width(m, c) : 0;
    }
    __syncthreads();
    if (warp == 0) {
      int base = 0;
      for (int g0 = 0; g0 < G; g0 += 32) {
        const int g = g0 + lane, c = g < G ? s_tile[g] : 0;
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
    s_tile[0] = 0, s_tile[1] = (P.t + P.wmax - 1) / P.wmax;
    s_w[0] = width(P.t, s_tile[1]);
  }
  __syncthreads();
  // the status of the call: one CTA's to set (a wait gives up long after)
  if (tid == 0 && blockIdx.x == 0) {
    if (P.zero_status) *P.status = B.bad ? kStatusDevice : 0;
    else if (B.bad) atomicCAS(P.status, 0, kStatusDevice);
  }
  const int ntiles = s_tile[G] * nmp, cl = (int)blockIdx.x / CG, ncl = (int)gridDim.x / CG;
  const int my_tiles = cl < ntiles ? (ntiles - 1 - cl) / ncl + 1 : 0;
  // tile i: the weight tiles of a token tile follow one another (their token
  // rows stay in L2).  A role walks its tiles by next_tile: without divisions,
  // and the warps (not the one thread that issues MMAs) look for the group 32
  // entries at a time, as the copies of the next tile wait for this
  // (with divisions and a binary search in every role: 427 us instead of 409
  // for 4096 rows through 10 of 512 experts).
  int tt = cl / nmp, mp = cl - tt * nmp;
  const int step_t = ncl / nmp, step_m = ncl - step_t * nmp;
  auto next_tile = [&](auto by_warp) {
    int lo = 0;  // the last group whose first token tile is <= tt
    if constexpr (decltype(by_warp)::value) {
      lo = 32 * (__popc(__ballot_sync(FULLM, 32 * lane < G && s_tile[32 * lane] <= tt)) - 1);
      lo += __popc(__ballot_sync(FULLM, lo + lane < G && s_tile[lo + lane] <= tt)) - 1;
    } else {
      for (int hi = G; hi - lo > 1;) {
        const int mid = (lo + hi) >> 1;
        if (s_tile[mid] <= tt) lo = mid; else hi = mid;
      }
    }
    const int m = s_off[lo + 1] - s_off[lo], w = s_w[lo], r0 = (tt - s_tile[lo]) * w;
    Tile T;
    T.g = lo, T.mt = mp * CG + rank;
    T.n0 = s_off[lo] + r0;
    T.nlen = max(0, min(w, m - r0));
    T.N = max(LY::step, (T.nlen + LY::step - 1) / LY::step * LY::step);
    tt += step_t, mp += step_m;
    if (mp >= nmp) mp -= nmp, tt++;
    return T;
  };
  using ByWarp = std::true_type;
  using ByThread = std::false_type;
  auto weight_row = [&](const Tile &T, int m) { return T.g * P.n + (MB == 2 ? m * (P.n / 2) : 0) + T.mt * 128; };
  // arrive on a barrier of the even CTA (this CTA's, without a pair)
  auto arrive_even = [&](uint64_t *bar) {
    if constexpr (CG == 1) tc05::mbar_arrive(bar);
    else tc05::mbar_arrive_cluster(tc05::map_rank(bar, 0));
  };
  // a pair's last tile may have no weight tile for the odd CTA: its rows are
  // some others' (or none), and nothing of them is stored

  if (warp == 8) {
    // ---------------------------------------------------------------- MMA issue
    // one thread walks the loop: no exchange with the rest of the warp
    // between a stage's arrival and its MMAs
    if (rank == 0 && tc05::elect_one()) {
      int s = 0, sl = 0;
      uint32_t ph = 0, slp = 0;
      bool ok = true;
      Tile Tn;
      if (my_tiles > 0) Tn = next_tile(ByThread());
      const uint32_t base = smem_u32(ring);
      for (int lt = 0; lt < my_tiles && ok; lt++) {
        const Tile T = Tn;
        const int b = lt & 1;
        if (!tc_wait<CG>(&B.acc_empty[b], (uint32_t)(((lt >> 1) & 1) ^ 1), P)) break;
        tc05::fence_after();
        const uint32_t d = tmem + (uint32_t)(b * LY::accCols), idesc = tc05::idesc_mx_e4m3(128 * CG, T.N);
        const uint32_t panel = (uint32_t)((T.N / CG + LY::unit - 1) / LY::unit * LY::unit * 128);  // token bytes a block
        for (int k0 = 0; k0 < nk; k0 += KB) {
          if (!tc_wait<CG>(&B.full[s], ph, P)) {
            ok = false;
            break;
          }
          const uint32_t st = base + (uint32_t)(s * P.stage);
#pragma unroll
          for (int kk = 0; kk < KB; kk++) {
            const int kb = k0 + kk;
            if ((kb & 3) == 0 && !tc_wait<CG>(&B.sc_full[sl], slp, P)) {
              ok = false;
              break;
            }
            tc05::fence_after();
            const uint32_t sfb = tmem + (uint32_t)(LY::scaleCol + 12 * sl), sfa = sfb + (MB == 1 ? 8 : 4);
            const uint32_t id = idesc | tc05::idesc_scale_byte(kb & 3);
            const uint64_t bd = tc05::sdesc(st + kk * panel);
#pragma unroll
            for (int m = 0; m < MB; m++) {
              const uint64_t ad = tc05::sdesc(st + (uint32_t)(KB * P.tok) + 16384 * (KB * m + kk));
#pragma unroll
              for (int j = 0; j < 4; j++)
                tc05::mma_mx<CG>(d + (uint32_t)(m * LY::N), ad + 2 * j, bd + 2 * j, id, sfa + 4 * m, sfb, (kb | j) != 0);
            }
            if ((kb & 3) == 3 || kb == nk - 1) {
              if constexpr (CG == 1) tc05::commit(&B.sc_empty[sl]);
              else tc05::commit_pair(&B.sc_empty[sl]);
              if (++sl == 4) sl = 0, slp ^= 1;
            }
          }
          if (!ok) break;
          if constexpr (CG == 1) tc05::commit(&B.empty[s]);
          else tc05::commit_pair(&B.empty[s]);
          if (++s == S) s = 0, ph ^= 1;
          if (k0 == 0 && lt + 1 < my_tiles) Tn = next_tile(ByThread());  // while the MMAs run
        }
        if (ok) {
          if constexpr (CG == 1) tc05::commit(&B.acc_full[b]);
          else tc05::commit_pair(&B.acc_full[b]);
        }
      }
      // every MMA issued here has completed before TMEM is released
      if constexpr (CG == 1) tc05::commit(&B.drain);
      else tc05::commit_pair(&B.drain);
      tc_wait<CG>(&B.drain, 0, P);
    }
    __syncwarp();
  } else if (warp == 9) {
    // ---------------------------------------------------------------- TMA
    int f = 0, s = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (int lt = 0; lt < my_tiles && ok; lt++) {
      const Tile T = next_tile(ByWarp());
      // this CTA's token rows of the tile: one box of as many rows (64 + 32 +
      // 16 in three boxes cost 7% at 8192 x 8192 x 2048).  One lane issues
      // the copies: their operands are uniform registers, and lanes with
      // operands of their own would be served one by one
      const int rows = T.N / CG, box = (rows + LY::unit - 1) / LY::unit, first = T.n0 + rank * rows;
      const uint32_t bytes = (uint32_t)(KB * (box * LY::unit * 128 + MB * 16384)) * CG;
      const CUtensorMap *map_a = &P.tm_a[box - 1];
      for (int kb = 0; kb < nk; kb += KB, f++) {
        // (failure-detection test: CTA 0 never expects its first stage's
        // copies, so the MMA warp's bounded wait runs out)
        if (!tc_warp_wait<CG>(&B.empty[s], ph ^ 1, P) || (P.withhold && blockIdx.x == 0 && f == 0)) {
          ok = false;
          break;
        }
        if (tc05::elect_one()) {
          uint8_t *st = ring + s * P.stage;
          if (rank == 0) mbar_expect_tx(&B.full[s], bytes);
          const uint32_t bar = CG == 1 ? smem_u32(&B.full[s]) : tc05::map_rank(&B.full[s], 0);
#pragma unroll
          for (int m = 0; m < MB; m++)
            tc05::tma_load_cg<CG, KB>(st + KB * P.tok + 16384 * KB * m, &P.tm_b, kb, weight_row(T, m), bar);
          tc05::tma_load_cg<CG, KB>(st, map_a, kb, first, bar);
        }
        __syncwarp();
        if (++s == S) s = 0, ph ^= 1;
      }
    }
    // copies still in flight land before the CTA (the pair) ends
    if (lane == 0 && rank == 0)
      for (int g = f > S ? f - S : 0; g < f; g++) tc_wait<CG>(&B.full[g % S], (uint32_t)((g / S) & 1), P);
    __syncwarp();
  } else if (warp < 4) {
    // ---------------------------------------------------------------- scales
    // Tokens: lane l has the rows l, l + 32, ... of the tile, four blocks'
    // bytes a word, the next four (the next tile's first) on their way;
    // weights: lane l has block (kb & ~31) + l of the tile's weight rows.
    int f = 0;
    bool ok = true;
    constexpr int R = (LY::N + 31) / 32, WB = MB == 1 ? 8 : 4;
    uint32_t nxt[R], wv[MB];
    auto fetch = [&](const Tile &T, int kb) {
#pragma unroll
      for (int i = 0; i < R; i++) {
        const int r = T.n0 + lane + 32 * i;
        nxt[i] = 32 * i < T.N && r < P.t ? *reinterpret_cast<const uint32_t *>(P.sa + (size_t)r * P.lds + kb) : 0u;
      }
    };
    Tile T, Tn;
    if (my_tiles > 0) Tn = next_tile(ByWarp()), fetch(Tn, 0);
    for (int lt = 0; lt < my_tiles && ok; lt++) {
      T = Tn;
      if (lt + 1 < my_tiles) Tn = next_tile(ByWarp());
      for (int kb = 0; kb < nk; kb += 4, f++) {
        if ((kb & 31) == 0)
#pragma unroll
          for (int m = 0; m < MB; m++)
            wv[m] = kb + lane < nk && T.mt < nmt
                        ? P.sb[((size_t)T.g * P.nb + (MB == 2 ? m * (P.nb / 2) : 0) + T.mt) * nk + kb + lane] : 0u;
        uint32_t w[12];  // token rows 0-31, 32-63, ...; then the weight blocks, the same for all rows
#pragma unroll
        for (int i = 0; i < WB; i++) w[i] = i < R ? nxt[i < R ? i : 0] : 0u;
        if (kb + 4 < nk) fetch(T, kb + 4);
        else if (lt + 1 < my_tiles) fetch(Tn, 0);
#pragma unroll
        for (int m = 0; m < MB; m++) {
          uint32_t x = 0;
#pragma unroll
          for (int i = 0; i < 4; i++) x |= __shfl_sync(FULLM, wv[m], (kb + i) & 31) << (8 * i);
#pragma unroll
          for (int i = 0; i < 4; i++) w[WB + 4 * m + i] = x;
        }
        const int sl = f & 3;
        if (!tc_warp_wait<CG>(&B.sc_empty[sl], (uint32_t)(((f >> 2) & 1) ^ 1), P)) {
          ok = false;
          break;
        }
        tc05::fence_after();
        tc05::st12(tmem + (uint32_t)(LY::scaleCol + 12 * sl) + ((uint32_t)(32 * warp) << 16), w);
        tc05::wait_st();
        tc05::fence_before();
        __syncwarp();
        if (lane == 0) arrive_even(&B.sc_full[sl]);
      }
    }
  } else {
    // ---------------------------------------------------------------- epilogue
    const int q = warp & 3;    // TMEM lane quadrant this warp may read
    const int et = tid - 128;  // 0..127 over the epilogue warps: the tile's weight row (channel)
    auto release = [&](int b) {  // the accumulator is read: the MMAs may fill it again
      tc05::fence_before();
      __syncwarp();
      if (lane == 0) arrive_even(&B.acc_empty[b]);
    };
    for (int lt = 0; lt < my_tiles; lt++) {
      const Tile T = next_tile(ByWarp());
      const int b = lt & 1;
      // the four epilogue warps stop together (they share named barriers)
      if (!tc05::named_and(2, 128, tc_warp_wait<CG>(&B.acc_full[b], (uint32_t)((lt >> 1) & 1), P))) break;
      tc05::fence_after();
      const uint32_t tl = tmem + (uint32_t)(b * LY::accCols) + ((uint32_t)(32 * q) << 16);
      if (T.mt >= nmt) {
        release(b);
      } else if constexpr (KIND == kOutSilu8) {
        uint8_t *hb = sm;                                     // [N][128] h in e4m3
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
            hb[(c0 + j) * 128 + et] = (uint8_t)e4m3x2<true>(v, 0.f);
          }
        }
        release(b);
        tc05::named_sync(1, 128);
        for (int i = et; i < T.nlen * 8; i += 128)
          *reinterpret_cast<uint4 *>(static_cast<uint8_t *>(P.out) + (size_t)(T.n0 + (i >> 3)) * P.ldo + T.mt * 128 +
                                     (i & 7) * 16) = *reinterpret_cast<const uint4 *>(hb + i * 16);
        tc05::named_sync(1, 128);  // hb and the maxima are free again
      } else {
        // 32 tokens at a time: the warp's 32 x 32 piece is turned in shared
        // memory so that a lane stores 16 bytes of a token's row (a store a
        // token of 64 bytes each took 17 cycles an instruction and bound the
        // kernel); rows that do not allow that are stored value by value
        using O = typename std::conditional<KIND == kOutF32, float, uint16_t>::type;
        constexpr int V = 16 / sizeof(O), per = 32 / V;  // values a 16-byte piece, pieces a token
        O *stg = reinterpret_cast<O *>(sm) + q * 1024;
        const int row0 = T.mt * 128 + 32 * q;
        O *o = static_cast<O *>(P.out) + (size_t)T.n0 * P.ldo + row0;
        const bool wide = P.wide && row0 + 32 <= P.n;
        for (int c0 = 0; c0 < T.N; c0 += 32) {
          float v[32];
          if (c0 + 32 <= T.N) tc05::ld32(tl + c0, v);
          else tc05::ld16(tl + c0, v);
          if (wide) {
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 32; j++) store_out(stg + j * 32 + lane, v[j]);
            __syncwarp();
#pragma unroll
            for (int i = 0; i < per; i++) {
              const int tok = i * (32 / per) + lane / per, piece = lane % per;
              if (c0 + tok < T.nlen)
                *reinterpret_cast<uint4 *>(o + (int64_t)(c0 + tok) * P.ldo + piece * V) =
                    *reinterpret_cast<const uint4 *>(stg + tok * 32 + piece * V);
            }
          } else if (row0 + lane < P.n) {
#pragma unroll
            for (int j = 0; j < 32; j++)
              if (c0 + j < T.nlen) store_out(o + (int64_t)(c0 + j) * P.ldo + lane, v[j]);
          }
        }
        release(b);
      }
    }
  }

  tc05::fence_before();
  if constexpr (CG == 1) {
    __syncthreads();
    if (warp == 8) tc05::dealloc(tmem, 512);
  } else {
    tc05::cluster_sync();
    if (warp == 8) tc05::dealloc_pair(tmem, 512);
  }
}

// bytes [rows] x cols, rows ld apart, 128B swizzle, zeros outside: boxes of
// 128 bytes x box_rows, or (kb == 2; cols % 128 == 0) x 2 k blocks as well
bool make_map8(CUtensorMap *m, const void *base, uint64_t cols, uint64_t rows, uint64_t ld, uint32_t box_rows, int kb) {
  const cuuint64_t dims2[2] = {cols, rows}, dims3[3] = {128, rows, cols / 128};
  const cuuint64_t strides[2] = {ld, 128};
  const cuuint32_t box[3] = {128, box_rows, 2};
  const cuuint32_t estr[3] = {1, 1, 1};
  return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, (cuuint32_t)kb + 1, const_cast<void *>(base),
                     kb == 2 ? dims3 : dims2, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// weight tiles of a group, and whether CTA pairs take them two at a time
int weight_tiles(const Mm8P &p, int out_kind) { return out_kind == kOutSilu8 ? p.n / 256 : p.nb; }
bool use_pairs(const Mm8P &p, int out_kind) { return weight_tiles(p, out_kind) > 1; }

// The launch of one form: the ring for the tile width p.wmax, the tensor
// maps, the kernel.
template <int MB, int KIND, int CG, int KB>
cudaError_t launch_tc(Mm8P &p, int grid, cudaStream_t st) {
  using LY = TcLay<MB, CG>;
  const int rows = (p.wmax / CG + LY::unit - 1) / LY::unit * LY::unit;
  p.tok = rows * 128;
  p.stage = (KB * (p.tok + MB * 16384) + 1023) / 1024 * 1024;
  p.stages = LY::room / p.stage < kMaxStages ? LY::room / p.stage : kMaxStages;
  // the most any launch asks for: another host thread's launch of the same
  // kernel may stand between this and the launch below.  Before the tensor
  // maps: it makes the device's context this thread's, which they need
  cudaError_t e = cudaFuncSetAttribute(mm8_tc<MB, KIND, CG, KB>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       LY::offRing + LY::room + 1024);
  if (e != cudaSuccess) return e;
  bool ok = encode_fn() != nullptr;
  ok = ok && make_map8(&p.tm_b, p.b, p.k, (uint64_t)(p.G > 0 ? p.G : 1) * p.n, p.k, 128, KB);
  for (int i = 0; i < rows / LY::unit; i++)
    ok = ok && make_map8(&p.tm_a[i], p.a, p.k, p.t, p.lda, (uint32_t)((i + 1) * LY::unit), KB);
  if (!ok) return cudaErrorNotSupported;
  const int smem = LY::offRing + p.stages * p.stage + 1024;
  cudaLaunchAttribute at[2];
  int n = 0;
  if (CG == 2) {
    at[n].id = cudaLaunchAttributeClusterDimension;
    at[n].val.clusterDim.x = 2, at[n].val.clusterDim.y = 1, at[n].val.clusterDim.z = 1;
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
  return cudaLaunchKernelEx(&cfg, mm8_tc<MB, KIND, CG, KB>, p);
}

}  // namespace

cudaError_t launch_mm8_small(const Mm8Args &p, int out_kind, cudaStream_t st) {
  const unsigned grid = (unsigned)((p.n + 15) / 16);
  const int nt = (p.t + 7) / 8;
  auto f = nt <= 1 ? mm8_few_rows<1, float> : (nt <= 2 ? mm8_few_rows<2, float> : mm8_few_rows<4, float>);
  if (out_kind == kOutBf16) f = nt <= 1 ? mm8_few_rows<1, uint16_t> : (nt <= 2 ? mm8_few_rows<2, uint16_t> : mm8_few_rows<4, uint16_t>);
  return launch_pdl(f, dim3(grid), 32 * kSmWarps, 0, st, p);
}

template <int MB, int KIND>
cudaError_t launch_tc_form(Mm8P p, int n_sms, cudaStream_t st) {
  const bool pairs = use_pairs(p, KIND);
  p.wide = ((reinterpret_cast<uintptr_t>(p.out) | (uintptr_t)(p.ldo * (KIND == kOutF32 ? 4 : 2))) & 15) == 0;
  p.wmax = pairs ? TcLay<MB, 2>::N : TcLay<MB, 1>::N;
  const int cg = pairs ? 2 : 1;
  if (!p.offs) {
    // dense: the tile width with the least (rounds of tiles) x (width + what
    // a tile costs whatever its width, some 48 columns' worth).  333 x 1000 x
    // 2000: 32 columns instead of 192 keep 44 pairs busy instead of 8
    const int64_t nmp = (weight_tiles(p, KIND) + cg - 1) / cg;
    int64_t best = INT64_MAX;
    int pick = p.wmax;
    for (int w = p.wmax; w >= 16 * cg; w -= 16 * cg) {
      const int64_t rounds = ((p.t + w - 1) / w * nmp + n_sms / cg - 1) / (n_sms / cg), cost = rounds * (w + 48);
      if (cost < best) best = cost, pick = w;
    }
    p.wmax = pick;
  }
  // no more CTAs than tiles (grouped: the bound of one partial tile a group)
  const int64_t tt = (p.t + p.wmax - 1) / p.wmax + (p.offs ? p.G : 0);
  const int64_t tiles = tt * ((weight_tiles(p, KIND) + cg - 1) / cg);
  const int grid = (int)(tiles < n_sms / cg ? tiles : n_sms / cg) * cg;
  if (!pairs) return launch_tc<MB, KIND, 1, 1>(p, grid, st);
  if constexpr (MB == 1)
    if (p.k % 256 == 0) return launch_tc<MB, KIND, 2, 2>(p, grid, st);
  return launch_tc<MB, KIND, 2, 1>(p, grid, st);
}

cudaError_t launch_mm8_tc(const Mm8P &p, int out_kind, int n_sms, cudaStream_t st) {
  if (out_kind == kOutF32) return launch_tc_form<1, kOutF32>(p, n_sms, st);
  if (out_kind == kOutBf16) return launch_tc_form<1, kOutBf16>(p, n_sms, st);
  return launch_tc_form<2, kOutSilu8>(p, n_sms, st);
}

}  // namespace moe
