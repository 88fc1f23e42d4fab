// gate.cu -- routing from given logits: softmax or sigmoid scores, a bias
// that steers the selection only, expert groups, top-k, renormalised weights.
//
// One warp per row; lane l holds the C consecutive experts from l * C on, so
// that among equal keys the lowest lane (and in it the lowest place) is the
// lowest id.  The selection works on 32-bit keys that order as the scores do
// (0: masked).  Without a bias the key is the logit's own and the order is
// exact.  With one, and for the sums of the group stage, 32-bit scores carry
// an error of a few 2^-22; wherever two candidates are closer than that (and
// are not the same numbers) the warp decides the row again in 64 bits.
#include <cuda_runtime.h>

#include "fp8.cuh"

namespace moe {
namespace {

constexpr unsigned FULLM = 0xffffffffu;
constexpr int kGateWarps = 4;
constexpr float kInf = __builtin_huge_valf();

__device__ __forceinline__ uint32_t okey(float f) {
  const uint32_t u = __float_as_uint(f == 0.f ? 0.f : f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float of_key(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(FULLM, v, o);
  return v;
}
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(FULLM, v, o);
  return v;
}
__device__ __forceinline__ float load_logit(const GateP &P, int row, int e) {
  const int64_t i = (int64_t)row * P.ld + e;
  if (P.bf16) return __uint_as_float((uint32_t)static_cast<const uint16_t *>(P.logits)[i] << 16);
  return static_cast<const float *>(P.logits)[i];
}
// How far a 32-bit selection score may be from the definition's: scores are
// at most 1, their exponential, sum and quotient are good to 2^-21 together,
// the sum with the bias to 2^-24 of itself.
__device__ __forceinline__ float tol_of(float sel) { return 9.5367431640625e-7f * (1.f + fabsf(sel)); }

// The row's choice in 64 bits; lane r < K ends with the r-th id (-1: none).
__device__ __noinline__ int gate_row64(const GateP &P, int row, double *sel) {
  const int lane = threadIdx.x & 31;
  const double ninf = -__longlong_as_double(0x7ff0000000000000ll);
  double m = ninf;
  for (int e = lane; e < P.E; e += 32) m = fmax(m, (double)load_logit(P, row, e));  // fmax drops NaN
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmax(m, __shfl_xor_sync(FULLM, m, o));
  double z = 0;
  for (int e = lane; e < P.E; e += 32) {
    const double l = load_logit(P, row, e);
    const float b = P.bias ? P.bias[e] : 0.f;
    double p = 0;
    if (l > ninf) p = P.sigmoid ? 1.0 / (1.0 + exp(-l)) : (m == -ninf ? (l == m ? 1.0 : 0.0) : exp(l - m));
    z += p;
    sel[e] = l > ninf && b > -kInf ? p : ninf;
  }
  z = warp_sum(z);
  __syncwarp();
  for (int e = lane; e < P.E; e += 32)
    if (sel[e] > ninf) sel[e] = (P.sigmoid ? sel[e] : sel[e] / z) + (P.bias ? (double)P.bias[e] : 0.0);
  __syncwarp();
  if (P.ng > 1) {
    double score = ninf;
    for (int g = 0; g < P.ng; g++) {
      double a = ninf, b = ninf;
      for (int e = g * P.gs + lane; e < (g + 1) * P.gs; e += 32) {
        const double v = sel[e];
        if (v > a) b = a, a = v;
        else if (v > b) b = v;
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) {
        const double oa = __shfl_xor_sync(FULLM, a, o), ob = __shfl_xor_sync(FULLM, b, o);
        b = fmax(fmin(a, oa), fmax(b, ob));
        a = fmax(a, oa);
      }
      if (lane == g) score = a > ninf && P.group_top == 2 && b > ninf ? a + b : a;
    }
    int rank = 0;
    for (int j = 0; j < P.ng; j++) {
      const double o = __shfl_sync(FULLM, score, j);
      rank += o > score || (o == score && j < lane);
    }
    const unsigned keep = __ballot_sync(FULLM, lane < P.ng && rank < P.top_groups);
    for (int e = lane; e < P.E; e += 32)
      if (!((keep >> (e / P.gs)) & 1u)) sel[e] = ninf;
  }
  // without a bias the logits order the experts (scores may underflow)
  if (!P.bias)
    for (int e = lane; e < P.E; e += 32)
      if (sel[e] > ninf) sel[e] = load_logit(P, row, e);
  __syncwarp();
  int mine = -1;
  for (int r = 0; r < P.K; r++) {
    double bv = ninf;
    int bi = 0x7fffffff;
    for (int e = lane; e < P.E; e += 32)
      if (sel[e] > bv) bv = sel[e], bi = e;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      const double ov = __shfl_xor_sync(FULLM, bv, o);
      const int oi = __shfl_xor_sync(FULLM, bi, o);
      if (ov > bv || (ov == bv && oi < bi)) bv = ov, bi = oi;
    }
    if (bv == ninf) break;
    if (lane == r) mine = bi;
    if (lane == (bi & 31)) sel[bi] = ninf;
    __syncwarp();
  }
  return mine;
}

template <int C>
__global__ void __launch_bounds__(32 * kGateWarps) gate_kernel(const __grid_constant__ GateP P) {
  extern __shared__ double sel64[];  // [kGateWarps][E]: rows decided in 64 bits
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row = blockIdx.x * kGateWarps + warp;
  if (row >= P.t) return;
  const int E = P.E, K = P.K, e0 = lane * C;

  float l[C];
  uint32_t key[C];
  float m = -kInf;
#pragma unroll
  for (int i = 0; i < C; i++) {
    l[i] = e0 + i < E ? load_logit(P, row, e0 + i) : -kInf;
    m = fmaxf(m, l[i]);
  }
  const bool biased = P.bias != nullptr;
  // scores: needed for the bias, the sums of a group, and the full softmax's weights
  const bool pair_groups = P.ng > 1 && P.group_top == 2;
  const bool scores = biased || pair_groups || (!P.sigmoid && !P.renorm);
  float z = 1.f;
  if (!P.sigmoid && scores) {
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(FULLM, m, o));
    z = 0.f;
#pragma unroll
    for (int i = 0; i < C; i++) {
      const float x = m == kInf ? (l[i] == kInf ? 0.f : -kInf) : l[i] - m;
      z += l[i] > -kInf ? expf(x) : 0.f;
    }
    z = warp_sum(z);
  }
  auto score_of = [&](float v) {
    if (P.sigmoid) return 1.f / (1.f + expf(-v));
    return expf(m == kInf ? (v == kInf ? 0.f : -kInf) : v - m) / z;
  };
#pragma unroll
  for (int i = 0; i < C; i++) {
    const float b = biased && e0 + i < E ? P.bias[e0 + i] : 0.f;
    key[i] = l[i] > -kInf && b > -kInf ? okey(biased ? score_of(l[i]) + b : l[i]) : 0u;
  }

  bool near = false;  // some comparison is too close for 32 bits
  if (P.ng > 1) {
    float score = -kInf;
    uint32_t top1 = 0, top2 = 0;
    for (int g = 0; g < P.ng; g++) {
      uint32_t a = 0, b = 0;
#pragma unroll
      for (int i = 0; i < C; i++) {
        const int e = e0 + i - g * P.gs;
        if ((unsigned)e < (unsigned)P.gs) {
          const uint32_t k = key[i];
          b = k > a ? a : (k > b ? k : b);
          a = k > a ? k : a;
        }
      }
      const uint32_t m1 = __reduce_max_sync(FULLM, a);
      const int src = __ffs(__ballot_sync(FULLM, a == m1)) - 1;
      const uint32_t m2 = __reduce_max_sync(FULLM, lane == src ? b : a);
      if (lane == g) top1 = m1, top2 = P.group_top == 2 ? m2 : 0u;
    }
    if (top1) {
      score = of_key(top1);
      if (pair_groups) {
        if (!biased) score = score_of(score);
        if (top2) score += biased ? of_key(top2) : score_of(of_key(top2));
      }
    }
    // rank among the groups; a kept and a dropped group within the error of
    // each other that are not the same numbers make the row a near one
    int rank = 0;
    for (int j = 0; j < P.ng; j++) {
      const float o = __shfl_sync(FULLM, score, j);
      rank += o > score || (o == score && j < lane);
    }
    const unsigned keep = __ballot_sync(FULLM, lane < P.ng && rank < P.top_groups);
    if (biased || pair_groups) {
      const bool kept = (keep >> lane) & 1u;
      bool close = false;
      for (int j = 0; j < P.ng; j++) {
        const float o = __shfl_sync(FULLM, score, j);
        const uint32_t o1 = __shfl_sync(FULLM, top1, j), o2 = __shfl_sync(FULLM, top2, j);
        if (kept && !((keep >> j) & 1u) && top1 && o1 && score - o <= 2.f * (tol_of(o) + tol_of(score)))
          close |= biased || o1 != top1 || o2 != top2;
      }
      near = __any_sync(FULLM, close);
    }
#pragma unroll
    for (int i = 0; i < C; i++)
      if (e0 + i < E && !((keep >> ((e0 + i) / P.gs)) & 1u)) key[i] = 0u;
  }

  uint32_t bk = 0;
  int bi = 0;
#pragma unroll
  for (int i = 0; i < C; i++)
    if (key[i] > bk) bk = key[i], bi = i;
  int mine = -1;
  uint32_t mykey = 0;
  if (!near) {
    for (int r = 0; r < K; r++) {
      const uint32_t mx = __reduce_max_sync(FULLM, bk);
      if (mx == 0) break;
      const int src = __ffs(__ballot_sync(FULLM, bk == mx)) - 1;
      const int id = __shfl_sync(FULLM, e0 + bi, src);
      if (lane == r) mine = id, mykey = mx;
      if (lane == src) {
        uint32_t nk = 0;
        int ni = 0;
#pragma unroll
        for (int i = 0; i < C; i++) {
          if (i == bi) key[i] = 0u;
          if (key[i] > nk) nk = key[i], ni = i;
        }
        bk = nk, bi = ni;
      }
    }
  }
  float lg = mine >= 0 ? load_logit(P, row, mine) : -kInf;
  if (biased && !near) {
    // the chosen ones among themselves, then what was left against the last
    // of them: two that are the same numbers are in order by their ids
    const float b = mine >= 0 ? P.bias[mine] : 0.f, sel = of_key(mykey);
    const float ps = __shfl_up_sync(FULLM, sel, 1), pl = __shfl_up_sync(FULLM, lg, 1), pb = __shfl_up_sync(FULLM, b, 1);
    bool c = lane > 0 && mine >= 0 && ps - sel <= tol_of(ps) + tol_of(sel) && !(pl == lg && pb == b);
    const float ls = __shfl_sync(FULLM, sel, K - 1), ll = __shfl_sync(FULLM, lg, K - 1), lb = __shfl_sync(FULLM, b, K - 1);
#pragma unroll
    for (int i = 0; i < C; i++)
      if (key[i]) {
        const float v = of_key(key[i]);
        if (ls - v <= tol_of(ls) + tol_of(v)) c |= !(l[i] == ll && P.bias[e0 + i] == lb);
      }
    near = __any_sync(FULLM, c);
  }
  if (near) {
    mine = gate_row64(P, row, sel64 + (size_t)warp * E);
    lg = mine >= 0 ? load_logit(P, row, mine) : -kInf;
  }

  // weights of the chosen experts (lane r: the r-th)
  const bool have = lane < K && mine >= 0;
  if (!have) lg = -kInf;
  float w = 0.f;
  float top = lg;
#pragma unroll
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(FULLM, top, o));
  if (P.renorm) {
    // softmax: exp(l - top) over their sum, whatever the full sum is; sigmoid
    // below e^-60 is exp(l) to 32 bits, so a common factor keeps it from 0
    if (have) {
      if (P.sigmoid && top > -60.f) w = 1.f / (1.f + expf(-lg));
      else w = expf(top == kInf ? (lg == kInf ? 0.f : -kInf) : lg - top);
    }
    const float sum = warp_sum(w);
    w = sum > 0.f ? w / sum : 0.f;
  } else if (have) {
    w = score_of(lg);
  }
  if (lane < K) {
    P.idx[(size_t)row * K + lane] = (uint32_t)mine;
    P.w[(size_t)row * K + lane] = w * P.scale;
  }
}

template <int C>
cudaError_t launch(const GateP &p, cudaStream_t st) {
  const size_t smem = (size_t)kGateWarps * p.E * 8;
  if (smem > 48 * 1024) return cudaErrorInvalidValue;  // E <= 1024: 32 KB
  gate_kernel<C><<<(unsigned)((p.t + kGateWarps - 1) / kGateWarps), 32 * kGateWarps, smem, st>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_gate(const GateP &p, cudaStream_t st) {
  if (p.E <= 64) return launch<2>(p, st);
  if (p.E <= 128) return launch<4>(p, st);
  if (p.E <= 256) return launch<8>(p, st);
  if (p.E <= 512) return launch<16>(p, st);
  return launch<32>(p, st);
}

}  // namespace moe
