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
  const uint32_t u = __float_as_uint(f + 0.f);  // -0 is 0
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
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
// How far a 32-bit selection score may be from the definition's, by the fast
// exponential (2 + 1.16 |x| ulp) and quotient (2 ulp).  Sigmoid: the score
// moves by p (1 - p) of the exponential's error, 0.6 ulp of 1 at most, and by
// the quotient's 2: below 2^-21 together.  Softmax: p |x| < 0.4 and the sum's
// error, at most that of the mean |x| < ln 1024, weigh in: below 2^-20.  The
// sum with the bias adds 2^-24 of itself.
__device__ __forceinline__ float tol_of(float sel, bool sigmoid) {
  return (sigmoid ? 4.76837158203125e-7f : 9.5367431640625e-7f) + 1.1920928955078125e-7f * fabsf(sel);
}

// unsigned key in the order of d (0 is left for what is masked)
__device__ __forceinline__ uint64_t okey64(double d) {
  const uint64_t u = (uint64_t)__double_as_longlong(d == 0.0 ? 0.0 : d);
  return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}
__device__ __forceinline__ double of_key64(uint64_t k) {
  return __longlong_as_double((long long)((k >> 63) ? (k & 0x7fffffffffffffffull) : ~k));
}
__device__ __forceinline__ uint64_t warp_max(uint64_t v) {
  const uint32_t hi = __reduce_max_sync(FULLM, (uint32_t)(v >> 32));
  const uint32_t lo = __reduce_max_sync(FULLM, (uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
  return (uint64_t)hi << 32 | lo;
}

// The whole row's choice in 64 bits; lane r < K ends with the r-th id (-1: none).
// Scores are computed in 64-bit floating point, of which this GPU does little;
// they are compared as integers.
__device__ __noinline__ int gate_row64(const GateP &P, int row, uint64_t *key) {
  const int lane = threadIdx.x & 31;
  float m = -kInf;
  for (int e = lane; e < P.E; e += 32) m = fmaxf(m, load_logit(P, row, e));  // fmaxf drops NaN
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(FULLM, m, o));
  double z = 0;
  for (int e = lane; e < P.E; e += 32) {
    const float l = load_logit(P, row, e);
    double p = 0;
    if (l > -kInf) p = P.sigmoid ? 1.0 / (1.0 + exp(-(double)l)) : (m == kInf ? (l == m ? 1.0 : 0.0) : exp((double)l - m));
    z += p;
    key[e] = (uint64_t)__double_as_longlong(p);
  }
  z = warp_sum(z);
  __syncwarp();
  for (int e = lane; e < P.E; e += 32) {
    const double p = __longlong_as_double((long long)key[e]);
    const float b = P.bias ? P.bias[e] : 0.f;
    key[e] = load_logit(P, row, e) > -kInf && b > -kInf ? okey64((P.sigmoid ? p : p / z) + (double)b) : 0ull;
  }
  __syncwarp();
  if (P.ng > 1) {
    uint64_t score = 0;
    for (int g = 0; g < P.ng; g++) {
      uint64_t a = 0, b = 0;
      for (int e = g * P.gs + lane; e < (g + 1) * P.gs; e += 32) {
        const uint64_t v = key[e];
        if (v > a) b = a, a = v;
        else if (v > b) b = v;
      }
      const uint64_t m1 = warp_max(a);
      const int src = __ffs(__ballot_sync(FULLM, a == m1)) - 1;
      const uint64_t m2 = warp_max(lane == src ? b : a);
      if (lane == g) score = m1 && P.group_top == 2 && m2 ? okey64(of_key64(m1) + of_key64(m2)) : m1;
    }
    int rank = 0;
    for (int j = 0; j < P.ng; j++) {
      const uint64_t o = __shfl_sync(FULLM, score, j);
      rank += o > score || (o == score && j < lane);
    }
    const unsigned keep = __ballot_sync(FULLM, lane < P.ng && rank < P.top_groups);
    for (int e = lane; e < P.E; e += 32)
      if (!((keep >> (e / P.gs)) & 1u)) key[e] = 0;
  }
  // without a bias the logits order the experts (scores may underflow)
  if (!P.bias)
    for (int e = lane; e < P.E; e += 32)
      if (key[e]) key[e] = okey64(load_logit(P, row, e));
  __syncwarp();
  int mine = -1;
  for (int r = 0; r < P.K; r++) {
    uint64_t bv = 0;
    int bi = 0x7fffffff;
    for (int e = lane; e < P.E; e += 32)
      if (key[e] > bv) bv = key[e], bi = e;
    const uint64_t mx = warp_max(bv);
    if (mx == 0) break;
    const int id = (int)__reduce_min_sync(FULLM, bv == mx ? (uint32_t)bi : 0x7fffffffu);
    if (lane == r) mine = id;
    if (lane == (id & 31)) key[id] = 0;
    __syncwarp();
  }
  return mine;
}

// The choice among up to 32 candidates in 64 bits, one a lane (id, or -1): an
// order of 32-bit scores that is right but for those too near one another.
// m, z: the row's largest logit and, in 64 bits, the sum of its exponentials
// (softmax).  Lane r < K ends with the r-th id.
__device__ __noinline__ int gate_candidates64(const GateP &P, int row, int id, int n, float m, double z, int *list) {
  const int lane = threadIdx.x & 31;
  uint64_t key = 0;
  if (id >= 0) {
    const float l = load_logit(P, row, id);
    const double p = P.sigmoid ? 1.0 / (1.0 + exp(-(double)l)) : (m == kInf ? (l == m ? 1.0 : 0.0) : exp((double)l - m)) / z;
    key = okey64(p + (double)P.bias[id]);
  }
  int rank = 0;
  for (int j = 0; j < n; j++) {
    const uint64_t o = __shfl_sync(FULLM, key, j);
    const int oi = __shfl_sync(FULLM, id, j);
    rank += o > key || (o == key && oi < id);
  }
  if (id >= 0) list[rank] = id;
  __syncwarp();
  id = lane < n ? list[lane] : -1;
  __syncwarp();
  return id;
}

// The C logits of lane `lane`, experts e0 .. e0 + C - 1; -inf past E.  VEC:
// rows start on 16 bytes and a lane's experts are all there or none are.
template <int C, bool VEC>
__device__ __forceinline__ void load_row(const GateP &P, int row, int e0, float (&l)[C]) {
  if (VEC && e0 >= P.E) {
#pragma unroll
    for (int i = 0; i < C; i++) l[i] = -kInf;
  } else if (VEC && P.bf16) {
    const uint16_t *p = static_cast<const uint16_t *>(P.logits) + (int64_t)row * P.ld + e0;
    uint32_t w[C / 2];
    if constexpr (C == 4) {
      const uint2 v = *reinterpret_cast<const uint2 *>(p);
      w[0] = v.x, w[1] = v.y;
    } else {
#pragma unroll
      for (int i = 0; i < C / 8; i++) {
        const uint4 v = reinterpret_cast<const uint4 *>(p)[i];
        w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
      }
    }
#pragma unroll
    for (int i = 0; i < C / 2; i++) l[2 * i] = bf16lo(w[i]), l[2 * i + 1] = bf16hi(w[i]);
  } else if (VEC) {
    const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(P.logits) + (int64_t)row * P.ld + e0);
#pragma unroll
    for (int i = 0; i < C / 4; i++) {
      const float4 v = p[i];
      l[4 * i] = v.x, l[4 * i + 1] = v.y, l[4 * i + 2] = v.z, l[4 * i + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < C; i++) l[i] = e0 + i < P.E ? load_logit(P, row, e0 + i) : -kInf;
  }
}

// What a warp does for a row is bound by its instructions: 65535 rows of 256
// experts in 8 groups with a bias take 85 us at 3.1 instructions a cycle and
// SM (some 1100 a row; the rows' 71 MB would take 10.5), 214 us with a full
// scan of the lane's experts per choice and per group.  So a lane keeps its
// best two keys: a choice costs a maximum over the warp, and a lane looks
// through its experts again only after two of them were taken; and where a
// lane's experts lie in one group (LPG lanes a group, 0: they do not) the
// group's best two come from those by a few exchanges.  Warps walk rows with their bias in registers.
template <int C, bool VEC>
__global__ void __launch_bounds__(32 * kGateWarps) gate_kernel(const __grid_constant__ GateP P) {
  extern __shared__ uint64_t key64[];  // [kGateWarps][E]: rows decided in 64 bits
  __shared__ uint2 picks[kGateWarps][32];  // the choices of a row: key, id
  pdl_wait_prev();
  pdl_launch_next();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int E = P.E, K = P.K, e0 = lane * C;
  const unsigned below = (1u << lane) - 1u;
  const bool biased = P.bias != nullptr;
  const bool pair_groups = P.ng > 1 && P.group_top == 2;
  // scores: needed for the bias, the sums of a group, and the full softmax's weights
  const bool scores = biased || pair_groups || (!P.sigmoid && !P.renorm);
  const int lpg = P.ng > 1 && P.gs % C == 0 && 32 % (P.gs / C) == 0 ? P.gs / C : 0;  // lanes of a group
  float bias[C];
#pragma unroll
  for (int i = 0; i < C; i++) bias[i] = biased && e0 + i < E ? fmaxf(P.bias[e0 + i], -kInf) : 0.f;  // NaN: -inf

  const int step = gridDim.x * kGateWarps;
  float next[C];
  if (blockIdx.x * kGateWarps + warp < P.t) load_row<C, VEC>(P, blockIdx.x * kGateWarps + warp, e0, next);
  for (int row = blockIdx.x * kGateWarps + warp; row < P.t; row += step) {
    float l[C];
#pragma unroll
    for (int i = 0; i < C; i++) l[i] = next[i];
    if (step < P.t - row) load_row<C, VEC>(P, row + step, e0, next);
    float m = -kInf, z = 1.f;
    if (!P.sigmoid && scores) {
#pragma unroll
      for (int i = 0; i < C; i++) m = fmaxf(m, l[i]);
#pragma unroll
      for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(FULLM, m, o));
      z = 0.f;
#pragma unroll
      for (int i = 0; i < C; i++) z += l[i] > -kInf ? __expf(m == kInf ? (l[i] == kInf ? 0.f : -kInf) : l[i] - m) : 0.f;
      z = warp_sum(z);
    }
    const float inv = 1.f / z;
    auto score_of = [&](float v) {
      if (P.sigmoid) return __fdividef(1.f, 1.f + __expf(-v));
      return __expf(m == kInf ? (v == kInf ? 0.f : -kInf) : v - m) * inv;
    };
    uint32_t key[C];
#pragma unroll
    for (int i = 0; i < C; i++) {
      float v = l[i];
      if (biased) v = score_of(v) + bias[i];
      key[i] = l[i] > -kInf && v > -kInf ? okey(v) : 0u;
    }
    // the lane's best two
    uint32_t b1 = 0, b2 = 0;
    int i1 = 0, i2 = 0;
#pragma unroll
    for (int i = 0; i < C; i++) {
      const bool g1 = key[i] > b1, g2 = key[i] > b2;
      b2 = g1 ? b1 : (g2 ? key[i] : b2), i2 = g1 ? i1 : (g2 ? i : i2);
      b1 = g1 ? key[i] : b1, i1 = g1 ? i : i1;
    }

    bool near = false;  // some comparison is too close for 32 bits
    if (P.ng > 1) {
      // lane g (of lpg lanes a group: every lane of the group) has the
      // group's best two keys
      uint32_t top1 = b1, top2 = b2;
      const int mine = lpg ? lane / lpg : lane;
      if (lpg) {
        for (int o = 1; o < lpg; o <<= 1) {
          const uint32_t o1 = __shfl_xor_sync(FULLM, top1, o), o2 = __shfl_xor_sync(FULLM, top2, o);
          top2 = max(min(top1, o1), max(top2, o2));
          top1 = max(top1, o1);
        }
      } else {
        uint32_t t1 = 0, t2 = 0;
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
          if (lane == g) t1 = m1, t2 = m2;
        }
        top1 = t1, top2 = t2;
      }
      if (P.group_top == 1) top2 = 0u;
      // The group's score, and how far it may be from the definition's: the
      // errors of its terms (a bias of each sign may cancel in the sum, the
      // roundings it brought do not) and the sum's own rounding.  A term that
      // is infinite makes the score exact; a sum past the 32-bit range is left
      // to 64.
      float score = -kInf, gtol = 0.f;
      bool over = false;
      if (top1) {
        score = of_key(top1);
        if (pair_groups) {
          if (!biased) score = score_of(score);
          gtol = tol_of(score, P.sigmoid);
          if (top2) {
            const float s1 = score, s2 = biased ? of_key(top2) : score_of(of_key(top2));
            gtol += tol_of(s2, P.sigmoid);
            score += s2;
            over = fabsf(score) == kInf && s1 < kInf;
          }
          gtol += 1.1920928955078125e-7f * fabsf(score);
        } else {
          gtol = tol_of(score, P.sigmoid);
        }
        if (score == kInf && !over) gtol = 0.f;
      }
      const int lanes = lpg ? lpg : 1;
      int rank = 0;
      for (int j = 0; j < P.ng; j++) {
        const float o = __shfl_sync(FULLM, score, j * lanes);
        rank += o > score || (o == score && j < mine);
      }
      const bool kept = mine < P.ng && rank < P.top_groups;
      if (biased || pair_groups) {
        // the lowest kept and the highest dropped score; where they are
        // within the largest error of each other, every such pair within its
        // own that is not the same numbers makes the row a near one
        const uint32_t lo = __reduce_min_sync(FULLM, kept && top1 ? okey(score) : 0xffffffffu);
        const uint32_t hi = __reduce_max_sync(FULLM, mine < P.ng && !kept && top1 ? okey(score) : 0u);
        const float tmax = __uint_as_float(__reduce_max_sync(FULLM, mine < P.ng ? __float_as_uint(gtol) : 0u));
        near = __any_sync(FULLM, mine < P.ng && over);
        if (!near && lo != 0xffffffffu && hi) {
          if (!(of_key(lo) - of_key(hi) > 2.f * tmax)) {
            bool close = false;
            for (int j = 0; j < P.ng; j++) {
              const float o = __shfl_sync(FULLM, score, j * lanes), ot = __shfl_sync(FULLM, gtol, j * lanes);
              const uint32_t o1 = __shfl_sync(FULLM, top1, j * lanes), o2 = __shfl_sync(FULLM, top2, j * lanes);
              const int ok = __shfl_sync(FULLM, kept ? 1 : 0, j * lanes);
              if (kept && !ok && top1 && o1 && !(score - o > gtol + ot))
                close |= biased || o1 != top1 || o2 != top2;
            }
            near = __any_sync(FULLM, close);
          }
        }
      }
      if (lpg) {
        if (!kept) {
          b1 = b2 = 0u;
#pragma unroll
          for (int i = 0; i < C; i++) key[i] = 0u;
        }
      } else {
        const unsigned keep = __ballot_sync(FULLM, kept);
        b1 = b2 = 0u, i1 = i2 = 0;
#pragma unroll
        for (int i = 0; i < C; i++) {
          if (e0 + i < E && !((keep >> ((e0 + i) / P.gs)) & 1u)) key[i] = 0u;
          const bool g1 = key[i] > b1, g2 = key[i] > b2;
          b2 = g1 ? b1 : (g2 ? key[i] : b2), i2 = g1 ? i1 : (g2 ? i : i2);
          b1 = g1 ? key[i] : b1, i1 = g1 ? i : i1;
        }
      }
    }

    int mine = -1;
    uint32_t mykey = 0, taken = 0;
    bool second = true;  // (b2, i2) is the best after (b1, i1)
    if (!near) {
      int r = 0;
      for (; r < K; r++) {
        const uint32_t mx = __reduce_max_sync(FULLM, b1);
        if (mx == 0) break;
        // the first lane that has it: the lowest id
        const bool has = b1 == mx;
        const unsigned who = __ballot_sync(FULLM, has);
        if (has && (who & below) == 0) {
          picks[warp][r] = make_uint2(mx, (uint32_t)(e0 + i1));
          taken |= 1u << i1;
          if (second) {
            b1 = b2, i1 = i2, second = false;
          } else {
            b1 = 0u, i1 = 0;
#pragma unroll
            for (int i = 0; i < C; i++) {
              const uint32_t k = (taken >> i) & 1u ? 0u : key[i];
              if (k > b1) b1 = k, i1 = i;
            }
          }
        }
        __syncwarp();
      }
      if (lane < r) mykey = picks[warp][lane].x, mine = (int)picks[warp][lane].y;
      __syncwarp();
    }
    float lg = -kInf;
    if (biased) {
      lg = mine >= 0 ? load_logit(P, row, mine) : -kInf;
      if (!near) {
        // the chosen ones among themselves, then what was left against the
        // last of them: two that are the same numbers are in order by their ids
        const float b = mine >= 0 ? P.bias[mine] : 0.f, sel = of_key(mykey);
        const float ps = __shfl_up_sync(FULLM, sel, 1), pl = __shfl_up_sync(FULLM, lg, 1), pb = __shfl_up_sync(FULLM, b, 1);
        bool c = lane > 0 && mine >= 0 && ps - sel <= tol_of(ps, P.sigmoid) + tol_of(sel, P.sigmoid) && !(pl == lg && pb == b);
        const float ls = __shfl_sync(FULLM, sel, K - 1), ll = __shfl_sync(FULLM, lg, K - 1), lb = __shfl_sync(FULLM, b, K - 1);
        const bool full = __shfl_sync(FULLM, mine, K - 1) >= 0;  // (fewer than K: nothing is left)
        const float v1 = of_key(b1);
        unsigned reach = 0;  // what was left within reach of the last
        if (__any_sync(FULLM, full && b1 && ls - v1 <= tol_of(ls, P.sigmoid) + tol_of(v1, P.sigmoid))) {
#pragma unroll
          for (int i = 0; i < C; i++)
            if (key[i] && !((taken >> i) & 1u)) {
              const float v = of_key(key[i]);
              if (ls - v <= tol_of(ls, P.sigmoid) + tol_of(v, P.sigmoid)) {
                reach |= 1u << i;
                c |= !(l[i] == ll && bias[i] == lb);
              }
            }
        }
        if (__any_sync(FULLM, c)) {
          // the chosen and those within reach, decided in 64 bits: a lane each
          int *list = reinterpret_cast<int *>(key64 + (size_t)warp * E);
          int n = __popc(__ballot_sync(FULLM, mine >= 0)), extra = __popc(reach), x = extra;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(FULLM, x, o);
            if (lane >= o) x += y;
          }
          const int total = n + __shfl_sync(FULLM, x, 31);
          if (total <= 32 && E >= 16) {
            int at = n + x - extra;
            for (unsigned left = reach; left; left &= left - 1) list[at++] = e0 + __ffs(left) - 1;
            __syncwarp();
            const int id = lane < n ? mine : (lane < total ? list[lane] : -1);
            __syncwarp();
            double z64 = 1.0;
            if (!P.sigmoid) {
              z64 = 0.0;
#pragma unroll
              for (int i = 0; i < C; i++)
                if (l[i] > -kInf) z64 += m == kInf ? (l[i] == kInf ? 1.0 : 0.0) : exp((double)l[i] - m);
              z64 = warp_sum(z64);
            }
            mine = gate_candidates64(P, row, id, total, m, z64, list);
            if (lane >= K) mine = -1;
            lg = mine >= 0 ? load_logit(P, row, mine) : -kInf;
          } else {
            near = true;
          }
        }
      }
    } else if (mine >= 0) {
      lg = of_key(mykey);
    }
    if (near) {
      __syncwarp();
      mine = gate_row64(P, row, key64 + (size_t)warp * E);
      __syncwarp();
      lg = mine >= 0 ? load_logit(P, row, mine) : -kInf;
    }

    // weights of the chosen experts (lane r: the r-th)
    const bool have = lane < K && mine >= 0;
    if (!have) lg = -kInf;
    float w = 0.f;
    if (P.renorm) {
      // softmax: exp(l - top) over their sum, whatever the full sum is; sigmoid
      // below e^-60 is exp(l) to 32 bits, so a common factor keeps it from 0
      float top = lg;
#pragma unroll
      for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(FULLM, top, o));
      if (have) {
        if (P.sigmoid && top > -60.f) w = 1.f / (1.f + expf(-lg));
        else w = expf(top == kInf ? (lg == kInf ? 0.f : -kInf) : lg - top);
      }
      const float sum = warp_sum(w);
      w = sum > 0.f ? w / sum : 0.f;
    } else if (have) {
      w = P.sigmoid ? 1.f / (1.f + expf(-lg)) : expf(m == kInf ? (lg == kInf ? 0.f : -kInf) : lg - m) / z;
    }
    if (lane < K) {
      P.idx[(size_t)row * K + lane] = (uint32_t)mine;
      P.w[(size_t)row * K + lane] = w * P.scale;
    }
  }
}

template <int C>
cudaError_t launch(const GateP &p, int n_sms, cudaStream_t st) {
  const size_t smem = (size_t)kGateWarps * p.E * 8;
  if (smem > 48 * 1024) return cudaErrorInvalidValue;  // E <= 1024: 32 KB
  const int size = p.bf16 ? 2 : 4;
  const bool vec = p.E % C == 0 && (p.ld * size) % 16 == 0 && (reinterpret_cast<uintptr_t>(p.logits) & 15) == 0;
  const int64_t need = ((int64_t)p.t + kGateWarps - 1) / kGateWarps, cap = (int64_t)n_sms * 64;
  const unsigned grid = (unsigned)(need < cap ? need : cap);
  return launch_pdl(vec ? gate_kernel<C, true> : gate_kernel<C, false>, dim3(grid), 32 * kGateWarps, smem, st, p);
}

}  // namespace

cudaError_t launch_gate(const GateP &p, int n_sms, cudaStream_t st) {
  if (p.E <= 128) return launch<4>(p, n_sms, st);
  if (p.E <= 256) return launch<8>(p, n_sms, st);
  if (p.E <= 512) return launch<16>(p, n_sms, st);
  return launch<32>(p, n_sms, st);
}

}  // namespace moe
