// logprobs.cu -- per row of logits l: log probabilities of given tokens, the
// entropy and the top_k tokens, p = softmax(scale * l).
//
// One pass over the row: every thread keeps a reference value (the largest
// logit that it knew of when it last moved it), s0 = sum of 2^u and s1 = sum
// of u 2^u with u = (l - reference) * scale * log2(e).  Then
//   log Z = ln(s0),  entropy = ln(2) (log2 s0 - s1 / s0),
// both whatever the reference.  Moving it by d: s1 = 2^-d (s1 - d s0), s0 =
// 2^-d s0.  The top_k tokens are the largest 64-bit keys (the logit in the
// order of unsigned numbers, then the complement of the id): a threshold that
// at least top_k of the row reach (of the maxima of 32 groups of the first
// values the top_k-th) lets only few values into a list in shared memory,
// which is cut to its largest 32 whenever it fills, raising the threshold.
//
// A row is a cluster of S blocks (few rows) or one block; the blocks' sums
// and lists meet in the first one's shared memory.  The bound is HBM; per
// value some eight instructions.
#include <cuda_runtime.h>

#include "block.cuh"
#include "fp8.cuh"
#include "tc05.cuh"

namespace moe {
namespace {

constexpr unsigned FULLM = 0xffffffffu;
constexpr float kInf = __builtin_huge_valf();
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kU = 4;         // 16-byte chunks of a thread in flight
constexpr int kSlack = 1024;  // list entries beyond what one chunk a thread can add
constexpr int kMaxS = 8;

typedef unsigned long long key_t64;

__device__ __forceinline__ uint32_t okey(float f) {
  const uint32_t u = __float_as_uint(f + 0.f);  // -0 is 0
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float of_okey(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ key_t64 shfl_xor64(key_t64 v, int m) {
  return (key_t64)__shfl_xor_sync(FULLM, (unsigned)(v >> 32), m) << 32 | __shfl_xor_sync(FULLM, (unsigned)v, m);
}

// Warp: 32 keys, one a lane, into descending order (a bitonic network), and
// the largest 32 of two such lists.
__device__ __forceinline__ key_t64 exchange(key_t64 v, int j, bool larger) {
  const key_t64 o = shfl_xor64(v, j);
  return (o > v) == larger ? o : v;
}
__device__ __forceinline__ key_t64 sort32(key_t64 v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int n = 2; n <= 32; n *= 2)
#pragma unroll
    for (int j = n / 2; j; j /= 2) v = exchange(v, j, ((lane & j) == 0) == ((lane & n) == 0 || n == 32));
  return v;
}
__device__ __forceinline__ key_t64 merge32(key_t64 a, key_t64 b) {
  const int lane = threadIdx.x & 31;
  const key_t64 r = (key_t64)__shfl_sync(FULLM, (unsigned)(b >> 32), 31 - lane) << 32 | __shfl_sync(FULLM, (unsigned)b, 31 - lane);
  key_t64 v = a > r ? a : r;
#pragma unroll
  for (int j = 16; j; j /= 2) v = exchange(v, j, (lane & j) == 0);
  return v;
}

// What a thread, a block or a row has summed.  ref: the reference logit (-inf:
// nothing yet); mu = ref * c, in 32 bits, is what the sums are relative to
// unless it is so large that l * c may overflow: then they are to ref itself.
struct Sums {
  float ref, mu, s0, s1;
  bool big;
};
__device__ __forceinline__ void set_ref(Sums &a, float ref, float c) {
  a.ref = ref, a.mu = ref * c, a.big = !(fabsf(a.mu) < 1e30f);
}
// how far (in powers of two, 0 or below) a's reference lies below one at M
__device__ __forceinline__ float below(const Sums &a, const Sums &M, float c) {
  const float d = a.ref == M.ref ? 0.f : (a.big || M.big ? (a.ref - M.ref) * c : a.mu - M.mu);
  return fmaxf(d, -300.f);
}
__device__ __forceinline__ void move_to(Sums &a, const Sums &M, float c) {
  const float d = below(a, M, c), w = ex2(d);
  a.s1 = w * fmaf(d, a.s0, a.s1), a.s0 *= w;
  a.ref = M.ref, a.mu = M.mu, a.big = M.big;
}

template <bool BF16>
struct Chunk {
  static constexpr int n = BF16 ? 8 : 4;
  static __device__ __forceinline__ void unpack(const uint4 &r, float (&v)[n]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int j = 0; j < 4; j++) {
      if constexpr (BF16) v[2 * j] = bf16lo(w[j]), v[2 * j + 1] = bf16hi(w[j]);
      else v[j] = __uint_as_float(w[j]);
    }
  }
  static __device__ __forceinline__ float load1(const void *p, int64_t i) {
    if constexpr (BF16) return __uint_as_float((uint32_t)static_cast<const uint16_t *>(p)[i] << 16);
    else return static_cast<const float *>(p)[i];
  }
};

template <bool BF16, int T>
__global__ void __launch_bounds__(T) logprobs_rows(const __grid_constant__ LogprobsP P) {
  using C = Chunk<BF16>;
  constexpr int CH = C::n, W = T / 32, kCap = T * CH + kSlack, kSize = BF16 ? 2 : 4;
  __shared__ key_t64 s_list[kCap];
  __shared__ key_t64 s_top[W][32], s_lists[kMaxS][32];  // of the block's warps, of the row's blocks
  __shared__ key_t64 s_tau;
  __shared__ float s_gm[32], s_ref[32], s_s0[32], s_s1[32];
  __shared__ int s_cnt, s_inf[32];
  __shared__ float s_rank[kMaxS][4];  // of the row's blocks: reference, s0, s1, infinities
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_wait_prev();
  pdl_launch_next();
  if (P.S > 1) tc05::cluster_arrive();
  const int S = P.S, rank = S > 1 ? (int)tc05::cluster_rank() : 0;
  const int64_t row = blockIdx.x / S;
  const float c = P.scale * kLog2e;
  const uint8_t *base = static_cast<const uint8_t *>(P.x) + row * P.ld * kSize;
  const int lo = min(P.v, rank * P.seg), len = min(P.v, lo + P.seg) - lo;
  // the block's values in 16-byte chunks: the first may start before lo
  const uint8_t *at = base + (int64_t)lo * kSize;
  const int off = (int)(((uintptr_t)at & 15u) / kSize), nch = (len + off + CH - 1) / CH;
  const uint4 *chunks = reinterpret_cast<const uint4 *>(at - off * kSize);
  const int niter = (nch + T * kU - 1) / (T * kU);

  float tok = 0.f;  // this thread's first given token
  int tok_id = -1;
  if (rank == 0 && tid < P.m) {
    tok_id = P.tokens[row * P.m + tid];
    if ((unsigned)tok_id < (unsigned)P.v) tok = C::load1(base, tok_id);
  }

  auto load = [&](uint4 (&r)[kU], int it) {
#pragma unroll
    for (int u = 0; u < kU; u++) {
      const int i = (it * kU + u) * T + tid, first = i * CH - off;
      if (first >= 0 && first + CH <= len) {
        r[u] = ldg_stream4(chunks + i);
      } else {  // edges, value by value; NaN (masked) outside
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; j++) {
          if constexpr (BF16) {
            uint32_t h[2];
#pragma unroll
            for (int e = 0; e < 2; e++) {
              const int x = first + 2 * j + e;
              h[e] = x >= 0 && x < len ? reinterpret_cast<const uint16_t *>(at)[x] : 0x7fffu;
            }
            w[j] = h[0] | h[1] << 16;
          } else {
            const int x = first + j;
            w[j] = x >= 0 && x < len ? reinterpret_cast<const uint32_t *>(at)[x] : 0x7fffffffu;
          }
        }
        r[u] = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  };
  auto max_of = [&](const float (&v)[CH]) {
    float m = -kInf;
#pragma unroll
    for (int e = 0; e < CH; e++) m = fmaxf(m, v[e]);  // drops NaN
    return m;
  };

  uint4 cur[kU], nxt[kU];
  load(cur, 0);
  if (tid == 0) s_cnt = 0;
  // ---- the first values: the reference, and a first threshold
  Sums sum;
  key_t64 tau = 0;
  {
    float m = -kInf;
#pragma unroll
    for (int u = 0; u < kU; u++) {
      float v[CH];
      C::unpack(cur[u], v);
      m = fmaxf(m, max_of(v));
    }
    constexpr int per = T / 32;  // threads of a group
#pragma unroll
    for (int o = 1; o < per && o < 32; o *= 2) m = fmaxf(m, __shfl_xor_sync(FULLM, m, o));
    if (lane % per == 0) s_gm[tid / per] = m;
    __syncthreads();
    const float g = s_gm[lane];
    float b = g;
#pragma unroll
    for (int o = 16; o; o >>= 1) b = fmaxf(b, __shfl_xor_sync(FULLM, b, o));
    set_ref(sum, b, c);
    sum.s0 = sum.s1 = 0.f;
    if (P.k > 0) {
      int r = 0;
#pragma unroll
      for (int j = 0; j < 32; j++) {
        const float o = __shfl_sync(FULLM, g, j);
        r += o > g || (o == g && j < lane);
      }
      const unsigned who = __ballot_sync(FULLM, r == P.k - 1);
      const float t = __shfl_sync(FULLM, g, __ffs(who) - 1);
      if (t > -kInf) tau = (key_t64)okey(t) << 32;
    }
  }
  if (tid == 0) s_tau = tau;
  float tau_v = tau ? of_okey((uint32_t)(tau >> 32)) : -kInf;
  int seen = 0;  // entries of the list, as far as this thread's own places tell

  // values of a chunk that pass the threshold, into the list
  auto push = [&](const uint4 &r, int i) {
    float v[CH];
    C::unpack(r, v);
#pragma unroll
    for (int e = 0; e < CH; e++) {
      if (v[e] >= tau_v && v[e] > -kInf) {
        const key_t64 key = (key_t64)okey(v[e]) << 32 | (uint32_t)~(uint32_t)(lo + i * CH - off + e);
        if (key > tau) {
          const int n = atomicAdd(&s_cnt, 1);
          if (n < kCap) s_list[n] = key;
          seen = n + 1;
        }
      }
    }
  };
  // All threads: the list's largest 32 become the list.  [drop0, drop1): ids
  // that are left out.
  auto compact = [&](int drop0, int drop1) {
    const int n = min(s_cnt, kCap);
    key_t64 r = 0;
    for (int b = warp * 32; b < n; b += T) {
      key_t64 x = b + lane < n ? s_list[b + lane] : 0;
      const int id = (int)~(uint32_t)x - lo;
      if (x && id >= drop0 && id < drop1) x = 0;
      r = merge32(r, sort32(x));
    }
    s_top[warp][lane] = r;
    __syncthreads();
#pragma unroll
    for (int s = W / 2; s; s /= 2) {
      if (warp < s) s_top[warp][lane] = r = merge32(r, s_top[warp + s][lane]);
      __syncthreads();
    }
    if (warp == 0) {
      s_list[lane] = r;
      const unsigned any = __ballot_sync(FULLM, r != 0);
      if (lane == 0) s_cnt = __popc(any);
      if (lane == P.k - 1 && r > s_tau) s_tau = r;
    }
    __syncthreads();
    tau = s_tau;
    tau_v = tau ? of_okey((uint32_t)(tau >> 32)) : -kInf;
    seen = 0;
  };

  for (int it = 0; it < niter; it++) {
    if (it + 1 < niter) load(nxt, it + 1);
#pragma unroll
    for (int u = 0; u < kU; u++) {
      float v[CH];
      C::unpack(cur[u], v);
      const float m = max_of(v);
      if (m > sum.ref) {
        Sums to;
        set_ref(to, m, c);
        move_to(sum, to, c);
      }
      if (!sum.big) {
#pragma unroll
        for (int e = 0; e < CH; e++) {
          const float x = fmaxf(fmaf(v[e], c, -sum.mu), -200.f), p = ex2(x);  // masked values: 2^-200 is 0
          sum.s0 += p, sum.s1 = fmaf(p, x, sum.s1);
        }
      } else {
#pragma unroll
        for (int e = 0; e < CH; e++) {
          const float x = fmaxf((v[e] - sum.ref) * c, -200.f), p = ex2(x);
          sum.s0 += p, sum.s1 = fmaf(p, x, sum.s1);
        }
      }
      if (P.k > 0 && m >= tau_v) push(cur[u], (it * kU + u) * T + tid);
    }
    if (P.k > 0 && __syncthreads_or(seen > kSlack)) {
      // the list is long: cut it, and if it did not hold all of these values,
      // take them again a chunk at a time
      const bool over = s_cnt > kCap;
      const int d0 = it * kU * T * CH - off, d1 = d0 + kU * T * CH;
      __syncthreads();
      compact(over ? d0 : 0, over ? d1 : 0);
      if (over)
#pragma unroll 1
        for (int u = 0; u < kU; u++) {
          push(u == 0 ? cur[0] : (u == 1 ? cur[1] : (u == 2 ? cur[2] : cur[3])), (it * kU + u) * T + tid);
          __syncthreads();
          compact(0, 0);
        }
    }
#pragma unroll
    for (int u = 0; u < kU; u++) cur[u] = nxt[u];
  }

  // ---- the block's sums and list
  float m = sum.ref;
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(FULLM, m, o));
  if (lane == 0) s_ref[warp] = m;
  __syncthreads();
  m = lane < W ? s_ref[lane] : -kInf;
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(FULLM, m, o));
  Sums all;
  set_ref(all, m, c);
  move_to(sum, all, c);
  int ninf = 0;
  if (m == kInf)  // p is shared by the infinities
    for (int i = tid; i < len; i += T) ninf += C::load1(at, i) == kInf;
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    sum.s0 += __shfl_xor_sync(FULLM, sum.s0, o);
    sum.s1 += __shfl_xor_sync(FULLM, sum.s1, o);
    ninf += __shfl_xor_sync(FULLM, ninf, o);
  }
  if (lane == 0) s_s0[warp] = sum.s0, s_s1[warp] = sum.s1, s_inf[warp] = ninf;
  if (P.k > 0) compact(0, 0);  // begins after a barrier of its own: the list's last entries are there
  __syncthreads();
  if (warp == 0) {
    all.s0 = lane < W ? s_s0[lane] : 0.f, all.s1 = lane < W ? s_s1[lane] : 0.f;
    ninf = lane < W ? s_inf[lane] : 0;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      all.s0 += __shfl_xor_sync(FULLM, all.s0, o);
      all.s1 += __shfl_xor_sync(FULLM, all.s1, o);
      ninf += __shfl_xor_sync(FULLM, ninf, o);
    }
  }
  __shared__ float s_row[4];  // the row's: reference, log Z relative to it
  key_t64 top = 0;
  if (S > 1) {
    tc05::cluster_wait();  // every block of the row has begun: its shared memory can be written
    if (warp == 0) {
      tc05::st_cluster(tc05::map_rank(&s_lists[rank][lane], 0), P.k > 0 ? s_list[lane] : 0ull);
      if (lane == 0) {
        const uint32_t f = tc05::map_rank(&s_rank[rank][0], 0);
        tc05::st_cluster(f, all.ref), tc05::st_cluster(f + 4, all.s0), tc05::st_cluster(f + 8, all.s1);
        tc05::st_cluster(f + 12, (float)ninf);
      }
    }
    __syncwarp();
    tc05::cluster_sync();
    if (rank != 0) return;
    if (warp == 0) {
      Sums a;
      const int r = lane < S ? lane : 0;
      set_ref(a, lane < S ? s_rank[r][0] : -kInf, c);
      a.s0 = lane < S ? s_rank[r][1] : 0.f, a.s1 = lane < S ? s_rank[r][2] : 0.f;
      float fi = lane < S ? s_rank[r][3] : 0.f;
      float mm = a.ref;
#pragma unroll
      for (int o = kMaxS / 2; o; o >>= 1) mm = fmaxf(mm, __shfl_xor_sync(FULLM, mm, o));
      mm = __shfl_sync(FULLM, mm, 0);
      set_ref(all, mm, c);
      move_to(a, all, c);
      all.s0 = a.s0, all.s1 = a.s1;
#pragma unroll
      for (int o = kMaxS / 2; o; o >>= 1) {
        all.s0 += __shfl_xor_sync(FULLM, all.s0, o);
        all.s1 += __shfl_xor_sync(FULLM, all.s1, o);
        fi += __shfl_xor_sync(FULLM, fi, o);
      }
      all.s0 = __shfl_sync(FULLM, all.s0, 0), all.s1 = __shfl_sync(FULLM, all.s1, 0);
      ninf = (int)__shfl_sync(FULLM, fi, 0);
      for (int b = 0; b < S; b++) top = merge32(top, s_lists[b][lane]);
    }
  } else if (warp == 0 && P.k > 0) {
    top = s_list[lane];
  }
  // ---- the answers
  if (warp == 0) {
    float lz, h;
    if (all.ref == kInf) {
      lz = logf((float)ninf), h = lz;
    } else if (all.s0 > 0.f) {
      const float l2 = log2f(all.s0);
      // relative to ref: mu is ref * c rounded
      lz = kLn2 * (all.big ? l2 : l2 + fmaf(-all.ref, c, all.mu)), h = kLn2 * (l2 - all.s1 / all.s0);
    } else {
      lz = 0.f, h = 0.f;
    }
    if (lane == 0) {
      s_row[0] = all.ref, s_row[1] = lz;
      if (P.entropy) P.entropy[row] = fmaxf(h, 0.f);
    }
    auto logp = [&](float x) { return x == all.ref ? -lz : fmaf(P.scale, x - all.ref, -lz); };
    if (lane < P.k) {
      const float x = of_okey((uint32_t)(top >> 32));
      P.top_idx[row * P.k + lane] = top ? ~(uint32_t)top : 0xffffffffu;
      P.top_logp[row * P.k + lane] = top ? logp(x) : -kInf;
    }
  }
  __syncthreads();
  const float ref = s_row[0], lz = s_row[1];
  for (int i = tid; i < P.m; i += T) {
    if (i >= T) {
      tok_id = P.tokens[row * P.m + i];
      if ((unsigned)tok_id < (unsigned)P.v) tok = C::load1(base, tok_id);
    }
    const bool in = (unsigned)tok_id < (unsigned)P.v && tok > -kInf;  // false for NaN
    P.logp[row * P.m + i] = !in ? -kInf : (tok == ref ? -lz : fmaf(P.scale, tok - ref, -lz));
  }
}

template <bool BF16, int T>
cudaError_t launch_t(const LogprobsP &p, cudaStream_t st) {
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = (unsigned)p.S, at[1].val.clusterDim.y = 1, at[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((int64_t)p.t * p.S));
  cfg.blockDim = dim3(T);
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = p.S > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, logprobs_rows<BF16, T>, p);
}

}  // namespace

cudaError_t launch_logprobs(LogprobsP p, int n_sms, cudaStream_t st) {
  // few rows: as many blocks a row as fill the SMs, of 4096 values or more
  p.S = 1;
  while (p.S < kMaxS && (int64_t)p.t * p.S * 2 <= 2 * n_sms && p.v / (p.S * 2) >= 4096) p.S *= 2;
  p.seg = ((p.v + p.S - 1) / p.S + 7) / 8 * 8;
  if (p.seg <= 2048) return p.bf16 ? launch_t<true, 128>(p, st) : launch_t<false, 128>(p, st);
  if (p.seg <= 8192) return p.bf16 ? launch_t<true, 256>(p, st) : launch_t<false, 256>(p, st);
  return p.bf16 ? launch_t<true, 512>(p, st) : launch_t<false, 512>(p, st);
}

}  // namespace moe
