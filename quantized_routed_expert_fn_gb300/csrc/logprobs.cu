// logprobs.cu -- per row of logits l: log probabilities of given tokens, the
// entropy and the top_k tokens, p = softmax(scale * l).
//
// One pass over the row: every thread keeps a reference value (the largest
// logit that it knew of when it last moved it), s0 = sum of 2^u and s1 = sum
// of u 2^u with u = (l - reference) * scale * log2(e).  Then
//   log Z = ln(s0),  entropy = ln(2) (log2 s0 - s1 / s0),
// both whatever the reference.  Moving it by d: s1 = 2^-d (s1 - d s0), s0 =
// 2^-d s0.  The top_k tokens are the largest 64-bit keys (the logit in the
// order of unsigned numbers, then the complement of the id).  Each thread keeps
// the largest value it saw; at least top_k of the row reach the top_k-th of
// those, and only threads whose own does have such values: those threads'
// values are looked at again, by the whole block, and the ones that reach it
// go through lists in shared memory that are cut to their largest 32.  (With
// candidates collected in the one pass, 4096 rows of 131072 with top 5 took half
// as long again.)
//
// A row is a cluster of S blocks (few rows) or one block; the blocks' sums
// and lists meet in the first one's shared memory.  The bound is HBM, beside
// some six instructions a value: 4096 x 131072 bf16, top 5, 175 us, 6.1 TB/s (without
// alternatives 158, 6.8); 1 x 131072 fp32, top 20: 7.6, of which launch, the
// orders and exchanges are nearly all.
#include <cuda_runtime.h>
#include <type_traits>

#include "block.cuh"
#include "fp8.cuh"
#include "tc05.cuh"

namespace moe {
namespace {

constexpr unsigned FULLM = 0xffffffffu;
constexpr float kInf = __builtin_huge_valf();
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kMaxS = 8;
constexpr int kFetch = 32 * 1024;

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
__device__ __forceinline__ key_t64 shfl_xor_of(key_t64 v, int m) {
  return (key_t64)__shfl_xor_sync(FULLM, (unsigned)(v >> 32), m) << 32 | __shfl_xor_sync(FULLM, (unsigned)v, m);
}
__device__ __forceinline__ uint32_t shfl_xor_of(uint32_t v, int m) { return __shfl_xor_sync(FULLM, v, m); }

// Warp: 32 keys, one a lane, into descending order (a bitonic network), and
// the largest 32 of two such lists.
template <class K>
__device__ __forceinline__ K exchange(K v, int j, bool larger) {
  const K o = shfl_xor_of(v, j);
  return (o > v) == larger ? o : v;
}
template <class K>
__device__ __forceinline__ K sort32(K v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int n = 2; n <= 32; n *= 2)
#pragma unroll
    for (int j = n / 2; j; j /= 2) v = exchange(v, j, ((lane & j) == 0) == ((lane & n) == 0 || n == 32));
  return v;
}
template <class K>
__device__ __forceinline__ K merge32(K a, K b) {
  const int lane = threadIdx.x & 31;
  const K r = shfl_xor_of(b, 31);  // the other way round
  K v = a > r ? a : r;
#pragma unroll
  for (int j = 16; j; j /= 2) v = exchange(v, j, (lane & j) == 0);
  return v;
}
// Block: the largest 32 of n sorted lists (a power of two of them, no more
// than the block's warps), into the first; mine: this warp's list (warps from n
// on: anything).
template <class K>
__device__ __forceinline__ void merge_lists(K (*lists)[32], int n, K mine) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp < n) lists[warp][lane] = mine;
  __syncthreads();
  for (n /= 2; n; n /= 2) {
    if (warp < n) lists[warp][lane] = mine = merge32(mine, lists[warp + n][lane]);
    __syncthreads();
  }
}

// What a thread, a block or a row has summed.  ref: the reference logit (-inf:
// nothing yet); mu = ref * c, rounded to 32 bits, is what the sums are relative
// to (a term is then one multiply-add) as long as its rounding stays small: of
// 2^20 it is up to 2^-5 of a power of two, of 2^32 more than the exponents
// hold.  From 2^20 on (masks, large logits or scales) they are to ref itself.
struct Sums {
  float ref, mu, s0, s1;
  bool big;
};
__device__ __forceinline__ void set_ref(Sums &a, float ref, float c) {
  a.ref = ref, a.mu = ref * c, a.big = !(fabsf(a.mu) < 1048576.f);
}
// how far ref * c lies above what the sums are relative to
__device__ __forceinline__ float slack(const Sums &a, float c) { return a.big ? 0.f : fmaf(a.ref, c, -a.mu); }
// how far (in powers of two, 0 or below but for that rounding) what a's sums
// are relative to lies below the same of M
__device__ __forceinline__ float below(const Sums &a, const Sums &M, float c) {
  const float d = a.ref == M.ref ? 0.f : (a.big || M.big ? (a.ref - M.ref) * c - slack(a, c) + slack(M, c) : a.mu - M.mu);
  return fmaxf(d, -300.f);
}
__device__ __forceinline__ void move_to(Sums &a, const Sums &M, float c) {
  const float d = below(a, M, c), w = ex2(d);
  a.s1 = w * fmaf(d, a.s0, a.s1), a.s0 *= w;
  a.ref = M.ref, a.mu = M.mu, a.big = M.big;
}

// ln p of a logit, lz being ln Z relative to ref (in halves: the difference may
// pass the 32-bit range and the scale bring it back)
__device__ __forceinline__ float ln_p(float l, float ref, float scale, float lz) {
  return l == ref ? -lz : fmaf(2.f * scale, 0.5f * l - 0.5f * ref, -lz);
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

// Largest of a chunk's values, without NaN.
template <bool BF16>
__device__ __forceinline__ float chunk_max(const uint4 &r) {
  if constexpr (BF16) {
    uint32_t m, n;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(r.x), "r"(r.y));
    asm("max.bf16x2 %0, %1, %2;" : "=r"(n) : "r"(r.z), "r"(r.w));
    asm("max.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(m), "r"(n));
    return fmaxf(bf16lo(m), bf16hi(m));
  } else {
    return fmaxf(fmaxf(__uint_as_float(r.x), __uint_as_float(r.y)), fmaxf(__uint_as_float(r.z), __uint_as_float(r.w)));
  }
}

// A chunk's terms.  SAFE: masked values (infinities below, NaN) count nothing,
// and references may be large; without it masked values leave s1 no number.
template <bool BF16, bool SAFE>
__device__ __forceinline__ void add_chunk(Sums &a, const uint4 &r, float c) {
  constexpr int CH = Chunk<BF16>::n;
  float v[CH], t0 = 0.f, t1 = 0.f;
  Chunk<BF16>::unpack(r, v);
  if (!SAFE || !a.big) {
#pragma unroll
    for (int e = 0; e < CH; e++) {
      float x = fmaf(v[e], c, -a.mu);
      if (SAFE) x = fmaxf(x, -200.f);  // 2^-200 is 0
      const float p = ex2(x);
      t0 += p, t1 = fmaf(p, x, t1);
    }
  } else {
#pragma unroll
    for (int e = 0; e < CH; e++) {
      const float x = fmaxf((v[e] - a.ref) * c, -200.f), p = ex2(x);
      t0 += p, t1 = fmaf(p, x, t1);
    }
  }
  a.s0 += t0, a.s1 += t1;
}

// T threads a block, U chunks of 16 bytes a thread at a time and as many on their way.
template <bool BF16, int T, int U>
__global__ void __launch_bounds__(T) logprobs_rows(const __grid_constant__ LogprobsP P) {
  using C = Chunk<BF16>;
  constexpr int CH = C::n, W = T / 32, kSize = BF16 ? 2 : 4;
  constexpr int kAdd = 32 * CH, kCap = 32 + kAdd;  // list entries that a warp's chunk can add; of a warp
  __shared__ key_t64 s_list[W][kCap];
  __shared__ key_t64 s_top[W][32], s_lists[kMaxS][32];  // of the block's warps, of the row's blocks
  __shared__ uint32_t s_max[W][32];
  __shared__ uint16_t s_cand[T];  // threads whose values may be among the largest
  __shared__ int s_cand_n;
  __shared__ float s_ref[32], s_s0[32], s_s1[32];
  __shared__ int s_inf[32];
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
  const int niter = (nch + T * U - 1) / (T * U);
  const int whole0 = off ? 1 : 0, whole1 = (len + off) / CH;  // chunks that lie in the row

  float tok = 0.f;  // this thread's first given token
  int tok_id = -1;
  if (rank == 0 && tid < P.m) {
    tok_id = P.tokens[row * P.m + tid];
    if ((unsigned)tok_id < (unsigned)P.v) tok = C::load1(base, tok_id);
  }

  // chunk i; edges value by value, NaN (masked) outside the row
  auto load_one = [&](int i) {
    const int first = i * CH - off;
    if (first >= 0 && first + CH <= len) return ldg_stream4(chunks + i);
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
    return make_uint4(w[0], w[1], w[2], w[3]);
  };
  // whether all of iteration it's chunks lie in the row
  auto inside = [&](int it) { return it * U * T >= whole0 && (it + 1) * U * T <= whole1; };
  auto load = [&](uint4 (&r)[U], int it) {
    if (inside(it)) {
#pragma unroll
      for (int u = 0; u < U; u++) r[u] = ldg_stream4(chunks + (it * U + u) * T + tid);
      return;
    }
#pragma unroll
    for (int u = 0; u < U; u++) r[u] = load_one((it * U + u) * T + tid);
  };
  auto max_of = [&](const uint4 (&r)[U]) {
    float m = -kInf;
#pragma unroll
    for (int u = 0; u < U; u++) m = fmaxf(m, chunk_max<BF16>(r[u]));  // drops NaN
    return m;
  };

  uint4 cur[U], nxt[U];
  load(cur, 0);
  // ---- the sums, and the largest value of each thread
  Sums sum;
  {
    float m = max_of(cur);
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(FULLM, m, o));
    set_ref(sum, m, c);
    sum.s0 = sum.s1 = 0.f;
  }
  const float room = 4.f / c;  // how far above its reference a value may lie
  float most = -kInf;
  // the values of one iteration with care; of many rows not unrolled, as that
  // doubles the registers
  auto careful_sums = [&] {
    if constexpr (U > 4) {
#pragma unroll
      for (int u = 0; u < U; u++) add_chunk<BF16, true>(sum, cur[u], c);
    } else {
#pragma unroll 1
      for (int u = 0; u < U; u++) add_chunk<BF16, true>(sum, u == 0 ? cur[0] : (u == 1 ? cur[1] : (u == 2 ? cur[2] : cur[3])), c);
    }
  };
  bool safe = false;
  for (int it = 0; it < niter; it++) {
    if (it + 1 < niter) load(nxt, it + 1);
    const float m = max_of(cur);
    most = fmaxf(most, m);
    if (__any_sync(FULLM, !(m <= sum.ref + room)) && m > sum.ref) {  // (not of an infinite reference)
      Sums to;
      set_ref(to, m, c);
      move_to(sum, to, c);
    }
    const Sums before = sum;
    const bool careful = safe || !inside(it) || __any_sync(FULLM, sum.big);
    if (careful) {
      careful_sums();
    } else {
#pragma unroll
      for (int u = 0; u < U; u++) add_chunk<BF16, false>(sum, cur[u], c);
      // masked values: these again, and the rest of the row, with care
      if (__any_sync(FULLM, !(fabsf(sum.s1) < kInf))) {
        safe = true;
        sum = before;
        careful_sums();
      }
    }
#pragma unroll
    for (int u = 0; u < U; u++) cur[u] = nxt[u];
  }

  // ---- the largest values
  key_t64 tau = 0;
  float tau_v = -kInf;
  int cnt = 0;  // entries of the warp's list

  // Warp: the list's largest 32 become the list, in descending order; the
  // threshold rises to its top_k-th.
  auto compact = [&] {
    __syncwarp();
    key_t64 r = 0;
    for (int b = 0; b < cnt; b += 32) r = merge32(r, sort32(b + lane < cnt ? s_list[warp][b + lane] : 0));
    __syncwarp();
    s_list[warp][lane] = r;
    cnt = __popc(__ballot_sync(FULLM, r != 0));
    const key_t64 t = (key_t64)__shfl_sync(FULLM, (unsigned)(r >> 32), P.k - 1) << 32 | __shfl_sync(FULLM, (unsigned)r, P.k - 1);
    if (t > tau) tau = t, tau_v = of_okey((uint32_t)(tau >> 32));
    __syncwarp();
  };
  // Warp: values of its chunk i that pass the threshold, into the list.
  auto push = [&](const uint4 &r, int i) {
    float v[CH];
    C::unpack(r, v);
    if (cnt > kCap - kAdd) compact();
    unsigned left = 0;  // values of this lane's that may
#pragma unroll
    for (int e = 0; e < CH; e++) left |= (unsigned)(v[e] >= tau_v && v[e] > -kInf) << e;  // false for NaN
    while (__any_sync(FULLM, left != 0)) {
      const int e = __ffs(left) - 1;
      float x = v[0];
#pragma unroll
      for (int j = 1; j < CH; j++) x = e == j ? v[j] : x;
      const key_t64 key = (key_t64)okey(x) << 32 | (uint32_t)~(uint32_t)(lo + i * CH - off + e);
      const bool in = left && key > tau;
      const unsigned who = __ballot_sync(FULLM, in);
      if (in) s_list[warp][cnt + __popc(who & ((1u << lane) - 1u))] = key;
      cnt += __popc(who);
      left &= left - 1;
    }
  };
  if (P.k > 0) {
    // the row that takes this one's place begins in L2, as the block asks HBM
    // for little until then
    if (P.fetch && tid == 0 && row + P.ahead < P.t) {
      const uintptr_t next = reinterpret_cast<uintptr_t>(base) + (uintptr_t)(P.ahead * P.ld * kSize);
      asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"((next + 15) & ~(uintptr_t)15), "r"(P.fetch) : "memory");
    }
    // the threads' maxima in order: top_k of the row reach the top_k-th, and
    // only the threads whose own does have such values: their chunks again,
    // shared out over the block (they lie in L2, or did not long ago)
    const uint32_t mine = most > -kInf ? okey(most) : 0u;
    if (tid == 0) s_cand_n = 0;
    merge_lists(s_max, W, sort32(mine));
    const uint32_t least = s_max[0][P.k - 1];
    tau = (key_t64)least << 32, tau_v = least ? of_okey(least) : -kInf;
    const bool has = mine != 0 && mine >= least;
    const unsigned who = __ballot_sync(FULLM, has);
    int first = 0;
    if (lane == 0 && who) first = atomicAdd(&s_cand_n, __popc(who));
    first = __shfl_sync(FULLM, first, 0);
    if (has) s_cand[first + __popc(who & ((1u << lane) - 1u))] = (uint16_t)tid;
    __syncthreads();
    const int n = s_cand_n, total = n * niter * U;
    constexpr int G = T == 256 ? 2 : 1;  // chunks of a thread at a time (4096 x 131072 bf16, top 20: 219 us; 1: 224)
    for (int b = 0; b < total; b += T * G) {
      uint4 r[G];
      int at_i[G];
#pragma unroll
      for (int u = 0; u < G; u++) {
        const int x = b + u * T + tid, j = n ? x / n : 0, i = j * T + (x < total ? s_cand[x - j * n] : 0);
        r[u] = x < total && i < nch ? load_one(i) : make_uint4(~0u, ~0u, ~0u, ~0u);  // (no numbers)
        at_i[u] = i;
      }
#pragma unroll
      for (int u = 0; u < G; u++)
        if (__any_sync(FULLM, chunk_max<BF16>(r[u]) >= tau_v)) push(r[u], at_i[u]);
    }
    compact();
    merge_lists(s_top, W, s_list[warp][lane]);
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
      tc05::st_cluster(tc05::map_rank(&s_lists[rank][lane], 0), P.k > 0 ? s_top[0][lane] : 0ull);
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
    }
    if (P.k > 0) {  // (a row of several blocks has 256 threads a block or more: a warp a list)
      merge_lists(s_lists, S, warp < S ? s_lists[warp][lane] : 0ull);
      top = s_lists[0][lane];
    }
  } else if (warp == 0 && P.k > 0) {
    top = s_top[0][lane];
  }
  // ---- the answers
  if (warp == 0) {
    float lz, h;
    if (all.ref == kInf) {
      lz = logf((float)ninf), h = lz;
    } else if (all.ref == -kInf) {  // no logit
      lz = 0.f, h = 0.f;
    } else {
      const float l2 = log2f(all.s0);
      // relative to ref: mu is ref * c rounded
      lz = kLn2 * (l2 - slack(all, c)), h = kLn2 * (l2 - all.s1 / all.s0);
    }
    if (lane == 0) {
      s_row[0] = all.ref, s_row[1] = lz;
      if (P.entropy) P.entropy[row] = h < 0.f ? 0.f : h;
    }
    if (lane < P.k) {
      const float x = of_okey((uint32_t)(top >> 32));
      P.top_idx[row * P.k + lane] = top ? ~(uint32_t)top : 0xffffffffu;
      P.top_logp[row * P.k + lane] = top ? ln_p(x, all.ref, P.scale, lz) : -kInf;
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
    P.logp[row * P.m + i] = in ? ln_p(tok, ref, P.scale, lz) : -kInf;
  }
}

template <bool BF16, int T, int U = 4>
cudaError_t launch_t(LogprobsP p, int n_sms, cudaStream_t st) {
  static const int fit = [] {
    int n = 0;
    return cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, logprobs_rows<BF16, T, U>, T, 0) == cudaSuccess ? n : 0;
  }();
  p.ahead = fit * n_sms;
  // 4096 x 131072 bf16 with 0 / 16 / 32 / 64 / 128 KB of the next row: top 1 178 /
  // 169 / 164 / 168 / 173 us, top 5 185 / 180 / 179 / 184 / 189, top 20 224 / 226 /
  // 227 / 232 / 230; shorter rows lose (16384 x 16000: 123 / 131 with 32)
  p.fetch = T == 256 && p.S == 1 && (int64_t)p.v * (BF16 ? 2 : 4) >= 2 * kFetch ? kFetch : 0;
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
  return cudaLaunchKernelEx(&cfg, logprobs_rows<BF16, T, U>, p);
}

}  // namespace

cudaError_t launch_logprobs(LogprobsP p, int n_sms, cudaStream_t st) {
  // Few rows: several blocks a row, of 16384 values or more while each has an
  // SM, of 25000 when some SMs have two.  us with 1 / 2 / 4 / 8, fp32: 1 x
  // 131072 18 / 12 / 9.4 / 7.9, 48 x 100003 14 / 11 / 10.2 / 12.2, 100 x 131072
  // 16 / 14 / 14 / 18, 100 x 32000 7.7 / 8.3 / 9.6 / 15, 30 x 20000 6.8 / 7.3 / 7.2 / 7.3.
  p.S = 1;
  while (p.S < kMaxS) {
    const int64_t blocks = (int64_t)p.t * p.S * 2, values = p.v / (p.S * 2);
    if (!(blocks <= n_sms ? values >= 16384 : (blocks <= n_sms * 4 / 3 && values >= 25000))) break;
    p.S *= 2;
  }
  p.seg = ((p.v + p.S - 1) / p.S + 7) / 8 * 8;
  // Threads of a block: what it does once a row (orders, exchanges) costs as
  // much as some values of each thread.  us, 16384 rows, top 5, fp32, with 32 /
  // 64 / 128 / 256 threads: of 1000 27 / 44 / 76 / 153, of 4000 61 / 68 / 94 /
  // 164, of 8000 136 / 103 / 121 / 189, of 32000 531 / 437 / 359 / 371; few
  // rows (256) of 4000 8.1 / 6.3 / 5.8 / 6.0, of 32000 33 / 17 / 10.6 / 9.4.
  const int64_t bytes = (int64_t)p.seg * (p.bf16 ? 2 : 4);
  const bool few = (int64_t)p.t < 8 * (int64_t)n_sms;
  int T = bytes <= (few ? 4096 : 20480) ? 32 : (bytes <= (few ? 8192 : 40960) ? 64 : (bytes <= (few ? 20480 : 131072) ? 128 : 256));
  if (p.S > 1) T = 256;  // a warp for each of a row's lists
  // fp32, no more than two blocks an SM: more of a row in flight for each (48 x 100003,
  // not in L2: 14.4 -> 11.5 us; 4096 x 131072: 186 -> 328). Not bf16, where its registers
  // leave one block an SM (16 x 131072: 7.9 -> 12.4).
  if (!p.bf16 && T == 256 && (int64_t)p.t * p.S <= 2 * n_sms) return launch_t<false, 256, 8>(p, n_sms, st);
  auto go = [&](auto n) { return p.bf16 ? launch_t<true, decltype(n)::value>(p, n_sms, st) : launch_t<false, decltype(n)::value>(p, n_sms, st); };
  if (T == 32) return go(std::integral_constant<int, 32>());
  if (T == 64) return go(std::integral_constant<int, 64>());
  if (T == 128) return go(std::integral_constant<int, 128>());
  return go(std::integral_constant<int, 256>());
}

}  // namespace moe
