// norm.cu -- root-mean-square norms before and after a block:
//   out = x / sqrt(mean(x^2) + eps) * w                            (norm)
//   r = res_scale * residual + scale * gate * v, out = norm of r   (add_norm)
// with v the block's output or its norm.
//
// A row stays in registers from its loads to its last store: every tensor is
// read and written once, so HBM is the bound, and instructions where values
// are bf16.  T threads hold a row, NV values each, in pieces of V neighbouring
// values: V = 8 where all rows start on 16 bytes, or anywhere but alike (the
// pieces then begin on 16 bytes in the row, see SH); 2 or 1 otherwise, so that
// neighbouring lanes always touch neighbouring bytes.  Sums are 32-bit, in a
// fixed tree.  65536 x 2048 bf16: 89 us, 6.0 TB/s; fp32 32768 x 2048: 80, 6.7;
// 32816 x 4090 bf16 122 (with pieces of 2: 160).
#include <cuda_runtime.h>

#include <type_traits>

#include "block.cuh"
#include "fp8.cuh"

namespace moe {
namespace {

constexpr unsigned FULLM = 0xffffffffu;
constexpr int kMaxThreads = 512;

// V neighbouring values: bf16 or fp32
template <int V, bool BF16>
__device__ __forceinline__ void load_as(const void *p, int64_t i, float *v) {
  if constexpr (BF16) {
    const uint16_t *x = static_cast<const uint16_t *>(p) + i;
    if constexpr (V == 8) {
      const uint4 u = *reinterpret_cast<const uint4 *>(x);
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int j = 0; j < 4; j++) v[2 * j] = bf16lo(w[j]), v[2 * j + 1] = bf16hi(w[j]);
    } else if constexpr (V == 2) {
      const uint32_t u = *reinterpret_cast<const uint32_t *>(x);
      v[0] = bf16lo(u), v[1] = bf16hi(u);
    } else {
      v[0] = __uint_as_float((uint32_t)*x << 16);
    }
  } else {
    const float *x = static_cast<const float *>(p) + i;
    if constexpr (V == 8) {
      const float4 a = *reinterpret_cast<const float4 *>(x), b = *reinterpret_cast<const float4 *>(x + 4);
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else if constexpr (V == 2) {
      const float2 a = *reinterpret_cast<const float2 *>(x);
      v[0] = a.x, v[1] = a.y;
    } else {
      v[0] = *x;
    }
  }
}

// two values to bf16 (nearest, ties to even), lo in the lower half
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

template <int V, bool BF16>
__device__ __forceinline__ void store_as(void *p, int64_t i, const float *v) {
  if constexpr (BF16) {
    uint16_t *x = static_cast<uint16_t *>(p) + i;
    if constexpr (V == 8)
      *reinterpret_cast<uint4 *>(x) = make_uint4(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]), bf16x2(v[4], v[5]), bf16x2(v[6], v[7]));
    else if constexpr (V == 2) *reinterpret_cast<uint32_t *>(x) = bf16x2(v[0], v[1]);
    else *x = (uint16_t)bf16x2(v[0], 0.f);
  } else {
    float *x = static_cast<float *>(p) + i;
    if constexpr (V == 8) {
      *reinterpret_cast<float4 *>(x) = make_float4(v[0], v[1], v[2], v[3]);
      *reinterpret_cast<float4 *>(x + 4) = make_float4(v[4], v[5], v[6], v[7]);
    } else if constexpr (V == 2) {
      *reinterpret_cast<float2 *>(x) = make_float2(v[0], v[1]);
    } else {
      *x = v[0];
    }
  }
}

// Sum over the T threads of each row: a power of two lanes, or all warps of a
// block; red:
// a word for each warp, used once.  large (the same for all threads of a warp,
// or of the block): whether any of their sums may be past 1e37.
__device__ __forceinline__ float row_sum(float v, int T, float *red, bool &large) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (T <= 32) {
    for (int o = T >> 1; o; o >>= 1) v += __shfl_xor_sync(FULLM, v, o);
    large = __any_sync(FULLM, !(v < 1e35f));
    return v;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(FULLM, v, o);
  if (lane == 0) red[warp] = v;
  __syncthreads();
  v = lane < (T >> 5) ? red[lane] : 0.f;
  large = __any_sync(FULLM, !(v < 1e35f));
#pragma unroll
  for (int o = kMaxThreads / 64; o; o >>= 1) v += __shfl_xor_sync(FULLM, v, o);
  return __shfl_sync(FULLM, v, 0);
}

// v and x *= 1 / sqrt(mean over the row of their squares + eps).  A row whose
// sum of squares comes near the end of the 32-bit range is summed again 2^-100
// smaller (exact: its largest value is at least 1e16); infinities and NaN stay
// what the formula makes of them.
template <int NV>
__device__ __forceinline__ void normalise(float (&v)[NV], float &x, const NormP &P, float *red) {
  float s4[4] = {x * x, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < NV; i++) s4[i & 3] = fmaf(v[i], v[i], s4[i & 3]);
  bool large, any;
  float ss = row_sum((s4[0] + s4[1]) + (s4[2] + s4[3]), P.T, red, any), eps = P.eps;
  if (any) {
    const float c = !(ss < 1e37f) ? 7.888609052210118e-31f : 1.f;
    x *= c, ss = x * x;
#pragma unroll
    for (int i = 0; i < NV; i++) v[i] *= c, ss = fmaf(v[i], v[i], ss);
    ss = row_sum(ss, P.T, red + 32, large);
    eps = eps * c * c;
  }
  const float inv = rsqrtf(fmaf(ss, P.inv_h, eps));
  x *= inv;
#pragma unroll
  for (int i = 0; i < NV; i++) v[i] *= inv;
}

// SH (V = 8): rows that do not start on 16 bytes, but all matrices' alike: the
// pieces begin `lead` values into a row, on 16 bytes; those before them and the
// last ones are one value more for 16 of the row's threads.  What is per column
// lies in shared memory as fp32, a word left out after each eight, so that
// lanes that read 8 words apart meet no bank twice; a block keeps it over its
// rows.
constexpr int kMaxVec = 96 * 1024;  // bytes of those
__host__ __device__ constexpr int vec_words(int h) { return (h + 7) / 8 * 9; }
struct Vecs {
  const float *w, *wp, *g;
};

__device__ __forceinline__ float load1(const void *p, int bf16, int64_t i) {
  float v;
  if (bf16) load_as<1, true>(p, i, &v);
  else load_as<1, false>(p, i, &v);
  return v;
}
__device__ __forceinline__ float gate_of(const NormP &P, float g) { return P.gate_sigmoid && g == g ? logistic(g) : g; }

// One row, in the registers of T threads (all of a warp's, or a block's, come
// here together).
template <int V, int NV, bool ADD, bool SH>
__device__ __forceinline__ void one_row(const NormP &P, int64_t row, float (&red)[4][32], const Vecs &vecs, uint32_t *s_max) {
  constexpr int N = NV / V;
  const int T = P.T, l = P.T >= (int)blockDim.x ? (int)threadIdx.x : (int)threadIdx.x & (T - 1);
  const bool live = row < P.t;
  const int h = live ? P.h : 0, lead = SH ? (int)(-((row & 7) * P.ld8) & 7) : 0;
  auto col = [&](int j) { return lead + (j * T + l) * V; };
  auto pieces = [&](auto f) {
#pragma unroll
    for (int j = 0; j < N; j++)
      if (col(j) + (SH ? V : 1) <= h) f(j);
  };
  // SH: the value more, of column xc (< 0: none)
  int xc = -1;
  if (SH && l < 8 && l < lead) xc = l;
  if (SH && l >= 8 && l < 16) xc = h - (h - lead) % 8 + l - 8;
  if (xc >= h) xc = -1;
  int word[SH ? 8 : 1];  // of a piece's i-th column, behind 9 words for each piece before it
  if constexpr (SH)
#pragma unroll
    for (int i = 0; i < 8; i++) word[i] = lead + i + ((lead + i) >> 3);
  auto load = [&](const void *p, int bf16, int64_t at, float *to, float &x) {
    if (bf16) pieces([&](int j) { load_as<V, true>(p, at + col(j), to + j * V); });
    else pieces([&](int j) { load_as<V, false>(p, at + col(j), to + j * V); });
    if (SH && xc >= 0) x = load1(p, bf16, at + xc);
  };
  float v[NV], x = 0.f;
  auto store = [&](void *p, int bf16, int64_t at) {
    if (bf16) {
      pieces([&](int j) { store_as<V, true>(p, at + col(j), v + j * V); });
      if (SH && xc >= 0) store_as<1, true>(p, at + xc, &x);
    } else {
      pieces([&](int j) { store_as<V, false>(p, at + col(j), v + j * V); });
      if (SH && xc >= 0) store_as<1, false>(p, at + xc, &x);
    }
  };
  auto weigh = [&](const float *weights, const float *words) {
    if constexpr (SH) {
      pieces([&](int j) {
#pragma unroll
        for (int i = 0; i < 8; i++) v[8 * j + i] *= words[9 * (j * T + l) + word[i]];
      });
      if (xc >= 0) x *= words[xc + (xc >> 3)];
    } else {
      pieces([&](int j) {
        float w[V];
        load_as<V, false>(weights, col(j), w);
#pragma unroll
        for (int i = 0; i < V; i++) v[j * V + i] *= w[i];
      });
    }
  };
#pragma unroll
  for (int i = 0; i < NV; i++) v[i] = 0.f;
  load(P.y, P.y_bf16, row * P.ldy, v, x);
  if constexpr (ADD) {
    float r[NV], rx = 0.f;  // on its way before the first store: the residual may be what is written
#pragma unroll
    for (int i = 0; i < NV; i++) r[i] = 0.f;
    load(P.res, P.res_bf16, row * P.ldr, r, rx);
    if (P.post) {
      normalise(v, x, P, red[0]);
      if (P.wp) weigh(P.wp, vecs.wp);
    }
    // (gate by value first: a gate of 0 closes, whatever the scale)
    if (P.gate) {
      if (P.gate_cols == 1) {
        const float g = live ? gate_of(P, load1(P.gate, P.gate_bf16, row * P.ldg)) : 1.f;
        x *= g;
#pragma unroll
        for (int i = 0; i < NV; i++) v[i] *= g;
      } else if (SH && P.ldg == 0) {
        weigh(nullptr, vecs.g);
      } else {
        auto by = [&](auto bf16, auto sigmoid) {
          pieces([&](int j) {
            float g[V];
            load_as<V, decltype(bf16)::value>(P.gate, row * P.ldg + col(j), g);
#pragma unroll
            for (int i = 0; i < V; i++) v[j * V + i] *= decltype(sigmoid)::value && g[i] == g[i] ? logistic(g[i]) : g[i];
          });
        };
        using Y = std::true_type;
        using No = std::false_type;
        if (P.gate_sigmoid) P.gate_bf16 ? by(Y(), Y()) : by(No(), Y());
        else P.gate_bf16 ? by(Y(), No()) : by(No(), No());
        if (SH && xc >= 0) x *= gate_of(P, load1(P.gate, P.gate_bf16, row * P.ldg + xc));
      }
    }
    x = fmaf(P.scale, x, P.res_scale * rx);
#pragma unroll
    for (int i = 0; i < NV; i++) v[i] = fmaf(P.scale, v[i], P.res_scale * r[i]);
    store(P.ro, P.ro_bf16, row * P.ldro);
    if (P.out_kind == kNormOutNone) return;
  }
  normalise(v, x, P, red[2]);
  if (P.w) weigh(P.w, vecs.w);
  if (P.out_kind != kNormOutE4m3) {
    store(P.out, P.out_kind == kNormOutBf16, row * P.ldo);
    return;
  }
  if constexpr (SH) return;  // (not launched so)
  uint8_t *q = static_cast<uint8_t *>(P.out) + row * P.ldo, *s = P.s + row * P.lds;
  if constexpr (V == 8) {
    // 16 lanes hold a scale block
#pragma unroll
    for (int j = 0; j < N; j++) {
      float b[8];
#pragma unroll
      for (int i = 0; i < 8; i++) b[i] = v[j * 8 + i];
      uint32_t w[2], e;
      quant_block<8>(b, w, e);
      if (col(j) < h) {
        *reinterpret_cast<uint2 *>(q + col(j)) = make_uint2(w[0], w[1]);
        if ((l & 15) == 0) s[col(j) >> 7] = (uint8_t)e;
      }
    }
  } else {
    // two or four neighbouring warps hold one (T is at least 128 / V)
    const int warp = threadIdx.x >> 5, W = blockDim.x >> 5;
#pragma unroll
    for (int j = 0; j < N; j++) {
      uint32_t a = 0;
#pragma unroll
      for (int i = 0; i < V; i++) a = max(a, mag_bits(v[j * V + i]));
      a = __reduce_max_sync(FULLM, a);
      if ((threadIdx.x & 31) == 0) s_max[j * W + warp] = a;
    }
    __syncthreads();
    constexpr int B = 4 / V;  // warps of a block
#pragma unroll
    for (int j = 0; j < N; j++) {
      uint32_t a = 0;
#pragma unroll
      for (int i = 0; i < B; i++) a = max(a, s_max[j * W + (warp & ~(B - 1)) + i]);
      const uint32_t e = e8m0_of_amax(a);
      const float f = e8m0_inv(e);
      if (col(j) < h) {
        const uint32_t w = e4m3x2<true>(v[j * V] * f, V == 2 ? v[j * V + V - 1] * f : 0.f);
        if constexpr (V == 2) *reinterpret_cast<uint16_t *>(q + col(j)) = (uint16_t)w;
        else q[col(j)] = (uint8_t)w;
        if ((col(j) & 127) == 0) s[col(j) >> 7] = (uint8_t)e;
      }
    }
  }
}

// Without SH the grid covers the rows; with it, blocks walk over them.
template <int V, int NV, bool ADD, bool SH>
__global__ void __launch_bounds__(kMaxThreads) norm_rows(const __grid_constant__ NormP P) {
  static_assert(!SH || V == 8, "");
  __shared__ float s_red[SH ? 2 : 1][4][32];
  extern __shared__ uint32_t s_dyn[];  // e4m3, V < 8: maxima [N][warps]; SH: vectors
  pdl_wait_prev();
  pdl_launch_next();
  const int per = P.T >= (int)blockDim.x ? 1 : (int)blockDim.x / P.T, mine = per > 1 ? (int)threadIdx.x / P.T : 0;
  if constexpr (!SH) {
    one_row<V, NV, ADD, SH>(P, (int64_t)blockIdx.x * per + mine, s_red[0], Vecs(), s_dyn);
  } else {
    float *at = reinterpret_cast<float *>(s_dyn);
    auto place = [&](auto get) {
      float *to = at;
      for (int i = threadIdx.x; i < P.h; i += blockDim.x) to[i + (i >> 3)] = get(i);
      at += vec_words(P.h);
      return to;
    };
    Vecs vecs = {};
    if (P.w) vecs.w = place([&](int c) { return P.w[c]; });
    if (ADD && P.wp) vecs.wp = place([&](int c) { return P.wp[c]; });
    if (ADD && P.gate && P.gate_cols != 1 && P.ldg == 0) vecs.g = place([&](int c) { return gate_of(P, load1(P.gate, P.gate_bf16, c)); });
    __syncthreads();
    int half = 0;  // the next row's sums lie in the other half
    for (int64_t first = (int64_t)blockIdx.x * per; first < P.t; first += (int64_t)gridDim.x * per, half ^= 1)
      one_row<V, NV, ADD, SH>(P, first + mine, s_red[half], vecs, s_dyn);
  }
}

// the widest pieces that every row of every tensor allows: 8, 2 or 1 values
int piece(const NormP &p) {
  int v = 8;
  auto need = [&](const void *a, int64_t ld, int size, int align8) {
    if (!a) return;
    const uintptr_t at = reinterpret_cast<uintptr_t>(a), step = (uintptr_t)(ld * size);
    while (v > 1 && ((at | step) & (uintptr_t)(v == 8 ? align8 - 1 : 2 * size - 1))) v = v == 8 ? 2 : 1;
  };
  auto size = [](int bf16) { return bf16 ? 2 : 4; };
  while (v > 1 && p.h % v) v = v == 8 ? 2 : 1;
  need(p.y, p.ldy, size(p.y_bf16), 16);
  need(p.res, p.ldr, size(p.res_bf16), 16);
  need(p.ro, p.ldro, size(p.ro_bf16), 16);
  if (p.gate && p.gate_cols != 1) need(p.gate, p.ldg, size(p.gate_bf16), 16);
  need(p.w, 0, 4, 16);
  need(p.wp, 0, 4, 16);
  if (p.out_kind == kNormOutE4m3) need(p.out, p.ldo, 1, 8);
  else if (p.out_kind != kNormOutNone) need(p.out, p.ldo, p.out_kind == kNormOutBf16 ? 2 : 4, 16);
  return v;
}

// Whether no row starts on 16 bytes, but all matrices' rows alike.
bool alike(NormP &p) {
  if (p.out_kind == kNormOutE4m3) return false;
  const int vecs = (p.w != nullptr) + (p.wp != nullptr) + (p.gate && p.gate_cols != 1 && p.ldg == 0);
  if (vecs * vec_words(p.h) * 4 > kMaxVec) return false;
  bool ok = true;
  int rem = -1;
  auto take = [&](const void *a, int64_t ld) {
    if (!a) return;
    ok = ok && (reinterpret_cast<uintptr_t>(a) & 15) == 0 && (rem < 0 || rem == (int)(ld & 7) || p.t == 1);
    rem = (int)(ld & 7);
  };
  take(p.y, p.ldy), take(p.res, p.ldr), take(p.ro, p.ldro);
  if (p.out_kind != kNormOutNone) take(p.out, p.ldo);
  if (p.gate && p.gate_cols != 1 && p.ldg) take(p.gate, p.ldg);
  p.ld8 = rem;
  return ok;
}

template <class F>
int registers(F f) {
  cudaFuncAttributes a;
  return cudaFuncGetAttributes(&a, f) == cudaSuccess && a.numRegs > 0 ? (a.numRegs + 7) / 8 * 8 : 128;
}

template <int NV>
cudaError_t launch_alike(NormP p, int T, int n_sms, cudaStream_t st) {
  p.T = T;
  const int block = T <= 32 ? 256 : T, rows = block / T;
  const int vecs = (p.w != nullptr) + (p.wp != nullptr) + (p.gate && p.gate_cols != 1 && p.ldg == 0);
  const size_t smem = (size_t)vecs * vec_words(p.h) * 4;
  auto f = p.res ? norm_rows<8, NV, true, true> : norm_rows<8, NV, false, true>;
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxVec);
    if (e != cudaSuccess) return e;
  }
  static const int regs[2] = {registers(norm_rows<8, NV, false, true>), registers(norm_rows<8, NV, true, true>)};
  // as many thread blocks as stay resident, each with the same number of rounds
  const int by_regs = 65536 / (regs[p.res != nullptr] * block), by_smem = (int)(220 * 1024 / (smem + 1024));
  const int fit = by_regs < by_smem ? by_regs : by_smem;
  const int64_t need = ((int64_t)p.t + rows - 1) / rows, cap = (int64_t)n_sms * (fit < 1 ? 1 : (fit > 2048 / block ? 2048 / block : fit));
  const int64_t rounds = (need + cap - 1) / cap;
  return launch_pdl(f, dim3((unsigned)((need + rounds - 1) / rounds)), block, smem, st, p);
}

template <int V, int NV>
cudaError_t launch_form(NormP p, int T, cudaStream_t st) {
  p.T = T;
  const int block = T <= 32 ? 128 : T, rows = block / T;  // (T above 32: a block a row)
  const size_t smem = p.out_kind == kNormOutE4m3 && V < 8 ? (size_t)(NV / V) * (block / 32) * 4 : 0;
  const dim3 grid((unsigned)(((int64_t)p.t + rows - 1) / rows));
  return p.res ? launch_pdl(norm_rows<V, NV, true, false>, grid, block, smem, st, p)
               : launch_pdl(norm_rows<V, NV, false, false>, grid, block, smem, st, p);
}

// Values a thread holds.  What a thread does whatever their number (addresses,
// exchanges, the root) costs as much as some 16: 32 of them, with a residual
// 16, as long as the rows give every SM 64 warps; few rows want many threads.
// us with 8 / 16 / 32 / 64 values, bf16, norm: 65536 rows x 2048 101 / 95 / 89
// / 111, 32768 x 4096 113 / 104 / 97 / 110; one row x 2048 1.8 / 2.1 / 2.4 /
// 3.1.  add_norm (fp32 residual): 65536 x 2048 305 / 286 / 297 / 324.
template <class T>
int values_a_thread(const NormP &p, int n_sms, T threads) {
  int nv = 8;
  const int most = p.res ? 16 : 32;
  while (nv < most && threads(2 * nv) < threads(nv) && (int64_t)p.t * threads(2 * nv) >= (int64_t)n_sms * 64 * 32) nv *= 2;
  while (threads(nv) > kMaxThreads) nv *= 2;
  return nv;
}

// Threads of a row: a power of two up to 32, or warps (`least` if that is more,
// and multiples of it).
int threads_for(int values, int nv, int least) {
  int T = least;
  while (T < 32 && T * nv < values) T *= 2;
  const int unit = least > 32 ? least : 32;
  return T * nv >= values ? T : ((values + nv - 1) / nv + unit - 1) / unit * unit;
}

template <int V>
cudaError_t launch_v(const NormP &p, int n_sms, cudaStream_t st) {
  auto threads = [&](int nv) { return threads_for(p.h, nv, p.out_kind == kNormOutE4m3 ? 128 / V : 4); };
  const int nv = values_a_thread(p, n_sms, threads), T = threads(nv);
  return nv == 8 ? launch_form<V, 8>(p, T, st) : (nv == 16 ? launch_form<V, 16>(p, T, st) :
         (nv == 32 ? launch_form<V, 32>(p, T, st) : launch_form<V, 64>(p, T, st)));
}

}  // namespace

cudaError_t launch_norm(NormP p, int n_sms, cudaStream_t st) {
  const int v = piece(p);
  if (v == 8) return launch_v<8>(p, n_sms, st);
  auto threads = [&](int nv) { return threads_for(p.h, nv, 16); };
  const int nv = values_a_thread(p, n_sms, threads), T = threads(nv);
  if (nv <= 32 && p.h >= 32 && alike(p))
    return nv == 8 ? launch_alike<8>(p, T, n_sms, st) : (nv == 16 ? launch_alike<16>(p, T, n_sms, st) : launch_alike<32>(p, T, n_sms, st));
  return v == 2 ? launch_v<2>(p, n_sms, st) : launch_v<1>(p, n_sms, st);
}

}  // namespace moe
