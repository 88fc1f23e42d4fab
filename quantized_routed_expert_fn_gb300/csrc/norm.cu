// norm.cu -- root-mean-square norms before and after a block:
//   out = x / sqrt(mean(x^2) + eps) * w                            (norm)
//   r = res_scale * residual + scale * gate * v, out = norm of r   (add_norm)
// with v the block's output or its norm.
//
// A row stays in registers from its loads to its last store: every tensor is
// read and written once, so HBM is the bound.  T threads (a power of two)
// hold a row, NV values each, in pieces of V neighbouring values: V = 8 where
// all rows start on 16 bytes, 2 or 1 where they do not, so that neighbouring
// lanes always touch neighbouring bytes.  Sums are 32-bit, in a fixed tree.
#include <cuda_runtime.h>

#include "block.cuh"
#include "fp8.cuh"

namespace moe {
namespace {

constexpr unsigned FULLM = 0xffffffffu;
constexpr int kMaxThreads = 512;

template <int V>
__device__ __forceinline__ void load_piece(const void *p, int bf16, int64_t i, float *v) {
  if (bf16) {
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

template <int V>
__device__ __forceinline__ void store_piece(void *p, int bf16, int64_t i, const float *v) {
  if (bf16) {
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

// Sum over the T threads of each row; red: a word for each warp, used once.
// large: (the same for all threads that share a barrier) whether any row's
// sum may be past 1e37.
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
  const int W = blockDim.x >> 5, nw = T >> 5;
  large = __any_sync(FULLM, lane < W && !(red[lane < W ? lane : 0] < 1e35f));
  v = red[(warp & ~(nw - 1)) + (lane & (nw - 1))];
  for (int o = nw >> 1; o; o >>= 1) v += __shfl_xor_sync(FULLM, v, o);
  return v;
}

// v *= 1 / sqrt(mean(v^2) + eps).  A row whose sum of squares comes near the
// end of the 32-bit range is summed again 2^-100 smaller (exact: its largest
// value is at least 1e16); infinities and NaN stay what the formula makes of
// them.
template <int NV>
__device__ __forceinline__ void normalise(float (&v)[NV], const NormP &P, float *red) {
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < NV; i++) ss = fmaf(v[i], v[i], ss);
  bool large, any;
  ss = row_sum(ss, P.T, red, any);
  float eps = P.eps;
  if (any) {
    const bool big = !(ss < 1e37f);
    const float c = big ? 7.888609052210118e-31f : 1.f;
    ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; i++) v[i] *= c, ss = fmaf(v[i], v[i], ss);
    ss = row_sum(ss, P.T, red + 32, large);
    eps = eps * c * c;
  }
  const float inv = 1.f / sqrtf(ss / (float)P.h + eps);
#pragma unroll
  for (int i = 0; i < NV; i++) v[i] *= inv;
}

template <int V, int NV, bool ADD>
__global__ void __launch_bounds__(kMaxThreads) norm_rows(const __grid_constant__ NormP P) {
  constexpr int N = NV / V;
  __shared__ float red[4][32];
  extern __shared__ uint32_t s_max[];  // e4m3, V < 8: [N][warps]
  pdl_wait_prev();
  pdl_launch_next();
  const int T = P.T, l = threadIdx.x & (T - 1);
  const int64_t row = (int64_t)blockIdx.x * (blockDim.x / T) + threadIdx.x / T;
  const bool live = row < P.t;
  auto col = [&](int j) { return (j * T + l) * V; };
  auto here = [&](int j) { return live && col(j) < P.h; };
  float v[NV];
#pragma unroll
  for (int j = 0; j < N; j++) {
    if (here(j)) load_piece<V>(P.y, P.y_bf16, row * P.ldy + col(j), v + j * V);
    else
#pragma unroll
      for (int i = 0; i < V; i++) v[j * V + i] = 0.f;
  }
  if constexpr (ADD) {
    if (P.post) {
      normalise(v, P, red[0]);
      if (P.wp) {
#pragma unroll
        for (int j = 0; j < N; j++)
          if (here(j)) {
            float w[V];
            load_piece<V>(P.wp, 0, col(j), w);
#pragma unroll
            for (int i = 0; i < V; i++) v[j * V + i] *= w[i];
          }
      }
    }
    float g1 = 1.f;
    auto sig = [&](float g) { return P.gate_sigmoid ? 1.f / (1.f + expf(-g)) : g; };
    if (P.gate && P.gate_cols == 1 && live) {
      load_piece<1>(P.gate, P.gate_bf16, row * P.ldg, &g1);
      g1 = sig(g1);
    }
#pragma unroll
    for (int j = 0; j < N; j++)
      if (here(j)) {
        float r[V], g[V];
        load_piece<V>(P.res, P.res_bf16, row * P.ldr + col(j), r);
        if (P.gate && P.gate_cols != 1) {
          load_piece<V>(P.gate, P.gate_bf16, row * P.ldg + col(j), g);
#pragma unroll
          for (int i = 0; i < V; i++) g[i] = sig(g[i]);
        } else {
#pragma unroll
          for (int i = 0; i < V; i++) g[i] = g1;
        }
#pragma unroll
        for (int i = 0; i < V; i++) {
          // gate by value first: a gate of 0 closes, whatever the scale
          r[i] = fmaf(P.scale, g[i] * v[j * V + i], P.res_scale * r[i]);
          v[j * V + i] = r[i];
        }
        store_piece<V>(P.ro, P.ro_bf16, row * P.ldro + col(j), r);
      }
    if (P.out_kind == kNormOutNone) return;
  }
  normalise(v, P, red[2]);
  if (P.w) {
#pragma unroll
    for (int j = 0; j < N; j++)
      if (here(j)) {
        float w[V];
        load_piece<V>(P.w, 0, col(j), w);
#pragma unroll
        for (int i = 0; i < V; i++) v[j * V + i] *= w[i];
      }
  }
  if (P.out_kind != kNormOutE4m3) {
#pragma unroll
    for (int j = 0; j < N; j++)
      if (here(j)) store_piece<V>(P.out, P.out_kind == kNormOutBf16, row * P.ldo + col(j), v + j * V);
    return;
  }
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
      if (here(j)) {
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
      if (here(j)) {
        const uint32_t w = e4m3x2<true>(v[j * V] * f, V == 2 ? v[j * V + V - 1] * f : 0.f);
        if constexpr (V == 2) *reinterpret_cast<uint16_t *>(q + col(j)) = (uint16_t)w;
        else q[col(j)] = (uint8_t)w;
        if ((col(j) & 127) == 0) s[col(j) >> 7] = (uint8_t)e;
      }
    }
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

template <int V, int NV>
cudaError_t launch_vn(NormP p, cudaStream_t st) {
  int T = 4;
  while (T * NV < p.h) T *= 2;
  if (p.out_kind == kNormOutE4m3 && T < 128 / V) T = 128 / V;
  p.T = T;
  const int block = T < 256 ? 256 : T, rows = block / T;
  const size_t smem = p.out_kind == kNormOutE4m3 && V < 8 ? (size_t)(NV / V) * (block / 32) * 4 : 0;
  const dim3 grid((unsigned)(((int64_t)p.t + rows - 1) / rows));
  return p.res ? launch_pdl(norm_rows<V, NV, true>, grid, block, smem, st, p)
               : launch_pdl(norm_rows<V, NV, false>, grid, block, smem, st, p);
}

template <int V>
cudaError_t launch_v(const NormP &p, cudaStream_t st) {
  if (p.h <= 8 * kMaxThreads) return launch_vn<V, 8>(p, st);
  if (p.h <= 16 * kMaxThreads) return launch_vn<V, 16>(p, st);
  if (p.h <= 32 * kMaxThreads) return launch_vn<V, 32>(p, st);
  return launch_vn<V, 64>(p, st);
}

}  // namespace

cudaError_t launch_norm(const NormP &p, int, cudaStream_t st) {
  const int v = piece(p);
  return v == 8 ? launch_v<8>(p, st) : (v == 2 ? launch_v<2>(p, st) : launch_v<1>(p, st));
}

}  // namespace moe
