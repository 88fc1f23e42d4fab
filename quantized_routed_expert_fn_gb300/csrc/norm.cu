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
// fixed tree.  65536 x 2048 bf16: 84 us, 6.4 TB/s; fp32 32768 x 2048: 79, 6.8;
// 32816 x 4090 bf16 107 (with pieces of 2: 160).  add_norm, 30000 x 4096, all
// bf16, a gate a channel: 157 us, 6.3 TB/s; 30011 x 4090 195.  Arithmetic goes two
// values an instruction (one by one 2 to 4 % longer).
#include <cuda_runtime.h>

#include <type_traits>

#include "block.cuh"
#include "fp8.cuh"
#include "tc05.cuh"

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

// Two values an instruction, each rounded as on its own.
__device__ __forceinline__ void mul2(float &x, float &y, float a, float b) {
  asm("{\n .reg .b64 u, v;\n mov.b64 u, {%0, %1};\n mov.b64 v, {%2, %3};\n mul.rn.f32x2 u, u, v;\n mov.b64 {%0, %1}, u;\n}\n"
      : "+f"(x), "+f"(y)
      : "f"(a), "f"(b));
}
// x, y = a x + c, b y + d
__device__ __forceinline__ void fma2(float &x, float &y, float a, float b, float c, float d) {
  asm("{\n .reg .b64 u, v, w;\n mov.b64 u, {%0, %1};\n mov.b64 v, {%2, %3};\n mov.b64 w, {%4, %5};\n fma.rn.f32x2 u, u, v, w;\n"
      " mov.b64 {%0, %1}, u;\n}\n"
      : "+f"(x), "+f"(y)
      : "f"(a), "f"(b), "f"(c), "f"(d));
}
// s, t += a^2, b^2
__device__ __forceinline__ void squares2(float &s, float &t, float a, float b) {
  asm("{\n .reg .b64 u, v;\n mov.b64 u, {%0, %1};\n mov.b64 v, {%2, %3};\n fma.rn.f32x2 u, v, v, u;\n mov.b64 {%0, %1}, u;\n}\n"
      : "+f"(s), "+f"(t)
      : "f"(a), "f"(b));
}
template <int N>
__device__ __forceinline__ void scale_all(float (&v)[N], float c) {
#pragma unroll
  for (int i = 0; i < N; i += 2) mul2(v[i], v[i + 1], c, c);
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
// sum of squares comes near the end of the 32-bit range is summed again with
// its values 2^-100 smaller (those that this makes inexact lie 2^70 and more
// below the largest), and its quotients are made 2^-100 smaller after the
// product; infinities and NaN stay what the formula makes of them.
template <int NV>
__device__ __forceinline__ void normalise(float (&v)[NV], float &x, const NormP &P, float *red) {
  float s4[4] = {x * x, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < NV; i += 2) squares2(s4[i & 3], s4[(i & 3) + 1], v[i], v[i + 1]);
  bool large, any;
  float ss = row_sum((s4[0] + s4[1]) + (s4[2] + s4[3]), P.T, red, any), eps = P.eps, c = 1.f;
  if (any) {
    if (!(ss < 1e37f)) c = 7.888609052210118e-31f;
    float again = c * x * (c * x);
#pragma unroll
    for (int i = 0; i < NV; i++) again = fmaf(c * v[i], c * v[i], again);
    again = row_sum(again, P.T, red + 32, large);
    if (c != 1.f) ss = again, eps = eps * c * c;  // (a row beside such a one keeps its own sum)
  }
  const float m = fmaf(ss, P.inv_h, eps), r = rsqrtf(m);
  // one step of Newton's: the root's error is the last bit's (e4m3 values
  // next to a border are told apart as by a division)
  const float inv = m < 1e38f ? fmaf(0.5f * r, fmaf(-m * r, r, 1.f), r) : r;
  x *= inv;
  scale_all(v, inv);
  if (any) x *= c, scale_all(v, c);
}

// SH (V = 8): rows that do not start on 16 bytes, but all matrices' alike: the
// pieces begin `lead` values into a row, on 16 bytes; those before them and the
// last ones are one value more for 16 of the row's threads.  Blocks walk over
// the rows by a multiple of 8, so that a thread's columns stay the same ones;
// what is per column lies in shared memory as each thread will read it.
constexpr int kMaxVec = 96 * 1024;  // bytes of those
struct Vecs {
  const float4 *w, *wp, *g;  // halves of pieces, blockDim apart
  float xw, xwp, xg;         // of the value more
};

__device__ __forceinline__ float load1(const void *p, int bf16, int64_t i) {
  float v;
  if (bf16) load_as<1, true>(p, i, &v);
  else load_as<1, false>(p, i, &v);
  return v;
}
__device__ __forceinline__ float gate_of(const NormP &P, float g) { return P.gate_sigmoid && g == g ? logistic(g) : g; }

// Which of a block's rows is a thread's (T up to 32 is a power of two; above, a
// block has one row).
__device__ __forceinline__ int row_of(int T, int thread) { return T <= 32 ? thread >> (31 - __clz(T)) : 0; }

// What a thread holds of a row: pieces of V columns, and, SH, one value more.
template <int V, int NV, bool SH>
struct Place {
  int T, l, h, lead, xc;  // xc: its column, < 0: none
  __device__ __forceinline__ Place(const NormP &P, int64_t row, int thread) {
    // (either is right; each where it costs fewer registers: 30011 x 4090 195 us
    // against 229, to e4m3 65536 x 2048 94 against 98)
    T = P.T, l = (SH ? T >= (int)blockDim.x : T > 32) ? thread : thread & (T - 1);
    h = row < P.t ? P.h : 0, lead = SH ? (int)(-((row & 7) * P.ld8) & 7) : 0, xc = -1;
    if (SH && l < 8 && l < lead) xc = l;
    if (SH && l >= 8 && l < 16) xc = h - (h - lead) % 8 + l - 8;
    if (xc >= h) xc = -1;
  }
  __device__ __forceinline__ int col(int j) const { return lead + (j * T + l) * V; }
  template <class F>
  __device__ __forceinline__ void pieces(F f) const {
#pragma unroll
    for (int j = 0; j < NV / V; j++)
      if (col(j) + (SH ? V : 1) <= h) f(j);
  }
};

// The next rows' values on their way to shared memory (RING), copied by the
// warp that will hold them, 16 bytes a lane, neighbouring lanes neighbouring
// bytes: of bf16 a thread copies its own pieces, of fp32 the first 16 lanes'
// pieces are a copy of the whole warp's and the others' the next (each lane
// its own two halves: every 32 bytes asked for twice, 310 us instead of 184 at
// 32768 x 2048).
constexpr int kRing = 2;  // (3: fewer blocks fit; 30011 x 4090 254 us instead of 214)
constexpr int kMaxRing = 200 * 1024;
struct Ring {
  uint8_t *y, *res;  // a place is [pieces][blockDim][values of a piece]
};
// bytes of a thread's row of NV values
__host__ __device__ constexpr int ring_row(int nv, int bf16) { return nv * (bf16 ? 2 : 4); }

// The copies of the rows first + (thread / T), into the ring's place `at`.
template <int V, int NV, bool ADD, bool SH>
__device__ __forceinline__ void row_copies(const NormP &P, int64_t first, const Ring &ring, int at) {
  const int lane = threadIdx.x & 31;
  auto copy = [&](const void *p, int bf16, int64_t ld, uint8_t *to) {
    to += (size_t)at * ring_row(NV, bf16) * blockDim.x;
    if (bf16) {
      const int64_t row = first + row_of(P.T, threadIdx.x);
      const Place<V, NV, SH> L(P, row, threadIdx.x);
      L.pieces([&](int j) {
        cp_async16(to + ((size_t)j * blockDim.x + threadIdx.x) * 16, static_cast<const uint16_t *>(p) + row * ld + L.col(j));
      });
    } else {
#pragma unroll
      for (int c = 0; c < 2; c++) {
        const int thread = (int)threadIdx.x - lane + 16 * c + (lane >> 1);
        const int64_t row = first + row_of(P.T, thread);
        const Place<V, NV, SH> L(P, row, thread);
        L.pieces([&](int j) {
          cp_async16(to + ((size_t)j * blockDim.x + thread) * 32 + 16 * (lane & 1),
                     static_cast<const float *>(p) + row * ld + L.col(j) + 4 * (lane & 1));
        });
      }
    }
  };
  copy(P.y, P.y_bf16, P.ldy, ring.y);
  if constexpr (ADD) copy(P.res, P.res_bf16, P.ldr, ring.res);
}

// One row, in the registers of T threads (all of a warp's, or a block's, come
// here together).  RING: its values lie in the ring's place `at`, but for the
// one more, which is x0 and r0.
template <int V, int NV, bool ADD, bool SH, bool RING>
__device__ __forceinline__ void one_row(const NormP &P, int64_t row, float (&red)[4][32], const Vecs &vecs, uint32_t *s_max,
                                        const Ring &ring = Ring(), int at_ring = 0, float x0 = 0.f, float r0 = 0.f) {
  constexpr int N = NV / V;
  const Place<V, NV, SH> L(P, row, threadIdx.x);
  const int T = L.T, l = L.l, h = L.h, xc = L.xc;
  const bool live = row < P.t;
  auto col = [&](int j) { return L.col(j); };
  auto pieces = [&](auto f) { L.pieces(f); };
  auto load = [&](const void *p, int bf16, int64_t at, float *to, float &x, const uint8_t *from, float value) {
    if constexpr (RING) {
      from += (size_t)at_ring * ring_row(NV, bf16) * blockDim.x;
      if (bf16) pieces([&](int j) { load_as<8, true>(from + ((size_t)j * blockDim.x + threadIdx.x) * 16, 0, to + j * 8); });
      else pieces([&](int j) { load_as<8, false>(from + ((size_t)j * blockDim.x + threadIdx.x) * 32, 0, to + j * 8); });
      x = value;
      return;
    }
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
  auto weigh = [&](const float *weights, const float4 *mine, float xw) {
    pieces([&](int j) {
      float w[V];
      if constexpr (SH) {
        const float4 a = mine[2 * j * blockDim.x], b = mine[(2 * j + 1) * blockDim.x];
        w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
      } else {
        load_as<V, false>(weights, col(j), w);
      }
      if constexpr (V > 1) {
#pragma unroll
        for (int i = 0; i < V; i += 2) mul2(v[j * V + i], v[j * V + i + 1], w[i], w[i + 1]);
      } else {
        v[j] *= w[0];
      }
    });
    if (SH) x *= xw;
  };
#pragma unroll
  for (int i = 0; i < NV; i++) v[i] = 0.f;
  load(P.y, P.y_bf16, row * P.ldy, v, x, ring.y, x0);
  if constexpr (ADD) {
    float r[NV], rx = 0.f;  // on its way before the first store: the residual may be what is written
#pragma unroll
    for (int i = 0; i < NV; i++) r[i] = 0.f;
    load(P.res, P.res_bf16, row * P.ldr, r, rx, ring.res, r0);
    if (P.post) {
      normalise(v, x, P, red[0]);
      if (P.wp) weigh(P.wp, vecs.wp, vecs.xwp);
    }
    // (gate by value first: a gate of 0 closes, whatever the scale)
    if (P.gate) {
      if (P.gate_cols == 1) {
        const float g = live ? gate_of(P, load1(P.gate, P.gate_bf16, row * P.ldg)) : 1.f;
        x *= g;
        scale_all(v, g);
      } else if (SH && P.ldg == 0) {
        weigh(nullptr, vecs.g, vecs.xg);
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
    scale_all(r, P.res_scale);
#pragma unroll
    for (int i = 0; i < NV; i += 2) fma2(v[i], v[i + 1], P.scale, P.scale, r[i], r[i + 1]);
    store(P.ro, P.ro_bf16, row * P.ldro);
    if (P.out_kind == kNormOutNone) return;
  }
  normalise(v, x, P, red[2]);
  if (P.w) weigh(P.w, vecs.w, vecs.xw);
  if (P.out_kind != kNormOutE4m3) {
    store(P.out, P.out_kind == kNormOutBf16, row * P.ldo);
    return;
  }
  if constexpr (SH) return;  // (not launched so)
  uint8_t *q = static_cast<uint8_t *>(P.out) + row * P.ldo, *s = P.s + row * P.lds;
  if constexpr (V == 8) {
    // 16 lanes hold a scale block.  All pieces' maxima together, as each is a
    // chain of exchanges (one piece after the other: 65536 x 2048 111 us
    // instead of 103).  NaN does not count in them and stays one in the
    // conversion; an infinity makes the warp do it with care.
    float a[N], am = 0.f;
#pragma unroll
    for (int j = 0; j < N; j++) {
      a[j] = 0.f;
#pragma unroll
      for (int i = 0; i < 8; i++) a[j] = fmaxf(a[j], fabsf(v[j * 8 + i]));
    }
#pragma unroll
    for (int o = 8; o; o >>= 1)
#pragma unroll
      for (int j = 0; j < N; j++) a[j] = fmaxf(a[j], __shfl_xor_sync(FULLM, a[j], o));
#pragma unroll
    for (int j = 0; j < N; j++) am = fmaxf(am, a[j]);
    const bool care = __any_sync(FULLM, !(am <= 3.402823466e38f));
#pragma unroll
    for (int j = 0; j < N; j++) {
      uint32_t w[2], e;
      float b[8];
#pragma unroll
      for (int i = 0; i < 8; i++) b[i] = v[j * 8 + i];
      if (care) {
        quant_block<8>(b, w, e);
      } else {
        e = e8m0_of_amax(__float_as_uint(a[j]));
        scale_all(b, e8m0_inv(e));
        w[0] = e4m3x4<false>(b[0], b[1], b[2], b[3]);
        w[1] = e4m3x4<false>(b[4], b[5], b[6], b[7]);
      }
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

// Without SH and RING the grid covers the rows; with them, blocks walk over them.
template <int V, int NV, bool ADD, bool SH, bool RING>
__global__ void __launch_bounds__(kMaxThreads, NV <= 16 ? 2 : 0) norm_rows(const __grid_constant__ NormP P) {
  static_assert(V == 8 || !(SH || RING), "");
  constexpr bool WALK = SH || RING;
  __shared__ float s_red[WALK ? 2 : 1][4][32];
  extern __shared__ __align__(16) uint32_t s_dyn[];  // e4m3, V < 8: maxima [N][warps]; the ring; SH: vectors
  pdl_wait_prev();
  pdl_launch_next();
  const int per = row_of(P.T, blockDim.x - 1) + 1, mine = row_of(P.T, threadIdx.x);
  if constexpr (!WALK) {
    one_row<V, NV, ADD, SH, false>(P, (int64_t)blockIdx.x * per + mine, s_red[0], Vecs(), s_dyn);
    return;
  }
  const int64_t step = (int64_t)gridDim.x * per;
  int64_t first = (int64_t)blockIdx.x * per;
  uint8_t *at = reinterpret_cast<uint8_t *>(s_dyn);
  Ring ring = {};
  float x = 0.f, rx = 0.f;
  // the value more of a row, a row ahead
  auto more = [&](int64_t row) {
    if constexpr (SH && RING) {
      const Place<V, NV, SH> L(P, row, threadIdx.x);
      if (L.xc >= 0) {
        x = load1(P.y, P.y_bf16, row * P.ldy + L.xc);
        if constexpr (ADD) rx = load1(P.res, P.res_bf16, row * P.ldr + L.xc);
      } else {
        x = rx = 0.f;
      }
    }
  };
  if constexpr (RING) {
    ring.y = at;
    at += (size_t)kRing * ring_row(NV, P.y_bf16) * blockDim.x;
    if (ADD) {
      ring.res = at;
      at += (size_t)kRing * ring_row(NV, P.res_bf16) * blockDim.x;
    }
#pragma unroll
    for (int i = 0; i < kRing - 1; i++) {
      row_copies<V, NV, ADD, SH>(P, first + i * step, ring, i);
      tc05::cp_commit();
    }
    more(first + mine);
  }
  Vecs vecs = {};
  if constexpr (SH) {
    Place<V, NV, SH> L(P, first + mine < P.t ? first + mine : 0, threadIdx.x);
    auto place = [&](auto get, float &xv) {
      float4 *to = reinterpret_cast<float4 *>(at) + threadIdx.x;
      L.pieces([&](int j) {
        const int c = L.col(j);
        to[2 * j * blockDim.x] = make_float4(get(c), get(c + 1), get(c + 2), get(c + 3));
        to[(2 * j + 1) * blockDim.x] = make_float4(get(c + 4), get(c + 5), get(c + 6), get(c + 7));
      });
      xv = L.xc >= 0 ? get(L.xc) : 0.f;
      at += (size_t)NV * 4 * blockDim.x;
      return to;
    };
    if (P.w) vecs.w = place([&](int c) { return P.w[c]; }, vecs.xw);
    if (ADD && P.wp) vecs.wp = place([&](int c) { return P.wp[c]; }, vecs.xwp);
    if (ADD && P.gate && P.gate_cols != 1 && P.ldg == 0)
      vecs.g = place([&](int c) { return gate_of(P, load1(P.gate, P.gate_bf16, c)); }, vecs.xg);
  }
  int half = 0, slot = 0;  // the next row's sums lie in the other half
  for (; first < P.t; first += step, half ^= 1) {
    if constexpr (RING) {
      __syncwarp();  // the place's values are read
      row_copies<V, NV, ADD, SH>(P, first + (kRing - 1) * step, ring, slot ? slot - 1 : kRing - 1);
      tc05::cp_commit();
      const float x0 = x, r0 = rx;
      more(first + step + mine);
      tc05::cp_wait_group<kRing - 1>();
      __syncwarp();  // of all the warp's copies
      one_row<V, NV, ADD, SH, true>(P, first + mine, s_red[half], vecs, s_dyn, ring, slot, x0, r0);
      if (++slot == kRing) slot = 0;
    } else {
      one_row<V, NV, ADD, SH, false>(P, first + mine, s_red[half], vecs, s_dyn);
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

// Whether the next rows' values are fetched ahead.  us without / with: add_norm
// of bf16 on an fp32 stream 65536 x 2048 286 / 250, 8192 x 8192 181 / 143, on a
// bf16 one 30000 x 4096 222 / 158, 30011 x 4090 243 / 216; all fp32 32768 x
// 2048 160 / 184.  norm of bf16 65536 x 2048 93 / 86, 8192 x 16384 121 / 83,
// 32816 x 4090 (SH) 109 / 116; fp32 32768 x 2048 79 / 88; to e4m3 65536 x 2048
// 102 / 116 (instructions), 8192 x 16384 122 / 104.
bool with_ring(const NormP &p, bool sh) {
  if (!p.y_bf16) return false;
  return p.res || (!sh && (p.out_kind != kNormOutE4m3 || p.h > 8192));
}

// vectors that SH holds in shared memory
int vecs_of(const NormP &p) { return (p.w != nullptr) + (p.wp != nullptr) + (p.gate && p.gate_cols != 1 && p.ldg == 0); }

// Whether no row starts on 16 bytes, but all matrices' rows alike.
bool alike(NormP &p) {
  if (p.out_kind == kNormOutE4m3) return false;
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

// Bytes of shared memory that rows on their way take.
int ring_bytes(const NormP &p, int nv, int block) {
  return kRing * block * (ring_row(nv, p.y_bf16) + (p.res ? ring_row(nv, p.res_bf16) : 0));
}

// Blocks that stay resident walk over the rows; where each has several and
// shared memory allows, with the next row's values on their way.  done:
// launched (without SH only in that case).
template <int NV, bool SH>
cudaError_t launch_walk(NormP p, int T, int n_sms, cudaStream_t st, bool &done) {
  p.T = T;
  const int block = T <= 32 ? 256 : T, rows = block / T;
  const int vecs = SH ? vecs_of(p) * NV * 4 * block : 0;
  const int64_t need = ((int64_t)p.t + rows - 1) / rows;
  static const int regs[4] = {SH ? registers(norm_rows<8, NV, false, SH, false>) : 128, SH ? registers(norm_rows<8, NV, true, SH, false>) : 128,
                              registers(norm_rows<8, NV, false, SH, true>), registers(norm_rows<8, NV, true, SH, true>)};
  if (vecs > kMaxVec) return cudaSuccess;
  for (int ring = with_ring(p, SH) ? 1 : 0; ring >= (SH ? 0 : 1); ring--) {
    const int smem = vecs + (ring ? ring_bytes(p, NV, block) : 0);
    if (smem > kMaxRing) continue;
    int fit = 65536 / (regs[2 * ring + (p.res != nullptr)] * block);
    if (fit > 2048 / block) fit = 2048 / block;
    if (fit > 226 * 1024 / (smem + 2048)) fit = 226 * 1024 / (smem + 2048);
    int64_t cap = (int64_t)n_sms * (fit < 1 ? 1 : fit);
    if (SH && cap > 8) cap -= cap % 8;
    const int64_t rounds = (need + cap - 1) / cap;
    if (ring && rounds < 6) continue;  // (4096 x 2048: 20 us without, 22 with)
    auto f = p.res ? norm_rows<8, NV, true, SH, true> : norm_rows<8, NV, false, SH, true>;
    if constexpr (SH)
      if (!ring) f = p.res ? norm_rows<8, NV, true, SH, false> : norm_rows<8, NV, false, SH, false>;
    if (smem > 46 * 1024) {  // (beside a kilobyte that is there anyway)
      const cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxRing);
      if (e != cudaSuccess) return e;
    }
    done = true;
    int64_t grid = (need + rounds - 1) / rounds;  // each with the same number of rounds
    if (SH && rounds > 1) grid = (grid + 7) / 8 * 8;
    return launch_pdl(f, dim3((unsigned)grid), block, smem, st, p);
  }
  return cudaSuccess;
}

template <int V, int NV>
cudaError_t launch_form(NormP p, int T, cudaStream_t st) {
  p.T = T;
  const int block = T <= 32 ? 128 : T, rows = block / T;  // (T above 32: a block a row)
  const size_t smem = p.out_kind == kNormOutE4m3 && V < 8 ? (size_t)(NV / V) * (block / 32) * 4 : 0;
  const dim3 grid((unsigned)(((int64_t)p.t + rows - 1) / rows));
  return p.res ? launch_pdl(norm_rows<V, NV, true, false, false>, grid, block, smem, st, p)
               : launch_pdl(norm_rows<V, NV, false, false, false>, grid, block, smem, st, p);
}

// Values a thread holds.  What a thread does whatever their number (addresses,
// exchanges, the root) costs as much as some 16: 32 of them, with a residual
// 16, as long as the rows give every SM 64 (200) warps; few rows want many threads.
// us with 8 / 16 / 32 / 64 values, bf16, norm: 65536 rows x 2048 101 / 95 / 89
// / 111, 32768 x 4096 113 / 104 / 97 / 110; one row x 2048 1.8 / 2.1 / 2.4 /
// 3.1.  add_norm (fp32 residual): 65536 x 2048 305 / 286 / 297 / 324.
template <class T>
int values_a_thread(const NormP &p, int n_sms, bool sh, T threads) {
  int nv = 8;
  const int most = p.res || with_ring(p, sh) ? 16 : 32;
  while (nv < most && threads(2 * nv) < threads(nv) && (int64_t)p.t * threads(2 * nv) >= (int64_t)n_sms * (p.res ? 200 : 64) * 32) nv *= 2;
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
  const int nv = values_a_thread(p, n_sms, false, threads), T = threads(nv);
  return nv == 8 ? launch_form<V, 8>(p, T, st) : (nv == 16 ? launch_form<V, 16>(p, T, st) :
         (nv == 32 ? launch_form<V, 32>(p, T, st) : launch_form<V, 64>(p, T, st)));
}

}  // namespace

cudaError_t launch_norm(NormP p, int n_sms, cudaStream_t st) {
  const int v = piece(p);
  const bool sh = v < 8 && p.h >= 32 && alike(p);
  auto threads = [&](int nv) { return threads_for(p.h, nv, 16); };
  if (sh || (v == 8 && p.h >= 256)) {  // (shorter rows of whole pieces have fewer threads than a walk takes)
    const int nv = values_a_thread(p, n_sms, sh, threads), T = threads(nv);
    bool done = false;
    cudaError_t e = cudaSuccess;
    if (sh) e = nv == 8 ? launch_walk<8, true>(p, T, n_sms, st, done) : (nv == 16 ? launch_walk<16, true>(p, T, n_sms, st, done) :
                (nv == 32 ? launch_walk<32, true>(p, T, n_sms, st, done) : cudaSuccess));
    else e = nv == 8 ? launch_walk<8, false>(p, T, n_sms, st, done) : (nv == 16 ? launch_walk<16, false>(p, T, n_sms, st, done) :
             (nv == 32 ? launch_walk<32, false>(p, T, n_sms, st, done) : cudaSuccess));
    if (done || e != cudaSuccess) return e;
  }
  return v == 8 ? launch_v<8>(p, n_sms, st) : (v == 2 ? launch_v<2>(p, n_sms, st) : launch_v<1>(p, n_sms, st));
}

}  // namespace moe
