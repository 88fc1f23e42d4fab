// experts8.cu -- the routed experts' step over 8-bit weights, from given ids
// and weights.
//
// Few rows (decode, verify): two kernels that stream the union's weights
// once.  Every row is a column of the m16n8 tiles, whether it chose the
// expert or not, so no row lists are built; a CTA whose expert stands
// earlier in the id table leaves at once, so no union is built either.
//   gate_up  a cluster of 8 CTAs per (entry, 128 channels): each CTA streams
//            16 gate and 16 up rows, its warps split k; the cluster shares
//            the 128 channels' maxima and every CTA writes its h in e4m3
//   down     a CTA per 16 output rows over all experts of the union: its
//            warps split (expert, k block), sums meet in a fixed order
// Many rows: the entries are grouped by expert (count, scan), x is quantised
// once per row and written to its entries' places, mm8_tc computes h8 and
// the outputs y, and a last kernel sums a row's weighted outputs in the
// order of its entries.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include "fp8.cuh"

namespace cg = cooperative_groups;

namespace moe {
namespace {

constexpr unsigned FULLM = 0xffffffffu;
constexpr int kWarps = 8, kThreads = 32 * kWarps;

__device__ __forceinline__ void pdl_launch_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void pdl_wait_prev() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

__device__ __forceinline__ void mma_e4m3(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// one k block of 128: 16 weight rows (pieces at 16q and 64 + 16q of rows g
// and g + 8) times eight rows of x (the same pieces of row g)
struct Frag {
  uint4 a[2][2];
};
__device__ __forceinline__ void load_frag(Frag &f, const uint8_t *row_g, size_t ld8) {
  f.a[0][0] = ldg_stream4(row_g);
  f.a[0][1] = ldg_stream4(row_g + ld8);
  f.a[1][0] = ldg_stream4(row_g + 64);
  f.a[1][1] = ldg_stream4(row_g + 64 + ld8);
}
__device__ __forceinline__ void mma_frag(float (&d)[4], const Frag &f, const uint4 &b0, const uint4 &b1) {
  mma_e4m3(d, f.a[0][0].x, f.a[0][1].x, f.a[0][0].y, f.a[0][1].y, b0.x, b0.y);
  mma_e4m3(d, f.a[0][0].z, f.a[0][1].z, f.a[0][0].w, f.a[0][1].w, b0.z, b0.w);
  mma_e4m3(d, f.a[1][0].x, f.a[1][1].x, f.a[1][0].y, f.a[1][1].y, b1.x, b1.y);
  mma_e4m3(d, f.a[1][0].z, f.a[1][1].z, f.a[1][0].w, f.a[1][1].w, b1.z, b1.w);
}

// eight consecutive values of x
template <bool BF16>
__device__ __forceinline__ void load_x8(const void *x, int64_t i, float (&v)[8]) {
  if (BF16) {
    const uint4 u = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(x) + i);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; j++) v[2 * j] = bf16lo(w[j]), v[2 * j + 1] = bf16hi(w[j]);
  } else {
    const float4 a = *reinterpret_cast<const float4 *>(static_cast<const float *>(x) + i);
    const float4 b = *reinterpret_cast<const float4 *>(static_cast<const float *>(x) + i + 4);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
}

// Half a warp: the 128 values its lanes hold eight each of -> e4m3, scale byte
__device__ __forceinline__ uint2 quant128(const float (&v)[8], uint32_t &e) {
  uint32_t a = 0;
#pragma unroll
  for (int j = 0; j < 8; j++) a = max(a, mag_bits(v[j]));
#pragma unroll
  for (int o = 8; o; o >>= 1) a = max(a, __shfl_xor_sync(FULLM, a, o));
  e = e8m0_of_amax(a);
  const float f = e8m0_inv(e);
  return make_uint2(e4m3x4(v[0] * f, v[1] * f, v[2] * f, v[3] * f), e4m3x4(v[4] * f, v[5] * f, v[6] * f, v[7] * f));
}

// ------------------------------------------------------------ few rows

__host__ __device__ constexpr int xs_stride(int H) { return H + 64; }  // rows 64 bytes apart in the banks
size_t gate_up_smem(int H) { return (size_t)kEx8SmallRows * (xs_stride(H) + (H / 128) * 4); }

template <bool BF16>
__global__ void __cluster_dims__(8, 1, 1) __launch_bounds__(kThreads) ex8_gate_up(const __grid_constant__ Ex8P P) {
  pdl_launch_next();
  extern __shared__ __align__(16) uint8_t xs[];  // [8][H + 64] e4m3 rows of x, then float [8][H / 128] scales
  __shared__ float red[kWarps][32][9];
  __shared__ uint32_t amax[8];  // this CTA's maxima of h per row
  float *sx = reinterpret_cast<float *>(xs + kEx8SmallRows * xs_stride(P.H));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q = lane & 3;
  const int H = P.H, I = P.I, K = P.K, nk = H / 128, n = P.t * K, entry = blockIdx.y;
  if (blockIdx.x == 0 && entry == 0 && tid == 0) *P.status = 0;
  const uint32_t ex = P.idx[entry];
  // the cluster leaves as one: its CTAs share the entry
  bool dup = false;
  for (int j = tid; j < entry; j += kThreads) dup |= P.idx[j] == ex;
  if (__syncthreads_or(dup) || ex >= (uint32_t)P.E) return;
  unsigned used = 0;  // rows that chose this expert
  for (int j = 0; j < n; j++)
    if (P.idx[j] == ex) used |= 1u << (j / K);

  const int c0 = blockIdx.x * 16;  // first of this CTA's channels
  const uint8_t *wg = P.gu + ((size_t)ex * 2 * I + c0 + g) * H + q * 16, *wu = wg + (size_t)I * H;
  const size_t ld8 = (size_t)8 * H;
  Frag fg, fu;
  if (warp < nk) {
    load_frag(fg, wg + (size_t)warp * 128, ld8);
    load_frag(fu, wu + (size_t)warp * 128, ld8);
  }
  // the rows that chose the expert, in e4m3 (the others' columns are zeros)
  for (int b = warp * 2; b < kEx8SmallRows * nk; b += 2 * kWarps) {
    const int bb = b + (lane >> 4), r = bb / nk, kb = bb - r * nk, c = kb * 128 + (lane & 15) * 8;
    const bool on = bb < kEx8SmallRows * nk && ((used >> r) & 1u);
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (on) load_x8<BF16>(P.x, (int64_t)r * H + c, v);
    uint32_t e;
    const uint2 u = quant128(v, e);
    if (bb < kEx8SmallRows * nk) {
      *reinterpret_cast<uint2 *>(xs + r * xs_stride(H) + c) = u;
      if ((lane & 15) == 0) sx[r * nk + kb] = e8m0_f(e);
    }
  }
  __syncthreads();
  const uint8_t *sgp = P.gus + ((size_t)ex * (2 * I / 128) + c0 / 128) * nk, *sup = sgp + (size_t)(I / 128) * nk;
  float ag[4] = {0.f, 0.f, 0.f, 0.f}, au[4] = {0.f, 0.f, 0.f, 0.f};
  for (int kb = warp; kb < nk; kb += kWarps) {
    const Frag cg_ = fg, cu_ = fu;
    if (kb + kWarps < nk) {
      load_frag(fg, wg + (size_t)(kb + kWarps) * 128, ld8);
      load_frag(fu, wu + (size_t)(kb + kWarps) * 128, ld8);
    }
    const uint8_t *xr = xs + g * xs_stride(H) + kb * 128 + q * 16;
    const uint4 b0 = *reinterpret_cast<const uint4 *>(xr), b1 = *reinterpret_cast<const uint4 *>(xr + 64);
    float dg[4] = {0.f, 0.f, 0.f, 0.f}, du[4] = {0.f, 0.f, 0.f, 0.f};
    mma_frag(dg, cg_, b0, b1);
    mma_frag(du, cu_, b0, b1);
    const float s0 = sx[2 * q * nk + kb], s1 = sx[(2 * q + 1) * nk + kb];
    const float bg = e8m0_f(sgp[kb]), bu = e8m0_f(sup[kb]);
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const float s = (i & 1) ? s1 : s0;
      ag[i] += dg[i] * s * bg;
      au[i] += du[i] * s * bu;
    }
  }
#pragma unroll
  for (int i = 0; i < 4; i++) {
    red[warp][g + 8 * (i >> 1)][2 * q + (i & 1)] = ag[i];
    red[warp][16 + g + 8 * (i >> 1)][2 * q + (i & 1)] = au[i];
  }
  __syncthreads();
  // thread (row of x r, channel c): h, its maximum over the CTA's 16
  // channels, then over the cluster's 128
  const int r = tid >> 4, c = tid & 15;  // the first four warps
  float h = 0.f;
  if (tid < 128) {
    float gv = 0.f, uv = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; w++) gv += red[w][c][r], uv += red[w][16 + c][r];
    h = gv / (1.f + expf(-gv)) * uv;
    uint32_t a = mag_bits(h);
#pragma unroll
    for (int o = 8; o; o >>= 1) a = max(a, __shfl_xor_sync(FULLM, a, o));
    if (c == 0) amax[r] = a;
  }
  cg::cluster_group cl = cg::this_cluster();
  cl.sync();
  if (tid < 128) {
    // lane c < 8 of a row reads CTA c's maximum
    uint32_t a = c < 8 ? *cl.map_shared_rank(&amax[r], c) : 0u;
#pragma unroll
    for (int o = 8; o; o >>= 1) a = max(a, __shfl_xor_sync(FULLM, a, o));
    const uint32_t e = e8m0_of_amax(a);
    const uint8_t v = (uint8_t)e4m3x2(h * e8m0_inv(e), 0.f);
    if (r < P.t && ((used >> r) & 1u)) {
      // at the row's first entry with this expert
      int j = r * K;
      while (P.idx[j] != ex) j++;
      P.h8[(size_t)j * I + c0 + c] = v;
      if ((blockIdx.x & 7) == 0 && c == 0) P.h8s[(size_t)j * P.ldi + c0 / 128] = (uint8_t)e;
    }
  }
  cl.sync();  // no CTA ends while another may read its maxima
}

constexpr int kMaxEntries = kEx8SmallRows * 32;

template <bool BF16>
__global__ void __launch_bounds__(kThreads) ex8_down(const __grid_constant__ Ex8P P) {
  __shared__ uint32_t ids[kMaxEntries];
  __shared__ int uni[kMaxEntries];  // entries that name an expert first
  __shared__ int nuni, wsum[kWarps];
  __shared__ float red[kWarps][16][9];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q = lane & 3;
  const int H = P.H, I = P.I, K = P.K, nk = I / 128, n = P.t * K, n0 = blockIdx.x * 16;
  if (tid < n) ids[tid] = P.idx[tid];
  __syncthreads();
  bool first = tid < n && ids[tid] < (uint32_t)P.E;
  for (int j = 0; j < tid && first; j++) first = ids[j] != ids[tid];
  const unsigned bal = __ballot_sync(FULLM, first);
  if (lane == 0) wsum[warp] = __popc(bal);
  __syncthreads();
  int base = 0;
  for (int w = 0; w < warp; w++) base += wsum[w];
  if (first) uni[base + __popc(bal & ((1u << lane) - 1u))] = tid;
  if (tid == kThreads - 1) nuni = base + __popc(bal);
  __syncthreads();

  const int items = nuni * nk;  // (expert, k block), k fastest
  auto wrow = [&](int it) {
    const int u = it / nk, kb = it - u * nk;
    return P.dn + ((size_t)ids[uni[u]] * H + n0 + g) * I + kb * 128 + q * 16;
  };
  const size_t ld8 = (size_t)8 * I;
  Frag f;
  if (warp < items) load_frag(f, wrow(warp), ld8);
  pdl_wait_prev();  // h8 is the previous kernel's; the weights above are not
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  for (int it = warp; it < items; it += kWarps) {
    const Frag c = f;
    if (it + kWarps < items) load_frag(f, wrow(it + kWarps), ld8);
    const int u = it / nk, kb = it - u * nk;
    const uint32_t ex = ids[uni[u]];
    // row g's first entry with this expert, and the sum of its weights
    auto entry_of = [&](int r, float *wt) {
      int at = -1;
      float s = 0.f;
      if (r < P.t)
        for (int j = r * K; j < (r + 1) * K; j++)
          if (ids[j] == ex) {
            if (at < 0) at = j;
            s += P.w[j];
          }
      *wt = s;
      return at;
    };
    float wg;
    const int eg = entry_of(g, &wg);
    uint4 b0 = make_uint4(0, 0, 0, 0), b1 = b0;
    float sg = 0.f;
    if (eg >= 0) {
      const uint8_t *hr = P.h8 + (size_t)eg * I + kb * 128 + q * 16;
      b0 = *reinterpret_cast<const uint4 *>(hr);
      b1 = *reinterpret_cast<const uint4 *>(hr + 64);
      sg = e8m0_f(P.h8s[(size_t)eg * P.ldi + kb]) * wg;
    }
    float d[4] = {0.f, 0.f, 0.f, 0.f};
    mma_frag(d, c, b0, b1);
    // scales of columns 2q, 2q + 1: lanes with g = 2q, 2q + 1 hold them
    const float s0 = __shfl_sync(FULLM, sg, 8 * q), s1 = __shfl_sync(FULLM, sg, 8 * q + 4);
    const float fb = e8m0_f(P.dns[((size_t)ex * (H / 128) + (n0 >> 7)) * nk + kb]);
#pragma unroll
    for (int i = 0; i < 4; i++) {
      // a column whose row did not choose the expert adds nothing, whatever
      // the product is (a NaN weight times zero)
      const float s = (i & 1) ? s1 : s0;
      const int col = 2 * q + (i & 1);
      const bool on = __shfl_sync(FULLM, eg, 4 * col) >= 0;
      if (on) acc[i] += d[i] * fb * s;
    }
  }
#pragma unroll
  for (int i = 0; i < 4; i++) red[warp][g + 8 * (i >> 1)][2 * q + (i & 1)] = acc[i];
  __syncthreads();
  if (tid < 128) {
    const int row = tid & 15, r = tid >> 4;
    if (r < P.t) {
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; w++) v += red[w][row][r];
      const size_t o = (size_t)r * H + n0 + row;
      if (BF16) {
        uint16_t b;
        asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(b) : "f"(v));
        static_cast<uint16_t *>(P.out)[o] = b;
      } else {
        static_cast<float *>(P.out)[o] = v;
      }
    }
  }
}

// ------------------------------------------------------------ many rows

constexpr int kCountEntries = 1024;

// Place of every entry within its expert's rows.  A block counts its entries
// in shared memory and takes a run of places per expert; which places an
// entry gets depends on the order of the blocks, its results do not.  The
// last block to finish scans the counts.
__global__ void __launch_bounds__(256) ex8_count(const __grid_constant__ Ex8P P) {
  extern __shared__ int hist[];  // [E]
  __shared__ int last, part[9];
  const int tid = threadIdx.x, lane = tid & 31, n = P.t * P.K, E = P.E;
  for (int e = tid; e < E; e += 256) hist[e] = 0;
  __syncthreads();
  uint32_t ex[4];
  int rank[4];
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const int j = blockIdx.x * kCountEntries + i * 256 + tid;
    ex[i] = j < n ? P.idx[j] : 0xffffffffu;
    rank[i] = ex[i] < (uint32_t)E ? atomicAdd(&hist[ex[i]], 1) : 0;
  }
  __syncthreads();
  for (int e = tid; e < E; e += 256) {
    const int c = hist[e];
    hist[e] = c ? atomicAdd(&P.counts[e], c) : 0;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const int j = blockIdx.x * kCountEntries + i * 256 + tid;
    if (j < n) P.place[j] = ex[i] < (uint32_t)E ? hist[ex[i]] + rank[i] : -1;
  }
  __threadfence();
  __syncthreads();
  if (tid == 0) last = atomicAdd(&P.counts[E], 1) == (int)gridDim.x - 1;
  __syncthreads();
  if (!last) return;
  __threadfence();
  // four experts a thread: exclusive scan of the counts
  int c[4], sum = 0;
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const int e = 4 * tid + i;
    c[i] = e < E ? __ldcg(&P.counts[e]) : 0;
    sum += c[i];
  }
  int x = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(FULLM, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) part[tid >> 5] = x;
  __syncthreads();
  int base = x - sum;
  for (int w = 0; w < (tid >> 5); w++) base += part[w];
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const int e = 4 * tid + i;
    if (e <= E) P.offs[e] = base;
    base += c[i];
  }
  if (E == 1024 && tid == 255) P.offs[E] = base;
}

// x rows -> e4m3, written to the places of their entries: a warp per row.
template <bool BF16>
__global__ void __launch_bounds__(kThreads) ex8_scatter(const __grid_constant__ Ex8P P) {
  const int row = blockIdx.x * kWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (row >= P.t) return;
  const int K = P.K, H = P.H;
  int at = -1;
  if (lane < K) {
    const int j = row * K + lane, pl = P.place[j];
    if (pl >= 0) at = P.offs[P.idx[j]] + pl;
    P.place[j] = at;  // from here on: the entry's row
  }
  for (int c0 = 0; c0 < H; c0 += 256) {
    const int c = c0 + lane * 8;
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (c < H) load_x8<BF16>(P.x, (int64_t)row * H + c, v);
    uint32_t e;
    const uint2 u = quant128(v, e);
    for (int j = 0; j < K; j++) {
      const int a = __shfl_sync(FULLM, at, j);
      if (a >= 0 && c < H) {
        *reinterpret_cast<uint2 *>(P.x8 + (size_t)a * H + c) = u;
        if ((lane & 15) == 0) P.x8s[(size_t)a * P.ldh + c / 128] = (uint8_t)e;
      }
    }
  }
}

// out[row] = sum over the row's entries, in order, of weight * y
template <bool BF16>
__global__ void __launch_bounds__(256) ex8_combine(const __grid_constant__ Ex8P P) {
  __shared__ int at[32];
  __shared__ float wt[32];
  pdl_wait_prev();
  const int row = blockIdx.x, K = P.K, H = P.H;
  if (threadIdx.x < K) {
    at[threadIdx.x] = P.place[row * K + threadIdx.x];
    wt[threadIdx.x] = P.w[row * K + threadIdx.x];
  }
  __syncthreads();
  for (int c = threadIdx.x * 8; c < H; c += 256 * 8) {
    float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int j = 0; j < K; j++) {
      if (at[j] < 0) continue;
      float v[8];
      load_x8<BF16>(P.y, (int64_t)at[j] * H + c, v);
#pragma unroll
      for (int i = 0; i < 8; i++) s[i] += wt[j] * v[i];
    }
    if (BF16) {
      uint32_t u[4];
#pragma unroll
      for (int i = 0; i < 4; i++) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u[i]) : "f"(s[2 * i + 1]), "f"(s[2 * i]));
      *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(P.out) + (size_t)row * H + c) = make_uint4(u[0], u[1], u[2], u[3]);
    } else {
      float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(P.out) + (size_t)row * H + c);
      o[0] = make_float4(s[0], s[1], s[2], s[3]);
      o[1] = make_float4(s[4], s[5], s[6], s[7]);
    }
  }
}

size_t al(size_t n) { return (n + 1023) & ~(size_t)1023; }

template <class F>
cudaError_t launch_pdl(F f, dim3 grid, unsigned block, size_t smem, cudaStream_t st, const Ex8P &p) {
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, f, p);
}

}  // namespace

bool ex8_small(int H, int I, int t, int K) { return t <= kEx8SmallRows && gate_up_smem(H) <= 200 * 1024; }

Ex8Sizes ex8_sizes(int H, int E, int I, int t, int K, int out_size) {
  const size_t n = (size_t)t * K;
  const size_t ldi = (size_t)(I / 128 + 3) / 4 * 4, ldh = (size_t)(H / 128 + 3) / 4 * 4;
  Ex8Sizes s{};
  s.h8 = al(n * I), s.h8s = al(n * ldi);
  s.total = s.h8 + s.h8s;
  if (!ex8_small(H, I, t, K)) {
    s.x8 = al(n * H), s.x8s = al(n * ldh);
    s.counts = al((size_t)(E + 1) * 4), s.offs = al((size_t)(E + 1) * 4), s.place = al(n * 4);
    s.y = al(n * H * out_size);
    s.total += s.x8 + s.x8s + s.counts + s.offs + s.place + s.y;
  }
  return s;
}

cudaError_t launch_ex8_small(const Ex8P &p, cudaStream_t st) {
  const size_t smem = gate_up_smem(p.H);
  auto f = p.x_bf16 ? ex8_gate_up<true> : ex8_gate_up<false>;
  if (smem > 32 * 1024) {
    cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  f<<<dim3((unsigned)(p.I / 16), (unsigned)(p.t * p.K)), kThreads, smem, st>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_pdl(p.out_bf16 ? ex8_down<true> : ex8_down<false>, dim3((unsigned)(p.H / 16)), kThreads, 0, st, p);
}

cudaError_t launch_ex8_group(const Ex8P &p, int n_sms, cudaStream_t st) {
  (void)n_sms;
  cudaError_t e = cudaMemsetAsync(p.counts, 0, (size_t)(p.E + 1) * 4, st);
  if (e != cudaSuccess) return e;
  const int n = p.t * p.K;
  ex8_count<<<(unsigned)((n + kCountEntries - 1) / kCountEntries), 256, (size_t)p.E * 4, st>>>(p);
  const unsigned grid = (unsigned)((p.t + kWarps - 1) / kWarps);
  if (p.x_bf16) ex8_scatter<true><<<grid, kThreads, 0, st>>>(p);
  else ex8_scatter<false><<<grid, kThreads, 0, st>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_ex8_combine(const Ex8P &p, cudaStream_t st) {
  return launch_pdl(p.out_bf16 ? ex8_combine<true> : ex8_combine<false>, dim3((unsigned)p.t), 256, 0, st, p);
}

}  // namespace moe
