// quant8.cu -- quantisation to e4m3 with one E8M0 scale per 128 values of a
// row (activations) or per 128 x 128 block (weights).
//
// The scale 2^e is a power of two, so x * 2^-e is exact and each value is
// rounded once, by the hardware conversion.  Both kernels read every value
// once and hold it in registers between the maximum and the conversion: the
// bound is HBM (2 or 4 bytes read, 1 written per value).  16300 x 4112 floats
// in blocks: 52 us, 6.5 TB/s.  4096 x 2048 bf16 in rows: 7.4 us back to back,
// the bytes 3.7.
#include <cuda_runtime.h>

#include "fp8.cuh"

namespace moe {
namespace {

constexpr unsigned FULLM = 0xffffffffu;

template <bool BF16>
__device__ __forceinline__ float load1(const void *x, int64_t i) {
  if (BF16) return __uint_as_float((uint32_t)static_cast<const uint16_t *>(x)[i] << 16);
  return static_cast<const float *>(x)[i];
}

// eight values from element i on; VEC: 16-byte loads, all inside the row
template <bool BF16, bool VEC>
__device__ __forceinline__ void load8(const void *x, int64_t i, int n, float (&v)[8]) {
  if (VEC) {
    if (n <= 0) {
#pragma unroll
      for (int j = 0; j < 8; j++) v[j] = 0.f;
    } else if (BF16) {
      const uint4 u = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(x) + i);
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int j = 0; j < 4; j++) v[2 * j] = bf16lo(w[j]), v[2 * j + 1] = bf16hi(w[j]);
    } else {
      const float4 a = *reinterpret_cast<const float4 *>(static_cast<const float *>(x) + i);
      const float4 b = *reinterpret_cast<const float4 *>(static_cast<const float *>(x) + i + 4);
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; j++) v[j] = j < n ? load1<BF16>(x, i + j) : 0.f;
  }
}

template <bool VEC>
__device__ __forceinline__ void store8(uint8_t *q, int n, uint32_t lo, uint32_t hi) {
  if (VEC) {
    if (n > 0) *reinterpret_cast<uint2 *>(q) = make_uint2(lo, hi);
  } else {
#pragma unroll
    for (int j = 0; j < 8; j++)
      if (j < n) q[j] = (uint8_t)((j < 4 ? lo : hi) >> (8 * (j & 3)));
  }
}

// Half a warp per row block of 128, eight values a lane; the half warps walk
// the blocks of all rows in turn, the next block's load in flight while one
// is converted.  The step from block to block is counted, not divided: some
// 80 instructions a block are what bounds this kernel beside HBM.
template <bool BF16, bool VEC>
__global__ void __launch_bounds__(256) quant_rows(const __grid_constant__ Quant8P P) {
  pdl_wait_prev();
  pdl_launch_next();
  const int cb = (P.cols + 127) / 128, sub = threadIdx.x & 15;
  const int step = gridDim.x * 16, step_r = step / cb, step_b = step - step_r * cb;
  const int i0 = blockIdx.x * 16 + (threadIdx.x >> 4);
  int row = i0 / cb, b = i0 - row * cb;
  float next[8];
  auto load = [&](int r, int bb) {
    const int c = bb * 128 + sub * 8;
    load8<BF16, VEC>(P.x, (int64_t)r * P.ldx + c, r < P.rows ? min(8, P.cols - c) : 0, next);
  };
  load(row, b);
  // both halves of a warp take part in the exchange: it walks on while either
  // has a block
  while (__any_sync(FULLM, row < P.rows)) {
    const int r = row, bb = b, n = r < P.rows ? min(8, P.cols - bb * 128 - sub * 8) : 0;
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; j++) v[j] = next[j];
    b += step_b, row = min(row + step_r, P.rows);
    if (b >= cb) b -= cb, row = min(row + 1, P.rows);
    load(row, b);
    uint32_t w[2], e;
    quant_block<8>(v, w, e);
    store8<VEC>(P.q + (int64_t)r * P.ldq + bb * 128 + sub * 8, n, w[0], w[1]);
    if (r < P.rows && sub == 0) P.s[(int64_t)r * P.lds + bb] = (uint8_t)e;
  }
}

// One block per 128 x 128 block: thread (16 lanes of a row, 16 rows a pass)
// holds eight rows' eight values.
template <bool BF16, bool VEC>
__global__ void __launch_bounds__(256) quant_blocks(const __grid_constant__ Quant8P P) {
  __shared__ uint32_t red[8];
  pdl_wait_prev();
  pdl_launch_next();
  const int sub = threadIdx.x & 15, r0 = blockIdx.y * 128 + (threadIdx.x >> 4), c = blockIdx.x * 128 + sub * 8;
  float v[8][8];
  uint32_t a = 0;
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const int row = r0 + 16 * i;
    load8<BF16, VEC>(P.x, (int64_t)row * P.ldx + c, row < P.rows ? min(8, P.cols - c) : 0, v[i]);
  }
#pragma unroll
  for (int i = 0; i < 8; i++)
#pragma unroll
    for (int j = 0; j < 8; j++) a = max(a, mag_bits(v[i][j]));
  a = __reduce_max_sync(FULLM, a);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = a;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; w++) a = max(a, red[w]);
  const uint32_t e = e8m0_of_amax(a);
  const float f = e8m0_inv(e);
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const int row = r0 + 16 * i;
    const uint32_t lo = e4m3x4<true>(v[i][0] * f, v[i][1] * f, v[i][2] * f, v[i][3] * f);
    const uint32_t hi = e4m3x4<true>(v[i][4] * f, v[i][5] * f, v[i][6] * f, v[i][7] * f);
    if (row < P.rows) store8<VEC>(P.q + (int64_t)row * P.ldq + c, min(8, P.cols - c), lo, hi);
  }
  if (threadIdx.x == 0) P.s[(int64_t)blockIdx.y * P.lds + blockIdx.x] = (uint8_t)e;
}

// 16-byte loads and 8-byte stores: rows start on them and end on a whole one
bool vec_ok(const Quant8P &p) {
  const uintptr_t xa = reinterpret_cast<uintptr_t>(p.x), qa = reinterpret_cast<uintptr_t>(p.q);
  return (xa & 15) == 0 && (qa & 7) == 0 && p.ldx % 8 == 0 && p.ldq % 8 == 0 && p.cols % 8 == 0;
}

}  // namespace

cudaError_t launch_quant8_rows(const Quant8P &p, int n_sms, cudaStream_t st) {
  // as many thread blocks as stay resident, each with the same number of rounds
  const int64_t need = ((int64_t)p.rows * ((p.cols + 127) / 128) + 15) / 16, cap = (int64_t)n_sms * 8;
  const int64_t rounds = (need + cap - 1) / cap;
  const unsigned grid = (unsigned)((need + rounds - 1) / rounds);
  const bool v = vec_ok(p);
  auto f = p.bf16 ? (v ? quant_rows<true, true> : quant_rows<true, false>) : (v ? quant_rows<false, true> : quant_rows<false, false>);
  return launch_pdl(f, dim3(grid), 256, 0, st, p);
}

cudaError_t launch_quant8_blocks(const Quant8P &p, cudaStream_t st) {
  const dim3 grid((unsigned)((p.cols + 127) / 128), (unsigned)((p.rows + 127) / 128));
  const bool v = vec_ok(p);
  auto f = p.bf16 ? (v ? quant_blocks<true, true> : quant_blocks<true, false>)
                  : (v ? quant_blocks<false, true> : quant_blocks<false, false>);
  return launch_pdl(f, grid, 256, 0, st, p);
}

}  // namespace moe
