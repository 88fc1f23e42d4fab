// api8.cu -- C ABI of the 8-bit experts: argument checks and launches.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <initializer_list>

#include "api.cuh"
#include "fp8.cuh"
#include "moe_api.h"

namespace {

using moe::fail;
using moe::overlap;

constexpr int kMaxRows = 1 << 20;   // 2^25 entries at the most
constexpr int kMaxCount = 1 << 30;  // row and column indices step within 32 bits

int dtype_size(int d) { return d == MOE_F32 ? 4 : (d == MOE_BF16 ? 2 : 0); }

int sm_count(int *n) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return fail(MOE_ECUDA, "device query failed");
  return MOE_OK;
}

// bytes from the first to the last element of rows x cols, ld elements apart
size_t span(int64_t rows, int64_t cols, int64_t ld, int size) {
  return rows < 1 ? 0 : ((size_t)(rows - 1) * ld + cols) * size;
}

// The device status is a word of its own: the kernels zero it while they read
// and write the other buffers.
struct Buf {
  const void *p;
  size_t n;
};
int check_status(const int *st, std::initializer_list<Buf> bufs) {
  if ((uintptr_t)st & 3u) return fail(MOE_EALIGN, "dev_status is misaligned");
  for (const Buf &b : bufs)
    if (b.p && overlap(st, 4, b.p, b.n)) return fail(MOE_EINVAL, "dev_status lies in another buffer");
  return MOE_OK;
}

int check_layer8(const moe_layer8 *L, int t, int top_k) {
  if (!L) return fail(MOE_EINVAL, "layer is NULL");
  if (t < 0 || t > kMaxRows) return fail(MOE_EINVAL, "t %d outside 0..%d", t, kMaxRows);
  if (top_k < 1 || top_k > 32) return fail(MOE_ESHAPE, "top_k %d outside 1..32", top_k);
  if (L->hidden < 128 || L->hidden % 128 || L->hidden > 16384)
    return fail(MOE_ESHAPE, "hidden %u must be a multiple of 128 in 128..16384", L->hidden);
  if (L->inter < 128 || L->inter % 128 || L->inter > 16384)
    return fail(MOE_ESHAPE, "inter %u must be a multiple of 128 in 128..16384", L->inter);
  if (L->n_experts < 1 || L->n_experts > 1024) return fail(MOE_ESHAPE, "n_experts %u outside 1..1024", L->n_experts);
  return MOE_OK;
}

}  // namespace

extern "C" {

int moe_gate(const moe_gate_cfg *c, const void *logits, int logit_dtype, int64_t ld, const float *bias, int t,
             uint32_t *topk_idx, float *topk_w, moe_stream_t stream) {
  if (!c) return fail(MOE_EINVAL, "cfg is NULL");
  if (c->n_experts < 1 || c->n_experts > 1024) return fail(MOE_ESHAPE, "n_experts %u outside 1..1024", c->n_experts);
  if (c->score != MOE_SCORE_SOFTMAX && c->score != MOE_SCORE_SIGMOID)
    return fail(MOE_EINVAL, "unknown score %u", c->score);
  if (c->flags & ~(uint32_t)MOE_GATE_RENORM) return fail(MOE_EINVAL, "unknown flags 0x%x", c->flags);
  if (!std::isfinite(c->scale)) return fail(MOE_EINVAL, "scale is not finite");
  if (c->n_groups < 1 || c->n_groups > 32 || c->n_experts % c->n_groups)
    return fail(MOE_ESHAPE, "n_groups %u must be in 1..32 and divide n_experts %u", c->n_groups, c->n_experts);
  if (c->top_groups < 1 || c->top_groups > c->n_groups)
    return fail(MOE_ESHAPE, "top_groups %u outside 1..n_groups", c->top_groups);
  if (c->group_top != 1 && c->group_top != 2) return fail(MOE_ESHAPE, "group_top %u is neither 1 nor 2", c->group_top);
  const uint32_t avail = c->n_experts / c->n_groups * c->top_groups;
  if (c->top_k < 1 || c->top_k > 32 || c->top_k > avail)
    return fail(MOE_ESHAPE, "top_k %u outside 1..min(32, %u experts of the chosen groups)", c->top_k, avail);
  const int size = dtype_size(logit_dtype);
  if (!size) return fail(MOE_EINVAL, "unknown logit_dtype %d", logit_dtype);
  if (t < 0 || t > kMaxCount) return fail(MOE_EINVAL, "t %d outside 0..2^30", t);
  if (t == 0) return MOE_OK;
  if (!logits || !topk_idx || !topk_w) return fail(MOE_EINVAL, "logits, topk_idx and topk_w are required");
  if (ld < (int64_t)c->n_experts) return fail(MOE_ESHAPE, "ld %lld below n_experts", (long long)ld);
  if (((uintptr_t)logits % size) || (((uintptr_t)topk_idx | (uintptr_t)topk_w | (uintptr_t)bias) & 3u))
    return fail(MOE_EALIGN, "misaligned pointer");
  const size_t nl = span(t, c->n_experts, ld, size), no = (size_t)t * c->top_k * 4;
  const size_t nb = bias ? (size_t)c->n_experts * 4 : 0;
  if (overlap(logits, nl, topk_idx, no) || overlap(logits, nl, topk_w, no) || overlap(topk_idx, no, topk_w, no) ||
      (bias && (overlap(bias, nb, topk_idx, no) || overlap(bias, nb, topk_w, no))))
    return fail(MOE_EINVAL, "the outputs overlap the inputs or one another");
  moe::GateP p{};
  p.logits = logits, p.bf16 = logit_dtype == MOE_BF16, p.ld = ld, p.bias = bias;
  p.t = t, p.E = (int)c->n_experts, p.K = (int)c->top_k;
  p.sigmoid = c->score == MOE_SCORE_SIGMOID, p.renorm = (c->flags & MOE_GATE_RENORM) != 0;
  p.ng = c->top_groups == c->n_groups ? 1 : (int)c->n_groups;  // every group stays: no group stage
  p.gs = p.E / p.ng, p.top_groups = (int)c->top_groups, p.group_top = (int)c->group_top;
  p.scale = c->scale;
  p.idx = topk_idx, p.w = topk_w;
  int n_sms = 0;
  if (int r = sm_count(&n_sms)) return r;
  const cudaError_t e = moe::launch_gate(p, n_sms, (cudaStream_t)stream);
  if (e != cudaSuccess) return fail(MOE_ECUDA, "launch failed: %s", cudaGetErrorString(e));
  return MOE_OK;
}

int moe_quant8(const void *x, int x_dtype, int64_t ldx, int rows, int cols, int block_rows, uint8_t *q, int64_t ldq,
               uint8_t *s, int64_t lds, moe_stream_t stream) {
  const int size = dtype_size(x_dtype);
  if (!size) return fail(MOE_EINVAL, "unknown x_dtype %d", x_dtype);
  if (block_rows != 1 && block_rows != 128) return fail(MOE_ESHAPE, "block_rows %d is neither 1 nor 128", block_rows);
  if (rows < 0 || rows > kMaxCount || cols < 1 || cols > kMaxCount)
    return fail(MOE_ESHAPE, "rows %d outside 0..2^30 or cols %d outside 1..2^30", rows, cols);
  if (rows == 0) return MOE_OK;
  const int64_t cb = ((int64_t)cols + 127) / 128, rb = ((int64_t)rows + block_rows - 1) / block_rows;
  if (!x || !q || !s) return fail(MOE_EINVAL, "x, q and s are required");
  if (ldx < cols || ldq < cols || lds < cb) return fail(MOE_ESHAPE, "a row stride is below the row's length");
  if (block_rows == 128 && rb > 65535) return fail(MOE_ESHAPE, "rows %d above 65535 blocks of 128", rows);
  if ((uintptr_t)x % size) return fail(MOE_EALIGN, "x is misaligned");
  const size_t nx = span(rows, cols, ldx, size), nq = span(rows, cols, ldq, 1), ns = span(rb, cb, lds, 1);
  if (overlap(x, nx, q, nq) || overlap(x, nx, s, ns) || overlap(q, nq, s, ns))
    return fail(MOE_EINVAL, "x, q and s overlap");
  moe::Quant8P p{};
  p.x = x, p.bf16 = x_dtype == MOE_BF16, p.ldx = ldx, p.rows = rows, p.cols = cols;
  p.q = q, p.ldq = ldq, p.s = s, p.lds = lds;
  int n_sms = 0;
  if (int r = sm_count(&n_sms)) return r;
  const cudaError_t e = block_rows == 1 ? moe::launch_quant8_rows(p, n_sms, (cudaStream_t)stream)
                                        : moe::launch_quant8_blocks(p, (cudaStream_t)stream);
  if (e != cudaSuccess) return fail(MOE_ECUDA, "launch failed: %s", cudaGetErrorString(e));
  return MOE_OK;
}

int moe_mm8(const uint8_t *a, int64_t lda, const uint8_t *sa, int64_t lds, int t, const uint8_t *b, const uint8_t *sb,
            int n, int k, void *out, int out_dtype, int64_t ldo, const int32_t *offs, int n_groups, uint32_t flags,
            int *dev_status, moe_stream_t stream) {
  const int size = dtype_size(out_dtype);
  if (!size) return fail(MOE_EINVAL, "unknown out_dtype %d", out_dtype);
  if (flags & ~(uint32_t)MOE_TEST_WITHHOLD) return fail(MOE_EINVAL, "unknown flags 0x%x", flags);
  if (t < 0 || t > kMaxCount || n < 1 || k < 1) return fail(MOE_ESHAPE, "t %d, n %d, k %d", t, n, k);
  if (k % 16) return fail(MOE_ESHAPE, "k %d must be a multiple of 16", k);
  if (k > 1 << 24) return fail(MOE_ESHAPE, "k %d above 2^24", k);
  if (!offs != !n_groups || n_groups < 0 || n_groups > 1024)
    return fail(MOE_EINVAL, "offs and n_groups (1..1024) go together");
  const int64_t G = n_groups ? n_groups : 1, nb = ((int64_t)n + 127) / 128, nk = ((int64_t)k + 127) / 128;
  if (G * n > INT32_MAX - 256) return fail(MOE_ESHAPE, "n_groups x n exceeds the 2^31 rows a tensor-map coordinate reaches");
  if (nb * (((int64_t)t + 15) / 16 + G) > INT32_MAX) return fail(MOE_ESHAPE, "too many output tiles");
  if (!dev_status) return fail(MOE_EINVAL, "dev_status is NULL");
  if (int r = check_status(dev_status, {})) return r;
  if (t > 0) {
    if (!a || !sa || !b || !sb || !out) return fail(MOE_EINVAL, "a, sa, b, sb and out are required");
    if (lda < k || lds < nk || ldo < n) return fail(MOE_ESHAPE, "a row stride is below the row's length");
    if (((uintptr_t)a & 15u) || lda % 16 || ((uintptr_t)b & 15u))
      return fail(MOE_EALIGN, "a, its row stride and b must be 16-byte aligned");
    if (lda >= (int64_t)1 << 40) return fail(MOE_ESHAPE, "lda too large");
    if (((uintptr_t)sa & 3u) || lds % 4) return fail(MOE_EALIGN, "sa and its row stride must be 4-byte aligned");
    if ((uintptr_t)out % size || ((uintptr_t)offs & 3u)) return fail(MOE_EALIGN, "out or offs is misaligned");
    const size_t no = span(t, n, ldo, size);
    if (overlap(out, no, a, span(t, k, lda, 1)) || overlap(out, no, sa, span(t, nk, lds, 1)) ||
        overlap(out, no, b, (size_t)(G * n) * k) || overlap(out, no, sb, (size_t)(G * nb * nk)) ||
        (offs && overlap(out, no, offs, (size_t)(G + 1) * 4)))
      return fail(MOE_EINVAL, "out overlaps an input");
    if (int r = check_status(dev_status, {{out, no}, {a, span(t, k, lda, 1)}, {sa, span(t, nk, lds, 1)},
                                          {b, (size_t)(G * n) * k}, {sb, (size_t)(G * nb * nk)}, {offs, (size_t)(G + 1) * 4}}))
      return r;
  }
  cudaStream_t st = (cudaStream_t)stream;
  cudaError_t e;
  moe::Mm8P p;
  memset(&p, 0, sizeof p);
  p.a = a, p.sa = sa, p.b = b, p.sb = sb, p.lda = lda, p.lds = lds;
  p.t = t, p.n = n, p.k = k, p.nk = (int)nk, p.nb = (int)nb;
  p.G = n_groups, p.offs = offs;
  p.out = out, p.ldo = ldo;
  p.withhold = (flags & MOE_TEST_WITHHOLD) != 0;
  p.status = dev_status;
  p.timeout_ns = moe::timeout_ns();
  const int kind = out_dtype == MOE_F32 ? moe::kOutF32 : moe::kOutBf16;
  if (t > 0 && !offs && moe::mm8_small(t, n, k) && !p.withhold) {
    e = moe::launch_mm8_small(p, kind, st);
  } else {
    e = cudaSuccess;
    p.zero_status = 1;
    // a wait may give up no sooner than the status is zeroed
    if (p.timeout_ns < 1000000) p.timeout_ns = 1000000;
    if (t == 0) {
      e = cudaMemsetAsync(dev_status, 0, 4, st);
    } else {
      int n_sms = 0;
      if (int r = sm_count(&n_sms)) return r;
      e = moe::launch_mm8_tc(p, kind, n_sms, st);
    }
  }
  if (e != cudaSuccess) return fail(MOE_ECUDA, "launch failed: %s", cudaGetErrorString(e));
  return MOE_OK;
}

size_t moe_experts8_workspace(const moe_layer8 *L, int t, int top_k) {
  if (check_layer8(L, t, top_k) != MOE_OK) return 0;
  // few rows have buffers of their own, which may need more than many rows':
  // the most that t rows or fewer need
  size_t n = 256;
  for (int r = t; r >= 0; r = r > moe::kEx8SmallRows ? moe::kEx8SmallRows : r - 1)
    n = std::max(n, moe::ex8_sizes((int)L->hidden, (int)L->n_experts, (int)L->inter, r, top_k).total);
  return n;
}

int moe_experts8(const moe_layer8 *L, const void *x, int x_dtype, int t, const uint32_t *topk_idx,
                 const float *topk_w, int top_k, void *out, int out_dtype, void *work, size_t work_bytes,
                 int *dev_status, moe_stream_t stream) {
  if (int r = check_layer8(L, t, top_k)) return r;
  const int xs = dtype_size(x_dtype), os = dtype_size(out_dtype);
  if (!xs || !os) return fail(MOE_EINVAL, "unknown x_dtype %d / out_dtype %d", x_dtype, out_dtype);
  if (!L->gate_up || !L->gate_up_s || !L->down || !L->down_s)
    return fail(MOE_EINVAL, "a weight or scale pointer is NULL");
  if (((uintptr_t)L->gate_up | (uintptr_t)L->down) & 15u)
    return fail(MOE_EALIGN, "gate_up and down must be 16-byte aligned");
  if (!dev_status) return fail(MOE_EINVAL, "dev_status is NULL");
  if (int r = check_status(dev_status, {})) return r;
  const int H = (int)L->hidden, E = (int)L->n_experts, I = (int)L->inter;
  if ((int64_t)E * 2 * I > INT32_MAX || (int64_t)E * H > INT32_MAX)
    return fail(MOE_ESHAPE, "weight rows exceed the 2^31 rows a tensor-map coordinate reaches");
  cudaStream_t st = (cudaStream_t)stream;
  cudaError_t e = cudaSuccess;
  if (t == 0) {
    e = cudaMemsetAsync(dev_status, 0, 4, st);
    return e == cudaSuccess ? MOE_OK : fail(MOE_ECUDA, "memset failed: %s", cudaGetErrorString(e));
  }
  if (!x || !topk_idx || !topk_w || !out || !work)
    return fail(MOE_EINVAL, "x, topk_idx, topk_w, out and work are required");
  if (((uintptr_t)x | (uintptr_t)out) & 15u) return fail(MOE_EALIGN, "x and out must be 16-byte aligned");
  if (((uintptr_t)topk_idx | (uintptr_t)topk_w) & 3u) return fail(MOE_EALIGN, "topk_idx / topk_w misaligned");
  if ((uintptr_t)work & 255u) return fail(MOE_EALIGN, "work must be 256-byte aligned");
  const size_t no = (size_t)t * H * os, ni = (size_t)t * top_k * 4;
  if (overlap(x, (size_t)t * H * xs, out, no)) return fail(MOE_EINVAL, "out overlaps x");
  if (overlap(topk_idx, ni, out, no) || overlap(topk_w, ni, out, no))
    return fail(MOE_EINVAL, "out overlaps the ids or weights");
  const moe::Ex8Sizes z = moe::ex8_sizes(H, E, I, t, top_k);
  if (work_bytes < z.total) return fail(MOE_ENOSPACE, "work holds %zu bytes, %zu needed", work_bytes, z.total);
  if (overlap(work, z.total, x, (size_t)t * H * xs) || overlap(work, z.total, out, no) ||
      overlap(work, z.total, topk_idx, ni) || overlap(work, z.total, topk_w, ni))
    return fail(MOE_EINVAL, "work overlaps x, out, the ids or the weights");
  const size_t ne = (size_t)E * H * I;  // bytes of down; gate_up has twice as many
  const Buf parts[4] = {{L->gate_up, 2 * ne}, {L->gate_up_s, 2 * ne >> 14}, {L->down, ne}, {L->down_s, ne >> 14}};
  for (const Buf &w : parts)
    if (overlap(w.p, w.n, out, no) || overlap(w.p, w.n, work, z.total))
      return fail(MOE_EINVAL, "out or work overlaps the layer's weights or scales");
  if (int r = check_status(dev_status, {{x, (size_t)t * H * xs}, {topk_idx, ni}, {topk_w, ni}, {out, no}, {work, z.total},
                                        parts[0], parts[1], parts[2], parts[3]}))
    return r;
  moe::Ex8P p{};
  p.H = H, p.E = E, p.I = I, p.t = t, p.K = top_k;
  p.gu = L->gate_up, p.gus = L->gate_up_s, p.dn = L->down, p.dns = L->down_s;
  p.x = x, p.x_bf16 = x_dtype == MOE_BF16, p.out_bf16 = out_dtype == MOE_BF16;
  p.idx = topk_idx, p.w = topk_w, p.out = out, p.status = dev_status;
  p.ldi = (I / 128 + 3) / 4 * 4, p.ldh = (H / 128 + 3) / 4 * 4;
  uint8_t *at = static_cast<uint8_t *>(work);
  auto take = [&](size_t bytes) {
    uint8_t *r = at;
    at += bytes;
    return r;
  };
  int n_sms = 0;
  if (int r = sm_count(&n_sms)) return r;
  if (moe::ex8_small(H, I, t, top_k)) {
    p.h32 = (float *)take(z.h32);
    p.timeout_ns = moe::timeout_ns();
    if (p.timeout_ns < 1000000) p.timeout_ns = 1000000;  // as in moe_mm8
    e = moe::launch_ex8_small(p, n_sms, st);
    return e == cudaSuccess ? MOE_OK : fail(MOE_ECUDA, "launch failed: %s", cudaGetErrorString(e));
  }
  p.h8 = take(z.h8), p.h8s = take(z.h8s), p.x8 = take(z.x8), p.x8s = take(z.x8s);
  p.counts = (int *)take(z.counts), p.offs = (int *)take(z.offs), p.place = (int *)take(z.place);
  p.y = (float *)take(z.y);
  moe::Mm8P u, d;
  memset(&u, 0, sizeof u);
  u.a = p.x8, u.lda = H, u.sa = p.x8s, u.lds = p.ldh, u.b = p.gu, u.sb = p.gus;
  u.t = t * top_k, u.n = 2 * I, u.k = H, u.nk = H / 128, u.nb = 2 * I / 128;
  u.G = E, u.offs = p.offs;
  u.out = p.h8, u.ldo = I, u.hs = p.h8s, u.ldhs = p.ldi;
  u.status = dev_status, u.timeout_ns = moe::timeout_ns();
  d = u;
  d.a = p.h8, d.lda = I, d.sa = p.h8s, d.lds = p.ldi, d.b = p.dn, d.sb = p.dns;
  d.n = H, d.k = I, d.nk = I / 128, d.nb = H / 128;
  d.out = p.y, d.ldo = H, d.hs = nullptr;
  e = moe::launch_ex8_group(p, st);
  if (e == cudaSuccess) e = moe::launch_mm8_tc(u, moe::kOutSilu8, n_sms, st);
  if (e == cudaSuccess) e = moe::launch_mm8_tc(d, moe::kOutF32, n_sms, st);
  if (e == cudaSuccess) e = moe::launch_ex8_combine(p, n_sms, st);
  if (e != cudaSuccess) return fail(MOE_ECUDA, "launch failed: %s", cudaGetErrorString(e));
  return MOE_OK;
}

}  // extern "C"
