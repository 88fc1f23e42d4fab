// api_block.cu -- C ABI of the operators around the experts' step (norms,
// products with an epilogue, log probabilities): argument checks and launches.
#include <cmath>
#include <cstring>
#include <initializer_list>

#include "api.cuh"
#include "block.cuh"
#include "moe_api.h"

namespace {

using moe::fail;
using moe::overlap;

constexpr int kMaxCount = 1 << 30;

int float_size(int d) { return d == MOE_F32 ? 4 : (d == MOE_BF16 ? 2 : 0); }
int out_size(int d) { return d == MOE_E4M3 ? 1 : float_size(d); }

int sm_count(int *n) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return fail(MOE_ECUDA, "device query failed");
  return MOE_OK;
}

// A matrix argument: rows of cols values of `size` bytes, ld values apart.
struct Mat {
  const void *p;
  int64_t rows, cols, ld;
  int size;
  size_t bytes() const { return !p || rows < 1 ? 0 : ((size_t)(rows - 1) * ld + cols) * size; }
};

int check_mat(const Mat &m, const char *name) {
  if (!m.p) return fail(MOE_EINVAL, "%s is NULL", name);
  if (m.ld < m.cols) return fail(MOE_ESHAPE, "%s: row stride %lld below the row's length", name, (long long)m.ld);
  if (m.ld >= (int64_t)1 << 40) return fail(MOE_ESHAPE, "%s: row stride too large", name);
  if ((uintptr_t)m.p % m.size) return fail(MOE_EALIGN, "%s is misaligned", name);
  return MOE_OK;
}

// Whether `out` may stand where `in` does: apart, or the same matrix in the
// same type (a thread reads a value before it writes the one in its place).
bool apart_or_same(const Mat &out, const Mat &in) {
  if (!overlap(out.p, out.bytes(), in.p, in.bytes())) return true;
  return out.p == in.p && out.size == in.size && (out.ld == in.ld || out.rows == 1);
}
bool apart(const Mat &out, const Mat &in) { return !overlap(out.p, out.bytes(), in.p, in.bytes()); }

// Beside an eps below the normal numbers squares would count that are cut off
// there; above 1e37 the mean and eps may pass the 32-bit range together.
int check_eps(float eps) {
  if (!(eps >= 0x1p-126f) || !(eps <= 1e37f)) return fail(MOE_EINVAL, "eps outside 2^-126..1e37");
  return MOE_OK;
}

// A norm's output and, in e4m3, its scales.
int check_norm_out(const Mat &out, int dtype, const Mat &s) {
  if (int r = check_mat(out, "out")) return r;
  if (dtype != MOE_E4M3) return s.p ? fail(MOE_EINVAL, "scales go with an e4m3 output") : MOE_OK;
  if (int r = check_mat(s, "scales")) return r;
  return apart(out, s) ? MOE_OK : fail(MOE_EINVAL, "out and scales overlap");
}

int norm_out_kind(int dtype) {
  return dtype == MOE_F32 ? moe::kNormOutF32 : (dtype == MOE_BF16 ? moe::kNormOutBf16 : moe::kNormOutE4m3);
}

int launch(const moe::NormP &p, moe_stream_t stream) {
  int n_sms = 0;
  if (int r = sm_count(&n_sms)) return r;
  const cudaError_t e = moe::launch_norm(p, n_sms, (cudaStream_t)stream);
  return e == cudaSuccess ? MOE_OK : fail(MOE_ECUDA, "launch failed: %s", cudaGetErrorString(e));
}

int check_norm_size(int t, int h) {
  if (t < 0 || t > kMaxCount) return fail(MOE_ESHAPE, "t %d outside 0..2^30", t);
  if (h < 1 || h > moe::kNormMaxCols) return fail(MOE_ESHAPE, "h %d outside 1..%d", h, moe::kNormMaxCols);
  return MOE_OK;
}

}  // namespace

extern "C" {

int moe_norm(const void *x, int x_dtype, int64_t ldx, const float *w, float eps, int t, int h, void *out, int out_dtype,
             int64_t ldo, uint8_t *scales, int64_t lds, moe_stream_t stream) {
  const int xs = float_size(x_dtype), os = out_size(out_dtype);
  if (!xs || !os) return fail(MOE_EINVAL, "unknown x_dtype %d / out_dtype %d", x_dtype, out_dtype);
  if (int r = check_norm_size(t, h)) return r;
  if (int r = check_eps(eps)) return r;
  if (t == 0) return MOE_OK;
  const Mat mx{x, t, h, ldx, xs}, mo{out, t, h, ldo, os}, ms{scales, t, (h + 127) / 128, lds, 1}, mw{w, 1, h, h, 4};
  if (int r = check_mat(mx, "x")) return r;
  if (int r = check_norm_out(mo, out_dtype, ms)) return r;
  if ((uintptr_t)w & 3u) return fail(MOE_EALIGN, "w is misaligned");
  if (!apart_or_same(mo, mx) || !apart(mo, mw) || !apart(ms, mx) || !apart(ms, mw))
    return fail(MOE_EINVAL, "out or scales overlap the inputs (out may be x itself, in its type)");
  moe::NormP p{};
  p.t = t, p.h = h, p.eps = eps, p.inv_h = 1.f / (float)h;
  p.y = x, p.ldy = ldx, p.y_bf16 = x_dtype == MOE_BF16;
  p.out_kind = norm_out_kind(out_dtype);
  p.w = w, p.out = out, p.ldo = ldo, p.s = scales, p.lds = lds;
  return launch(p, stream);
}

int moe_add_norm(const moe_add_norm_cfg *c, const void *y, int y_dtype, int64_t ldy, const void *residual, int res_dtype,
                 int64_t ldr, void *res_out, int res_out_dtype, int64_t ldro, int t, int h, void *out, int out_dtype,
                 int64_t ldo, uint8_t *scales, int64_t lds, moe_stream_t stream) {
  if (!c) return fail(MOE_EINVAL, "cfg is NULL");
  const int ys = float_size(y_dtype), rs = float_size(res_dtype), ros = float_size(res_out_dtype), os = out_size(out_dtype);
  if (!ys || !rs || !ros || !os)
    return fail(MOE_EINVAL, "unknown y_dtype %d / res_dtype %d / res_out_dtype %d / out_dtype %d", y_dtype, res_dtype,
                res_out_dtype, out_dtype);
  if (c->flags & ~(uint32_t)(MOE_NORM_POST | MOE_NORM_GATE_SIGMOID)) return fail(MOE_EINVAL, "unknown flags 0x%x", c->flags);
  if (!std::isfinite(c->scale) || !std::isfinite(c->res_scale)) return fail(MOE_EINVAL, "a scale is not finite");
  if (int r = check_norm_size(t, h)) return r;
  if (int r = check_eps(c->eps)) return r;
  const bool post = (c->flags & MOE_NORM_POST) != 0;
  if (c->w_post && !post) return fail(MOE_EINVAL, "w_post goes with MOE_NORM_POST");
  int gs = 2;
  if (c->gate) {
    gs = float_size(c->gate_dtype);
    if (!gs) return fail(MOE_EINVAL, "unknown gate_dtype %d", c->gate_dtype);
    if (c->gate_cols != 1 && c->gate_cols != h) return fail(MOE_ESHAPE, "gate_cols %d is neither 1 nor h", c->gate_cols);
  }
  if (t == 0) return MOE_OK;
  const Mat my{y, t, h, ldy, ys}, mr{residual, t, h, ldr, rs}, mro{res_out, t, h, ldro, ros}, mo{out, t, h, ldo, os};
  const Mat ms{scales, t, (h + 127) / 128, lds, 1}, mw{c->w, 1, h, h, 4}, mp{c->w_post, 1, h, h, 4};
  const Mat mg{c->gate, c->ldg ? t : 1, c->gate_cols, c->ldg ? c->ldg : c->gate_cols, gs};
  if (int r = check_mat(my, "y")) return r;
  if (int r = check_mat(mr, "residual")) return r;
  if (int r = check_mat(mro, "res_out")) return r;
  if (c->gate)
    if (int r = check_mat(mg, "gate")) return r;
  if (((uintptr_t)c->w | (uintptr_t)c->w_post) & 3u) return fail(MOE_EALIGN, "w or w_post is misaligned");
  if (!apart_or_same(mro, my) || !apart_or_same(mro, mr) || !apart(mro, mg) || !apart(mro, mw) || !apart(mro, mp))
    return fail(MOE_EINVAL, "res_out overlaps an input (it may be y or residual itself, in its type)");
  if (out) {
    if (int r = check_norm_out(mo, out_dtype, ms)) return r;
    for (const Mat *o : {&mo, &ms})
      if (!apart(*o, mro) || !apart(*o, mg) || !apart(*o, mw) || !apart(*o, mp) || !apart(*o, mr) ||
          !(o == &mo ? apart_or_same(mo, my) : apart(ms, my)))
        return fail(MOE_EINVAL, "out or scales overlap another buffer (out may be y itself, in its type)");
  } else if (scales) {
    return fail(MOE_EINVAL, "scales without out");
  }
  moe::NormP p{};
  p.t = t, p.h = h, p.eps = c->eps, p.inv_h = 1.f / (float)h;
  p.y = y, p.ldy = ldy, p.y_bf16 = y_dtype == MOE_BF16;
  p.post = post, p.scale = c->scale, p.res_scale = c->res_scale, p.wp = c->w_post;
  p.gate = c->gate, p.ldg = c->ldg, p.gate_bf16 = c->gate_dtype == MOE_BF16, p.gate_cols = c->gate_cols;
  p.gate_sigmoid = (c->flags & MOE_NORM_GATE_SIGMOID) != 0;
  p.res = residual, p.ldr = ldr, p.res_bf16 = res_dtype == MOE_BF16;
  p.ro = res_out, p.ldro = ldro, p.ro_bf16 = res_out_dtype == MOE_BF16;
  p.out_kind = out ? norm_out_kind(out_dtype) : moe::kNormOutNone;
  p.w = c->w, p.out = out, p.ldo = ldo, p.s = scales, p.lds = lds;
  return launch(p, stream);
}

int moe_logprobs(const void *logits, int logit_dtype, int64_t ld, int t, int v, float scale, const int32_t *tokens, int m,
                 float *logp, float *entropy, uint32_t *top_idx, float *top_logp, int top_k, moe_stream_t stream) {
  const int size = float_size(logit_dtype);
  if (!size) return fail(MOE_EINVAL, "unknown logit_dtype %d", logit_dtype);
  if (t < 0 || t > kMaxCount / 8) return fail(MOE_ESHAPE, "t %d outside 0..2^27", t);
  if (v < 1 || v > 1 << 24) return fail(MOE_ESHAPE, "v %d outside 1..2^24", v);
  if (!(scale > 0.f) || !(scale <= 1e6f)) return fail(MOE_EINVAL, "scale must be positive, 1e6 at most");
  if (m < 0 || m > 1024) return fail(MOE_ESHAPE, "m %d outside 0..1024", m);
  if (top_k < 0 || top_k > 32 || top_k > v) return fail(MOE_ESHAPE, "top_k %d outside 0..min(32, v)", top_k);
  if (t == 0) return MOE_OK;
  if (m == 0 && top_k == 0 && !entropy) return fail(MOE_EINVAL, "nothing is asked for");
  if ((m > 0) != (tokens != nullptr) || (m > 0) != (logp != nullptr))
    return fail(MOE_EINVAL, "tokens, logp and m go together");
  if ((top_k > 0) != (top_idx != nullptr) || (top_k > 0) != (top_logp != nullptr))
    return fail(MOE_EINVAL, "top_idx, top_logp and top_k go together");
  const Mat ml{logits, t, v, ld, size}, mt{tokens, t, m, m, 4}, mk{top_idx, t, top_k, top_k, 4};
  const Mat outs[4] = {{logp, t, m, m, 4}, {entropy, t, 1, 1, 4}, mk, {top_logp, t, top_k, top_k, 4}};
  if (int r = check_mat(ml, "logits")) return r;
  if (((uintptr_t)tokens | (uintptr_t)logp | (uintptr_t)entropy | (uintptr_t)top_idx | (uintptr_t)top_logp) & 3u)
    return fail(MOE_EALIGN, "misaligned pointer");
  for (int i = 0; i < 4; i++) {
    if (!apart(outs[i], ml) || !apart(outs[i], mt)) return fail(MOE_EINVAL, "an output overlaps the logits or the tokens");
    for (int j = 0; j < i; j++)
      if (!apart(outs[i], outs[j])) return fail(MOE_EINVAL, "two outputs overlap");
  }
  moe::LogprobsP p{};
  p.x = logits, p.ld = ld, p.bf16 = logit_dtype == MOE_BF16, p.t = t, p.v = v, p.scale = scale;
  p.tokens = tokens, p.m = m, p.logp = logp, p.entropy = entropy;
  p.top_idx = top_idx, p.top_logp = top_logp, p.k = top_k;
  int n_sms = 0;
  if (int r = sm_count(&n_sms)) return r;
  const cudaError_t e = moe::launch_logprobs(p, n_sms, (cudaStream_t)stream);
  return e == cudaSuccess ? MOE_OK : fail(MOE_ECUDA, "launch failed: %s", cudaGetErrorString(e));
}

int moe_mm16(const uint16_t *a, int64_t lda, int t, const uint16_t *b, int64_t ldb, int n, int k, const moe_epilogue *epi,
             void *out, int out_dtype, int64_t ldo, uint32_t flags, int *dev_status, moe_stream_t stream) {
  static const moe_epilogue none = {};
  const moe_epilogue &E = epi ? *epi : none;
  const int os = float_size(out_dtype);
  if (!os) return fail(MOE_EINVAL, "unknown out_dtype %d", out_dtype);
  if (flags & ~(uint32_t)(MOE_MM16_GATED | MOE_TEST_WITHHOLD)) return fail(MOE_EINVAL, "unknown flags 0x%x", flags);
  if (E.act > MOE_ACT_SIGMOID) return fail(MOE_EINVAL, "unknown act %u", E.act);
  const bool gated = (flags & MOE_MM16_GATED) != 0;
  if (t < 0 || t > kMaxCount || n < 1 || k < 1 || k > 1 << 24) return fail(MOE_ESHAPE, "t %d, n %d, k %d", t, n, k);
  const int64_t wrows = gated ? 2 * (int64_t)n : n;
  if (wrows > INT32_MAX - 256) return fail(MOE_ESHAPE, "more weight rows than a tensor-map coordinate reaches");
  if (((int64_t)t / 16 + 1) * (n / 64 + 2) > INT32_MAX) return fail(MOE_ESHAPE, "too many output tiles");
  int rs = 2;
  if (E.residual) {
    rs = float_size(E.res_dtype);
    if (!rs) return fail(MOE_EINVAL, "unknown res_dtype %d", E.res_dtype);
  }
  if (!dev_status) return fail(MOE_EINVAL, "dev_status is NULL");
  if ((uintptr_t)dev_status & 3u) return fail(MOE_EALIGN, "dev_status is misaligned");
  cudaStream_t st = (cudaStream_t)stream;
  if (t == 0) {
    const cudaError_t e = cudaMemsetAsync(dev_status, 0, 4, st);
    return e == cudaSuccess ? MOE_OK : fail(MOE_ECUDA, "memset failed: %s", cudaGetErrorString(e));
  }
  const Mat ma{a, t, k, lda, 2}, mb{b, wrows, k, ldb, 2}, mo{out, t, n, ldo, os}, mr{E.residual, t, n, E.ldr, rs};
  const Mat mbias{E.bias, 1, wrows, wrows, 4}, mrs{E.row_scale, 1, t, t, 4}, mst{dev_status, 1, 1, 1, 4};
  if (int r = check_mat(ma, "a")) return r;
  if (int r = check_mat(mb, "b")) return r;
  if (int r = check_mat(mo, "out")) return r;
  if (E.residual)
    if (int r = check_mat(mr, "residual")) return r;
  if ((((uintptr_t)a | (uintptr_t)b) & 15u) || lda % 8 || ldb % 8)
    return fail(MOE_EALIGN, "a, b and their rows must start on 16 bytes");
  if (((uintptr_t)E.bias | (uintptr_t)E.row_scale) & 3u) return fail(MOE_EALIGN, "bias or row_scale is misaligned");
  if (!apart(mo, ma) || !apart(mo, mb) || !apart(mo, mbias) || !apart(mo, mrs)) return fail(MOE_EINVAL, "out overlaps an input");
  if (!apart_or_same(mo, mr)) return fail(MOE_EINVAL, "out overlaps the residual (it may be the residual itself, in its type)");
  for (const Mat *m : {&ma, &mb, &mo, &mr, &mbias, &mrs})
    if (!apart(mst, *m)) return fail(MOE_EINVAL, "dev_status lies in another buffer");
  moe::Mm16P p;
  memset(&p, 0, sizeof p);
  p.a = a, p.lda = lda, p.b = b, p.ldb = ldb, p.t = t, p.n = n, p.k = k, p.gated = gated, p.act = (int)E.act;
  p.bias = E.bias, p.row_scale = E.row_scale, p.res = E.residual, p.ldr = E.ldr, p.res_bf16 = E.res_dtype == MOE_BF16;
  p.out = out, p.ldo = ldo, p.out_bf16 = out_dtype == MOE_BF16;
  auto whole = [](const Mat &m) { return !m.p || (((uintptr_t)m.p | (uintptr_t)(m.ld * m.size)) & (4u * m.size - 1)) == 0; };
  p.wide = whole(mo) && whole(mr);
  auto runs = [](const Mat &m) { return !m.p || (((uintptr_t)m.p | (uintptr_t)(m.ld * m.size)) & 31u) == 0; };
  p.wide8 = runs(mo) && runs(mr);
  p.withhold = (flags & MOE_TEST_WITHHOLD) != 0;
  p.status = dev_status;
  p.timeout_ns = moe::timeout_ns();
  if (p.timeout_ns < 1000000) p.timeout_ns = 1000000;  // a wait gives up no sooner than the status is zeroed
  int n_sms = 0;
  if (int r = sm_count(&n_sms)) return r;
  const cudaError_t e = moe::mm16_few(p, n_sms) && !p.withhold ? moe::launch_mm16_few(p, n_sms, st) : moe::launch_mm16_tc(p, n_sms, st);
  return e == cudaSuccess ? MOE_OK : fail(MOE_ECUDA, "launch failed: %s", cudaGetErrorString(e));
}

}  // extern "C"
