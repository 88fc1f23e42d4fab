"""Cases and plain forms of the operators around the experts' step: norms before and after a block with its gate,
residual scale and residual (norm, add_norm), matrix products with bias, activation, gate and residual in their epilogue
(mm16), and log probabilities of given tokens with entropy and top alternatives (logprobs).

Formats: bf16 or f32; norms also give e4m3 values (torch.float8_e4m3fn) with E8M0 scales (torch.float8_e8m0fnu, byte e
stands for 2^(e - 127)), one per 128 consecutive values of a row.
"""
import math

import torch

own = False

E4M3 = torch.float8_e4m3fn
E8M0 = torch.float8_e8m0fnu
BF16 = torch.bfloat16
F32 = torch.float32
F64 = torch.float64
TYPES = {"bf16": BF16, "f32": F32, "e4m3": E4M3}
SIZES = {"bf16": 2, "f32": 4, "e4m3": 1, "none": 0}


def listed():
    return [
        # one decoded token's norm before the router and the experts: launch latency
        dict(name="norm_token", op="norm", t=1, h=2048, x="f32", out="bf16", weight=True, pad=0),
        # the same for a prefill chunk, straight into the 8-bit form that the experts' first product takes
        dict(name="norm_quant", op="norm", t=4096, h=2048, x="bf16", out="e4m3", weight=True, pad=0),
        # the end of a block over a prefill chunk: the experts' output normalised, gated by row, added to a 32-bit residual
        # stream, and the next block's norm
        dict(name="add_norm_chunk", op="add_norm", t=4096, h=2048, y="bf16", res="f32", gate="row", sigmoid=True, post=True,
             scale=0.5, res_scale=1.0, out="bf16", weight=True, pad=0),
        # a large batch with a gate per channel and an odd width (rows that start on no 16 bytes)
        dict(name="add_norm_large", op="add_norm", t=30011, h=4090, y="bf16", res="bf16", gate="channel", sigmoid=False,
             post=False, scale=1.0, res_scale=0.7, out="bf16", weight=True, pad=0),
        # one token's router logits (512 experts): launch latency
        dict(name="mm_router_token", op="mm16", t=1, n=512, k=2048, gated=False, act="none", bias=False, residual="none",
             row_scale=False, out="f32", pad=0),
        # the shared expert's first product over a prefill chunk: silu(gate) * up
        dict(name="mm_shared_up", op="mm16", t=4096, n=768, k=2048, gated=True, act="silu", bias=False, residual="none",
             row_scale=False, out="bf16", pad=0),
        # odd sizes: a ragged batch through a small projection with everything in the epilogue
        dict(name="mm_odd", op="mm16", t=333, n=1001, k=2008, gated=False, act="gelu", bias=True, residual="bf16",
             row_scale=True, out="f32", pad=8),
        # four rows of a verify step through the vocabulary's product: the weights' bytes
        dict(name="mm_head", op="mm16", t=4, n=131072, k=2048, gated=False, act="none", bias=False, residual="none",
             row_scale=False, out="f32", pad=0),
        # a large prefill batch through a dense layer with bias, activation and residual
        dict(name="mm_large", op="mm16", t=8192, n=8192, k=2048, gated=False, act="gelu_tanh", bias=True, residual="bf16",
             row_scale=False, out="bf16", pad=0),
        # one decoded token: its probability, the entropy, 20 alternatives
        dict(name="logprobs_token", op="logprobs", t=1, v=131072, m=1, top=20, dtype="f32", scale=1.0, masked=0.0),
        # a batch of verify steps, four drafted tokens asked of each row, an odd vocabulary, some tokens switched off
        dict(name="logprobs_verify", op="logprobs", t=48, v=100003, m=4, top=8, dtype="f32", scale=1.25, masked=0.01),
        # scoring a prompt chunk: bf16 logits (many ties), the next token's probability, five alternatives
        dict(name="logprobs_chunk", op="logprobs", t=4096, v=131072, m=1, top=5, dtype="bf16", scale=1.0, masked=0.0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["norm", "add_norm", "mm16", "mm16", "logprobs"])
    if op == "norm":
        h = _log(rng, 16, 8192)
        return dict(op=op, t=_log(rng, 1, min(65536, 120_000_000 // h)), h=h, x=rng.choice(["bf16", "f32"]),
                    out=rng.choice(["bf16", "f32", "e4m3"]), weight=rng.random() < 0.8, pad=rng.choice([0, 0, 8, 13]))
    if op == "add_norm":
        h = _log(rng, 16, 8192)
        return dict(op=op, t=_log(rng, 1, min(65536, 60_000_000 // h)), h=h, y=rng.choice(["bf16", "f32"]),
                    res=rng.choice(["bf16", "f32"]), gate=rng.choice(["none", "row", "channel", "full"]),
                    sigmoid=rng.random() < 0.5, post=rng.random() < 0.5, scale=rng.choice([1.0, 0.25]),
                    res_scale=rng.choice([1.0, 0.9]), out=rng.choice(["bf16", "f32", "e4m3", "none"]),
                    weight=rng.random() < 0.8, pad=rng.choice([0, 0, 8, 13]))
    if op == "mm16":
        gated = rng.random() < 0.3
        k = 8 * _log(rng, 2, 1024)
        n = _log(rng, 8, min(131072, 250_000_000 // k) // (2 if gated else 1))
        t = _log(rng, 1, max(1, min(16384, 64_000_000 // n, int(1.2e11 / (n * k * (2 if gated else 1))))))
        return dict(op=op, t=t, n=n, k=k, gated=gated,
                    act=rng.choice(["silu", "gelu", "gelu_tanh", "relu", "sigmoid"] + ["none"] * (not gated) * 3), bias=rng.random() < 0.4, residual=rng.choice(["none", "bf16", "f32"]), row_scale=rng.random() < 0.3,
                    out=rng.choice(["bf16", "f32"]), pad=rng.choice([0, 8, 16]))
    v = _log(rng, 1000, 262144)
    return dict(op=op, t=_log(rng, 1, min(16384, 260_000_000 // v)), v=v, m=rng.randint(1, 8), top=rng.randint(1, 32),
                dtype=rng.choice(["bf16", "f32"]), scale=rng.choice([1.0, 0.7, 1.6]), masked=rng.choice([0.0, 0.05]))


# ---- inputs

def _rows(values, pad):
    """The same rows, `pad` values further apart than they are long."""
    if not pad:
        return values
    wide = torch.empty(values.shape[0], values.shape[1] + pad, dtype=values.dtype, device="cuda")
    wide[:, : values.shape[1]] = values
    return wide[:, : values.shape[1]]


def _stream(t, h, g):
    """A residual stream: rows of different sizes, and a few channels that are much larger than the others."""
    x = torch.randn(t, h, device="cuda", generator=g) * torch.exp(0.5 * torch.randn(t, 1, device="cuda", generator=g))
    return x * torch.where(torch.rand(h, device="cuda", generator=g) < 0.01, 20.0, 1.0)


def _empty_out(s, t, h):
    if s["out"] == "e4m3":
        s["scales"] = torch.empty(t, -(-h // 128), dtype=torch.uint8, device="cuda").view(E8M0)
    else:
        s["scales"] = None
    s["out_values"] = torch.empty(t, h, dtype=TYPES[s["out"]], device="cuda") if s["out"] != "none" else None


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case)
    if own:
        from quantized_routed_expert_fn_gb300 import moe
        s["moe"] = moe
    t = s["t"]
    if s["op"] in ("norm", "add_norm"):
        h = s["h"]
        s["w"] = 1 + 0.2 * torch.randn(h, device="cuda", generator=g) if s["weight"] else None
        _empty_out(s, t, h)
        if s["op"] == "norm":
            s["x_values"] = _rows(_stream(t, h, g).to(TYPES[s["x"]]), s["pad"])
            return s
        s["y_values"] = _rows(torch.randn(t, h, device="cuda", generator=g).to(TYPES[s["y"]]), s["pad"])
        s["residual"] = _rows(_stream(t, h, g).to(TYPES[s["res"]]), s["pad"])
        s["res_out"] = torch.empty(t, h, dtype=TYPES[s["res"]], device="cuda")
        s["w_post"] = 1 + 0.2 * torch.randn(h, device="cuda", generator=g) if s["post"] else None
        shape = {"none": None, "row": (t, 1), "channel": (1, h), "full": (t, h)}[s["gate"]]
        s["gate_values"] = None if shape is None else torch.randn(shape, device="cuda", generator=g)
        if s["gate"] == "full":
            s["gate_values"] = s["gate_values"].to(BF16)
    elif s["op"] == "mm16":
        n, k = s["n"], s["k"]
        rows = 2 * n if s["gated"] else n
        s["a"] = _rows(torch.randn(t, k, device="cuda", generator=g).to(BF16), s["pad"])
        s["b"] = (torch.randn(rows, k, device="cuda", generator=g) * k ** -0.5).to(BF16)
        s["bias_values"] = 0.1 * torch.randn(rows, device="cuda", generator=g) if s["bias"] else None
        s["residual_values"] = None
        if s["residual"] != "none":
            s["residual_values"] = _rows(torch.randn(t, n, device="cuda", generator=g).to(TYPES[s["residual"]]), s["pad"])
        s["row_scale_values"] = torch.rand(t, device="cuda", generator=g) if s["row_scale"] else None
        s["out_values"] = torch.empty(t, n, dtype=TYPES[s["out"]], device="cuda")
        if own:
            s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    else:
        v = s["v"]
        # rows between flat and peaked
        x = torch.randn(t, v, device="cuda", generator=g) * (1.5 + 2 * torch.rand(t, 1, device="cuda", generator=g))
        if s["masked"]:
            x.masked_fill_(torch.rand(v, device="cuda", generator=g) < s["masked"], -math.inf)
        s["logits"] = x.to(TYPES[s["dtype"]])
        # half of the given tokens are likely ones
        likely = (x + torch.randn(t, v, device="cuda", generator=g)).argmax(1, keepdim=True)
        other = torch.randint(0, v, (t, s["m"]), device="cuda", generator=g)
        s["tokens"] = torch.where(torch.rand(t, s["m"], device="cuda", generator=g) < 0.5, likely, other).to(torch.int32)
        s["logp"] = torch.empty(t, s["m"], device="cuda")
        s["entropy"] = torch.empty(t, device="cuda")
        s["top_idx"] = torch.empty(t, s["top"], dtype=torch.int32, device="cuda")
        s["top_logp"] = torch.empty(t, s["top"], device="cuda")
    return s


# ---- plain forms

def _quantised(x):
    """e4m3 values and E8M0 scales of x [t][h], a scale per 128 of a row: the least power of two 2^e with |x| <= 448 * 2^e."""
    t, h = x.shape
    blocks = -(-h // 128)
    p = torch.zeros(t, blocks * 128, device=x.device)
    p[:, :h] = x
    p = p.view(t, blocks, 128)
    m, e = torch.frexp(p.abs().amax(2))  # m 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
    e = torch.where(m > 0, e - 9 + (m > 0.875), 0).to(torch.int32)
    q = p * ((127 - e) << 23).view(F32)[:, :, None]
    return q.view(t, -1)[:, :h].to(E4M3), (e + 127).to(torch.uint8).view(E8M0)


def _normed(s, x, w):
    y = x / torch.sqrt((x * x).mean(1, keepdim=True) + 1e-6)
    y = y * w if w is not None else y
    return _quantised(y) if s["out"] == "e4m3" else y.to(TYPES[s["out"]])


def _add_norm_plain(s):
    v = s["y_values"].float()
    if s["post"]:
        v = v / torch.sqrt((v * v).mean(1, keepdim=True) + 1e-6) * s["w_post"]
    if s["gate_values"] is not None:
        g = s["gate_values"].float()
        v = v * (1 / (1 + torch.exp(-g)) if s["sigmoid"] else g)
    r = s["res_scale"] * s["residual"].float() + s["scale"] * v
    out = r.to(TYPES[s["res"]])
    return (out, _normed(s, r, s["w"])) if s["out"] != "none" else out


def _act(name, z):
    if name == "silu":
        return z / (1 + torch.exp(-z))
    if name == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if name == "relu":
        return z.clamp(min=0)
    return 1 / (1 + torch.exp(-z)) if name == "sigmoid" else z


def _mm16_plain(s):
    z = s["a"].float() @ s["b"].float().T
    if s["bias_values"] is not None:
        z = z + s["bias_values"]
    n = s["n"]
    h = _act(s["act"], z[:, :n]) * z[:, n:] if s["gated"] else _act(s["act"], z)
    if s["row_scale_values"] is not None:
        h = h * s["row_scale_values"][:, None]
    if s["residual_values"] is not None:
        h = h + s["residual_values"].float()
    return h.to(TYPES[s["out"]])


def _logprobs_plain(s):
    # 64 bits: sums over the vocabulary; the order is the logits' own, ties to the lowest id
    x, v = s["logits"], s["v"]
    bits = x.float().view(torch.int32).long()
    bits = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits)  # as the values order; -0 and 0 are one
    idx = (v - 1 - (bits * 2 ** 20 + (v - 1 - torch.arange(v, device=x.device))).topk(s["top"], dim=1).values % 2 ** 20)
    x = x.double()
    d = s["scale"] * (x - x.amax(1, keepdim=True))
    e = torch.exp(d)
    z = e.sum(1, keepdim=True)
    entropy = torch.log(z) - torch.where(e > 0, e * d, 0.0).sum(1, keepdim=True) / z
    logp = d - torch.log(z)
    return (logp.gather(1, s["tokens"].long()).float(), entropy[:, 0].float(), idx.to(torch.int32),
            logp.gather(1, idx).float())


def run(s):
    op = s["op"]
    if not own:
        if op == "norm":
            return _normed(s, s["x_values"].float(), s["w"])
        return _add_norm_plain(s) if op == "add_norm" else (_mm16_plain(s) if op == "mm16" else _logprobs_plain(s))
    moe = s["moe"]
    if op == "mm16":
        moe.mm16(s["a"], s["b"], s["out_values"], s["status"], bias=s["bias_values"], act=s["act"], gated=s["gated"],
                 row_scale=s["row_scale_values"], residual=s["residual_values"])
        return s["out_values"]
    if op == "logprobs":
        moe.logprobs(s["logits"], tokens=s["tokens"], logp=s["logp"], entropy=s["entropy"], top_idx=s["top_idx"],
                     top_logp=s["top_logp"], scale=s["scale"])
        return s["logp"], s["entropy"], s["top_idx"], s["top_logp"]
    if op == "norm":
        moe.norm(s["x_values"], s["out_values"], w=s["w"], scales=s["scales"])
    else:
        moe.add_norm(s["y_values"], s["residual"], s["res_out"], post=s["post"], w_post=s["w_post"], gate=s["gate_values"],
                     gate_sigmoid=s["sigmoid"], scale=s["scale"], res_scale=s["res_scale"], out=s["out_values"], w=s["w"],
                     scales=s["scales"])
    out = (s["out_values"], s["scales"]) if s["out"] == "e4m3" else s["out_values"]
    if op == "norm":
        return out
    return (s["res_out"], out) if s["out"] != "none" else s["res_out"]


# ---- the same from the definitions, in 64 bits

def _exact_norm(x, w):
    y = x * (math.sqrt(x.shape[1]) / torch.sqrt(torch.linalg.vector_norm(x, dim=1) ** 2 + x.shape[1] * 1e-6))[:, None]
    return y * w.double() if w is not None else y


def _exact_e4m3(x):
    """The values after rounding, in units of their block's scale, and the scales."""
    q, scales = torch.empty_like(x), []
    for at in range(0, x.shape[1], 128):
        p = x[:, at:at + 128]
        a = p.abs().amax(1)
        e = torch.floor(torch.log2(torch.clamp(a, min=1e-300) / 448))
        e = torch.where(a > 0, torch.where(a <= 448 * torch.exp2(e), e, e + 1), torch.zeros_like(e))
        u = p * torch.exp2(-e)[:, None]
        step = torch.exp2(torch.clamp(torch.floor(torch.log2(torch.clamp(u.abs(), min=1e-300))), min=-6) - 3)
        q[:, at:at + 128] = torch.round(u / step) * step
        scales.append(torch.exp2(e))
    return q, torch.stack(scales, 1)


def _exact_act(name, z):
    if name == "silu":
        return z * torch.special.expit(z)
    if name == "gelu":
        return z * torch.special.ndtr(z)
    if name == "gelu_tanh":
        return z * torch.special.expit(math.sqrt(8 / math.pi) * (z + 0.044715 * z ** 3))
    if name == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    return torch.special.expit(z) if name == "sigmoid" else z


def _exact_logprobs(s):
    parts = []
    for x, tokens in zip(torch.split(s["logits"], 256), torch.split(s["tokens"], 256)):
        order = torch.sort(x.float(), dim=1, descending=True, stable=True).indices[:, : s["top"]]
        logp = torch.log_softmax(s["scale"] * x.double(), dim=1)
        parts.append((logp.gather(1, tokens.long()), -torch.special.xlogy(torch.exp(logp), torch.exp(logp)).sum(1),
                      order.to(torch.int32), logp.gather(1, order)))
    return tuple(torch.cat(p) for p in zip(*parts))


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "logprobs":
        return _exact_logprobs(s)
    if s["op"] == "mm16":
        z = torch.matmul(s["a"].double(), s["b"].double().transpose(0, 1))
        if s["bias"]:
            z += s["bias_values"].double()
        up = z[:, s["n"]:]
        z = _exact_act(s["act"], z[:, : s["n"]])
        z = z * up if s["gated"] else z
        z = z * s["row_scale_values"].double()[:, None] if s["row_scale"] else z
        return z + s["residual_values"].double() if s["residual"] != "none" else z
    if s["op"] == "norm":
        y = _exact_norm(s["x_values"].double(), s["w"])
        return _exact_e4m3(y) if s["out"] == "e4m3" else y
    v = s["y_values"].double()
    v = _exact_norm(v, s["w_post"]) if s["post"] else v
    if s["gate"] != "none":
        g = s["gate_values"].double()
        v = v * (torch.special.expit(g) if s["sigmoid"] else g)
    r = torch.add(s["residual"].double() * s["res_scale"], v, alpha=s["scale"])
    if s["out"] == "none":
        return r
    y = _exact_norm(r, s["w"])
    return r, _exact_e4m3(y) if s["out"] == "e4m3" else y


def work(case):
    c, t = case, case["t"]
    if c["op"] == "norm":
        n = t * c["h"]
        return {"bytes": n * (SIZES[c["x"]] + SIZES[c["out"]]) + c["h"] * 4 * c["weight"]
                + (t * -(-c["h"] // 128) if c["out"] == "e4m3" else 0), "flops": 4 * n}
    if c["op"] == "add_norm":
        h = c["h"]
        n = t * h
        return {"bytes": n * (SIZES[c["y"]] + 2 * SIZES[c["res"]] + SIZES[c["out"]]) + h * 4 * (c["weight"] + c["post"])
                + {"none": 0, "row": 4 * t, "channel": 4 * h, "full": 2 * n}[c["gate"]]
                + (t * -(-h // 128) if c["out"] == "e4m3" else 0), "flops": 10 * n}
    if c["op"] == "mm16":
        rows = c["n"] * (2 if c["gated"] else 1)
        return {"bytes": (t + rows) * c["k"] * 2 + t * c["n"] * (SIZES[c["out"]] + SIZES[c["residual"]])
                + rows * 4 * c["bias"] + t * 4 * c["row_scale"], "flops": 2 * t * rows * c["k"]}
    return {"bytes": t * (c["v"] * SIZES[c["dtype"]] + c["m"] * 8 + c["top"] * 8 + 4), "flops": 6 * t * c["v"]}
