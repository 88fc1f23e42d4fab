"""Cases and plain forms of the 8-bit expert operators: routing (gate), quantisation to e4m3 with a power-of-two
scale per block of 128 (quant8), the block-scaled matrix product, dense and grouped by expert (mm8), and the routed
experts as one step (experts8).

Formats: e4m3 values (torch.float8_e4m3fn) with E8M0 scales (torch.float8_e8m0fnu, byte e stands for 2^(e - 127)): one
per 128 consecutive k of a row for activations, one per 128 x 128 block for weights.
"""
import math

import numpy as np
import torch

own = False

E4M3 = torch.float8_e4m3fn
E8M0 = torch.float8_e8m0fnu
BF16 = torch.bfloat16
F32 = torch.float32


def listed():
    return [
        # one decoded token of a 128-expert layer, top 8, weights renormalised: launch latency
        dict(name="gate_token", op="gate", t=1, experts=128, top_k=8, score="softmax", bias=False, groups=1, top_groups=1,
             group_top=1, renorm=True, scale=1.0, dtype="f32", masked=0.0),
        # a prefill chunk of a 512-expert layer, top 10, bf16 logits straight from a bf16 router product (many ties)
        dict(name="gate_chunk", op="gate", t=4096, experts=512, top_k=10, score="softmax", bias=False, groups=1,
             top_groups=1, group_top=1, renorm=True, scale=1.0, dtype="bf16", masked=0.0),
        # a large padded batch with sigmoid scores, a balance bias and 8 expert groups of which 4 stay
        dict(name="gate_groups", op="gate", t=65535, experts=256, top_k=8, score="sigmoid", bias=True, groups=8,
             top_groups=4, group_top=2, renorm=True, scale=2.5, dtype="f32", masked=0.02),
        # the activations of a prefill chunk, quantised by rows before a product
        dict(name="quant_rows", op="quant8", rows=4096, cols=2048, block_rows=1, dtype="bf16"),
        # a layer's projection weights, quantised once at load in 128 x 128 blocks; ragged edges
        dict(name="quant_blocks", op="quant8", rows=16300, cols=4112, block_rows=128, dtype="f32"),
        # one token through a square projection: the weights are streamed once
        dict(name="mm_token", op="mm8", t=1, n=2048, k=2048, groups=0, skew=0.0, pad=0, out="bf16"),
        # an odd batch and ragged sizes, 32-bit output
        dict(name="mm_odd", op="mm8", t=333, n=1000, k=2000, groups=0, skew=0.0, pad=0, out="f32"),
        # a large prefill chunk through a wide projection
        dict(name="mm_chunk", op="mm8", t=8192, n=8192, k=2048, groups=0, skew=0.0, pad=0, out="bf16"),
        # the rows of 4096 tokens x top 8 grouped by 128 experts of uneven popularity, with unused rows behind the last
        dict(name="mm_grouped", op="mm8", t=32768, n=1536, k=2048, groups=128, skew=1.1, pad=100, out="bf16"),
        # one decoded token through its 8 experts
        dict(name="experts_token", op="experts8", t=1, hidden=2048, experts=128, top_k=8, inter=768, skew=0.0, x="f32"),
        # a verify batch of 4 rows
        dict(name="experts_verify", op="experts8", t=4, hidden=2048, experts=512, top_k=10, inter=512, skew=0.0, x="f32"),
        # a prefill chunk with Zipf(1.1) expert popularity
        dict(name="experts_chunk", op="experts8", t=4096, hidden=2048, experts=512, top_k=10, inter=512, skew=1.1, x="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gate", "quant8", "mm8", "mm8", "experts8", "experts8"])
    if op == "gate":
        groups = rng.choice([1, 1, 2, 4, 8])
        experts = groups * _log(rng, 8, 1024 // groups if groups > 1 else 1000)
        top_groups = rng.randint(1, groups)
        top_k = rng.randint(1, min(16, top_groups * (experts // groups)))
        t = _log(rng, 1, max(1, min(70000, 16000000 // experts)))
        score = rng.choice(["softmax", "sigmoid"])
        return dict(op=op, t=t, experts=experts, top_k=top_k, score=score, bias=rng.random() < 0.5, groups=groups,
                    top_groups=top_groups, group_top=rng.choice([1, 2]), renorm=rng.random() < 0.6,
                    scale=round(rng.uniform(0.5, 3.0), 3), dtype=rng.choice(["f32", "bf16"]), masked=rng.choice([0.0, 0.1]))
    if op == "quant8":
        cols = 16 * _log(rng, 8, 512)
        rows = _log(rng, 1, max(2, 67000000 // cols))
        return dict(op=op, rows=rows, cols=cols, block_rows=rng.choice([1, 128]), dtype=rng.choice(["f32", "bf16"]))
    if op == "mm8":
        groups = rng.choice([0, 0, _log(rng, 2, 256)])
        k = 16 * _log(rng, 8, 512)
        n = _log(rng, 16, 8192 if not groups else 2048)
        t = _log(rng, 1, max(2, min(32768, int(1.0e11 / (n * k)))))
        return dict(op=op, t=t, n=n, k=k, groups=groups, skew=rng.choice([0.0, 1.1]) if groups else 0.0,
                    pad=rng.randint(0, min(64, t - 1)) if groups else 0, out=rng.choice(["bf16", "f32"]))
    experts = _log(rng, 8, 512)
    return dict(op=op, t=_log(rng, 1, 4096), hidden=128 * rng.randint(2, 16), experts=experts,
                top_k=rng.randint(1, min(10, experts)), inter=128 * rng.randint(1, 6), skew=rng.choice([0.0, 1.1]),
                x=rng.choice(["f32", "bf16"]))


# ---- inputs

def _bits(e, dtype):
    """Bytes as the 8-bit floating-point type they are."""
    return e.to(torch.uint8).view(dtype)


def _values8(shape, g, sigma):
    """Normal values of standard deviation sigma, held in e4m3."""
    return (torch.randn(shape, device="cuda", generator=g) * sigma).clamp_(-448, 448).to(E4M3)


def _scales8(shape, g, lo, hi):
    """Block scales 2^lo .. 2^(hi - 1)."""
    return _bits(torch.randint(127 + lo, 127 + hi, shape, device="cuda", generator=g), E8M0)


def _pad4(n):
    return (n + 3) // 4 * 4


def _popularity(n, skew, g):
    p = torch.arange(1, n + 1, device="cuda", dtype=torch.float64) ** -skew
    return (p / p.sum())[torch.randperm(n, device="cuda", generator=g)]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case)
    if own:
        from quantized_routed_expert_fn_gb300 import moe
        s["moe"] = moe
    if s["op"] == "gate":
        t, e = s["t"], s["experts"]
        logits = torch.randn(t, e, device="cuda", generator=g) * 2
        # rows of a padded batch have every expert masked; other rows a few of them (experts that are switched off)
        if s["masked"]:
            logits[torch.rand(t, e, device="cuda", generator=g) < s["masked"] / 4] = -math.inf
            logits[torch.rand(t, device="cuda", generator=g) < s["masked"]] = -math.inf
        s["logits"] = logits.to(BF16) if s["dtype"] == "bf16" else logits
        s["bias_values"] = torch.randn(e, device="cuda", generator=g) * 0.05 if s["bias"] else None
        s["idx"] = torch.empty(t, s["top_k"], dtype=torch.int32, device="cuda")
        s["w"] = torch.empty(t, s["top_k"], device="cuda")
    elif s["op"] == "quant8":
        rows, cols, br = s["rows"], s["cols"], s["block_rows"]
        # normal values whose size varies from row to row, as activations and weight rows do
        x = torch.randn(rows, cols, device="cuda", generator=g) * torch.exp(torch.randn(rows, 1, device="cuda", generator=g))
        s["x_values"] = x.to(BF16) if s["dtype"] == "bf16" else x
        s["q"] = torch.empty(rows, cols, dtype=E4M3, device="cuda")
        s["s"] = torch.empty(-(-rows // br), -(-cols // 128), dtype=torch.uint8, device="cuda").view(E8M0)
    elif s["op"] == "mm8":
        t, n, k, groups = s["t"], s["n"], s["k"], s["groups"]
        kb, nb = -(-k // 128), -(-n // 128)
        s["a"] = _values8((t, k), g, 120.0)
        s["sa"] = _scales8((t, _pad4(kb)), g, -9, -5)[:, :kb]
        lead = (groups,) if groups else ()
        s["b"] = _values8(lead + (n, k), g, 120.0)
        s["sb"] = _scales8(lead + (nb, kb), g, -14, -11)
        s["out_values"] = torch.full((t, n), 0.5, dtype=BF16 if s["out"] == "bf16" else F32, device="cuda")
        s["offs"] = None
        if groups:
            p = _popularity(groups, s["skew"], g)
            of = torch.multinomial(p, t - s["pad"], replacement=True, generator=g)
            s["offs"] = torch.cat([torch.zeros(1, device="cuda", dtype=torch.int64),
                                   torch.bincount(of, minlength=groups).cumsum(0)]).to(torch.int32)
    else:
        t, h, e, k, i = s["t"], s["hidden"], s["experts"], s["top_k"], s["inter"]
        x = torch.randn(t, h, device="cuda", generator=g)
        s["x_values"] = x.to(BF16) if s["x"] == "bf16" else x
        s["gate_up"] = _values8((e, 2 * i, h), g, 120.0)
        s["gate_up_s"] = _scales8((e, 2 * i // 128, h // 128), g, -13, -11)
        s["down"] = _values8((e, h, i), g, 120.0)
        s["down_s"] = _scales8((e, h // 128, i // 128), g, -13, -11)
        p = _popularity(e, s["skew"], g)
        noise = -torch.log(-torch.log(torch.rand(t, e, device="cuda", generator=g, dtype=torch.float64).clamp_(1e-300, 1 - 1e-16)))
        s["idx"] = (p.log() + noise).topk(k, dim=1).indices.to(torch.int32)
        w = torch.rand(t, k, device="cuda", generator=g) + 0.05
        s["w"] = w / w.sum(1, keepdim=True)
        s["out_values"] = torch.empty(t, h, dtype=BF16, device="cuda")
        if own:
            s["layer"] = moe.Layer8(s["gate_up"], s["gate_up_s"], s["down"], s["down_s"])
            s["work"] = moe.alloc_workspace(moe.experts8_workspace(s["layer"], t, k))
    if own and s["op"] in ("mm8", "experts8"):
        s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    return s


# ---- plain forms

def _gate_plain(s):
    # 64 bits: scores next to one another decide which expert is chosen
    logits, bias = s["logits"].double(), s["bias_values"]
    t, e = logits.shape
    dead = ~(logits > -math.inf)
    x = torch.where(dead, torch.full_like(logits, -math.inf), logits)
    if s["score"] == "softmax":
        m = x.amax(1, keepdim=True).clamp(min=-1e300)
        p = torch.exp(x - m)
        p = p / p.sum(1, keepdim=True).clamp(min=1e-300)
    else:
        p = 1 / (1 + torch.exp(-x))
    sel = p + bias.double() if bias is not None else p
    sel = sel.masked_fill(dead, -math.inf)
    key = sel if bias is not None else x  # without a bias the logit orders as the score does
    if s["groups"] > 1:
        per = sel.view(t, s["groups"], -1)
        best = per.topk(min(s["group_top"], per.shape[2]), dim=2).values
        score = torch.where(best > -math.inf, best, 0.0).sum(2).masked_fill(best[:, :, 0] == -math.inf, -math.inf)
        order = torch.sort(score, dim=1, descending=True, stable=True).indices[:, : s["top_groups"]]
        keep = torch.zeros(t, s["groups"], dtype=torch.bool, device=p.device).scatter_(1, order, True)
        key = key.masked_fill(~keep.repeat_interleave(e // s["groups"], 1), -math.inf)
    top = torch.sort(key, dim=1, descending=True, stable=True)
    idx = top.indices[:, : s["top_k"]]
    none = top.values[:, : s["top_k"]] == -math.inf
    w = p.gather(1, idx).masked_fill(none, 0.0)
    if s["renorm"]:
        w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
    return idx.masked_fill(none, -1).to(torch.int32), (w * s["scale"]).float()


def _exp2(e):
    """2^e for whole e in -126 .. 127, exactly."""
    return ((e + 127) << 23).view(F32)


def _quantise(x, br):
    """e4m3 values (as 32-bit numbers) and scale exponents of x [rows][cols], per br x 128 block."""
    rows, cols = x.shape
    rb, cb = -(-rows // br), -(-cols // 128)
    p = torch.zeros(rb * br, cb * 128, device=x.device)
    p[:rows, :cols] = x
    p = p.view(rb, br, cb, 128)
    a = p.abs().amax((1, 3))
    m, e = torch.frexp(a)  # a = m 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
    e = torch.where(a > 0, e - 9 + (m > 0.875), 0).to(torch.int32)
    q = (p * _exp2(-e)[:, None, :, None]).to(E4M3).float()
    return q.view(rb * br, cb * 128)[:rows, :cols], e


def _spread(values, exps, br):
    """values [..][rows][cols] times the scale 2^exps of each br x 128 block."""
    f = _exp2(exps).repeat_interleave(128, -1)[..., : values.shape[-1]]
    return values * (f.repeat_interleave(br, -2)[..., : values.shape[-2], :] if br > 1 else f)


def _exponents(s):
    return s.view(torch.uint8).to(torch.int32) - 127


def _grouped_product(a, w, offs):
    """Row r of a, in group g (offs[g] <= r < offs[g + 1]), times w[g]^T; rows in no group give zero."""
    r = torch.arange(a.shape[0], device=a.device)
    g = torch.searchsorted(offs, r, right=True) - 1
    r = r[g < w.shape[0]]
    g = g[g < w.shape[0]]
    slot = r - offs[g]
    y = torch.zeros(a.shape[0], w.shape[1], device=a.device)
    if r.numel():
        packed = torch.zeros(w.shape[0], int(slot.max()) + 1, a.shape[1], device=a.device)
        packed[g, slot] = a[r]
        y[r] = torch.bmm(packed, w.transpose(1, 2))[g, slot]
    return y


def _mm8_plain(s):
    a = _spread(s["a"].float(), _exponents(s["sa"]), 1)
    b = _spread(s["b"].float(), _exponents(s["sb"]), 128)
    out = s["out_values"]
    if s["offs"] is None:
        return (a @ b.T).to(out.dtype)
    offs = s["offs"].long()
    inside = torch.arange(s["t"], device=a.device) < offs[-1]
    return torch.where(inside[:, None], _grouped_product(a, b, offs).to(out.dtype), out)


def _experts8_plain(s):
    t, k, i, e = s["t"], s["top_k"], s["inter"], s["experts"]
    ids, order = torch.sort(s["idx"].reshape(-1).long(), stable=True)
    offs = torch.searchsorted(ids, torch.arange(e + 1, device=ids.device))
    x = _spread(*_quantise(s["x_values"].float(), 1), 1)
    gu = _grouped_product(x[order // k], _spread(s["gate_up"].float(), _exponents(s["gate_up_s"]), 128), offs)
    gate, up = gu[:, :i], gu[:, i:]
    h = _spread(*_quantise(gate / (1 + torch.exp(-gate)) * up, 1), 1)
    y = _grouped_product(h, _spread(s["down"].float(), _exponents(s["down_s"]), 128), offs)
    back = torch.empty_like(order)
    back[order] = torch.arange(t * k, device=order.device)
    return (y[back].view(t, k, -1) * s["w"][:, :, None]).sum(1).to(BF16)


def run(s):
    op = s["op"]
    if not own:
        if op == "gate":
            return _gate_plain(s)
        if op == "quant8":
            q, e = _quantise(s["x_values"].float(), s["block_rows"])
            return q.to(E4M3), _bits(e + 127, E8M0)
        return _mm8_plain(s) if op == "mm8" else _experts8_plain(s)
    moe = s["moe"]
    if op == "gate":
        moe.gate(s["logits"], s["idx"], s["w"], bias=s["bias_values"], score=s["score"], n_groups=s["groups"],
                 top_groups=s["top_groups"], group_top=s["group_top"], renorm=s["renorm"], scale=s["scale"])
        return s["idx"], s["w"]
    if op == "quant8":
        moe.quant8(s["x_values"], s["q"], s["s"], block_rows=s["block_rows"])
        return s["q"], s["s"]
    if op == "mm8":
        moe.mm8(s["a"], s["sa"], s["b"], s["sb"], s["out_values"], s["status"], offs=s["offs"])
    else:
        moe.experts8(s["layer"], s["x_values"], s["idx"], s["w"], s["out_values"], s["work"], s["status"])
    return s["out_values"]


# ---- the same from the definitions, in 64 bits

def _round_e4m3(x):
    """Nearest e4m3 value (ties to even) of 64-bit x, |x| <= 448."""
    e = torch.frexp(x.abs()).exponent.to(torch.float64) - 1
    step = torch.exp2(torch.clamp(e, min=-6) - 3)
    return torch.round(x / step) * step


def _block_exponent(a):
    """Least whole e with a <= 448 * 2^e (0 where a is 0)."""
    e = torch.ceil(torch.log2(torch.clamp(a, min=1e-300) / 448)) - 1
    e = e + (a > 448 * torch.exp2(e)) + (a > 448 * torch.exp2(e + 1))
    return torch.where(a > 0, e, torch.zeros_like(e))


def _exact_rows(x):
    """x [rows][cols] rounded to e4m3 under a power-of-two scale per 128 of a row, as the values it stands for."""
    parts = torch.split(x, 128, dim=1)
    done = []
    for p in parts:
        f = torch.exp2(_block_exponent(p.abs().amax(1, keepdim=True)))
        done.append(_round_e4m3(p / f) * f)
    return torch.cat(done, 1)


def _exact_weights(q, s):
    w = q.to(torch.float64)
    f = torch.exp2(s.view(torch.uint8).to(torch.float64) - 127)
    rows = torch.arange(w.shape[0], device=w.device) // 128
    cols = torch.arange(w.shape[1], device=w.device) // 128
    return w * f[rows][:, cols]


def _exact_gate(s):
    x = s["logits"].double().cpu().numpy()
    bias = np.zeros(x.shape[1]) if s["bias_values"] is None else s["bias_values"].double().cpu().numpy()
    t, e = x.shape
    k, groups = s["top_k"], s["groups"]
    live = x > -np.inf
    with np.errstate(all="ignore"):
        if s["score"] == "softmax":
            top = np.where(live.any(1), np.where(live, x, -np.inf).max(1), 0.0)
            num = np.where(live, np.exp(x - top[:, None]), 0.0)
            p = num / np.maximum(num.sum(1), 1e-300)[:, None]
        else:
            p = np.where(live, np.exp(-np.logaddexp(0, -x)), 0.0)
    sel = np.where(live, p + bias, -np.inf)
    rank = sel if s["bias_values"] is not None else np.where(live, x, -np.inf)
    if groups > 1:
        ordered = -np.sort(-sel.reshape(t, groups, -1), axis=2)[:, :, : s["group_top"]]
        score = np.where(np.isfinite(ordered), ordered, 0.0).sum(2)
        score[ordered[:, :, 0] == -np.inf] = -np.inf
        chosen = np.argsort(-score, axis=1, kind="stable")[:, : s["top_groups"]]
        allowed = np.zeros((t, groups), dtype=bool)
        np.put_along_axis(allowed, chosen, True, axis=1)
        rank = np.where(np.repeat(allowed, e // groups, axis=1), rank, -np.inf)
    idx = np.argsort(-rank, axis=1, kind="stable")[:, :k]
    none = np.take_along_axis(rank, idx, 1) == -np.inf
    w = np.where(none, 0.0, np.take_along_axis(p, idx, 1))
    if s["renorm"]:
        w = w / np.maximum(w.sum(1, keepdims=True), 1e-300)
    return np.where(none, -1, idx).astype(np.int32), w * s["scale"]


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "gate":
        return _exact_gate(s)
    if op == "quant8":
        x, br = s["x_values"].double(), s["block_rows"]
        rows, cols = x.shape
        a = torch.stack([p.abs().amax(1) for p in torch.split(x, 128, dim=1)], 1)
        a = torch.stack([p.amax(0) for p in torch.split(a, br, dim=0)], 0) if br > 1 else a
        e = _block_exponent(a)
        f = torch.exp2(e)[torch.arange(rows, device="cuda") // br][:, torch.arange(cols, device="cuda") // 128]
        return _round_e4m3(x / f), torch.exp2(e)
    if op == "mm8":
        t, offs = s["t"], s["offs"]
        a = s["a"].double() * torch.exp2(s["sa"].view(torch.uint8).double() - 127)[:, torch.arange(s["k"], device="cuda") // 128]
        if offs is None:
            return a @ _exact_weights(s["b"], s["sb"]).T
        out, offs = s["out_values"].double(), offs.tolist()
        for g in range(s["groups"]):
            if offs[g + 1] > offs[g]:
                out[offs[g]:offs[g + 1]] = a[offs[g]:offs[g + 1]] @ _exact_weights(s["b"][g], s["sb"][g]).T
        return out
    x, i = _exact_rows(s["x_values"].double()), s["inter"]
    out = torch.zeros(s["t"], s["hidden"], dtype=torch.float64, device="cuda")
    for e in torch.unique(s["idx"]).tolist():
        tok, j = torch.nonzero(s["idx"] == e, as_tuple=True)
        gu = x[tok] @ _exact_weights(s["gate_up"][e], s["gate_up_s"][e]).T
        h = _exact_rows(gu[:, :i] * torch.sigmoid(gu[:, :i]) * gu[:, i:])
        out.index_add_(0, tok, s["w"][tok, j].double()[:, None] * (h @ _exact_weights(s["down"][e], s["down_s"][e]).T))
    return out


def _visited(n, k, t, skew):
    """Expected number of n experts of that popularity that t tokens with k choices each visit."""
    p = np.arange(1, n + 1) ** -skew
    return float((1 - (1 - np.minimum(1.0, k * p / p.sum())) ** t).sum())


def work(case):
    c = case
    if c["op"] == "gate":
        size = 2 if c["dtype"] == "bf16" else 4
        return {"bytes": c["t"] * (c["experts"] * size + c["top_k"] * 8) + c["experts"] * 4 * c["bias"],
                "flops": c["t"] * c["experts"] * 10}
    if c["op"] == "quant8":
        n = c["rows"] * c["cols"]
        return {"bytes": n * (3 if c["dtype"] == "bf16" else 5) + -(-c["rows"] // c["block_rows"]) * -(-c["cols"] // 128),
                "flops": 3 * n}
    if c["op"] == "mm8":
        t = c["t"] - c["pad"]
        kb, nb = -(-c["k"] // 128), -(-c["n"] // 128)
        used = _visited(c["groups"], 1, t, c["skew"]) if c["groups"] else 1
        return {"bytes": t * (c["k"] + kb) + used * (c["n"] * c["k"] + nb * kb) + t * c["n"] * (2 if c["out"] == "bf16" else 4),
                "flops": 2 * t * c["n"] * c["k"]}
    t, h, i, k = c["t"], c["hidden"], c["inter"], c["top_k"]
    used = _visited(c["experts"], k, t, c["skew"])
    return {"bytes": used * 3 * h * i * (1 + 1 / 16384) + t * h * ((2 if c["x"] == "bf16" else 4) + 2) + t * k * 8,
            "flops": 6 * t * k * h * i}
