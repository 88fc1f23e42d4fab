"""GPU parity of moe_norm and moe_add_norm against plain 64-bit implementations.

Tolerances (refblock): 32-bit sums of squares, root and quotient, in units of 2^-24 of the result; the sum's error where
terms cancel in the residual; half a step of the output's type.  e4m3: the bytes of a value within those bounds."""
import threading

import numpy as np
import pytest

import refblock as rb

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from quantized_routed_expert_fn_gb300 import build, moe as m
    build.build()
    m.lib()
    return m


TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def cuda(a, kind="f32", pad=0, shift=0):
    """a on the GPU in that type, rows `pad` values further apart, the first `shift` values into its buffer."""
    x = torch.from_numpy(np.ascontiguousarray(a)).to(TYPES[kind])
    if not pad and not shift:
        return x.cuda()
    r, c = x.shape
    wide = torch.full((r * (c + pad) + shift,), float("nan"), dtype=x.dtype, device="cuda")
    view = wide[shift:].view(r, c + pad)[:, :c]
    view.copy_(x)
    return view


def f64(t):
    return t.double().cpu().numpy()


def outputs(t, h, kind, pad=0):
    """(out, scales) with a sentinel behind every row and around the buffer."""
    if kind == "e4m3":
        return (torch.full((t, h + pad), 0x55, dtype=torch.uint8, device="cuda")[:, :h],
                torch.full((t, -(-h // 128) + pad), 0x55, dtype=torch.uint8, device="cuda")[:, : -(-h // 128)])
    return torch.full((t, h + pad), 7.0, dtype=TYPES[kind], device="cuda")[:, :h], None


def untouched(view, value):
    whole = view._base if view._base is not None else view
    if whole.dim() == 2:
        assert (whole[:, view.shape[1]:] == value).all()


def check_out(out, s, kind, ref, bound, what=""):
    if kind == "e4m3":
        rb.check_e4m3(out.cpu().numpy(), s.cpu().numpy(), ref, bound, what)
        untouched(s, 0x55)
    else:
        rb.check(f64(out), ref, bound, kind, what)
    untouched(out, 0x55 if kind == "e4m3" else 7.0)


SHAPES = [(1, 1), (1, 2048), (3, 7), (5, 128), (2, 130), (7, 4096), (4, 4090), (3, 8200), (2, 16384), (2, 20002), (1, 32768),
          (37, 16), (1000, 64), (65, 200), (300, 257), (9, 4097), (2, 16387)]


@pytest.mark.parametrize("out", ["f32", "bf16", "e4m3"])
@pytest.mark.parametrize("x", ["f32", "bf16"])
@pytest.mark.parametrize("t,h", SHAPES, ids=[f"{a}x{b}" for a, b in SHAPES])
def test_norm(moe, t, h, x, out):
    g = np.random.default_rng(t * 7919 + h)
    for pad, shift, weight in ((0, 0, True), (8, 0, False), (5, 1, True), (2, 2, True)):
        a = g.normal(size=(t, h)) * np.exp(g.normal(size=(t, 1)))
        xt = cuda(a.astype(np.float32), x, pad, shift)
        w = cuda((1 + 0.3 * g.normal(size=h)).astype(np.float32)) if weight else None
        o, s = outputs(t, h, out, pad)
        moe.norm(xt, o, w=w, eps=1e-5, scales=s)
        torch.cuda.synchronize()
        ref = rb.norm(f64(xt), None if w is None else f64(w), 1e-5)
        check_out(o, s, out, ref, np.abs(ref) * (rb.NORM + 2) * rb.U, (pad, shift))


ADD = [dict(), dict(post=True), dict(post=True, w_post=True, gate="row", sig=True, scale=0.5),
       dict(gate="channel", res_scale=0.75), dict(gate="full", sig=True, w=True), dict(gate="full", gk="bf16", post=True),
       dict(gate="one", scale=-1.5, w=True), dict(gate="row", gk="bf16", res_scale=0.0, w=True)]


@pytest.mark.parametrize("kinds", [("f32", "f32", "f32", "f32"), ("bf16", "f32", "f32", "bf16"), ("bf16", "bf16", "bf16", "e4m3"),
                                   ("f32", "bf16", "f32", "e4m3"), ("bf16", "f32", "bf16", None)], ids=lambda k: "-".join(map(str, k)))
@pytest.mark.parametrize("o", ADD, ids=range(len(ADD)))
def test_add_norm(moe, o, kinds):
    yk, rk, rok, out = kinds
    g = np.random.default_rng(11)
    for t, h, pad, shift in ((1, 2048, 0, 0), (5, 96, 0, 0), (33, 257, 3, 1), (7, 4090, 0, 0), (130, 1000, 8, 0), (2, 16386, 2, 2), (3, 1, 0, 0),
                             (3, 12288, 0, 0), (2, 20008, 8, 0)):
        y = cuda(g.normal(size=(t, h)).astype(np.float32), yk, pad, shift)
        res = cuda((g.normal(size=(t, h)) * 3).astype(np.float32), rk, pad, shift)
        shape = {None: None, "row": (t, 1), "channel": (1, h), "full": (t, h), "one": (1, 1)}[o.get("gate")]
        gate = None if shape is None else cuda(g.normal(size=shape).astype(np.float32), o.get("gk", "f32"))
        wp = cuda((1 + 0.3 * g.normal(size=h)).astype(np.float32)) if o.get("w_post") else None
        w = cuda((1 + 0.3 * g.normal(size=h)).astype(np.float32)) if o.get("w") else None
        ro, _ = outputs(t, h, rok, pad)
        to, s = outputs(t, h, out, pad) if out else (None, None)
        moe.add_norm(y, res, ro, post=o.get("post", False), w_post=wp, gate=gate, gate_sigmoid=o.get("sig", False),
                     scale=o.get("scale", 1.0), res_scale=o.get("res_scale", 1.0), out=to, w=w, scales=s)
        torch.cuda.synchronize()
        arr = lambda x: None if x is None else f64(x)  # noqa: E731
        r, dr, n, dn = rb.add_norm(f64(y), f64(res), o.get("post", False), arr(wp), arr(gate), o.get("sig", False),
                                   o.get("scale", 1.0), o.get("res_scale", 1.0), arr(w))
        rb.check(f64(ro), r, dr, rok, (t, h))
        untouched(ro, 7.0)
        if out:
            check_out(to, s, out, n, dn, (t, h))


@pytest.mark.parametrize("out", ["f32", "bf16", "e4m3", None])
@pytest.mark.parametrize("t,h,pad,yk,rk", [(20000, 72, 0, "bf16", "bf16"), (40000, 33, 0, "bf16", "f32"), (6000, 1000, 8, "bf16", "f32"),
                                           (4001, 4090, 0, "bf16", "bf16"), (9000, 2047, 0, "f32", "f32"), (2500, 8191, 0, "bf16", "f32"),
                                           (2000, 16376, 0, "f32", "bf16"), (30000, 130, 3, "bf16", "bf16"), (5000, 2048, 0, "bf16", "f32")])
def test_many_rows(moe, t, h, pad, yk, rk, out):
    """Blocks that walk over rows, with the next ones on their way: every row against 64 bits (on the GPU)."""
    g = torch.Generator(device="cuda")
    g.manual_seed(t + h)
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    y, res = (rnd(t, h + pad).to(TYPES[k])[:, :h] for k in (yk, rk))
    w, wp, gate = 1 + 0.2 * rnd(h), 1 + 0.2 * rnd(h), rnd(1, h)
    y0, r0 = y.double(), res.double()
    ro, (to, s) = torch.empty(t, h, dtype=TYPES[rk], device="cuda"), outputs(t, h, out) if out else (None, None)
    moe.add_norm(y, res, ro, post=True, w_post=wp, gate=gate, gate_sigmoid=True, scale=0.5, out=to, w=w, scales=s)
    n64 = lambda x, v: x / torch.sqrt((x * x).mean(1, keepdim=True) + 1e-6) * v  # noqa: E731
    v = n64(y0, wp.double()) * torch.sigmoid(gate.double())
    r = r0 + 0.5 * v
    dr = ((0.5 * v).abs() * (rb.NORM + 12) + r0.abs() * 2 + r.abs()) * rb.U
    assert ((ro.double() - r).abs() <= dr * 1.01 + r.abs() * rb.HALF[rk]).all()
    if out:
        rms = torch.sqrt((r * r).mean(1, keepdim=True) + 1e-6)
        ref = n64(r, w.double())
        bound = dr / rms * w.abs() + ref.abs() * (torch.sqrt((dr * dr).mean(1, keepdim=True)) / rms + (rb.NORM + 2) * rb.U)
        if out == "e4m3":
            step = torch.exp2(s.double() - 127).repeat_interleave(128, 1)[:, :h]
            got = to.view(torch.float8_e4m3fn).double() * step
            # half a step: 2^-4 of the value, or 2^-10 of the scale
            assert ((got - ref).abs() <= bound * 1.1 + torch.maximum(ref.abs() * 2.0 ** -4, step * 2.0 ** -10)).all()
            top = (ref.abs() / step).amax(1)
            assert (top <= 448 * 1.001).all()
        else:
            assert ((to.double() - ref).abs() <= bound * 1.01 + ref.abs() * rb.HALF[out]).all()
    # in place, and the plain norm
    moe.add_norm(y, res, res, post=True, w_post=wp, gate=gate, gate_sigmoid=True, scale=0.5)
    # (another form of the kernel may take it, whose sums have another order)
    assert ((res.double() - r).abs() <= dr * 1.01 + r.abs() * rb.HALF[rk]).all()
    n = torch.empty(t, h, dtype=TYPES[yk], device="cuda")
    moe.norm(y, n, w=w)
    ref = n64(y0, w.double())
    assert ((n.double() - ref).abs() <= ref.abs() * ((rb.NORM + 2) * rb.U * 1.01 + rb.HALF[yk])).all()


@pytest.mark.parametrize("h", [64, 2048, 2047])
@pytest.mark.parametrize("out", ["f32", "bf16", "e4m3"])
def test_norm_special_rows(moe, h, out):
    """Zeros, infinities, NaN, rows whose squares leave the 32-bit range at either end."""
    g = np.random.default_rng(3)
    a = g.normal(size=(12, h))
    a[0] = 0
    a[1] *= 1e30
    a[2] = 3.4e38
    a[3] *= 1e-30
    a[4, 5] = np.inf
    a[5, 9] = np.nan
    a[6, 3], a[6, 60] = np.inf, -np.inf
    a[7] *= 1e18
    a[8, 1:] = 0
    a[9] = 1e-45
    a[10, 1] = 3e38
    xt = cuda(a.astype(np.float32))
    o, s = outputs(12, h, out)
    moe.norm(xt, o, scales=s)
    torch.cuda.synchronize()
    ref = rb.norm(f64(xt))
    # squares below the normal numbers: an absolute 2^-149 each, beside eps = 1e-6 nothing
    check_out(o, s, out, ref, np.abs(np.nan_to_num(ref)) * (rb.NORM + 4) * rb.U)


def test_in_place(moe):
    """The residual stream updated where it stands, and the norm written over the block's output."""
    g = np.random.default_rng(1)
    t, h = 70, 1000
    for out_in_y in (False, True):
        y, res = cuda(g.normal(size=(t, h)).astype(np.float32), "bf16"), cuda(g.normal(size=(t, h)).astype(np.float32))
        y0, r0 = f64(y), f64(res)
        moe.add_norm(y, res, res, post=True, out=y if out_in_y else None)
        r, dr, n, dn = rb.add_norm(y0, r0, post=True)
        rb.check(f64(res), r, dr, "f32")
        if out_in_y:
            rb.check(f64(y), n, dn, "bf16")
        moe.norm(res, res)
        assert np.abs(f64(res) - rb.norm(r)).max() < 1e-4


def test_norm_gives_quant8s_bytes(moe):
    """The e4m3 output is quant8 of the 32-bit output, bit for bit, at any alignment."""
    g = np.random.default_rng(2)
    for t, h, pad in ((300, 2048, 0), (33, 1002, 2), (33, 1001, 0), (5, 40, 0)):
        x = cuda(g.normal(size=(t, h)).astype(np.float32), "bf16", pad)
        o32, _ = outputs(t, h, "f32")
        moe.norm(x, o32)
        q, s = outputs(t, h, "e4m3")
        moe.norm(x, q, scales=s)
        q2, s2 = torch.empty_like(q), torch.empty_like(s)
        moe.quant8(o32.contiguous(), q2, s2)
        assert torch.equal(q, q2) and torch.equal(s, s2)


def test_repeats_streams_graphs_and_threads(moe):
    g = np.random.default_rng(4)
    t, h = 1500, 2048
    y, res = cuda(g.normal(size=(t, h)).astype(np.float32), "bf16"), cuda(g.normal(size=(t, h)).astype(np.float32))
    gate = cuda(g.normal(size=(t, 1)).astype(np.float32))

    def call(ro, out, stream=None):
        moe.add_norm(y, res, ro, post=True, gate=gate, gate_sigmoid=True, out=out, stream=stream)
    ro, out = torch.empty_like(res), torch.empty_like(y)
    call(ro, out)
    torch.cuda.synchronize()
    side, bufs = torch.cuda.Stream(), [(torch.empty_like(res), torch.empty_like(y)) for _ in range(4)]
    side.wait_stream(torch.cuda.current_stream())
    call(*bufs[0], stream=side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(*bufs[1])
        moe.norm(bufs[1][0], bufs[1][1])
        call(*bufs[1])
    for _ in range(3):
        graph.replay()
    workers = [threading.Thread(target=lambda b=b: [call(*b) for _ in range(5)]) for b in bufs[2:]]
    [w.start() for w in workers]
    [w.join() for w in workers]
    torch.cuda.synchronize()
    for r, n in bufs:
        assert torch.equal(r, ro) and torch.equal(n, out)


def test_empty_and_far_rows(moe):
    """No rows: nothing is touched; offsets past 32 bits: the last of 1.1 million rows of 4000."""
    o, _ = outputs(0, 64, "f32")
    moe.norm(torch.empty(0, 64, device="cuda"), o)
    t, h = 1_100_000, 4000
    x = torch.ones(t, h, dtype=torch.bfloat16, device="cuda")
    x[-1] = torch.linspace(-1, 1, h, device="cuda")
    out = torch.empty_like(x)
    moe.norm(x, out)
    ref = rb.norm(f64(x[-1:]))
    rb.check(f64(out[-1:]), ref, np.abs(ref) * (rb.NORM + 2) * rb.U, "bf16")
    assert (out[: t - 1].sum(1, dtype=torch.float32) == h).all()
