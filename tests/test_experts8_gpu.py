"""GPU parity of the 8-bit experts (moe_gate, moe_quant8, moe_mm8, moe_experts8) against plain 64-bit implementations.

Tolerances.  Ids, scale bytes, e4m3 bytes: equal.  Gate weights: a relative 2^-19 (32-bit exponential, sum and
quotients) of the largest weight of the row.  Products: terms of e4m3 values and powers of two are exact; each 32-wide
step may drop what lies below 2^-23 of its sum for each of its 33 terms, in all k * 2^-23 of the sum of magnitudes;
the output's rounding adds half a step, eps / 2 relative.  Inputs whose every partial sum is a small whole number have
to come out exactly."""
import numpy as np
import pytest

import ref8

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}  # half a step, relative: eps / 2


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from quantized_routed_expert_fn_gb300 import build, moe as m
    build.build()
    m.lib()
    return m


def dt(name):
    return torch.float32 if name == "f32" else torch.bfloat16


def cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def f64(t):
    return t.double().cpu().numpy()


# ------------------------------------------------------------ gate

def run_gate(m, lg, k, bias=None, ld=None, **kw):
    t, e = lg.shape
    if ld:
        wide = torch.full((t, ld), 1e30, dtype=lg.dtype, device="cuda")
        wide[:, :e] = lg
        lg = wide[:, :e]
    idx = torch.full((t, k), 77, dtype=torch.int32, device="cuda")
    w = torch.full((t, k), 77.0, device="cuda")
    m.gate(lg, idx, w, bias=bias, **kw)
    torch.cuda.synchronize()
    return idx.cpu().numpy(), w.cpu().numpy()


def check_gate(m, lg, k, bias=None, ld=None, score="softmax", n_groups=1, top_groups=1, group_top=1, renorm=False, scale=1.0):
    idx, w = run_gate(m, lg, k, bias, ld, score=score, n_groups=n_groups, top_groups=top_groups, group_top=group_top,
                      renorm=renorm, scale=scale)
    ri, rw = ref8.gate(f64(lg), k, score, None if bias is None else f64(bias), n_groups, top_groups, group_top, renorm, scale)
    assert np.array_equal(idx, ri), np.nonzero((idx != ri).any(1))[0][:5]
    assert (np.abs(w - rw) <= 2.0 ** -19 * np.abs(rw).max(1, keepdims=True) + 1e-37).all()
    return idx, w


GATES = [  # t, E, k, options
    (1, 1, 1, {}), (3, 7, 3, dict(renorm=True)), (5, 8, 2, dict(score="sigmoid")), (37, 33, 8, dict(score="sigmoid", bias=True)),
    (64, 128, 8, dict(renorm=True)), (130, 100, 10, dict(bias=True, renorm=True, scale=2.5)), (9, 512, 10, dict(renorm=True)),
    (31, 1000, 16, dict(score="sigmoid", bias=True, renorm=True)), (17, 1024, 32, dict(renorm=True)),
    (6, 1024, 32, dict(score="sigmoid", bias=True)), (5, 40, 31, dict(bias=True)),
    (65, 256, 8, dict(score="sigmoid", bias=True, n_groups=8, top_groups=4, group_top=2, renorm=True, scale=2.5)),
    (65, 256, 8, dict(n_groups=8, top_groups=3, group_top=1)), (33, 160, 6, dict(n_groups=8, top_groups=3, group_top=1, scale=16.0)),
    (33, 96, 5, dict(n_groups=32, top_groups=7, group_top=2, score="sigmoid")), (20, 60, 4, dict(n_groups=4, top_groups=2, group_top=2)),
    (20, 60, 30, dict(n_groups=4, top_groups=2, group_top=1, bias=True)), (11, 72, 9, dict(n_groups=24, top_groups=5, group_top=2, bias=True)),
    (8, 64, 4, dict(n_groups=4, top_groups=4, group_top=2, bias=True)), (12, 32, 1, dict(n_groups=32, top_groups=1)),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("t,e,k,o", GATES, ids=[f"{g[0]}x{g[1]}k{g[2]}_{i}" for i, g in enumerate(GATES)])
def test_gate(moe, t, e, k, o, dtype):
    g = np.random.default_rng(e * 1000 + t)
    lg = cuda((g.normal(size=(t, e)) * 2).astype(np.float32)).to(dt(dtype))
    o = dict(o)
    bias = cuda((g.normal(size=e) * 0.1).astype(np.float32)) if o.pop("bias", False) else None
    check_gate(moe, lg, k, bias, **o)
    check_gate(moe, lg, k, bias, ld=e + 5, **o)


SPECIAL = [dict(renorm=True), dict(), dict(score="sigmoid"), dict(score="sigmoid", renorm=True), dict(bias=True, renorm=True),
           dict(score="sigmoid", bias=True), dict(n_groups=8, top_groups=2, group_top=2, score="sigmoid", bias=True, renorm=True),
           dict(n_groups=8, top_groups=3, group_top=1), dict(n_groups=8, top_groups=3, group_top=2)]


@pytest.mark.parametrize("o", SPECIAL, ids=range(len(SPECIAL)))
def test_gate_special_rows(moe, o):
    """Masked, tied, infinite and NaN logits, and masked biases."""
    g = np.random.default_rng(5)
    e, k = 64, 6
    lg = g.normal(size=(14, e)).astype(np.float32)
    lg[0] = -np.inf
    lg[1] = 0.0
    lg[2, ::2] = -np.inf
    lg[3, 5:] = -np.inf           # fewer experts than top_k
    lg[4] = np.nan
    lg[5, 3:40] = np.nan
    lg[6, 7] = np.inf
    lg[7, [9, 50]] = np.inf
    lg[8] = np.where(g.random(e) < 0.5, -0.0, 0.0)
    lg[9] = np.round(lg[9])       # many ties
    lg[10] = -200.0 + lg[10]      # sigmoids below the 32-bit range's normal numbers
    lg[11] = 100.0 + lg[11]
    lg[12, 1:] = -np.inf
    lg[13] *= 1e4
    o = dict(o)
    bias = None
    if o.pop("bias", False):
        b = (g.normal(size=e) * 0.1).astype(np.float32)
        b[11], b[12] = -np.inf, np.nan
        bias = cuda(b)
    # rows 10 and 11 differ in scores by less than 64 bits hold when a sigmoid saturates: leave what has no order out
    rows = [r for r in range(14) if not (o.get("score") == "sigmoid" and r in (10, 11, 13) and (bias is not None or o.get("group_top") == 2))]
    check_gate(moe, cuda(lg[rows]), k, bias, **o)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,e", [(1, 64), (4, 64), (1, 20), (1, 32), (4, 24)])
def test_gate_scores_a_last_place_apart(moe, score, groups, e):
    """Logits one 32-bit step apart under a bias: 32-bit scores cannot tell them, the choice has to."""
    g = np.random.default_rng(3)
    t, k = 200, 4
    base = g.normal(size=(t, 1)).astype(np.float32)
    lg = np.repeat(base, e, axis=1)
    steps = g.integers(-3, 4, size=(t, e))
    for _ in range(3):
        lg = np.where(steps > 0, np.nextafter(lg, np.float32(np.inf)), np.where(steps < 0, np.nextafter(lg, np.float32(-np.inf)), lg))
        steps = steps - np.sign(steps)
    bias = cuda(np.zeros(e, np.float32))
    lg[::3, : e // 2] -= 1  # half of the experts out of reach
    check_gate(moe, cuda(lg), k, bias, score=score, n_groups=groups, top_groups=1 if groups == 1 else 2, group_top=2, renorm=True)


def test_gate_empty_and_many_rows(moe):
    idx, w = run_gate(moe, torch.empty(0, 16, device="cuda"), 2)
    assert idx.shape == (0, 2)
    g = np.random.default_rng(0)
    lg = cuda(g.normal(size=(9001, 40)).astype(np.float32))
    check_gate(moe, lg, 3, score="sigmoid", bias=cuda((g.normal(size=40) * 0.1).astype(np.float32)), renorm=True)


# ------------------------------------------------------------ quant8

def run_quant(m, x, br, pad=0):
    rows, cols = x.shape
    cb, rb = -(-cols // 128), -(-rows // br)
    q = torch.full((rows, cols + pad), 0x55, dtype=torch.uint8, device="cuda")
    s = torch.full((rb, cb + pad), 0x55, dtype=torch.uint8, device="cuda")
    if pad:
        wide = torch.full((rows, cols + pad), 7.0, dtype=x.dtype, device="cuda")
        wide[:, :cols] = x
        x = wide[:, :cols]
    m.quant8(x, q[:, :cols], s[:, :cb], block_rows=br)
    torch.cuda.synchronize()
    if pad:
        assert (q[:, cols:] == 0x55).all() and (s[:, cb:] == 0x55).all()
    return q[:, :cols].cpu().numpy(), s[:, :cb].cpu().numpy()


def special_values(g, rows, cols):
    x = (g.normal(size=(rows, cols)) * np.exp(g.normal(size=(rows, 1)) * 4)).astype(np.float32)
    flat = x.reshape(-1)
    n = flat.size
    put = [0.0, -0.0, np.inf, -np.inf, np.nan, 1e-45, -1e-40, 448.0, 449.0, 2.0 ** -118, 1e38]
    at = g.choice(n, size=min(n // 3, len(put)), replace=False)
    flat[at] = np.array(put[: len(at)], np.float32)
    return x


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("br", [1, 128])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 128), (3, 129), (2, 127), (5, 1000), (128, 128), (129, 257), (300, 144), (257, 2048)])
def test_quant8(moe, rows, cols, br, dtype):
    g = np.random.default_rng(rows * 7 + cols)
    for special in (False, True):
        x = special_values(g, rows, cols) if special else g.normal(size=(rows, cols)).astype(np.float32)
        xt = cuda(x).to(dt(dtype))
        rq, rs = ref8.quant8(f64(xt), br)
        for pad in (0, 3, 8):
            q, s = run_quant(moe, xt, br, pad)
            assert np.array_equal(s, rs)
            same = (q == rq) | ((q & 127 == 127) & (rq & 127 == 127))
            assert same.all(), np.argwhere(~same)[:5]


def test_quant8_borders(moe):
    """Every tie between two neighbouring e4m3 values, and maxima around 448 * 2^e."""
    v = ref8.E4M3[:127]
    ties = (v[1:] + v[:-1]) / 2
    x = np.concatenate([v, ties, -v, -ties, np.nextafter(ties.astype(np.float32), np.float32(0))]).astype(np.float32)
    x = np.concatenate([x, np.zeros(-len(x) % 127, np.float32)]).reshape(-1, 127)
    x = np.concatenate([x, np.full((x.shape[0], 1), 448, np.float32)], 1)  # scale 1
    rows = [x]
    for e in (-120, -30, -1, 0, 5, 60, 118):
        for a in (448.0, np.nextafter(np.float32(448), np.float32(500)), np.nextafter(np.float32(448), np.float32(0))):
            r = np.linspace(-1, 1, 128, dtype=np.float32) * 0
            r[3], r[9] = np.float32(a) * np.float32(2.0) ** e, np.float32(a) * np.float32(2.0) ** e / 3
            rows.append(r[None])
    rows.append(np.zeros((1, 128), np.float32))
    rows.append(np.full((1, 128), np.inf, np.float32))
    x = np.concatenate(rows)
    rq, rs = ref8.quant8(x)
    q, s = run_quant(moe, cuda(x), 1)
    assert np.array_equal(s, rs) and np.array_equal(q & 127, rq & 127)


# ------------------------------------------------------------ mm8

def operands(g, t, n, k, whole=False, lead=()):
    nk, nb = -(-k // 128), -(-n // 128)
    if whole:  # partial sums are whole numbers below 2^24 * 2^-4: exact in 32 bits in any order
        codes = ref8.round_e4m3(np.arange(-2, 3))
        a, b = g.choice(codes, size=(t, k)), g.choice(codes, size=lead + (n, k))
        return a, g.integers(125, 128, size=(t, nk)).astype(np.uint8), b, g.integers(126, 129, size=lead + (nb, nk)).astype(np.uint8)
    a = ref8.round_e4m3(np.clip(g.normal(size=(t, k)) * 100, -448, 448))
    b = ref8.round_e4m3(np.clip(g.normal(size=lead + (n, k)) * 100, -448, 448))
    return a, g.integers(118, 123, size=(t, nk)).astype(np.uint8), b, g.integers(114, 117, size=lead + (nb, nk)).astype(np.uint8)


def padded(x, ld, fill):
    w = np.full((x.shape[0], ld), fill, x.dtype)
    w[:, : x.shape[1]] = x
    return cuda(w)[:, : x.shape[1]]


def run_mm8(m, a, sa, b, sb, out="bf16", offs=None, pad=0, flags=0, fill=0.5):
    t, k = a.shape
    n = b.shape[-2]
    nk = sa.shape[1]
    # what lies between the rows must not be read as data: NaN codes and scales
    at = padded(a, k + 16 * (pad > 0), 0x7F)
    st = padded(sa, -(-nk // 4) * 4 + 4 * (pad > 0), 255)
    o = torch.full((t, n + pad), fill, dtype=dt(out), device="cuda")
    status = torch.full((1,), 99, dtype=torch.int32, device="cuda")
    m.mm8(at, st, cuda(b), cuda(sb), o[:, :n], status, offs=None if offs is None else cuda(np.asarray(offs, np.int32)), flags=flags)
    torch.cuda.synchronize()
    if pad:
        assert (o[:, n:] == fill).all()
    return f64(o[:, :n]), status.item()


def check_mm8(got, ref, mag, k, out):
    tol = k * 2.0 ** -23 * mag
    tol = tol + (np.abs(ref) + tol) * HALF[out]
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], ref[bad][:4])


SIZES = [(1, 16, 128), (1, 1, 16), (2, 2048, 2048), (4, 100, 144), (7, 129, 4112), (8, 16, 256), (9, 300, 400), (16, 128, 2048),
         (31, 33, 1008), (32, 257, 640), (33, 128, 128), (64, 128, 16), (100, 1, 512), (129, 130, 272), (224, 256, 2048),
         (225, 100, 384), (449, 384, 1024), (1000, 333, 2000),
         (34, 256, 1280), (48, 300, 144), (97, 640, 2048), (193, 129, 128), (700, 1000, 528)]


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("t,n,k", SIZES)
def test_mm8(moe, t, n, k, out):
    g = np.random.default_rng(t * 13 + n)
    a, sa, b, sb = operands(g, t, n, k)
    ref, mag = ref8.mm8(a, sa, b, sb)
    for pad in (0, 7):
        got, status = run_mm8(moe, a, sa, b, sb, out, pad=pad)
        assert status == 0
        check_mm8(got, ref, mag, k, out)


@pytest.mark.parametrize("t,n,k", [(1, 128, 1024), (5, 200, 2048), (32, 130, 528), (33, 130, 528), (150, 260, 2048), (500, 500, 1040)])
def test_mm8_whole_numbers_are_exact(moe, t, n, k):
    g = np.random.default_rng(t + n)
    a, sa, b, sb = operands(g, t, n, k, whole=True)
    ref, _ = ref8.mm8(a, sa, b, sb)
    got, status = run_mm8(moe, a, sa, b, sb, "f32")
    assert status == 0 and np.array_equal(got, ref)


@pytest.mark.parametrize("t", [3, 70])
def test_mm8_nan_and_wide_scales_stay_in_their_rows(moe, t):
    g = np.random.default_rng(t)
    n, k = 140, 384
    a, sa, b, sb = operands(g, t, n, k)
    a[1, 5] = 0x7F
    b[130, 300] = 0xFF
    sa[2, 1] = 255                 # a NaN scale
    sa[0], sb[:] = 127 - 60, 127 + 60  # scales far from 1 that cancel
    ref, mag = ref8.mm8(a, sa, b, sb)
    got, _ = run_mm8(moe, a, np.where(sa == 255, 255, sa).astype(np.uint8), b, sb, "f32")
    nan = np.zeros((t, n), bool)
    nan[1], nan[2], nan[:, 130] = True, True, True
    assert np.array_equal(np.isnan(got), nan)
    x, w = ref8.dequant8(np.where(a == 0x7F, 0, a).astype(np.uint8), np.where(sa == 255, 0, sa).astype(np.uint8)), ref8.dequant8(np.where(b & 127 == 127, 0, b).astype(np.uint8), sb, 128)
    r, mg = x @ w.T, np.abs(x) @ np.abs(w).T
    tol = k * 2.0 ** -23 * mg + np.abs(r) * HALF["f32"]
    assert (np.abs(got - r)[~nan] <= tol[~nan] * 1.001).all()


@pytest.mark.parametrize("shift", [114, -118])
@pytest.mark.parametrize("t", [3, 20, 70])
def test_mm8_scales_that_cancel(moe, t, shift):
    """Row scales times 2^shift and weight scales times 2^-shift: the same numbers, bit for bit."""
    g = np.random.default_rng(t)
    a, sa, b, sb = operands(g, t, 140, 384)
    sa = sa + 4  # 122 to 126
    want, _ = run_mm8(moe, a, sa, b, sb, "f32")
    got, _ = run_mm8(moe, a, (sa.astype(int) + shift).astype(np.uint8), b, (sb.astype(int) - shift).astype(np.uint8), "f32")
    assert np.isfinite(want).all() and np.array_equal(got, want)


GROUPS = [  # rows of each group, rows before, rows behind, n, k
    ([5], 0, 0, 128, 128), ([0, 3, 0, 0, 200, 1, 224, 225, 16, 0], 0, 13, 130, 272), ([1] * 40, 2, 0, 96, 2048),
    ([0, 0, 0], 0, 9, 64, 128), ([300, 17], 5, 40, 256, 512), ([2, 0] * 512, 0, 3, 16, 144), ([33, 31, 32, 47, 48, 49], 0, 0, 384, 1024),
]


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("sizes,before,behind,n,k", GROUPS, ids=range(len(GROUPS)))
def test_mm8_grouped(moe, sizes, before, behind, n, k, out):
    g = np.random.default_rng(len(sizes) + n)
    t, G = before + sum(sizes) + behind, len(sizes)
    offs = before + np.concatenate([[0], np.cumsum(sizes)])
    for whole in (False, True):
        a, sa, b, sb = operands(g, t, n, k, whole, (G,))
        got, status = run_mm8(moe, a, sa, b, sb, out, offs)
        assert status == 0
        for i in range(G):
            r = slice(offs[i], offs[i + 1])
            ref, mag = ref8.mm8(a[r], sa[r], b[i], sb[i])
            if whole and out == "f32":
                assert np.array_equal(got[r], ref)
            else:
                check_mm8(got[r], ref, mag, k, out)
        assert (got[:before] == 0.5).all() and (got[offs[-1]:] == 0.5).all()


@pytest.mark.parametrize("offs", [[0, 50, 40, 64], [-1, 10, 20, 30], [0, 10, 20, 65], [70, 70, 70, 70]])
def test_mm8_reports_bad_offsets_and_writes_nothing(moe, offs):
    g = np.random.default_rng(1)
    a, sa, b, sb = operands(g, 64, 128, 256, lead=(3,))
    got, status = run_mm8(moe, a, sa, b, sb, "f32", offs)
    assert status == moe.EDEVICE and (got == 0.5).all()
    got, status = run_mm8(moe, a, sa, b, sb, "f32", [0, 10, 20, 64])  # the next call starts clean
    assert status == 0


@pytest.mark.parametrize("n", [128, 256])
def test_mm8_bounded_wait_reports(moe, monkeypatch, n):
    """A stage whose copies are never issued: the waits give up, the status says so, the context stays usable."""
    monkeypatch.setenv("MOE_TIMEOUT_MS", "50")
    g = np.random.default_rng(1)
    a, sa, b, sb = operands(g, 64, n, 256)
    _, status = run_mm8(moe, a, sa, b, sb, "f32", flags=moe.TEST_WITHHOLD)
    assert status == moe.ETIMEOUT
    monkeypatch.delenv("MOE_TIMEOUT_MS")
    ref, mag = ref8.mm8(a, sa, b, sb)
    got, status = run_mm8(moe, a, sa, b, sb, "f32")
    assert status == 0
    check_mm8(got, ref, mag, 256, "f32")


def test_mm8_empty(moe):
    g = np.random.default_rng(1)
    a, sa, b, sb = operands(g, 0, 64, 128)
    got, status = run_mm8(moe, a, sa, b, sb, "f32")
    assert got.shape == (0, 64) and status == 0


# ------------------------------------------------------------ experts8

def make_experts(g, e, h, i, whole=False):
    def w(rows, cols):
        if whole:
            q = g.choice(ref8.round_e4m3(np.arange(-2, 3)), size=(e, rows, cols))
            return q, g.integers(121, 123, size=(e, rows // 128, cols // 128)).astype(np.uint8)
        q = ref8.round_e4m3(np.clip(g.normal(size=(e, rows, cols)) * 100, -448, 448))
        return q, g.integers(113, 115, size=(e, rows // 128, cols // 128)).astype(np.uint8)
    gu, gus = w(2 * i, h)
    dn, dns = w(h, i)
    return gu, gus, dn, dns


def run_experts(m, ws, x, idx, w, out="bf16", stream=None):
    L = m.Layer8(*[cuda(v) for v in ws])
    t, h = x.shape
    o = torch.full((t, h), 9.0, dtype=dt(out), device="cuda")
    work = m.alloc_workspace(m.experts8_workspace(L, t, idx.shape[1]))
    work.fill_(0xA5)
    status = torch.full((1,), 99, dtype=torch.int32, device="cuda")
    m.experts8(L, x, cuda(idx.astype(np.int32)), cuda(w.astype(np.float32)), o, work, status)
    torch.cuda.synchronize()
    assert status.item() == 0, m.STATUS_NAMES.get(status.item())
    return f64(o)


EX = [  # t, H, I, E, k, x type, out type
    (1, 128, 128, 1, 1, "f32", "f32"), (1, 256, 128, 8, 2, "f32", "bf16"), (1, 2048, 768, 16, 8, "bf16", "bf16"),
    (3, 384, 256, 5, 5, "f32", "f32"), (4, 1024, 512, 40, 10, "f32", "bf16"), (8, 256, 384, 12, 4, "bf16", "f32"),
    (9, 256, 128, 8, 2, "f32", "f32"), (12, 384, 256, 64, 3, "f32", "bf16"), (40, 256, 256, 3, 2, "bf16", "bf16"),
    (150, 128, 128, 2, 1, "f32", "f32"), (2, 1152, 1152, 6, 2, "f32", "f32"), (8, 640, 128, 20, 8, "bf16", "bf16"),
    (7, 1408, 896, 9, 3, "f32", "bf16"), (8, 128, 512, 64, 32, "f32", "f32"),
    (2, 4096, 256, 40, 16, "f32", "f32"), (1, 6144, 128, 12, 12, "bf16", "f32"), (8, 512, 1024, 70, 9, "f32", "bf16"),
    (3, 256, 2048, 24, 8, "f32", "f32"),
]


@pytest.mark.parametrize("whole", [False, True])
@pytest.mark.parametrize("t,h,i,e,k,xd,od", EX)
def test_experts8(moe, t, h, i, e, k, xd, od, whole):
    """whole: x and the weights are small whole numbers, so that the first product is exact and the allowance, which
    otherwise adds the worst truncation of every step, is far below the result."""
    g = np.random.default_rng(t * 7 + h)
    ws = make_experts(g, e, h, i, whole)
    x = cuda((g.integers(-2, 3, size=(t, h)) if whole else g.normal(size=(t, h))).astype(np.float32)).to(dt(xd))
    idx = np.stack([g.choice(e, size=k, replace=False) for _ in range(t)])
    w = g.random(size=(t, k)).astype(np.float32)
    if t > 2:
        idx[1] = -1                 # a row without experts
        idx[2, 0] = e + 3           # another rank's expert
        if k > 1:
            idx[0, 1] = idx[0, 0]   # the same expert twice
    ref, allow = ref8.experts8(f64(x), *ws, idx, w, HALF[od], whole)
    got = run_experts(moe, ws, x, idx, w, od)
    bad = ~(np.abs(got - ref) <= allow)
    assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], ref[bad][:4], allow[bad][:4])
    if t > 2:
        assert (got[1] == 0).all()
    if whole:
        assert np.sqrt((allow ** 2).mean()) < 0.1 * np.sqrt((ref ** 2).mean())


def test_experts8_one_expert_gets_every_row(moe):
    g = np.random.default_rng(0)
    ws = make_experts(g, 4, 256, 128)
    x = cuda(g.normal(size=(260, 256)).astype(np.float32))
    idx, w = np.full((260, 2), 3), np.full((260, 2), 0.25, np.float32)
    ref, allow = ref8.experts8(f64(x), *ws, idx, w, HALF["f32"])
    assert (np.abs(run_experts(moe, ws, x, idx, w, "f32") - ref) <= allow).all()


def test_experts8_group_sizes_around_a_tile(moe):
    """Groups of every size at which a tile's token boxes, its columns or the number of tiles change."""
    g = np.random.default_rng(8)
    sizes = [1, 16, 17, 31, 32, 33, 80, 95, 96, 97, 103, 111, 112, 113, 127, 128, 129, 223, 224, 225]
    e, t = len(sizes), sum(sizes)
    ws = make_experts(g, e, 128, 128, whole=True)
    x = cuda(g.integers(-2, 3, size=(t, 128)).astype(np.float32))
    idx, w = g.permutation(np.repeat(np.arange(e), sizes))[:, None], np.ones((t, 1), np.float32)
    ref, allow = ref8.experts8(f64(x), *ws, idx, w, HALF["f32"], True)
    for _ in range(5):
        bad = (~(np.abs(run_experts(moe, ws, x, idx, w, "f32") - ref) <= allow)).any(1)
        assert not bad.any(), np.bincount(idx[bad, 0], minlength=e)


@pytest.mark.parametrize("shift", [118, -100])
@pytest.mark.parametrize("t", [4, 30])
def test_experts8_scales_that_cancel(moe, t, shift):
    """x times 2^shift through gate_up scales times 2^-shift: the same numbers, bit for bit."""
    g = np.random.default_rng(t)
    gu, gus, dn, dns = make_experts(g, 6, 256, 128)
    gus = gus + 10  # 123, 124
    x = g.normal(size=(t, 256)).astype(np.float32)
    idx, w = np.stack([g.choice(6, size=2, replace=False) for _ in range(t)]), g.random(size=(t, 2)).astype(np.float32)
    want = run_experts(moe, (gu, gus, dn, dns), cuda(x), idx, w, "f32")
    x2, gus2 = (x * np.float32(2.0) ** shift).astype(np.float32), (gus.astype(int) - shift).astype(np.uint8)
    got = run_experts(moe, (gu, gus2, dn, dns), cuda(x2), idx, w, "f32")
    assert np.isfinite(want).all() and np.array_equal(got, want)


@pytest.mark.parametrize("t", [5, 70])
def test_experts8_nan_row_stays_alone(moe, t):
    g = np.random.default_rng(t)
    ws = make_experts(g, 6, 256, 128)
    x = g.normal(size=(t, 256)).astype(np.float32)
    idx = np.stack([g.choice(6, size=2, replace=False) for _ in range(t)])
    w = g.random(size=(t, 2)).astype(np.float32)
    clean = run_experts(moe, ws, cuda(x), idx, w)
    x[2, 100], x[3, 7] = np.nan, np.inf
    got = run_experts(moe, ws, cuda(x), idx, w)
    assert np.isnan(got[2]).all() and np.isnan(got[3]).all()
    rest = [r for r in range(t) if r not in (2, 3)]
    assert np.array_equal(got[rest], clean[rest])


@pytest.mark.parametrize("t", [4, 40])
def test_experts8_nan_weights_stay_in_their_channels(moe, t):
    """A NaN weight of one expert: the rows that chose it become NaN (its channel's h is), a NaN in its down rows only
    that output; rows that did not choose it are as they were."""
    g = np.random.default_rng(t + 1)
    gu, gus, dn, dns = make_experts(g, 6, 256, 128)
    x = cuda(g.normal(size=(t, 256)).astype(np.float32))
    idx = np.stack([g.choice(5, size=2, replace=False) for _ in range(t)])
    idx[::2, 1] = 5
    w = g.random(size=(t, 2)).astype(np.float32) + 0.1
    clean = run_experts(moe, (gu, gus, dn, dns), x, idx, w)
    dn2 = dn.copy()
    dn2[5, 77, 100] = 0xFF
    got = run_experts(moe, (gu, gus, dn2, dns), x, idx, w)
    want = np.zeros(got.shape, bool)
    want[::2, 77] = True
    assert np.array_equal(np.isnan(got), want) and np.array_equal(got[~want], clean[~want])
    gu2 = gu.copy()
    gu2[5, 130, 3] = 0x7F
    got = run_experts(moe, (gu2, gus, dn, dns), x, idx, w)
    assert np.isnan(got[::2]).all() and np.array_equal(got[1::2], clean[1::2])


@pytest.mark.parametrize("t", [4, 300])
def test_route_quantise_experts_together(moe, t):
    """Router logits -> gate -> experts, and a dense product beside them, captured into two graphs that share a
    workspace and replayed in turn: every replay gives what the plain calls gave, bit for bit."""
    g = np.random.default_rng(t)
    e, k, h, i = 16, 4, 256, 128
    ws = make_experts(g, e, h, i)
    L = moe.Layer8(*[cuda(v) for v in ws])
    router = cuda(g.normal(size=(h, e)).astype(np.float32) / 16)
    bias = cuda((g.normal(size=e) * 0.05).astype(np.float32))
    proj = cuda(g.normal(size=(200, h)).astype(np.float32))
    pq, ps = torch.empty(200, h, dtype=torch.uint8, device="cuda"), torch.empty(2, 2, dtype=torch.uint8, device="cuda")
    moe.quant8(proj, pq, ps, block_rows=128)
    work = moe.alloc_workspace(moe.experts8_workspace(L, t, k))

    def buffers():
        z = lambda *s, d=torch.float32: torch.zeros(*s, dtype=d, device="cuda")  # noqa: E731
        return dict(x=z(t, h), idx=z(t, k, d=torch.int32), w=z(t, k), out=z(t, h), st=z(1, d=torch.int32),
                    q=z(t, h, d=torch.uint8), s=z(t, 4, d=torch.uint8), p=z(t, 200), st2=z(1, d=torch.int32))

    def step(b):
        moe.gate(b["x"] @ router, b["idx"], b["w"], bias=bias, score="sigmoid", n_groups=4, top_groups=2, group_top=2,
                 renorm=True, scale=1.5)
        moe.experts8(L, b["x"], b["idx"], b["w"], b["out"], work, b["st"])
        moe.quant8(b["x"], b["q"], b["s"][:, :2])
        moe.mm8(b["q"], b["s"][:, :2], pq, ps, b["p"], b["st2"])

    sets, graphs, want = [buffers(), buffers()], [], []
    for b in sets:
        b["x"].copy_(torch.from_numpy(g.normal(size=(t, h)).astype(np.float32)))
        step(b)
        torch.cuda.synchronize()
        assert b["st"].item() == 0 and b["st2"].item() == 0
        want.append({n: b[n].clone() for n in ("idx", "w", "out", "p")})
        ids, wt = ref8.gate(f64(b["x"] @ router), k, "sigmoid", f64(bias), 4, 2, 2, True, 1.5)
        assert np.array_equal(b["idx"].cpu().numpy(), ids)
        if t <= 8:
            ref, allow = ref8.experts8(f64(b["x"]), *ws, ids, b["w"].cpu().numpy(), HALF["f32"])
            assert (np.abs(f64(b["out"]) - ref) <= allow).all()
    side = torch.cuda.Stream()
    for b in sets:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=side):
            step(b)
        graphs.append(gr)
    for rep in range(3):
        for gr, b, w in zip(graphs, sets, want):
            for n in w:
                b[n].fill_(3)
            gr.replay()
        torch.cuda.synchronize()
        for b, w in zip(sets, want):
            for n in w:
                assert torch.equal(b[n], w[n]), n


def test_other_stream_and_repeated_calls(moe):
    """The calls run on the stream they are given; repeats give the same bits."""
    g = np.random.default_rng(4)
    e, k, h, i, t = 32, 4, 512, 256, 500
    L = moe.Layer8(*[cuda(v) for v in make_experts(g, e, h, i)])
    x = cuda(g.normal(size=(t, h)).astype(np.float32))
    idx = cuda(np.stack([g.choice(e, size=k, replace=False) for _ in range(t)]).astype(np.int32))
    w = cuda(g.random(size=(t, k)).astype(np.float32))
    work = moe.alloc_workspace(moe.experts8_workspace(L, t, k))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    outs = [torch.empty(t, h, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for o in outs[:2]:
        moe.experts8(L, x, idx, w, o, work, status, stream=s)
    with torch.cuda.stream(s):
        for o in outs[2:]:
            moe.experts8(L, x, idx, w, o, work, status)
    s.synchronize()
    assert status.item() == 0
    for o in outs[1:]:
        assert torch.equal(o, outs[0])


@pytest.mark.parametrize("t", [2, 30])
def test_captured_behind_other_work(moe, t):
    """In a graph: first, behind a copy, behind a fill, behind a kernel, where two streams join, behind itself; and the
    same calls without a graph.  Each must see what came before it."""
    g = np.random.default_rng(t)
    L = moe.Layer8(*[cuda(v) for v in make_experts(g, 6, 256, 128)])
    src = torch.randn(t, 256, device="cuda")
    idx = cuda(np.stack([g.choice(6, size=2, replace=False) for _ in range(t)]).astype(np.int32))
    w = torch.rand(t, 2, device="cuda")
    work = moe.alloc_workspace(moe.experts8_workspace(L, t, 2))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()

    def sequence(outs):
        call = lambda x, i: moe.experts8(L, x, idx, w, outs[i], work, status)  # noqa: E731
        x = outs[6]
        call(src, 0)
        x.copy_(src)
        call(x, 1)
        x.zero_()
        call(x, 2)
        torch.add(src, src, out=x)
        call(x, 3)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            x.mul_(0.5)
        torch.mul(src, 3.0, out=outs[7])
        torch.cuda.current_stream().wait_stream(side)
        call(x, 4)
        call(outs[4], 5)

    new = lambda: [torch.full((t, 256), 5.0, device="cuda") for _ in range(8)]  # noqa: E731
    plain = new()
    sequence(plain)
    torch.cuda.synchronize()
    outs = new()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sequence(outs)
    for _ in range(3):
        for o in outs:
            o.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, plain):
            assert torch.equal(a, b)
    assert torch.equal(plain[0], plain[1]) and torch.equal(plain[0], plain[4]) and (plain[2] == 0).all()
    assert not torch.equal(plain[3], plain[0]) and not torch.equal(plain[5], plain[4])
    assert status.item() == 0


@pytest.mark.parametrize("t", [4, 24, 2500])
def test_calls_behind_one_another_without_a_wait(moe, t):
    """A chain in which each call reads what the one before it writes, and one that overwrites what the one before it
    reads, over and over: as with a synchronisation after every call."""
    g = np.random.default_rng(17)
    h, i, e, k = 256, 128, 6, 2
    L = moe.Layer8(*[cuda(v) for v in make_experts(g, e, h, i)])
    router = cuda(ref8.round_e4m3(g.normal(size=(e, h)) * 50))
    rs = torch.full((1, h // 128), 118, dtype=torch.uint8, device="cuda")
    xs = [torch.randn(t, h, device="cuda") for _ in range(3)]

    def chain(wait):
        z = lambda *s, d=torch.float32: torch.zeros(*s, dtype=d, device="cuda")  # noqa: E731
        x, q, s, lg = z(t, h), z(t, h, d=torch.uint8), z(t, 4, d=torch.uint8)[:, : h // 128], z(t, e)
        idx, w, st, out = z(t, k, d=torch.int32), z(t, k), z(1, d=torch.int32), []
        work = moe.alloc_workspace(moe.experts8_workspace(L, t, k))
        y = z(t, h)
        done = torch.cuda.synchronize if wait else (lambda: None)
        for n in range(30):
            x.copy_(xs[n % 3])
            done()
            for _ in range(2):
                moe.quant8(x, q, s)
                done()
                moe.mm8(q, s, router, rs, lg, st)
                done()
                moe.gate(lg, idx, w, renorm=True)
                done()
                moe.experts8(L, x, idx, w, y, work, st)
                done()
                x.copy_(y)
                done()
            out.append((idx.clone(), y.clone()))
        torch.cuda.synchronize()
        assert st.item() == 0
        return out

    want, got = chain(True), chain(False)
    for (i0, y0), (i1, y1) in zip(want, got):
        assert torch.equal(i0, i1) and torch.equal(y0, y1)
    assert not torch.equal(want[0][1], want[1][1])


def test_calls_from_two_threads_and_streams(moe):
    """Calls of different sizes from two host threads on their own streams, with their own workspaces, at once."""
    import threading
    g = np.random.default_rng(6)
    e, h, i, k = 12, 512, 256, 3
    L = moe.Layer8(*[cuda(v) for v in make_experts(g, e, h, i)])
    work = []
    for t in (3, 40, 130, 700):
        x = cuda(g.normal(size=(t, h)).astype(np.float32))
        idx = cuda(np.stack([g.choice(e, size=k, replace=False) for _ in range(t)]).astype(np.int32))
        w = cuda(g.random(size=(t, k)).astype(np.float32))
        a, sa, b, sb = operands(g, t, 300, 768)
        work.append(dict(x=x, idx=idx, w=w, a=cuda(a), sa=padded(sa, 8, 255), b=cuda(b), sb=cuda(sb)))
    torch.cuda.synchronize()

    def run(out, order):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for n in order:
                d, t = work[n], work[n]["x"].shape[0]
                ws = moe.alloc_workspace(moe.experts8_workspace(L, t, k))
                o, p = torch.empty(t, h, device="cuda"), torch.empty(t, 300, device="cuda")
                st = torch.zeros(2, dtype=torch.int32, device="cuda")
                moe.experts8(L, d["x"], d["idx"], d["w"], o, ws, st[:1])
                moe.mm8(d["a"], d["sa"], d["b"], d["sb"], p, st[1:])
                out.append((n, o, p, st, ws))
        s.synchronize()

    ref = []
    run(ref, range(4))
    got = [[], []]
    threads = [threading.Thread(target=run, args=(got[0], [0, 3, 1, 2] * 10)),
               threading.Thread(target=run, args=(got[1], [2, 0, 3, 1] * 10))]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert [len(v) for v in got] == [40, 40]
    for n, o, p, st, _ in got[0] + got[1]:
        assert st.tolist() == [0, 0]
        assert torch.equal(o, ref[n][1]) and torch.equal(p, ref[n][2])


def test_a_single_row_of_any_stride(moe):
    """The stride of one row means nothing: a row of a transposed or odd view is taken."""
    g = np.random.default_rng(1)
    a, sa, b, sb = operands(g, 1, 40, 272)
    ref, mag = ref8.mm8(a, sa, b, sb)
    at = cuda(np.concatenate([a, a], 1)).as_strided((1, 272), (287, 1))
    st = cuda(np.concatenate([sa, sa], 1)).as_strided((1, 3), (4, 1))
    o = torch.zeros(1, 40, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    moe.mm8(at, st, cuda(b), cuda(sb), o, status)
    check_mm8(f64(o), ref, mag, 272, "f32")
    x = torch.randn(1, 300, device="cuda")
    want = run_quant(moe, x, 1)
    q, s = torch.zeros(1, 300, dtype=torch.uint8, device="cuda"), torch.zeros(1, 3, dtype=torch.uint8, device="cuda")
    moe.quant8(x.expand(5, 300)[:1], q.as_strided((1, 300), (1, 1)), s)
    assert np.array_equal(q.cpu().numpy(), want[0]) and np.array_equal(s.cpu().numpy(), want[1])


def test_binding_refusals(moe):
    z = lambda *s, d=torch.uint8: torch.zeros(*s, dtype=d, device="cuda")  # noqa: E731
    st = z(1, d=torch.int32)
    for bad in [dict(a=z(4, 128, d=torch.float32)), dict(sa=z(4, 3)), dict(b=z(64, 128).t()), dict(out=z(4, 65, d=torch.float32)),
                dict(sa=z(4, 2)[:, :1]), dict(out=z(64, 4, d=torch.float32).t()), dict(b=z(2, 64, 128)),
                dict(sa=z(16)[:13].as_strided((4, 1), (4, 1))[:, :1])]:
        args = dict(a=z(4, 128), sa=z(4, 4)[:, :1], b=z(64, 128), sb=z(1, 1), out=z(4, 64, d=torch.float32)) | bad
        if "sa" in bad and bad["sa"].shape == (4, 1) and bad["sa"].stride(0) == 4:
            args["sa"] = torch.zeros(13, dtype=torch.uint8, device="cuda").as_strided((4, 1), (4, 1))
        with pytest.raises(moe.MoeError):
            moe.mm8(args["a"], args["sa"], args["b"], args["sb"], args["out"], st)
    with pytest.raises(moe.MoeError):
        moe.gate(z(4, 8, d=torch.float32), z(4, 2, d=torch.int64), z(4, 2, d=torch.float32))
    with pytest.raises(moe.MoeError):
        moe.gate(z(4, 8, d=torch.float32), z(4, 2, d=torch.int32), z(4, 2, d=torch.float32), score="tanh")
    with pytest.raises(moe.MoeError):
        moe.quant8(z(4, 8, d=torch.float16), z(4, 8), z(4, 1))
    for offs in (z(1, d=torch.int32), z(1, 2, d=torch.int32), z(0, d=torch.int32)):
        with pytest.raises(moe.MoeError):
            moe.mm8(z(4, 128), z(4, 4)[:, :1], z(1, 64, 128), z(1, 1, 1), z(4, 64, d=torch.float32), st, offs=offs)
    L = moe.Layer8(z(2, 256, 128), z(2, 2, 1), z(2, 128, 128), z(2, 1, 1))
    with pytest.raises(moe.MoeError):
        moe.experts8(L, z(4, 128, d=torch.float32), z(8, d=torch.int32), z(8, d=torch.float32), z(4, 128, d=torch.float32),
                     moe.alloc_workspace(1 << 20), st)
    with pytest.raises(moe.MoeError):
        moe.Layer8(z(2, 256, 100), z(2, 2, 1), z(2, 100, 128), z(2, 1, 1))


# ------------------------------------------------------------ experts8: terms in 32 bits whatever the number of rows

@pytest.mark.parametrize("t,h,i,e,k", [(3, 256, 128, 8, 4), (8, 384, 256, 12, 4), (9, 256, 128, 8, 4), (40, 384, 256, 12, 6),
                                       (300, 256, 128, 16, 8), (1500, 640, 128, 30, 5)])
def test_experts8_rounds_the_sum_once(moe, t, h, i, e, k):
    """A bf16 output is the 32-bit one rounded once: the experts' terms are in 32 bits for few rows and for many."""
    g = np.random.default_rng(t)
    ws = make_experts(g, e, h, i)
    x = cuda(g.normal(size=(t, h)).astype(np.float32))
    idx, w = np.stack([g.choice(e, size=k, replace=False) for _ in range(t)]), g.random(size=(t, k)).astype(np.float32)
    whole = run_experts(moe, ws, x, idx, w, "f32")
    got = run_experts(moe, ws, x, idx, w, "bf16")
    assert np.array_equal(got, f64(torch.from_numpy(whole).float().bfloat16()))


# ------------------------------------------------------------ gate: bounds and ranges at their edges

@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("size", [2, 4, 8, 5])
@pytest.mark.parametrize("big", [16.0, 100.0, 1e4])
def test_gate_large_biases_that_cancel_in_a_group(moe, big, size, score):
    """A group's best two have biases big and -big (a forced expert beside one switched off): their scores carry the
    rounding of numbers as large as big, their sum is about 1.  Groups' sums some 1e-6 apart: the order is 64-bit
    arithmetic's."""
    g = np.random.default_rng(int(big) + size)
    groups, t = 8, 300
    bias = np.full((groups, size), -np.inf, np.float32)
    bias[:, 0], bias[:, 1] = big, -big
    bias[:, 2:] = np.where(g.random((groups, size - 2)) < 0.5, -np.inf, -3 * big)
    bias = g.permuted(bias, axis=1).reshape(-1)
    lg = (g.normal(size=(t, 1)) * 0.3 + g.normal(size=(t, groups * size)) * np.exp(g.normal(size=(t, 1))) * 1e-5).astype(np.float32)
    for top_groups, k in ((1, 1), (3, 4)):
        check_gate(moe, cuda(lg), k, cuda(bias), score=score, n_groups=groups, top_groups=top_groups, group_top=2, renorm=True)


def test_gate_group_sums_by_hand(moe):
    """Two groups of two, biases 1000 and -1000: sums 1.00004 and 1.00002 in 64 bits, 1.0 and 1.000061 in 32."""
    p = np.array([[0.50002, 0.50002, 0.50004, 0.49998]])
    bias = cuda(np.array([1000, -1000, 1000, -1000], np.float32))
    idx, _ = check_gate(moe, cuda(np.log(p / (1 - p)).astype(np.float32)), 1, bias, score="sigmoid", n_groups=2, group_top=2)
    assert idx.tolist() == [[0]]


@pytest.mark.parametrize("top_groups", [1, 2, 3, 4])
def test_gate_group_sums_past_32_bits(moe, top_groups):
    """Biases whose sums leave the 32-bit range on either side, beside a group that is masked throughout."""
    bias = np.array([-np.inf, -np.inf, -3e38, -3e38, 3e38, 2e38, 3e38, 3e38, -3e38, -2e38], np.float32)
    lg = np.random.default_rng(2).normal(size=(20, 10)).astype(np.float32)
    check_gate(moe, cuda(lg), 2 * top_groups, cuda(bias), score="sigmoid", n_groups=5, top_groups=top_groups, group_top=2)


# ------------------------------------------------------------ scales: the whole range of their sum

@pytest.mark.parametrize("ea,eb", [(65, 64), (126, 3), (3, 126), (-75, -75), (-123, -27), (-27, -123)])
@pytest.mark.parametrize("t", [3, 8, 13, 20, 70])
def test_mm8_scales_that_add_up_past_32_bits(moe, t, ea, eb):
    """Scales 2^ea and 2^eb whose product no 32-bit number holds (or only a rounded one), of operands that bring the
    result back: the same numbers times a power of two, bit for bit, and zeros stay zeros."""
    g = np.random.default_rng(t)
    a, sa, b, sb = operands(g, t, 140, 256, whole=True)  # values -2 .. 2, every sum exact
    a[0] = 0
    ref, _ = ref8.mm8(a, sa, b, sb)
    f = 2.0 ** (-7 if ea + eb > 0 else 7)
    a, b = ref8.round_e4m3(ref8.E4M3[a] * f), ref8.round_e4m3(ref8.E4M3[b] * f)
    sa, sb = np.minimum(sa, 127), np.minimum(sb, 127)
    ref, _ = ref8.mm8(a, sa, b, sb)
    ref = ref * 2.0 ** (ea + eb)
    assert np.abs(ref).max() < 2.0 ** 128 and np.array_equal(ref, ref.astype(np.float32))
    got, status = run_mm8(moe, a, (sa.astype(int) + ea).astype(np.uint8), b, (sb.astype(int) + eb).astype(np.uint8), "f32")
    assert status == 0 and np.array_equal(got, ref)


@pytest.mark.parametrize("t", [4, 30])
def test_experts8_blocks_of_zeros_under_large_scales(moe, t):
    """A block of weights that are zero adds nothing, whatever its scale and however large x or h is there."""
    g = np.random.default_rng(t)
    gu, gus, dn, dns = make_experts(g, 6, 256, 256)
    x = g.normal(size=(t, 256)).astype(np.float32)
    x[:, :128] *= np.float32(2.0) ** 118
    gu[:, :, :128], dn[:, :, :128] = 0, 0
    gus[:, :, 0], dns[:, :, 0] = 127, 127
    gus[:, 0, 1], gus[:, 2, 1] = 113 + 59, 113 + 59  # the first 128 channels of h: some 2^110
    idx, w = np.stack([g.choice(6, size=2, replace=False) for _ in range(t)]), g.random(size=(t, 2)).astype(np.float32)
    want = run_experts(moe, (gu, gus, dn, dns), cuda(x), idx, w, "f32")
    assert np.isfinite(want).all() and (want != 0).any()
    for big in (150, 254):
        gus2, dns2 = gus.copy(), dns.copy()
        gus2[:, :, 0] = big
        assert np.array_equal(run_experts(moe, (gu, gus2, dn, dns), cuda(x), idx, w, "f32"), want)
        dns2[:, :, 0] = big
        assert np.array_equal(run_experts(moe, (gu, gus, dn, dns2), cuda(x), idx, w, "f32"), want)


def test_experts8_one_workspace_for_every_smaller_batch(moe):
    """A workspace for the largest batch serves all smaller ones, where h is wider than x too."""
    g = np.random.default_rng(3)
    e, h, i, k = 10, 256, 768, 8
    L = moe.Layer8(*[cuda(v) for v in make_experts(g, e, h, i)])
    work = moe.alloc_workspace(moe.experts8_workspace(L, 9, k))
    x = cuda(g.normal(size=(9, h)).astype(np.float32))
    idx = cuda(np.stack([g.choice(e, size=k, replace=False) for _ in range(9)]).astype(np.int32))
    w = cuda(g.random(size=(9, k)).astype(np.float32))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for t in range(9, 0, -1):
        o = torch.empty(t, h, device="cuda")
        moe.experts8(L, x[:t], idx[:t], w[:t], o, work, status)
        assert status.item() == 0 and torch.isfinite(o).all()


@pytest.mark.parametrize("e,o", [(64, {}), (64, dict(n_groups=8, top_groups=3, group_top=2)), (300, dict(scale=2.0))])
def test_gate_softmax_runs_over_experts_a_bias_masks(moe, e, o):
    """A bias of -inf or NaN takes an expert out of the choice and of its group's score; the softmax still runs over
    every expert with a logit, so that an expert's weight does not depend on which others are switched off."""
    g = np.random.default_rng(e)
    lg = g.normal(size=(40, e)).astype(np.float32) * 2
    lg[:, 7] = -np.inf
    bias = (g.normal(size=e) * 0.1).astype(np.float32)
    bias[::5], bias[3::7] = -np.inf, np.nan
    idx, w = check_gate(moe, cuda(lg), 6, cuda(bias), **o)
    p = np.exp(lg.astype(np.float64))
    p /= p.sum(1, keepdims=True)
    assert np.abs(w / o.get("scale", 1.0) - np.take_along_axis(p, idx.astype(np.int64), 1)).max() <= 2.0 ** -19


# ------------------------------------------------------------ mm8: both sides of the few-row rule at large weights

@pytest.mark.parametrize("t,n,k", [(1, 8192, 4096), (8, 8192, 4096), (1, 8192, 4224), (8, 8320, 4096), (5, 2048, 16512), (16, 8192, 2048), (16, 4096, 4096), (16, 4096, 4224),
                                   (32, 2048, 2048), (32, 2048, 2064)])
def test_mm8_few_rows_of_large_weights(moe, t, n, k):
    g = np.random.default_rng(n + t)
    a, sa, b, sb = operands(g, t, n, k)
    got, status = run_mm8(moe, a, sa, b, sb, "f32")
    assert status == 0
    for r in (slice(0, 128), slice(n // 2 // 128 * 128, n // 2 // 128 * 128 + 128), slice(n - 128, n)):
        ref, mag = ref8.mm8(a, sa, b[r], sb[r.start // 128: -(-r.stop // 128)])
        check_mm8(got[:, r], ref, mag, k, "f32")
