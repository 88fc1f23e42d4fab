"""GPU parity of moe_mm16 against a plain 64-bit implementation.

Tolerances: refblock.mm16 (sums, activations) and half a step of the output.  Inputs that are small whole numbers, whose
every partial sum 32 bits hold, have to come out exactly; so have products that are zero."""
import os
import threading

import numpy as np
import pytest

import refblock as rb

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from quantized_routed_expert_fn_gb300 import build, moe as m
    build.build()
    m.lib()
    return m


def f64(t):
    return t.double().cpu().numpy()


def rows16(a, pad=0):
    """bf16 rows that start on 16 bytes, NaN between them."""
    r, c = a.shape
    ld = -(-c // 8) * 8 + pad
    wide = torch.full((r, ld), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, :c] = torch.from_numpy(np.ascontiguousarray(a.astype(np.float32))).cuda().bfloat16()
    return wide[:, :c]


def run(m, a, b, kind="f32", pad=0, res=None, flags=0, expect=0, **kw):
    t, n = a.shape[0], b.shape[0] // (2 if kw.get("gated") else 1)
    out = torch.full((t + 1, n + pad), 7.0, dtype=TYPES[kind], device="cuda")
    st = torch.full((1,), 55, dtype=torch.int32, device="cuda")
    m.mm16(a, b, out[:t, :n], st, residual=res, flags=flags, **kw)
    torch.cuda.synchronize()
    assert st.item() == expect
    assert (out[t] == 7).all() and (out[:, n:] == 7).all()
    return out[:t, :n]


def whole(g, shape, top=3):
    return g.integers(-top, top + 1, size=shape).astype(np.float64)


SIZES = [  # t, n, k
    (1, 1, 1), (1, 512, 2048), (3, 17, 65), (8, 128, 64), (5, 130, 2048), (9, 100, 40), (9, 128, 2048), (16, 256, 64), (33, 512, 2048),
    (31, 40, 8200), (64, 1000, 130), (100, 2048, 512), (128, 64, 128), (129, 128, 129), (200, 300, 72), (257, 257, 257), (333, 1001, 2008),
    (700, 129, 64), (1000, 513, 100), (513, 2000, 320), (2, 4000, 1000), (7, 20001, 72), (2050, 256, 64), (1500, 1100, 192), (40, 9000, 64),
]


@pytest.mark.parametrize("t,n,k", SIZES, ids=["x".join(map(str, s)) for s in SIZES])
def test_whole_numbers_are_exact(moe, t, n, k):
    """Every size, plain and gated, both output types: the exact product (of 32-bit results)."""
    g = np.random.default_rng(t * 31 + n * 7 + k)
    a = whole(g, (t, k))
    for gated in (False, True):
        b = whole(g, (2 * n if gated else n, k), 2)
        z = a @ b.T
        ref = np.maximum(z[:, :n], 0) * (z[:, n:] if gated else 1)
        at, bt = rows16(a), rows16(b, 8)
        got = f64(run(moe, at, bt, pad=3, act="relu", gated=gated))
        if np.abs(ref).max() < 2 ** 24:
            assert np.array_equal(got, ref), np.argwhere(got != ref)[:5].tolist()
        got16 = f64(run(moe, at, bt, "bf16", act="relu", gated=gated))
        assert np.array_equal(got16, f64(torch.from_numpy(got).bfloat16()))


EPI = [dict(), dict(act="silu", gated=True), dict(act="gelu", bias=True, res="bf16"), dict(act="gelu_tanh", gated=True, bias=True, scale=True),
       dict(act="sigmoid", scale=True, res="f32"), dict(bias=True, scale=True, res="bf16", gated=True), dict(act="relu", res="f32")]


@pytest.mark.parametrize("res", [None, "f32", "bf16"])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("t,n,k", [(2300, 1296, 136), (1300, 2000, 64), (3100, 784, 72), (260, 5008, 40), (700, 1200, 5000), (300, 4000, 8200),
                                   (20000, 48, 64), (9000, 160, 200), (333, 1008, 4160)], ids=lambda v: str(v))
def test_large_tiles_are_exact(moe, t, n, k, gated, kind, res):
    """Several tiles a block, whole rows, residuals by pieces, k in two halves: exact products of whole numbers, on the GPU."""
    g = torch.Generator(device="cuda")
    g.manual_seed(t + n)
    whole = lambda *s: torch.randint(-2, 3, s, device="cuda", generator=g).float()  # noqa: E731
    a, b = whole(t, k), whole(2 * n if gated else n, k)
    r = None if res is None else whole(t, n).to(TYPES[res])
    bias, scale = whole(b.shape[0]), whole(t)
    z = a @ b.T + bias  # sums below 2^24: exact
    ref = torch.relu(z[:, :n]).double() * (z[:, n:] if gated else 1) * scale[:, None] + (0 if r is None else r)
    out = run(moe, a.bfloat16(), b.bfloat16(), kind, res=r, act="relu", gated=gated, bias=bias, row_scale=scale)
    if kind == "f32":
        fine = ref.abs() < 2 ** 24  # (products of the two halves may be larger: rounded once or twice)
        assert torch.equal(out.double()[fine], ref[fine])
        assert ((out.double() - ref).abs() <= ref.abs() * 2.0 ** -23).all()
    else:
        assert ((out.double() - ref).abs() <= ref.abs() * (2.0 ** -8 + 2.0 ** -22)).all()
        small = ref.abs() <= 256
        assert torch.equal(out.double()[small], ref[small])


@pytest.mark.parametrize("res", [None, "f32", "bf16"])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("t,n,k", [(100, 4992, 72), (128, 8192, 64), (17, 10240, 40), (64, 10256, 136), (101, 14336, 64), (128, 20000, 48)],
                         ids=lambda v: str(v))
def test_gated_wide_products_of_few_rows(moe, t, n, k, kind, res):
    """One tile of tokens and many columns, whose tiles have to end where the next begins: exact products of whole numbers."""
    test_large_tiles_are_exact(moe, t, n, k, True, kind, res)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("t,n,k", [(1, 96, 256), (7, 513, 2048), (20, 200, 520), (150, 264, 1024), (300, 1001, 200), (1100, 640, 96)],
                         ids=lambda v: str(v))
@pytest.mark.parametrize("o", EPI, ids=range(len(EPI)))
def test_epilogues(moe, o, t, n, k, kind):
    g = np.random.default_rng(n + t)
    gated = o.get("gated", False)
    rows = 2 * n if gated else n
    for pad in (0, 1):
        a, b = rows16(g.normal(size=(t, k))), rows16(g.normal(size=(rows, k)) * 1.5 * k ** -0.5)
        bias = torch.from_numpy(g.normal(size=rows).astype(np.float32)).cuda() if o.get("bias") else None
        scale = torch.from_numpy(g.normal(size=t).astype(np.float32)).cuda() if o.get("scale") else None
        res = None
        if o.get("res"):
            res = torch.from_numpy(g.normal(size=(t, n + pad)).astype(np.float32)).cuda().to(TYPES[o["res"]])[:, :n]
        out = run(moe, a, b, kind, pad=pad, res=res, act=o.get("act", "none"), gated=gated, bias=bias, row_scale=scale)
        arr = lambda x: None if x is None else f64(x)  # noqa: E731
        ref, bound = rb.mm16(f64(a), f64(b), gated, o.get("act", "none"), arr(bias), arr(scale), arr(res))
        rb.check(f64(out), ref, bound, kind, pad)


@pytest.mark.parametrize("act", ["none", "silu", "gelu", "gelu_tanh", "relu", "sigmoid"])
def test_activations_over_their_range(moe, act):
    """One-term products whose z runs over the type's range, infinities and NaN among them."""
    z = np.concatenate([np.linspace(-30, 30, 241), [0.0, 1e-30, -1e-30, 1e30, -1e30, 3e38, -3e38, np.inf, -np.inf, np.nan, 88, -88, 100, -100, 200]])
    a, b = rows16(z[:, None]), rows16(np.ones((1, 1)))
    for t in (a.shape[0], 5):
        for at in range(0, a.shape[0] - t + 1, t):
            x = a[at:at + t].contiguous() if t > 8 else rows16(f64(a[at:at + t]))
            got = f64(run(moe, rows16(f64(x)), b, act=act))
            with np.errstate(all="ignore"):
                zx = f64(x)
                ref = rb.act(act, zx)
                # z is exact here: only the activation's own error counts, and that of factors below the normal numbers
                own = rb.act_bound(act, zx, ref) + np.abs(zx) * 2.0 ** -146 + 2.0 ** -146
                rb.check(got, ref, np.nan_to_num(own, nan=0.0, posinf=0.0), "f32")


@pytest.mark.parametrize("t", [3, 24, 100, 600])
def test_rows_do_not_touch_one_another(moe, t):
    """A row or a weight row of NaN or infinities spoils its own outputs only; what a row gives does not depend on the others."""
    g = np.random.default_rng(6)
    n, k = 300, 200
    a, b = whole(g, (t, k)), whole(g, (n, k))
    ref = a @ b.T
    a2, b2 = a.copy(), b.copy()
    a2[1] = np.nan
    b2[7, 3] = np.inf
    got = f64(run(moe, rows16(a2), rows16(b2)))
    keep = np.ones((t, n), bool)
    keep[1], keep[:, 7] = False, False
    assert np.array_equal(got[keep], ref[keep])
    assert np.isnan(got[1]).all() and not np.isfinite(got[:, 7]).any()


def test_in_place_residual(moe):
    """The shared expert added to the experts' output where it stands, at every kernel's sizes."""
    g = np.random.default_rng(8)
    for t, n, k, kind in ((4, 256, 128, "f32"), (40, 256, 512, "bf16"), (700, 520, 64, "f32"), (700, 513, 64, "bf16")):
        a, b = rows16(whole(g, (t, k))), rows16(whole(g, (n, k)))
        out = torch.from_numpy(whole(g, (t, n))).cuda().to(TYPES[kind])
        before, st = f64(out), torch.zeros(1, dtype=torch.int32, device="cuda")
        moe.mm16(a, b, out, st, residual=out)
        want = torch.from_numpy(before + f64(a) @ f64(b).T).to(TYPES[kind]).double().numpy()
        assert np.array_equal(f64(out), want) and st.item() == 0


def test_repeats_streams_graphs_and_threads(moe):
    """The same bits on every call: another stream, a replayed graph, two threads at once."""
    g = np.random.default_rng(9)
    for t, n, k in ((4, 512, 2048), (64, 512, 2048), (900, 1024, 512)):
        a, b = rows16(g.normal(size=(t, k))), rows16(g.normal(size=(n, k)))
        ref = run(moe, a, b, "bf16", act="silu")
        bufs = [torch.empty(t, n, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
        sts = [torch.zeros(1, dtype=torch.int32, device="cuda") for _ in range(4)]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        moe.mm16(a, b, bufs[0], sts[0], act="silu", stream=side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _ in range(3):
                moe.mm16(a, b, bufs[1], sts[1], act="silu")
        graph.replay()
        graph.replay()
        workers = [threading.Thread(target=lambda i=i: [moe.mm16(a, b, bufs[i], sts[i], act="silu") for _ in range(5)]) for i in (2, 3)]
        [w.start() for w in workers]
        [w.join() for w in workers]
        torch.cuda.synchronize()
        for o, s in zip(bufs, sts):
            assert torch.equal(o, ref) and s.item() == 0


@pytest.mark.parametrize("t,n", [(2, 64), (40, 128), (300, 1024)])
def test_a_wait_that_runs_out_is_reported(moe, t, n):
    g = np.random.default_rng(1)
    a, b = rows16(g.normal(size=(t, 512))), rows16(g.normal(size=(n, 512)))
    old = os.environ.get("MOE_TIMEOUT_MS")
    os.environ["MOE_TIMEOUT_MS"] = "20"
    try:
        out, st = torch.empty(t, n, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
        moe.mm16(a, b, out, st, flags=moe.TEST_WITHHOLD)
        torch.cuda.synchronize()
        assert st.item() == moe.ETIMEOUT
    finally:
        os.environ.pop("MOE_TIMEOUT_MS") if old is None else os.environ.__setitem__("MOE_TIMEOUT_MS", old)
    run(moe, a, b)  # the next call is well


def test_empty_and_far(moe):
    """No rows zero the status; weights past 32-bit offsets: the last of 1.1 million rows of 2048."""
    st = torch.full((1,), 9, dtype=torch.int32, device="cuda")
    moe.mm16(torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(8, 64, dtype=torch.bfloat16, device="cuda"),
             torch.empty(0, 8, device="cuda"), st)
    assert st.item() == 0
    n, k = 1_100_000, 2048
    b = torch.zeros(n, k, dtype=torch.bfloat16, device="cuda")
    b[-1] = 1
    for t in (2, 40, 300):
        a = torch.ones(t, k, dtype=torch.bfloat16, device="cuda")
        out = torch.empty(t, n, dtype=torch.bfloat16, device="cuda")
        moe.mm16(a, b, out, st)
        assert (out[:, -1] == k).all() and (out[:, :-1] == 0).all() and st.item() == 0
