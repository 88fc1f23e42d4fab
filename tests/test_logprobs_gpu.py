"""GPU parity of moe_logprobs against a plain 64-bit implementation.

Ids: equal (ties to the lowest).  Log probabilities: the bound of the 32-bit sum over the row (refblock.logprobs) and three
roundings of the result.  Entropy: the sum's bound twice, relative to it and absolute."""
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


def run(m, x, tokens, k, scale=1.0, stream=None):
    t = x.shape[0]
    tk = torch.from_numpy(np.ascontiguousarray(tokens.astype(np.int32))).cuda()
    lp = torch.full(tokens.shape, 7.0, device="cuda")
    ent = torch.full((t,), 7.0, device="cuda")
    idx = torch.full((t, k), 77, dtype=torch.int32, device="cuda") if k else None
    tl = torch.full((t, k), 7.0, device="cuda") if k else None
    m.logprobs(x, tokens=tk, logp=lp, entropy=ent, top_idx=idx, top_logp=tl, scale=scale, stream=stream)
    torch.cuda.synchronize()
    return [None if a is None else a.cpu().numpy() for a in (lp, ent, idx, tl)]


def compare(got, x, tokens, k, scale):
    lp, ent, idx, tl = got
    rlp, rent, ridx, rtl, dz = rb.logprobs(x.double().cpu().numpy(), tokens, k, scale)
    rb.check(lp, rlp, dz + np.abs(np.nan_to_num(rlp)) * 3 * rb.U, "f32", "logp")
    rb.check(ent, rent, (2 + 2 * rent) * dz[:, 0], "f32", "entropy")
    if k:
        assert np.array_equal(idx, ridx), np.argwhere(idx != ridx)[:4]
        rb.check(tl, rtl, dz + np.abs(np.nan_to_num(rtl)) * 3 * rb.U, "f32", "top")


def logits(a, dtype, ld=None, shift=0):
    x = torch.from_numpy(np.ascontiguousarray(a.astype(np.float32))).cuda().to(dtype)
    t, v = x.shape
    ld = ld or v
    buf = torch.full((t * ld + shift,), 1e30, dtype=dtype, device="cuda")
    view = buf[shift:].view(t, ld)[:, :v]
    view.copy_(x)
    return view


CASES = [  # t, v, m, k, ld past v, first element
    (1, 1, 1, 1, 0, 0), (3, 2, 2, 2, 0, 0), (5, 33, 3, 32, 0, 0), (2, 1000, 1, 5, 0, 0), (7, 1001, 4, 20, 0, 0), (1, 4096, 1, 0, 0, 0),
    (4, 8191, 8, 8, 3, 1), (2, 20000, 2, 31, 0, 3), (1, 131072, 1, 20, 0, 0), (2, 100003, 3, 32, 0, 0), (3, 131071, 2, 1, 1, 5),
    (160, 30001, 1, 7, 0, 0), (400, 5000, 2, 10, 0, 0), (40, 65537, 2, 3, 0, 0), (1, 1 << 20, 2, 9, 0, 0), (1, 40000, 700, 4, 0, 0),
    (2000, 300, 1, 3, 0, 0),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("t,v,m,k,pad,shift", CASES, ids=[f"{c[0]}x{c[1]}k{c[3]}" for c in CASES])
def test_logprobs(moe, t, v, m, k, pad, shift, dtype):
    g = np.random.default_rng(v + t)
    a = g.normal(size=(t, v)) * np.exp(g.normal(size=(t, 1)))
    x = logits(a, torch.float32 if dtype == "f32" else torch.bfloat16, v + pad, shift)
    tokens = g.integers(-2, v + 2, size=(t, m))
    tokens[:, 0] = a.argmax(1)
    for scale in (1.0, 0.3, 7.0):
        compare(run(moe, x, tokens, k, scale), x, tokens, k, scale)


@pytest.mark.parametrize("v", [37, 5000, 70001])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_special_rows(moe, v, dtype):
    """Masks, infinities, NaN, the type's lowest value, equal and ordered rows, far apart logits."""
    g = np.random.default_rng(9)
    low = -3.3895313892515355e38 if dtype == "bf16" else -3.4028234663852886e38
    a = g.normal(size=(20, v))
    a[0] = -np.inf
    a[1] = np.nan
    a[2] = 1.25                           # every value a tie
    a[3] = np.sort(a[3])                  # every value above those before it
    a[4] = np.sort(a[4])[::-1]
    a[5] = low                            # a mask of the lowest value that leaves nothing
    a[6, 3:] = low
    a[7, 3:] = -np.inf                    # fewer values than alternatives
    a[8, ::2] = np.nan
    a[9, 11] = np.inf
    a[10, [5, 30]] = np.inf
    a[11] = np.where(g.random(v) < 0.5, -0.0, 0.0)
    a[12] *= 1e4
    a[13] = a[13] * 1e-3 + 5000
    a[14] = a[14] * 1e-3 - 5000
    a[15, 0] = 90.0
    a[16] = a[16] * 1e37
    a[17, v - 1] = 300.0
    a[18] = low
    a[18, v // 2] = 3.0
    a[19] = np.round(a[19])               # many ties
    x = logits(a, torch.float32 if dtype == "f32" else torch.bfloat16)
    tokens = np.stack([np.arange(20) % v, np.full(20, v - 1), np.full(20, 30), np.full(20, v)], 1)
    for k, scale in ((32, 1.0), (1, 0.5), (6, 1.0), (0, 1.0)):
        compare(run(moe, x, tokens, k, scale), x, tokens, k, scale)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_long_lists_of_candidates(moe, dtype):
    """Rows whose order makes the threshold rise as slowly as it can, through every way that the list is cut."""
    v = 60000
    n = np.arange(v)
    rows = [n / 1000.0, n // 7 / 100.0, (n % 4096) / 100.0 + n // 4096, np.where(n % 3 == 0, n / 100.0, -5.0), -(n % 16384) / 50.0,
            np.where(n < 50000, -1.0, 1.0), np.where(n < 16384, -3.0, (n % 5000) / 10.0)]
    x = logits(np.stack(rows * 30), torch.float32 if dtype == "f32" else torch.bfloat16)
    tokens = np.full((x.shape[0], 1), v - 1)
    for part in (x, x[:7], x[:1], x[1:2]):  # a block a row, and several
        for k in (32, 1):
            compare(run(moe, part, tokens[: part.shape[0]], k), part, tokens[: part.shape[0]], k, 1.0)


def test_parts_streams_graphs_and_repeats(moe):
    """Each output by itself, the same bits on every call, on another stream and from a graph."""
    g = np.random.default_rng(3)
    x = logits(g.normal(size=(9, 50000)) * 2, torch.bfloat16)
    tokens = g.integers(0, 50000, size=(9, 3))
    lp, ent, idx, tl = run(moe, x, tokens, 12)
    ids = torch.from_numpy(tokens.astype(np.int32)).cuda()
    a, b = torch.empty(9, 3, device="cuda"), torch.empty(9, device="cuda")
    c, d = torch.empty(9, 12, dtype=torch.int32, device="cuda"), torch.empty(9, 12, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    moe.logprobs(x, tokens=ids, logp=a, stream=side)
    moe.logprobs(x, entropy=b, stream=side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.logprobs(x, top_idx=c, top_logp=d)
        moe.logprobs(x, tokens=ids, logp=a, entropy=b)
    graph.replay()
    torch.cuda.synchronize()
    assert np.array_equal(a.cpu().numpy(), lp) and np.array_equal(b.cpu().numpy(), ent)
    assert np.array_equal(c.cpu().numpy(), idx) and np.array_equal(d.cpu().numpy(), tl)
    e = torch.empty(0, 7, device="cuda")
    moe.logprobs(e, entropy=torch.empty(0, device="cuda"))


def test_far_rows(moe):
    """Offsets past 32 bits: the last of 80000 rows of 60000."""
    x = torch.zeros(80000, 60000, dtype=torch.bfloat16, device="cuda")
    x[-1, 59999] = 20
    ent = torch.empty(80000, device="cuda")
    idx = torch.empty(80000, 2, dtype=torch.int32, device="cuda")
    tl = torch.empty(80000, 2, device="cuda")
    moe.logprobs(x, entropy=ent, top_idx=idx, top_logp=tl)
    assert idx[-1].tolist() == [59999, 0] and (idx[:-1] == torch.tensor([0, 1], device="cuda", dtype=torch.int32)).all()
    assert (ent[:-1] - np.log(60000)).abs().max() < 1e-4
