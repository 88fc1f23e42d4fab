"""moe_mm16 of long k: sums of one sign, whose losses add up, against 64 bits, and exact products of whole numbers.

Tolerances: the tensor cores cut off less than 2^-23 of a sum at every step of 16; a sum of theirs has 256 steps at most (bf16
outputs: 2048), and what they are added up with rounds to nearest: 2^-24 for each of a tile's sums, eight warps or CTAs and
the two halves.  Inputs are positive, so every partial sum is below the result."""
import numpy as np
import pytest

from test_mm16_gpu import moe, run, test_large_tiles_are_exact as large_tiles  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def product64(a, b, part=1 << 14):
    z = 0
    for i in range(0, a.shape[1], part):
        z = z + a[:, i:i + part].double() @ b[:, i:i + part].double().T
    return z


SAME_SIGN = [  # t, n, k, gated, type, row padding of the output
    (1, 64, 1 << 18, False, "f32", 0), (8, 100, 70001, False, "f32", 0), (16, 40, 40000, True, "f32", 0),       # few rows
    (40, 256, 1 << 18, False, "f32", 0), (300, 256, 70001, False, "f32", 0), (64, 200, 40000, True, "f32", 1),  # k split over a cluster
    (2100, 1024, 20000, False, "f32", 1), (10000, 100, 9001, False, "f32", 1), (1100, 700, 30000, True, "f32", 1),
    (1300, 1024, 65536, False, "f32", 0), (100, 10016, 20000, False, "f32", 0), (700, 1024, 20008, True, "f32", 0),
    (2048, 2048, 4096, False, "f32", 0), (2048, 2048, 8192, False, "f32", 0),
    (40, 256, 1 << 20, False, "bf16", 0), (1300, 1024, 1 << 19, False, "bf16", 0), (1300, 1000, 40000, False, "bf16", 1),
]


@pytest.mark.parametrize("t,n,k,gated,kind,pad", SAME_SIGN, ids=["x".join(map(str, c[:3])) + c[4] for c in SAME_SIGN])
def test_sums_of_one_sign(moe, t, n, k, gated, kind, pad):  # noqa: F811
    g = torch.Generator(device="cuda")
    g.manual_seed(t + k)
    ld = -(-k // 8) * 8
    a, b = ((torch.rand(r, ld, device="cuda", generator=g) * 0.5 + 0.5).bfloat16()[:, :k] for r in (t, 2 * n if gated else n))
    z = product64(a, b)
    out = run(moe, a, b, kind, pad=pad, gated=gated).double()
    steps, half = (256, 2.0 ** -24) if kind == "f32" else (2048, 2.0 ** -8)
    loss = min(steps, -(-k // 16)) * 2.0 ** -23 + (k / (16 * steps) + 20) * 2.0 ** -24
    if gated:
        z, loss = z[:, :n] * z[:, n:], 2 * loss + loss * loss + 2.0 ** -24
    worst = ((out - z).abs() / z).max().item()
    assert worst <= loss + half, (worst, loss, half)


@pytest.mark.parametrize("res", [None, "f32", "bf16"])
@pytest.mark.parametrize("kind,k", [("f32", 9001), ("f32", 20000), ("bf16", 33000), ("bf16", 70001)], ids=lambda v: str(v))
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("t,n", [(1300, 1200), (700, 1201), (100, 10016), (10000, 96), (2500, 264)], ids=lambda v: str(v))
def test_long_products_are_exact(moe, t, n, k, kind, gated, res):  # noqa: F811
    """Tiles of several sums, of every form: whole numbers."""
    k = -(-k // 8) * 8
    large_tiles(moe, t, n, k, gated, kind, res)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("t,n,k", [(3, 70, 50000), (16, 100, 70000), (33, 300, 70000), (120, 512, 280000), (300, 130, 40000)], ids=lambda v: str(v))
def test_long_products_of_few_rows_are_exact(moe, t, n, k, kind):  # noqa: F811
    for gated in (False, True):
        large_tiles(moe, t, n, k, gated, kind, "f32")


def test_long_sums_repeat(moe):  # noqa: F811
    """The same bits on every call, in a chain of calls and from a graph."""
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    for t, n, k in ((1500, 1024, 12000), (64, 512, 70000), (5, 512, 70000)):
        a, b = (torch.randn(r, k, device="cuda", generator=g).bfloat16() for r in (t, n))
        ref = run(moe, a, b)
        out, st = torch.empty(t, n, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _ in range(3):
                moe.mm16(a, b, out, st)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref) and st.item() == 0
        assert np.isfinite(ref.sum().item())
