"""moe_norm and moe_add_norm: what a row gives is its own, whatever lies beside it."""
import numpy as np
import pytest

import refblock as rb
from test_norm_gpu import cuda, f64, moe, outputs  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("out", ["f32", "bf16", "e4m3"])
@pytest.mark.parametrize("h", [1, 16, 64, 200, 257, 512])
def test_neighbours_do_not_change_a_row(moe, h, out):  # noqa: F811
    """The bits of ordinary rows alone, among ordinary ones, and beside rows of 1e30, NaN and infinities (several rows a warp)."""
    g = np.random.default_rng(h)
    t = 64
    plain = g.normal(size=(t, h)).astype(np.float32)
    far = plain.copy()
    far[1::5] *= 1e30
    far[2::5, h // 2] = np.nan
    far[3::5, 0] = np.inf
    for pad in (0, 5):
        got = []
        for a in (plain, far):
            o, s = outputs(t, h, out)
            moe.norm(cuda(a, "f32", pad), o, scales=s)
            r, _ = outputs(t, h, out)
            ro = torch.empty(t, h, device="cuda")
            moe.add_norm(cuda(a, "f32", pad), cuda(plain * 2, "f32", pad), ro, post=True, out=r, scales=None if s is None else torch.empty_like(s))
            got.append([x.clone() for x in (o, r, ro)])
        torch.cuda.synchronize()
        for a, b in zip(*got):
            for keep in (0, 4):
                assert torch.equal(a[keep::5], b[keep::5])
    one, s1 = outputs(1, h, out)
    moe.norm(cuda(plain[:1]), one, scales=s1)
    o, s = outputs(t, h, out)
    moe.norm(cuda(plain), o, scales=s)
    assert torch.equal(o[:1], one)
