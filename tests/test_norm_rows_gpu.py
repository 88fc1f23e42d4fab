"""moe_norm and moe_add_norm: what a row gives is its own, whatever lies beside it, and rows of far apart values."""
import numpy as np
import pytest

import ref8
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


@pytest.mark.parametrize("out", ["f32", "bf16", "e4m3"])
@pytest.mark.parametrize("h", [64, 257, 2048, 4090])
def test_values_far_below_a_rows_largest(moe, h, out):  # noqa: F811
    """Rows whose squares leave the 32-bit range and whose values run over all of it: the small ones keep their bits."""
    g = np.random.default_rng(h)
    t = 16
    a = np.sign(g.normal(size=(t, h))) * 10.0 ** g.uniform(-37, 19, size=(t, h))
    for r in range(t):
        a[r, r] = 10.0 ** (19 + 1.2 * r)
    x = cuda(a.astype(np.float32))
    w = cuda((10.0 ** g.uniform(-1, 20, size=h)).astype(np.float32))  # (the largest are the first ones: no product overflows)
    w[:t] = 1
    for weight in (None, w):
        o, s = outputs(t, h, out)
        moe.norm(x, o, w=weight, scales=s)
        torch.cuda.synchronize()
        # the norm, and its product with the weight, are numbers of 32 bits each: below 2^-126 they have a step of 2^-149 and
        # may be off by half of it, the first times w
        ref = rb.norm(f64(x), None if weight is None else f64(weight))
        bound = np.abs(ref) * (rb.NORM + 4) * rb.U + (1 + (0 if weight is None else f64(weight))) * 2.0 ** -150
        if out != "e4m3":
            rb.check(f64(o), ref, bound, out)
            continue
        # half a step: 2^-4 of the value, or 2^-10 of the scale; blocks of numbers from 2^-100 on have the least scale
        step = np.repeat(np.exp2(s.cpu().numpy().astype(np.float64) - 127), 128, 1)[:, :h]
        got = ref8.E4M3[o.cpu().numpy()] * step
        assert (np.abs(got - ref) <= bound * 1.1 + np.maximum(np.abs(ref) * 2.0 ** -4, step * 2.0 ** -10)).all()
        for at in range(0, h, 128):
            top = np.abs(ref[:, at:at + 128]).max(1)
            use = top / step[:, at]
            assert (use <= 448 * 1.001).all() and ((use > 224 * 0.999) | (top < 2.0 ** -100)).all()
