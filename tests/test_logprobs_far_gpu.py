"""moe_logprobs where logits or their scaled values are large: masks between 1e9 and 1e35 in size over nearly all of a row,
rows of large offsets, scales up to the limit.  Bounds as in test_logprobs_gpu: the 32-bit sum over the row
(refblock.logprobs) and three roundings of the result; the ids are equal."""
import numpy as np
import pytest

import refblock as rb
from test_logprobs_gpu import logits, moe, run  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def check_rows(m, a, dtype, tokens, ks, scale, copies):
    """The rows by themselves in groups (several blocks a row where it is long), and `copies` times over (one block)."""
    x = logits(a, TYPES[dtype])
    x64 = x.double().cpu().numpy()
    for k in ks:
        rlp, rent, ridx, rtl, dz = rb.logprobs(x64, tokens, k, scale)
        t = len(a)
        for lo, hi, n in ((0, t, 1), (0, 3, 1), (t - 1, t, 1), (0, t, copies)):
            lp, ent, idx, tl = run(m, x[lo:hi].repeat(n, 1), np.tile(tokens[lo:hi], (n, 1)), k, scale)
            part = lambda r: np.tile(r[lo:hi], (n,) + (1,) * (r.ndim - 1))  # noqa: E731
            d = part(dz)
            rb.check(lp, part(rlp), d + np.abs(np.nan_to_num(part(rlp))) * 3 * rb.U, "f32", "logp")
            rb.check(ent, part(rent), (2 + 2 * part(rent)) * d[:, 0], "f32", "entropy")
            if k:
                assert np.array_equal(idx, part(ridx)), np.argwhere(idx != part(ridx))[:4]
                rb.check(tl, part(rtl), d + np.abs(np.nan_to_num(part(rtl))) * 3 * rb.U, "f32", "top")


MASKS = [-1e9, -4e9, -5e9, -1e10, -1e11, -1e12, -1e15, -1e20, -1e24, -1e29, -6e29, -1e30, -1e35]


@pytest.mark.parametrize("v,copies", [(300, 40), (5000, 40), (70001, 12)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_finite_masks(moe, v, copies, dtype):  # noqa: F811
    """All tokens masked by one value, all but one, all but a short run, half of them."""
    g = np.random.default_rng(v)
    rows, tokens = [], []
    for mask in MASKS:
        for left in (0, 1, 50, v // 2):
            a = np.full(v, mask)
            at = int(g.integers(0, v - left + 1)) if left < v // 2 else 0
            keep = np.arange(at, at + left) if left < v // 2 else g.permutation(v)[:left]
            a[keep] = g.normal(size=left) * 2
            rows.append(a)
            tokens.append([keep[0] if left else 0, v - 1, int(g.integers(0, v))])
    check_rows(moe, np.stack(rows), dtype, np.array(tokens), (32, 1), 1.0, copies)


@pytest.mark.parametrize("v,copies", [(300, 40), (40000, 20)])
@pytest.mark.parametrize("scale", [1.0, 1e3, 1e6, 1e-4])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_large_offsets_and_scales(moe, v, copies, scale, dtype):  # noqa: F811
    """Rows around a large value, with ties; rows whose values rise through the sizes where the sums' reference changes its
    form (2^20 powers of two: 726817 at scale 1); logits up to 1e5 under scales of 1e3 and 1e6."""
    g = np.random.default_rng(int(v + scale))
    spread = lambda mid, s: mid + s * g.normal(size=v)  # noqa: E731
    rows = [np.full(v, 6.55e9), np.full(v, -6.55e9), np.full(v, 1e15), spread(5e9, 3e3), spread(1e15, 3e8), spread(1e5, 1.0),
            np.sort(spread(1e5, 2.0 / scale)), np.sort(spread(726817.0 / scale, 4.0 / scale)), np.sort(spread(726817.0 / scale, 4.0 / scale))[::-1],
            np.sort(spread(-726817.0 / scale, 4.0 / scale)), spread(726817.0 / scale, 30.0 / scale), spread(0, 1e5), np.round(spread(0, 1e5)),
            np.round(spread(3e4, 2)), spread(0, 2 / scale), g.permutation(np.where(np.arange(v) % 2, 726800.0, 726830.0) / scale)]
    a = np.stack(rows)
    tokens = np.stack([a.argmax(1), np.full(len(a), v // 3), np.full(len(a), v - 1)], 1)
    check_rows(moe, a, dtype, tokens, (20, 0), scale, copies)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_differences_past_the_range(moe, dtype):  # noqa: F811
    """Logits whose difference no 32-bit number holds, under a scale that brings it back: ln p is a number."""
    g = np.random.default_rng(5)
    a = np.stack([np.where(g.random(3000) < 0.5, -3e38, 3e38), np.where(np.arange(3000) == 77, 3e38, -3e38)])
    tokens = np.array([[0, 1, 2], [77, 5, 6]])
    check_rows(moe, a, dtype, tokens, (8,), 1e-38, 20)
