"""moe_mm16's fp32 results to their last bits, at every kernel's sizes, with all that the epilogue does.

A weight row's terms have one sign, so no partial sum is larger than the product z, and the tensor cores lose less than 2^-23 of
z at each of the ceil(k / 16) steps; ten roundings are allowed for halves, warps or CTAs added up.  Then the bias, the activation
(refblock.act_bound; its slope is 1.2 at most), the product of a gated pair, row scale and residual, a rounding each.  At k = 2048
that is 1.6e-5 of the result."""
import math

import numpy as np
import pytest

import refblock as rb
from test_mm16_gpu import moe, run  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ACTS = {"none": lambda z: z, "relu": lambda z: z.clamp(min=0), "silu": lambda z: z * torch.sigmoid(z),
        "gelu": lambda z: z * 0.5 * torch.special.erfc(-z * math.sqrt(0.5)), "sigmoid": torch.sigmoid,
        "gelu_tanh": lambda z: z * torch.sigmoid(math.sqrt(8 / math.pi) * (z + 0.044715 * z ** 3))}


@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("t,n,k", [(1, 512, 2048), (5, 130, 2047), (16, 200, 1000), (16, 4000, 72), (64, 512, 2048), (333, 1001, 2008),
                                   (120, 264, 4096), (700, 1200, 2048), (700, 1201, 2048), (2300, 1296, 1000), (260, 5008, 512),
                                   (100, 10016, 264), (1500, 1200, 8192)], ids=lambda v: str(v))
def test_results_to_their_last_bits(moe, t, n, k, gated, act):  # noqa: F811
    g = torch.Generator(device="cuda")
    g.manual_seed(t + n + k)
    rnd = lambda *s: torch.rand(*s, device="cuda", generator=g)  # noqa: E731
    rows, ld = 2 * n if gated else n, -(-k // 8) * 8
    a = (rnd(t, ld) * 0.5 + 0.5).bfloat16()[:, :k]
    size = torch.where(rnd(rows, 1) < 0.5, -1.0, 1.0) * torch.exp2(4 * rnd(rows, 1) - 1) / k  # z from 0.3 to 7
    b = ((rnd(rows, ld) * 0.5 + 0.5) * size).bfloat16()[:, :k]
    bias, scale, res = rnd(rows) - 0.5, rnd(t) * 2 - 1, (rnd(t, n) - 0.5)
    for parts in ((), ("bias", "scale", "f32"), ("bias", "bf16")):
        z = a.double() @ b.double().T
        dz = (-(-k // 16) + 10) * 2.0 ** -23 * z.abs()
        if "bias" in parts:
            z = z + bias.double()
            dz = dz + z.abs() * rb.U
        x, dx = z[:, :n], dz[:, :n]
        h = ACTS[act](x)
        own = torch.from_numpy(np.ascontiguousarray(rb.act_bound(act, x.cpu().numpy(), h.cpu().numpy()))).cuda()
        dh = dx * 1.2 + own
        if gated:
            u, du = z[:, n:], dz[:, n:]
            h, dh = h * u, dh * u.abs() + h.abs() * du + dh * du + (h * u).abs() * rb.U
        if "scale" in parts:
            h, dh = h * scale.double()[:, None], dh * scale.double().abs()[:, None] + (h * scale[:, None]).abs() * rb.U
        r = None
        if "f32" in parts or "bf16" in parts:
            r = res if "f32" in parts else res.bfloat16()
            h = h + r.double()
            dh = dh + h.abs() * rb.U
        out = run(moe, a, b, act=act, gated=gated, bias=bias if "bias" in parts else None, row_scale=scale if "scale" in parts else None,
                  res=r).double()
        room = dh * (1 + 2.0 ** -20) + h.abs() * rb.U + 2.0 ** -149
        bad = (out - h).abs() > room
        assert not bad.any(), (parts, ((out - h).abs() / room).max().item(), bad.nonzero()[:3].tolist())
