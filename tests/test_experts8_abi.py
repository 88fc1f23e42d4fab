"""Host-side checks of the 8-bit experts' entry points: bad arguments are refused before any CUDA call."""
import ctypes

import numpy as np
import pytest

import ref8
from quantized_routed_expert_fn_gb300 import build


@pytest.fixture(scope="module")
def m():
    build.build()
    from quantized_routed_expert_fn_gb300 import moe
    moe.lib()
    return moe


A, B, C, D, O, W, S = 0x100000, 0x200000, 0x300000, 0x400000, 0x10000000, 0x20000000, 0x30000000


def _gate(m, t=4, dtype=0, ld=64, logits=A, idx=B, w=C, bias=None, **over):
    cfg = dict(n_experts=64, top_k=4, score=0, n_groups=1, top_groups=1, group_top=1, flags=0, scale=1.0) | over
    return m.lib().moe_gate(m.MoeGateCfg(*cfg.values()), logits, dtype, ld, bias, t, idx, w, None)


@pytest.mark.parametrize("over,code", [
    (dict(n_experts=0), -2), (dict(n_experts=1025, ld=1025), -2), (dict(top_k=0), -2), (dict(top_k=33), -2),
    (dict(score=2), -1), (dict(flags=2), -1), (dict(scale=float("inf")), -1), (dict(scale=float("nan")), -1),
    (dict(n_groups=0), -2), (dict(n_groups=3), -2), (dict(n_groups=64, top_groups=1), -2),
    (dict(n_groups=8, top_groups=9), -2), (dict(n_groups=8, top_groups=0), -2), (dict(group_top=3), -2),
    (dict(n_groups=32, top_groups=1, top_k=3), -2), (dict(dtype=2), -1), (dict(t=-1), -1), (dict(ld=63), -2),
    (dict(logits=None), -1), (dict(idx=None), -1), (dict(w=None), -1), (dict(logits=A + 2), -3), (dict(idx=B + 2), -3),
    (dict(bias=D + 1), -3), (dict(idx=A), -1), (dict(w=B), -1),
    (dict(bias=B), -1), (dict(t=(1 << 30) + 1), -1),
])
def test_gate_refusals(m, over, code):
    assert _gate(m, **over) == code, m.last_error()
    assert m.last_error()


def test_empty_calls_need_no_pointers(m):
    assert _gate(m, t=0, logits=None, idx=None, w=None) == 0
    assert m.lib().moe_quant8(None, 0, 128, 0, 128, 1, None, 128, None, 1, None) == 0


def _quant(m, x=A, dtype=0, ldx=256, rows=4, cols=256, br=1, q=O, ldq=256, s=S, lds=2):
    return m.lib().moe_quant8(x, dtype, ldx, rows, cols, br, q, ldq, s, lds, None)


@pytest.mark.parametrize("over,code", [
    (dict(dtype=7), -1), (dict(br=64), -2), (dict(rows=-1), -2), (dict(cols=0), -2), (dict(x=None), -1),
    (dict(q=None), -1), (dict(s=None), -1), (dict(ldx=255), -2), (dict(ldq=255), -2), (dict(lds=1), -2),
    (dict(x=A + 2), -3), (dict(q=A), -1), (dict(s=A + 16), -1), (dict(s=O), -1),
    (dict(rows=128 * 65535 + 1, br=128, ldx=256), -2), (dict(rows=(1 << 30) + 1), -2), (dict(cols=(1 << 30) + 1), -2),
])
def test_quant8_refusals(m, over, code):
    assert _quant(m, **over) == code, m.last_error()


def _mm8(m, a=A, lda=256, sa=B, lds=4, t=64, b=C, sb=D, n=128, k=256, out=O, dt=0, ldo=128, offs=None, g=0, flags=0, st=S):
    return m.lib().moe_mm8(a, lda, sa, lds, t, b, sb, n, k, out, dt, ldo, offs, g, flags, st, None)


@pytest.mark.parametrize("over,code", [
    (dict(dt=2), -1), (dict(flags=1), -1), (dict(t=-1), -2), (dict(n=0), -2), (dict(k=0), -2), (dict(k=24), -2),
    (dict(offs=W), -1), (dict(g=4), -1), (dict(offs=W, g=1025), -1), (dict(offs=W, g=-1), -1), (dict(st=None), -1),
    (dict(a=None), -1), (dict(sa=None), -1), (dict(b=None), -1), (dict(sb=None), -1), (dict(out=None), -1),
    (dict(lda=240), -2), (dict(lds=0), -2), (dict(ldo=127), -2), (dict(a=A + 8), -3), (dict(lda=264), -3),
    (dict(b=C + 4), -3), (dict(sa=B + 1), -3), (dict(lds=6), -3), (dict(out=O + 2), -3), (dict(offs=W + 2, g=2), -3),
    (dict(out=A + 64), -1), (dict(out=C), -1), (dict(out=D - 16), -1), (dict(n=1 << 22, g=1024, offs=W, ldo=1 << 22), -2),
    (dict(t=(1 << 30) + 1), -2),
])
def test_mm8_refusals(m, over, code):
    assert _mm8(m, **over) == code, m.last_error()


def _layer(m, **over):
    return m.MoeLayer8(*(dict(hidden=256, n_experts=8, inter=128, gu=A, gus=B, dn=C, dns=D) | over).values())


def _ex(m, L=None, x=O, xd=0, t=4, idx=W, w=W + 4096, k=2, out=O + (1 << 20), od=0, work=S, wb=1 << 24, st=S - 256):
    return m.lib().moe_experts8(L if L is not None else _layer(m), x, xd, t, idx, w, k, out, od, work, wb, st, None)


@pytest.mark.parametrize("layer,code", [
    (dict(hidden=0), -2), (dict(hidden=192), -2), (dict(hidden=16512), -2), (dict(inter=64), -2), (dict(inter=0), -2),
    (dict(n_experts=0), -2), (dict(n_experts=1025), -2), (dict(gu=None), -1), (dict(gus=None), -1), (dict(dn=None), -1),
    (dict(dns=None), -1), (dict(gu=A + 8), -3), (dict(dn=C + 1), -3),
])
def test_experts8_refuses_bad_layers(m, layer, code):
    assert _ex(m, _layer(m, **layer)) == code, m.last_error()


@pytest.mark.parametrize("over,code", [
    (dict(xd=2), -1), (dict(od=5), -1), (dict(t=-1), -1), (dict(t=(1 << 20) + 1), -1), (dict(k=0), -2), (dict(k=33), -2),
    (dict(x=None), -1), (dict(idx=None), -1), (dict(w=None), -1), (dict(out=None), -1), (dict(work=None), -1),
    (dict(st=None), -1), (dict(x=O + 4), -3), (dict(out=O + (1 << 20) + 8), -3), (dict(idx=W + 1), -3),
    (dict(work=S + 16), -3), (dict(wb=16), -7), (dict(out=O + 64), -1), (dict(out=W), -1),
    (dict(work=O), -1), (dict(x=S), -1),
    # out or work in the layer's weights (8 x 256 x 256 and 8 x 256 x 128 bytes) or scales (32 and 16 bytes)
    (dict(out=A + (1 << 19) - 64), -1), (dict(out=B + 16), -1), (dict(out=C + (1 << 18) - 64), -1), (dict(out=D), -1),
    (dict(work=A + 4096), -1), (dict(work=C), -1), (dict(work=D), -1),
])
def test_experts8_refuses_bad_calls(m, over, code):
    assert _ex(m, **over) == code, m.last_error()


def test_experts8_workspace(m):
    L = _layer(m)
    ws = m.lib().moe_experts8_workspace
    small, large = ws(L, 8, 2), ws(L, 9, 2)
    assert 0 < small < large < ws(L, 4096, 2)
    assert ws(L, 0, 2) > 0
    assert ws(L, -1, 2) == 0 and ws(L, 4, 33) == 0 and ws(_layer(m, hidden=100), 4, 2) == 0
    assert ctypes.sizeof(m.MoeLayer8) == 48


@pytest.mark.parametrize("st,code", [
    (S + 2, -3), (S - 1, -3), (O, -1), (O + 64 * 128 * 4 - 4, -1), (A + 16, -1), (B + 4, -1), (C + 128, -1), (D, -1), (W + 8, -1),
])
def test_mm8_refuses_a_status_in_another_buffer(m, st, code):
    """A misaligned status, or one within out (64 x 128 floats), a, sa, b, sb or the offsets, is refused on the host."""
    assert _mm8(m, st=st, offs=W, g=2) == code, m.last_error()


@pytest.mark.parametrize("st,code", [
    (S - 254, -3), (S - 255, -3), (S + 64, -1), (O + 16, -1), (O + (1 << 20) + 4092, -1), (W + 4, -1), (W + 4096 + 28, -1),
    (A + 1024, -1), (B + 28, -1), (C, -1), (D + 12, -1),
])
def test_experts8_refuses_a_status_in_another_buffer(m, st, code):
    """The same for work, x, out (4 x 256 floats), the ids and weights (4 x 2 words) and the layer's four buffers."""
    assert _ex(m, st=st) == code, m.last_error()
    if code == -3:
        assert _ex(m, st=st, t=0) == code


@pytest.mark.parametrize("k", [1, 8, 32])
@pytest.mark.parametrize("h,i", [(256, 768), (1024, 2048), (128, 16384), (2048, 512), (16384, 128), (4096, 2048)])
def test_experts8_workspace_does_not_fall_with_rows(m, h, i, k):
    """A workspace for the largest batch serves every smaller one (few rows have buffers of their own)."""
    ws = [m.lib().moe_experts8_workspace(_layer(m, hidden=h, inter=i), t, k) for t in list(range(40)) + [100, 4096]]
    assert ws[0] > 0 and all(a <= b for a, b in zip(ws, ws[1:]))


def test_python_binding_refuses_host_tensors(m):
    torch = pytest.importorskip("torch")
    x = torch.zeros(2, 128)
    q, s = torch.empty(2, 128, dtype=torch.uint8), torch.empty(2, 1, dtype=torch.uint8)
    with pytest.raises(m.MoeError):
        m.quant8(x, q, s)
    with pytest.raises(m.MoeError):
        m.gate(x, torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, 2))


# ---- the tests' own reference

def test_reference_e4m3_table():
    assert ref8.E4M3[0x7E] == 448 and ref8.E4M3[0x01] == 2.0 ** -9 and ref8.E4M3[0x38] == 1.0 and np.isnan(ref8.E4M3[0x7F])
    finite = [b for b in range(256) if (b & 127) != 127]
    assert np.array_equal(ref8.round_e4m3(ref8.E4M3[finite]), np.array(finite, np.uint8))
    # ties to the even code: 1 + 1/16 lies between 0x38 and 0x39, 1 + 3/16 between 0x39 and 0x3a
    assert list(ref8.round_e4m3([1.0625, 1.1875, 2.0 ** -10, 3 * 2.0 ** -10, np.inf, np.nan])) == [0x38, 0x3A, 0x00, 0x02, 0x7F, 0x7F]


def test_reference_scale_exponent():
    assert ref8.scale_exponent(448.0) == 0 and ref8.scale_exponent(448.1) == 1 and ref8.scale_exponent(224.0) == -1
    assert ref8.scale_exponent(0.0) == 0 and ref8.scale_exponent(1e-45) == -127


def test_reference_gate_by_hand():
    lg = np.array([[0.0, 1.0, 1.0, -np.inf]])
    idx, w = ref8.gate(lg, 2, renorm=True)
    assert idx.tolist() == [[1, 2]] and np.allclose(w, 0.5)
    idx, w = ref8.gate(lg, 2, score="sigmoid", bias=np.array([1.0, 0, 0, 9.0]))
    assert idx.tolist() == [[0, 1]] and np.allclose(w, [[0.5, 1 / (1 + np.exp(-1.0))]])
    idx, w = ref8.gate(lg, 3, groups=2, top_groups=1, group_top=2)
    assert idx.tolist() == [[1, 0, -1]] and w[0, 2] == 0


def test_reference_gate_softmax_runs_over_experts_a_bias_masks():
    """The bias moves no p: an expert that it masks is not chosen, but its logit stays in the softmax."""
    lg = np.log(np.array([[1.0, 2.0, 3.0, 4.0]]))
    idx, w = ref8.gate(lg, 2, bias=np.array([0.0, 0.0, 0.0, -np.inf]))
    assert idx.tolist() == [[2, 1]] and np.allclose(w, [[0.3, 0.2]])
    idx, w = ref8.gate(np.log(np.array([[1.0, 2.0, 3.0, 1e-300]])) + [[0, 0, 0, -np.inf]], 2)
    assert idx.tolist() == [[2, 1]] and np.allclose(w, [[0.5, 1 / 3]])
