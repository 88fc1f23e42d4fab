"""Host-side checks of the operators around the experts' step: bad arguments are refused before any CUDA call."""
import ctypes

import numpy as np
import pytest

import refblock
from quantized_routed_expert_fn_gb300 import build


@pytest.fixture(scope="module")
def m():
    build.build()
    from quantized_routed_expert_fn_gb300 import moe
    moe.lib()
    return moe


X, Y, O, P, W, G, S = 0x100000, 0x200000, 0x300000, 0x400000, 0x500000, 0x600000, 0x700000
INF, NAN = float("inf"), float("nan")


def _norm(m, x=X, xd=0, ldx=256, w=W, eps=1e-6, t=4, h=256, out=O, od=0, ldo=256, s=None, lds=0):
    return m.lib().moe_norm(x, xd, ldx, w, eps, t, h, out, od, ldo, s, lds, None)


@pytest.mark.parametrize("over,code", [
    (dict(xd=2), -1), (dict(xd=3), -1), (dict(od=3), -1), (dict(od=-1), -1), (dict(t=-1), -2), (dict(t=(1 << 30) + 1), -2),
    (dict(h=0), -2), (dict(h=32769, ldx=32769, ldo=32769), -2), (dict(eps=0.0), -1), (dict(eps=-1.0), -1), (dict(eps=INF), -1),
    (dict(eps=NAN), -1), (dict(eps=1e-60), -1), (dict(x=None), -1), (dict(out=None), -1), (dict(ldx=255), -2), (dict(ldx=0), -2),
    (dict(ldo=255), -2), (dict(ldx=1 << 40), -2), (dict(x=X + 2), -3), (dict(out=O + 1), -3), (dict(w=W + 2), -3),
    (dict(out=X + 16), -1), (dict(out=X, od=1), -1), (dict(out=X, ldo=257, ldx=256), -1), (dict(out=W), -1),
    (dict(s=S, lds=2), -1), (dict(od=2), -1), (dict(od=2, s=S, lds=1), -2), (dict(od=2, s=O + 8, lds=2), -1),
    (dict(od=2, s=X + 8, lds=2), -1), (dict(od=2, s=W, lds=2), -1), (dict(od=2, s=S, lds=2, out=X), -1),
])
def test_norm_refusals(m, over, code):
    assert _norm(m, **over) == code, m.last_error()
    assert m.last_error()


def _cfg(m, **over):
    c = dict(flags=0, eps=1e-6, scale=1.0, res_scale=1.0, w_post=None, w=W, gate=None, ldg=0, gate_dtype=0, gate_cols=1) | over
    return m.MoeAddNormCfg(*c.values())


def _add(m, cfg=None, y=Y, yd=0, ldy=256, r=X, rd=0, ldr=256, ro=P, rod=0, ldro=256, t=4, h=256, out=O, od=0, ldo=256, s=None, lds=0, **c):
    cfg = cfg or _cfg(m, **c)
    return m.lib().moe_add_norm(cfg, y, yd, ldy, r, rd, ldr, ro, rod, ldro, t, h, out, od, ldo, s, lds, None)


@pytest.mark.parametrize("over,code", [
    (dict(yd=2), -1), (dict(rd=2), -1), (dict(rod=2), -1), (dict(od=3), -1), (dict(flags=4), -1), (dict(scale=INF), -1),
    (dict(res_scale=NAN), -1), (dict(eps=0.0), -1), (dict(t=-1), -2), (dict(h=0), -2), (dict(w_post=G), -1),
    (dict(gate=G, gate_dtype=2), -1), (dict(gate=G, gate_cols=2), -2), (dict(gate=G, gate_cols=256, ldg=255), -2),
    (dict(gate=G + 2), -3), (dict(w=W + 1), -3), (dict(flags=1, w_post=G + 1), -3), (dict(y=None), -1), (dict(r=None), -1),
    (dict(ro=None), -1), (dict(ldy=255), -2), (dict(ldr=1), -2), (dict(ldro=0), -2), (dict(y=Y + 1), -3), (dict(r=X + 3), -3),
    (dict(ro=P + 2), -3), (dict(ro=X + 4), -1), (dict(ro=X, rod=1), -1), (dict(ro=Y + 1024), -1), (dict(ro=W), -1),
    (dict(ro=G, gate=G), -1), (dict(ro=G, gate=G, gate_cols=256, ldg=256), -1), (dict(out=P), -1), (dict(out=X), -1),
    (dict(out=Y, od=1), -1), (dict(out=Y + 16), -1), (dict(out=W), -1), (dict(out=None, s=S, lds=2), -1), (dict(od=2), -1),
    (dict(od=2, s=P, lds=2), -1), (dict(od=2, s=Y, lds=2), -1), (dict(od=2, s=S, lds=1), -2),
])
def test_add_norm_refusals(m, over, code):
    assert _add(m, **over) == code, m.last_error()


def test_empty_norms_need_no_pointers(m):
    assert _norm(m, t=0, x=None, out=None, w=None) == 0
    assert _add(m, t=0, y=None, r=None, ro=None, out=None) == 0
    assert m.lib().moe_add_norm(None, Y, 0, 1, X, 0, 1, P, 0, 1, 0, 1, None, 0, 1, None, 0, None) == -1
    assert ctypes.sizeof(m.MoeAddNormCfg) == 56


def test_e4m3_is_an_output_of_norms_only(m):
    """The type's number is refused everywhere else, as any unknown type."""
    assert m.lib().moe_quant8(X, 2, 256, 4, 256, 1, O, 256, S, 2, None) == -1


def test_bindings_refuse(m):
    torch = pytest.importorskip("torch")
    x = torch.zeros(2, 128)
    with pytest.raises(m.MoeError):
        m.norm(x, x)
    with pytest.raises(m.MoeError):
        m.norm(x[0], x[0])
    with pytest.raises(m.MoeError):
        m.add_norm(x, x, x)


# ---- the tests' own reference

def test_reference_norms_by_hand():
    x = np.array([[3.0, 4.0]])
    assert np.allclose(refblock.norm(x, np.array([1.0, 2.0]), 1e-30), [[3 / 12.5 ** 0.5, 8 / 12.5 ** 0.5]])
    s, _, n, _ = refblock.add_norm(x, np.array([[1.0, -4.0]]), gate=np.array([[0.0]]), sig=True, scale=2.0, res_scale=0.5)
    assert np.allclose(s, [[3.5, 2.0]]) and np.allclose(n, refblock.norm(s))


def test_reference_activations_by_hand():
    z = np.array([-2.0, 0.0, 3.0])
    assert np.allclose(refblock.act("silu", z), z / (1 + np.exp(-z)))
    assert np.allclose(refblock.act("gelu", z), [-0.04550026389635842, 0, 2.99595030634], atol=1e-9)
    assert np.allclose(refblock.act("gelu_tanh", z), 0.5 * z * (1 + np.tanh((2 / np.pi) ** 0.5 * (z + 0.044715 * z ** 3))))
    assert np.allclose(refblock.act("relu", z), [0, 0, 3]) and np.allclose(refblock.act("sigmoid", z), 1 / (1 + np.exp(-z)))


def _lp(m, x=X, xd=0, ld=1000, t=4, v=1000, scale=1.0, tok=Y, n=2, lp=O, ent=P, idx=W, tl=G, k=8):
    return m.lib().moe_logprobs(x, xd, ld, t, v, scale, tok, n, lp, ent, idx, tl, k, None)


@pytest.mark.parametrize("over,code", [
    (dict(xd=2), -1), (dict(t=-1), -2), (dict(t=(1 << 27) + 1), -2), (dict(v=0), -2), (dict(v=(1 << 24) + 1, ld=1 << 25), -2),
    (dict(scale=0.0), -1), (dict(scale=-1.0), -1), (dict(scale=NAN), -1), (dict(scale=INF), -1), (dict(scale=2e6), -1),
    (dict(n=-1), -2), (dict(n=1025), -2), (dict(k=33), -2), (dict(k=-1), -2), (dict(v=4, k=5), -2), (dict(x=None), -1),
    (dict(tok=None), -1), (dict(lp=None), -1), (dict(n=0), -1), (dict(idx=None), -1), (dict(tl=None), -1), (dict(k=0), -1),
    (dict(n=0, tok=None, lp=None, k=0, idx=None, tl=None, ent=None), -1), (dict(ld=999), -2), (dict(x=X + 2), -3), (dict(tok=Y + 2), -3),
    (dict(ent=P + 1), -3), (dict(lp=X + 64), -1), (dict(ent=Y), -1), (dict(idx=O), -1), (dict(tl=W), -1), (dict(ent=G + 4), -1),
])
def test_logprobs_refusals(m, over, code):
    assert _lp(m, **over) == code, m.last_error()


def test_empty_logprobs_need_no_pointers(m):
    assert _lp(m, t=0, x=None, tok=None, lp=None, idx=None, tl=None) == 0


def test_reference_logprobs_by_hand():
    x = np.log(np.array([[1.0, 2.0, 2.0, 5.0]]))
    lp, ent, idx, tl, _ = refblock.logprobs(x, np.array([[0, 3, 4, -1]]), 3)
    assert np.allclose(lp[0, :2], np.log([0.1, 0.5])) and np.isneginf(lp[0, 2:]).all()
    assert np.allclose(ent, -sum(p * np.log(p) for p in (0.1, 0.2, 0.2, 0.5)))
    assert idx.tolist() == [[3, 1, 2]] and np.allclose(tl, np.log([[0.5, 0.2, 0.2]]))
    lp, ent, idx, tl, _ = refblock.logprobs(np.array([[np.nan, -np.inf]]), np.array([[0]]), 2)
    assert np.isneginf(lp).all() and ent[0] == 0 and idx.tolist() == [[-1, -1]]


A, B2, RES, ST = 0x1000000, 0x2000000, 0x3000000, 0x4000000


def _mm(m, a=A, lda=256, t=64, b=B2, ldb=256, n=128, k=256, out=O, od=0, ldo=128, flags=0, st=ST, epi=True, **e):
    ep = m.MoeEpilogue(*(dict(act=0, res_dtype=0, bias=None, row_scale=None, residual=None, ldr=128) | e).values()) if epi else None
    return m.lib().moe_mm16(a, lda, t, b, ldb, n, k, ep, out, od, ldo, flags, st, None)


@pytest.mark.parametrize("over,code", [
    (dict(od=2), -1), (dict(flags=2), -1), (dict(act=6), -1), (dict(t=-1), -2), (dict(n=0), -2), (dict(k=0), -2), (dict(k=(1 << 24) + 1), -2),
    (dict(t=(1 << 30) + 1), -2), (dict(n=1 << 30, flags=1), -2), (dict(t=1 << 30, n=1 << 20, ldo=1 << 20), -2), (dict(residual=RES, res_dtype=2), -1),
    (dict(st=None), -1), (dict(st=ST + 2), -3), (dict(a=None), -1), (dict(b=None), -1), (dict(out=None), -1), (dict(lda=248), -2),
    (dict(ldb=0), -2), (dict(ldo=127), -2), (dict(residual=RES, ldr=127), -2), (dict(a=A + 8), -3), (dict(b=B2 + 2), -3), (dict(lda=260), -3),
    (dict(ldb=257), -3), (dict(out=O + 2), -3), (dict(residual=RES + 1), -3), (dict(bias=W + 1), -3), (dict(row_scale=W + 2), -3),
    (dict(out=A + 64), -1), (dict(out=B2), -1), (dict(bias=O + 4), -1), (dict(row_scale=O), -1), (dict(residual=O + 512), -1),
    (dict(residual=O, res_dtype=1), -1), (dict(residual=O, ldr=136), -1), (dict(st=A + 8), -1), (dict(st=B2 + 4), -1), (dict(st=O), -1),
    (dict(st=RES + 4, residual=RES), -1), (dict(st=W + 4, bias=W), -1), (dict(st=W + 8, row_scale=W), -1), (dict(flags=1, st=B2 + 65536 + 8), -1),
])
def test_mm16_refusals(m, over, code):
    assert _mm(m, **over) == code, m.last_error()


def test_mm16_struct_and_bindings(m):
    assert ctypes.sizeof(m.MoeEpilogue) == 40
    assert _mm(m, epi=False, k=0) == -2
    torch = pytest.importorskip("torch")
    x = torch.zeros(2, 128, dtype=torch.bfloat16)
    with pytest.raises(m.MoeError):
        m.mm16(x, x, torch.zeros(2, 2), torch.zeros(1, dtype=torch.int32))


def test_reference_mm16_by_hand():
    a, b = np.array([[1.0, 2.0]]), np.array([[3.0, 1.0], [1.0, -1.0]])
    assert np.allclose(refblock.mm16(a, b)[0], [[5, -1]])
    assert np.allclose(refblock.mm16(a, b, True, "relu", np.array([1.0, 2.0]), np.array([2.0]), np.array([[10.0]]))[0], [[22.0]])
