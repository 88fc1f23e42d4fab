"""A block of a served model through the operators as they are used together: norm, router product, routing, 8-bit experts,
shared expert with its gate on top of them, the next norm, the vocabulary's product, the answer's probabilities.

Each step is held to a 64-bit computation of that step from the inputs that it was given (refblock, ref8), the whole run to
the same bits when it is captured and replayed, on one token, a verify step and a prompt chunk."""
import subprocess
import sys
import threading

import numpy as np
import pytest

import ref8
import refblock as rb

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

H, E, K, I, V = 512, 16, 4, 256, 5003


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


class Block:
    """Weights, buffers and the calls of a block over t rows."""

    def __init__(self, m, t):
        g = torch.Generator(device="cuda")
        g.manual_seed(t)
        rnd = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
        bf = torch.bfloat16
        self.m, self.t = m, t
        self.stream0 = rnd(t, H) * 2
        self.w1, self.w2, self.wp = (1 + 0.2 * rnd(H) for _ in range(3))
        self.router, self.gate_w = (rnd(E, H) * H ** -0.5).to(bf), (rnd(1, H) * H ** -0.5).to(bf)
        self.s_up, self.s_down = (rnd(2 * I, H) * H ** -0.5).to(bf), (rnd(H, I) * I ** -0.5).to(bf)
        self.head = (rnd(V, H) * 3 * H ** -0.5).to(bf)
        q = []
        for shape in ((E, 2 * I, H), (E, H, I)):
            w = rnd(*shape) * shape[2] ** -0.5
            qw = torch.empty(shape, dtype=torch.float8_e4m3fn, device="cuda")
            s = torch.empty(shape[0], shape[1] // 128, shape[2] // 128, dtype=torch.uint8, device="cuda")
            for e in range(E):
                m.quant8(w[e], qw[e], s[e], block_rows=128)
            q += [qw, s]
        self.layer = m.Layer8(*q)
        self.work = m.alloc_workspace(m.experts8_workspace(self.layer, t, K))
        self.status = torch.zeros(6, dtype=torch.int32, device="cuda")
        e = lambda *s, d=torch.float32: torch.empty(*s, dtype=d, device="cuda")  # noqa: E731
        self.stream, self.n1, self.logits, self.idx, self.wts = e(t, H), e(t, H, d=bf), e(t, E), e(t, K, d=torch.int32), e(t, K)
        self.y, self.h, self.sg, self.n2 = e(t, H), e(t, I, d=bf), e(t, 1), e(t, H, d=bf)
        self.shared = e(t, H)
        self.vocab, self.tok = e(t, V), torch.randint(0, V, (t, 2), device="cuda", generator=g).to(torch.int32)
        self.logp, self.ent, self.top, self.top_lp = e(t, 2), e(t), e(t, 5, d=torch.int32), e(t, 5)

    def run(self):
        m, st = self.m, self.status
        self.stream.copy_(self.stream0)
        m.norm(self.stream, self.n1, w=self.w1)
        m.mm16(self.n1, self.router, self.logits, st[0:1])
        m.gate(self.logits, self.idx, self.wts, renorm=True)
        m.experts8(self.layer, self.n1, self.idx, self.wts, self.y, self.work, st[1:2])
        m.mm16(self.n1, self.gate_w, self.sg, st[2:3], act="sigmoid")
        m.mm16(self.n1, self.s_up, self.h, st[3:4], act="silu", gated=True)
        m.mm16(self.h, self.s_down, self.shared, st[4:5], row_scale=self.sg.view(-1), residual=self.y)
        m.add_norm(self.shared, self.stream, self.stream, post=True, w_post=self.wp, scale=0.5, out=self.n2, w=self.w2)
        m.mm16(self.n2, self.head, self.vocab, st[5:6])
        m.logprobs(self.vocab, tokens=self.tok, logp=self.logp, entropy=self.ent, top_idx=self.top, top_logp=self.top_lp)

    def results(self):
        return [x.clone() for x in (self.stream, self.n1, self.logits, self.idx, self.wts, self.y, self.sg, self.h, self.shared, self.n2,
                                    self.vocab, self.logp, self.ent, self.top, self.top_lp)]


@pytest.mark.parametrize("t", [1, 4, 11, 150])
def test_a_block_step_by_step(moe, t):
    b = Block(moe, t)
    b.run()
    torch.cuda.synchronize()
    assert (b.status == 0).all()
    x0 = f64(b.stream0)
    ref = rb.norm(x0, f64(b.w1))
    rb.check(f64(b.n1), ref, np.abs(ref) * (rb.NORM + 2) * rb.U, "bf16", "norm")
    n1 = f64(b.n1)
    rb.check(f64(b.logits), *rb.mm16(n1, f64(b.router)), "f32", "router")
    ri, rw = ref8.gate(f64(b.logits), K, renorm=True)
    assert np.array_equal(b.idx.cpu().numpy(), ri)
    assert (np.abs(f64(b.wts) - rw) <= 2.0 ** -19 * rw.max(1, keepdims=True)).all()
    gu, gus, dn, dns = b.layer.keep
    byte = lambda x: x.view(torch.uint8).cpu().numpy()  # noqa: E731
    rows = slice(0, 12)
    ref, allow = ref8.experts8(n1[rows], byte(gu), byte(gus), byte(dn), byte(dns), ri[rows], f64(b.wts)[rows], 2.0 ** -24)
    assert (np.abs(f64(b.y)[rows] - ref) <= allow + 1e-30).all()
    rb.check(f64(b.sg), *rb.mm16(n1, f64(b.gate_w), False, "sigmoid"), "f32", "shared gate")
    rb.check(f64(b.h), *rb.mm16(n1, f64(b.s_up), True, "silu"), "bf16", "shared up")
    rb.check(f64(b.shared), *rb.mm16(f64(b.h), f64(b.s_down), False, "none", None, f64(b.sg)[:, 0], f64(b.y)), "f32", "shared down")
    r, dr, n, dn_ = rb.add_norm(f64(b.shared), x0, True, f64(b.wp), None, False, 0.5, 1.0, f64(b.w2))
    rb.check(f64(b.stream), r, dr, "f32", "stream")
    rb.check(f64(b.n2), n, dn_, "bf16", "next norm")
    rb.check(f64(b.vocab), *rb.mm16(f64(b.n2), f64(b.head)), "f32", "head")
    lp, ent, idx, tl, dz = rb.logprobs(f64(b.vocab), b.tok.cpu().numpy(), 5)
    rb.check(f64(b.logp), lp, dz + np.abs(lp) * 3 * rb.U, "f32", "logp")
    rb.check(f64(b.ent), ent, (2 + 2 * ent) * dz[:, 0], "f32", "entropy")
    assert np.array_equal(b.top.cpu().numpy(), idx)
    rb.check(f64(b.top_lp), tl, dz + np.abs(tl) * 3 * rb.U, "f32", "top")


@pytest.mark.parametrize("t", [1, 4, 150, 700])
def test_a_block_captured_and_replayed(moe, t):
    b = Block(moe, t)
    b.run()
    torch.cuda.synchronize()
    ref = b.results()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(2):
            b.run()
    for x in (b.n1, b.logits, b.idx, b.y, b.h, b.shared, b.n2, b.vocab, b.top):
        x.zero_()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert (b.status == 0).all()
    for a, c in zip(ref, b.results()):
        assert torch.equal(a, c)


def test_two_blocks_at_once(moe):
    """Two threads, each with its block on a stream of its own."""
    blocks = [Block(moe, 9), Block(moe, 300)]
    refs = []
    for b in blocks:
        b.run()
        torch.cuda.synchronize()
        refs.append(b.results())

    def go(b, s):
        with torch.cuda.stream(s):
            for _ in range(20):
                b.run()
    streams = [torch.cuda.Stream() for _ in blocks]
    [s.wait_stream(torch.cuda.current_stream()) for s in streams]
    workers = [threading.Thread(target=go, args=a) for a in zip(blocks, streams)]
    [w.start() for w in workers]
    [w.join() for w in workers]
    torch.cuda.synchronize()
    for b, ref in zip(blocks, refs):
        assert (b.status == 0).all()
        for a, c in zip(ref, b.results()):
            assert torch.equal(a, c)


FIRST = """
import torch
from quantized_routed_expert_fn_gb300 import moe
a, b = torch.ones(40, 128, dtype=torch.bfloat16, device="cuda"), torch.ones(600, 128, dtype=torch.bfloat16, device="cuda")
o, st = torch.zeros(40, 600, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
n, ent = torch.zeros(40, 600, device="cuda"), torch.zeros(40, device="cuda")
s = torch.cuda.Stream()
with torch.cuda.stream(s):
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        moe.mm16(a, b, o, st)
        moe.norm(o, n)
        moe.logprobs(n, entropy=ent)
g.replay()
torch.cuda.synchronize()
assert (o == 128).all() and (n - 1).abs().max() < 1e-5 and (ent - 6.39693).abs().max() < 1e-4 and st.item() == 0
"""


def test_a_first_call_may_be_captured(moe):
    """A process whose first calls are made while a stream is captured."""
    r = subprocess.run([sys.executable, "-c", FIRST], capture_output=True, text=True, timeout=120,
                       cwd=__file__.rsplit("/", 2)[0])
    assert r.returncode == 0, r.stderr[-2000:]
