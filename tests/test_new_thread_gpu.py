"""The first call that a new host thread makes, before anything else there has touched CUDA, of each kernel with tensor maps."""
import threading

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def in_a_new_thread(f):
    failed = []

    def go():
        try:
            f()
        except Exception as e:  # noqa: BLE001
            failed.append(e)
    th = threading.Thread(target=go)
    th.start()
    th.join()
    torch.cuda.synchronize()
    assert not failed, failed


def test_products_from_a_new_thread():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from quantized_routed_expert_fn_gb300 import build, moe
    build.build()
    st = torch.zeros(2, dtype=torch.int32, device="cuda")
    one = torch.full((600, 256), 0x38, dtype=torch.uint8, device="cuda")  # 1 in e4m3
    sa, sb = torch.full((600, 4), 127, dtype=torch.uint8, device="cuda")[:, :2], torch.full((5, 2), 127, dtype=torch.uint8, device="cuda")
    out8, out16 = torch.zeros(600, 600, device="cuda"), torch.zeros(600, 600, device="cuda")
    b16 = torch.ones(600, 256, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    in_a_new_thread(lambda: moe.mm8(one, sa, one, sb, out8, st[0:1]))
    in_a_new_thread(lambda: moe.mm16(b16, b16, out16, st[1:2]))
    assert (out8 == 256).all() and (out16 == 256).all() and (st == 0).all()


def test_prefill_from_a_new_thread():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import numpy as np
    from quantized_routed_expert_fn_gb300 import build, moe, synth
    build.build()
    rng = np.random.default_rng(1)
    dl = moe.DeviceLayers([synth.make_layer(rng, 256, 8, 2, 128, 4, shared=True)], device="cuda:0")
    x = torch.from_numpy(rng.normal(size=(37, 256)).astype(np.float32)).cuda()
    work, st = moe.alloc_workspace(moe.prefill_workspace(dl, 37)), torch.zeros(1, dtype=torch.int32, device="cuda")
    outs = [torch.zeros(37, 256, dtype=torch.int16, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    in_a_new_thread(lambda: moe.prefill(dl, x, outs[0], work, st))
    moe.prefill(dl, x, outs[1], work, st)
    torch.cuda.synchronize()
    assert torch.equal(*outs) and st.item() == 0 and outs[0].any()
