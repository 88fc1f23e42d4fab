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
