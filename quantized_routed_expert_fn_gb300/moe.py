"""Python binding of the C ABI in include/moe_api.h (argument marshalling only).

Every step of the path runs in libmoe_gb300.so; this module only turns torch
tensors into pointers, fills the ABI structs and checks return codes.  There
is no fallback: if the library is missing the import of `lib()` raises.
"""
from __future__ import annotations

import ctypes
import functools
import os

import numpy as np
import torch

from . import build as _build
from . import synth

RESIDUAL = 1
PRENORM = 2
LOOKAHEAD = 4
TEST_WITHHOLD = 0x100

F32, BF16 = 0, 1
SCORES = {"softmax": 0, "sigmoid": 1}
GATE_RENORM = 1

OK, EINVAL, ESHAPE, EALIGN, ECUDA, ETIMEOUT, EDEVICE, ENOSPACE = 0, -1, -2, -3, -4, -5, -6, -7
STATUS_NAMES = {0: "MOE_OK", -1: "MOE_EINVAL", -2: "MOE_ESHAPE", -3: "MOE_EALIGN", -4: "MOE_ECUDA",
                -5: "MOE_ETIMEOUT", -6: "MOE_EDEVICE", -7: "MOE_ENOSPACE"}

EXPORTS = ["moe_route", "moe_forward", "moe_forward_traced", "moe_forward_noalloc", "moe_forward_workspace",
           "moe_prefill", "moe_prefill_timed", "moe_prefill_workspace", "moe_prefill_group", "moe_last_error",
           "moe_gate", "moe_quant8", "moe_mm8", "moe_experts8", "moe_experts8_workspace", "moe_tier_create", "moe_tier_update", "moe_tier_slot", "moe_tier_get_stats", "moe_tier_addresses",
           "moe_tier_destroy", "moe_tier_last_error"]
PREFILL_KERNELS = 10
PREFILL_KERNEL_NAMES = ["prep", "router_gemm", "topk", "group_count", "group_scan", "group_fill", "gather",
                        "gate_up_gemm", "down_gemm", "output"]
NOALLOC_MAX_WORKSPACE = 4 << 20
TRACE_CTAS, TRACE_PHASES = 1024, 16


class MoeQ(ctypes.Structure):
    _fields_ = [("w", ctypes.c_uint64), ("s", ctypes.c_uint64), ("b", ctypes.c_uint64),
                ("out", ctypes.c_uint32), ("inp", ctypes.c_uint32)]


class MoeLayer(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_uint32), ("n_experts", ctypes.c_uint32), ("top_k", ctypes.c_uint32),
                ("inter", ctypes.c_uint32), ("bits", ctypes.c_uint32), ("group", ctypes.c_uint32),
                ("flags", ctypes.c_uint32),
                ("router", ctypes.c_void_p), ("shared_gate", ctypes.c_void_p), ("shared_record", ctypes.c_void_p),
                ("sh_gate_up", MoeQ), ("sh_down", MoeQ),
                ("expert_addr", ctypes.c_void_p),
                ("gate_up", MoeQ), ("down", MoeQ),
                ("expert_bits", ctypes.c_void_p), ("gate_up_w", MoeQ * 3), ("down_w", MoeQ * 3),
                ("expert_tier", ctypes.c_void_p), ("cut_weak", ctypes.c_float),
                ("lookahead_idx", ctypes.c_void_p)]


class TierStats(ctypes.Structure):
    _fields_ = [("resident", ctypes.c_int), ("last_host_reads", ctypes.c_int), ("last_promoted", ctypes.c_int),
                ("promotions", ctypes.c_longlong), ("evictions", ctypes.c_longlong)]


class MoeGateCfg(ctypes.Structure):
    _fields_ = [("n_experts", ctypes.c_uint32), ("top_k", ctypes.c_uint32), ("score", ctypes.c_uint32),
                ("n_groups", ctypes.c_uint32), ("top_groups", ctypes.c_uint32), ("group_top", ctypes.c_uint32),
                ("flags", ctypes.c_uint32), ("scale", ctypes.c_float)]


class MoeLayer8(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_uint32), ("n_experts", ctypes.c_uint32), ("inter", ctypes.c_uint32),
                ("gate_up", ctypes.c_void_p), ("gate_up_s", ctypes.c_void_p), ("down", ctypes.c_void_p),
                ("down_s", ctypes.c_void_p)]


class MoeError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"{STATUS_NAMES.get(code, code)}: {msg}")
        self.code = code


_lib = None


def lib(path: str | None = None) -> ctypes.CDLL:
    """Load libmoe_gb300.so (built by build.build()); raise if it is absent."""
    global _lib
    if _lib is None:
        path = path or _build.LIB
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it with quantized_routed_expert_fn_gb300.build.build()")
        L = ctypes.CDLL(path)
        vp, i32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
        L.moe_last_error.restype = ctypes.c_char_p
        L.moe_forward_workspace.restype = sz
        L.moe_forward_workspace.argtypes = [ctypes.POINTER(MoeLayer), i32, i32]
        L.moe_forward.restype = i32
        L.moe_forward.argtypes = [ctypes.POINTER(MoeLayer), i32, vp, i32, vp, vp, sz, vp, vp, vp, vp, vp]
        L.moe_forward_traced.restype = i32
        L.moe_forward_traced.argtypes = [ctypes.POINTER(MoeLayer), i32, vp, i32, vp, vp, sz, vp, vp, vp, vp, vp, vp]
        L.moe_forward_noalloc.restype = i32
        L.moe_forward_noalloc.argtypes = [ctypes.POINTER(MoeLayer), i32, vp, i32, vp, vp, vp, vp, vp, vp]
        L.moe_route.restype = i32
        L.moe_route.argtypes = [ctypes.POINTER(MoeLayer), vp, i32, vp, vp, vp, vp, vp, vp, sz, vp, vp]
        L.moe_prefill_workspace.restype = sz
        L.moe_prefill_workspace.argtypes = [ctypes.POINTER(MoeLayer), i32]
        L.moe_prefill.restype = i32
        L.moe_prefill.argtypes = [ctypes.POINTER(MoeLayer), vp, i32, vp, vp, sz, vp, vp, vp]
        L.moe_prefill_timed.restype = i32
        L.moe_prefill_timed.argtypes = [ctypes.POINTER(MoeLayer), vp, i32, vp, vp, sz, vp, vp, vp, vp]
        L.moe_prefill_group.restype = i32
        L.moe_prefill_group.argtypes = [ctypes.POINTER(MoeLayer), vp, i32, vp, vp, vp, vp, vp, vp, sz, vp, vp]
        i64, u32 = ctypes.c_int64, ctypes.c_uint32
        L.moe_gate.restype = i32
        L.moe_gate.argtypes = [ctypes.POINTER(MoeGateCfg), vp, i32, i64, vp, i32, vp, vp, vp]
        L.moe_quant8.restype = i32
        L.moe_quant8.argtypes = [vp, i32, i64, i32, i32, i32, vp, i64, vp, i64, vp]
        L.moe_mm8.restype = i32
        L.moe_mm8.argtypes = [vp, i64, vp, i64, i32, vp, vp, i32, i32, vp, i32, i64, vp, i32, u32, vp, vp]
        L.moe_experts8_workspace.restype = sz
        L.moe_experts8_workspace.argtypes = [ctypes.POINTER(MoeLayer8), i32, i32]
        L.moe_experts8.restype = i32
        L.moe_experts8.argtypes = [ctypes.POINTER(MoeLayer8), vp, i32, i32, vp, vp, i32, vp, i32, vp, sz, vp, vp]
        L.moe_tier_create.restype = i32
        L.moe_tier_create.argtypes = [i32, i32, sz, vp, vp, i32, vp, vp, vp, ctypes.POINTER(vp)]
        L.moe_tier_update.restype = i32
        L.moe_tier_update.argtypes = [vp, vp, i32, vp]
        L.moe_tier_slot.restype = i32
        L.moe_tier_slot.argtypes = [vp, i32, i32]
        L.moe_tier_get_stats.restype = i32
        L.moe_tier_get_stats.argtypes = [vp, ctypes.POINTER(TierStats)]
        L.moe_tier_addresses.restype = ctypes.POINTER(ctypes.c_uint64)
        L.moe_tier_addresses.argtypes = [vp]
        L.moe_tier_destroy.restype = None
        L.moe_tier_destroy.argtypes = [vp]
        L.moe_tier_last_error.restype = ctypes.c_char_p
        _lib = L
    return _lib


def last_error() -> str:
    return lib().moe_last_error().decode()


def _check(code: int) -> None:
    if code != OK:
        raise MoeError(code, last_error())


def _p(t) -> int | None:
    return None if t is None else t.data_ptr()


def _stream(stream) -> int | None:
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _q(q) -> MoeQ:
    return MoeQ(q.w, q.s, q.b, q.out, q.inp)


class DeviceLayers:
    """Device copies of synth.Layer weights plus the ABI structs that point at them."""

    def __init__(self, layers, device="cuda"):
        self.tensors = []  # per layer: router, records, expert addresses, shared gate, shared record
        self.keep = []
        arr = (MoeLayer * len(layers))()
        for i, L in enumerate(layers):
            if isinstance(L, synth.DeviceLayer):
                router, recs, sg, srec = L.router, L.records, L.shared_gate, L.shared_record
            else:
                router = torch.from_numpy(L.router.view(np.int16)).to(device)
                recs = torch.from_numpy(L.records).to(device)
                sg = srec = None
                if L.shared_gate is not None:
                    sg = torch.from_numpy(L.shared_gate.view(np.int16)).to(device)
                    srec = torch.from_numpy(L.shared_record).to(device)
            stride = L.layout.stride
            base = recs.data_ptr()
            eaddr = torch.arange(L.n_experts, dtype=torch.int64, device=recs.device) * stride + base
            self.tensors += [router, recs, eaddr, sg, srec]
            c = arr[i]
            c.hidden, c.n_experts, c.top_k, c.inter = L.hidden, L.n_experts, L.top_k, L.inter
            c.bits, c.group, c.flags = L.bits, 64, L.flags
            c.router = router.data_ptr()
            c.shared_gate = _p(sg)
            c.shared_record = _p(srec)
            if L.shared_layout is not None:
                c.sh_gate_up, c.sh_down = _q(L.shared_layout.gate_up), _q(L.shared_layout.down)
            c.expert_addr = eaddr.data_ptr()
            c.gate_up, c.down = _q(L.layout.gate_up), _q(L.layout.down)
            if getattr(L, "expert_bits", None) is not None:
                # mixed widths: a width per routed record, offsets per width
                eb = L.expert_bits
                eb = eb if isinstance(eb, torch.Tensor) else torch.from_numpy(np.ascontiguousarray(eb))
                eb = eb.to(device=recs.device, dtype=torch.uint8)
                self.keep.append(eb)
                c.expert_bits = eb.data_ptr()
                for j, b in enumerate((4, 3, 2)):
                    c.gate_up_w[j], c.down_w[j] = _q(L.layouts[b].gate_up), _q(L.layouts[b].down)
        self.c = arr
        self.n = len(layers)
        self.src = layers

    def set_tier(self, layer: int, expert_addr: torch.Tensor, expert_tier: torch.Tensor | None,
                 cut_weak: float = 0.0) -> None:
        """Point layer `layer` at other record addresses (device or host
        memory) with their tiers (uint8 [E], 1 = host memory), and set its cut."""
        self.keep += [expert_addr, expert_tier]
        c = self.c[layer]
        c.expert_addr = expert_addr.data_ptr()
        c.expert_tier = None if expert_tier is None else expert_tier.data_ptr()
        c.cut_weak = cut_weak

    def set_flags(self, flags: int) -> None:
        for i in range(self.n):
            self.c[i].flags = flags


def forward_workspace(layers: DeviceLayers | ctypes.Array, nb: int, n_layers: int | None = None) -> int:
    arr = layers.c if isinstance(layers, DeviceLayers) else layers
    n = n_layers if n_layers is not None else len(arr)
    return int(lib().moe_forward_workspace(arr, n, nb))


def alloc_workspace(nbytes: int, device="cuda") -> torch.Tensor:
    return torch.empty(nbytes + 256, dtype=torch.uint8, device=device)


def _aligned(ws: torch.Tensor) -> tuple[int, int]:
    p = ws.data_ptr()
    a = (p + 255) // 256 * 256
    return a, ws.numel() - (a - p)


def forward(layers: DeviceLayers, x: torch.Tensor, out: torch.Tensor, work: torch.Tensor, status: torch.Tensor,
            slot_tab=None, wmap=None, topk_idx=None, n_layers: int | None = None, stream=None,
            layer_offset: int = 0) -> None:
    """moe_forward over layers[layer_offset : layer_offset + n_layers]."""
    n = n_layers if n_layers is not None else layers.n - layer_offset
    arr = ctypes.cast(ctypes.byref(layers.c, layer_offset * ctypes.sizeof(MoeLayer)), ctypes.POINTER(MoeLayer))
    wp, wb = _aligned(work)
    _check(lib().moe_forward(arr, n, _p(x), x.shape[0], _p(out), wp, wb, _p(slot_tab), _p(wmap), _p(topk_idx),
                             _p(status), _stream(stream)))


def forward_traced(layers: DeviceLayers, x: torch.Tensor, out: torch.Tensor, work: torch.Tensor,
                   status: torch.Tensor, trace: torch.Tensor, slot_tab=None, wmap=None, topk_idx=None,
                   stream=None) -> None:
    """moe_forward with per-phase timestamps into trace (int64 [n_layers][1024][16])."""
    wp, wb = _aligned(work)
    _check(lib().moe_forward_traced(layers.c, layers.n, _p(x), x.shape[0], _p(out), wp, wb, _p(slot_tab), _p(wmap),
                                    _p(topk_idx), _p(status), _p(trace), _stream(stream)))


def forward_noalloc(layers: DeviceLayers, x: torch.Tensor, out: torch.Tensor, status: torch.Tensor,
                    slot_tab=None, wmap=None, topk_idx=None, stream=None) -> None:
    """moe_forward on the library's fixed scratch (no workspace, no allocation)."""
    _check(lib().moe_forward_noalloc(layers.c, layers.n, _p(x), x.shape[0], _p(out), _p(slot_tab), _p(wmap),
                                     _p(topk_idx), _p(status), _stream(stream)))


def route(layers: DeviceLayers, x: torch.Tensor, topk_idx, topk_w, slot_row, wmap_row, work, status,
          logits=None, layer: int = 0, stream=None) -> None:
    arr = ctypes.cast(ctypes.byref(layers.c, layer * ctypes.sizeof(MoeLayer)), ctypes.POINTER(MoeLayer))
    wp, wb = _aligned(work)
    _check(lib().moe_route(arr, _p(x), x.shape[0], _p(logits), _p(topk_idx), _p(topk_w), _p(slot_row),
                           _p(wmap_row), wp, wb, _p(status), _stream(stream)))


def _layer_ptr(layers: DeviceLayers, layer: int):
    return ctypes.cast(ctypes.byref(layers.c, layer * ctypes.sizeof(MoeLayer)), ctypes.POINTER(MoeLayer))


def prefill_workspace(layers: DeviceLayers, t: int, layer: int = 0) -> int:
    return int(lib().moe_prefill_workspace(_layer_ptr(layers, layer), t))


def prefill(layers: DeviceLayers, x: torch.Tensor, out: torch.Tensor, work: torch.Tensor, status: torch.Tensor,
            topk_idx=None, layer: int = 0, stream=None) -> None:
    """moe_prefill: x float32 [t][H] -> out bf16 bits (int16 tensor) [t][H]."""
    wp, wb = _aligned(work)
    _check(lib().moe_prefill(_layer_ptr(layers, layer), _p(x), x.shape[0], _p(out), wp, wb, _p(topk_idx),
                             _p(status), _stream(stream)))


def prefill_group(layers: DeviceLayers, x: torch.Tensor, topk_idx, topk_w, group_offs, group_rows, group_w,
                  work, status, layer: int = 0, stream=None) -> None:
    """moe_prefill_group: routing and the stable expert grouping of a prefill chunk."""
    wp, wb = _aligned(work)
    _check(lib().moe_prefill_group(_layer_ptr(layers, layer), _p(x), x.shape[0], _p(topk_idx), _p(topk_w),
                                   _p(group_offs), _p(group_rows), _p(group_w), wp, wb, _p(status),
                                   _stream(stream)))


def prefill_timed(layers: DeviceLayers, x: torch.Tensor, out: torch.Tensor, work: torch.Tensor,
                  status: torch.Tensor, events, topk_idx=None, layer: int = 0, stream=None) -> None:
    """moe_prefill recording events[i] (torch.cuda.Event, already recorded once so
    that it exists) before kernel i and events[PREFILL_KERNELS] after the last."""
    assert len(events) == PREFILL_KERNELS + 1
    arr = (ctypes.c_void_p * len(events))(*[e.cuda_event for e in events])
    wp, wb = _aligned(work)
    _check(lib().moe_prefill_timed(_layer_ptr(layers, layer), _p(x), x.shape[0], _p(out), wp, wb, _p(topk_idx),
                                   _p(status), arr, _stream(stream)))


# ---- 8-bit experts: routing from given logits, quantisation, products

_FLOATS = {torch.float32: F32, torch.bfloat16: BF16}
_E4M3 = (torch.uint8, torch.float8_e4m3fn)
_E8M0 = (torch.uint8, getattr(torch, "float8_e8m0fnu", torch.uint8))
_I32 = (torch.int32, getattr(torch, "uint32", torch.int32))
_F32 = (torch.float32,)


def _bad(code: int, msg: str):
    raise MoeError(code, msg)


def _arg(t, name: str, shape: tuple, dtypes, dev: int) -> int:
    """Address of a CUDA tensor after checking type, shape, device and that its
    last dimension is contiguous (the strides of the others are the caller's)."""
    if t.dtype not in dtypes:
        _bad(EINVAL, f"{name} is {t.dtype}")
    if t.shape != shape:
        _bad(ESHAPE, f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.get_device() != dev:
        _bad(EINVAL, f"{name} is on {t.device}, expected cuda:{dev}")
    if not t.is_contiguous() and t.stride(-1) != 1 and t.shape[-1] > 1 and t.numel():
        _bad(EINVAL, f"{name}'s last dimension is not contiguous")
    return t.data_ptr()


def _whole(t, name: str, shape: tuple, dtypes, dev: int) -> int:
    if t.dtype not in dtypes:
        _bad(EINVAL, f"{name} is {t.dtype}")
    if t.shape != shape:
        _bad(ESHAPE, f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.get_device() != dev:
        _bad(EINVAL, f"{name} is on {t.device}, expected cuda:{dev}")
    if not t.is_contiguous():
        _bad(EINVAL, f"{name} is not contiguous")
    return t.data_ptr()


def _device(t, name: str) -> int:
    """The call's device: the current one, where the stream and every tensor have to be."""
    dev = t.get_device()
    if dev < 0 or dev != _current_device():
        _bad(EINVAL, f"{name} is on {t.device}, not on the current CUDA device")
    return dev


# The current stream's handle without a torch.cuda.Stream object around it
# (the object costs as much as a small call), where torch has that call.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


# The same for the current device, once a tensor says that CUDA is there.
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream_on(stream, dev: int) -> int:
    if stream is None and _raw_stream is not None:
        return _raw_stream(dev)
    return _stream(stream)


def _ld(t, rows: int, cols: int) -> int:
    """Row stride; of a single row, whose stride means nothing, its length."""
    return t.stride(0) if rows > 1 else cols


@functools.lru_cache(maxsize=64)
def _gate_cfg(n_experts, top_k, score, n_groups, top_groups, group_top, flags, scale) -> MoeGateCfg:
    if score not in SCORES:
        _bad(EINVAL, f"unknown score {score!r}")
    return MoeGateCfg(n_experts, top_k, SCORES[score], n_groups, top_groups, group_top, flags, scale)


def gate(logits: torch.Tensor, topk_idx: torch.Tensor, topk_w: torch.Tensor, bias=None, score: str = "softmax",
         n_groups: int = 1, top_groups: int = 1, group_top: int = 1, renorm: bool = False, scale: float = 1.0,
         stream=None) -> None:
    """moe_gate: logits float32 / bfloat16 [t][E] (any row stride) -> topk_idx int32 [t][k]
    (-1: no expert left), topk_w float32 [t][k]; bias float32 [E] steers the choice only."""
    if logits.dim() != 2 or topk_idx.dim() != 2:
        _bad(ESHAPE, "logits and topk_idx are matrices")
    t, e = logits.shape
    k = topk_idx.shape[1]
    dev = _device(logits, "logits")
    lp = _arg(logits, "logits", (t, e), _FLOATS, dev)
    ip = _whole(topk_idx, "topk_idx", (t, k), _I32, dev)
    wp = _whole(topk_w, "topk_w", (t, k), _F32, dev)
    bp = None if bias is None else _whole(bias, "bias", (e,), _F32, dev)
    cfg = _gate_cfg(e, k, score, n_groups, top_groups, group_top, GATE_RENORM if renorm else 0, scale)
    _check((_lib or lib()).moe_gate(cfg, lp, _FLOATS[logits.dtype], _ld(logits, t, e), bp, t, ip, wp,
                                    _stream_on(stream, dev)))


def quant8(x: torch.Tensor, q: torch.Tensor, s: torch.Tensor, block_rows: int = 1, stream=None) -> None:
    """moe_quant8: x float32 / bfloat16 [rows][cols] -> q e4m3 [rows][cols] (float8_e4m3fn or uint8) and
    s E8M0 [ceil(rows / block_rows)][ceil(cols / 128)] (float8_e8m0fnu or uint8); row strides as they are."""
    if x.dim() != 2 or block_rows not in (1, 128):
        _bad(ESHAPE, "x is a matrix; block_rows is 1 or 128")
    rows, cols = x.shape
    dev = _device(x, "x")
    xp = _arg(x, "x", (rows, cols), _FLOATS, dev)
    qp = _arg(q, "q", (rows, cols), _E4M3, dev)
    sr, sc = -(-rows // block_rows), -(-cols // 128)
    sp = _arg(s, "s", (sr, sc), _E8M0, dev)
    _check((_lib or lib()).moe_quant8(xp, _FLOATS[x.dtype], _ld(x, rows, cols), rows, cols, block_rows, qp,
                                      _ld(q, rows, cols), sp, _ld(s, sr, sc), _stream_on(stream, dev)))


def mm8(a: torch.Tensor, sa: torch.Tensor, b: torch.Tensor, sb: torch.Tensor, out: torch.Tensor, status: torch.Tensor,
        offs=None, flags: int = 0, stream=None) -> None:
    """moe_mm8: a e4m3 [t][k] with sa E8M0 [t][ceil(k / 128)] (its rows a multiple of 4 bytes apart, the last
    one held whole) times b e4m3 [n][k] with sb [ceil(n / 128)][ceil(k / 128)] -> out float32 / bfloat16 [t][n].
    With offs int32 [G + 1]: b [G][n][k], sb [G][..][..], group g has the rows offs[g] .. offs[g + 1] - 1."""
    if offs is not None and (offs.dim() != 1 or offs.shape[0] < 2):
        _bad(ESHAPE, "offs is a vector of the groups' G + 1 row offsets")
    groups = 0 if offs is None else offs.shape[0] - 1
    if a.dim() != 2 or b.dim() != (3 if groups else 2):
        _bad(ESHAPE, "a is [t][k]; b is [n][k], with offs [G][n][k]")
    t, k = a.shape
    n = b.shape[-2]
    dev = _device(a, "a")
    lead = (groups,) if groups else ()
    ap = _arg(a, "a", (t, k), _E4M3, dev)
    sap = _arg(sa, "sa", (t, -(-k // 128)), _E8M0, dev)
    bp = _whole(b, "b", lead + (n, k), _E4M3, dev)
    sbp = _whole(sb, "sb", lead + (-(-n // 128), -(-k // 128)), _E8M0, dev)
    op = _arg(out, "out", (t, n), _FLOATS, dev)
    fp = None if offs is None else _whole(offs, "offs", (groups + 1,), _I32, dev)
    lds = sa.stride(0)
    if t == 1 and lds % 4:  # one row: only what it holds can be read
        lds = -(-lds // 4) * 4
    if t and not (lds == sa.shape[1] and sa.is_contiguous()):
        if sa.untyped_storage().nbytes() < sa.storage_offset() + t * lds:
            _bad(EINVAL, "sa's last row is not held whole")
    _check((_lib or lib()).moe_mm8(ap, _ld(a, t, k), sap, lds, t, bp, sbp, n, k, op, _FLOATS[out.dtype], _ld(out, t, n),
                                   fp, groups, flags, _whole(status, "status", (1,), _I32, dev), _stream_on(stream, dev)))


class Layer8:
    """Routed experts in 8 bits: gate_up e4m3 [E][2 * inter][hidden] (the gate rows first), down e4m3
    [E][hidden][inter], with E8M0 scales per 128 x 128 block (quant8 with block_rows=128, expert by expert)."""

    def __init__(self, gate_up: torch.Tensor, gate_up_s: torch.Tensor, down: torch.Tensor, down_s: torch.Tensor):
        if gate_up.dim() != 3 or gate_up.shape[1] % 2:
            _bad(ESHAPE, "gate_up is [E][2 * inter][hidden]")
        e, i2, h = gate_up.shape
        i = i2 // 2
        if h % 128 or i % 128:
            _bad(ESHAPE, f"hidden {h} and inter {i} must be multiples of 128")
        dev = _device(gate_up, "gate_up")
        self.hidden, self.n_experts, self.inter, self.device = h, e, i, dev
        self.keep = (gate_up, gate_up_s, down, down_s)
        self.c = MoeLayer8(h, e, i, _whole(gate_up, "gate_up", (e, i2, h), _E4M3, dev),
                           _whole(gate_up_s, "gate_up_s", (e, i2 // 128, h // 128), _E8M0, dev),
                           _whole(down, "down", (e, h, i), _E4M3, dev),
                           _whole(down_s, "down_s", (e, h // 128, i // 128), _E8M0, dev))


def experts8_workspace(layer: Layer8, t: int, top_k: int) -> int:
    """Bytes experts8 needs for t rows or fewer of this layer and top_k: one workspace for the largest batch serves all."""
    return int(lib().moe_experts8_workspace(layer.c, t, top_k))


def experts8(layer: Layer8, x: torch.Tensor, topk_idx: torch.Tensor, topk_w: torch.Tensor, out: torch.Tensor,
             work: torch.Tensor, status: torch.Tensor, stream=None) -> None:
    """moe_experts8: x float32 / bfloat16 [t][hidden] through the experts topk_idx int32 [t][k] (ids outside
    0 .. E - 1 contribute nothing) with weights topk_w -> out float32 / bfloat16 [t][hidden]."""
    if topk_idx.dim() != 2:
        _bad(ESHAPE, "topk_idx is a matrix")
    t, k = topk_idx.shape
    dev = _device(x, "x")
    shape = (t, layer.hidden)
    wp, wb = _aligned(work)
    if layer.device != dev or work.get_device() != dev:
        _bad(EINVAL, f"layer on cuda:{layer.device}, work on {work.device}, x on cuda:{dev}")
    _check((_lib or lib()).moe_experts8(layer.c, _whole(x, "x", shape, _FLOATS, dev), _FLOATS[x.dtype], t,
                                        _whole(topk_idx, "topk_idx", (t, k), _I32, dev),
                                        _whole(topk_w, "topk_w", (t, k), _F32, dev), k,
                                        _whole(out, "out", shape, _FLOATS, dev), _FLOATS[out.dtype], wp, wb,
                                        _whole(status, "status", (1,), _I32, dev), _stream_on(stream, dev)))


class Tier:
    """The two-tier expert store (moe_tier_*): records in pinned host memory,
    the most recently used ones cached in device slots.

    host_records: address (int) or pinned uint8 tensor [n_layers][n_experts][stride];
    slots: device uint8 tensor [n_slots][stride] or None; expert_addr /
    expert_tier: device int64 / uint8 tensors [n_layers][n_experts], or None
    for a policy-only store (no CUDA call)."""

    def __init__(self, n_layers, n_experts, stride, host_records, n_slots, slots=None, expert_addr=None,
                 expert_tier=None, stream=None):
        self.n_layers, self.n_experts, self.stride = n_layers, n_experts, stride
        self._keep = [host_records, slots, expert_addr, expert_tier]
        h = host_records if isinstance(host_records, int) else host_records.data_ptr()
        self.dry = expert_addr is None
        t = ctypes.c_void_p()
        code = lib().moe_tier_create(n_layers, n_experts, stride, h, _p(slots), n_slots, _p(expert_addr),
                                     _p(expert_tier), None if self.dry else _stream(stream), ctypes.byref(t))
        if code != OK:
            raise MoeError(code, lib().moe_tier_last_error().decode())
        self.t = t

    def update(self, slot_tab, stream=None) -> int:
        """slot_tab: host uint64 array [n_layers][64] of the step just run."""
        st = np.ascontiguousarray(slot_tab, dtype=np.uint64)
        r = lib().moe_tier_update(self.t, st.ctypes.data, st.shape[0], None if self.dry else _stream(stream))
        if r < 0:
            raise MoeError(r, lib().moe_tier_last_error().decode())
        return r

    def slot(self, layer: int, expert: int) -> int:
        return int(lib().moe_tier_slot(self.t, layer, expert))

    def stats(self) -> dict:
        s = TierStats()
        _check(lib().moe_tier_get_stats(self.t, ctypes.byref(s)))
        return {f: getattr(s, f) for f, _ in TierStats._fields_}

    def addresses(self) -> np.ndarray:
        p = lib().moe_tier_addresses(self.t)
        return np.ctypeslib.as_array(p, shape=(self.n_layers, self.n_experts)).copy()

    def close(self) -> None:
        if self.t:
            lib().moe_tier_destroy(self.t)
            self.t = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
