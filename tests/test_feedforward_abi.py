"""Refusals of the feed-forward entry points, which need no GPU: bad arguments get the
documented status before any HIP call (the pointers are never dereferenced), and the
binding refuses tensors that the library could not address."""
import contextlib
import ctypes
import types

import pytest
import torch

from fp4_block_quantization_amd import fos
from test_serving_abi import Devices

F = ctypes.c_void_p(0x100000)
BIG = ctypes.c_void_p(0x1000000)


def at(n):
    return ctypes.c_void_p(0x100000 + n)


L = fos.lib()
OK, NULL, SHAPE, ALIGN, FLAGS, WS = (fos.FOS_OK, fos.FOS_E_NULL, fos.FOS_E_SHAPE, fos.FOS_E_ALIGN,
                                     fos.FOS_E_FLAGS, fos.FOS_E_WORKSPACE)


def norm(**kw):
    a = dict(x=F, xs=64, r=F, rs=64, w=F, M=4, K=64, eps=1e-6, h=F, rstd=F, y=F, rec=0, rule=0,
             data=F, scales=F, t=F, given=1, ws=F, wsb=4096) | kw
    return L.fos_rmsnorm_fwd(a["x"], a["xs"], a["r"], a["rs"], a["w"], a["M"], a["K"], a["eps"], a["h"],
                             a["rstd"], a["y"], a["rec"], a["rule"], a["data"], a["scales"], a["t"],
                             a["given"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(M=0), OK), (dict(M=0, x=None, w=None, y=None, h=None, rstd=None), OK),
    (dict(M=0, rec=2, data=None, scales=None), OK),
    (dict(M=-1), SHAPE), (dict(M=1 << 31), SHAPE), (dict(K=0), SHAPE), (dict(K=8), SHAPE),
    (dict(K=72), SHAPE), (dict(K=32784, xs=32784, rs=32784), SHAPE), (dict(rec=2, K=48), SHAPE),
    (dict(M=1 << 30, K=32768, xs=32768, rs=32768), SHAPE), (dict(xs=56), SHAPE), (dict(rs=56), SHAPE),
    (dict(xs=-64), SHAPE), (dict(xs=1 << 39), SHAPE),
    (dict(rec=-1), FLAGS), (dict(rec=3), FLAGS), (dict(rule=2), FLAGS), (dict(eps=0.0), FLAGS),
    (dict(eps=-1.0), FLAGS), (dict(eps=float("nan")), FLAGS), (dict(eps=float("inf")), FLAGS),
    (dict(eps=1e-39), FLAGS),
    (dict(x=None), NULL), (dict(w=None), NULL), (dict(y=None), NULL), (dict(rec=1, data=None), NULL),
    (dict(rec=2, scales=None), NULL), (dict(rec=1, t=None), NULL),
    (dict(rec=1, given=0, rstd=None), NULL), (dict(rec=1, given=0, h=None), NULL),
    (dict(x=at(8)), ALIGN), (dict(r=at(8)), ALIGN), (dict(w=at(8)), ALIGN), (dict(h=at(8)), ALIGN),
    (dict(y=at(2)), ALIGN), (dict(rstd=at(2)), ALIGN), (dict(xs=68), ALIGN), (dict(rs=68), ALIGN),
    (dict(rec=1, data=at(4)), ALIGN), (dict(rec=2, data=at(4)), ALIGN), (dict(rec=1, t=at(2)), ALIGN),
    (dict(rec=1, given=0, ws=None), WS), (dict(rec=1, given=0, ws=at(8)), WS),
    (dict(rec=1, given=0, wsb=4095), WS),
])
def test_norm_refusals(kw, want):
    if want == OK:
        kw = dict(kw, given=1)
    assert norm(**kw) == want


def norm_bwd(**kw):
    a = dict(dy=F, h=F, w=F, rstd=F, dh=F, M=4, K=64, dx=F, dw=F, ws=F, wsb=1 << 20) | kw
    return L.fos_rmsnorm_bwd(a["dy"], a["h"], a["w"], a["rstd"], a["dh"], a["M"], a["K"], a["dx"], a["dw"],
                             a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(M=0, dw=None, dy=None, h=None, dx=None), OK), (dict(M=-1), SHAPE), (dict(K=24), SHAPE),
    (dict(K=32784), SHAPE), (dict(dy=None), NULL), (dict(h=None), NULL), (dict(w=None), NULL),
    (dict(rstd=None), NULL), (dict(dx=None), NULL), (dict(dy=at(8)), ALIGN), (dict(h=at(8)), ALIGN),
    (dict(w=at(8)), ALIGN), (dict(rstd=at(2)), ALIGN), (dict(dh=at(8)), ALIGN), (dict(dx=at(8)), ALIGN),
    (dict(dw=at(4)), ALIGN), (dict(ws=None), WS), (dict(ws=at(8)), WS), (dict(wsb=64 * 4 - 1), WS),
])
def test_norm_bwd_refusals(kw, want):
    assert norm_bwd(**kw) == want


def test_workspace_sizes():
    assert L.fos_rmsnorm_bwd_workspace_bytes(0, 64) == 256
    assert L.fos_rmsnorm_bwd_workspace_bytes(1, 64) == 256
    assert L.fos_rmsnorm_bwd_workspace_bytes(1 << 20, 4096) <= 4096 * 4 * 1024
    for m, k in ((-1, 64), (4, 60), (4, 32784), (1 << 31, 64)):
        assert L.fos_rmsnorm_bwd_workspace_bytes(m, k) == 0
    assert L.fos_epilogue_bwd_workspace_bytes(0, 1, 0) > 0
    assert L.fos_epilogue_bwd_workspace_bytes(100, 64, 1) > L.fos_epilogue_bwd_workspace_bytes(100, 64, 0)
    for m, n, g in ((-1, 64, 0), (4, 0, 0), (4, 1 << 30, 0), (1 << 31, 64, 0), (4, 64, 2), (1 << 20, 1 << 25, 0)):
        assert L.fos_epilogue_bwd_workspace_bytes(m, n, g) == 0


def epilogue(**kw):
    a = dict(struct_size=ctypes.sizeof(fos.FosEpilogue), activation=4, gated=0, out_dtype=1,
             bias_bf16=None, residual_bf16=None, residual_stride=0, preact_bf16=None, reserved=0) | kw
    return fos.FosEpilogue(**{k: getattr(v, "value", v) for k, v in a.items()})


def products(e, **kw):
    """The status of the four products with these arguments (those that a product does not
    have are left out of it)."""
    a = dict(x=F, xs=256, xsc=F, xt=F, w=F, ws=F, wt=F, M=2, N=16, K=256, y=F) | kw
    p = None if e is None else ctypes.byref(e)
    size = a["M"], a["N"], a["K"]
    return {
        "q": L.fos_qlinear_epilogue_fwd(a["x"], a["xsc"], a["xt"], a["w"], a["ws"], a["wt"], *size, p, a["y"], None),
        "mxq": L.fos_mx_qlinear_epilogue_fwd(a["x"], a["xsc"], a["w"], a["ws"], *size, p, a["y"], None),
        "w": L.fos_wlinear_epilogue_fwd(a["x"], a["xs"], a["w"], a["ws"], a["wt"], *size, p, a["y"], None),
        "mxw": L.fos_mx_wlinear_epilogue_fwd(a["x"], a["xs"], a["w"], a["ws"], *size, p, a["y"], None),
    }


@pytest.mark.parametrize("kw,want", [
    (dict(struct_size=8), FLAGS), (dict(activation=5), FLAGS), (dict(gated=2), FLAGS),
    (dict(out_dtype=2), FLAGS), (dict(reserved=1), FLAGS),
    (dict(gated=1, residual_bf16=F, residual_stride=16), FLAGS),
    (dict(residual_bf16=F, residual_stride=15), SHAPE), (dict(residual_bf16=F, residual_stride=-16), SHAPE),
    (dict(residual_bf16=F, residual_stride=1 << 40), SHAPE), (dict(bias_bf16=at(1)), ALIGN),
    (dict(residual_bf16=at(1), residual_stride=16), ALIGN), (dict(preact_bf16=at(1)), ALIGN),
])
def test_epilogue_refusals(kw, want):
    assert set(products(epilogue(**kw)).values()) == {want}


def test_product_refusals():
    e = epilogue()
    assert set(products(None).values()) == {NULL}
    for kw in (dict(N=0), dict(K=0), dict(K=40), dict(M=-1), dict(M=1 << 31), dict(N=1 << 31), dict(K=1 << 31)):
        assert set(products(e, **kw).values()) == {SHAPE}, kw
    assert products(e, M=0)["q"] == SHAPE and products(e, M=0)["mxq"] == SHAPE
    assert products(e, M=0)["w"] == OK and products(e, M=0, x=None, w=None, y=None)["mxw"] == OK
    assert products(e, K=320)["mxq"] == SHAPE and products(e, K=48, xs=48)["mxw"] == SHAPE
    # a packed operand of 4 GiB: the weight's rows count twice with a gate
    big = dict(N=(1 << 20) - 512, K=8192)
    assert products(e, **big, y=None)["q"] == NULL
    assert products(epilogue(gated=1), **big)["q"] == SHAPE
    assert products(epilogue(gated=1), **big)["mxq"] == SHAPE
    assert products(epilogue(gated=1), N=1 << 30, K=64, xs=64)["w"] == SHAPE
    for name in ("x", "w", "ws", "y"):
        assert set(products(e, **{name: None}).values()) == {NULL}, name
    assert products(e, xsc=None)["q"] == NULL and products(e, xsc=None)["mxq"] == NULL
    assert products(e, xt=None)["q"] == NULL and products(e, wt=None)["q"] == NULL
    assert products(e, wt=None)["w"] == NULL
    for kw in (dict(x=at(8)), dict(w=at(8)), dict(ws=at(2)), dict(y=at(1))):
        assert set(products(e, **kw).values()) == {ALIGN}, kw
    assert set(products(epilogue(out_dtype=0), y=at(2)).values()) == {ALIGN}
    assert products(e, xs=260)["w"] == ALIGN and products(e, xs=248)["mxw"] == SHAPE


def bwd(**kw):
    a = dict(dy=F, z=F, M=4, N=16, act=4, gated=0, dz=F, db=F, t=F, ws=F, wsb=1 << 20) | kw
    return L.fos_epilogue_bwd(a["dy"], a["z"], a["M"], a["N"], a["act"], a["gated"], a["dz"], a["db"],
                              a["t"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(M=0, db=None, t=None, dy=None, z=None, dz=None), OK), (dict(act=5), FLAGS), (dict(act=-1), FLAGS),
    (dict(gated=2), FLAGS), (dict(M=-1), SHAPE), (dict(N=0), SHAPE), (dict(N=1 << 30), SHAPE),
    (dict(M=1 << 31), SHAPE), (dict(M=1 << 20, N=1 << 25), SHAPE), (dict(dy=None), NULL),
    (dict(z=None), NULL), (dict(dz=None), NULL), (dict(dy=at(1)), ALIGN), (dict(z=at(1)), ALIGN),
    (dict(dz=at(1)), ALIGN), (dict(db=at(2)), ALIGN), (dict(t=at(2)), ALIGN), (dict(ws=None), WS),
    (dict(ws=at(8)), WS), (dict(wsb=16), WS),
])
def test_epilogue_bwd_refusals(kw, want):
    assert bwd(**kw) == want


@contextlib.contextmanager
def refused():
    with pytest.raises(ValueError):
        yield


def test_binding_refuses_cpu_tensors_and_bad_names():
    """CPU tensors reach no C call."""
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.ones(64, dtype=torch.bfloat16)
    rec = fos.NVFP4Tensor(torch.zeros(32, 32, dtype=torch.uint8), torch.zeros(32, 4, dtype=torch.uint8),
                          torch.zeros(1))
    mx = fos.MXFP4Tensor(rec.data, torch.zeros(32, 2, dtype=torch.uint8))
    for call in (lambda: fos.rmsnorm_fwd(x, w), lambda: fos.rmsnorm_bwd(x, x, w, torch.zeros(4)),
                 lambda: fos.qlinear_epilogue_fwd(rec, rec), lambda: fos.qlinear_epilogue_fwd(rec, mx),
                 lambda: fos.qglu_fwd(mx, rec), lambda: fos.mx_qglu_fwd(mx, rec), lambda: fos.wglu_fwd(x, mx),
                 lambda: fos.mx_wglu_fwd(x, rec), lambda: fos.mx_qlinear_epilogue_fwd(mx, mx),
                 lambda: fos.qglu_fwd(rec, rec), lambda: fos.mx_qglu_fwd(mx, mx),
                 lambda: fos.wlinear_epilogue_fwd(x, rec), lambda: fos.mx_wlinear_epilogue_fwd(x, mx),
                 lambda: fos.wglu_fwd(x, rec), lambda: fos.mx_wglu_fwd(x, mx),
                 lambda: fos.epilogue_bwd(x, x), lambda: fos.epilogue_bwd(x, x, "tanh"),
                 lambda: fos.qglu_bwd(x, x, None, None), lambda: fos.qlinear_epilogue_bwd(x, x, rec, rec)):
        with refused():
            call()


def test_binding_refuses_outputs_that_overlap_what_is_read():
    flat = torch.zeros(8 * 64, dtype=torch.bfloat16)
    t = flat.view(8, 64)
    ok = fos._no_overlap
    ok(t[1:4], t[1:4], "it")                             # in place
    ok(t[0:4], t[4:8], "it"), ok(t[4:8], t[0:4], "it")    # side by side
    ok(t[:0], t[:0], "it")
    ok(t[:, :32], t[:, :32], "it")                       # equal rows of a wider tensor
    for out, other in ((t[0:4], t[1:5]), (t[1:5], t[0:4]), (t[0:4], t[3:7]),
                       (flat[:256].view(8, 32), t[:, :32]), (flat[:256].view(8, 32), t[:, 32:]),
                       (t[0:1], t.view(torch.int16)[0:1]), (flat[8:72].view(1, 64), t[0:1])):
        with refused():
            ok(out, other, "it")
    with refused():
        ok(t[1:4], t[1:4], "it", whole=False)


def test_calls_run_with_their_device_current(monkeypatch):
    devices = Devices(monkeypatch, current=1)
    seen = []
    entry = lambda *args: seen.append((devices.current, args)) or fos.FOS_OK
    monkeypatch.setattr(fos, "_lib", types.SimpleNamespace(fos_entry=entry))
    monkeypatch.setattr(fos, "_raw_stream", lambda index: 100 + index)
    fos._call(3, "fos_entry", 7)
    fos._call(1, "fos_entry", 8)
    assert seen == [(3, (7, 103)), (1, (8, 101))]
    assert devices.entered == [3] and devices.current == 1
