"""Refusals of the token-serving entry points, which need no GPU: bad arguments get the
documented status before any HIP call (the pointers are never dereferenced), and the
binding refuses tensors that the library could not address."""
import contextlib
import ctypes

import pytest
import torch

from fp4_block_quantization_amd import fos

F = ctypes.c_void_p(0x100000)
MIS = ctypes.c_void_p(0x100002)
L = fos.lib()
OK, NULL, SHAPE, ALIGN, FLAGS, WS = (fos.FOS_OK, fos.FOS_E_NULL, fos.FOS_E_SHAPE, fos.FOS_E_ALIGN,
                                     fos.FOS_E_FLAGS, fos.FOS_E_WORKSPACE)


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("args,want", [
    (dict(M=0), OK), (dict(M=0, x=None, wd=None, y=None), OK),
    (dict(M=-1), SHAPE), (dict(N=0), SHAPE), (dict(K=0), SHAPE), (dict(K=40), SHAPE),
    (dict(M=1 << 31), SHAPE), (dict(N=1 << 31), SHAPE), (dict(K=1 << 31), SHAPE),
    (dict(N=1 << 30, K=1 << 20), SHAPE), (dict(xs=32), SHAPE), (dict(xs=-64), SHAPE),
    (dict(x=None), NULL), (dict(wd=None), NULL), (dict(ws=None), NULL), (dict(y=None), NULL),
    (dict(x=MIS), ALIGN), (dict(xs=68), ALIGN), (dict(wd=MIS), ALIGN), (dict(ws=MIS), ALIGN),
    (dict(bias=ctypes.c_void_p(0x100001)), ALIGN), (dict(y=MIS, out=0), ALIGN),
    (dict(y=ctypes.c_void_p(0x100001)), ALIGN), (dict(out=2), FLAGS), (dict(out=-1), FLAGS),
])
def test_wlinear_refusals(mx, args, want):
    a = dict(x=F, xs=64, wd=F, ws=F, wt=F, bias=None, M=2, N=16, K=64, out=1, y=F) | args
    if mx:
        got = L.fos_mx_wlinear_fwd(a["x"], a["xs"], a["wd"], a["ws"], a["bias"], a["M"], a["N"], a["K"],
                                   a["out"], a["y"], None)
    else:
        got = L.fos_wlinear_fwd(a["x"], a["xs"], a["wd"], a["ws"], a["wt"], a["bias"], a["M"], a["N"],
                                a["K"], a["out"], a["y"], None)
    assert got == want


def test_wlinear_block_and_scale():
    assert L.fos_mx_wlinear_fwd(F, 48, F, F, None, 1, 16, 48, 1, F, None) == SHAPE      # K % 32
    assert L.fos_wlinear_fwd(F, 64, F, F, None, None, 1, 16, 64, 1, F, None) == NULL    # no t
    assert L.fos_wlinear_fwd(F, 64, F, F, MIS, None, 1, 16, 64, 1, F, None) == ALIGN


def cache(**kw):
    a = dict(struct_size=ctypes.sizeof(fos.FosKVCache), format=1, num_pages=8, page_size=16,
             num_kv_heads=2, head_dim=64, reserved=0, k_data=F, v_data=F, k_scales=F, v_scales=F,
             k_tensor_scale=F, v_tensor_scale=F) | kw
    return fos.FosKVCache(**{k: getattr(v, "value", v) for k, v in a.items()})


BAD_CACHES = [
    (dict(struct_size=8), FLAGS), (dict(format=2), FLAGS), (dict(reserved=1), FLAGS),
    (dict(num_pages=-1), SHAPE), (dict(num_pages=1 << 31), SHAPE), (dict(page_size=8), SHAPE),
    (dict(page_size=24), SHAPE), (dict(page_size=8192), SHAPE), (dict(num_kv_heads=0), SHAPE),
    (dict(head_dim=16), SHAPE), (dict(head_dim=80), SHAPE), (dict(head_dim=288), SHAPE),
    (dict(num_pages=1 << 30, num_kv_heads=1024), SHAPE), (dict(num_kv_heads=(1 << 31) - 1, page_size=4096), SHAPE),
    (dict(k_data=None), NULL), (dict(v_data=None), NULL), (dict(k_scales=None), NULL),
    (dict(v_scales=None), NULL), (dict(k_tensor_scale=None), NULL), (dict(v_tensor_scale=None), NULL),
    (dict(k_data=MIS), ALIGN), (dict(v_scales=MIS), ALIGN), (dict(v_tensor_scale=MIS), ALIGN),
]


def append(c=None, rule=0, k=F, ks=128, v=F, vs=128, slots=F, T=4):
    return L.fos_kv_append(None if c is None else ctypes.byref(c), rule, k, ks, v, vs, slots, T, None)


def gather(c=None, k=F, ks=128, v=F, vs=128, slots=F, T=4):
    return L.fos_kv_gather(None if c is None else ctypes.byref(c), slots, T, k, ks, v, vs, None)


BIG = ctypes.c_void_p(0x1000000)


def decode(c, q=F, qs=256, B=2, Hq=4, table=F, ts=3, pages=3, lens=F, scale=0.125, window=0, out=F,
           lse=None, ws=BIG, wsb=None):
    need = L.fos_paged_decode_workspace_bytes(2, 4, 2, 64)
    return L.fos_paged_decode(None if c is None else ctypes.byref(c), q, qs, B, Hq, table, ts, pages,
                              lens, scale, window, out, lse, ws, need if wsb is None else wsb, None)


@pytest.mark.parametrize("kw,want", BAD_CACHES)
def test_cache_refusals(kw, want):
    assert append(cache(**kw)) == want
    assert gather(cache(**kw)) == want
    assert decode(cache(**kw)) == want


def test_cache_of_no_pages_needs_no_memory():
    c = cache(num_pages=0, k_data=None, v_data=None, k_scales=None, v_scales=None,
              k_tensor_scale=None, v_tensor_scale=None)
    assert append(c) == OK                                     # every slot is outside


@pytest.mark.parametrize("call", [append, gather])
def test_rows_refusals(call):
    c = cache()
    assert call(None) == NULL
    assert call(c, T=-1) == SHAPE and call(c, T=1 << 31) == SHAPE
    assert call(c, ks=64) == SHAPE and call(c, vs=120) == SHAPE and call(c, ks=-128) == SHAPE
    assert call(c, ks=132) == ALIGN and call(c, k=MIS) == ALIGN and call(c, v=MIS) == ALIGN
    assert call(c, slots=ctypes.c_void_p(0x100004)) == ALIGN
    assert call(c, k=None) == NULL and call(c, v=None) == NULL and call(c, slots=None) == NULL
    assert call(c, T=0, k=None, v=None, slots=None) == OK
    # more than 2^32 - 1 work-items
    assert call(cache(num_kv_heads=1024, head_dim=256), ks=1 << 18, vs=1 << 18, T=1 << 20) == SHAPE


def test_append_rule():
    assert append(cache(), rule=2) == FLAGS and append(cache(), rule=-1) == FLAGS


def test_decode_refusals():
    c = cache()
    assert decode(None) == NULL
    assert decode(c, B=-1) == SHAPE and decode(c, Hq=3) == SHAPE and decode(c, Hq=0) == SHAPE
    assert decode(c, qs=128) == SHAPE and decode(c, ts=2) == SHAPE and decode(c, pages=-1) == SHAPE
    assert decode(c, pages=1 << 27, ts=1 << 27) == SHAPE       # 2^31 tokens
    assert decode(c, B=1 << 30) == SHAPE
    assert decode(c, window=-1) == FLAGS
    assert decode(c, scale=float("nan")) == FLAGS and decode(c, scale=float("inf")) == FLAGS
    for name in ("q", "table", "lens", "out"):
        assert decode(c, **{name: None}) == NULL, name
        assert decode(c, **{name: MIS}) == ALIGN, name
    assert decode(c, qs=260) == ALIGN and decode(c, lse=MIS) == ALIGN
    assert decode(c, ws=None) == WS and decode(c, ws=ctypes.c_void_p(0x1000010)) == WS
    assert decode(c, wsb=0) == WS
    assert decode(c, B=0, q=None, table=None, lens=None, out=None, ws=None) == OK


def test_decode_workspace_sizes():
    size = L.fos_paged_decode_workspace_bytes
    assert size(1, 1, 1, 32) > 0 and size(0, 8, 8, 128) >= 0
    for bad in ((-1, 8, 8, 128), (1, 0, 1, 128), (1, 8, 0, 128), (1, 8, 3, 128), (1, 8, 8, 0), (1, 8, 8, 512)):
        assert size(*bad) == 0
    assert size(64, 64, 8, 128) < 1 << 30


def bf(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def test_binding_refuses_host_tensors_and_wrong_shapes():
    """Nothing here reaches the library: the tensors are on the host."""
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)
    w = fos.NVFP4Tensor(u8(4, 16), u8(4, 2), torch.zeros(1))
    with pytest.raises(ValueError):
        fos.wlinear_fwd(bf(1, 32), w)
    with pytest.raises(ValueError):
        fos.mx_wlinear_fwd(bf(1, 32), fos.MXFP4Tensor(u8(4, 16), u8(4, 1)))
    with pytest.raises(ValueError, match="Hadamard"):
        fos.wlinear_fwd(bf(1, 32), fos.NVFP4Tensor(u8(4, 16), u8(4, 2), torch.zeros(1), hadamard_seed=3))
    with pytest.raises(ValueError):
        fos.PagedKVCache(bf(2, 2, 16, 64), bf(2, 2, 16, 64))
    with pytest.raises(ValueError):
        fos.PagedKVCache(bf(2, 2, 16, 64).float(), bf(2, 2, 16, 64).float())
    with pytest.raises(ValueError):
        fos.kv_cache(2, 16, 2, 64, format="fp8", device="cpu")
    with pytest.raises(ValueError):
        fos.kv_cache(2, 16, 2, 64, format="nvfp4", device="cpu")    # no tensor scales


def test_too_many_kv_heads():
    """More than 65536 kv heads are refused by every call, also with no page and one token."""
    c = cache(num_kv_heads=65537, num_pages=0, head_dim=32)
    width = 65537 * 32
    assert append(c, ks=width, vs=width, T=1) == SHAPE
    assert gather(c, ks=width, vs=width, T=1) == SHAPE
    assert gather(cache(num_kv_heads=65536, num_pages=0, head_dim=32), T=0) == OK


class Devices:
    """torch.cuda.device as a record of what was made current."""

    def __init__(self, monkeypatch, current):
        self.current, self.entered = current, []
        monkeypatch.setattr(fos, "_current_device", lambda: self.current)
        monkeypatch.setattr(torch.cuda, "device", self.enter)

    @contextlib.contextmanager
    def enter(self, index):
        before, self.current = self.current, index
        self.entered.append(index)
        yield
        self.current = before


def test_calls_run_with_their_device_current(monkeypatch):
    devices = Devices(monkeypatch, current=1)
    report = lambda *args: (devices.current, args)
    assert fos._on(3, report)("a", 2) == (3, ("a", 2))
    assert devices.entered == [3] and devices.current == 1
