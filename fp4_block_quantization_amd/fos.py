"""Thin ctypes binding of libfos.so (the C ABI declared in include/fos.h).

Argument marshalling only: every step of quantize / dequantize / qlinear runs in the
library's HIP kernels.  PyTorch provides device memory and the current HIP stream.
There is no fallback: if libfos.so is missing or fails to load, importing this
module raises.

Low-level functions carry the C names (fos_quantize, fos_dequantize, ...) and take
device tensors; ``quantize`` / ``dequantize`` / ``qlinear_fwd`` allocate the outputs.
The calls that serve one token at a time run on their tensors' device; all others want it to
be the current one (``torch.cuda.device``).
"""
from __future__ import annotations

import ctypes
import functools
import os
from dataclasses import dataclass
from typing import Optional, Sequence, Tuple, Union

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfos.so")

FOS_OK, FOS_E_NULL, FOS_E_SHAPE, FOS_E_ALIGN, FOS_E_FLAGS, FOS_E_WORKSPACE, FOS_E_HIP = range(7)
FOS_RULE_4OVER6, FOS_RULE_6ONLY = 0, 1
FOS_ROUND_RNE, FOS_ROUND_STOCHASTIC, FOS_ROUND_STOCHASTIC_FULL = 0, 1, 2
FOS_BLOCK_1D, FOS_BLOCK_2D = 0, 1
FOS_OUT_ROWWISE, FOS_OUT_COLWISE = 1, 2
FOS_OUT_F32, FOS_OUT_BF16 = 0, 1
FOS_KV_BF16, FOS_KV_NVFP4 = 0, 1


class FosError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {_lib.fos_status_string(status).decode()} (status {status})")


class FosQuantConfig(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_uint32), ("rule", ctypes.c_uint32),
                ("rounding", ctypes.c_uint32), ("block", ctypes.c_uint32),
                ("outputs", ctypes.c_uint32), ("hadamard", ctypes.c_uint32),
                ("hadamard_seed", ctypes.c_uint64), ("sr_seed", ctypes.c_uint64)]


class FosKVCache(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_uint32), ("format", ctypes.c_uint32),
                ("num_pages", ctypes.c_int64), ("page_size", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("k_data", ctypes.c_void_p),
                ("v_data", ctypes.c_void_p), ("k_scales", ctypes.c_void_p),
                ("v_scales", ctypes.c_void_p), ("k_tensor_scale", ctypes.c_void_p),
                ("v_tensor_scale", ctypes.c_void_p)]


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built; run `python -m fp4_block_quantization_amd.build`")
    lib = ctypes.CDLL(LIB_PATH)
    P, I64, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t
    cfgp = ctypes.POINTER(FosQuantConfig)
    cachep = ctypes.POINTER(FosKVCache)
    sigs = {
        "fos_abi_version": ([], ctypes.c_int),
        "fos_status_string": ([ctypes.c_int], ctypes.c_char_p),
        "fos_quantize_workspace_bytes": ([], SZ),
        "fos_workspace_bytes": ([], SZ),
        "fos_tensor_scale": ([cfgp, P, I64, I64, P, P, SZ, P], ctypes.c_int),
        "fos_quantize_scaled": ([cfgp, P, I64, I64, P, P, P, P, P, P], ctypes.c_int),
        "fos_quantize": ([cfgp, P, I64, I64, P, P, P, P, P, P, SZ, P], ctypes.c_int),
        "fos_quantize_noalloc": ([cfgp, P, I64, I64, P, P, P, P, P, P], ctypes.c_int),
        "fos_selftest_e4m3": ([P, P], ctypes.c_int),
        "fos_selftest_e2m1": ([P, P], ctypes.c_int),
        "fos_selftest_e2m1_sr": ([P, P], ctypes.c_int),
        "fos_selftest_e2m1_sr_full": ([P, P], ctypes.c_int),
        "fos_dequantize": ([P, P, P, I64, I64, ctypes.c_int, P, P], ctypes.c_int),
        "fos_dequantize_hadamard": ([P, P, P, I64, I64, ctypes.c_uint64, ctypes.c_int, P, P],
                                    ctypes.c_int),
        "fos_qlinear_fwd": ([P, P, P, P, P, P, I64, I64, I64, P, P], ctypes.c_int),
        "fos_qlinear_bwd": ([P] * 12 + [I64, I64, I64, P, P, P], ctypes.c_int),
        "fos_qlinear_act_workspace_bytes": ([I64, I64], SZ),
        "fos_qlinear_fwd_act": ([cfgp, P, P, ctypes.c_int, P, P, P, I64, I64, I64, P, P, SZ, P],
                                ctypes.c_int),
        "fos_mx_quantize": ([P, I64, I64, P, P, P], ctypes.c_int),
        "fos_mx_dequantize": ([P, P, I64, I64, ctypes.c_int, P, P], ctypes.c_int),
        "fos_mx_qlinear_fwd": ([P, P, P, P, I64, I64, I64, P, P], ctypes.c_int),
        "fos_wlinear_fwd": ([P, I64, P, P, P, P, I64, I64, I64, ctypes.c_int, P, P], ctypes.c_int),
        "fos_mx_wlinear_fwd": ([P, I64, P, P, P, I64, I64, I64, ctypes.c_int, P, P], ctypes.c_int),
        "fos_kv_append": ([cachep, ctypes.c_int, P, I64, P, I64, P, I64, P], ctypes.c_int),
        "fos_kv_gather": ([cachep, P, I64, P, I64, P, I64, P], ctypes.c_int),
        "fos_paged_decode_workspace_bytes": ([I64, I64, I64, I64], SZ),
        "fos_paged_decode_counter_bytes": ([], SZ),
        "fos_paged_decode": ([cachep, P, I64, I64, I64, P, I64, I64, P, ctypes.c_float, I64, P, P,
                              P, SZ, P], ctypes.c_int),
    }
    for name, (args, res) in sigs.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    return lib


_lib = _load()
ABI_VERSION = _lib.fos_abi_version()


def lib() -> ctypes.CDLL:
    return _lib


# ---------------------------------------------------------------- marshalling helpers

def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device) -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _check(status: int, what: str):
    if status != FOS_OK:
        raise FosError(status, what)


def make_config(rule: str = "4/6", rounding: str = "rne", block: str = "1d",
                outputs: Sequence[str] = ("row",), hadamard_seed: Optional[int] = None,
                sr_seed: Optional[int] = None) -> FosQuantConfig:
    rules = {"4/6": FOS_RULE_4OVER6, "6": FOS_RULE_6ONLY}
    roundings = {"rne": FOS_ROUND_RNE, "sr": FOS_ROUND_STOCHASTIC,
                 "sr_full": FOS_ROUND_STOCHASTIC_FULL}
    blocks = {"1d": FOS_BLOCK_1D, "2d": FOS_BLOCK_2D}
    out = 0
    for o in outputs:
        out |= {"row": FOS_OUT_ROWWISE, "col": FOS_OUT_COLWISE}[o]
    if rounding in ("sr", "sr_full") and sr_seed is None:
        raise ValueError("stochastic rounding needs sr_seed")
    return FosQuantConfig(ctypes.sizeof(FosQuantConfig), rules[rule], roundings[rounding],
                          blocks[block], out, 0 if hadamard_seed is None else 1,
                          0 if hadamard_seed is None else int(hadamard_seed) & (2 ** 64 - 1),
                          0 if sr_seed is None else int(sr_seed) & (2 ** 64 - 1))


_workspaces = {}


def workspace(device: torch.device) -> torch.Tensor:
    """Scratch workspace for the current stream of ``device`` (one per stream, so
    that calls on different streams never share one; its contents are scratch)."""
    device = torch.device(device)
    key = (device.index, torch.cuda.current_stream(device).cuda_stream)
    ws = _workspaces.get(key)
    if ws is None:
        ws = torch.zeros(int(_lib.fos_quantize_workspace_bytes()), dtype=torch.uint8, device=device)
        _workspaces[key] = ws
    return ws


# ---------------------------------------------------------------- C-named wrappers

def fos_tensor_scale(cfg: FosQuantConfig, x: torch.Tensor, tensor_scale: torch.Tensor,
                     ws: Optional[torch.Tensor] = None) -> None:
    ws = workspace(x.device) if ws is None else ws
    _check(_lib.fos_tensor_scale(ctypes.byref(cfg), _ptr(x), x.shape[0], x.shape[1],
                                 _ptr(tensor_scale), _ptr(ws), ws.numel(), _stream(x.device)),
           "fos_tensor_scale")


def fos_quantize_scaled(cfg: FosQuantConfig, x: torch.Tensor, tensor_scale: torch.Tensor,
                        row_data=None, row_scales=None, col_data=None, col_scales=None) -> None:
    _check(_lib.fos_quantize_scaled(ctypes.byref(cfg), _ptr(x), x.shape[0], x.shape[1],
                                    _ptr(tensor_scale), _ptr(row_data), _ptr(row_scales),
                                    _ptr(col_data), _ptr(col_scales), _stream(x.device)),
           "fos_quantize_scaled")


def fos_quantize(cfg: FosQuantConfig, x: torch.Tensor, row_data, row_scales, col_data,
                 col_scales, tensor_scale: torch.Tensor,
                 ws: Optional[torch.Tensor] = None) -> None:
    ws = workspace(x.device) if ws is None else ws
    _check(_lib.fos_quantize(ctypes.byref(cfg), _ptr(x), x.shape[0], x.shape[1],
                             _ptr(row_data), _ptr(row_scales), _ptr(col_data), _ptr(col_scales),
                             _ptr(tensor_scale), _ptr(ws), ws.numel(), _stream(x.device)),
           "fos_quantize")


def fos_quantize_noalloc(cfg: FosQuantConfig, x: torch.Tensor, row_data, row_scales, col_data,
                         col_scales, tensor_scale: torch.Tensor) -> None:
    """fos_quantize without a workspace: the library's own per-GPU scratch array holds
    the tensor-scale pass's partial maxima (calls on one GPU must not overlap)."""
    _check(_lib.fos_quantize_noalloc(ctypes.byref(cfg), _ptr(x), x.shape[0], x.shape[1],
                                     _ptr(row_data), _ptr(row_scales), _ptr(col_data),
                                     _ptr(col_scales), _ptr(tensor_scale), _stream(x.device)),
           "fos_quantize_noalloc")


def selftest_e4m3(device="cuda:0") -> int:
    """Number of fp32 values in [0, 448] whose hardware E4M3 conversion (used by the
    quantize kernels for the block scales) differs from the bit-level rule; 0 on a
    correct device."""
    n = torch.zeros(1, dtype=torch.int64, device=device)
    _check(_lib.fos_selftest_e4m3(_ptr(n), _stream(n.device)), "fos_selftest_e4m3")
    return int(n.item())


def selftest_e2m1(device="cuda:0") -> int:
    """Number of finite fp32 values whose hardware E2M1 conversion (used by the quantize
    kernels for the element codes) differs from the rounding rule; 0 on a correct
    device."""
    n = torch.zeros(1, dtype=torch.int64, device=device)
    _check(_lib.fos_selftest_e2m1(_ptr(n), _stream(n.device)), "fos_selftest_e2m1")
    return int(n.item())


def selftest_e2m1_sr(device="cuda:0") -> int:
    """Number of (finite fp32 value, draw byte, pair position) cases where the
    hardware stochastic rounding to E2M1, under the operands the quantize kernels
    build from their draws, differs from the draw rule; 0 on a correct device."""
    n = torch.zeros(1, dtype=torch.int64, device=device)
    _check(_lib.fos_selftest_e2m1_sr(_ptr(n), _stream(n.device)), "fos_selftest_e2m1_sr")
    return int(n.item())


def selftest_e2m1_sr_full(device="cuda:0") -> int:
    """Number of disagreements at the rounding boundary of the full-resolution
    stochastic rounding (every finite fp32 value, both pair positions); 0 on a
    correct device."""
    n = torch.zeros(1, dtype=torch.int64, device=device)
    _check(_lib.fos_selftest_e2m1_sr_full(_ptr(n), _stream(n.device)), "fos_selftest_e2m1_sr_full")
    return int(n.item())


def fos_dequantize(data: torch.Tensor, scales: torch.Tensor, tensor_scale: torch.Tensor,
                   rows: int, cols: int, out: torch.Tensor) -> None:
    dt = {torch.float32: FOS_OUT_F32, torch.bfloat16: FOS_OUT_BF16}[out.dtype]
    _check(_lib.fos_dequantize(_ptr(data), _ptr(scales), _ptr(tensor_scale), rows, cols, dt,
                               _ptr(out), _stream(out.device)), "fos_dequantize")


def fos_dequantize_hadamard(data: torch.Tensor, scales: torch.Tensor, tensor_scale: torch.Tensor,
                            rows: int, cols: int, hadamard_seed: int, out: torch.Tensor) -> None:
    dt = {torch.float32: FOS_OUT_F32, torch.bfloat16: FOS_OUT_BF16}[out.dtype]
    _check(_lib.fos_dequantize_hadamard(_ptr(data), _ptr(scales), _ptr(tensor_scale), rows, cols,
                                        hadamard_seed, dt, _ptr(out), _stream(out.device)),
           "fos_dequantize_hadamard")


def fos_qlinear_fwd(x_data, x_scales, x_t, w_data, w_scales, w_t, M: int, N: int, K: int,
                    y: torch.Tensor) -> None:
    _check(_lib.fos_qlinear_fwd(_ptr(x_data), _ptr(x_scales), _ptr(x_t), _ptr(w_data),
                                _ptr(w_scales), _ptr(w_t), M, N, K, _ptr(y), _stream(y.device)),
           "fos_qlinear_fwd")


def fos_qlinear_bwd(dy, dyt, xt, wt, M: int, N: int, K: int, dx: Optional[torch.Tensor],
                    dw: Optional[torch.Tensor]) -> None:
    """dy, dyt, xt, wt: (data, scales, tensor_scale) triples (a skipped product's
    operands may be None)."""
    def trip(r):
        return [_ptr(v) for v in r] if r is not None else [_ptr(None)] * 3
    dev = (dx if dx is not None else dw).device
    _check(_lib.fos_qlinear_bwd(*trip(dy), *trip(dyt), *trip(xt), *trip(wt), M, N, K, _ptr(dx),
                                _ptr(dw), _stream(dev)), "fos_qlinear_bwd")


def fos_qlinear_fwd_act(cfg: FosQuantConfig, x: torch.Tensor, x_t: torch.Tensor,
                        x_scale_given: bool, w_data, w_scales, w_t, N: int, y: torch.Tensor,
                        ws: torch.Tensor) -> None:
    M, K = x.shape
    _check(_lib.fos_qlinear_fwd_act(ctypes.byref(cfg), _ptr(x), _ptr(x_t), int(bool(x_scale_given)),
                                    _ptr(w_data), _ptr(w_scales), _ptr(w_t), M, N, K, _ptr(y),
                                    _ptr(ws), ws.numel(), _stream(x.device)),
           "fos_qlinear_fwd_act")


# ---------------------------------------------------------------- tensor-level API

@dataclass
class NVFP4Tensor:
    """One NVFP4 record: data [R, C/2] nibbles, scales [R, C/16] E4M3 bytes, and the
    per-tensor fp32 scale (device tensor of one element).  ``layout`` is "row" for
    the row-wise record of X and "col" for the record of X^T."""
    data: torch.Tensor
    scales: torch.Tensor
    tensor_scale: torch.Tensor
    layout: str = "row"
    block: str = "1d"
    hadamard_seed: Optional[int] = None

    @property
    def shape(self) -> Tuple[int, int]:
        return (self.data.shape[0], self.data.shape[1] * 2)


def _check_input(x: torch.Tensor):
    if x.dim() != 2 or x.dtype != torch.bfloat16 or not x.is_cuda or not x.is_contiguous():
        raise ValueError("x must be a contiguous 2-D bfloat16 CUDA tensor")


def _check_record(q, *others):
    """A record's tensors must be contiguous CUDA tensors on one device (the library
    dereferences them on the GPU), with the shapes the layout implies."""
    dev = q.data.device
    tensors = [q.data, q.scales] + ([q.tensor_scale] if hasattr(q, "tensor_scale") else [])
    for o in others:
        tensors += [o.data, o.scales] + ([o.tensor_scale] if hasattr(o, "tensor_scale") else [])
    for t in tensors:
        if not t.is_cuda or t.device != dev or not t.is_contiguous():
            raise ValueError("record tensors must be contiguous CUDA tensors on one device")
    for r in (q,) + others:
        if r.data.dtype != torch.uint8 or r.scales.dtype != torch.uint8 or r.data.dim() != 2:
            raise ValueError("record data and scales must be 2-D uint8 tensors")
        block = 32 if not hasattr(r, "tensor_scale") else 16
        R, C = r.shape
        if tuple(r.scales.shape) != (R, C // block):
            raise ValueError(f"scales must be [{R}, {C // block}]")


def tensor_scale(x: torch.Tensor, hadamard_seed: Optional[int] = None,
                 outputs: Sequence[str] = ("row",), out: Optional[torch.Tensor] = None
                 ) -> torch.Tensor:
    """The per-tensor FP32 scale t of x (device fp32 [1]), on the current stream;
    ``out``: optional destination."""
    _check_input(x)
    cfg = make_config(outputs=outputs, hadamard_seed=hadamard_seed)
    t = out if out is not None else torch.empty(1, dtype=torch.float32, device=x.device)
    if t.dtype != torch.float32 or t.numel() != 1 or t.device != x.device:
        raise ValueError("out must be a one-element fp32 tensor on x's device")
    fos_tensor_scale(cfg, x, t)
    return t


def quantize(x: torch.Tensor, rule: str = "4/6", rounding: str = "rne", block: str = "1d",
             outputs: Sequence[str] = ("row",), hadamard_seed: Optional[int] = None,
             sr_seed: Optional[int] = None, tensor_scale: Optional[torch.Tensor] = None
             ) -> Union[NVFP4Tensor, Tuple[NVFP4Tensor, NVFP4Tensor]]:
    """4/6 NVFP4 quantization of a bf16 [R, C] tensor.  Returns the row-wise record,
    the column-wise record (quantization of X^T), or both as (row, col).  With
    ``tensor_scale`` given (device fp32 [1]) the amax pass is skipped."""
    _check_input(x)
    cfg = make_config(rule, rounding, block, outputs, hadamard_seed, sr_seed)
    R, C = x.shape
    dev = x.device
    u8 = dict(dtype=torch.uint8, device=dev)
    rd = rs = cd = cs = None
    if "row" in outputs:
        rd, rs = torch.empty(R, C // 2, **u8), torch.empty(R, C // 16, **u8)
    if "col" in outputs:
        cd, cs = torch.empty(C, R // 2, **u8), torch.empty(C, R // 16, **u8)
    if tensor_scale is None:
        t = torch.empty(1, dtype=torch.float32, device=dev)
        fos_quantize(cfg, x, rd, rs, cd, cs, t)
    else:
        t = tensor_scale
        fos_quantize_scaled(cfg, x, t, rd, rs, cd, cs)
    res = []
    if rd is not None:
        res.append(NVFP4Tensor(rd, rs, t, "row", block, hadamard_seed))
    if cd is not None:
        res.append(NVFP4Tensor(cd, cs, t, "col", block, hadamard_seed))
    return res[0] if len(res) == 1 else tuple(res)


def dequantize(q: NVFP4Tensor, dtype: torch.dtype = torch.float32,
               inverse_hadamard: bool = False) -> torch.Tensor:
    """Dequantize a record ([R, C] as stored).  With ``inverse_hadamard`` a record made
    with the random Hadamard transform is returned to the original basis."""
    _check_record(q)
    R, C = q.shape
    out = torch.empty(R, C, dtype=dtype, device=q.data.device)
    if inverse_hadamard:
        if q.hadamard_seed is None:
            raise ValueError("the record was not made with the Hadamard transform")
        fos_dequantize_hadamard(q.data, q.scales, q.tensor_scale, R, C, q.hadamard_seed, out)
    else:
        fos_dequantize(q.data, q.scales, q.tensor_scale, R, C, out)
    return out


def qlinear_fwd(xq: NVFP4Tensor, wq: NVFP4Tensor, out: Optional[torch.Tensor] = None
                ) -> torch.Tensor:
    """Y = deq(A) deq(B)^T in bf16 for two records blocked along their shared inner
    dimension: A [M, K], B [N, K] as stored (a column-wise record of W is the record
    of W^T; 2D records carry one scale per 16 values too).  ``out``: optional bf16
    [M, N] destination."""
    _check_record(xq, wq)
    M, K = xq.shape
    N, K2 = wq.shape
    if K != K2:
        raise ValueError("inner dimensions differ")
    y = out if out is not None else torch.empty(M, N, dtype=torch.bfloat16,
                                                device=xq.data.device)
    if y.shape != (M, N) or y.dtype != torch.bfloat16 or not y.is_contiguous():
        raise ValueError("out must be a contiguous bf16 [M, N] tensor")
    fos_qlinear_fwd(xq.data, xq.scales, xq.tensor_scale, wq.data, wq.scales, wq.tensor_scale,
                    M, N, K, y)
    return y


def qlinear_act_workspace(M: int, K: int, device) -> torch.Tensor:
    """A workspace for qlinear_fwd_act on X [M, K] (torch allocations are 256-byte
    aligned)."""
    n = int(_lib.fos_qlinear_act_workspace_bytes(M, K))
    if n == 0:
        raise ValueError("unsupported activation shape")
    return torch.empty(n, dtype=torch.uint8, device=device)


def act_record(ws: torch.Tensor, M: int, K: int, tensor_scale: torch.Tensor,
               block: str = "1d", hadamard_seed: Optional[int] = None) -> NVFP4Tensor:
    """Views of the record of X that qlinear_fwd_act leaves in its workspace."""
    up = lambda v: (v + 255) // 256 * 256
    nd, ns = M * K // 2, M * K // 16
    data = ws[:nd].view(M, K // 2)
    scales = ws[up(nd):up(nd) + ns].view(M, K // 16)
    return NVFP4Tensor(data, scales, tensor_scale, "row", block, hadamard_seed)


def qlinear_fwd_act(x: torch.Tensor, wq: NVFP4Tensor, rule: str = "4/6", rounding: str = "rne",
                    block: str = "1d", hadamard_seed: Optional[int] = None,
                    sr_seed: Optional[int] = None, x_tensor_scale: Optional[torch.Tensor] = None,
                    out: Optional[torch.Tensor] = None, return_record: bool = False):
    """Y = deq(Q(X)) deq(Wq)^T in bf16 from a bf16 activation X [M, K] and a weight
    record Wq [N, K]: X is quantized with the given options inside the call.  With
    ``x_tensor_scale`` (device fp32 [1], e.g. a delayed scale) X is read once;
    otherwise its tensor scale is computed.  ``return_record`` also returns X's
    record (views of a fresh workspace)."""
    _check_input(x)
    _check_record(wq)
    M, K = x.shape
    N, K2 = wq.shape
    if K != K2:
        raise ValueError("inner dimensions differ")
    if wq.data.device != x.device:
        raise ValueError("x and the weight record are on different devices")
    cfg = make_config(rule, rounding, block, ("row",), hadamard_seed, sr_seed)
    y = out if out is not None else torch.empty(M, N, dtype=torch.bfloat16, device=x.device)
    if y.shape != (M, N) or y.dtype != torch.bfloat16 or not y.is_contiguous():
        raise ValueError("out must be a contiguous bf16 [M, N] tensor")
    given = x_tensor_scale is not None
    t = x_tensor_scale if given else torch.empty(1, dtype=torch.float32, device=x.device)
    ws = qlinear_act_workspace(M, K, x.device)
    fos_qlinear_fwd_act(cfg, x, t, given, wq.data, wq.scales, wq.tensor_scale, N, y, ws)
    if return_record:
        return y, act_record(ws, M, K, t, block, hadamard_seed)
    return y


def qlinear_bwd(dyq: Optional[NVFP4Tensor], dyq_t: Optional[NVFP4Tensor],
                xq_t: Optional[NVFP4Tensor], wq_t: Optional[NVFP4Tensor],
                need_dx: bool = True, need_dw: bool = True
                ) -> Tuple[Optional[torch.Tensor], Optional[torch.Tensor]]:
    """Backward of Y = X W^T from NVFP4 records: dX = deq(dY) deq(W^T)^T and
    dW = deq(dY^T) deq(X^T)^T (bf16).  dyq: row-wise record of dY [M, N]; dyq_t,
    xq_t, wq_t: column-wise records of dY, X and W (records of dY^T [N, M], X^T [K, M],
    W^T [K, N])."""
    if not (need_dx or need_dw):
        raise ValueError("nothing to compute")
    used = ([dyq, wq_t] if need_dx else []) + ([dyq_t, xq_t] if need_dw else [])
    _check_record(*used)
    if need_dx:
        M, N = dyq.shape
        K, N2 = wq_t.shape
        if N2 != N:
            raise ValueError("dY and W disagree on N")
    if need_dw:
        N3, M3 = dyq_t.shape
        K3, M4 = xq_t.shape
        if M3 != M4:
            raise ValueError("dY and X disagree on M")
        if need_dx and (N3 != N or M3 != M or K3 != K):
            raise ValueError("inconsistent shapes")
        M, N, K = M3, N3, K3
    ref = dyq if need_dx else dyq_t
    dev = ref.data.device
    dx = torch.empty(M, K, dtype=torch.bfloat16, device=dev) if need_dx else None
    dw = torch.empty(N, K, dtype=torch.bfloat16, device=dev) if need_dw else None
    trip = lambda q: (q.data, q.scales, q.tensor_scale) if q is not None else None
    fos_qlinear_bwd(trip(dyq) if need_dx else None, trip(dyq_t) if need_dw else None,
                    trip(xq_t) if need_dw else None, trip(wq_t) if need_dx else None,
                    M, N, K, dx, dw)
    return dx, dw


# ---------------------------------------------------------------- MXFP4

@dataclass
class MXFP4Tensor:
    """One MXFP4 record: data [R, C/2] nibbles and scales [R, C/32] E8M0 bytes."""
    data: torch.Tensor
    scales: torch.Tensor

    @property
    def shape(self) -> Tuple[int, int]:
        return (self.data.shape[0], self.data.shape[1] * 2)


def mx_quantize(x: torch.Tensor) -> MXFP4Tensor:
    """MXFP4 quantization of a bf16 [R, C] tensor (C % 32 == 0)."""
    _check_input(x)
    R, C = x.shape
    u8 = dict(dtype=torch.uint8, device=x.device)
    data, scales = torch.empty(R, C // 2, **u8), torch.empty(R, C // 32, **u8)
    _check(_lib.fos_mx_quantize(_ptr(x), R, C, _ptr(data), _ptr(scales), _stream(x.device)),
           "fos_mx_quantize")
    return MXFP4Tensor(data, scales)


def mx_dequantize(q: MXFP4Tensor, dtype: torch.dtype = torch.float32) -> torch.Tensor:
    _check_record(q)
    R, C = q.shape
    out = torch.empty(R, C, dtype=dtype, device=q.data.device)
    dt = {torch.float32: FOS_OUT_F32, torch.bfloat16: FOS_OUT_BF16}[dtype]
    _check(_lib.fos_mx_dequantize(_ptr(q.data), _ptr(q.scales), R, C, dt, _ptr(out),
                                  _stream(out.device)), "fos_mx_dequantize")
    return out


def mx_qlinear_fwd(aq: MXFP4Tensor, bq: MXFP4Tensor, out: Optional[torch.Tensor] = None
                   ) -> torch.Tensor:
    """Y = deq(A) deq(B)^T in bf16 on the FP4 matrix cores; A [M, K], B [N, K]."""
    _check_record(aq, bq)
    M, K = aq.shape
    N, K2 = bq.shape
    if K != K2:
        raise ValueError("inner dimensions differ")
    y = out if out is not None else torch.empty(M, N, dtype=torch.bfloat16, device=aq.data.device)
    if y.shape != (M, N) or y.dtype != torch.bfloat16 or not y.is_contiguous():
        raise ValueError("out must be a contiguous bf16 [M, N] tensor")
    _check(_lib.fos_mx_qlinear_fwd(_ptr(aq.data), _ptr(aq.scales), _ptr(bq.data), _ptr(bq.scales),
                                   M, N, K, _ptr(y), _stream(y.device)), "fos_mx_qlinear_fwd")
    return y


# ---------------------------------------------------------------- serving one token at a time
# These calls run once per layer and token, so their wrappers marshal raw addresses and
# check no more than the library needs to stay inside its tensors.  A call on a small
# problem takes as long as its launch (3 of 6 to 8 us) and what happens here, so devices are
# compared by index and a tensor's shape and stride are taken once.
_BF16, _U8, _F32, _I32, _I64 = (torch.bfloat16, torch.uint8, torch.float32, torch.int32,
                                torch.int64)

# The handle of a device's current stream; torch's own accessor where this build of torch
# has it (0.1 us; building a Stream object for it takes 1.9 us of a call's 10).
_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _raw_stream(index: int) -> int:
    if _current_raw_stream is None:
        return torch.cuda.current_stream(index).cuda_stream
    return _current_raw_stream(index)


_is_capturing = getattr(torch._C, "_cuda_isCurrentStreamCapturing",
                        torch.cuda.is_current_stream_capturing)


# A launch goes to the current device, whichever device its stream and its tensors are of.
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _with_device(index: int, fn, *args):
    with torch.cuda.device(index):
        return fn(*args)


def _on(index: int, fn):
    """fn, called with device ``index`` as the current one."""
    return functools.partial(_with_device, index, fn)


_OUT_CODE = {torch.float32: FOS_OUT_F32, torch.bfloat16: FOS_OUT_BF16}


def _wlinear_args(x, wq, bias, out_dtype, out, block):
    """Checked (device, M, N, K, row stride, y) of a weight-only product."""
    data, scales = wq.data, wq.scales
    dev, strides = data.get_device(), x.stride()
    if len(strides) != 2 or strides[1] != 1 or x.dtype != _BF16 or x.get_device() < 0:
        raise ValueError("x must be a 2-D bfloat16 CUDA tensor with contiguous rows")
    M, K = x.shape
    N, half = data.shape
    if K != 2 * half:
        raise ValueError("inner dimensions differ")
    if (data.dtype != _U8 or scales.dtype != _U8 or not data.is_contiguous()
            or not scales.is_contiguous() or scales.shape != (N, K // block)):
        raise ValueError(f"the record must be contiguous uint8 data [N, K/2] and scales [N, K/{block}]")
    if x.get_device() != dev or scales.get_device() != dev:
        raise ValueError("x and the weight record are on different devices")
    if bias is not None and (bias.shape != (N,) or bias.dtype != _BF16
                             or bias.get_device() != dev or not bias.is_contiguous()):
        raise ValueError("bias must be a contiguous bf16 [N] tensor on x's device")
    if out is None:
        if out_dtype not in _OUT_CODE:
            raise ValueError("out_dtype must be torch.bfloat16 or torch.float32")
        out = x.new_empty(M, N) if out_dtype == _BF16 else x.new_empty(M, N, dtype=out_dtype)
    elif (out.shape != (M, N) or out.dtype != out_dtype or out_dtype not in _OUT_CODE
          or out.get_device() != dev or not out.is_contiguous()):
        raise ValueError("out must be a contiguous [M, N] tensor of out_dtype on x's device")
    return dev, M, N, K, (strides[0] if M > 1 else K), out


def wlinear_fwd(x: torch.Tensor, wq: NVFP4Tensor, bias: Optional[torch.Tensor] = None,
                out_dtype: torch.dtype = torch.bfloat16, out: Optional[torch.Tensor] = None
                ) -> torch.Tensor:
    """Y = X deq(W)^T (+ bias) for a bf16 activation X [M, K], which is not quantized, and
    a weight record W [N, K]: the layer of a decode step (M = the sequences of the
    batch; made for up to 64; from several hundred on, ``dequantize`` and a dense product
    are faster).  X's rows may be strided.  ``bias``: bf16 [N];
    ``out``: optional [M, N] destination of ``out_dtype`` (bf16 or fp32)."""
    if wq.hadamard_seed is not None:
        raise ValueError("the weight record carries a Hadamard transform that x does not")
    t = wq.tensor_scale
    if t.dtype != _F32 or t.numel() != 1 or t.get_device() != x.get_device():
        raise ValueError("tensor_scale must be a one-element fp32 tensor on x's device")
    dev, M, N, K, stride, y = _wlinear_args(x, wq, bias, out_dtype, out, 16)
    call = _lib.fos_wlinear_fwd
    if dev != _current_device():
        call = _on(dev, call)
    _check(call(x.data_ptr(), stride, wq.data.data_ptr(), wq.scales.data_ptr(),
                t.data_ptr(), None if bias is None else bias.data_ptr(), M, N, K,
                _OUT_CODE[out_dtype], y.data_ptr(), _raw_stream(dev)),
           "fos_wlinear_fwd")
    return y


def mx_wlinear_fwd(x: torch.Tensor, wq: MXFP4Tensor, bias: Optional[torch.Tensor] = None,
                   out_dtype: torch.dtype = torch.bfloat16, out: Optional[torch.Tensor] = None
                   ) -> torch.Tensor:
    """wlinear_fwd for an MXFP4 weight record."""
    dev, M, N, K, stride, y = _wlinear_args(x, wq, bias, out_dtype, out, 32)
    call = _lib.fos_mx_wlinear_fwd
    if dev != _current_device():
        call = _on(dev, call)
    _check(call(x.data_ptr(), stride, wq.data.data_ptr(), wq.scales.data_ptr(),
                None if bias is None else bias.data_ptr(), M, N, K,
                _OUT_CODE[out_dtype], y.data_ptr(), _raw_stream(dev)),
           "fos_mx_wlinear_fwd")
    return y


class PagedKVCache:
    """A paged key-value cache over caller-owned CUDA tensors (not copied; they must not
    be replaced afterwards): k, v [pages, kv heads, page size, head dim] bf16, or, for
    an NVFP4 cache, uint8 nibbles [.., head dim / 2] with k_scales, v_scales uint8
    [.., head dim / 16] and the static tensor scales k_tensor_scale, v_tensor_scale
    (fp32 [1]).  ``kv_cache`` allocates one."""

    __slots__ = ("k", "v", "k_scales", "v_scales", "k_tensor_scale", "v_tensor_scale",
                 "num_pages", "num_kv_heads", "page_size", "head_dim", "format", "device", "_index", "_c",
                 "_ref")

    def __init__(self, k, v, k_scales=None, v_scales=None, k_tensor_scale=None,
                 v_tensor_scale=None):
        nvfp4 = k.dtype == torch.uint8
        if not nvfp4 and k.dtype != torch.bfloat16:
            raise ValueError("k and v must be bf16, or uint8 nibbles")
        if k.dim() != 4 or k.shape != v.shape or k.dtype != v.dtype:
            raise ValueError("k and v must be [pages, kv heads, page size, ..] of one shape and type")
        P, H, S, D = k.shape
        D = 2 * D if nvfp4 else D
        tensors = [k, v]
        if nvfp4:
            if None in (k_scales, v_scales, k_tensor_scale, v_tensor_scale):
                raise ValueError("an NVFP4 cache needs block scales and tensor scales of K and V")
            for s in (k_scales, v_scales):
                if s.dtype != torch.uint8 or tuple(s.shape) != (P, H, S, D // 16):
                    raise ValueError("block scales must be uint8 [pages, kv heads, page size, head dim / 16]")
            for t in (k_tensor_scale, v_tensor_scale):
                if t.dtype != torch.float32 or t.numel() != 1:
                    raise ValueError("tensor scales must be one-element fp32 tensors")
            tensors += [k_scales, v_scales, k_tensor_scale, v_tensor_scale]
        for t in tensors:
            if not t.is_cuda or t.device != k.device or not t.is_contiguous():
                raise ValueError("cache tensors must be contiguous CUDA tensors on one device")
        if not (16 <= S <= 4096 and S % 16 == 0 and 32 <= D <= 256 and D % 32 == 0
                and 1 <= H <= 65536):
            raise ValueError("page size must be a multiple of 16 from 16 to 4096, head dim a "
                             "multiple of 32 from 32 to 256, kv heads 1 to 65536")
        self.k, self.v, self.k_scales, self.v_scales = k, v, k_scales, v_scales
        self.k_tensor_scale, self.v_tensor_scale = k_tensor_scale, v_tensor_scale
        self.num_pages, self.num_kv_heads, self.page_size, self.head_dim = P, H, S, D
        self.format, self.device = ("nvfp4" if nvfp4 else "bf16"), k.device
        self._index = k.get_device()
        ptr = lambda t: t.data_ptr() if nvfp4 else None
        self._c = FosKVCache(ctypes.sizeof(FosKVCache), FOS_KV_NVFP4 if nvfp4 else FOS_KV_BF16, P,
                             S, H, D, 0, k.data_ptr(), v.data_ptr(), ptr(k_scales), ptr(v_scales),
                             ptr(k_tensor_scale), ptr(v_tensor_scale))
        self._ref = ctypes.byref(self._c)


def kv_cache(num_pages: int, page_size: int, num_kv_heads: int, head_dim: int,
             format: str = "nvfp4", k_tensor_scale: Optional[torch.Tensor] = None,
             v_tensor_scale: Optional[torch.Tensor] = None, device="cuda") -> PagedKVCache:
    """An empty (zeroed) cache.  An NVFP4 cache needs the static tensor scales of K and V:
    fp32 [1] device tensors, e.g. ``tensor_scale`` of keys and values seen beforehand."""
    shape = (num_pages, num_kv_heads, page_size)
    if format == "bf16":
        return PagedKVCache(*(torch.zeros(*shape, head_dim, dtype=torch.bfloat16, device=device)
                              for _ in range(2)))
    if format != "nvfp4":
        raise ValueError("format must be 'nvfp4' or 'bf16'")
    u8 = dict(dtype=torch.uint8, device=device)
    k, v = (torch.zeros(*shape, head_dim // 2, **u8) for _ in range(2))
    ks, vs = (torch.zeros(*shape, head_dim // 16, **u8) for _ in range(2))
    return PagedKVCache(k, v, ks, vs, k_tensor_scale, v_tensor_scale)


def _check_rows(cache: PagedKVCache, x: torch.Tensor, T: int, what: str) -> int:
    """The token stride of x."""
    H, D, s = cache.num_kv_heads, cache.head_dim, x.stride()
    if (len(s) != 3 or x.shape[1:] != (H, D) or x.dtype != _BF16 or x.get_device() != cache._index
            or s[2] != 1 or (H > 1 and s[1] != D)):
        raise ValueError(f"{what} must be bf16 [tokens, kv heads, head dim] on the cache's device, "
                         "each token's heads in one run")
    if x.shape[0] != T:
        raise ValueError("k, v and slots disagree on the number of tokens")
    return s[0]


def _check_slots(cache: PagedKVCache, slots: torch.Tensor) -> int:
    """The number of slots."""
    if (slots.dim() != 1 or slots.dtype != _I64 or slots.get_device() != cache._index
            or not slots.is_contiguous()):
        raise ValueError("slots must be a contiguous 1-D int64 tensor on the cache's device")
    return slots.shape[0]


_KV_RULES = {"4/6": FOS_RULE_4OVER6, "6": FOS_RULE_6ONLY}


def kv_append(cache: PagedKVCache, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor,
              rule: str = "4/6") -> None:
    """Write the keys and values of new tokens (bf16 [T, kv heads, head dim]; the token
    stride is free, so columns of a fused projection need no copy) to ``slots`` (int64
    [T], page * page_size + token of the page; negative or past the cache: skipped).
    An NVFP4 cache quantizes each 16 values with ``rule`` ("4/6" or "6") under the
    cache's tensor scales.  Slots of one call must be distinct."""
    T = _check_slots(cache, slots)
    k_stride, v_stride = _check_rows(cache, k, T, "k"), _check_rows(cache, v, T, "v")
    call = _lib.fos_kv_append
    if cache._index != _current_device():
        call = _on(cache._index, call)
    _check(call(cache._ref, _KV_RULES[rule], k.data_ptr(), k_stride, v.data_ptr(),
                v_stride, slots.data_ptr(), T, _raw_stream(cache._index)),
           "fos_kv_append")


def kv_gather(cache: PagedKVCache, slots: torch.Tensor) -> Tuple[torch.Tensor, torch.Tensor]:
    """Keys and values of ``slots`` (int64 [T]) as bf16 [T, kv heads, head dim]; zeros for
    slots outside the cache."""
    T, H, D = _check_slots(cache, slots), cache.num_kv_heads, cache.head_dim
    k = torch.empty(T, H, D, dtype=_BF16, device=cache.device)
    v = torch.empty(T, H, D, dtype=_BF16, device=cache.device)
    call = _lib.fos_kv_gather
    if cache._index != _current_device():
        call = _on(cache._index, call)
    _check(call(cache._ref, slots.data_ptr(), T, k.data_ptr(), H * D, v.data_ptr(),
                H * D, _raw_stream(cache._index)), "fos_kv_gather")
    return k, v


@functools.lru_cache(maxsize=4096)
def _decode_need(B: int, Hq: int, Hkv: int, D: int) -> int:
    return int(_lib.fos_paged_decode_workspace_bytes(B, Hq, Hkv, D))


_decode_workspaces = {}


def paged_decode_workspace(B: int, Hq: int, Hkv: int, D: int, device="cuda") -> torch.Tensor:
    """A workspace for paged_decode of these sizes, its counters cleared (by work on the
    current stream): what a captured graph passes as ``ws``."""
    need = _decode_need(B, Hq, Hkv, D)
    if need == 0:
        raise ValueError("sizes that paged_decode does not take")
    ws = torch.empty(1 << (need - 1).bit_length(), dtype=torch.uint8, device=device)
    ws[:int(_lib.fos_paged_decode_counter_bytes())].zero_()
    return ws


def _decode_workspace(device: torch.device, stream: int, capturing: bool, sizes) -> torch.Tensor:
    """The current stream's scratch for paged_decode, grown by powers of two.  A captured
    call gets one of its own, cleared in the graph: the graph may be replayed on another
    stream, or later than the next eager call on this one."""
    if capturing:
        return paged_decode_workspace(*sizes, device=device)
    key = (device.index, stream)
    ws = _decode_workspaces.get(key)
    if ws is None or ws.numel() < _decode_need(*sizes):
        ws = _decode_workspaces[key] = paged_decode_workspace(*sizes, device=device)
    return ws


def paged_decode(q: torch.Tensor, cache: PagedKVCache, block_table: torch.Tensor,
                 seq_lens: torch.Tensor, scale: Optional[float] = None, window: int = 0,
                 return_lse: bool = False, out: Optional[torch.Tensor] = None,
                 ws: Optional[torch.Tensor] = None):
    """Attention of one new token per sequence over the paged cache.

    q: bf16 [B, query heads, head dim] (the sequence stride is free; query heads a
    multiple of the cache's kv heads).  block_table: int32 [B, pages], rows may be
    strided; an id outside the cache is a page no longer held, whose tokens are not
    visible.  seq_lens: int32 [B], the new token included.  scale: default
    1/sqrt(head dim).  window > 0: only the last ``window`` tokens are visible.
    ``ws``: a ``paged_decode_workspace`` that no overlapping call uses; by default the
    current stream's (in a graph capture a new one, cleared by every replay).
    Returns bf16 [B, query heads, head dim] (``out`` if given), and with
    ``return_lse`` also the fp32 [B, query heads] log-sum-exp of the scaled scores.
    Where nothing is visible the output is 0 and its lse -inf."""
    dev, D, s = cache._index, cache.head_dim, q.stride()
    if len(s) != 3 or q.dtype != _BF16 or q.get_device() != dev:
        raise ValueError("q must be bf16 [sequences, query heads, head dim] on the cache's device")
    B, Hq, Dq = q.shape
    if Dq != D or s[2] != 1 or (Hq > 1 and s[1] != D):
        raise ValueError("q must have the cache's head dim, each sequence's heads in one run")
    if Hq < 1 or Hq % cache.num_kv_heads:
        raise ValueError("query heads must be a multiple of the cache's kv heads")
    t = block_table.stride()
    if len(t) != 2 or block_table.dtype != _I32 or block_table.get_device() != dev:
        raise ValueError("block_table must be int32 [sequences, pages] on the cache's device")
    rows, pages = block_table.shape
    if rows != B or (pages > 1 and t[1] != 1):
        raise ValueError("block_table must have a row of pages for each sequence")
    if (seq_lens.shape != (B,) or seq_lens.dtype != _I32 or seq_lens.get_device() != dev
            or not seq_lens.is_contiguous()):
        raise ValueError("seq_lens must be a contiguous int32 [sequences] tensor on the cache's device")
    if out is None:
        out = q.new_empty(B, Hq, D)
    elif (out.shape != (B, Hq, D) or out.dtype != _BF16 or out.get_device() != dev
          or not out.is_contiguous()):
        raise ValueError("out must be a contiguous bf16 tensor of q's shape on the cache's device")
    lse = q.new_empty(B, Hq, dtype=_F32) if return_lse else None
    stream, call, capturing = _raw_stream(dev), _lib.fos_paged_decode, _is_capturing
    if dev != _current_device():
        call, capturing = _on(dev, call), _on(dev, capturing)
    if ws is None:
        ws = _decode_workspace(cache.device, stream, capturing(), (B, Hq, cache.num_kv_heads, D))
    elif ws.dtype != _U8 or ws.get_device() != dev or not ws.is_contiguous():
        raise ValueError("ws must be a contiguous uint8 tensor on the cache's device")
    _check(call(cache._ref, q.data_ptr(), s[0], B, Hq, block_table.data_ptr(), t[0],
                pages, seq_lens.data_ptr(), D ** -0.5 if scale is None else scale,
                int(window), out.data_ptr(), None if lse is None else lse.data_ptr(),
                ws.data_ptr(), ws.numel(), stream), "fos_paged_decode")
    return (out, lse) if return_lse else out
