"""GPU tests of the token-serving operators at the ends of their ranges.  Bounds as in
test_gpu_serving.py, with what a test claims beyond them said there.
"""
import ctypes

import numpy as np
import pytest
import torch

from fp4_block_quantization_amd import workloads as W
from oracle import serving as S
from test_gpu_serving import DEV, U, dev, f64, fos, within  # noqa: F401

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ weight-only linear

@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_wlinear_longest_inner_dimension(fos, fmt):
    """K at the end of its range, 2^31 - 32: a weight row of 1 GiB, an activation of 4 GiB
    that is zero but in 300 blocks, the first and the last among them."""
    K, blocks = 2 ** 31 - 32, 300
    block = 16 if fmt == "nvfp4" else 32
    g = torch.Generator(device=DEV).manual_seed(3)
    data = torch.randint(0, 256, (1, K // 2), dtype=torch.uint8, device=DEV, generator=g)
    lo, hi = (40, 72) if fmt == "nvfp4" else (120, 130)
    scales = torch.randint(lo, hi, (1, K // block), dtype=torch.uint8, device=DEV, generator=g)
    at = np.random.RandomState(4).choice(K // 32, blocks, replace=False)
    at[:3] = 0, K // 32 - 1, K // 32 - 2
    some = W.random_bf16(blocks, 32, 5, "normal").to(DEV)
    x = torch.zeros(1, K, dtype=torch.bfloat16, device=DEV)
    x.view(-1, 32)[dev(at)] = some
    bias = torch.ones(1, dtype=torch.bfloat16, device=DEV)
    t = torch.full((1,), 0.01, device=DEV)
    if fmt == "nvfp4":
        y = fos.wlinear_fwd(x, fos.NVFP4Tensor(data, scales, t), bias=bias, out_dtype=torch.float32)
    else:
        y = fos.mx_wlinear_fwd(x, fos.MXFP4Tensor(data, scales), bias=bias, out_dtype=torch.float32)
    part = lambda r, n: r.view(-1, n)[dev(at)].reshape(1, -1).cpu().numpy()
    ref, mag = S.wlinear_ref64(f64(some).reshape(1, -1), part(data, 16), part(scales, 32 // block),
                               np.float32(0.01) if fmt == "nvfp4" else None, np.ones(1))
    # the other products are zeros: only sums with these blocks' values round
    within(f64(y), ref, U * np.abs(ref) + (32 * blocks + 8) * U * mag, "y")


# ------------------------------------------------------------------ attention

@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("D", [32, 128, 192])
def test_decode_over_a_cache_without_memory(fos, fmt, D):
    """A cache of no pages may have every pointer null, its tensor scales among them."""
    B, Hq, Hkv = 3, 4, 2
    cache = fos.FosKVCache(ctypes.sizeof(fos.FosKVCache), fmt, 0, 16, Hkv, D, 0)
    q = torch.ones(B, Hq, D, dtype=torch.bfloat16, device=DEV)
    table = torch.zeros(B, 2, dtype=torch.int32, device=DEV)
    lens = torch.tensor([5, 0, 32], dtype=torch.int32, device=DEV)
    out, lse = torch.ones_like(q), torch.zeros(B, Hq, device=DEV)
    ws = fos.paged_decode_workspace(B, Hq, Hkv, D, DEV)
    status = fos.lib().fos_paged_decode(
        ctypes.byref(cache), q.data_ptr(), Hq * D, B, Hq, table.data_ptr(), 2, 2, lens.data_ptr(), 0.125,
        0, out.data_ptr(), lse.data_ptr(), ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream)
    assert status == fos.FOS_OK
    torch.cuda.synchronize()
    assert not out.any() and (lse == -float("inf")).all()


def test_decode_over_an_empty_nvfp4_cache(fos):
    t = torch.ones(1, device=DEV)
    cache = fos.kv_cache(0, 16, 2, 64, "nvfp4", t, t, device=DEV)
    q = torch.ones(2, 4, 64, dtype=torch.bfloat16, device=DEV)
    out, lse = fos.paged_decode(q, cache, torch.zeros(2, 3, dtype=torch.int32, device=DEV),
                                torch.tensor([5, 48], dtype=torch.int32, device=DEV), return_lse=True)
    assert not out.any() and (lse == -float("inf")).all()
