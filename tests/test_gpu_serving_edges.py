"""GPU tests of the token-serving operators at the ends of their ranges.  Bounds as in
test_gpu_serving.py, with what a test claims beyond them said there.
"""
import ctypes

import pytest
import torch

from test_gpu_serving import DEV, fos  # noqa: F401

pytestmark = pytest.mark.gpu


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
