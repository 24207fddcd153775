"""The decode-step example: what its launches compute stage by stage against the fp64
references, and its replayed graph against eager launches bit for bit."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from oracle import serving as S
from test_gpu_serving import DEV, check_attention, check_linear, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example(root_dir):
    spec = importlib.util.spec_from_file_location(
        "decode_step", os.path.join(root_dir, "examples", "decode_step.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def rows(t):
    return t.cpu().numpy()


def held_rows(d, b):
    """Keys and values of sequence b as they lie in its cache, fp64."""
    c, page = d.cache, d.pages.page_size
    j = np.arange(d.pages.count[b])
    ids, off = np.asarray(d.pages.held[b])[j // page], j % page
    out = []
    for data, scales, t in ((c.k, c.k_scales, c.k_tensor_scale), (c.v, c.v_scales, c.v_tensor_scale)):
        data = f64(data) if scales is None else rows(data)
        out.append(S.cache_rows_f64(data[ids, :, off], None if scales is None else rows(scales)[ids, :, off],
                                    None if t is None else float(t)))
    return out


@pytest.mark.parametrize("fmt", ["nvfp4", "bf16"])
def test_decode_steps(example, fmt):
    layer = example.Layer(256, 8, 2, 64, 512, seed=3, device=DEV)
    batch, prompt, steps = 3, 70, 9
    decoders = [example.Decoder(layer, fmt, batch, prompt + steps, 16, seed=4, graph=g)
                for g in (True, False)]
    gen = torch.Generator().manual_seed(5)
    first = torch.randn(prompt, batch, 256, generator=gen).to(DEV, torch.bfloat16)
    for d in decoders:
        d.prefill(first)
    for _ in range(steps):
        x = torch.randn(batch, 256, generator=gen).to(DEV, torch.bfloat16)
        (y, parts), (want, eager) = (d.step(x) for d in decoders)
        torch.cuda.synchronize()
        assert torch.equal(y, want)
        for name in eager:
            assert torch.equal(parts[name], eager[name]), name
    d = decoders[1]
    w = layer.w_qkv
    qkv = torch.cat([eager[n].flatten(1) for n in "qkv"], dim=1)
    check_linear(qkv, example.normed(x), rows(w.data), rows(w.scales), float(w.tensor_scale), layer.b_qkv)
    for b in range(batch):
        k, v = held_rows(d, b)
        assert len(k) == prompt + steps
        check_attention(eager["attention"][b], None, f64(eager["q"][b]), k, v, 0.125, f"sequence {b}")
    w = layer.w_down
    check_linear(example.fos.mx_wlinear_fwd(eager["u"], w), eager["u"], rows(w.data), rows(w.scales), None)
