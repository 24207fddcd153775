"""The feed-forward binding's own work, without a GPU: CPU tensors stand for a device's, and
the entry points' names are noted instead of called."""
import pytest
import torch

import fp4_block_quantization_amd as package
from fp4_block_quantization_amd import fos

BF16 = torch.bfloat16


@pytest.fixture
def calls(monkeypatch):
    """Names of the entry points that a call of the binding reaches."""
    seen = []
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: 0)
    monkeypatch.setattr(fos, "_call", lambda dev, name, *args: seen.append(name))
    return seen


def record(rows, cols):
    return fos.NVFP4Tensor(torch.zeros(rows, cols // 2, dtype=torch.uint8),
                           torch.zeros(rows, cols // 16, dtype=torch.uint8), torch.zeros(1))


def product_bwd(m, n, k, gated=False, x=None, w=None, **kw):
    rows = 2 * n if gated else n
    dy, z = torch.zeros(m, n, dtype=BF16), torch.zeros(m, rows, dtype=BF16)
    f = fos.qglu_bwd if gated else fos.qlinear_epilogue_bwd
    return f(dy, z, x or record(k, m), w or record(k, rows), **kw)


# dX has W's rows as its inner dimension, dW those of X; only the wanted ones count
@pytest.mark.parametrize("m,n,gated,kw", [
    (48, 64, False, {}), (48, 64, True, {}), (64, 48, False, {}), (64, 16, True, {}),
    (64, 48, False, dict(need_dw=False)), (80, 64, True, dict(need_dx=False)),
    (32, 64, False, {}), (0, 64, False, {}), (0, 64, False, dict(need_dw=False)),
])
def test_backward_of_a_product_refuses_sizes_before_the_first_launch(calls, m, n, gated, kw):
    with pytest.raises(fos.FosError) as e:
        product_bwd(m, n, 64, gated, **kw)
    assert e.value.status == fos.FOS_E_SHAPE and calls == []


@pytest.mark.parametrize("m,n,gated,kw", [
    (64, 64, False, {}), (128, 32, True, {}), (64, 48, False, dict(need_dx=False)),
    (48, 64, False, dict(need_dw=False)), (1, 64, True, dict(need_dw=False))])
def test_backward_of_a_product_launches_what_it_accepts(calls, m, n, gated, kw):
    product_bwd(m, n, 48, gated, **kw)
    assert calls == ["fos_epilogue_bwd", "fos_quantize_scaled"] + ["fos_qlinear_epilogue_fwd"] * (2 - len(kw))


def test_backward_of_a_product_refuses_what_is_too_large_or_misaligned(calls):
    # a packed operand of 4 GiB, and more columns than an epilogue addresses; no memory behind them
    many = torch.zeros(1, dtype=torch.uint8)
    for rows, inner in (((1 << 20) + 64, 64), (1 << 20, 8192)):
        big = fos.NVFP4Tensor(many.expand(rows, inner // 2), many.expand(rows, inner // 16), torch.zeros(1))
        with pytest.raises(fos.FosError) as e:
            fos._check_plain_product(64, rows, inner, big)
        assert e.value.status == fos.FOS_E_SHAPE
    buf = torch.zeros(64 * 32 + 32, dtype=torch.uint8)
    start = -buf.data_ptr() % 16
    x = record(64, 64)
    x.data = buf[start + 8:][:64 * 32].view(64, 32)
    with pytest.raises(fos.FosError) as e:
        product_bwd(64, 64, 64, x=x)
    assert e.value.status == fos.FOS_E_ALIGN and calls == []
    x.data = buf[start:][:64 * 32].view(64, 32)
    product_bwd(64, 64, 64, x=x)
    assert len(calls) == 4


def test_backward_of_a_product_refuses_operands_of_different_inner_dimensions(calls):
    with pytest.raises(ValueError, match="inner dimension"):
        product_bwd(64, 64, None, x=record(48, 64), w=record(80, 64))
    assert calls == []
    product_bwd(64, 64, None, x=record(48, 64), w=record(80, 64), need_dw=False)     # X is not looked at
    assert len(calls) == 3


def test_backward_of_the_norm_takes_the_rows_that_its_forward_took(calls):
    """Without a residual h is x itself, whose rows may be strided."""
    wide, w, rstd = torch.zeros(6, 200, dtype=BF16), torch.ones(64, dtype=BF16), torch.ones(6)
    dy = torch.zeros(6, 64, dtype=BF16)
    for h in (wide[:, 8:72], wide[:, :64], dy):
        fos.rmsnorm_bwd(dy, h, w, rstd)
    assert calls == ["fos_rmsnorm_bwd"] * 3
    for h in (torch.zeros(64, 6, dtype=BF16).T, wide[:, :128:2], wide[:4, :64], wide[:, :64].float(), w):
        with pytest.raises(ValueError):
            fos.rmsnorm_bwd(dy, h, w, rstd)
    with pytest.raises(ValueError):
        fos.rmsnorm_bwd(wide[:, :64], dy, w, rstd)
    assert len(calls) == 3


@pytest.mark.parametrize("name", [
    "rmsnorm_fwd", "rmsnorm_bwd", "RMSNormOutput", "qlinear_epilogue_fwd", "mx_qlinear_epilogue_fwd", "qglu_fwd",
    "mx_qglu_fwd", "wlinear_epilogue_fwd", "mx_wlinear_epilogue_fwd", "wglu_fwd", "mx_wglu_fwd", "epilogue_bwd",
    "qlinear_epilogue_bwd", "qglu_bwd"])
def test_the_package_offers_the_operators(name):
    """As it does the quantizers, the plain products and the calls of a decode step."""
    assert getattr(package, name) is getattr(fos, name)
