"""GPU tests of the feed-forward operators against fp64 references (oracle/feedforward.py)
and, for what is stored in 4 bits, the oracle's records bit for bit.

Bounds (u = 2^-24, half a step of fp32).

Norm: a square of a bf16 value is exact in fp64, so the mean of K of them is off by at most
K 2^-53 and rstd, rounded once to fp32, by (1 + 2^-10) u.  y is then a fixed sequence of fp32
roundings of h, rstd and w, which the tests repeat bit for bit.

Backward of the norm: n and g carry one rounding (u); a product of the two at most 4 u, the
sum of K of them K u of the magnitudes more; dx's own terms add 6 u and dh's addition one.
dw: each term 3 u, and M u of the magnitudes for their sum.

Epilogue: Z is a sum of K exact products, off by at most (K + 8) u S (S the magnitudes; the
scale and the bias are a few u).  The activations' slopes are at most 1.13 in size.  The
activation itself: the exponent -z log2 e carries 1.5 |z| u (gelu_tanh: its argument, of
size at most |u|, is off by 4 u |u|, and s (1 - s) |z| |u| is at most 1.2), the hardware's
exponential and reciprocal 2 u each, so with s (1 - s) z^2 <= 0.44 an activation is off by
at most 16 u (1 + |z|); the fit behind gelu by 5 u of a tail that is at most 1 / 2.  A
rounding to bf16 adds 2^-8 of the value, to fp32 u.

Slopes: the same errors, times at most |z| du/dz where a slope has that factor: 32 u (1 + |z|)
for |z| below 16, beyond which a slope is 0 or 1 to fp32.
"""
import numpy as np
import pytest
import torch

from fp4_block_quantization_amd import workloads as W
from oracle import feedforward as FF
from oracle import formats as F
from oracle import mxfp4 as MX
from oracle import nvfp4 as N
from oracle import serving as S
from oracle.qlinear import operand_exact
from test_gpu_parity import assert_same_bytes, bits_of
from test_gpu_serving import dev, f64, mx_weight, nv_weight, within

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def fos():
    from fp4_block_quantization_amd import fos as mod
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    return mod


def rnd(dtype):
    return 2.0 ** -8 if dtype == BF16 else U


def bits(t):
    """The bf16 bit patterns of a GPU tensor."""
    return t.cpu().contiguous().view(torch.int16).numpy().view(np.uint16)


# ------------------------------------------------------------------------------- norm

NORM_SHAPES = [(1, 16), (3, 32), (5, 48), (1, 4096), (17, 512), (40, 528), (64, 1040), (1030, 1024),
               (1100, 2080), (1025, 4096), (9, 4112), (7, 8192), (3, 16384), (2, 16400), (2, 32768), (1027, 2064),
               (2500, 96), (9000, 64), (4, 4096), (3, 2064), (2, 1040), (5, 1040), (16, 512)]


def norm_inputs(m, k, seed, residual):
    x = W.random_bf16(m, k, seed, "student_t").to(DEV)
    r = W.random_bf16(m, k, seed + 1, "normal", scale=3.0).to(DEV) if residual else None
    w = W.random_bf16(1, k, seed + 2, "normal")[0].to(DEV)
    return x, r, w


def check_norm(o, x, r, w, eps):
    """h, rstd and the bits of y, which are returned (as a CPU bf16 tensor)."""
    h = x.cpu() if r is None else (x.cpu().float() + r.cpu().float()).to(BF16)
    assert torch.equal(o.h.cpu(), h)
    _, rstd = FF.rmsnorm64(h.double().numpy(), w.cpu().double().numpy(), eps)
    within(o.rstd.cpu().double().numpy(), rstd, (1 + 2.0 ** -10) * U * rstd, "rstd")
    y = (h.float() * o.rstd.cpu()[:, None] * w.cpu().float()).to(BF16)
    if o.y is not None:
        assert torch.equal(o.y.cpu(), y)
    return y


@pytest.mark.parametrize("m,k", NORM_SHAPES)
@pytest.mark.parametrize("residual", [False, True])
def test_norm_bf16(fos, m, k, residual):
    x, r, w = norm_inputs(m, k, m + k, residual)
    check_norm(fos.rmsnorm_fwd(x, w, eps=1e-5, residual=r), x, r, w, 1e-5)


@pytest.mark.parametrize("m,k", NORM_SHAPES)
@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("residual", [False, True])
def test_norm_nvfp4(fos, m, k, given, residual):
    x, r, w = norm_inputs(m, k, m + k + 7, residual)
    t = torch.tensor([0.002], device=DEV) if given else None
    o = fos.rmsnorm_fwd(x, w, residual=r, format="nvfp4", tensor_scale=t, return_y=not given)
    y = check_norm(o, x, r, w, 1e-6)
    want = N.quantize(bits(y), N.Config(), None if t is None else np.float32(0.002))
    assert np.float32(o.record.tensor_scale.cpu()[0]) == want["t"]
    assert_same_bytes(o.record.data.cpu().numpy(), want["row_data"], "data")
    assert_same_bytes(o.record.scales.cpu().numpy(), want["row_scales"], "scales")


@pytest.mark.parametrize("m,k", [s for s in NORM_SHAPES if s[1] % 32 == 0])
def test_norm_mxfp4(fos, m, k):
    x, r, w = norm_inputs(m, k, m + k + 9, m % 2)
    o = fos.rmsnorm_fwd(x, w, residual=r, format="mxfp4", return_y=bool(k % 64))
    want = MX.quantize(bits(check_norm(o, x, r, w, 1e-6)))
    assert_same_bytes(o.record.data.cpu().numpy(), want["data"], "data")
    assert_same_bytes(o.record.scales.cpu().numpy(), want["scales"], "scales")


def test_norm_rule_six(fos):
    x, r, w = norm_inputs(33, 160, 3, True)
    o = fos.rmsnorm_fwd(x, w, residual=r, format="nvfp4", rule="6")
    want = N.quantize(bits(check_norm(o, x, r, w, 1e-6)), N.Config(rule="6"))
    assert_same_bytes(o.record.data.cpu().numpy(), want["row_data"], "data")
    assert_same_bytes(o.record.scales.cpu().numpy(), want["row_scales"], "scales")


@pytest.mark.parametrize("fmt", ["bf16", "nvfp4", "mxfp4"])
@pytest.mark.parametrize("m", [1, 5, 1200])
def test_norm_strided_rows(fos, fmt, m):
    k = 320
    wide = torch.full((m, 2 * k + 48), float("nan"), dtype=BF16, device=DEV)
    x, r, w = norm_inputs(m, k, 4, True)
    wide[:, 8:8 + k], wide[:, k + 24:2 * k + 24] = x, r
    want = fos.rmsnorm_fwd(x, w, residual=r, format=fmt)
    got = fos.rmsnorm_fwd(wide[:, 8:8 + k], w, residual=wide[:, k + 24:2 * k + 24], format=fmt)
    assert torch.equal(got.h, want.h) and torch.equal(got.rstd, want.rstd)
    if fmt == "bf16":
        assert torch.equal(got.y, want.y)
    else:
        assert torch.equal(got.record.data, want.record.data)
        assert torch.equal(got.record.scales, want.record.scales)


@pytest.mark.parametrize("fmt", ["bf16", "nvfp4", "mxfp4"])
def test_norm_sum_in_place(fos, fmt):
    """The residual stream updated where it lies, rows around it untouched."""
    m, k = 37, 544
    x, r, w = norm_inputs(m, k, 5, True)
    want = fos.rmsnorm_fwd(x, w, residual=r, format=fmt)
    stream = torch.full((m + 2, k), 7.0, dtype=BF16, device=DEV)
    stream[1:-1] = r
    got = fos.rmsnorm_fwd(x, w, residual=stream[1:-1], format=fmt, h=stream[1:-1])
    assert torch.equal(stream[1:-1], want.h) and torch.equal(got.rstd, want.rstd)
    assert (stream[0] == 7).all() and (stream[-1] == 7).all()
    for a, b in ((got.y, want.y),) if fmt == "bf16" else ((got.record.data, want.record.data),):
        assert torch.equal(a, b)


@pytest.mark.parametrize("fmt", ["bf16", "nvfp4", "mxfp4"])
def test_norm_extreme_rows(fos, fmt):
    """A row of zeros, one of values whose squares pass fp32, one of subnormals, one value alone."""
    k = 96
    x = torch.zeros(4, k)
    x[1], x[2] = 1.0e37 * torch.sign(torch.randn(k, generator=torch.Generator().manual_seed(1))), 1e-39
    x[3, 95] = -5.0
    x, w = x.to(BF16).to(DEV), W.random_bf16(1, k, 6, "normal")[0].to(DEV)
    o = fos.rmsnorm_fwd(x, w, eps=1e-30, format=fmt, return_y=True)
    y = check_norm(o, x, None, w, 1e-30)
    assert torch.isfinite(y).all() and (o.y[0] == 0).all()
    if fmt == "nvfp4":
        want = N.quantize(bits(y), N.Config())
        assert_same_bytes(o.record.data.cpu().numpy(), want["row_data"], "data")
    if fmt == "mxfp4":
        assert_same_bytes(o.record.data.cpu().numpy(), MX.quantize(bits(y))["data"], "data")


@pytest.mark.parametrize("m,k", [(5, 96), (2, 4096), (1200, 4096), (3, 16384), (2, 32768), (17, 512), (6, 4096)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_norm_of_values_that_are_not_finite(fos, m, k, bad):
    """One such value makes its row NaN; the records are those of y, whatever it holds."""
    x, r, w = norm_inputs(m, k, 3, True)
    clean = fos.rmsnorm_fwd(x, w, residual=r).y
    x[1, 7] = bad
    for given in (None, torch.full((1,), 2.0 ** -7, device=DEV)):
        o = fos.rmsnorm_fwd(x, w, residual=r, format="nvfp4", tensor_scale=given, return_y=True)
        q = fos.quantize(o.y, tensor_scale=given)
        assert torch.equal(o.record.data, q.data) and torch.equal(o.record.scales, q.scales)
        assert torch.equal(o.record.tensor_scale.view(torch.int32), q.tensor_scale.view(torch.int32))
    o = fos.rmsnorm_fwd(x, w, residual=r, format="mxfp4", return_y=True)
    q = fos.mx_quantize(o.y)
    assert torch.equal(o.record.data, q.data) and torch.equal(o.record.scales, q.scales)
    rest = torch.arange(m, device=DEV) != 1
    assert torch.equal(o.y[rest], clean[rest]) and o.y[1].isnan().any()


def test_norm_of_no_rows(fos):
    x, w = torch.empty(0, 64, dtype=BF16, device=DEV), torch.ones(64, dtype=BF16, device=DEV)
    for fmt in ("bf16", "nvfp4", "mxfp4"):
        o = fos.rmsnorm_fwd(x, w, residual=x, format=fmt)
        assert o.h.shape == (0, 64) and o.rstd.shape == (0,)
        if fmt == "nvfp4":
            assert float(o.record.tensor_scale) == 0.0
    dx, dw = fos.rmsnorm_bwd(x, x, w, torch.empty(0, device=DEV))
    assert dx.shape == (0, 64) and (dw == 0).all()


@pytest.mark.parametrize("m,k", NORM_SHAPES)
@pytest.mark.parametrize("direct", [False, True])
def test_norm_bwd(fos, m, k, direct):
    h, dh, w = norm_inputs(m, k, m + k + 11, direct)
    dy = W.random_bf16(m, k, m + 1, "normal", scale=0.1).to(DEV)
    rstd = fos.rmsnorm_fwd(h, w).rstd
    dx, dw = fos.rmsnorm_bwd(dy, h, w, rstd, dh=dh)
    ref, rdw, size, sdw = FF.rmsnorm_bwd64(f64(dy), f64(h), f64(w), rstd.cpu().double().numpy(),
                                           None if dh is None else f64(dh))
    err = (k + 12) * U * size
    within(f64(dx), ref, 2.0 ** -8 * (np.abs(ref) + err) + err, "dx")
    within(dw.cpu().double().numpy(), rdw, (m + 4) * U * sdw, "dw")
    again = fos.rmsnorm_bwd(dy, h, w, rstd, dh=dh)
    assert torch.equal(dx, again[0]) and torch.equal(dw, again[1])
    assert fos.rmsnorm_bwd(dy, h, w, rstd, dh=dh, need_dweight=False)[1] is None


# --------------------------------------------------------------------------- epilogue

def product_bound(z, size, act, k, dtype):
    """(y's error before its rounding is added, for an activation of z)"""
    return 1.13 * (k + 8) * U * size + 16 * U * (1 + np.abs(z))


def check_epilogue(y, z_kept, x, w, bias, act, gated, residual, k):
    """x, w: operands in fp64, scales applied."""
    z, size = x @ w.T, np.abs(x) @ np.abs(w).T
    if bias is not None:
        z, size = z + bias, size + np.abs(bias)
    ez = (k + 8) * U * size
    if z_kept is not None:
        within(f64(z_kept), z, 2.0 ** -8 * (np.abs(z) + ez) + ez + 2.0 ** -133, "preact")
    ref = FF.epilogue64(z, act, gated, residual)
    if gated:
        half = z.shape[1] // 2
        f = np.abs(FF.activation64(act, z[:, :half])[0])
        ef = 1.13 * ez[:, :half] + 16 * U * (1 + np.abs(z[:, :half]))
        err = ef * (np.abs(z[:, half:]) + ez[:, half:]) + f * ez[:, half:] + 2 * U * np.abs(ref)
    else:
        err = 1.13 * ez + 16 * U * (1 + np.abs(z))
        if residual is not None:
            err = err + 2 * U * (np.abs(ref) + np.abs(residual))
    within(f64(y), ref, rnd(y.dtype) * (np.abs(ref) + err) + err + 2.0 ** -133, "y")


Q_SHAPES = [(1, 1, 64), (16, 16, 64), (3, 130, 256), (130, 100, 256), (256, 256, 256), (257, 300, 512),
            (100, 515, 320), (300, 128, 1024), (513, 260, 192), (64, 1027, 768), (700, 64, 512)]


def nv_act(fos, m, k, seed):
    return nv_weight(fos, m, k, seed, scale=1.0)


@pytest.mark.parametrize("m,n,k", Q_SHAPES)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_qlinear_epilogue(fos, m, n, k, gated, fmt):
    nv = fmt == "nvfp4"
    if not nv and k % 256:
        pytest.skip("MXFP4 products take whole 256s")
    i = Q_SHAPES.index((m, n, k))
    act = FF.ACTIVATIONS[(i + 2 * gated + nv) % 5]
    out = BF16 if (i + gated) % 3 else torch.float32
    rows = 2 * n if gated else n
    xd, xs, xt, xq = (nv_act if nv else mx_weight)(fos, m, k, m + k)
    wd, ws, wt, wq = (nv_weight if nv else mx_weight)(fos, rows, k, n + k)
    bias = W.random_bf16(1, rows, m, "normal")[0].to(DEV) if i % 2 else None
    res = W.random_bf16(m, n, n, "normal").to(DEV) if not gated and i % 3 == 0 else None
    kw = dict(bias=bias, activation=act, out_dtype=out, return_preact=i % 2 == 0)
    if gated:
        f = fos.qglu_fwd if nv else fos.mx_qglu_fwd
    else:
        f = fos.qlinear_epilogue_fwd if nv else fos.mx_qlinear_epilogue_fwd
        kw["residual"] = res
    got = f(xq, wq, **kw)
    y, z = got if kw["return_preact"] else (got, None)
    a = operand_exact(xd, xs) * xt if nv else MX.operand_exact(xd, xs)
    b = operand_exact(wd, ws) * wt if nv else MX.operand_exact(wd, ws)
    check_epilogue(y, z, a, b, None if bias is None else f64(bias), act, gated,
                   None if res is None else f64(res), k)
    again = f(xq, wq, **kw)
    assert torch.equal(y, again[0] if kw["return_preact"] else again)


# tiles of 256 x 256, and of 128 x 128 with one K step, in more than half a round of
# workgroups, and split over K, where sums have another order
@pytest.mark.parametrize("m,n,k,same", [(2300, 7700, 512, True), (260, 390, 256, True),
                                        (2050, 2304, 512, True), (260, 390, 768, False)])
def test_qlinear_epilogue_without_one_is_qlinear(fos, m, n, k, same):
    x, w = (W.random_bf16(r, k, r, "normal").to(DEV) for r in (m, n))
    xq, wq = fos.quantize(x), fos.quantize(w)
    want = fos.qlinear_fwd(xq, wq)
    got = fos.qlinear_epilogue_fwd(xq, wq)
    y, z = fos.qlinear_epilogue_fwd(xq, wq, activation="relu", return_preact=True)
    assert torch.equal(z, got) and torch.equal(y, got.relu())
    if same:
        assert torch.equal(got, want)
    else:
        size = fos.dequantize(xq).abs() @ fos.dequantize(wq).abs().t()
        within(f64(got), f64(want), 2.0 ** -7 * f64(want).__abs__() + 2.1 * (k + 8) * U * f64(size), "y")


@pytest.mark.parametrize("m,n,k", [(2300, 7700, 512), (700, 390, 768), (1100, 8200, 256)])
def test_mx_qlinear_epilogue_without_one_is_mx_qlinear(fos, m, n, k):
    """The same sums in the same order on tiles of 256 x 256, 128 x 128 and 256 x 128."""
    aq, bq = (fos.mx_quantize(W.random_bf16(r, k, r, "normal").to(DEV)) for r in (m, n))
    want = fos.mx_qlinear_fwd(aq, bq)
    assert torch.equal(fos.mx_qlinear_epilogue_fwd(aq, bq), want)
    y, z = fos.mx_qlinear_epilogue_fwd(aq, bq, activation="relu", return_preact=True)
    assert torch.equal(z, want) and torch.equal(y, want.relu())


# more rows than one 256 x 256 tile of the largest kernels, with every option
@pytest.mark.parametrize("m,n,k,gated,fmt,act", [
    (4097, 2100, 512, False, "nvfp4", "gelu"), (4097, 1100, 320, True, "nvfp4", "silu"),
    (4097, 4400, 512, False, "mxfp4", "gelu_tanh"), (8300, 1100, 256, True, "mxfp4", "silu"),
    (4097, 2099, 256, False, "nvfp4", "silu"), (4097, 4399, 512, False, "mxfp4", "silu"),
    # more tiles of 64 x 64 than there are CUs, fewer of 128 x 128: K split over two groups of waves
    (600, 2000, 832, False, "nvfp4", "silu"), (600, 1100, 576, True, "nvfp4", "gelu"),
    (2100, 2000, 192, False, "nvfp4", "gelu_tanh"), (2100, 1100, 256, True, "nvfp4", "relu")])
def test_epilogue_of_many_tiles(fos, m, n, k, gated, fmt, act):
    """Against fp32 products of the dequantized records, whose own error the bound counts."""
    rows = 2 * n if gated else n
    x, w = W.random_bf16(m, k, 1, "normal").to(DEV), W.random_bf16(rows, k, 2, "normal", scale=0.02).to(DEV)
    bias = W.random_bf16(1, rows, 3, "normal")[0].to(DEV)
    res = None if gated else W.random_bf16(m, n, 4, "normal").to(DEV)
    nv = fmt == "nvfp4"
    xq, wq = (fos.quantize(x), fos.quantize(w)) if nv else (fos.mx_quantize(x), fos.mx_quantize(w))
    a, b = ((fos.dequantize if nv else fos.mx_dequantize)(q).double() for q in (xq, wq))
    z, size = a @ b.t() + bias.double(), a.abs() @ b.abs().t() + bias.double().abs()
    kw = dict(bias=bias, activation=act, return_preact=True)
    if gated:
        y, got = (fos.qglu_fwd if nv else fos.mx_qglu_fwd)(xq, wq, **kw)
    else:
        y, got = (fos.qlinear_epilogue_fwd if nv else fos.mx_qlinear_epilogue_fwd)(xq, wq, residual=res, **kw)
    z, size = z.cpu().numpy(), size.cpu().numpy()
    # a dequantized NVFP4 value carries one rounding more (its block scale times the tensor's)
    ez = (k + 8 + 4) * U * size
    within(f64(got), z, 2.0 ** -8 * (np.abs(z) + ez) + ez, "preact")
    ref = FF.epilogue64(z, act, gated, None if res is None else f64(res))
    e = 1.13 * ez + 16 * U * (1 + np.abs(z))
    if gated:
        f = np.abs(FF.activation64(act, z[:, :n])[0])
        e = e[:, :n] * (np.abs(z[:, n:]) + ez[:, n:]) + f * ez[:, n:] + 2 * U * np.abs(ref)
    else:
        e = e + 2 * U * (np.abs(ref) + np.abs(f64(res)))
    within(f64(y), ref, 2.0 ** -8 * (np.abs(ref) + e) + e, "y")


@pytest.mark.parametrize("n", [256, 258, 131])
def test_qlinear_epilogue_residual_in_place_and_strided(fos, n):
    """The residual stream updated where it lies; a residual of odd stride beside NaNs."""
    m, k = 270, 256
    _, _, _, xq = nv_act(fos, m, k, 3)
    _, _, _, wq = nv_weight(fos, n, k, 4)
    res = W.random_bf16(m, n, 5, "normal").to(DEV)
    want = fos.qlinear_epilogue_fwd(xq, wq, residual=res)
    for shift in (0, 1):
        wide = torch.full((m, n + 3), float("nan"), dtype=BF16, device=DEV)
        wide[:, shift:shift + n] = res
        assert torch.equal(fos.qlinear_epilogue_fwd(xq, wq, residual=wide[:, shift:shift + n]), want)
    stream = torch.full((m + 2, n), 7.0, dtype=BF16, device=DEV)
    stream[1:-1] = res
    fos.qlinear_epilogue_fwd(xq, wq, residual=stream[1:-1], out=stream[1:-1])
    assert torch.equal(stream[1:-1], want)
    assert (stream[0] == 7).all() and (stream[-1] == 7).all()


@pytest.mark.parametrize("m", [1, 3, 17, 33, 130, 257])
@pytest.mark.parametrize("n", [256, 131])
@pytest.mark.parametrize("out", [BF16, torch.float32])
def test_rows_behind_the_last_are_left_as_they_were(fos, m, n, out):
    """The rows that a tile has past M, in the memory behind y: not written."""
    k = 512
    for nv in (True, False):
        _, _, _, xq = (nv_act if nv else mx_weight)(fos, m, k, 3)
        _, _, _, wq = (nv_weight if nv else mx_weight)(fos, 2 * n, k, 4)
        x = W.random_bf16(m, k, 5, "normal").to(DEV)
        for call in ((fos.qlinear_epilogue_fwd, fos.qglu_fwd) if nv else
                     (fos.mx_qlinear_epilogue_fwd, fos.mx_qglu_fwd)):
            cols = 2 * n if "epilogue" in call.__name__ else n
            held = torch.full((m + 600, cols), 7.0, dtype=out, device=DEV)
            call(xq, wq, activation="relu", out_dtype=out, out=held[300:300 + m])
            assert torch.equal(held[300:300 + m], call(xq, wq, activation="relu", out_dtype=out))
            assert (held[:300] == 7).all() and (held[300 + m:] == 7).all(), call.__name__
        for call in ((fos.wlinear_epilogue_fwd, fos.wglu_fwd) if nv else
                     (fos.mx_wlinear_epilogue_fwd, fos.mx_wglu_fwd)):
            cols = 2 * n if "epilogue" in call.__name__ else n
            held = torch.full((m + 600, cols), 7.0, dtype=out, device=DEV)
            call(x, wq, activation="relu", out_dtype=out, out=held[300:300 + m])
            assert (held[300:300 + m] != 7).any()
            assert (held[:300] == 7).all() and (held[300 + m:] == 7).all(), call.__name__


W_SHAPES = [(1, 1, 32), (1, 256, 256), (1, 4096, 512), (2, 130, 1024), (3, 17, 96), (4, 64, 2080),
            (5, 33, 1056), (7, 300, 64), (16, 512, 1024), (17, 100, 288), (31, 63, 544),
            (33, 16, 2048), (61, 259, 1312), (64, 1024, 512), (65, 40, 352), (130, 96, 160),
            (16, 3, 12320), (1, 6000, 128), (24, 9000, 64), (60, 9000, 64)]


@pytest.mark.parametrize("m,n,k", W_SHAPES)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_wlinear_epilogue(fos, m, n, k, gated, fmt):
    nv = fmt == "nvfp4"
    i = W_SHAPES.index((m, n, k))
    act = FF.ACTIVATIONS[(i + 3 * gated + nv) % 5]
    out = BF16 if (i + gated) % 3 else torch.float32
    rows = 2 * n if gated else n
    wd, ws, wt, wq = (nv_weight if nv else mx_weight)(fos, rows, k, n + k)
    wide = torch.full((m, k + 24), float("nan"), dtype=BF16, device=DEV)
    wide[:, 8:8 + k] = W.random_bf16(m, k, m + k, "student_t").to(DEV)
    x = wide[:, 8:8 + k]
    bias = W.random_bf16(1, rows, m, "normal")[0].to(DEV) if i % 2 else None
    res = W.random_bf16(m, n, n, "normal").to(DEV) if not gated and i % 3 == 0 else None
    kw = dict(bias=bias, activation=act, out_dtype=out, return_preact=i % 2 == 0)
    if gated:
        f = fos.wglu_fwd if nv else fos.mx_wglu_fwd
    else:
        f = fos.wlinear_epilogue_fwd if nv else fos.mx_wlinear_epilogue_fwd
        kw["residual"] = res
    got = f(x, wq, **kw)
    y, z = got if kw["return_preact"] else (got, None)
    b = operand_exact(wd, ws) * wt if nv else MX.operand_exact(wd, ws)
    check_epilogue(y, z, f64(x), b, None if bias is None else f64(bias), act, gated,
                   None if res is None else f64(res), k)


@pytest.mark.parametrize("m", [1, 20])
def test_wlinear_epilogue_residual_in_place(fos, m):
    n, k = 272, 512
    _, _, _, wq = mx_weight(fos, n, k, 4)
    x, res = W.random_bf16(m, k, 1, "normal").to(DEV), W.random_bf16(m, n, 5, "normal").to(DEV)
    want = fos.mx_wlinear_epilogue_fwd(x, wq, residual=res)
    stream = torch.full((m + 2, n), 7.0, dtype=BF16, device=DEV)
    stream[1:-1] = res
    fos.mx_wlinear_epilogue_fwd(x, wq, residual=stream[1:-1], out=stream[1:-1])
    assert torch.equal(stream[1:-1], want)
    assert (stream[0] == 7).all() and (stream[-1] == 7).all()


@pytest.mark.parametrize("m", [1, 5, 40, 65])
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_plain_weight_only_product_between_epilogues(fos, m, fmt):
    """A plain product has no epilogue, whatever calls came before it."""
    nv = fmt == "nvfp4"
    n, k = 40, 352
    wd, ws, wt, wq = (nv_weight if nv else mx_weight)(fos, n, k, m)
    x, bias = W.random_bf16(m, k, 1, "normal").to(DEV), W.random_bf16(1, n, 2, "normal")[0].to(DEV)
    plain = fos.wlinear_fwd if nv else fos.mx_wlinear_fwd
    glu = fos.wglu_fwd if nv else fos.mx_wglu_fwd
    epi = fos.wlinear_epilogue_fwd if nv else fos.mx_wlinear_epilogue_fwd
    b = operand_exact(wd, ws) * wt if nv else MX.operand_exact(wd, ws)
    for i in range(8):
        glu(x, wq, activation="gelu", bias=bias, return_preact=True)
        y = plain(x, wq, bias=bias, out_dtype=torch.float32)
        check_epilogue(y, None, f64(x), b, f64(bias), "none", False, None, k)
        epi(x, wq, activation="silu", bias=bias, residual=y.to(BF16), return_preact=True)
        assert torch.equal(plain(x, wq, bias=bias, out_dtype=torch.float32), y)


def test_wlinear_epilogue_of_no_rows(fos):
    _, _, _, wq = nv_weight(fos, 32, 64, 1)
    x = torch.empty(0, 64, dtype=BF16, device=DEV)
    assert fos.wlinear_epilogue_fwd(x, wq, activation="silu").shape == (0, 32)
    y, z = fos.wglu_fwd(x, wq, return_preact=True)
    assert y.shape == (0, 16) and z.shape == (0, 32)


@pytest.mark.parametrize("act", FF.ACTIVATIONS)
def test_a_nan_is_kept(fos, act):
    """A NaN in a bias, a residual or an activation row gives NaN in its column, element or row
    and nowhere else, and a NaN pre-activation a NaN gradient."""
    m, n, k = 20, 64, 512
    _, _, _, xq = nv_act(fos, m, k, 1)
    _, _, _, wq = nv_weight(fos, n, k, 2)
    _, _, _, mxq = mx_weight(fos, m, k, 1)
    _, _, _, mwq = mx_weight(fos, n, k, 2)
    x = W.random_bf16(m, k, 3, "normal").to(DEV)
    bias, res = W.random_bf16(1, n, 4, "normal")[0].to(DEV), W.random_bf16(m, n, 5, "normal").to(DEV)
    nan_bias, nan_res, nan_x = bias.clone(), res.clone(), x.clone()
    nan_bias[5] = nan_res[3, 7] = nan_x[2, 100] = float("nan")
    for f, a, w in ((fos.qlinear_epilogue_fwd, xq, wq), (fos.mx_qlinear_epilogue_fwd, mxq, mwq),
                    (fos.wlinear_epilogue_fwd, x, wq), (fos.mx_wlinear_epilogue_fwd, x, mwq),
                    (fos.wlinear_epilogue_fwd, x[:2], wq)):
        r, rn = res[:f(a, w).shape[0]], nan_res[:f(a, w).shape[0]]
        want = f(a, w, bias=bias, activation=act, residual=r)
        got = f(a, w, bias=nan_bias, activation=act, residual=rn)
        bad = rn.isnan()
        bad[:, 5] = True
        assert torch.equal(got.isnan(), bad) and torch.equal(got[~bad], want[~bad])
    for w in (wq, mwq):
        f = fos.wlinear_epilogue_fwd if w is wq else fos.mx_wlinear_epilogue_fwd
        want, got = f(x, w, activation=act), f(nan_x, w, activation=act)
        keep = torch.arange(m, device=DEV) != 2
        assert got[2].isnan().all() and torch.equal(got[keep], want[keep])
    z = res.clone()
    want, got = fos.epilogue_bwd(res, z, act), fos.epilogue_bwd(res, nan_res, act)
    there = nan_res.isnan()
    assert torch.equal(got[~there], want[~there])
    assert act in ("none", "relu") or got[there].isnan().all()      # their slopes do not take z's value
    g = fos.epilogue_bwd(res[:, :32].contiguous(), nan_res, act, gated=True)
    assert g[3, 39].isnan() and (act in ("none", "relu") or g[3, 7].isnan())
    n = fos.rmsnorm_fwd(nan_x, torch.ones(k, dtype=BF16, device=DEV)).y
    assert n[2].isnan().all() and not n[3:].isnan().any()


# --------------------------------------------------------------------------- backward

B_SHAPES = [(1, 1), (1, 16), (3, 8), (17, 33), (64, 512), (5, 520), (130, 1000), (300, 72), (2100, 64),
            (70, 4099), (5000, 8)]


@pytest.mark.parametrize("m,n", B_SHAPES)
@pytest.mark.parametrize("gated", [False, True])
def test_epilogue_bwd(fos, m, n, gated):
    act = FF.ACTIVATIONS[(B_SHAPES.index((m, n)) + 2 * gated) % 5]
    z = W.random_bf16(m, 2 * n if gated else n, m + n, "student_t").to(DEV)
    dy = W.random_bf16(m, n, m, "normal", scale=0.1).to(DEV)
    check_bwd(fos, dy, z, act, gated)


def check_bwd(fos, dy, z, act, gated):
    dz, dbias, t = fos.epilogue_bwd(dy, z, act, gated=gated, return_dbias=True, return_tensor_scale=True)
    d, zz = f64(dy), f64(z)
    ref = FF.epilogue_bwd64(d, zz, act, gated)
    half = d.shape[1]
    gate = zz[:, :half]
    slope = 32 * U * (1 + np.minimum(np.abs(gate), 16)) + 2 * U * np.abs(FF.activation64(act, gate)[1])
    if gated:
        value = 16 * U * (1 + np.abs(gate))
        err = np.concatenate((np.abs(d * zz[:, half:]) * slope, np.abs(d) * value), 1) + 2 * U * np.abs(ref)
    else:
        err = np.abs(d) * slope + 2 * U * np.abs(ref)
    within(f64(dz), ref, 2.0 ** -8 * (np.abs(ref) + err) + err + 2.0 ** -133, "dz")
    m = d.shape[0]
    within(dbias.cpu().double().numpy(), ref.sum(0), (err + (m + 1) * U * np.abs(ref)).sum(0) + 2.0 ** -126,
           "dbias")
    assert float(t) == float(N.tensor_scale_from_amax(np.float32(f64(dz).__abs__().max())))
    assert torch.equal(fos.epilogue_bwd(dy, z, act, gated=gated), dz)
    again = fos.epilogue_bwd(dy, z, act, gated=gated, return_dbias=True)
    assert torch.equal(again[0], dz) and torch.equal(again[1], dbias)
    only = fos.epilogue_bwd(dy, z, act, gated=gated, return_tensor_scale=True)
    assert torch.equal(only[1], t)


@pytest.mark.parametrize("act", FF.ACTIVATIONS)
@pytest.mark.parametrize("gated", [False, True])
def test_epilogue_bwd_over_the_whole_range(fos, act, gated):
    """Every finite bf16 pre-activation (of the gate), from -3.4e38 to 3.4e38."""
    pat = np.arange(1 << 16, dtype=np.uint32).astype(np.uint16)
    pat = pat[np.isfinite(F.bf16_bits_to_f32(pat))]
    z = torch.from_numpy(pat.view(np.int16).copy()).view(BF16).to(DEV).reshape(-1, 16)
    dy = W.random_bf16(z.shape[0], 16, 1, "normal", scale=0.1).to(DEV)
    if gated:
        z = torch.cat((z, torch.full_like(z, 0.5)), 1)
        # act(z) dY of the largest z passes fp32 where |dY| is above 1
        assert float(dy.abs().max()) < 1
    dz = fos.epilogue_bwd(dy, z, act, gated=gated)
    assert torch.isfinite(dz).all()
    keep = (z[:, :16].float().abs() < 1e4).all(1)
    check_bwd(fos, dy[keep].contiguous(), z[keep].contiguous(), act, gated)
    far = f64(z[~keep][:, :16])
    want = FF.epilogue_bwd64(f64(dy[~keep]), f64(z[~keep]), act, gated)
    got = f64(dz[~keep])
    assert (np.abs(got - want) <= 2.0 ** -7 * np.abs(want) + 1e-36).all(), far


def test_epilogue_bwd_unaligned_and_empty(fos):
    z = W.random_bf16(40, 64, 1, "normal").to(DEV)
    dy = W.random_bf16(40, 64, 2, "normal").to(DEV)
    want = fos.epilogue_bwd(dy, z, "silu", return_dbias=True)
    flat = torch.empty(40 * 64 + 1, dtype=BF16, device=DEV)
    flat[1:] = z.flatten()
    got = fos.epilogue_bwd(dy, flat[1:].view(40, 64), "silu", return_dbias=True)
    assert torch.equal(got[0], want[0])
    within(got[1].cpu().double().numpy(), want[1].cpu().double().numpy(),
           2 * 41 * U * np.abs(f64(want[0])).sum(0) * (1 + 2.0 ** -7), "dbias")
    dz, dbias, t = fos.epilogue_bwd(dy[:0], z[:0], return_dbias=True, return_tensor_scale=True)
    assert dz.shape == (0, 64) and (dbias == 0).all() and float(t) == 0


@pytest.mark.parametrize("gated", [False, True])
def test_product_backward(fos, gated):
    """dX and dW are the products of the records of dZ with the given options."""
    m, n, k = 192, 128, 320
    rows = 2 * n if gated else n
    x, w = W.random_bf16(m, k, 1, "normal").to(DEV), W.random_bf16(rows, k, 2, "normal", scale=0.02).to(DEV)
    xt, wt = fos.quantize(x, outputs=("col",)), fos.quantize(w, outputs=("col",), block="2d")
    z = W.random_bf16(m, rows, 3, "normal").to(DEV)
    dy = W.random_bf16(m, n, 4, "normal", scale=1e-3).to(DEV)
    f = fos.qglu_bwd if gated else fos.qlinear_epilogue_bwd
    for rounding, seed in (("rne", None), ("sr", 5)):
        dx, dw, db = f(dy, z, xt, wt, activation="silu", return_dbias=True, rounding=rounding, sr_seed=seed)
        dz, dbias = fos.epilogue_bwd(dy, z, "silu", gated=gated, return_dbias=True)
        a, b = fos.quantize(dz, outputs=("row", "col"), rounding=rounding, sr_seed=seed)
        want = fos.qlinear_epilogue_fwd(a, wt), fos.qlinear_epilogue_fwd(b, xt)
        assert torch.equal(dx, want[0]) and torch.equal(dw, want[1]) and torch.equal(db, dbias)
        for got, q, other in ((dx, a, wt), (dw, b, xt)):
            u, v = (operand_exact(r.data.cpu().numpy(), r.scales.cpu().numpy()) * float(r.tensor_scale)
                    for r in (q, other))
            ref, size = u @ v.T, np.abs(u) @ np.abs(v).T
            err = (u.shape[1] + 8) * U * size
            within(f64(got), ref, 2.0 ** -8 * (np.abs(ref) + err) + err, "product")
    dx, none = f(dy, z, None, wt, activation="silu", need_dw=False)
    assert none is None and torch.equal(dx, f(dy, z, xt, wt, activation="silu")[0])
    none, dw = f(dy, z, xt, None, activation="silu", need_dx=False)
    assert none is None and torch.equal(dw, f(dy, z, xt, wt, activation="silu")[1])


# ------------------------------------------------------------------- refusals on the device

def test_binding_refuses_what_the_library_could_not_address(fos):
    """Wrong shapes, types and overlaps are refused on the host, before any launch."""
    x, r, w = norm_inputs(8, 64, 1, True)
    rec, up = fos.quantize(x.repeat(2, 1)), fos.quantize(x.repeat(4, 1))
    mx = fos.mx_quantize(torch.cat((x, x, x, x), 1))
    y = torch.zeros(16, 32, dtype=BF16, device=DEV)
    short = fos.NVFP4Tensor(rec.data, rec.scales[:, :2].contiguous(), rec.tensor_scale)
    turned = fos.NVFP4Tensor(rec.data, rec.scales, rec.tensor_scale, hadamard_seed=3)
    calls = [
        lambda: fos.rmsnorm_fwd(x, w[:32]), lambda: fos.rmsnorm_fwd(x.float(), w),
        lambda: fos.rmsnorm_fwd(x, w.float()), lambda: fos.rmsnorm_fwd(x.T, w),
        lambda: fos.rmsnorm_fwd(x, w, residual=r[:4]), lambda: fos.rmsnorm_fwd(x, w, format="fp8"),
        lambda: fos.rmsnorm_fwd(x, w, rule="5"), lambda: fos.rmsnorm_fwd(x, w, h=r),
        lambda: fos.rmsnorm_fwd(x, w, tensor_scale=rec.tensor_scale),
        lambda: fos.rmsnorm_fwd(x, w, format="nvfp4", tensor_scale=rec.tensor_scale.double()),
        lambda: fos.rmsnorm_fwd(x[1:5], w, residual=r[:4], h=x[:4]),
        lambda: fos.rmsnorm_fwd(x[:4], w, residual=r[1:5], h=r[:4]),
        lambda: fos.rmsnorm_bwd(x, r, w, torch.ones(4, device=DEV)),
        lambda: fos.rmsnorm_bwd(x, r[:4], w, torch.ones(8, device=DEV)),
        lambda: fos.rmsnorm_bwd(x, r, w, torch.ones(8, device=DEV), dh=x[:4]),
        lambda: fos.qlinear_epilogue_fwd(rec, mx), lambda: fos.qlinear_epilogue_fwd(rec, short),
        lambda: fos.qlinear_epilogue_fwd(rec, turned), lambda: fos.wlinear_epilogue_fwd(x, turned),
        lambda: fos.qlinear_epilogue_fwd(rec, up, bias=w), lambda: fos.qlinear_epilogue_fwd(rec, up, activation="tanh"),
        lambda: fos.qlinear_epilogue_fwd(rec, up, residual=y[:, :16]),
        lambda: fos.qlinear_epilogue_fwd(rec, up, out=y.float()),
        lambda: fos.qlinear_epilogue_fwd(rec, up, out_dtype=torch.float16),
        lambda: fos.qlinear_epilogue_fwd(rec, rec, residual=torch.zeros(17, 16, dtype=BF16, device=DEV)[1:],
                                         out=y.view(-1)[:128].view(16, 8)),
        lambda: fos.qlinear_epilogue_fwd(rec, up, residual=torch.cat((y, y))[1:17], out=y.T),
        lambda: fos.qglu_fwd(rec, fos.NVFP4Tensor(up.data[:15], up.scales[:15], up.tensor_scale)),
        lambda: fos.wlinear_epilogue_fwd(x[:, :32], rec), lambda: fos.mx_wlinear_epilogue_fwd(x, mx),
        lambda: fos.wlinear_epilogue_fwd(x.repeat(1, 2)[:, :64].T, rec),
        lambda: fos.epilogue_bwd(y, y[:8]), lambda: fos.epilogue_bwd(y, y, gated=True),
        lambda: fos.epilogue_bwd(y.float(), y), lambda: fos.epilogue_bwd(y[:, :16], y[:, :16].contiguous()),
        lambda: fos.qlinear_epilogue_bwd(y, y, None, None, need_dx=False, need_dw=False),
        lambda: fos.qlinear_epilogue_bwd(y, y, None, rec), lambda: fos.qlinear_epilogue_bwd(y, y, rec, mx),
        lambda: fos.qlinear_epilogue_bwd(y, y, None, rec, need_dw=False),
        lambda: fos.qlinear_epilogue_bwd(y, y, rec, None, need_dx=False),
        lambda: fos.qglu_bwd(y, y, None, rec, need_dw=False),
        lambda: fos.qglu_bwd(torch.cat((y, y), 1)[:, :32].contiguous(), torch.cat((y, y), 1), None, turned, need_dw=False)]
    for i, call in enumerate(calls):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was not refused")
    rows = torch.zeros(18, 32, dtype=BF16, device=DEV)
    for out in (rows[1:17], rows[2:18]):
        with pytest.raises(ValueError, match="overlaps"):
            fos.qlinear_epilogue_fwd(rec, up, residual=rows[:16], out=out)
    same = torch.zeros(16, 64, dtype=BF16, device=DEV)
    square = fos.quantize(torch.ones(64, 64, dtype=BF16, device=DEV))
    with pytest.raises(ValueError, match="overlaps"):
        fos.wlinear_epilogue_fwd(same, square, residual=same, out=same)
    with pytest.raises(fos.FosError):                    # K of 96: not a multiple of 64
        a = fos.quantize(torch.ones(16, 96, dtype=BF16, device=DEV))
        fos.qlinear_epilogue_fwd(a, a)
    with pytest.raises(fos.FosError):
        fos.rmsnorm_fwd(x, w, eps=0.0)
    with pytest.raises(fos.FosError):
        fos.rmsnorm_fwd(x[:, :40].contiguous(), w[:40].contiguous())


# --------------------------------------------------------------- together, as they are used

class Block:
    """A gated feed-forward block on NVFP4 records with its backward pass."""

    def __init__(self, fos, m, k, hidden, seed):
        self.fos, self.hidden = fos, hidden
        self.x, self.r, self.w = norm_inputs(m, k, seed, True)
        self.dout = W.random_bf16(m, k, seed + 3, "normal", scale=0.05).to(DEV)
        self.in_w = W.random_bf16(2 * hidden, k, seed + 4, "normal", scale=k ** -0.5).to(DEV)
        self.out_w = W.random_bf16(k, hidden, seed + 5, "normal", scale=hidden ** -0.5).to(DEV)
        self.win, self.win_t = fos.quantize(self.in_w, block="2d", outputs=("row", "col"))
        self.wout, self.wout_t = fos.quantize(self.out_w, block="2d", outputs=("row", "col"))

    def inputs(self, seed):
        m, k = self.x.shape
        for t, s in ((self.x, 0), (self.r, 1), (self.dout, 2)):
            t.copy_(W.random_bf16(m, k, seed + s, "normal", scale=(1.0, 3.0, 0.05)[s]))

    def forward(self):
        f = self.fos
        n = f.rmsnorm_fwd(self.x, self.w, residual=self.r, format="nvfp4", return_y=True)
        y, z = f.qglu_fwd(n.record, self.win, return_preact=True)
        a, at = f.quantize(y, outputs=("row", "col"))
        out = f.qlinear_epilogue_fwd(a, self.wout, residual=n.h)
        return dict(n=n, y=y, z=z, a=a, at=at, out=out)

    def backward(self, s):
        f = self.fos
        dq, dqt = f.quantize(self.dout, outputs=("row", "col"))
        da, dw_out = f.qlinear_bwd(dq, dqt, s["at"], self.wout_t)
        xt = f.quantize(s["n"].y, outputs=("col",))
        dx, dw_in, db = f.qglu_bwd(da, s["z"], xt, self.win_t, return_dbias=True)
        dh, dw = f.rmsnorm_bwd(dx, s["n"].h, self.w, s["n"].rstd, dh=self.dout)
        return dict(da=da, dw_out=dw_out, dx=dx, dw_in=dw_in, db=db, dh=dh, dw=dw)

    def run(self):
        s = self.forward()
        g = self.backward(s)
        n = s["n"]
        return [n.h, n.rstd, n.y, n.record.data, n.record.scales, n.record.tensor_scale, s["y"], s["z"],
                s["out"], *g.values()]


def values_of(q):
    return operand_exact(q.data.cpu().numpy(), q.scales.cpu().numpy()) * float(q.tensor_scale)


@pytest.mark.parametrize("m,k,hidden", [(64, 128, 64), (192, 320, 448), (320, 1024, 192)])
def test_block_forward_and_backward(fos, m, k, hidden):
    """Every stage against the references, from what the stage before it gave."""
    b = Block(fos, m, k, hidden, m)
    s = b.forward()
    g = b.backward(s)
    n = s["n"]
    yb = check_norm(n, b.x, b.r, b.w, 1e-6)
    assert torch.equal(n.y.cpu(), yb)
    q = fos.quantize(n.y)
    assert torch.equal(n.record.data, q.data) and torch.equal(n.record.scales, q.scales)
    assert torch.equal(n.record.tensor_scale, q.tensor_scale)
    check_epilogue(s["y"], s["z"], values_of(n.record), values_of(b.win), None, "silu", True, None, k)
    check_epilogue(s["out"], None, values_of(s["a"]), values_of(b.wout), None, "none", False, f64(n.h), hidden)
    check_bwd(fos, g["da"], s["z"], "silu", True)
    dz, db, t = fos.epilogue_bwd(g["da"], s["z"], "silu", gated=True, return_dbias=True, return_tensor_scale=True)
    assert torch.equal(db, g["db"])
    rows, cols = fos.quantize(dz, outputs=("row", "col"))
    xt = fos.quantize(n.y, outputs=("col",))
    for got, u, v in ((g["dx"], rows, b.win_t), (g["dw_in"], cols, xt)):
        u, v = values_of(u), values_of(v)
        err = (u.shape[1] + 8) * U * (np.abs(u) @ np.abs(v).T)
        within(f64(got), u @ v.T, 2.0 ** -8 * (np.abs(u @ v.T) + err) + err, "product")
    ref, rdw, size, sdw = FF.rmsnorm_bwd64(f64(g["dx"]), f64(n.h), f64(b.w), n.rstd.cpu().double().numpy(),
                                           f64(b.dout))
    err = (k + 12) * U * size
    within(f64(g["dh"]), ref, 2.0 ** -8 * (np.abs(ref) + err) + err, "dh")
    within(g["dw"].cpu().double().numpy(), rdw, (m + 4) * U * sdw, "dw")


def same(got, want):
    return all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, want, strict=True))


def test_block_replayed_from_graphs(fos):
    """The whole step, forward and backward, captured and replayed with new inputs and eager
    work between; a second graph of it, captured meanwhile, replays beside the first."""
    blocks = [Block(fos, 192, 320, 448, 1), Block(fos, 128, 512, 320, 2)]
    graphs, outs, sides = [], [], [torch.cuda.Stream() for _ in blocks]
    for b, side in zip(blocks, sides):
        side.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            outs.append(b.run())
        graphs.append(g)
    for i in range(4):
        for b in blocks:
            b.inputs(10 * i + 5)
        torch.cuda.synchronize()
        for g, side in zip(graphs, sides):          # at the same time, on streams of their own
            with torch.cuda.stream(side):
                g.replay()
        torch.cuda.synchronize()
        for b, got in zip(blocks, outs):
            assert same(got, b.run()), i
        torch.cuda.synchronize()


def test_backward_captured_while_eager_results_live(fos):
    """The forward pass ran eagerly; the backward pass of what it left is captured."""
    b = Block(fos, 128, 256, 192, 3)
    s = b.forward()
    want = b.backward(s)
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        got = b.backward(s)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert same(got.values(), want.values())
        assert same(b.backward(s).values(), want.values())


def test_decode_block_on_two_streams(fos):
    """The few-row path (norm, gated product, product with the residual in place), issued on
    two streams at once, gives each its own results."""
    k, hidden, m = 1024, 768, 3
    _, _, _, win = nv_weight(fos, 2 * hidden, k, 1)
    _, _, _, wout = mx_weight(fos, k, hidden, 2)
    _, _, w = norm_inputs(1, k, 3, False)
    xs = [W.random_bf16(m, k, 7 + i, "normal").to(DEV) for i in range(2)]

    def step(x, h):
        n = fos.rmsnorm_fwd(x, w)
        u = fos.wglu_fwd(n.y, win, activation="gelu_tanh")
        fos.mx_wlinear_epilogue_fwd(u, wout, residual=h, out=h)
        t = fos.rmsnorm_fwd(h, w, format="nvfp4")
        return h, t.record.data, t.record.scales, t.record.tensor_scale

    want = [step(x, x.clone()) for x in xs]
    hs = [[x.clone() for _ in range(20)] for x in xs]
    sides = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    got = [[], []]
    for i in range(20):
        for j, side in enumerate(sides):
            with torch.cuda.stream(side):
                got[j].append(step(xs[j], hs[j][i]))
    torch.cuda.synchronize()
    for j in range(2):
        for g in got[j]:
            assert same(g, want[j])


# ------------------------------------------------------------------------- past 32 bits

def test_rows_past_32_bit_offsets(fos):
    """More than 2^31 elements: the last rows are those of a call on them alone."""
    m, k = 66000, 32768
    gen = torch.Generator(device=DEV).manual_seed(1)
    x = torch.empty(m, k, dtype=BF16, device=DEV).normal_(generator=gen)
    w = W.random_bf16(1, k, 2, "normal")[0].to(DEV)
    t = torch.full((1,), 2.0 ** -6, device=DEV)
    last = slice(m - 3, m)
    n = fos.rmsnorm_fwd(x, w, format="nvfp4", tensor_scale=t, return_y=True)
    few = fos.rmsnorm_fwd(x[last], w, format="nvfp4", tensor_scale=t, return_y=True)
    assert same([n.rstd[last], n.y[last], n.record.data[last], n.record.scales[last]],
                [few.rstd, few.y, few.record.data, few.record.scales])
    y = n.y
    del n
    dx, _ = fos.rmsnorm_bwd(y, x, w, fos.rmsnorm_fwd(x, w).rstd)
    assert torch.equal(dx[last], fos.rmsnorm_bwd(y[last], x[last], w, few.rstd)[0])
    del dx
    dz = fos.epilogue_bwd(y, x, "silu")
    assert torch.equal(dz[last], fos.epilogue_bwd(y[last], x[last], "silu"))


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_outputs_past_32_bit_offsets(fos, fmt):
    m, n, k = 140000, 16400, 256
    nv = fmt == "nvfp4"
    a, b = (W.random_bf16(r, k, s, "normal").to(DEV) for r, s in ((m, 1), (n, 2)))
    make = fos.quantize if nv else fos.mx_quantize
    f = fos.qlinear_epilogue_fwd if nv else fos.mx_qlinear_epilogue_fwd
    aq, bq = make(a), make(b)
    res = torch.zeros(m, n, dtype=BF16, device=DEV)
    last = slice(m - 5, m)
    res[last] = W.random_bf16(5, n, 3, "normal").to(DEV)
    f(aq, bq, activation="silu", residual=res, out=(y := res))
    want = W.random_bf16(5, n, 3, "normal")
    if nv:
        u, v = operand_exact(aq.data[last].cpu().numpy(), aq.scales[last].cpu().numpy()), values_of(bq)
        u = u * float(aq.tensor_scale)
    else:
        u, v = (MX.operand_exact(q.cpu().numpy(), s.cpu().numpy())
                for q, s in ((aq.data[last], aq.scales[last]), (bq.data, bq.scales)))
    check_epilogue(y[last], None, u, v, None, "silu", False, f64(want), k)
