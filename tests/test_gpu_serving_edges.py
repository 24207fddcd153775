"""GPU tests of the token-serving operators at the ends of their ranges.  Bounds as in
test_gpu_serving.py, with what a test claims beyond them said there.
"""
import ctypes

import numpy as np
import pytest
import torch

import test_gpu_serving as T
from fp4_block_quantization_amd import workloads as W
from oracle import formats as F
from oracle import nvfp4 as N
from oracle import serving as S
from test_gpu_serving import DEV, FMTS, U, dev, f64, fos, within  # noqa: F401
from test_serving_abi import Devices

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


# More than 1024 weight rows and more than four activation rows are products of 16x16x32 tiles
# (fewer weight rows fit the GPU as groups of 4 or 8 that get a CU each and take the kernel
# of few rows).

def records(fmt):
    return T.nv_weight if fmt == "nvfp4" else T.mx_weight


def linear(fos, fmt):
    return fos.wlinear_fwd if fmt == "nvfp4" else fos.mx_wlinear_fwd


def some_rows(n):
    return np.unique(np.concatenate([np.arange(0, n, 37), np.arange(16), np.arange(n - 70, n)]))


@pytest.mark.parametrize("m", [5, 16, 24, 40, 64])
@pytest.mark.parametrize("k", [16, 48, 80, 1008, 4112])
def test_wlinear_tiles_of_rows_that_end_in_half_a_load(fos, m, k):
    """K a multiple of 16 but not of 32: a weight row starts at 8-byte alignment."""
    n = 1203
    data, scales, t, w = T.nv_weight(fos, n, k, m + k)
    x = W.random_bf16(m, k, k, "normal").to(DEV)
    T.check_linear(fos.wlinear_fwd(x, w, out_dtype=torch.float32), x, data, scales, t, rows=some_rows(n))


@pytest.mark.parametrize("m,n", [(5, 1203), (16, 2050), (9, 6000), (16, 8200), (250, 1000), (17, 12300),
                                 (61, 4099), (33, 16400), (100, 6000)])
@pytest.mark.parametrize("fmt,k,out", [("nvfp4", 304, torch.float32), ("nvfp4", 1056, torch.bfloat16),
                                       ("mxfp4", 1056, torch.float32)])
def test_wlinear_tiles_with_bias_strided_rows_and_given_output(fos, m, n, fmt, k, out):
    """Sizes for which the GPU is filled with each of the tiles; NaN next to the activation
    rows, and rows of the output next to the given ones that stay."""
    data, scales, t, w = records(fmt)(fos, n, k, m + n)
    wide = torch.full((m, k + 72), float("nan"), dtype=torch.bfloat16, device=DEV)
    x = wide[:, 40:40 + k]
    x.copy_(W.random_bf16(m, k, n, "normal"))
    bias = W.random_bf16(1, n, 3, "normal")[0].to(DEV)
    full = torch.full((m + 2, n), 7.0, dtype=out, device=DEV)
    y = linear(fos, fmt)(x, w, bias=bias, out_dtype=out, out=full[1:m + 1])
    rows = some_rows(n)
    ref, mag = S.wlinear_ref64(f64(x), data, scales, t, rows=rows)
    ref, mag = ref + f64(bias)[rows], mag + np.abs(f64(bias)[rows])
    rnd = 2.0 ** -8 if out == torch.bfloat16 else U
    within(f64(y[:, dev(rows)]), ref, rnd * np.abs(ref) + (k + 8) * U * mag * (1 + rnd), "y")
    assert not y.isnan().any() and (full[0] == 7).all() and (full[m + 1] == 7).all()


@pytest.mark.parametrize("m", [6, 32, 64])
@pytest.mark.parametrize("block", ["1d", "2d"])
def test_wlinear_tiles_of_wide_values(fos, m, block):
    """Activations from 2^-100 to 2^100 side by side, a weight that uses the whole range of
    block scales, and a 2D record."""
    n, k = 1200, 1024
    data, scales, t, w = T.nv_weight(fos, n, k, 9, N.Config(block=block), scale=1.0)
    g = np.random.RandomState(m)
    x = np.ldexp(g.randn(m, k), g.randint(-100, 100, (m, k)))
    x = T.to_gpu_bf16(F.f32_to_bf16_bits(x.astype(np.float32)))
    T.check_linear(fos.wlinear_fwd(x, w, out_dtype=torch.float32), x, data, scales, t, rows=some_rows(n))


@pytest.mark.parametrize("m", [9, 33, 64])
@pytest.mark.parametrize("lo,hi,e", [(0, 7, 100), (7, 120, 60), (100, 150, 0), (130, 228, -60), (228, 253, -100)])
def test_mx_wlinear_tiles_of_every_block_scale(fos, m, lo, hi, e):
    """E8M0 codes from 0 (2^-127, where the weights are below bf16's normal range) to the
    largest whose products with E2M1 are finite."""
    n, k = 1200, 640
    g = np.random.RandomState(m)
    data = g.randint(0, 256, (n, k // 2)).astype(np.uint8)
    scales = g.randint(lo, hi, (n, k // 32)).astype(np.uint8)
    x = T.to_gpu_bf16(F.f32_to_bf16_bits(np.ldexp(g.randn(m, k), e).astype(np.float32)))
    y = fos.mx_wlinear_fwd(x, fos.MXFP4Tensor(dev(data), dev(scales)), out_dtype=torch.float32)
    T.check_linear(y, x, data, scales, None, rows=some_rows(n))


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


def one_sequence(fos, fmt, k, v, page=16):
    """A cache with these rows (bf16 [tokens, heads, dim]) as one sequence, and what to call
    paged_decode with."""
    n, heads, dim = k.shape
    pages = -(-n // page)
    cache = T.new_cache(fos, fmt, pages, page, heads, dim)
    fos.kv_append(cache, k.to(DEV), v.to(DEV), torch.arange(n, device=DEV))
    return cache, (torch.arange(pages, dtype=torch.int32, device=DEV)[None],
                   torch.tensor([n], dtype=torch.int32, device=DEV))


@FMTS
@pytest.mark.parametrize("top,others,scale", [(10, 0, None), (17, 0, None), (20, 0, None), (24, 0, None),
                                              (45, 0, None), (100, 0, 0.25), (0, -100, 1e30),
                                              (-3, -20, 1e5)])
def test_decode_query_of_wide_range(fos, fmt, top, others, scale):
    """Some heads have a value of 2^top beside others of about 2^others, where K is zero: the
    scores are the others'."""
    n, Hq, Hkv, D = 300, 8, 2, 128
    k = W.random_bf16(n, Hkv * D, 1, "normal").view(n, Hkv, D)
    v = W.random_bf16(n, Hkv * D, 2, "normal").view(n, Hkv, D)
    q = W.random_bf16(Hq, D, 3, "normal", scale=2.0 ** others)
    for h, d in ((0, 5), (1, 126), (6, 64)):
        q[h, d] = 1.75 * 2.0 ** top
        k[:, h // 4, d] = 0.0
    cache, args = one_sequence(fos, fmt, k, v)
    out, lse = fos.paged_decode(q[None].to(DEV), cache, *args, scale=scale, return_lse=True)
    kk, vv = (T.N_rows(cache, name)[:n] for name in "kv")
    T.check_attention(out[0], lse[0], f64(q), kk, vv, D ** -0.5 if scale is None else scale)


@FMTS
@pytest.mark.parametrize("top,others,scale", [(127, 0, 2.0), (60, -100, 1e30), (127, -100, 1e30),
                                              (-100, -120, 1e36), (127, 120, 2.0 ** -119)])
def test_decode_query_and_scale_at_their_ends(fos, fmt, top, others, scale):
    """The same at the ends of the range of bf16, with a scale that the large values alone
    would take past fp32."""
    test_decode_query_of_wide_range(fos, fmt, top, others, scale)


@FMTS
@pytest.mark.parametrize("q", [1.0, 2.0 ** 127])
def test_decode_scores_of_zero_under_any_scale(fos, fmt, q):
    """K is 0: every token has the same weight, however large the query and the scale."""
    n = 70
    v = W.random_bf16(n, 64, 2, "normal").view(n, 1, 64)
    cache, args = one_sequence(fos, fmt, torch.zeros(n, 1, 64, dtype=torch.bfloat16), v)
    out, lse = fos.paged_decode(torch.full((1, 1, 64), q, dtype=torch.bfloat16, device=DEV), cache, *args,
                                scale=3.4e38, return_lse=True)
    T.check_attention(out[0], lse[0], np.zeros((1, 64)), np.zeros((n, 1, 64)), T.N_rows(cache, "v")[:n], 1.0)


@FMTS
@pytest.mark.parametrize("n", [3, 60, 64, 1000])
@pytest.mark.parametrize("gap", [8.0, 12.0, 16.0, 24.0, 28.0, 30.0, 33.0, 36.0, 56.0])
def test_decode_beside_a_token_that_takes_the_weight(fos, fmt, n, gap):
    """The first token's score is about ``gap`` above all others and its value is 0: the output
    is what the others leave.  A weight may be rounded to 11 bits, or by 2^-32 of the largest
    weight if that is more."""
    Hq, Hkv, D = 4, 2, 64
    k = W.random_bf16(n, Hkv * D, 1, "normal", scale=0.25).view(n, Hkv, D)
    v = W.random_bf16(n, Hkv * D, 2, "uniform").view(n, Hkv, D) + 2.0
    q = torch.ones(Hq, D, dtype=torch.bfloat16)
    k[0], v[0] = gap / D, 0.0
    cache, args = one_sequence(fos, fmt, k.bfloat16(), v.bfloat16())
    out, lse = fos.paged_decode(q[None].to(DEV), cache, *args, scale=1.0, return_lse=True)
    kk, vv = (T.N_rows(cache, name)[:n] for name in "kv")
    ref, rl, A, V, E = S.attend_ref64(f64(q), kk, vv, 1.0)
    dS, adds = (D + 8) * U * A, (n / 4 + 64) * U
    rel = 2 * dS + 2.0 ** -20 + adds + 2.0 ** -11
    low = n * 2.0 ** -32 * np.abs(vv).max(axis=0).repeat(2, axis=0) / E[:, None]
    within(f64(out[0]), ref, 2.0 ** -8 * np.abs(ref) + (rel[:, None] * V + low) * (1 + 2.0 ** -8)
           + 2.0 ** -133, "out")
    within(f64(lse[0]), rl, dS + 2.0 ** -20 + adds + 4 * U * np.abs(rl), "lse")


def test_every_call_runs_on_the_device_of_its_tensors(fos, monkeypatch):
    """With another device current, each call makes its tensors' device current for its launch
    and for what it asks about the stream's capture."""
    t = torch.ones(1, device=DEV)
    cache = fos.kv_cache(4, 16, 2, 64, "nvfp4", t, t, device=DEV)
    x = torch.ones(3, 128, dtype=torch.bfloat16, device=DEV)
    k, slots = x.view(3, 2, 64), torch.arange(3, device=DEV)
    table = torch.arange(4, dtype=torch.int32, device=DEV).expand(3, 4).contiguous()
    lens = torch.full((3,), 3, dtype=torch.int32, device=DEV)
    w, mx = fos.quantize(x), fos.mx_quantize(x)
    calls = [lambda: fos.wlinear_fwd(x, w), lambda: fos.mx_wlinear_fwd(x, mx),
             lambda: fos.kv_append(cache, k, k, slots), lambda: fos.kv_gather(cache, slots),
             lambda: fos.paged_decode(k, cache, table, lens)]
    want = [f() for f in calls]
    index = torch.device(DEV).index
    devices = Devices(monkeypatch, current=index + 5)
    for f, y in zip(calls, want):
        devices.entered.clear()
        got = f()
        assert devices.entered and set(devices.entered) == {index}
        for a, b in zip(got if isinstance(got, tuple) else (got,), y if isinstance(y, tuple) else (y,)):
            assert a is b is None or torch.equal(a, b)
    devices.current = index
    devices.entered.clear()
    for f in calls:
        f()
    assert not devices.entered


@FMTS
def test_decode_batch_of_several_launches(fos, fmt):
    """64 kv heads and 1030 sequences are more segments than a launch counts (65536): the
    second one starts at sequence 1024.  Long sequences on both sides of it leave partial
    results."""
    lens = np.random.RandomState(3).randint(0, 20, 1030)
    lens[[0, 500, 1022, 1023, 1024, 1027, 1029]] = 700, 24000, 0, 1500, 1300, 900, 600
    T.run_decode(fos, fmt, 1030, 64, 64, 32, 16, lens, seed=51)


@FMTS
@pytest.mark.parametrize("Hq,Hkv,D,lens", [(800, 800, 32, [40, 0, 600]), (300, 300, 160, [30, 5, 300]),
                                           (1036, 518, 128, [17, 270]), (5100, 300, 160, [3, 290])])
def test_decode_more_head_groups_than_fit_at_once(fos, fmt, Hq, Hkv, D, lens):
    """Head groups that are more than the workgroups the GPU holds (256 to 768, by head dim):
    one workgroup of each walks every sequence."""
    T.run_decode(fos, fmt, len(lens), Hq, Hkv, D, 16, lens, seed=52)


def test_decode_infinities_where_masked(fos, monkeypatch):
    """Infinities of either sign, alone, together and beside NaN, past the length, before the
    window and in foreign pages of a bf16 cache leave no trace, at every offset of the length
    inside a tile."""
    inf, nan = float("inf"), float("nan")
    for values in ((inf,), (-inf,), (inf, -inf), (inf, nan, -inf, 3.0e38)):
        def fill(cache):
            for x in (cache.k, cache.v):
                x.view(-1)[:] = torch.tensor(values, device=DEV).bfloat16().repeat(
                    -(-x.numel() // len(values)))[:x.numel()]
        monkeypatch.setattr(T, "fill_garbage", fill)
        T.run_decode(fos, "bf16", 40, 2, 2, 64, 16, list(range(90, 130)), window=45, seed=15)
        T.run_decode(fos, "bf16", 7, 6, 3, 96, 16, [90, 16, 1, 333, 700, 64, 65], holes=True, seed=8)
