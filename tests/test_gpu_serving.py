"""GPU tests of the token-serving operators against fp64 references (oracle/serving.py)
and, for what is stored, the oracle's records bit for bit.

Bounds (u = 2^-24).  A product of a bf16 and a dequantized 4-bit value is exact in fp32,
so a sum of n of them in any order is off by at most n u S, S the sum of magnitudes; the
scale, the bias and the exponent of the softmax add a few u.  Rounding to bf16 adds
2^-8 of the value (8 significant bits), to fp32 u.

Attention: a score is off by at most dS = ((D + 8) u) A, A its magnitude sum; the weight
exp(s - lse) then by the factor 2 dS + 2^-20 (argument and exponential).  The weights may
enter the product with V rounded to 11 bits or more (2^-11 each, and 2^-25 of the largest
weight for those below the half-precision range), and each accumulator takes at most
L/4 + 64 rounded additions of L tokens.
"""
import numpy as np
import pytest
import torch

from fp4_block_quantization_amd import workloads as W
from oracle import formats as F
from oracle import mxfp4 as MX
from oracle import nvfp4 as N
from oracle import serving as S
from test_gpu_parity import assert_same_bytes, bits_of, to_gpu_bf16

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24


@pytest.fixture(scope="module")
def fos():
    from fp4_block_quantization_amd import fos as mod
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    return mod


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def within(got, ref, bound, what):
    bad = ~(np.abs(got - ref) <= bound)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} outside, worst "
                           f"{np.nanmax(np.abs(got - ref) / np.maximum(bound, 1e-300)):.3g} of the bound, "
                           f"first at {np.argwhere(bad)[0].tolist()}")


# ------------------------------------------------------------------ weight-only linear

def nv_weight(fos, n, k, seed, cfg=N.Config(), scale=0.02):
    o = N.quantize(bits_of(W.random_bf16(n, k, seed, "normal", scale=scale, outlier_every=97)), cfg)
    t = torch.tensor([o["t"]], dtype=torch.float32, device=DEV)
    return o["row_data"], o["row_scales"], float(o["t"]), \
        fos.NVFP4Tensor(dev(o["row_data"]), dev(o["row_scales"]), t, block=cfg.block)


def mx_weight(fos, n, k, seed, scale=0.02):
    o = MX.quantize(bits_of(W.random_bf16(n, k, seed, "normal", scale=scale, outlier_every=97)))
    return o["data"], o["scales"], None, fos.MXFP4Tensor(dev(o["data"]), dev(o["scales"]))


def check_linear(y, x, data, scales, t, bias=None, rows=None):
    ref, mag = S.wlinear_ref64(f64(x), data, scales, t, None if bias is None else f64(bias), rows)
    got = f64(y) if rows is None else f64(y)[:, rows]
    rnd = 2.0 ** -8 if y.dtype == torch.bfloat16 else U
    # the smallest normal bf16 / fp32 step for results that round to subnormals
    within(got, ref, rnd * np.abs(ref) + (x.shape[1] + 8) * U * mag * (1 + rnd) + 2.0 ** -133, "y")


SHAPES = [(1, 1, 32), (1, 256, 256), (1, 4096, 512), (2, 130, 4096), (3, 17, 96), (4, 64, 2080),
          (5, 33, 1056), (7, 300, 64), (8, 48, 4128), (16, 512, 1024), (17, 100, 288),
          (31, 63, 544), (32, 4096, 128), (33, 16, 2048), (61, 259, 1312), (64, 1024, 512),
          (65, 40, 352), (130, 96, 160), (1, 5, 12288), (16, 3, 12320), (64, 2, 4096)]


@pytest.mark.parametrize("m,n,k", SHAPES)
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_wlinear(fos, m, n, k, fmt, out):
    data, scales, t, w = (nv_weight if fmt == "nvfp4" else mx_weight)(fos, n, k, m + n + k)
    f = fos.wlinear_fwd if fmt == "nvfp4" else fos.mx_wlinear_fwd
    x = W.random_bf16(m, k, 3 * m + k, "student_t").to(DEV)
    bias = W.random_bf16(1, n, m, "normal")[0].to(DEV) if (m + n) % 2 else None
    y = f(x, w, bias=bias, out_dtype=out)
    check_linear(y, x, data, scales, t, bias)
    assert torch.equal(y, f(x, w, bias=bias, out_dtype=out))        # the same every time


@pytest.mark.parametrize("m", [1, 2, 3, 5, 16, 40, 64])
@pytest.mark.parametrize("k", [16, 48, 80, 1008, 4112])
def test_wlinear_rows_that_end_in_half_a_load(fos, m, k):
    """K a multiple of 16 but not of 32: a weight row starts at 8-byte alignment."""
    data, scales, t, w = nv_weight(fos, 77, k, m + k)
    x = W.random_bf16(m, k, k, "normal").to(DEV)
    check_linear(fos.wlinear_fwd(x, w, out_dtype=torch.float32), x, data, scales, t)


@pytest.mark.parametrize("m", [1, 4, 24])
def test_wlinear_strided_rows_and_given_output(fos, m):
    n, k = 96, 320
    data, scales, t, w = nv_weight(fos, n, k, 5)
    wide = W.random_bf16(m, k + 72, 6, "normal").to(DEV)
    wide[:, :40], wide[:, 40 + k:] = float("nan"), float("nan")     # next to the rows
    x = wide[:, 40:40 + k]
    out = torch.full((m + 2, n), 7.0, dtype=torch.bfloat16, device=DEV)
    y = fos.wlinear_fwd(x, w, out=out[1:m + 1])
    assert y.data_ptr() == out[1].data_ptr()
    check_linear(y, x, data, scales, t)
    assert (out[0] == 7).all() and (out[m + 1] == 7).all()


def test_wlinear_empty_batch(fos):
    _, _, _, w = nv_weight(fos, 32, 64, 1)
    y = fos.wlinear_fwd(torch.empty(0, 64, dtype=torch.bfloat16, device=DEV), w)
    assert y.shape == (0, 32)


@pytest.mark.parametrize("m", [1, 6, 32])
@pytest.mark.parametrize("block", ["1d", "2d"])
def test_wlinear_wide_values(fos, m, block):
    """Activations from 2^-100 to 2^100 side by side, a weight that uses the whole range
    of block scales, and a 2D record."""
    n, k = 48, 1024
    data, scales, t, w = nv_weight(fos, n, k, 9, N.Config(block=block), scale=1.0)
    g = np.random.RandomState(m)
    x = np.ldexp(g.randn(m, k), g.randint(-100, 100, (m, k)))
    x = to_gpu_bf16(F.f32_to_bf16_bits(x.astype(np.float32)))
    check_linear(fos.wlinear_fwd(x, w, out_dtype=torch.float32), x, data, scales, t)


@pytest.mark.parametrize("m", [1, 2, 9, 33])
def test_mx_wlinear_scale_range(fos, m):
    """Every block scale from 2^-120 to 2^100 (E8M0 codes 7 to 227)."""
    n, k = 64, 640
    g = np.random.RandomState(m)
    data = g.randint(0, 256, (n, k // 2)).astype(np.uint8)
    for lo, hi, e in ((7, 120, 60), (100, 150, 0), (130, 228, -60)):
        scales = g.randint(lo, hi, (n, k // 32)).astype(np.uint8)
        x = to_gpu_bf16(F.f32_to_bf16_bits(np.ldexp(g.randn(m, k), e).astype(np.float32)))
        y = fos.mx_wlinear_fwd(x, fos.MXFP4Tensor(dev(data), dev(scales)), out_dtype=torch.float32)
        check_linear(y, x, data, scales, None)


def test_wlinear_on_another_stream(fos):
    data, scales, t, w = nv_weight(fos, 512, 512, 21)
    x = W.random_bf16(4, 512, 22, "normal").to(DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y = fos.wlinear_fwd(x, w)
    side.synchronize()
    check_linear(y, x, data, scales, t)


@pytest.mark.parametrize("m", [1, 3, 16])
def test_wlinear_weight_past_32_bits(fos, m):
    """A weight of more than 4 GiB of nibbles: rows on either side of 2^31 and 2^32."""
    n, k = 140000, 65536
    g = torch.Generator(device=DEV).manual_seed(m)
    data = torch.randint(0, 256, (n, k // 2), dtype=torch.uint8, device=DEV, generator=g)
    scales = torch.randint(40, 72, (n, k // 16), dtype=torch.uint8, device=DEV, generator=g)
    t = torch.full((1,), 0.01, device=DEV)
    x = W.random_bf16(m, k, 2, "normal").to(DEV)
    y = fos.wlinear_fwd(x, fos.NVFP4Tensor(data, scales, t), out_dtype=torch.float32)
    rows = [0, 65535, 65536, 131071, 131072, n - 17, n - 1]
    ref, mag = S.wlinear_ref64(f64(x), data[rows].cpu().numpy(), scales[rows].cpu().numpy(),
                               np.float32(0.01))
    within(f64(y[:, rows]), ref, U * np.abs(ref) + (k + 8) * U * mag, "y")


# ------------------------------------------------------------------ cache

KT, VT = np.float32(12.0625 / 2688), np.float32(6.59375 / 2688)


def new_cache(fos, fmt, pages, page, heads, dim):
    ts = [torch.tensor([t], dtype=torch.float32, device=DEV) for t in (KT, VT)]
    return fos.kv_cache(pages, page, heads, dim, fmt, *(ts if fmt == "nvfp4" else ()), device=DEV)


def fill_garbage(cache):
    """NaN everywhere: bf16 NaNs, or E4M3 NaN block scales over random nibbles."""
    if cache.format == "bf16":
        cache.k.fill_(float("nan")), cache.v.fill_(float("nan"))
    else:
        for d, s in ((cache.k, cache.k_scales), (cache.v, cache.v_scales)):
            d.random_(0, 256), s.fill_(0x7F)


def expected_record(x, t, rule):
    """(nibbles, scales) of bf16 rows [n, heads, dim] under the tensor scale t."""
    n, h, d = x.shape
    o = N.quantize(bits_of(x.cpu()).reshape(n * h, d), N.Config(rule=rule), t=t)
    return o["row_data"].reshape(n, h, d // 2), o["row_scales"].reshape(n, h, d // 16)


@pytest.mark.parametrize("rule", ["4/6", "6"])
@pytest.mark.parametrize("tokens,heads,dim,page", [(1, 1, 32, 16), (3, 8, 128, 16), (50, 2, 96, 48),
                                                   (257, 5, 64, 256), (33, 3, 256, 4096),
                                                   (130, 1, 224, 32)])
def test_append_nvfp4_matches_the_quantizer(fos, tokens, heads, dim, page, rule):
    g = np.random.RandomState(tokens)
    pages = max(2, 2 * -(-tokens // page))
    cache = new_cache(fos, "nvfp4", pages, page, heads, dim)
    before = [x.random_(0, 127).clone() for x in (cache.k, cache.v, cache.k_scales, cache.v_scales)]
    # columns of a wider row, as a fused projection gives them; some blocks saturate
    wide = W.random_bf16(tokens, 2 * heads * dim + 16, tokens + dim, "student_t", scale=2.0,
                         outlier_every=101).to(DEV)
    wide[0, 8:40] = 0.0
    k = wide[:, 8:8 + heads * dim].unflatten(1, (heads, dim))
    v = wide[:, 8 + heads * dim:8 + 2 * heads * dim].unflatten(1, (heads, dim))
    slots = g.choice(pages * page, tokens, replace=False)
    skip = g.rand(tokens) < 0.2
    given = np.where(skip, g.choice([-1, -7, pages * page, 2 ** 40, -2 ** 62], tokens), slots)
    fos.kv_append(cache, k, v, dev(given), rule=rule)
    want = [b.cpu().numpy().copy() for b in before]
    for x, t, i in ((k, KT, 0), (v, VT, 1)):
        data, scales = expected_record(x, t, rule)
        for j in np.flatnonzero(~skip):
            want[i][slots[j] // page, :, slots[j] % page] = data[j]
            want[2 + i][slots[j] // page, :, slots[j] % page] = scales[j]
    for got, w, name in zip((cache.k, cache.v, cache.k_scales, cache.v_scales), want,
                            ("k", "v", "k_scales", "v_scales")):
        assert_same_bytes(got.cpu().numpy(), w, name)


@pytest.mark.parametrize("tokens,heads,dim,page", [(1, 1, 32, 16), (5, 8, 128, 64), (70, 3, 96, 48)])
def test_append_and_gather_bf16(fos, tokens, heads, dim, page):
    cache = new_cache(fos, "bf16", 5, page, heads, dim)
    fill_garbage(cache)
    k = W.random_bf16(tokens, heads * dim, 1, "normal").to(DEV).view(tokens, heads, dim)
    v = W.random_bf16(tokens, heads * dim, 2, "normal").to(DEV).view(tokens, heads, dim)
    slots = np.random.RandomState(0).choice(5 * page, tokens, replace=False)
    fos.kv_append(cache, k, v, dev(slots))
    for j in range(tokens):
        assert torch.equal(cache.k[slots[j] // page, :, slots[j] % page], k[j])
        assert torch.equal(cache.v[slots[j] // page, :, slots[j] % page], v[j])
    assert torch.isnan(cache.k.float()).sum() == (5 * page - tokens) * heads * dim
    ask = np.concatenate([slots, [-1, 5 * page, slots[0]]])
    gk, gv = fos.kv_gather(cache, dev(ask))
    z = torch.zeros(2, heads, dim, dtype=torch.bfloat16, device=DEV)
    assert torch.equal(gk, torch.cat([k, z, k[:1]])) and torch.equal(gv, torch.cat([v, z, v[:1]]))


def test_gather_nvfp4_matches_the_dequantizer(fos):
    pages, page, heads, dim = 3, 48, 2, 160
    cache = new_cache(fos, "nvfp4", pages, page, heads, dim)
    cache.k.random_(0, 256), cache.v.random_(0, 256)
    cache.k_scales.random_(0, 127), cache.v_scales.random_(0, 127)
    ask = np.random.RandomState(3).randint(-20, pages * page + 20, 300)
    got = fos.kv_gather(cache, dev(ask))
    ok = (ask >= 0) & (ask < pages * page)
    at = np.where(ok, ask, 0)
    for g, d, s, t in ((got[0], cache.k, cache.k_scales, KT), (got[1], cache.v, cache.v_scales, VT)):
        d, s = d.cpu().numpy()[at // page, :, at % page], s.cpu().numpy()[at // page, :, at % page]
        x = N.dequantize(d.reshape(-1, dim // 2), s.reshape(-1, dim // 16), t)
        want = F.f32_to_bf16_bits(x).reshape(-1, heads, dim) * ok[:, None, None].astype(np.uint16)
        assert_same_bytes(bits_of(g.cpu()), want, "gather")


def test_append_nothing(fos):
    cache = new_cache(fos, "nvfp4", 1, 16, 2, 64)
    none = torch.empty(0, 2, 64, dtype=torch.bfloat16, device=DEV)
    slots = torch.empty(0, dtype=torch.int64, device=DEV)
    fos.kv_append(cache, none, none, slots)
    k, v = fos.kv_gather(cache, slots)
    assert k.shape == (0, 2, 64) and not cache.k.any()


def test_cache_past_32_bits(fos):
    """A bf16 cache of more than 4 GiB: slots and pages on either side of 2^31 and 2^32
    bytes, appended, gathered and attended to."""
    page, heads, dim = 64, 8, 128                        # 128 KiB a page
    pages = 33000
    cache = fos.kv_cache(pages, page, heads, dim, "bf16", device=DEV)
    ids = np.array([1, 16383, 16384, 32767, 32768, pages - 1])
    T = len(ids) * page
    k = W.random_bf16(T, heads * dim, 5, "normal").to(DEV).view(T, heads, dim)
    v = W.random_bf16(T, heads * dim, 6, "normal").to(DEV).view(T, heads, dim)
    slots = (ids[:, None] * page + np.arange(page)).reshape(-1)
    fos.kv_append(cache, k, v, dev(slots))
    gk, gv = fos.kv_gather(cache, dev(slots))
    assert torch.equal(gk, k) and torch.equal(gv, v)
    q = W.random_bf16(16, dim, 7, "normal").to(DEV).view(1, 16, dim)
    out, lse = fos.paged_decode(q, cache, dev(ids.astype(np.int32)[None]),
                                torch.tensor([T - 3], dtype=torch.int32, device=DEV), return_lse=True)
    check_attention(out[0], lse[0], f64(q[0]), f64(k[:T - 3]), f64(v[:T - 3]), dim ** -0.5)


# ------------------------------------------------------------------ attention

def check_attention(out, lse, q, k, v, scale, what=""):
    ref, rl, A, V, E = S.attend_ref64(q, k, v, scale)
    n, D = len(k), q.shape[1]
    if n == 0:
        assert not f64(out).any() and (lse is None or (f64(lse) == -np.inf).all()), what
        return
    dS = (D + 8) * U * A
    adds = (n / 4 + 64) * U
    rel = 2 * dS + 2.0 ** -20 + adds + 2.0 ** -11
    top = np.abs(v).max(axis=0).repeat(q.shape[0] // v.shape[1], axis=0)
    low = n * 2.0 ** -25 * top / E[:, None]
    within(f64(out), ref, 2.0 ** -8 * np.abs(ref) + (rel[:, None] * V + low) * (1 + 2.0 ** -8)
           + 2.0 ** -133, what + " out")
    if lse is not None:
        within(f64(lse), rl, dS + 2.0 ** -20 + adds + 4 * U * np.abs(rl), what + " lse")


def run_decode(fos, fmt, B, Hq, Hkv, D, page, lens, window=0, holes=False, scale=None, seed=0,
               slack=0, qscale=1.5, garbage=True):
    """A cache whose pages hold the sequences' tokens at random page ids, NaN everywhere
    else, read back against the reference."""
    g = np.random.RandomState(seed)
    lens = np.asarray(lens)
    held = [-(-max(0, int(n)) // page) for n in lens]
    width = max(1, max(held) + slack)
    pages = sum(held) + 2
    cache = new_cache(fos, fmt, pages, page, Hkv, D)
    if garbage:
        fill_garbage(cache)
    order = g.permutation(pages - 1)                    # the last page belongs to nobody
    table = g.choice([-1, pages - 1, pages, 2 ** 31 - 1, -2 ** 31], (B, width))
    at, slots = 0, []
    for b in range(B):
        table[b, :held[b]] = order[at:at + held[b]]
        at += held[b]
        j = np.arange(max(0, int(lens[b])))
        slots.append(table[b][j // page] * page + j % page)
    if holes:
        gone = g.rand(B, width) < 0.3
        gone[0] = True                                  # one sequence has no page left
        lost = g.choice([-1, pages, pages + 5], (B, width))
        shown = np.where(gone, lost, table)
    else:
        shown = table
    slots = np.concatenate(slots).astype(np.int64)
    T = len(slots)
    if T:
        k = W.random_bf16(T, Hkv * D, seed + 1, "normal", outlier_every=61, outlier_mult=3.0)
        v = W.random_bf16(T, Hkv * D, seed + 2, "normal")
        fos.kv_append(cache, k.to(DEV).view(T, Hkv, D), v.to(DEV).view(T, Hkv, D), dev(slots))
    wide = W.random_bf16(B, Hq * D + 24, seed + 3, "normal", scale=qscale).to(DEV)
    q = wide[:, 8:8 + Hq * D].unflatten(1, (Hq, D))
    tab = torch.full((B, width + 3), -5, dtype=torch.int32, device=DEV)
    tab[:, :width] = dev(shown.astype(np.int64)).int()
    out, lse = fos.paged_decode(q, cache, tab[:, :width], dev(lens.astype(np.int32)), scale=scale,
                                window=window, return_lse=True)
    again = fos.paged_decode(q, cache, tab[:, :width], dev(lens.astype(np.int32)), scale=scale,
                             window=window)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))
    ks, vs = ((x.float().cpu().numpy() if fmt == "bf16" else x.cpu().numpy()) for x in (cache.k, cache.v))
    sc = [None, None] if fmt == "bf16" else [cache.k_scales.cpu().numpy(), cache.v_scales.cpu().numpy()]
    for b in range(B):
        ids, off = S.visible(lens[b], shown[b], page, pages, window)
        kk, vv = (S.cache_rows_f64(x[ids, :, off], None if s is None else s[ids, :, off], t)
                  for x, s, t in ((ks, sc[0], KT), (vs, sc[1], VT)))
        check_attention(out[b], lse[b], f64(q[b]), kk, vv, D ** -0.5 if scale is None else scale,
                        f"sequence {b} of {len(ids)} tokens")


FMTS = pytest.mark.parametrize("fmt", ["bf16", "nvfp4"])


@FMTS
@pytest.mark.parametrize("D", [32, 64, 96, 128, 160, 192, 224, 256])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (8, 2), (7, 1)])
def test_decode_head_layouts(fos, fmt, D, Hq, Hkv):
    run_decode(fos, fmt, 3, Hq, Hkv, D, 16, [1, 77, 300], seed=D + Hq)


@FMTS
@pytest.mark.parametrize("Hq,Hkv", [(4, 4), (16, 1), (17, 1), (48, 1), (32, 2), (30, 3), (64, 8)])
def test_decode_shared_heads(fos, fmt, Hq, Hkv):
    run_decode(fos, fmt, 2, Hq, Hkv, 64, 32, [129, 500], seed=Hq)


@FMTS
@pytest.mark.parametrize("page", [16, 32, 48, 80, 256, 4096])
def test_decode_lengths_around_pages_and_tiles(fos, fmt, page):
    lens = [0, 1, 2, 7, 8, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 511, 513]
    run_decode(fos, fmt, len(lens), 4, 2, 64, page, lens, slack=2, seed=page)


@FMTS
def test_decode_every_short_length(fos, fmt):
    run_decode(fos, fmt, 70, 2, 1, 128, 16, list(range(70)), seed=5)


@FMTS
def test_decode_nothing_to_see(fos, fmt):
    run_decode(fos, fmt, 5, 4, 2, 96, 16, [0, -3, 0, -2 ** 31, 0], seed=6)


@FMTS
@pytest.mark.parametrize("window", [1, 5, 31, 32, 33, 100, 1000, 2 ** 40])
def test_decode_window(fos, fmt, window):
    run_decode(fos, fmt, 6, 4, 2, 64, 48, [0, 1, 33, 99, 400, 1500], window=window, seed=window % 97)


@FMTS
@pytest.mark.parametrize("window", [0, 60])
def test_decode_pages_given_up(fos, fmt, window):
    run_decode(fos, fmt, 7, 6, 3, 64, 16, [90, 16, 1, 333, 700, 64, 65], window=window, holes=True, seed=8)


@FMTS
def test_decode_length_past_the_table(fos, fmt):
    """A length beyond the table's pages sees what the table names; a window counts from
    the length."""
    for window in (0, 40):
        cache = new_cache(fos, fmt, 2, 32, 2, 64)
        T = 64
        k = W.random_bf16(T, 128, 1, "normal").to(DEV).view(T, 2, 64)
        v = W.random_bf16(T, 128, 2, "normal").to(DEV).view(T, 2, 64)
        fos.kv_append(cache, k, v, torch.arange(T, device=DEV))
        gk, gv = fos.kv_gather(cache, torch.arange(T, device=DEV))
        q = W.random_bf16(3, 256, 3, "normal").to(DEV).view(3, 4, 64)
        table = torch.tensor([[0, 1]] * 3, dtype=torch.int32, device=DEV)
        lens = torch.tensor([70, 2 ** 31 - 1, 64], dtype=torch.int32, device=DEV)
        out, lse = fos.paged_decode(q, cache, table, lens, window=window, return_lse=True)
        kv = (N_rows(cache, "k"), N_rows(cache, "v"))
        for b in range(3):
            first = max(0, int(lens[b]) - window) if window else 0
            check_attention(out[b], lse[b], f64(q[b]), kv[0][first:T], kv[1][first:T], 0.125, f"{b}")


def N_rows(cache, name):
    """Every row of a cache of one run of pages as fp64 [tokens, heads, dim]."""
    x, s = getattr(cache, name), getattr(cache, name + "_scales")
    rows = S.cache_rows_f64(x.float().cpu().numpy() if s is None else x.cpu().numpy(),
                            None if s is None else s.cpu().numpy(), KT if name == "k" else VT)
    return rows.transpose(0, 2, 1, 3).reshape(-1, rows.shape[1], rows.shape[3])


@FMTS
@pytest.mark.parametrize("scale", [None, 0.0, -0.3, 1.7])
def test_decode_scale(fos, fmt, scale):
    run_decode(fos, fmt, 2, 8, 4, 128, 64, [200, 1000], scale=scale, qscale=0.7, seed=11)


@FMTS
def test_decode_peaked_and_far_scores(fos, fmt):
    """Scores in the hundreds: one token takes all the weight, the maximum moves late."""
    run_decode(fos, fmt, 2, 8, 2, 128, 64, [3000, 129], qscale=40.0, seed=12)


@FMTS
@pytest.mark.parametrize("exponent", [-110, -20, 20, 60])
def test_decode_query_range(fos, fmt, exponent):
    """Queries far from 1, with the scale that brings the scores back."""
    run_decode(fos, fmt, 1, 4, 2, 64, 16, [100], qscale=2.0 ** exponent, scale=2.0 ** (-exponent - 3),
               seed=13)


@FMTS
@pytest.mark.parametrize("B,Hq,Hkv,D,L", [(1, 8, 1, 128, 70001), (2, 4, 2, 64, 40000), (1, 2, 2, 256, 20011)])
def test_decode_long(fos, fmt, B, Hq, Hkv, D, L):
    run_decode(fos, fmt, B, Hq, Hkv, D, 128, [L - 31 * b for b in range(B)], seed=L, garbage=False)


@FMTS
def test_decode_many_sequences(fos, fmt):
    lens = np.random.RandomState(4).randint(0, 120, 700)
    lens[13] = 5000
    run_decode(fos, fmt, 700, 4, 2, 32, 16, lens, seed=14)


@FMTS
def test_decode_values_that_are_infinite_where_masked(fos, fmt):
    """NaN and infinities past the length, before the window and in foreign pages leave
    no trace, at every offset of the length inside a tile."""
    run_decode(fos, fmt, 40, 2, 2, 64, 16, list(range(90, 130)), window=45, seed=15)


@FMTS
def test_decode_on_another_stream(fos, fmt):
    cache = new_cache(fos, fmt, 40, 16, 2, 64)
    T = 640
    k = W.random_bf16(T, 128, 1, "normal").to(DEV).view(T, 2, 64)
    v = W.random_bf16(T, 128, 2, "normal").to(DEV).view(T, 2, 64)
    slots = torch.arange(T, device=DEV)
    q = W.random_bf16(1, 256, 3, "normal").to(DEV).view(1, 4, 64)
    table = torch.arange(40, dtype=torch.int32, device=DEV)[None]
    lens = torch.tensor([T], dtype=torch.int32, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fos.kv_append(cache, k, v, slots)
        out, lse = fos.paged_decode(q, cache, table, lens, return_lse=True)
    side.synchronize()
    check_attention(out[0], lse[0], f64(q[0]), N_rows(cache, "k"), N_rows(cache, "v"), 0.125)


def test_decode_empty_batch_and_empty_cache(fos):
    cache = new_cache(fos, "nvfp4", 4, 16, 2, 64)
    q = torch.empty(0, 4, 64, dtype=torch.bfloat16, device=DEV)
    out = fos.paged_decode(q, cache, torch.empty(0, 3, dtype=torch.int32, device=DEV),
                           torch.empty(0, dtype=torch.int32, device=DEV))
    assert out.shape == (0, 4, 64)
    q = torch.ones(2, 4, 64, dtype=torch.bfloat16, device=DEV)
    lens = torch.tensor([5, 9], dtype=torch.int32, device=DEV)
    # no page in the table, and no page in the cache
    for c, width in ((cache, 0), (new_cache(fos, "bf16", 0, 16, 2, 64), 2)):
        out, lse = fos.paged_decode(q, c, torch.zeros(2, width, dtype=torch.int32, device=DEV), lens,
                                    return_lse=True)
        assert not out.any() and (lse == -float("inf")).all()


@FMTS
def test_decode_replayed_from_a_graph(fos, fmt):
    """A captured step (append, attention) replayed with other tokens and lengths gives
    the eager results."""
    page, Hkv, D, B = 16, 2, 64, 3
    cache, eager = (new_cache(fos, fmt, 60, page, Hkv, D) for _ in range(2))
    table = torch.arange(60, dtype=torch.int32, device=DEV).view(B, 20)
    q = torch.zeros(B, 4, D, dtype=torch.bfloat16, device=DEV)
    k, v = (torch.zeros(B, Hkv, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    slots = torch.zeros(B, dtype=torch.int64, device=DEV)
    lens = torch.zeros(B, dtype=torch.int32, device=DEV)
    out = torch.zeros_like(q)

    def step():
        fos.kv_append(cache, k, v, slots)
        fos.paged_decode(q, cache, table, lens, out=out)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()                                          # the workspace exists before the capture
    torch.cuda.current_stream().wait_stream(side)
    cache.k.zero_(), cache.v.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for i in range(6):
        n = 1 + 50 * i
        j = torch.tensor([n - 1, n + 2, n + 7], device=DEV)
        slots.copy_(table[torch.arange(B, device=DEV), j // page].long() * page + j % page)
        lens.copy_(j + 1)
        for x, seed in ((q, 1), (k, 2), (v, 3)):
            x.copy_(W.random_bf16(B, x.shape[1] * D, 10 * i + seed, "normal").view(x.shape))
        graph.replay()
        fos.kv_append(eager, k, v, slots)
        want = fos.paged_decode(q, eager, table, lens)
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), want.view(torch.int16)), i


@FMTS
@pytest.mark.parametrize("L", [5, 300, 5000])
def test_decode_keeps_a_nan(fos, fmt, L):
    """A NaN query gives NaN in its head's output and lse, one sequence, few tokens or
    many workgroups alike, and touches no other head."""
    cache = new_cache(fos, fmt, 320, 16, 2, 64)
    k, v = (W.random_bf16(L, 128, s, "normal").to(DEV).view(L, 2, 64) for s in (1, 2))
    fos.kv_append(cache, k, v, torch.arange(L, device=DEV))
    q = W.random_bf16(1, 256, 3, "normal").to(DEV).view(1, 4, 64)
    args = (torch.arange(320, dtype=torch.int32, device=DEV)[None],
            torch.tensor([L], dtype=torch.int32, device=DEV))
    out, lse = fos.paged_decode(q, cache, *args, return_lse=True)
    q[0, 1, 17] = float("nan")
    got, got_lse = fos.paged_decode(q, cache, *args, return_lse=True)
    assert got[0, 1].isnan().all() and got_lse[0, 1].isnan()
    rest = [0, 2, 3]
    assert torch.equal(got[0, rest], out[0, rest]) and torch.equal(got_lse[0, rest], lse[0, rest])


def test_decode_captured_before_any_call(fos):
    """A capture that is the first call of its stream, and whose graph is replayed only
    after an eager call there, changes neither; a workspace of the caller's serves both."""
    cache = new_cache(fos, "nvfp4", 320, 16, 2, 64)
    L = 5000
    k, v = (W.random_bf16(L, 128, s, "normal").to(DEV).view(L, 2, 64) for s in (1, 2))
    fos.kv_append(cache, k, v, torch.arange(L, device=DEV))
    q = W.random_bf16(1, 256, 3, "normal").to(DEV).view(1, 4, 64)
    args = (torch.arange(320, dtype=torch.int32, device=DEV)[None],
            torch.tensor([L], dtype=torch.int32, device=DEV))
    want = fos.paged_decode(q, cache, *args)
    own = fos.paged_decode_workspace(1, 4, 2, 64, DEV)
    outs = [torch.zeros_like(want) for _ in range(3)]
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        fos.paged_decode(q, cache, *args, out=outs[0])
        fos.paged_decode(q, cache, *args, out=outs[1], ws=own)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fos.paged_decode(q, cache, *args, out=outs[2])
    torch.cuda.current_stream().wait_stream(side)
    for _ in range(3):
        outs[0].zero_(), outs[1].zero_()
        graph.replay()
        eager = fos.paged_decode(q, cache, *args, ws=own)
        torch.cuda.synchronize()
        for o in (outs[0], outs[1], outs[2], eager):
            assert torch.equal(o, want)


def test_decode_refuses_a_workspace_that_is_too_small(fos):
    cache = new_cache(fos, "bf16", 4, 16, 2, 64)
    q = torch.ones(1, 4, 64, dtype=torch.bfloat16, device=DEV)
    args = (torch.zeros(1, 4, dtype=torch.int32, device=DEV),
            torch.ones(1, dtype=torch.int32, device=DEV))
    with pytest.raises(fos.FosError):
        fos.paged_decode(q, cache, *args, ws=torch.zeros(4096, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError):
        fos.paged_decode(q, cache, *args, ws=torch.zeros(4096, device=DEV))
    with pytest.raises(ValueError):
        fos.paged_decode_workspace(1, 3, 2, 64, DEV)


@pytest.mark.parametrize("m", [1, 3, 9, 33])
def test_mx_wlinear_scale_ends(fos, m):
    """The ends of E8M0's range: codes 0 (2^-127, below fp32's normal range) to 6, and
    228 up to the largest whose products with E2M1 are finite."""
    n, k = 64, 640
    g = np.random.RandomState(m)
    data = g.randint(0, 256, (n, k // 2)).astype(np.uint8)
    for lo, hi, e in ((0, 7, 100), (228, 253, -100)):
        scales = g.randint(lo, hi, (n, k // 32)).astype(np.uint8)
        x = to_gpu_bf16(F.f32_to_bf16_bits(np.ldexp(g.randn(m, k), e).astype(np.float32)))
        y = fos.mx_wlinear_fwd(x, fos.MXFP4Tensor(dev(data), dev(scales)), out_dtype=torch.float32)
        check_linear(y, x, data, scales, None)


@FMTS
@pytest.mark.parametrize("short", [False, True])
def test_decode_several_parts_per_sequence(fos, fmt, short):
    """Batches whose sequences fall to a few workgroups each, of one length in steps or
    with much shorter and empty ones between."""
    g = np.random.RandomState(31)
    lens = g.randint(1025, 1281, 20)
    if short:
        lens[[3, 7, 8, 19]] = 0, 1, 257, 40
    run_decode(fos, fmt, 20, 8, 8, 128, 32, list(lens), seed=32)


@pytest.mark.parametrize("m,n", [(2, 8200), (4, 300), (16, 2050), (9, 6000), (16, 8200), (250, 1000),
                                 (17, 12300), (61, 4099), (33, 16400), (100, 6000)])
@pytest.mark.parametrize("fmt,k", [("nvfp4", 1040), ("nvfp4", 2208), ("mxfp4", 2208)])
def test_wlinear_many_weight_rows(fos, m, n, fmt, k):
    """Sizes for which the GPU is filled with each of the tiles."""
    data, scales, t, w = (nv_weight if fmt == "nvfp4" else mx_weight)(fos, n, k, m + n)
    x = W.random_bf16(m, k, n, "normal").to(DEV)
    run = fos.wlinear_fwd if fmt == "nvfp4" else fos.mx_wlinear_fwd
    y = torch.full((m, n), float("nan"), dtype=torch.float32, device=DEV)
    run(x, w, out_dtype=torch.float32, out=y)
    rows = np.unique(np.concatenate([np.arange(0, n, 7), np.arange(max(0, n - 80), n)]))
    check_linear(y, x, data, scales, t, rows=rows)
    assert not y.isnan().any()


@FMTS
@pytest.mark.parametrize("Hq,Hkv,D,lens", [
    (2, 1, 256, [27000]), (16, 1, 192, [9000]), (16, 2, 96, [300, 11000, 2]), (1, 1, 32, [40000, 0, 39000]),
    (4, 1, 64, [5000, 5000, 9, 12345]), (35, 5, 128, [14000, 1000])])
def test_decode_many_partial_results(fos, fmt, Hq, Hkv, D, lens):
    """Few heads and long sequences: a hundred workgroups and more leave parts of one
    output, next to sequences that fall to one."""
    run_decode(fos, fmt, len(lens), Hq, Hkv, D, 64, lens, seed=41, garbage=False)


@pytest.mark.parametrize("m,n", [(1, 1), (3, 1023), (4, 1025), (1, 2051), (3, 4099), (5, 7), (6, 510),
                                 (7, 1000), (13, 255), (16, 256), (33, 111), (64, 61), (90, 40)])
@pytest.mark.parametrize("fmt,k", [("nvfp4", 16), ("nvfp4", 528), ("nvfp4", 4640), ("mxfp4", 96), ("mxfp4", 2592)])
def test_wlinear_few_weight_rows(fos, m, n, fmt, k):
    """Few weight rows, where each workgroup takes few of them and groups of activation
    rows share them."""
    data, scales, t, w = (nv_weight if fmt == "nvfp4" else mx_weight)(fos, n, k, m + n)
    wide = W.random_bf16(m, k + 24, n, "normal").to(DEV)
    x = wide[:, 8:8 + k]
    bias = W.random_bf16(1, n, 3, "normal")[0].to(DEV) if n % 2 else None
    run = fos.wlinear_fwd if fmt == "nvfp4" else fos.mx_wlinear_fwd
    check_linear(run(x, w, bias=bias, out_dtype=torch.float32), x, data, scales, t, bias)
