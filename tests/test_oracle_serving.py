"""Pins of the fp64 references of the token-serving operators."""
import numpy as np
import pytest

from oracle import mxfp4 as MX
from oracle import nvfp4 as N
from oracle import serving as S


def test_visible_tokens():
    ids, off = S.visible(10, [3, 1], 8, 4)
    assert ids.tolist() == [3] * 8 + [1] * 2 and off.tolist() == list(range(8)) + [0, 1]
    ids, off = S.visible(10, [3, 1], 8, 4, window=3)
    assert ids.tolist() == [3, 1, 1] and off.tolist() == [7, 0, 1]
    ids, off = S.visible(10, [4, 1], 8, 4)                       # page 4 is not in the cache
    assert ids.tolist() == [1, 1]
    assert len(S.visible(0, [0], 8, 4)[0]) == 0 and len(S.visible(-5, [0], 8, 4)[0]) == 0
    assert len(S.visible(100, [0, 1], 8, 4)[0]) == 16            # past the table
    assert len(S.visible(100, [0, 1], 8, 4, window=90)[0]) == 6
    assert len(S.visible(100, [0, 1], 8, 4, window=10)[0]) == 0


def test_attention_against_the_definition():
    g = np.random.RandomState(0)
    q, k, v = g.randn(4, 32), g.randn(9, 2, 32), g.randn(9, 2, 32)
    out, lse, A, V, E = S.attend_ref64(q, k, v, 0.3)
    for h in range(4):
        w = np.exp(0.3 * np.array([np.dot(q[h], k[j, h // 2]) for j in range(9)]))
        assert np.isclose(lse[h], np.log(w.sum()), rtol=1e-13)
        assert np.allclose(out[h], sum(w[j] * v[j, h // 2] for j in range(9)) / w.sum(), rtol=1e-12)
        assert np.isclose(E[h] * w.max(), w.sum())
        assert (V[h] >= np.abs(out[h]) - 1e-15).all()


def test_attention_shift_and_nothing():
    """Adding one vector to every key shifts the scores and leaves the output; one token
    returns its value; none returns zeros."""
    g = np.random.RandomState(1)
    q, k, v = g.randn(2, 16), g.randn(5, 1, 16), g.randn(5, 1, 16)
    c = g.randn(16)
    a, b = S.attend_ref64(q, k, v, 1.0), S.attend_ref64(q, k + c, v, 1.0)
    assert np.allclose(a[0], b[0]) and np.allclose(b[1] - a[1], q @ c)
    one = S.attend_ref64(q, k[:1], v[:1], 1.0)
    assert np.allclose(one[0], v[0]) and np.allclose(one[1], q @ k[0, 0])
    none = S.attend_ref64(q, k[:0], v[:0], 1.0)
    assert not none[0].any() and (none[1] == -np.inf).all()


@pytest.mark.parametrize("mx", [False, True])
def test_wlinear_against_the_dequantized_product(mx):
    g = np.random.RandomState(2)
    w, x, bias = g.randn(6, 64).astype(np.float32), g.randn(3, 64), g.randn(6)
    if mx:
        o = MX.quantize(w)
        rec, deq = (o["data"], o["scales"], None), MX.dequantize(o["data"], o["scales"])
    else:
        o = N.quantize(w, N.Config())
        rec = (o["row_data"], o["row_scales"], o["t"])
        deq = N.dequantize(*rec)
    y, s = S.wlinear_ref64(x, *rec, bias)
    assert np.allclose(y, x @ deq.astype(np.float64).T + bias, rtol=1e-5, atol=1e-6)
    assert (s >= np.abs(y) - 1e-12).all()
    y2, _ = S.wlinear_ref64(x, *rec, None, [4, 1])
    assert np.allclose(y2, (y - bias)[:, [4, 1]])


def test_cache_rows_are_the_dequantized_record():
    g = np.random.RandomState(3)
    x = g.randn(2 * 3 * 4, 32).astype(np.float32)
    o = N.quantize(x, N.Config(), t=0.01)
    d, s = o["row_data"].reshape(2, 3, 4, 16), o["row_scales"].reshape(2, 3, 4, 2)
    assert np.array_equal(S.cache_rows_f64(d, s, 0.01).reshape(-1, 32),
                          N.dequantize(o["row_data"], o["row_scales"], 0.01).astype(np.float64))
    assert np.array_equal(S.cache_rows_f64(x), x.astype(np.float64))
