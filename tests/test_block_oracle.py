"""Pins of ``oracle.block`` (CPU): formats against their tables and torch's casts, gradients against
central differences, the generator against its authors' known answers."""
import os
import sys

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from oracle import block as K  # noqa: E402

torch = pytest.importorskip("torch")


def test_e4m3_table():
    codes = torch.arange(256, dtype=torch.uint8)
    ref = codes.view(torch.float8_e4m3fn).float().numpy().astype(np.float64)
    np.testing.assert_array_equal(K.e4m3_values(), ref)
    assert np.nanmax(K.e4m3_values()) == 448.0


def test_e4m3_round():
    rng = np.random.default_rng(0)
    table = K.e4m3_values()
    table = np.unique(table[np.isfinite(table)])
    v = np.concatenate([rng.uniform(-448, 448, 20000), rng.standard_normal(20000) * 0.02, table,
                        (table[1:] + table[:-1]) / 2, [0.0, 2.0 ** -10, 3 * 2.0 ** -10, -2.0 ** -10]])
    v = v.astype(np.float32).astype(np.float64)
    ref = torch.from_numpy(v).float().to(torch.float8_e4m3fn).float().numpy()
    np.testing.assert_array_equal(K.e4m3_round(v), ref)
    assert np.isin(K.e4m3_round(v), table).all()


def test_scales_are_the_smallest_that_do_not_saturate():
    rng = np.random.default_rng(1)
    v = rng.standard_normal((200, 96)) * 2.0 ** rng.integers(-40, 40, (200, 1))
    for edge in (448.0, 447.999, 448.001, 1.75, 1.7500001, 1.0, 2.0 ** -126, 2.0 ** -149):
        row = np.zeros((1, 96))
        row[0, 5], row[0, 40], row[0, 95] = edge, -edge, edge / 2
        v = np.concatenate([v, row])
    s = K.scale_exponents(v)
    top = np.abs(v).reshape(*s.shape, 32).max(-1)
    assert (top <= 448 * 2.0 ** s).all()
    tight = (top > 448 * 2.0 ** (s - 1)) | (s == -127)
    assert tight.all()
    q, b = K.quantize(v)
    assert np.abs(q).max() <= 448 and b.shape == (v.shape[0], 16) and not b[:, 3:].any()


def test_quantize_of_what_is_not_finite():
    v = np.zeros((1, 64))
    v[0, 3], v[0, 4], v[0, 5] = np.inf, 3.0, np.nan
    q, b = K.quantize(v)
    assert np.isnan(q[0, [3, 5]]).all() and q[0, 4] == 3.0 * 2.0 ** (127 - int(b[0, 0]))
    assert b[0, 1] == 0 and not q[0, 32:].any()


def test_decode_undoes_quantize():
    rng = np.random.default_rng(2)
    v = rng.standard_normal((7, 160))
    q, b = K.quantize(v)
    codes = torch.from_numpy(q).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    back = K.decode(codes, b)
    # half a step of e4m3, 2^-4 of the value, or of the smallest ones, 2^-10 of the scale
    s = np.repeat(2.0 ** (b[:, :5].astype(np.float64) - 127), 32, axis=1)
    assert (np.abs(back - v) <= np.maximum(2.0 ** -4 * np.abs(v), 2.0 ** -10 * s)).all()


def differences(f, x, d, h=1e-5):
    """The derivative of f along d at x, centrally."""
    return (f(x + h * d) - f(x - h * d)) / (2 * h)


def test_rms_norm_backward():
    rng = np.random.default_rng(3)
    s, dy, dsum = (rng.standard_normal((5, 24)) for _ in range(3))
    gamma = 1 + 0.3 * rng.standard_normal(24)
    _, r = K.rms_norm(s, gamma, 1e-3)
    ds, dg = K.rms_norm_backward(dy, dsum, s, gamma, r)
    for _ in range(4):
        d, dgam = rng.standard_normal(s.shape), rng.standard_normal(24)
        along = differences(lambda v: (dy * K.rms_norm(v, gamma, 1e-3)[0]).sum() + (dsum * v).sum(), s, d)
        assert abs(along - (ds * d).sum()) < 1e-7
        along = differences(lambda g: (dy * K.rms_norm(s, g, 1e-3)[0]).sum(), gamma, dgam)
        assert abs(along - (dg * dgam).sum()) < 1e-7


def test_grouped_gemm_backward():
    rng = np.random.default_rng(4)
    off = [0, 3, 3, 8]
    x, w, dy = rng.standard_normal((8, 6)), rng.standard_normal((3, 5, 6)), rng.standard_normal((8, 5))
    dx, dw = K.grouped_gemm_backward(x, dy, off, w)
    assert not dw[1].any()
    d, e = rng.standard_normal(x.shape), rng.standard_normal(w.shape)
    along = differences(lambda v: (dy * K.grouped_gemm(v, off, w)).sum(), x, d)
    assert abs(along - (dx * d).sum()) < 1e-7
    along = differences(lambda v: (dy * K.grouped_gemm(x, off, v)).sum(), w, e)
    assert abs(along - (dw * e).sum()) < 1e-7


@pytest.mark.parametrize("counter,key,words", [
    ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
     (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1))])
def test_philox_known_answers(counter, key, words):
    got = K.philox([np.array([c]) for c in counter], key)
    assert tuple(int(w[0]) for w in got) == words


def test_keep():
    n = 200000
    m = K.keep(n, 0.3, 12345678901, 7)
    # a share of n independent draws: five standard deviations
    assert abs(m.mean() - 0.7) < 5 * (0.3 * 0.7 / n) ** 0.5
    np.testing.assert_array_equal(m[1001:5000], K.keep(3999, 0.3, 12345678901, 7, first=1001))
    assert K.keep(1000, 0.0, 1, 1).all()
    for other in (K.keep(n, 0.3, 12345678902, 7), K.keep(n, 0.3, 12345678901, 8)):
        assert abs((m == other).mean() - (0.49 + 0.09)) < 0.01
