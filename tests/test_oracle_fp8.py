"""Pins of the 8-bit operators' oracle: the e4m3 table and rounding against
torch's float8_e4m3fn conversion and hand-derived values, the operators
against loops."""
import numpy as np
import torch

from oracle import fp8_oracle as F


def test_table_matches_torch():
    codes = np.arange(256, dtype=np.uint8)
    ref = torch.from_numpy(codes).view(torch.float8_e4m3fn).float().numpy()
    got = F.decode(codes)
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    assert np.array_equal(got[~np.isnan(got)], ref[~np.isnan(ref)])
    assert F.VALUES[126] == 448.0 and F.VALUES[1] == 2.0 ** -9 and F.VALUES[8] == 2.0 ** -6


def test_encode_rounds_to_nearest_even():
    # every value, every midpoint (ties go to the even code) and its neighbours
    pos = F.VALUES[:127]
    assert np.array_equal(F.encode(pos), np.arange(127))
    mid = (pos[1:] + pos[:-1]) / 2
    lo = np.arange(126)
    assert np.array_equal(F.encode(mid), np.where(lo % 2 == 0, lo, lo + 1))
    assert np.array_equal(F.encode(mid * (1 - 1e-12)), lo)
    assert np.array_equal(F.encode(mid * (1 + 1e-12)), lo + 1)
    assert np.array_equal(F.encode(-pos[1:]), np.arange(1, 127) | 128)
    v = np.random.default_rng(3).standard_normal(4096) * 30
    ref = torch.from_numpy(v.astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(F.encode(v.astype(np.float32)), ref)


def test_codes_hold_half_a_step():
    v = np.random.default_rng(4).standard_normal((5, 300))
    q, s = F.code_rows(v)
    full = F.spread(s.astype(np.float64), 300)
    assert np.all(np.abs(F.decode(q) * full - v) <= np.maximum(2.0 ** -4 * np.abs(v),
                                                              2.0 ** -10 * full) * (1 + 1e-12))
    assert F.code_rows(np.zeros((1, 16)))[1][0, 0] == np.float32(2.0 ** -126)


def test_product_and_norm_against_loops():
    rng = np.random.default_rng(5)
    a, w = rng.standard_normal((3, 144)), rng.standard_normal((130, 144))
    qa, sa = F.code_rows(a)
    qw, sw = F.code_weight(w)
    y, mag = F.product(qa, sa, qw, sw)
    for m, n in ((0, 0), (2, 127), (1, 128), (2, 129)):
        t = [float(F.VALUES[qa[m, k]]) * float(sa[m, k // 128]) * float(F.VALUES[qw[n, k]]) *
             float(sw[n // 128, k // 128]) for k in range(144)]
        assert abs(sum(t) - y[m, n]) <= 1e-12 * mag[m, n]
    h, out = F.rmsnorm(a, a[::-1], w[0], 0.5)
    row = a[1] + a[1]
    assert np.allclose(out[1], row / (np.mean(row ** 2) + 0.5) ** 0.5 * w[0], rtol=1e-13)
    v = F.silu_mul(np.array([[0.0, 1.0, 3.0, -2.0]]))
    assert v[0, 0] == 0.0 and abs(v[0, 1] + 2 / (1 + np.exp(-1))) < 1e-15
