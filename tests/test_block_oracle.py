"""Pins of the fp64 definitions of the operators around the layer: published
test vectors, brute-force loops, central differences, and planted mistakes
that the pins must catch."""
import numpy as np
import pytest

from oracle import block_oracle as bo


@pytest.mark.parametrize("ctr, key, want", [
    # known-answer vectors of Philox4x32-10 (published with the Random123 library)
    ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
     (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1)),
])
def test_philox_known_answers(ctr, key, want):
    assert tuple(bo.philox4x32(ctr, key)) == want


def test_draws_follow_the_documented_counter():
    T, D, seed, offset, site = 5, 19, 0x0123456789ABCDEF, (1 << 64) - 2, 3
    u = bo.dropout_draws(T, D, seed, offset, site)
    G = 3
    for t, d in ((0, 0), (0, 18), (4, 7), (4, 17), (2, 9)):
        n = t * G + d // 8
        hi = (offset + site) % (1 << 64)          # wraps
        w = bo.philox4x32((n & bo.MASK32, n >> 32, hi & bo.MASK32, hi >> 32),
                          (seed & bo.MASK32, seed >> 32))
        i = d % 8
        want = w[i // 2] >> 16 if i & 1 else w[i // 2] & 0xFFFF
        assert u[t, d] == want


def test_dropout_rate_and_limits():
    f = bo.dropout_factors(400, 256, 0.25, 7, 0, 0)
    n = f.size
    # binomial: six standard deviations
    assert abs((f == 0).mean() - 0.25) < 6 * np.sqrt(0.25 * 0.75 / n)
    assert set(np.unique(f)) == {0.0, 65536.0 / 49152}
    assert (bo.dropout_factors(3, 5, 0.0, 1, 1, 1) == 1).all()
    assert (bo.dropout_factors(3, 5, 1.0, 1, 1, 1) == 0).all()


def _loss(s, w, b, dy, eps, rms):
    return (bo.norm_fwd(s, w, b, eps, rms)[0] * dy).sum()


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("weighted", [False, True])
def test_norm_gradients_against_differences(rms, weighted):
    r = np.random.default_rng(3)
    T, D, eps = 3, 7, 1e-2
    s, dy = r.normal(size=(T, D)), r.normal(size=(T, D))
    w = 1 + 0.3 * r.normal(size=D) if weighted else None
    b = r.normal(size=D) if weighted else None
    _, mean, rstd = bo.norm_fwd(s, w, b, eps, rms)
    ds, dw, db = bo.norm_bwd(dy, s, mean, rstd, w, rms)
    h = 1e-5

    def diff(a, i):
        keep = a[i]
        a[i] = keep + h
        up = _loss(s, w, b, dy, eps, rms)
        a[i] = keep - h
        dn = _loss(s, w, b, dy, eps, rms)
        a[i] = keep
        return (up - dn) / (2 * h)

    got = np.array([[diff(s, (t, d)) for d in range(D)] for t in range(T)])
    np.testing.assert_allclose(got, ds, atol=1e-8)
    if weighted:
        np.testing.assert_allclose([diff(w, d) for d in range(D)], dw, atol=1e-8)
        np.testing.assert_allclose([diff(b, d) for d in range(D)], db, atol=1e-8)
    # a dropped projection term or a missing mean would not pass
    wrong = (dy if w is None else dy * w) * rstd[:, None]
    assert np.abs(wrong - ds).max() > 1e-2


def test_norm_by_hand():
    y, mean, rstd = bo.norm_fwd([[1.0, 3.0]], [2.0, 1.0], [0.0, 5.0], 0.0)
    assert mean[0] == 2 and rstd[0] == 1
    np.testing.assert_allclose(y, [[-2.0, 6.0]])
    y, mean, rstd = bo.norm_fwd([[3.0, 4.0]], eps=0.0, rms=True)
    np.testing.assert_allclose(y, np.array([[3.0, 4.0]]) / np.sqrt(12.5))


def test_quant_rows_by_hand():
    x = np.array([[127.0, 0.5, 1.5, 2.5, -0.5, -1.5, 126.5, -127.0],
                  [0.0] * 8,
                  [np.inf, 1, 2, 3, 4, 5, 6, 7],
                  [np.nan, np.inf, 2, 3, 4, 5, 6, 7]], dtype=np.float32)
    q, s = bo.quant_rows(x)
    assert s[0] == 1 and s[1] == 0 and np.isinf(s[2]) and np.isnan(s[3])
    assert q[0].tolist() == [127, 0, 2, 2, 0, -2, 126, -127]   # ties to even
    assert not q[1:].any()


def test_matmul_i8_by_loops():
    r = np.random.default_rng(1)
    a, b = (r.integers(-128, 128, size=(n, 16)).astype(np.int8) for n in (3, 5))
    sa, sb = r.random(3).astype(np.float32), r.random(5).astype(np.float32)
    y = bo.matmul_i8(a, sa, b, sb)
    for t in range(3):
        for n in range(5):
            acc = sum(int(a[t, k]) * int(b[n, k]) for k in range(16))
            assert y[t, n] == pytest.approx(acc * float(sa[t]) * float(sb[n]), rel=1e-12)
