"""Pins of the few-bits reference: the formats' rules on values worked out by hand, and its gradient
against differences."""
import numpy as np
import pytest

from oracle import few_bits_ref as ref


def _row(first, n=32):
    v = np.zeros(n)
    v[:len(first)] = first
    return v


@pytest.mark.parametrize("amax,byte", [(6.0, 127), (6.0001, 128), (3.0, 126), (1.0, 125), (1.5, 125), (1.50001, 126),
                                       (0.0, 1), (2.0 ** -130, 1)])
def test_mx4_scale(amax, byte):
    assert ref.mx4_quantize(_row([amax]))[1][0] == byte


def test_mx4_rounds_to_the_even_code():
    v = _row([6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.75, -5.0, 0.2500001, 4.9999])
    q, s = ref.mx4_quantize(v)
    assert s[0] == 127
    got = ref.mx4_values(q, s)[:12]
    assert got.tolist() == [6, 0, 1, 1, 2, 2, 4, 4, -1, -4, 0.5, 4]
    assert q[0] == 7 and q[1] == (2 | 2 << 4)


@pytest.mark.parametrize("amax,byte", [(127 / 64, 127), (127.01 / 64, 128), (1.0, 127), (0.99, 126), (0.0, 7),
                                       (2.0 ** -128, 7), (2.0 ** 127, 254), (255 / 128 * 2.0 ** 127, 254)])
def test_ck8_scale(amax, byte):
    q, s = ref.ck8_pack(_row([amax, -amax]))
    assert s[0] == byte and abs(int(q[0])) <= 127


def test_ck8_rounds_to_even_and_stays_near():
    v = _row([127 / 64, 0.5 / 64, 1.5 / 64, -2.5 / 64, 3.49 / 64])
    q, s = ref.ck8_pack(v)
    assert q[:5].tolist() == [127, 0, 2, -2, 3]
    r = np.random.default_rng(0).standard_normal((50, 64)) * np.exp2(np.arange(50) - 25)[:, None]
    q, s = ref.ck8_pack(r)
    err = np.abs(ref.ck8_values(q, s) - r).reshape(50, 2, 32).max(-1)
    assert (err <= np.abs(r).reshape(50, 2, 32).max(-1) / 127).all()


def test_blocks_with_no_number_come_back_as_nan():
    for bad in (np.inf, -np.inf, np.nan):
        v = np.ones(64)
        v[40] = bad
        for pack, values in ((ref.mx4_quantize, ref.mx4_values), (ref.ck8_pack, ref.ck8_values)):
            got = values(*pack(v))
            assert np.isfinite(got[:32]).all() and np.isnan(got[32:]).all()


def test_every_code_survives():
    codes = np.arange(256, dtype=np.uint8).reshape(16, 16)
    s = np.full((16, 1), 130, dtype=np.uint8)
    v = ref.mx4_values(codes, s)
    v[:, 0] = np.where(np.abs(v).max(1) < 48, 48, v[:, 0])  # the block's largest fixes its scale
    q, s2 = ref.mx4_quantize(v)
    assert np.array_equal(ref.mx4_values(q, s2), v) and (s2 == 130).all()


def test_dswiglu_against_differences():
    r = np.random.default_rng(1)
    a, b, dh = (r.standard_normal((5, 7)) for _ in range(3))
    f = lambda a, b: (dh * ref.silu(a) * b).sum()  # noqa: E731
    g = ref.dswiglu(dh, a, b)
    for i in range(5):
        for j in range(7):
            for n, v in ((0, a), (7, b)):
                v[i, j] += 1e-6
                up = f(a, b)
                v[i, j] -= 2e-6
                down = f(a, b)
                v[i, j] += 1e-6
                assert abs((up - down) / 2e-6 - g[i, j + n]) < 1e-7
