"""The ends of the MXINT8 range in the few-bits reference: where the scale stops, how far a value may be off."""
import numpy as np
import pytest

from oracle import few_bits_ref as ref

MAX = float(np.finfo(np.float32).max)


def _blocks(amax, n=200):
    v = np.random.default_rng(int(np.log2(amax)) + 500).uniform(-1, 1, (n, 32)) * amax
    v[:, 0], v[1::2, 1] = amax, -amax
    return v


@pytest.mark.parametrize("amax", [2.0 ** -149, 2.0 ** -130, 2.0 ** -124, 126.9 * 2.0 ** -127, 127 * 2.0 ** -127,
                                  2.0 ** -120, 1.0, 127 / 64, 1.99, 127 / 64 * 2.0 ** 127, MAX])
def test_an_element_is_off_by_its_blocks_largest_over_127_or_half_the_lowest_step(amax):
    v = _blocks(amax)
    q, s = ref.ck8_pack(v)
    assert np.abs(q.astype(int)).max() <= 127
    err = np.abs(ref.ck8_values(q, s) - v)
    assert err.max() <= max(amax / 127, 2.0 ** -127)


def test_the_lowest_step_passes_the_blocks_largest_over_127():
    v = np.zeros(32)
    v[0], v[1] = 2.0 ** -124, 1.9 * 2.0 ** -128
    q, s = ref.ck8_pack(v)
    err = np.abs(ref.ck8_values(q, s) - v).max()
    assert s[0] == 7 and v[0] / 127 < err <= 2.0 ** -127


def test_only_the_last_byte_holds_a_code():
    v = np.zeros((2, 32))
    v[0, :2] = MAX, -MAX                                # 128 2^121 in whole steps
    v[1, 0] = np.nextafter(np.float32(127 / 64 * 2.0 ** 126), np.float32(np.inf))  # the next scale takes it
    q, s = ref.ck8_pack(v)
    assert q[0, :2].tolist() == [127, -127] and s[:, 0].tolist() == [254, 254] and q[1, 0] == 64
