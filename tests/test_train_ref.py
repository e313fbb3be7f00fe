"""The plain implementations behind the training operators' tests, pinned without a GPU: the generator to the
published vectors, the gate's gradient to differences."""
import numpy as np
import pytest

import _train_ref as R


@pytest.mark.parametrize("counter,key,want", [
    # the known answers that the generator's authors publish for Philox4x32-10
    ([0, 0, 0, 0], [0, 0], [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]),
    ([0xFFFFFFFF] * 4, [0xFFFFFFFF] * 2, [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]),
    ([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], [0xA4093822, 0x299F31D0],
     [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]),
])
def test_generator_known_answers(counter, key, want):
    assert [int(x) for x in R.philox(np.array(counter), key)] == want


def test_keep_rate_is_the_threshold():
    n = 1 << 20
    for p in (0.1, 0.5):
        q = 1 - R.threshold(p) / 65536
        kept = R.keep_mask(0, n, p, seed=7, offset=3).mean()
        assert abs(kept - q) < 6 * np.sqrt(q * (1 - q) / n)      # six standard deviations
    assert R.keep_mask(0, 1000, 0.0, 1, 2).all()


def test_gate_gradient_against_differences():
    """Central differences with step e: truncation e²/6 · max|h'''| (third derivatives of silu are below 1 for
    these u), rounding 2^-52·|h|/e."""
    rng = np.random.default_rng(0)
    g, u = rng.uniform(-12, 12, 500), rng.uniform(-3, 3, 500)
    e = 1e-4
    dg, du = R.gate_grad(g, u, 1.0)
    num_g = (R.gate(g + e, u) - R.gate(g - e, u)) / (2 * e)
    num_u = (R.gate(g, u + e) - R.gate(g, u - e)) / (2 * e)
    bound = e * e / 6 * 3 + 2.0 ** -52 * 40 / e
    assert np.abs(dg - num_g).max() < bound
    assert np.abs(du - num_u).max() < bound


def test_cast_reference_on_known_groups():
    x = np.zeros((1, 128), np.float32)
    codes, s = R.cast_groups(x, 1, 128, False)
    assert (codes == 0).all() and s[0, 0] == 1
    x[0, 3], x[0, 4] = 448.0, -224.0
    for ue in (False, True):
        codes, s = R.cast_groups(x, 1, 128, ue)
        assert R.e4m3_values(codes)[0, 3] == 448 and R.e4m3_values(codes)[0, 4] == -224
        assert s[0, 0] == (127 if ue else 1)
    x[0, 3] = np.nextafter(np.float32(448), np.float32(500))
    assert R.cast_groups(x, 1, 128, True)[1][0, 0] == 128        # just past 448: the next power of two
