"""How the few-token products are laid out, over the whole range of sizes that the calls take (no GPU)."""
import itertools

import pytest

import _few_plan as P

SM, CTA = 227 << 10, 1 << 10
TOKENS = [1, 2, 7, 8, 9, 16, 17, 31, 32, 33, 500]
EXPERTS = [(1, 1), (1, 32), (2, 4), (8, 32), (8, 256), (8, 1024), (32, 33), (32, 512), (32, 1022), (32, 1023), (32, 1024)]
ROWS = [16, 48, 512, 2432, 2448, 4096, 4864, 4880, 7168, 24576, 300000]
UNITS = [1, 2, 3, 8, 16, 17, 56, 64, 1000, 16384]
FORMS = [(False, True), (True, True), (True, False)]


def _domain():
    return itertools.product(TOKENS, EXPERTS, ROWS, UNITS, FORMS)


def test_every_layout_fits():
    for T, (k, E), rows, units, (four, whole) in _domain():
        for capped in (False, True):
            R, warps, ctas, stages, smem, _ = at = P.choice(T, k, E, rows, units, four, whole, capped)
            assert ctas >= 1 and warps >= 4 and 2 <= stages <= 4, (T, k, E, rows, units, four, at)
            assert smem + CTA <= SM and ctas * (smem + CTA) <= SM, (T, k, E, rows, units, four, at)
            assert smem >= warps * (stages * 16 * R * 144), at


def test_a_cap_keeps_the_order_of_the_sums():
    for T, (k, E), rows, units, (four, whole) in _domain():
        a, b = P.choice(T, k, E, rows, units, four, whole), P.choice(T, k, E, rows, units, four, whole, True)
        assert a[:2] == b[:2] and b[2] == 1, (T, k, E, rows, units, four)


@pytest.mark.parametrize("E", [1023, 1024])
@pytest.mark.parametrize("N", [2448, 4096, 4864])
def test_tables_of_many_experts_leave_room(N, E):
    """32 choices of about a thousand experts: twelve warps of two tiles and the sums of 32 tokens are 16 bytes too many."""
    for I in (128, 2048):
        for T in (32, 33):
            up, down = P.layer(T, 32, E, 128, I, N, "")
            assert up[2] >= 1 and down[2] >= 1 and down[1] < 12


def _cost(rows, units, R, warps, ctas):
    rounds = -(-(-(-rows // (16 * R))) // (152 * ctas))
    return rounds * (-(-units // warps) + 0.3) * (12 if R == 2 else 16)


def test_the_layout_that_was_weighed_is_the_one_that_runs():
    """The cost is that of the CTAs an SM that fit, and no layout that fits costs less."""
    for T, (k, E), rows, units, (four, whole) in _domain():
        R, warps, ctas, _, _, cost = at = P.choice(T, k, E, rows, units, four, whole)
        assert cost == pytest.approx(_cost(rows, units, R, warps, ctas)), (T, k, E, rows, units, four, at)
        most = 12 if R == 2 else 16
        for w in range(4, most + 1):
            for c in range(1, most // w + 1):
                if P.stages(T, k, E, w, c, R):
                    assert _cost(rows, units, R, w, c) >= cost * (1 - 1e-6), (T, k, E, rows, units, four, at, w, c)


def test_units_of_two_tiles_are_weighed_by_what_fits():
    """32 tokens through 8 of 64 experts of 7168x2048: six warps at two CTAs an SM do not fit, twelve at one do."""
    for product in P.layer(32, 8, 64, 7168, 2048, 7168, ""):
        assert product[:3] == (2, 12, 1)
