"""The rotation's angles at the ends of their range, against angles in whole numbers.

The angle is p * inv_freq modulo a turn. Here it is a fraction in exact arithmetic: inv_freq is a double, p a whole
number, and pi is known to 80 digits, so p * inv_freq / (2 pi) has an error below 2^31 * 2^53 * 10^-79.
"""

from fractions import Fraction

import numpy as np
import pytest
import torch

import attention_fa2_attn_gb300 as fa
import fa_inputs as fi

pytestmark = pytest.mark.gpu
DEV = "cuda:0"

PI = Fraction(31415926535897932384626433832795028841971693993751058209749445923078164062862090, 10**79)


def _turn(p, f):
    """p * f as a part of a turn in [-1/2, 1/2)."""
    x = Fraction(int(p)) * Fraction(float(f)) / (2 * PI)
    x -= x.numerator // x.denominator
    return float(x - 1 if x >= Fraction(1, 2) else x)


def _rotated(freqs, positions, interleaved=False, call=None, dtype=torch.float32, ab=(1.0, 0.0)):
    """The pair `ab` turned by each angle -> (first, second) [positions][freqs], on the CPU."""
    n = len(freqs)
    x = torch.empty(1, 1, len(positions), 2 * n, dtype=dtype, device=DEV)
    first, second = (slice(0, None, 2), slice(1, None, 2)) if interleaved else (slice(0, n), slice(n, None))
    x[..., first], x[..., second] = ab
    pos = torch.tensor([positions], dtype=torch.int32, device=DEV)
    f = torch.tensor(freqs, dtype=torch.float64, device=DEV)
    y = (call or fa.fa_rope)(x, None, pos, f, interleaved=interleaved)[0][0, 0].float().cpu().double()
    return y[:, first], y[:, second]


POSITIONS = [1, 2, -1, 3, 1000003, 2**31 - 1, -(2**31)]


@pytest.mark.parametrize("interleaved", [False, True])
def test_fast_angles(interleaved):
    # turns a position up to 2^50: the fraction of a turn is off by at most 2^-32 (|p| * 2^-63 turns), so the sines are
    # as right as those of slow pairs: 2^-21 for a pair of (1, 0)
    freqs = [1.0, 6.25, 98765.4321, -(2.0**31) - 0.5, 1e12 + 0.125, 2.0**51 + 1, -(2.0**52) - 1, 2.0**53 - 1]
    cos, sin = _rotated(freqs, POSITIONS, interleaved)
    want = 2 * np.pi * np.array([[_turn(p, f) for f in freqs] for p in POSITIONS])
    assert np.abs(cos.numpy() - np.cos(want)).max() <= 2.0**-21
    assert np.abs(sin.numpy() - np.sin(want)).max() <= 2.0**-21


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("n", [1, 2, 4, 8, 32])
def test_an_angle_that_is_none_leaves_nan(n, interleaved, dtype):
    # NaN, infinite and past 2^53: the pair is NaN at every position, forward and backward; its neighbours are as without it
    for call in (fa.fa_rope, fa.fa_rope_bwd):
        good = [0.5 + i for i in range(n)]
        for bad in (float("nan"), float("inf"), -float("inf"), 2.0**53, -1e300):
            freqs = list(good)
            freqs[n // 2] = bad
            got = _rotated(freqs, [0, 1, -7], interleaved, call, dtype)
            want = _rotated(good, [0, 1, -7], interleaved, call, dtype)
            keep = torch.arange(n) != n // 2
            for g, w in zip(got, want):
                assert torch.isnan(g[:, n // 2]).all(), bad
                assert torch.equal(g[:, keep], w[:, keep])


def test_the_largest_angle_that_is_one_and_the_smallest():
    below = float(np.nextafter(2.0**53, 0))
    cos, sin = _rotated([below, 0.0, 5e-324, 2.0**-70], [1, 0, 7])
    assert torch.isfinite(cos).all() and torch.isfinite(sin).all()
    assert (cos[:, 1:] == 1).all() and (sin[:, 1:].abs() <= 2.0**-60).all() and (cos[1] == 1).all() and (sin[1] == 0).all()


def test_append_takes_the_same_angles():
    q, k, v = (fi.randn((1, 2, 3, 64), 80 + i).to(DEV) for i in range(3))
    pools = [torch.zeros(2, 16, 2, 64, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    f = torch.full((32,), 0.25, dtype=torch.float64, device=DEV)
    f[3], f[5] = float("inf"), 2.0**40
    pos = torch.tensor([[0, 5, 1000]], dtype=torch.int32, device=DEV)
    slots = torch.tensor([[3, 17, 30]], dtype=torch.int32, device=DEV)
    qo = fa.fa_rope_append_paged(q, k, v, pos, slots, f, *pools)
    qr, kr = fa.fa_rope(q, k, pos, f)
    nan = torch.zeros(64, dtype=torch.bool, device=DEV)
    nan[3] = nan[35] = True
    rows = pools[0].view(32, 2, 64)[slots[0].long()].transpose(0, 1)
    for a, b in ((qo, qr), (rows[None], kr)):
        assert torch.isnan(a[..., nan]).all() and torch.equal(a[..., ~nan], b[..., ~nan]) and torch.isfinite(a[..., ~nan]).all()
    assert torch.equal(pools[1].view(32, 2, 64)[slots[0].long()].transpose(0, 1)[None], v)


@pytest.mark.parametrize("interleaved", [False, True])
def test_sines_of_a_pair_are_right_to_their_own_last_place(interleaved):
    """The angle that the sine sees is brought within an eighth of a turn before it is rounded to 24 bits: r, |r| <= pi/4,
    off by at most |r| * 2^-24, beside the whole-number angle's |p| * 2^-63 <= 2^-43 turns. cos moves by |sin| times
    that and the reverse; sine and cosine themselves are off by at most one unit in the last place, 2^-23 of the value;
    a product with 1 and a sum with 0 round nothing. Rounded before that the angle would be off by up to pi * 2^-25,
    which a small sine near half a turn shows."""
    rng = np.random.default_rng(90)
    freqs = list(10.0 ** rng.uniform(-5, 1, 64))
    positions = [int(p) for p in rng.integers(-(2**20), 2**20, 200)]
    cos, sin = (x.numpy() for x in _rotated(freqs, positions, interleaved))
    turn = np.array([[_turn(p, f) for f in freqs] for p in positions])
    r = 2 * np.pi * np.abs(turn - np.round(turn * 4) / 4)  # from the nearest quarter
    off = r * 2.0**-24 + 2 * np.pi * 2.0**-43
    for got, want, slope in ((cos, np.cos(2 * np.pi * turn), np.sin(2 * np.pi * turn)),
                             (sin, np.sin(2 * np.pi * turn), np.cos(2 * np.pi * turn))):
        assert np.all(np.abs(got - want) <= np.abs(slope) * off + 2.0**-23 * np.abs(want))
