"""Sampling at borders between tokens that a few units of the weights' last
binary place decide: the weights are what the documentation says, exp of the
distance to the maximum rounded to 46 places."""
from fractions import Fraction

import numpy as np
import pytest

import oracle
from tests.test_gpu_sample import f32, run

PLACES = 46
STEP = np.log(2.0) / 256               # of the kernels' table of weights


def weight(x):
    """exp(x) in units of 2^-46, to a hundredth of one: by its series, of
    which 40 terms leave under 2^-60 for |x| <= 2, and squared up from there."""
    halvings = max(0, int(np.ceil(np.log2(max(-float(x), 1e-30) / 2))))
    y = Fraction(float(x)) / 2 ** halvings
    term, total = Fraction(1), Fraction(1)
    for n in range(1, 41):
        term = Fraction(int(term * y / n * 2 ** 200), 2 ** 200)
        total += term
    for _ in range(halvings):
        total = Fraction(int(total * total * 2 ** 200), 2 ** 200)
    return total * 2 ** PLACES


def units(x):
    return int(weight(x) + Fraction(1, 2))


def row_with_rest(rest, seed):
    """Logits whose first is the maximum, 0, and whose others weigh `rest`
    units together, the large ones of them between two steps of 1/256 octave
    (where a short series for the step's fraction errs most)."""
    rng = np.random.RandomState(seed)
    x, left = [np.float32(0.0)], rest
    for share in (0.5, 0.8):               # of what is left
        n = np.ceil(-np.log(share * left / 2.0 ** PLACES) / STEP - 0.5)
        v = np.float32(-(n + 0.5 + 0.04 * (rng.rand() - 0.5)) * STEP)
        x.append(v)
        left -= units(v)
    while left > 0:
        v = np.float32(np.log(left / 2.0 ** PLACES))
        while units(v) > left:
            v = np.nextafter(v, np.float32(-100))
        x.append(v)
        left -= units(v)
    assert left == 0 and len(x) < 12
    return np.array(x + [np.float32(-200)] * (12 - len(x)), np.float32)


CASES = [(seed, over) for seed in range(8) for over in (4, -4)]


def rows():
    one = 2 ** PLACES
    return np.stack([row_with_rest(one + over, seed) for seed, over in CASES])


def test_rows_weigh_what_they_should():
    """The oracle's double-precision weights agree on every row: half of the
    mass lies before or behind the first token by four units."""
    for x, (_, over) in zip(rows(), CASES):
        assert sum(units(v) for v in x[1:]) == 2 ** PLACES + over
        assert (oracle.sample_row(x.astype(np.float64), 0.5) > 0) == (over > 0)


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 16, 160])
def test_half_of_the_mass(M):
    """u = 1/2 against rows whose first token weighs half, four units more or
    less (in fp64 the weights of a row can be off by one unit where they lie
    next to the middle of two): few rows, and many."""
    x = np.resize(rows(), (M, 12))
    got = run(f32(x), np.full(M, 0.5))["tokens"]
    want = np.resize([over > 0 for _, over in CASES], M)
    assert np.array_equal(got > 0, want)
    assert np.array_equal(got, [oracle.sample_row(r.astype(np.float64), 0.5)
                                for r in x])


@pytest.mark.gpu
@pytest.mark.parametrize("k", [None, 12, 11])
def test_top_p_of_one_half(k):
    """top-p = 1/2 keeps the first token alone, or one more."""
    x, n = rows(), len(CASES)
    ks = None if k is None else np.full(n, k)
    got = run(f32(x), np.full(n, 0.999), k=ks, p=np.full(n, 0.5))["tokens"]
    assert np.array_equal(got > 0, [over > 0 for _, over in CASES])


@pytest.mark.gpu
@pytest.mark.parametrize("k,p", [(None, None), (6, None), (None, 0.999999),
                                 (6, 0.99)])
def test_uniform_numbers_from_one_on(k, p):
    """u is held to [0, 1): to the largest number below 1, so that a number
    that was rounded up to 1 does not take the last token with any weight."""
    u = np.array([1.0, 1.5, 4.0, 1e20, 3e38, np.inf, 1 - 2.0 ** -24])
    x = np.full((len(u), 9), -25.0, np.float32)
    x[:, 1] = 0.0
    n = len(u)
    got = run(f32(x), u, k=None if k is None else np.full(n, k),
              p=None if p is None else np.full(n, p))["tokens"]
    assert got.tolist() == [1] * n
