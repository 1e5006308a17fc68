"""The launch schemes of sampling, which go by the number of workgroups: each
gives the tokens that the oracle gives, and the same ones on every call."""
import numpy as np
import pytest

from tests.test_gpu_sample import expect, logits, run


def batch(M, V, seed):
    """Rows of every filter, and of none."""
    rng = np.random.RandomState(seed)
    T = rng.choice([0.0, 0.7, 1.0, 1.0], size=M)
    k = rng.choice([0, 0, 1, 30, 400, 2500], size=M)
    p = rng.choice([1.0, 0.8, 0.95], size=M)
    mp = rng.choice([0.0, 0.0, 0.05], size=M)
    return logits(M, V, seed=seed, std=1.5), rng.rand(M), T, k, p, mp


@pytest.mark.gpu
@pytest.mark.parametrize("M,V", [
    (64, 9000), (65, 9000),            # 128 and 130 workgroups of 16 groups
    (8, 131072), (9, 120000),          # 128, 135
    (128, 700), (129, 700)])           # 128 rows, one workgroup each
def test_few_workgroups_and_more(M, V):
    """A row's last workgroup plans and picks, or kernels of their own do."""
    args = batch(M, V, M)
    want = expect(*args)
    for _ in range(3):
        assert np.array_equal(run(*args)["tokens"], want)


@pytest.mark.gpu
@pytest.mark.parametrize("M,V", [(682, 17500), (683, 17500), (2047, 900),
                                 (2048, 900)])
def test_thousands_of_workgroups(M, V):
    """From 2048 workgroups on each takes twice the groups of a row's sums
    (2046 and 2049 of them here, 2047 and 2048): the tokens of the same rows
    in small batches, and the oracle's on every tenth."""
    args = batch(M, V, M)
    got = run(*args)["tokens"]
    parts = [run(*(a[s:s + 42] for a in args))["tokens"]
             for s in range(0, M, 42)]
    assert np.array_equal(got, np.concatenate(parts))
    some = [a[::10] for a in args]
    assert np.array_equal(got[::10], expect(*some))
