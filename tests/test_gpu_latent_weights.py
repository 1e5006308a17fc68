"""Softmax weights of the bf16 attention kernels hold 16 bits of each weight,
and requests whose block tables exceed what LDS holds of them."""
import numpy as np
import pytest
import torch

import linear_attention_speculative_amd as kda
from tests import test_gpu_latent as absorbed
from tests import test_gpu_latent_prompt as prompts
from tests.latent_check import f64, hold, make


def halves(ref, dims):
    """Largest errors of a bf16 output whose weights are two bf16 values: the
    first keeps the leading 8 bits of a weight, the second the rest, below 2^-7
    of it, rounded to half a step, 2^-8: 2^-15 of the weight (and 2^-23 for
    what keeps that rest above 0).  Scores, sums and the last rounding as in
    `bounds`."""
    u = 2.0 ** -24
    score = (dims + 4) * u * ref["size"]
    rel = 2 * (np.expm1(score) + (ref["keys"] + 8) * u) + 2.0 ** -15 + 2 * u
    out = rel[..., None] * ref["weight"] + 1e-30
    return out + 2.0 ** -8 * (np.abs(ref["out"]) + out)


@pytest.mark.gpu
@pytest.mark.parametrize("R,P,scale", [(128, 0, 0.02), (512, 64, 0.005),
                                       (256, 64, -0.01)])
def test_latent_attention(R, P, scale):
    kw = make([1, 4, 30], [9, 33, 500], H=8, R=R, P=P, block=16, act="bf16",
              seed=R)
    kw["softmax_scale"] = scale
    ref = absorbed.expect(kw)
    absorbed.run(kw)
    torch.cuda.synchronize()
    hold(f64(kw["out"]), ref["out"], halves(ref, R + P), "out")


@pytest.mark.gpu
@pytest.mark.parametrize("D,P", [(128, 64), (64, 0)])
def test_prefill(D, P):
    kw = prompts.prompt([3, 40, 300], [3, 90, 300], H=3, D=D, P=P, act="bf16",
                        seed=D)
    kw["softmax_scale"] = 0.01
    ref = prompts.expect(kw)
    kda.latent_prefill(**kw)
    torch.cuda.synchronize()
    hold(f64(kw["out"]), ref["out"], halves(ref, D + P), "out")


@pytest.mark.gpu
def test_infinite_values_at_any_weight():
    """Weights that the first half holds whole (1, and its powers of two), and
    others: an infinite value leaves its sum infinite, not NaN."""
    n = 200
    kw = prompts.prompt([n], [n], H=2, D=64, P=0, act="bf16", seed=3)
    kw["q"][:, 0] = 0                      # head 0: equal weights
    inf = float("inf")
    for tok, dim, v in ((0, 1, inf), (0, 2, -inf), (100, 3, inf),
                        (199, 4, -inf)):
        kw["value"][tok, :, dim] = v
    kda.latent_prefill(**kw)
    torch.cuda.synchronize()
    out = f64(kw["out"])
    assert (out[:, :, 1] == np.inf).all() and (out[:, :, 2] == -np.inf).all()
    assert (out[100:, :, 3] == np.inf).all()
    assert np.isfinite(out[:100, :, 3]).all()
    assert (out[199:, :, 4] == -np.inf).all()
    assert np.isfinite(out[:199, :, 4]).all()
    assert np.isfinite(out[:, :, 5:]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_runs_past_the_table_in_lds(act):
    """512 entries of a block table are in LDS at a time: with a block a token
    and 140 requests of some 1500 tokens a workgroup's run passes that."""
    computed = [1400 + 3 * i for i in range(140)]
    kw = make([1] * 140, computed, H=2, R=128, P=0, block=1, act=act, seed=4)
    steps = sum(-(-(c + 1) // 32) + 4 for c in computed)
    assert (steps // 256 - 8) * 32 > 512
    kw["block_table"][5:60:7, 700:900:3] = 0        # null blocks among them
    ref = absorbed.expect(kw)
    absorbed.run(kw)
    torch.cuda.synchronize()
    absorbed.check(kw, ref, act)
