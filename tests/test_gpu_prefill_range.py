"""Prefill where magnitudes inside a request lie far apart: outputs that are
what is left of large terms, columns of the state that vanish and come back,
gates at the edge of the fp32 range; against the token-by-token fp64 oracle."""
import numpy as np
import pytest

from tests.layer_check import HALF_STEP, f64, make_layer, reference
from tests.test_gpu_prefill import DEV, run

# A product of the chunked form takes each operand as a pair of fp16 numbers
# (each half rounded to its 11 bits: 2^-24 of the operand; the product of the
# two low halves left out: another 2^-24) and adds up in fp32.  A term passes
# three such products on its way from the state to an output (r = V - K S,
# c = T r, o = Q S + B c), so it is off by at most 3 * 3 * 2^-24 of itself,
# plus, for sums of up to 128 of them, half a step of the partial sum at each
# addition, whose expected size is sqrt(128) 2^-24 of the terms' 2-norm:
# together under 24 * 2^-24 of the largest |q| |S| or |v|.
TERM_TOL = 24 * 2.0 ** -24


def one_key(act, out, D, scale, L=80):
    """Prompts that ask for the one key they write, under betas near 1 and no
    decay, from a state that holds `scale` times as much under that key:
    o_t is what the delta rule left of two large terms."""
    H = 2
    kw = make_layer(L, 4, H, D, 4, act=act, out=out, conv=False, seed=81,
                    lb=-1e-6)
    HD = H * D
    key = kw["mixed_qkv"][:1, HD:2 * HD].clone()
    kw["mixed_qkv"][:, HD:2 * HD] = key
    kw["mixed_qkv"][:, :HD] = key
    kw["raw_beta"].fill_(6.0)
    k = key.float().view(H, D)
    k = k / k.norm(dim=1, keepdim=True)
    v = kw["mixed_qkv"][0, 2 * HD:].float().view(H, D)
    kw["state"][1] = scale * v[:, :, None] * k[:, None, :]
    return kw


@pytest.mark.gpu
@pytest.mark.parametrize("D", [16, 32, 64, 128])
@pytest.mark.parametrize("act,out", [("bf16", "act"), ("bf16", "f32"),
                                     ("f32", "act")])
@pytest.mark.parametrize("scale", [16.0, 64.0])
def test_outputs_left_of_terms_that_cancel(scale, act, out, D):
    """The error of an output goes by the terms' fp32-like accuracy, not by a
    16-bit rounding of what cancels."""
    L = 80
    kw = one_key(act, out, D, scale, L)
    ref = reference(kw, [0, L], [2], [1])
    run(kw, [0, L], [2], [1])
    o, r = f64(kw["out"]), ref["out"]
    v = np.abs(f64(kw["mixed_qkv"])[:, 2 * 2 * D:]).max()
    # a query has norm D^-1/2, the state `scale` times a v row; other sums
    # (the gate's, the state's own over three chunks) stay below these
    term = (scale + 1) * v / np.sqrt(D)
    half = HALF_STEP["bf16" if act == "bf16" and out == "act" else "f32"]
    off = np.abs(o - r) - half * np.abs(r)
    assert off.max() <= TERM_TOL * term, (off.max() / term, np.abs(r).max())
    # the first chunk's last tokens: less than a hundredth of the terms is left
    if scale == 64.0:
        assert np.abs(r[8:]).max() < 0.1 * term
