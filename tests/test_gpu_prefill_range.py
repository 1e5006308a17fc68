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


# A decay e^G over a chunk: every log-decay g is off by a few roundings of
# itself (2^-22 of it), its exponential by (|g| + 1) 2^-23 (the product with
# log2 e), so the decay by at most |G| (2^-22 + 2^-23) + 32 * 2^-23 of itself:
# 3.6e-5 at G = -89.  Twice that, for a state and the output read from it.
DECAY_TOL = 8e-5


# Where nothing is written, what a chunk leaves of a state is its decay e^G
# and a correction for each token, beta k^ (k^ . S), decayed in two factors of
# the chunked form: e^G_t before the token (in k e^G_t, T and r) and e^(G-G_t)
# after it.  Each factor is rounded to a multiple of a fixed step, by at most
# itself; a term of four such factors is off by at most 2^4 - 1 times itself,
# and there are 32, of at most e^G times the column each: under 512 e^G.
LEFT_TOL = 512.0


def vanishing(D, act, v_later, held, total=-88.7, L=120):
    """A state of `held` that the first chunk's gates bring down by e^total
    while nothing is written; from token 64 on values of `v_later`, without
    decay."""
    H = 2
    kw = make_layer(L, 4, H, D, 4, act=act, out="f32", conv=False, seed=82,
                    lb=-5.0)
    kw["A_log"].zero_()
    kw["dt_bias"].zero_()
    g = total / 32 / -5.0                      # share of the bound, a token
    kw["raw_gate"][:32] = float(np.log(g / (1 - g)))
    kw["raw_gate"][32:] = -30.0                # 5e^-30: none
    v = kw["mixed_qkv"][:, 2 * H * D:]
    v[:64] = 0
    v[64:] *= v_later
    kw["state"].mul_(held / kw["state"][1].abs().max())
    return kw


def agree(kw, ref, slot, tol, parts):
    """Outputs of the row ranges `parts`, each against its own largest, and
    the slot's state."""
    o, r = f64(kw["out"]), ref["out"]
    assert np.isfinite(o).all() and np.isfinite(f64(kw["state"])).all()
    for s, e in parts:
        top = np.abs(r[s:e]).max()
        err = np.abs(o[s:e] - r[s:e]).max()
        assert err <= tol * top, (s, e, err / max(top, 1e-300), top)
    s, r = f64(kw["state"])[slot], ref["state"][slot]
    err = np.abs(s - r).max() / np.abs(r).max()
    assert err <= tol, err


@pytest.mark.gpu
@pytest.mark.parametrize("D", [16, 32, 64, 128])
@pytest.mark.parametrize("held", [3e5, 4e7, 1.5e8, 1e9, 1e12])
def test_large_states_that_decay_to_nothing(held, D):
    """A column of 1e5 to 1e12 that one chunk decays by 2^-128, and no values
    after it: what is left stays as small as that."""
    kw = vanishing(D, "f32", 0.0, held)
    ref = reference(kw, [0, 120], [2], [1])
    run(kw, [0, 120], [2], [1])
    # a column of D channels, each at most `held`
    left = LEFT_TOL * np.exp(-88.7) * held * np.sqrt(D)
    o, s = f64(kw["out"]), f64(kw["state"])[2]
    assert np.abs(o[32:] - ref["out"][32:]).max() <= left
    assert np.abs(s - ref["state"][2]).max() <= left
    # the first chunk's outputs, from the state as it was
    top = np.abs(ref["out"][:32]).max()
    assert np.abs(o[:32] - ref["out"][:32]).max() <= DECAY_TOL * top


@pytest.mark.gpu
@pytest.mark.parametrize("D", [32, 128])
@pytest.mark.parametrize("held", [0.0, 1e-12, 1.0, 1e9])
@pytest.mark.parametrize("v_later", [1e-20, 1.0, 3e5, 1e9, 1e30])
def test_values_after_a_column_vanished(v_later, held, D):
    """Values of any size after chunks of zeros over a state that decayed to
    (almost) nothing: the scale that followed it down does not overflow."""
    kw = vanishing(D, "f32", v_later, held)
    ref = reference(kw, [0, 120], [2], [1])
    run(kw, [0, 120], [2], [1])
    # (what was left of the state, at most 1e9 e^-88.7 = 3e-30, is under the
    # smallest step of 1e-20)
    agree(kw, ref, 2, DECAY_TOL, [(64, 120)])


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
def test_values_near_the_largest_fp32(D):
    """Values of up to 1e38, some at a time."""
    L, H = 100, 2
    kw = make_layer(L, 4, H, D, 4, act="f32", conv=False, seed=83, lb=-5.0)
    v = kw["mixed_qkv"][:, 2 * H * D:]
    v.div_(v.abs().max())
    v[np.arange(L) % 9 > 0] = 0
    v.mul_(1e38)
    kw["raw_gate"].fill_(-1.0)
    ref = reference(kw, [0, L], [2], None)
    assert np.abs(ref["state"]).max() < 3e38
    run(kw, [0, L], [2], None)
    agree(kw, ref, 2, DECAY_TOL, [(0, 32), (32, 100)])
