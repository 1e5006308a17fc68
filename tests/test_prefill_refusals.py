"""Calls that the prefill's argument checks refuse (CPU): gates that could
grow a state, and, as the decode's, conv states whose entries share memory."""
import pytest
import torch

import linear_attention_speculative_amd as kda
from linear_attention_speculative_amd import _abi
from tests.layer_check import make_layer


def layer(conv):
    kw = make_layer(20, 6, 2, 16, 4, act="f32", device="cpu", conv=conv)
    n = kda.prefill_workspace_size(20, 2, 2, 16, torch.float32)
    kw.update(query_start_loc=torch.tensor([0, 8, 20], dtype=torch.int32),
              state_indices=torch.tensor([1, 2], dtype=torch.int32),
              workspace=torch.empty(n, dtype=torch.uint8))
    return kw


@pytest.mark.parametrize("conv", [True, False])
@pytest.mark.parametrize("bound,code", [
    (None, _abi.KDA_OK), (-5.0, _abi.KDA_OK), (0.0, _abi.KDA_OK),
    (-0.0, _abi.KDA_OK), (1e-30, _abi.KDA_E_UNSUPPORTED),
    (3.0, _abi.KDA_E_UNSUPPORTED), (float("inf"), _abi.KDA_E_UNSUPPORTED),
    (float("nan"), _abi.KDA_E_UNSUPPORTED)])
def test_bounds_above_zero_are_refused(bound, code, conv):
    """A log-decay above 0 leaves the range that the chunked form's operands
    have (every factor at most 1)."""
    check = kda.check_prefill if conv else kda.check_prefill_qkv
    assert check(**dict(layer(conv), lower_bound=bound)) == code
    if code != _abi.KDA_OK:
        assert b"lower_bound" in _abi.load().kda_last_error()


def test_an_unused_bound_is_not_looked_at():
    a = kda.prefill_args(**dict(layer(True), lower_bound=None))
    a.lower_bound = 7.0
    assert _abi.load().kda_check_prefill(a) == _abi.KDA_OK


@pytest.mark.parametrize("op", ["prefill", "decode"])
@pytest.mark.parametrize("dim_first", [True, False])
def test_conv_entries_that_share_memory_are_refused(dim_first, op):
    """Writes of two slots, channels or positions to one element would race."""
    kw = make_layer(2, 6, 2, 16, 4, act="f32", device="cpu",
                    dim_first=dim_first)
    index = dict(state_indices=torch.tensor([1, 2], dtype=torch.int32))
    check = kda.check_decode
    if op == "prefill":
        n = kda.prefill_workspace_size(2, 2, 2, 16, torch.float32)
        index.update(workspace=torch.empty(n, dtype=torch.uint8),
                     query_start_loc=torch.tensor([0, 1, 2],
                                                  dtype=torch.int32))
        check = kda.check_prefill
    N, C, Lc = 6, 96, 6
    shape = (N, C, Lc) if dim_first else (N, Lc, C)
    flat = torch.zeros(4 * N * C * Lc)

    def status(slot, chan, tok):
        strides = (slot, chan, tok) if dim_first else (slot, tok, chan)
        return check(**dict(kw, **index, conv_state=flat.as_strided(
            shape, strides)))

    for ok in ((C * Lc, Lc, 1), (C * Lc, 1, C), (2 * C * Lc, 2 * Lc, 1),
               (C * Lc + 8, 1, C + 1), (1, N * Lc, N), (1, N, N * C)):
        assert status(*ok) == _abi.KDA_OK, ok
    for bad in ((C * Lc - 1, Lc, 1), (Lc, Lc, 1), (C * Lc, Lc - 1, 1),
                (C * Lc, 1, 1), (C * Lc, 1, C - 1), (1, Lc, 1)):
        assert status(*bad) == _abi.KDA_E_LAYOUT, bad
    # one slot has nothing to overlap with
    one = dict(kw, **index, state=kw["state"][:1],
               conv_state=flat.as_strided((1, *shape[1:]),
                                          (0, *((Lc, 1) if dim_first
                                                else (C, 1)))))
    assert check(**one) == _abi.KDA_OK
