"""Chunked prefill of a KDA layer against the token-by-token fp64 oracle:
lengths around the chunk and its sub-blocks, head dims, dtypes, layouts, both
gates, strong decays that underflow inside a chunk, continued and in-place
states, null slots, rows behind the last request, a prompt in pieces, the
decode that follows, streams and graph replays; and the refusals (CPU)."""
import numpy as np
import pytest
import torch

import linear_attention_speculative_amd as kda
from linear_attention_speculative_amd import _abi
from tests.layer_check import TORCH, compare, f64, i32, make_layer, reference

DEV = "cuda"


def workspace(kw, B, device=DEV):
    T, H = kw["raw_beta"].shape
    n = kda.prefill_workspace_size(T, B, H, kw["state"].shape[3],
                                   kw["mixed_qkv"].dtype, kw["out"].dtype)
    return torch.full((n,), 0xff, dtype=torch.uint8, device=device)


def run(kw, qsl, slots, initial, accepted=None, **more):
    call = kda.conv_prefill if "conv_state" in kw else kda.prefill_qkv
    args = dict(kw, query_start_loc=i32(qsl, DEV),
                state_indices=i32(slots, DEV),
                initial_state_indices=None if initial is None
                else i32(initial, DEV), workspace=workspace(kw, len(slots)),
                **more)
    if accepted is not None:
        args["num_accepted_tokens"] = i32(accepted, DEV)
    call(**args)
    torch.cuda.synchronize()
    return args


def check(kw, lens, slots, initial, accepted=None, tail=0):
    """One launch against the oracle; `tail` rows behind the last request."""
    qsl = np.concatenate([[0], np.cumsum(lens)])
    assert kw["out"].shape[0] == qsl[-1] + tail
    ref = reference(kw, qsl, slots, initial, accepted)
    run(kw, qsl, slots, initial, accepted)
    N = kw["state"].shape[0]
    written = [s for s, n in zip(slots, lens) if 0 < s < N and n > 0]
    compare(kw, ref, written, pairs=True)


LENGTHS = [[1], [2, 1, 3], [15, 16, 17], [31, 32, 33, 0, 34], [64, 65, 63],
           [100, 0, 1, 47], [193]]
CASES = [
    dict(H=2, D=128), dict(H=3, D=64, dim_first=False),
    dict(H=1, D=32, lb=-5.0, act="f32"), dict(H=5, D=16),
    dict(H=2, D=128, act="f32", lb=-5.0), dict(H=1, D=16, act="f32"),
    dict(H=2, D=64, out="f32", weight="f32", gentle=False),
]


@pytest.mark.gpu
@pytest.mark.parametrize("ci", range(len(CASES)))
@pytest.mark.parametrize("li", range(len(LENGTHS)))
def test_prefill_matches_oracle(li, ci):
    lens, B = LENGTHS[li], len(LENGTHS[li])
    rng = np.random.RandomState(100 * li + ci)
    kw = make_layer(sum(lens) + 3, 2 * B + 2, Q=4, seed=100 * li + ci,
                    **CASES[ci])
    perm = 1 + rng.permutation(2 * B)
    initial = perm[B:].copy()
    initial[::2] = 0                       # every other prompt starts afresh
    check(kw, lens, perm[:B], initial, rng.randint(-1, 7, size=B), tail=3)


@pytest.mark.gpu
@pytest.mark.parametrize("ci", range(len(CASES)))
def test_prefill_of_convolved_inputs(ci):
    kw = make_layer(150, 8, Q=4, seed=ci, conv=False,
                    **{k: v for k, v in CASES[ci].items()
                       if k not in ("dim_first", "weight")})
    check(kw, [37, 1, 112], [3, 1, 7], [3, 0, 5])


@pytest.mark.gpu
@pytest.mark.parametrize("strong", [40.0, 2000.0])
def test_decays_that_empty_the_state(strong):
    """Gates whose decays underflow within a few tokens, next to tokens that
    keep everything: products of decays of any size stay exact."""
    kw = make_layer(90, 3, 2, 64, 4, act="f32", conv=False, seed=5)
    gate = torch.randn(90, 128, device=DEV)
    gate[torch.rand(90, 128, device=DEV) < 0.2] = strong
    gate[torch.rand(90, 128, device=DEV) < 0.3] = -60.0
    kw["raw_gate"] = gate
    kw["dt_bias"] = torch.zeros_like(kw["dt_bias"])
    check(kw, [90], [1], [2])


@pytest.mark.gpu
def test_repeated_keys_and_unit_betas():
    """The triangular system at its stiffest: every key the same, betas 1,
    no decay."""
    kw = make_layer(70, 2, 1, 32, 4, act="f32", conv=False, seed=6)
    kw["mixed_qkv"][:, 32:64] = kw["mixed_qkv"][:1, 32:64].clone()
    kw["raw_beta"].fill_(40.0)
    kw["raw_gate"].fill_(-80.0)
    check(kw, [70], [1], None)


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [1e-20, 1e-3, 3e4, 1e18])
def test_values_of_any_magnitude(scale):
    """Scales of v (and of the states they make) far outside the range of the
    16-bit operand pairs."""
    kw = make_layer(80, 3, 2, 64, 4, act="f32", conv=False, seed=7)
    kw["mixed_qkv"][:, 256:] *= scale
    kw["mixed_qkv"][:, 256::7] *= 1e-3
    kw["state"].mul_(scale)
    check(kw, [50, 30], [1, 2], [1, 0])


@pytest.mark.gpu
def test_zero_inputs_and_states():
    kw = make_layer(40, 3, 2, 64, 4, act="f32", conv=False, seed=7)
    kw["mixed_qkv"].zero_()
    kw["state"].zero_()
    check(kw, [40], [1], [2])
    assert (kw["out"] == 0).all()


@pytest.mark.gpu
def test_null_slots_and_rows_behind():
    """Null, negative and out-of-range state slots: zeros for their rows,
    nothing else; null initial slots mean zeros."""
    lens = [20, 35, 1, 40]
    kw = make_layer(sum(lens) + 9, 5, 2, 32, 4, seed=9)
    check(kw, lens, [0, 2, -3, 5], [1, -1, 2, 3], tail=9)
    assert (f64(kw["out"])[-9:] == 7.0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_non_finite_inputs_stay_in_their_request(act):
    """A NaN or infinite input spoils its own request from its chunk on: the
    chunks before it and the other requests stay as without it."""
    lens, slots = [40, 100, 70], [1, 2, 3]
    qsl = np.concatenate([[0], np.cumsum(lens)])
    a = make_layer(210, 5, 2, 64, 3, act=act, seed=61)
    b = {k: v.clone() if isinstance(v, torch.Tensor) else v
         for k, v in a.items()}
    t = 40 + 70                           # token 70 of the second request
    b["mixed_qkv"][t, :128] = float("nan")
    b["raw_gate"][t + 3, 5] = float("nan")
    b["mixed_qkv"][t + 9, -3] = float("inf")
    run(a, qsl, slots, None)
    run(b, qsl, slots, None)
    whole = np.r_[0:40 + 64, 140:210]     # chunks of 32 before token 70
    assert torch.equal(a["out"][whole], b["out"][whole])
    for s in (1, 3):
        assert torch.equal(a["state"][s], b["state"][s])
        assert torch.equal(a["conv_state"][s], b["conv_state"][s])
    assert bool(torch.isnan(b["out"][t:140]).any())


@pytest.mark.gpu
def test_in_place_continuation_in_pieces():
    """A prompt in pieces through one slot, the pieces continuing in place,
    equals the whole prompt."""
    pieces = [5, 64, 1, 2, 43]
    kw = make_layer(sum(pieces), 4, 2, 64, 3, act="f32", seed=11)
    ref = reference(kw, [0, sum(pieces)], [2], None)
    at = 0
    for i, n in enumerate(pieces):
        part = dict(kw, **{k: kw[k][at:at + n] for k in (
            "mixed_qkv", "raw_gate", "raw_beta", "out")})
        run(part, [0, n], [2], [2] if i else None)
        at += n
    compare(kw, ref, [2], pairs=True)


@pytest.mark.gpu
def test_prefill_then_decode():
    """The slot a prefill leaves is what the decode reads: a prompt, then ten
    single tokens, against the oracle over all of them."""
    L, D, H = 45, 128, 2
    kw = make_layer(L + 10, 3, H, D, 4, act="f32", seed=12, lb=-5.0)
    ref = reference(kw, [0, L + 10], [1], None)
    rows = ("mixed_qkv", "raw_gate", "raw_beta", "out")
    run(dict(kw, **{k: kw[k][:L] for k in rows}), [0, L], [1], None)
    for t in range(L, L + 10):
        kda.conv_update_decode(**dict(kw, **{k: kw[k][t:t + 1]
                                             for k in rows}),
                               state_indices=i32([1], DEV))
    torch.cuda.synchronize()
    compare(kw, ref, [1], pairs=True)


@pytest.mark.gpu
def test_many_requests_of_one_token():
    B = 300
    kw = make_layer(B, 2 * B + 1, 1, 16, 4, act="f32", seed=13)
    rng = np.random.RandomState(1)
    perm = 1 + rng.permutation(2 * B)
    check(kw, [1] * B, perm[:B], perm[B:])


@pytest.mark.gpu
def test_unordered_offsets_stay_inside():
    """Offsets that run backwards or past the rows are clamped: no result is
    defined, nothing outside the tensors is touched."""
    kw = make_layer(40, 4, 1, 32, 4, act="f32", conv=False, seed=3)
    run(kw, [-5, 90, 20, 10 ** 9], [1, 2, 3], None)


@pytest.mark.gpu
@pytest.mark.parametrize("qsl", [[0, 0, 0, 0], [40, 40, 40, 40],
                                 [33, 0, 70, 0], [40, 5, 5, 39]])
def test_workspace_content_is_never_an_index(qsl):
    """A batch of rows without any request's token (as a padded launch has
    them) changes nothing, and no batch takes an index from what an earlier
    call left in the workspace."""
    kw = make_layer(40, 4, 3, 64, 3, act="f32", seed=17)
    before = {n: kw[n].clone() for n in ("out", "state", "conv_state")}
    work = workspace(kw, 3)
    work.view(torch.int32).fill_(2)
    args = dict(kw, query_start_loc=i32(qsl, DEV),
                state_indices=i32([1, 2, 3], DEV), workspace=work)
    kda.conv_prefill(**args)
    torch.cuda.synchronize()
    if len(set(qsl)) == 1:
        for name, old in before.items():
            assert torch.equal(kw[name], old), name
        # the same rows as one request, over the same workspace
        args["query_start_loc"] = i32([0, 40, 40, 40], DEV)
        ref = reference(kw, [0, 40, 40, 40], [1, 2, 3], None)
        kda.conv_prefill(**args)
        torch.cuda.synchronize()
        compare(kw, ref, [1], pairs=True)


@pytest.mark.gpu
def test_graph_replays_and_streams():
    """A captured prefill replayed over new inputs, with eager work between
    the replays, against eager calls; the call runs on the stream given."""
    lens = [50, 3]
    qsl, slots = [0, 50, 53], [1, 2]
    kw = make_layer(53, 3, 2, 64, 4, act="f32", seed=21)
    args = dict(kw, query_start_loc=i32(qsl, DEV),
                state_indices=i32(slots, DEV), workspace=workspace(kw, 2))
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    kda.conv_prefill(stream=stream, **args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.conv_prefill(**args)
    for i in range(3):
        kw["mixed_qkv"].copy_(torch.randn_like(kw["mixed_qkv"]))
        eager = {k: v.clone() if isinstance(v, torch.Tensor) else v
                 for k, v in kw.items()}
        graph.replay()
        torch.cuda.synchronize()
        run(eager, qsl, slots, None)
        for name in ("out", "state", "conv_state"):
            assert torch.equal(kw[name], eager[name]), (i, name)
    assert lens


@pytest.mark.gpu
def test_two_prefills_at_once_on_two_streams():
    """Launches in flight together, each with its own workspace."""
    sets = [make_layer(300, 3, 4, 64, 4, act="f32", seed=30 + i)
            for i in range(2)]
    alone = []
    for kw in sets:
        c = {k: v.clone() if isinstance(v, torch.Tensor) else v
             for k, v in kw.items()}
        run(c, [0, 300], [1], None)
        alone.append(c)
    args = [dict(kw, query_start_loc=i32([0, 300], DEV),
                 state_indices=i32([1], DEV), workspace=workspace(kw, 1))
            for kw in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(3):
        for a, s in zip(args, streams):
            kda.conv_prefill(stream=s, **a)
    torch.cuda.synchronize()
    for kw, c in zip(sets, alone):
        assert torch.equal(kw["out"], c["out"])
        assert torch.equal(kw["state"][1], c["state"][1])


def _cpu(**over):
    kw = make_layer(20, 6, 2, 16, 4, act="f32", device="cpu", **over)
    kw.update(query_start_loc=torch.tensor([0, 8, 20], dtype=torch.int32),
              state_indices=torch.tensor([1, 2], dtype=torch.int32),
              workspace=workspace(kw, 2, "cpu"))
    return kw


def test_prefill_checks():
    ok = _cpu()
    assert kda.check_prefill(**ok) == _abi.KDA_OK, \
        _abi.load().kda_last_error()
    small = ok["workspace"][:-256]
    bad = [
        (dict(workspace=small), _abi.KDA_E_CAPACITY),
        (dict(state=ok["state"].bfloat16()), _abi.KDA_E_DTYPE),
        (dict(state=ok["state"][:, :, :, :8]), _abi.KDA_E_UNSUPPORTED),
        (dict(out=ok["out"][:19]), _abi.KDA_E_SHAPE),
        (dict(out=ok["out"].bfloat16()), _abi.KDA_E_DTYPE),
        (dict(mixed_qkv=ok["mixed_qkv"].t().contiguous().t()),
         _abi.KDA_E_LAYOUT),
        (dict(conv_state=ok["conv_state"].bfloat16()), _abi.KDA_E_DTYPE),
        (dict(conv_state=ok["conv_state"][:5]), _abi.KDA_E_SHAPE),
        (dict(spec_query_len=0), _abi.KDA_E_UNSUPPORTED),
        (dict(conv_state=ok["conv_state"][:1].expand(6, -1, -1)),
         _abi.KDA_E_LAYOUT),
        (dict(conv_state=ok["conv_state"][:, :, :1].expand(-1, -1, 6)),
         _abi.KDA_E_LAYOUT),
    ]
    for over, code in bad:
        assert kda.check_prefill(**dict(ok, **over)) == code, over.keys()
    lib = _abi.load()
    assert lib.kda_check_prefill(None) == _abi.KDA_E_ARG
    a = kda.prefill_args(**ok)
    a.workspace = None
    assert lib.kda_check_prefill(a) == _abi.KDA_E_ARG
    a = kda.prefill_args(**ok)
    a.workspace += 8
    assert lib.kda_check_prefill(a) == _abi.KDA_E_UNALIGNED
    a = kda.prefill_args(**ok)
    a.query_start_loc = None
    assert lib.kda_check_prefill(a) == _abi.KDA_E_ARG
    a.batch = 0                      # nothing to do needs nothing
    assert lib.kda_check_prefill(a) == _abi.KDA_OK


def test_prefill_binding_refusals():
    ok = _cpu()
    with pytest.raises(ValueError, match="GPU"):
        kda.conv_prefill(**ok)
    with pytest.raises(ValueError, match="entries"):
        kda.check_prefill(**dict(ok, query_start_loc=torch.zeros(
            2, dtype=torch.int32)))
    with pytest.raises(ValueError):
        kda.prefill_workspace_size(10, 1, 2, 48, torch.bfloat16)
    with pytest.raises(ValueError):
        kda.prefill_workspace_size(-1, 1, 2, 64, torch.bfloat16)
    with pytest.raises(ValueError):       # work items of a launch past 2^32
        kda.prefill_workspace_size(1 << 24, 1, 32, 64, torch.bfloat16)
    with pytest.raises(ValueError):
        kda.prefill_workspace_size(1 << 20, 1 << 20, 32, 128, torch.bfloat16)
    with pytest.raises(ValueError):
        kda.prefill_workspace_size(10, 1, 2, 64, torch.float16)
    with pytest.raises(ValueError, match="conv_weight|conv_state"):
        kda.check_prefill_qkv(**ok)
    assert TORCH
