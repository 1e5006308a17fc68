"""Single-token decode of a KDA layer against the fp64 oracle: head dims,
dtypes, layouts, both gates, null slots, moved and in-place states, padded
rows, streams, graph replays, and a run of single tokens against one prompt;
and the refusals of its checks (CPU)."""
import numpy as np
import pytest
import torch

import linear_attention_speculative_amd as kda
from linear_attention_speculative_amd import _abi
from tests.layer_check import compare, f64, i32, make_layer, reference

DEV = "cuda"


def _run(kw, slots, final, accepted, **more):
    conv = "conv_state" in kw
    call = kda.conv_update_decode if conv else kda.decode_qkv
    args = dict(kw, state_indices=i32(slots, DEV),
                final_state_indices=None if final is None
                else i32(final, DEV), **more)
    if conv:
        args["num_accepted_tokens"] = None if accepted is None \
            else i32(accepted, DEV)
    call(**args)
    torch.cuda.synchronize()


def _expected(kw, slots, final, accepted, null=0):
    """The layer on one token per request: sources are the initial slots,
    the final slots receive; a null source writes only zeros."""
    N, B = kw["state"].shape[0], len(slots)
    slots = np.asarray(slots)
    fin = slots if final is None else np.asarray(final)
    live = (slots > null) & (slots < N)
    keep = live & (fin > null) & (fin < N)
    # requests that keep nothing run into a scratch slot of the oracle
    ref = dict(out=f64(kw["out"]), state=f64(kw["state"]), conv_state=None)
    dst = np.where(keep, fin, null)
    r = reference(kw, np.arange(B + 1), dst, slots, accepted, null)
    ref.update(r)
    for b in np.nonzero(live & ~keep)[0]:
        one = np.full(B, null)
        free = [s for s in range(null + 1, N) if s not in slots][0]
        one[b] = free
        ref["out"][b] = reference(kw, np.arange(B + 1), one, slots, accepted,
                                  null)["out"][b]
    return ref, sorted(set(fin[keep].tolist()))


CASES = [
    dict(B=1, H=2, D=128), dict(B=5, H=3, D=64, dim_first=False),
    dict(B=9, H=1, D=32, lb=-5.0), dict(B=17, H=5, D=16, act="f32"),
    dict(B=4, H=2, D=128, act="f32", conv=False),
    dict(B=4, H=2, D=64, conv=False, out="f32"),
    dict(B=6, H=2, D=128, weight="f32", out="f32", gentle=False),
    dict(B=3, H=4, D=16, lb=-5.0, row_pad=32, slot_pad=64),
    dict(B=40, H=7, D=128, lb=-5.0, dim_first=False),
]


@pytest.mark.gpu
@pytest.mark.parametrize("moved", [False, True])
@pytest.mark.parametrize("ci", range(len(CASES)))
def test_decode_matches_oracle(ci, moved):
    c = dict(CASES[ci])
    B, Q = c.pop("B"), 4
    rng = np.random.RandomState(ci)
    kw = make_layer(B, 2 * B + 4, Q=Q, seed=ci, **c)
    perm = 1 + rng.permutation(2 * B + 2)
    slots, final = perm[:B].copy(), perm[B:2 * B].copy() if moved else None
    if B > 3:                     # null, out-of-range and negative slots
        slots[1], slots[2] = 0, 10 ** 6
        if moved:
            final[0], final[3] = -5, 2 * B + 4
    acc = rng.randint(-1, Q + 3, size=B) if "conv_state" in kw else None
    ref, written = _expected(kw, slots, final, acc)
    _run(kw, slots, final, acc)
    compare(kw, ref, written)


@pytest.mark.gpu
def test_decode_without_tokens_does_nothing():
    kw = make_layer(0, 3, 2, 64, 4)
    before = kw["state"].clone()
    _run(kw, np.zeros(0, int), None, None)
    assert torch.equal(kw["state"], before)


@pytest.mark.gpu
def test_decode_on_its_own_stream_and_in_a_graph():
    """A captured step replayed with eager work in between equals eager
    steps; the call runs on the stream it is given."""
    B, H, D, Q = 3, 2, 64, 2
    slots = np.array([2, 1, 4])
    kw = make_layer(B, 6, H, D, Q, act="f32", seed=3)
    eager = {k: v.clone() if isinstance(v, torch.Tensor) else v
             for k, v in kw.items()}
    args = dict(kw, state_indices=i32(slots, DEV))
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    kda.conv_update_decode(stream=stream, **args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.conv_update_decode(**args)
    _run(eager, slots, None, None)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        _run(eager, slots, None, None)
        for name in ("out", "state", "conv_state"):
            assert torch.equal(kw[name], eager[name]), name
        torch.randn(1000, device=DEV).sum().item()


@pytest.mark.gpu
def test_many_single_tokens_equal_one_sequence():
    """Forty in-place decode steps of one request against the oracle over the
    whole sequence."""
    H, D, Q, L = 2, 64, 4, 40
    kw = make_layer(L, 4, H, D, Q, act="f32", seed=8)
    ref = reference(kw, [0, L], [2], [2])
    rows = {n: kw[n] for n in ("mixed_qkv", "raw_gate", "raw_beta", "out")}
    for t in range(L):
        step = dict(kw, **{n: v[t:t + 1] for n, v in rows.items()})
        _run(step, [2], None, [1])
    compare(kw, ref, [2])


@pytest.mark.gpu
def test_large_pool_offsets_pass_32_bits():
    """A slot whose element offset is past 2^31: the pool is a strided view of
    one buffer of 9 GB."""
    H, D, B = 1, 128, 2
    kw = make_layer(B, 2, H, D, 2, conv=False, act="f32", seed=4)
    stride = (1 << 30) + 4096
    flat = torch.zeros(2 * stride + H * D * D, device=DEV)
    pool = torch.as_strided(flat, (3, H, D, D), (stride, D * D, D, 1))
    pool[1], pool[2] = kw["state"][0], kw["state"][1]
    small = dict(kw, state=pool.contiguous())
    kw["state"] = pool
    ref = reference(small, [0, 1, 2], [1, 2], [1, 2])
    _run(kw, [1, 2], None, None)
    compare(dict(kw, state=pool.contiguous()), ref, [1, 2])


def _cpu(**over):
    kw = make_layer(3, 6, 2, 16, 4, act=over.pop("act", "f32"),
                    device="cpu", **over)
    kw["state_indices"] = torch.arange(3, dtype=torch.int32)
    return kw


def test_decode_checks():
    ok = _cpu()
    assert kda.check_decode(**ok) == _abi.KDA_OK
    bad = [
        (dict(state=ok["state"][:, :1]), _abi.KDA_E_SHAPE),
        (dict(state=ok["state"].double()), _abi.KDA_E_DTYPE),
        (dict(state=ok["state"].transpose(2, 3)), _abi.KDA_E_LAYOUT),
        (dict(state=ok["state"][:1].expand(6, -1, -1, -1)),
         _abi.KDA_E_LAYOUT),
        (dict(raw_gate=ok["raw_gate"].bfloat16()), _abi.KDA_E_DTYPE),
        (dict(raw_beta=ok["raw_beta"][:, :1]), _abi.KDA_E_SHAPE),
        (dict(out=ok["out"].half()), _abi.KDA_E_DTYPE),
        (dict(out=ok["out"][:1].expand(3, -1)), _abi.KDA_E_LAYOUT),
        (dict(conv_state=ok["conv_state"][:, :, :5]),
         _abi.KDA_E_UNSUPPORTED),
        (dict(conv_state=ok["conv_state"][:1].expand(6, -1, -1)),
         _abi.KDA_E_LAYOUT),
        (dict(conv_weight=ok["conv_weight"][:, :3]), _abi.KDA_E_SHAPE),
        (dict(spec_query_len=17), _abi.KDA_E_UNSUPPORTED),
        (dict(dt_bias=ok["dt_bias"][:, :8]), _abi.KDA_E_SHAPE),
        (dict(mixed_qkv=torch.zeros(3 * 96 + 1)[1:].view(3, 96)),
         _abi.KDA_E_UNALIGNED),
        (dict(state_indices=torch.arange(2, dtype=torch.int32)),
         _abi.KDA_E_SHAPE),
    ]
    for over, code in bad:
        assert kda.check_decode(**dict(ok, **over)) == code, over.keys()
    lib = _abi.load()
    assert lib.kda_check_decode(None) == _abi.KDA_E_ARG
    a = kda.decode_args(**ok)
    a.state_indices = None
    assert lib.kda_check_decode(a) == _abi.KDA_E_ARG
    a.batch = -1
    assert lib.kda_check_decode(a) == _abi.KDA_E_ARG
    a = kda.decode_args(**ok)               # work items of a launch past 2^32
    a.batch = (1 << 23) // 2
    for t in (a.mixed_qkv, a.raw_gate, a.raw_beta, a.out):
        t.shape[0] = a.batch
    assert lib.kda_check_decode(a) == _abi.KDA_E_CAPACITY


def test_decode_binding_refusals():
    ok = _cpu()
    with pytest.raises(ValueError, match="GPU"):
        kda.conv_update_decode(**ok)
    with pytest.raises(TypeError):
        kda.check_decode(**dict(ok, state_indices=torch.arange(3)))
    with pytest.raises(ValueError, match="entries"):
        kda.check_decode(**ok, final_state_indices=torch.zeros(
            2, dtype=torch.int32))
    plain = {k: v for k, v in ok.items() if not k.startswith("conv")
             and k != "spec_query_len"}
    assert kda.check_decode_qkv(**plain) == _abi.KDA_OK
    with pytest.raises(ValueError, match="conv_state"):
        kda.check_decode_qkv(**ok)
