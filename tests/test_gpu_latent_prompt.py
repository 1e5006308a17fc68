"""The expanded form of latent attention: keys and values from cached latents,
and causal attention over prompts, against the fp64 oracle: types, dims,
ragged and empty requests, pieces behind computed tokens, more queries than
keys, strided rows, graphs; and the refusals (CPU)."""
import numpy as np
import pytest
import torch

import linear_attention_speculative_amd as kda
import oracle
from linear_attention_speculative_amd import _abi
from tests.latent_check import ACT, bounds, f64, hold, ints, paged

DEV = "cuda"
I32 = torch.int32


def randn(shape, g, dt, device=DEV, gap=0):
    if not gap:
        return torch.randn(shape, generator=g).to(dt).to(device)
    wide = torch.randn(*shape[:-2], shape[-2] + 1, shape[-1] + 8 * gap,
                       generator=g).to(dt).to(device)
    return wide[..., :shape[-2], :shape[-1]]


def starts(lens, device=DEV):
    return torch.as_tensor(np.concatenate([[0], np.cumsum(lens)]),
                           dtype=I32).to(device)


def prompt(q, k, *, H, D, P, act, seed=0, tail=0, device=DEV, gap=0):
    g = torch.Generator().manual_seed(seed)
    dt, T, S = ACT[act], sum(q) + tail, sum(k) + tail
    kw = dict(q=randn((T, H, D + P), g, dt, device, gap),
              key=randn((S, H, D), g, dt, device, gap),
              value=randn((S, H, D), g, dt, device, gap),
              out=randn((T, H, D), g, dt, device, gap),
              lse=torch.full((T, H), 7.0, device=device),
              query_start_loc=starts(q, device),
              key_start_loc=starts(k, device), softmax_scale=(D + P) ** -0.5)
    if P:
        kw["rope_key"] = randn((S, P), g, dt, device)
    return kw


def expect(kw):
    host = {k: f64(v) if v.is_floating_point() else ints(v)
            for k, v in kw.items() if isinstance(v, torch.Tensor)}
    return oracle.latent_prefill(**host, softmax_scale=kw["softmax_scale"])


def check(kw, ref, act):
    b_out, b_lse = bounds(ref, act, kw["q"].shape[2])
    hold(f64(kw["out"]), ref["out"], b_out, "out")
    hold(f64(kw["lse"]), ref["lse"], b_lse, "lse")


CASES = [
    dict(q=[1], k=[1], H=1, D=64, P=0, act="f32"),
    dict(q=[300], k=[300], H=3, D=128, P=64, act="bf16"),
    # ragged, empty, behind computed tokens; odd heads
    dict(q=[5, 0, 33, 257, 1], k=[5, 7, 97, 600, 64], H=5, D=128, P=64,
         act="bf16"),
    dict(q=[31, 64, 65, 0], k=[31, 200, 65, 0], H=8, D=64, P=64, act="bf16"),
    dict(q=[256, 255], k=[256, 511], H=2, D=128, P=0, act="bf16"),
    dict(q=[513], k=[513], H=1, D=64, P=0, act="bf16"),
    # fewer keys than queries: the first see nothing
    dict(q=[70, 10, 4], k=[30, 0, 4], H=3, D=128, P=64, act="bf16"),
    dict(q=[90, 3], k=[150, 2], H=3, D=128, P=64, act="f32"),
    dict(q=[260], k=[300], H=2, D=64, P=64, act="f32"),
    dict(q=[40, 1, 100], k=[41, 70, 100], H=9, D=128, P=0, act="f32"),
]


@pytest.mark.gpu
@pytest.mark.parametrize("ci", range(len(CASES)))
def test_prefill_matches_oracle(ci):
    kw = prompt(seed=ci, tail=3, **CASES[ci])
    ref = expect(kw)
    kda.latent_prefill(**kw)
    torch.cuda.synchronize()
    check(kw, ref, CASES[ci]["act"])       # rows behind the last: as they were


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_strided_rows_and_large_scores(act):
    kw = prompt([100, 30], [100, 90], H=3, D=128, P=64, act=act, gap=1,
                seed=4)
    kw["softmax_scale"] = 8.0
    kw["lse"] = torch.full((3, 130), 7.0, device=DEV).t()
    ref = expect(kw)
    kda.latent_prefill(**kw)
    torch.cuda.synchronize()
    check(kw, ref, act)


@pytest.mark.gpu
def test_more_requests_than_threads():
    rng = np.random.RandomState(2)
    q = list(rng.randint(0, 5, size=1100))
    k = [n + int(e) for n, e in zip(q, rng.randint(0, 9, size=1100))]
    kw = prompt(q, k, H=2, D=64, P=0, act="bf16", seed=7)
    ref = expect(kw)
    kda.latent_prefill(**kw)
    torch.cuda.synchronize()
    check(kw, ref, "bf16")


@pytest.mark.gpu
def test_values_behind_the_last_key_are_not_read_into_sums():
    """NaN in the rows of another request, in the same step of keys."""
    kw = prompt([10, 20], [10, 20], H=2, D=128, P=64, act="bf16", seed=3)
    ref = expect(kw)
    for n in ("key", "value", "rope_key"):
        kw[n][10:] = float("nan")
    kda.latent_prefill(**kw)
    torch.cuda.synchronize()
    b_out, _ = bounds(ref, "bf16", 192)
    hold(f64(kw["out"])[:10], ref["out"][:10], b_out[:10], "out")
    assert torch.isnan(kw["out"][10:].float()).all()


@pytest.mark.gpu
@pytest.mark.parametrize("act,D", [("bf16", 128), ("bf16", 64), ("f32", 128),
                                   ("f32", 64)])
def test_not_finite_keys_and_values_of_later_tokens(act, D):
    """They reach the queries that see them: of a value its own dimension."""
    n, ahead = 150, 23
    kw = prompt([n, 40], [n + ahead, 40], H=2, D=D, P=64, act=act, seed=8)
    ref = expect(kw)
    want = ref["out"]
    inf, nan = float("inf"), float("nan")
    for tok, dim, v in ((20, 3, inf), (41, 33, -inf), (97, 60, nan),
                        (45, 5, inf), (120, 5, -inf), (149, 9, -inf)):
        kw["value"][ahead + tok, 1, dim] = v
        with np.errstate(invalid="ignore"):
            want[tok:n, 1, dim] += v
    kw["key"][ahead + 140, 0, 7] = nan
    want[140:n, 0] = nan
    ref["lse"][140:n, 0] = nan
    kda.latent_prefill(**kw)
    torch.cuda.synchronize()
    check(kw, ref, act)


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [-0.05, 0.0, -2.0])
def test_scales_not_above_zero(act, scale):
    kw = prompt([70, 33], [100, 33], H=2, D=64, P=64, act=act, seed=6)
    kw["softmax_scale"] = scale
    ref = expect(kw)
    kda.latent_prefill(**kw)
    torch.cuda.synchronize()
    check(kw, ref, act)


@pytest.mark.gpu
def test_prefill_graph_replays_over_other_lengths():
    kw = prompt([200, 100], [250, 100], H=4, D=128, P=64, act="bf16", seed=5)
    kda.latent_prefill(**kw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.latent_prefill(**kw)
    for cut in (200, 90, 290):
        kw["query_start_loc"][1] = cut
        kw["key_start_loc"][1] = cut + 50
        ref = expect(kw)
        kw["out"].fill_(2.0)
        graph.replay()
        torch.randn(1000, device=DEV).sum().item()
        check(kw, ref, "bf16")


def expansion(lens, *, H, D, R, P, block, act, seed=0, tail=0, rope=True,
              device=DEV, gap=0, null=0):
    kw, N = paged([0] * len(lens), lens, block=block, seed=seed, null=null,
                  device=device)
    del kw["num_computed_tokens"], kw["query_start_loc"]
    g = torch.Generator().manual_seed(seed)
    dt, S = ACT[act], sum(lens) + tail
    kw.update(cache=randn((N, block, R + P), g, dt, device, gap),
              weight=(randn((H, 2 * D, R), g, torch.float32, device)
                      * R ** -0.5).to(dt),
              key=randn((S, H, D), g, dt, device, gap),
              value=randn((S, H, D), g, dt, device, gap),
              key_start_loc=starts(lens, device), null_block_id=null)
    if rope and P:
        kw["rope_key"] = randn((S, P), g, dt, device)
    return kw


def expand_expect(kw):
    host = {k: f64(v) if v.is_floating_point() else ints(v)
            for k, v in kw.items() if isinstance(v, torch.Tensor)}
    host.setdefault("rope_key", None)
    return oracle.latent_expand(**host, null_block_id=kw["null_block_id"])


def expand_check(kw, ref, act):
    """fp32 sums of R products, rounded once."""
    u, half = 2.0 ** -24, 2.0 ** -8 if act == "bf16" else 2.0 ** -24
    R = kw["weight"].shape[2]
    for n in ("key", "value"):
        off = R * u * ref[n + "_size"]
        hold(f64(kw[n]), ref[n], off + half * (np.abs(ref[n]) + off), n)
    if "rope_key" in kw:
        assert np.array_equal(f64(kw["rope_key"]), ref["rope_key"])


EXPAND = [
    dict(lens=[1], H=1, D=64, R=128, P=0, block=16, act="f32"),
    dict(lens=[130, 0, 5, 260], H=3, D=128, R=512, P=64, block=16,
         act="bf16"),
    dict(lens=[127, 1, 300], H=5, D=64, R=256, P=64, block=7, act="bf16"),
    dict(lens=[50, 200], H=2, D=128, R=128, P=8, block=1, act="bf16"),
    dict(lens=[128, 20], H=3, D=64, R=512, P=64, block=100, act="f32"),
    dict(lens=[40], H=2, D=128, R=128, P=64, block=16, act="f32",
         rope=False),
    # groups of tokens and tiles of W shared by workgroups
    dict(lens=[700, 1, 900], H=9, D=64, R=128, P=64, block=16, act="bf16"),
    dict(lens=[520], H=33, D=128, R=256, P=0, block=32, act="bf16"),
    dict(lens=[300, 230], H=2, D=64, R=512, P=64, block=16, act="bf16"),
]


@pytest.mark.gpu
@pytest.mark.parametrize("gap", [0, 1])
@pytest.mark.parametrize("ci", range(len(EXPAND)))
def test_expand_matches_oracle(ci, gap):
    kw = expansion(seed=ci, tail=2, gap=gap, **EXPAND[ci])
    ref = expand_expect(kw)
    kda.latent_expand(**kw)
    torch.cuda.synchronize()
    expand_check(kw, ref, EXPAND[ci]["act"])


@pytest.mark.gpu
def test_expand_null_blocks_and_rows_outside():
    kw = expansion([60, 40, 50], H=2, D=64, R=128, P=64, block=16, act="bf16",
                   seed=2, null=1)
    req = ints(kw["request_indices"])
    kw["block_table"][int(req[0]), 1] = 1
    kw["block_table"][int(req[0]), 2] = 10 ** 6
    kw["request_indices"][1] = -3
    kw["block_table"] = kw["block_table"][:, :3]
    ref = expand_expect(kw)
    assert (ref["key"][16:48] == 0).all()
    kda.latent_expand(**kw)
    torch.cuda.synchronize()
    expand_check(kw, ref, "bf16")


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_expand_offsets_in_front_of_the_first_row(act):
    """They are clamped: the first row is the request's position 0."""
    kw = expansion([40, 30], H=2, D=64, R=128, P=64, block=16, act=act,
                   seed=9)
    ref = expand_expect(kw)
    kw["key_start_loc"][0] = -5
    kda.latent_expand(**kw)
    torch.cuda.synchronize()
    expand_check(kw, ref, act)


def test_prefill_refusals():
    ok = prompt([3, 4], [5, 4], H=2, D=64, P=64, act="bf16", device="cpu")
    chk = lambda **d: kda.check_latent_prefill(**dict(ok, **d))  # noqa: E731
    assert chk() == _abi.KDA_OK
    assert chk(lse=None) == _abi.KDA_OK
    with pytest.raises(ValueError, match="GPU"):
        kda.latent_prefill(**ok)
    assert chk(rope_key=None) == _abi.KDA_E_SHAPE
    assert chk(rope_key=ok["rope_key"][:3]) == _abi.KDA_E_SHAPE
    assert chk(q=ok["q"][..., :96]) == _abi.KDA_E_SHAPE
    assert chk(q=ok["q"].float()) == _abi.KDA_E_DTYPE
    assert chk(value=ok["value"].float()) == _abi.KDA_E_DTYPE
    assert chk(out=ok["out"][:1].expand(7, -1, -1)) == _abi.KDA_E_LAYOUT
    assert chk(key=ok["key"][..., :32], value=ok["value"][..., :32],
               out=ok["out"][..., :32]) == _abi.KDA_E_UNSUPPORTED
    for scale in (float("inf"), float("nan"), -3.4e38):
        assert chk(softmax_scale=scale) == _abi.KDA_E_ARG
    wide = torch.zeros((9, 2, 66), dtype=torch.bfloat16)
    assert chk(key=wide[..., :64]) == _abi.KDA_E_UNALIGNED
    with pytest.raises(ValueError, match="entries"):
        chk(key_start_loc=ok["key_start_loc"][:2])
    lib = _abi.load()
    assert lib.kda_check_latent_prefill(None) == _abi.KDA_E_ARG
    for name, value in (("query_start_loc", None), ("key_start_loc", None),
                        ("batch", -1)):
        a = kda.latent_prefill_args(**ok)
        setattr(a, name, value)
        assert lib.kda_check_latent_prefill(a) == _abi.KDA_E_ARG, name


def test_expand_refusals():
    ok = expansion([3, 9], H=2, D=64, R=128, P=64, block=4, act="bf16",
                   device="cpu")
    chk = lambda **d: kda.check_latent_expand(**dict(ok, **d))  # noqa: E731
    assert chk() == _abi.KDA_OK
    assert chk(rope_key=None) == _abi.KDA_OK
    with pytest.raises(ValueError, match="GPU"):
        kda.latent_expand(**ok)
    assert chk(weight=ok["weight"][:1]) == _abi.KDA_E_SHAPE
    assert chk(weight=ok["weight"].float()) == _abi.KDA_E_DTYPE
    assert chk(weight=ok["weight"][..., :96]) == _abi.KDA_E_SHAPE
    assert chk(rope_key=None, weight=ok["weight"][..., :96]) == \
        _abi.KDA_E_UNSUPPORTED
    assert chk(key=ok["key"][:1].expand(12, -1, -1)) == _abi.KDA_E_LAYOUT
    assert chk(value=ok["value"][:5]) == _abi.KDA_E_SHAPE
    assert chk(null_block_id=-1) == _abi.KDA_E_ARG
    with pytest.raises(ValueError, match="row per request"):
        chk(request_indices=None, block_table=ok["block_table"][:1])
    lib = _abi.load()
    assert lib.kda_check_latent_expand(None) == _abi.KDA_E_ARG
    for name in ("key_start_loc", "block_table"):
        a = kda.latent_expand_args(**ok)
        setattr(a, name, None)
        assert lib.kda_check_latent_expand(a) == _abi.KDA_E_ARG, name
