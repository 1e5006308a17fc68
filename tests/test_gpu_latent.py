"""Latent attention over paged caches, and the write into them, against the
fp64 oracle: types, dims, heads, block sizes, ragged and empty windows, strided
rows, null blocks, cache places of other tokens that hold NaN, requests cut
over many workgroups, graphs and streams; and the refusals (CPU)."""
import numpy as np
import pytest
import torch

import linear_attention_speculative_amd as kda
import oracle
from linear_attention_speculative_amd import _abi
from tests.latent_check import ACT, bounds, f64, hold, ints, make

DEV = "cuda"


def run(kw, **more):
    T, H, W = kw["q"].shape
    R = kw["out"].shape[2]
    B = kw["query_start_loc"].numel() - 1
    work = torch.full((kda.latent_attention_workspace_size(
        T, B, H, R, W - R, kw["q"].dtype),), 255, dtype=torch.uint8,
        device=DEV)
    kda.latent_attention(workspace=work, **kw, **more)
    return work


def expect(kw):
    host = {k: f64(v) if v.is_floating_point() else ints(v)
            for k, v in kw.items() if isinstance(v, torch.Tensor)}
    return oracle.latent_attention(
        **host, softmax_scale=kw["softmax_scale"],
        null_block_id=kw["null_block_id"], latent_dim=kw["out"].shape[2])


def check(kw, ref, act):
    b_out, b_lse = bounds(ref, act, kw["q"].shape[2])
    hold(f64(kw["out"]), ref["out"], b_out, "out")
    hold(f64(kw["lse"]), ref["lse"], b_lse, "lse")


CASES = [
    # one token of one request, with and without computed ones
    dict(lens=[1], computed=[0], H=1, R=128, P=0, block=16, act="f32"),
    dict(lens=[1], computed=[37], H=32, R=512, P=64, block=16, act="bf16"),
    dict(lens=[1], computed=[700], H=33, R=512, P=64, block=7, act="bf16"),
    # ragged, empty requests in front, between and behind
    dict(lens=[0, 3, 0, 1, 4, 0], computed=[5, 0, 9, 31, 64, 2], H=6, R=128,
         P=64, block=5, act="f32"),
    dict(lens=[2, 0, 4, 1], computed=[95, 3, 128, 300], H=8, R=256, P=64,
         block=64, act="bf16"),
    # a block a token; blocks larger than a step
    dict(lens=[2, 1], computed=[600, 31], H=5, R=256, P=0, block=1,
         act="bf16"),
    dict(lens=[1, 2, 1], computed=[1, 700, 130], H=3, R=512, P=0, block=1000,
         act="f32"),
    # more rows than a workgroup's; a prompt in this form
    dict(lens=[70, 5], computed=[10, 0], H=3, R=512, P=64, block=16,
         act="bf16"),
    dict(lens=[40], computed=[33], H=7, R=512, P=64, block=32, act="f32"),
    dict(lens=[33, 64], computed=[0, 0], H=4, R=128, P=0, block=16,
         act="bf16"),
    dict(lens=[4] * 9, computed=list(range(28, 37)), H=16, R=256, P=64,
         block=16, act="f32"),
]


@pytest.mark.gpu
@pytest.mark.parametrize("ci", range(len(CASES)))
def test_latent_attention_matches_oracle(ci):
    kw = make(seed=ci, tail=2, **CASES[ci])
    ref = expect(kw)
    run(kw)
    torch.cuda.synchronize()
    check(kw, ref, CASES[ci]["act"])       # rows behind the last: as they were


@pytest.mark.gpu
@pytest.mark.parametrize("act,P", [("bf16", 64), ("f32", 0)])
def test_many_workgroups_share_requests(act, P):
    """Requests of several thousand tokens beside short ones: runs that start
    and end inside requests, row tiles joined from up to all workgroups."""
    kw = make([2, 1, 1, 3], [9000, 3, 2500, 6100], H=20, R=128, P=P, block=16,
              act=act, seed=5)
    ref = expect(kw)
    run(kw)
    torch.cuda.synchronize()
    check(kw, ref, act)


@pytest.mark.gpu
def test_more_requests_than_threads():
    B = 700
    rng = np.random.RandomState(3)
    kw = make(list(rng.randint(0, 3, size=B)), list(rng.randint(0, 40, size=B)),
              H=2, R=128, P=0, block=8, act="f32", seed=8)
    ref = expect(kw)
    run(kw)
    torch.cuda.synchronize()
    check(kw, ref, "f32")


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_strided_rows(act):
    kw = make([3, 1], [40, 70], H=5, R=256, P=64, block=16, act=act, seed=2,
              gap=1)
    wide = torch.full((kw["block_table"].shape[0], 40), -7, dtype=torch.int32,
                      device=DEV)
    n = kw["block_table"].shape[1]
    wide[:, :2 * n:2] = kw["block_table"]
    kw["block_table"] = wide[:, :2 * n:2]
    kw["lse"] = torch.full((5, kw["q"].shape[0]), 7.0, device=DEV).t()
    ref = expect(kw)
    run(kw)
    torch.cuda.synchronize()
    check(kw, ref, act)


@pytest.mark.gpu
def test_nothing_seen_and_null_blocks():
    """Null blocks, ids past the cache, rows outside the tables, tables
    narrower than the request; queries that see nothing get 0 and -inf."""
    kw = make([2, 1, 2, 1, 3], [60, 33, 20, 90, 0], H=4, R=128, P=64,
              block=16, act="bf16", seed=4, null=2)
    req = ints(kw["request_indices"])
    kw["block_table"][int(req[0]), 1] = 2               # null inside
    kw["block_table"][int(req[0]), 2] = 10 ** 6         # past the cache
    kw["block_table"][int(req[1])] = 0                  # nothing at all
    kw["request_indices"][2] = -1
    kw["request_indices"][4] = kw["block_table"].shape[0]
    kw["block_table"] = kw["block_table"][:, :5]        # 90 + 1 > 5 * 16
    ref = expect(kw)
    assert np.isinf(ref["lse"]).any() and np.isfinite(ref["lse"]).any()
    run(kw)
    torch.cuda.synchronize()
    check(kw, ref, "bf16")
    assert (kw["out"][2:3].float() == 0).all()


@pytest.mark.gpu
def test_large_scores():
    """Scores over several hundreds, rising and falling along the keys: the
    running maximum moves, most weights are nothing."""
    for act in ("bf16", "f32"):
        kw = make([2, 1], [200, 500], H=8, R=128, P=0, block=16, act=act,
                  seed=9)
        kw["softmax_scale"] = 20.0
        ref = expect(kw)
        run(kw)
        torch.cuda.synchronize()
        check(kw, ref, act)


@pytest.mark.gpu
def test_not_finite_entries_spoil_their_request_alone():
    kw = make([1, 1, 2], [50, 40, 90], H=4, R=128, P=64, block=16, act="bf16",
              seed=1)
    req, table = ints(kw["request_indices"]), ints(kw["block_table"])
    ref = expect(kw)
    kw["cache"][int(table[req[1], 1]), 3] = float("inf")
    run(kw)
    torch.cuda.synchronize()
    out = f64(kw["out"])
    assert not np.isfinite(out[1]).any()
    b_out, _ = bounds(ref, "bf16", 192)
    for t in (0, 2, 3):
        hold(out[t], ref["out"][t], b_out[t], "out")


@pytest.mark.gpu
@pytest.mark.parametrize("act,R", [("bf16", 512), ("bf16", 128), ("f32", 512),
                                   ("f32", 256)])
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
def test_not_finite_entries_of_later_tokens(act, R, value):
    """A window's tokens do not see the entries of those behind them."""
    lens, computed = [4, 3, 40], [50, 30, 90]
    kw = make(lens, computed, H=5, R=R, P=64, block=16, act=act, seed=2)
    ref = expect(kw)
    req, table = ints(kw["request_indices"]), ints(kw["block_table"])
    first = [2, 1, 11]                      # tokens of the windows
    for b in range(3):
        pos = computed[b] + first[b]
        at = kw["cache"][int(table[req[b], pos // 16]), pos % 16]
        at[3 + 40 * b] = value
        at[R - 1] = -value
    run(kw)
    torch.cuda.synchronize()
    b_out, b_lse = bounds(ref, act, R + 64)
    out, lse = f64(kw["out"]), f64(kw["lse"])
    start = ints(kw["query_start_loc"])
    for b in range(3):
        own = slice(start[b], start[b] + first[b])
        hold(out[own], ref["out"][own], b_out[own], "out")
        hold(lse[own], ref["lse"][own], b_lse[own], "lse")
        for t in range(start[b] + first[b], start[b + 1]):
            # (scores of +-inf, half of them NaN with a latent's second one)
            assert not np.isfinite(out[t]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [-0.05, 0.0, -3.0])
def test_scales_not_above_zero(act, scale):
    kw = make([2, 5], [70, 40], H=9, R=128, P=64, block=16, act=act, seed=5)
    kw["softmax_scale"] = scale
    ref = expect(kw)
    run(kw)
    torch.cuda.synchronize()
    check(kw, ref, act)


@pytest.mark.gpu
def test_graph_replays_and_other_stream():
    kw = make([2, 1, 4], [100, 900, 31], H=16, R=512, P=64, block=16,
              act="bf16", seed=6)
    lens = kw["num_computed_tokens"].clone()
    req = kw["request_indices"].long()
    work = run(kw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.latent_attention(workspace=work, **kw)
    for step in range(3):
        # (shorter contexts: their places are in the cache)
        kw["num_computed_tokens"][req] = (lens[req] - 17 * step).clamp(min=0)
        ref = expect(kw)
        kw["out"].fill_(3.0)
        graph.replay()
        torch.randn(1000, device=DEV).sum().item()
        check(kw, ref, "bf16")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    kw["out"].fill_(3.0)
    side.wait_stream(torch.cuda.current_stream())
    kda.latent_attention(workspace=work, stream=side, **kw)
    side.synchronize()
    check(kw, ref, "bf16")


@pytest.mark.gpu
def test_two_streams_at_once_and_same_bits():
    sets = [make([1, 3, 2], [500 + 64 * i, 90, 700], H=32, R=512, P=64,
                 block=16, act="bf16", seed=i) for i in range(2)]
    alone = []
    for kw in sets:
        run(kw)
        torch.cuda.synchronize()
        alone.append((kw["out"].clone(), kw["lse"].clone()))
        kw["out"].fill_(1.0)
    streams = [torch.cuda.Stream() for _ in sets]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    works = []
    for _ in range(3):
        for kw, s in zip(sets, streams):
            with torch.cuda.stream(s):
                works.append(run(kw, stream=s))
    torch.cuda.synchronize()
    for kw, (o, l) in zip(sets, alone):
        assert torch.equal(kw["out"], o) and torch.equal(kw["lse"], l)


@pytest.mark.gpu
def test_cache_past_32_bits():
    """A cache of over 4 GiB, its used blocks at its far end."""
    kw = make([1, 2], [70, 30], H=4, R=512, P=64, block=64, act="bf16",
              seed=3)
    N = kw["cache"].shape[0]
    big = torch.empty((60000, 64, 576), dtype=torch.bfloat16, device=DEV)
    far = 60000 - N
    big[far:] = kw["cache"]
    ref = expect(kw)
    kw["cache"] = big
    live = kw["block_table"] > 0
    kw["block_table"] += live.int() * far
    assert far * 64 * 576 * 2 > 1 << 32
    run(kw)
    torch.cuda.synchronize()
    check(kw, ref, "bf16")


@pytest.mark.gpu
@pytest.mark.parametrize("act,R,P", [("bf16", 512, 64), ("f32", 128, 0),
                                     ("bf16", 8, 16)])
def test_latent_write(act, R, P):
    g = torch.Generator().manual_seed(1)
    T, N, bs = 37, 9, 7
    dt = ACT[act]
    cache = torch.randn((N, bs, R + P + 16), generator=g).to(dt).to(DEV)
    wide = cache.clone()
    latent = torch.randn((T, R + 8), generator=g).to(dt).to(DEV)[:, :R]
    rope = torch.randn((T, P), generator=g).to(dt).to(DEV) if P else None
    rng = np.random.RandomState(0)
    slots = rng.permutation(N * bs)[:T + 4]
    slots[[3, 9]] = -1, N * bs + 2          # (the null block takes some, too)
    ref = oracle.latent_write(
        latent=f64(latent), rope_key=f64(rope) if P else None,
        cache=f64(cache)[..., :R + P], slot_mapping=slots, null_block_id=1)
    kda.latent_write(latent=latent, rope_key=rope, cache=cache[..., :R + P],
                     slot_mapping=torch.as_tensor(slots).to(DEV),
                     null_block_id=1)
    torch.cuda.synchronize()
    assert np.array_equal(f64(cache)[..., :R + P], ref)
    assert torch.equal(cache[..., R + P:], wide[..., R + P:])


@pytest.mark.gpu
def test_latent_write_null_blocks_past_32_bits_of_slots():
    cache = torch.zeros((3, 16, 128), device=DEV)
    kda.latent_write(latent=torch.ones((40, 128), device=DEV), cache=cache,
                     slot_mapping=torch.arange(40, device=DEV),
                     null_block_id=(1 << 28) - 1)   # slots below 2^32
    torch.cuda.synchronize()
    assert (cache == 0).all()


@pytest.mark.gpu
def test_empty_calls_launch_nothing():
    kw = make([1], [3], H=2, R=128, P=0, block=4, act="f32")
    kw["q"], kw["out"], kw["lse"] = (kw[n][:0] for n in ("q", "out", "lse"))
    kda.latent_attention(workspace=torch.empty(0, dtype=torch.uint8,
                                               device=DEV), **kw)
    kda.latent_write(latent=kw["q"][:, 0], cache=kw["cache"],
                     slot_mapping=torch.zeros(0, dtype=torch.int64,
                                              device=DEV))
    torch.cuda.synchronize()


def test_refusals():
    ok = make([1, 2], [3, 9], H=4, R=128, P=64, block=4, act="bf16",
              device="cpu")
    ok["workspace"] = torch.empty(kda.latent_attention_workspace_size(
        3, 2, 4, 128, 64, torch.bfloat16), dtype=torch.uint8)
    chk = lambda **d: kda.check_latent_attention(**dict(ok, **d))  # noqa: E731
    assert chk() == _abi.KDA_OK
    assert chk(lse=None) == _abi.KDA_OK
    with pytest.raises(ValueError, match="GPU"):
        kda.latent_attention(**ok)
    assert chk(q=ok["q"].float()) == _abi.KDA_E_DTYPE
    assert chk(q=ok["q"].half()) == _abi.KDA_E_DTYPE
    assert chk(out=ok["out"][:2]) == _abi.KDA_E_SHAPE
    assert chk(out=ok["out"][..., :64]) == _abi.KDA_E_UNSUPPORTED
    assert chk(cache=ok["cache"][..., :128]) == _abi.KDA_E_SHAPE
    assert chk(out=ok["out"][:1].expand(3, -1, -1)) == _abi.KDA_E_LAYOUT
    wide = torch.zeros((3, 4, 196), dtype=torch.bfloat16)
    assert chk(q=wide[..., 4:]) == _abi.KDA_E_UNALIGNED
    assert chk(q=wide[..., :192]) == _abi.KDA_E_UNALIGNED
    assert chk(lse=ok["lse"].double()) == _abi.KDA_E_DTYPE
    assert chk(lse=ok["lse"][:1].expand(3, 4)) == _abi.KDA_E_LAYOUT
    assert chk(workspace=ok["workspace"][:-1]) == _abi.KDA_E_CAPACITY
    for scale in (float("inf"), float("nan"), -3.4e38):
        assert chk(softmax_scale=scale) == _abi.KDA_E_ARG
    assert chk(null_block_id=-1) == _abi.KDA_E_ARG
    with pytest.raises(ValueError, match="row per request"):
        chk(request_indices=None, block_table=ok["block_table"][:1])
    with pytest.raises(ValueError, match="entries"):
        chk(num_computed_tokens=ok["num_computed_tokens"][:2])
    with pytest.raises(ValueError, match="two-dimensional"):
        chk(block_table=ok["block_table"].long())
    with pytest.raises(ValueError):
        kda.latent_attention_workspace_size(3, 2, 4, 96, 64, torch.bfloat16)
    lib = _abi.load()
    assert lib.kda_check_latent_attention(None) == _abi.KDA_E_ARG
    for name, value in (("query_start_loc", None),
                        ("num_computed_tokens", None), ("workspace", None),
                        ("block_table", None), ("batch", -1)):
        a = kda.latent_args(**ok)
        setattr(a, name, value)
        assert lib.kda_check_latent_attention(a) == _abi.KDA_E_ARG, name


def test_write_refusals():
    ok = dict(latent=torch.zeros(3, 128), rope_key=torch.zeros(3, 64),
              cache=torch.zeros(4, 5, 192),
              slot_mapping=torch.arange(3))
    chk = lambda **d: kda.check_latent_write(**dict(ok, **d))  # noqa: E731
    assert chk() == _abi.KDA_OK
    with pytest.raises(ValueError, match="GPU"):
        kda.latent_write(**ok)
    assert chk(rope_key=None) == _abi.KDA_E_SHAPE
    assert chk(rope_key=ok["rope_key"][:2]) == _abi.KDA_E_SHAPE
    assert chk(latent=ok["latent"].bfloat16()) == _abi.KDA_E_DTYPE
    assert chk(cache=ok["cache"][:, :1].expand(4, 5, 192)) == \
        _abi.KDA_E_LAYOUT
    assert chk(cache=torch.zeros(4, 5, 194)[..., :192]) == \
        _abi.KDA_E_UNALIGNED
    assert chk(latent=torch.zeros(3, 130), rope_key=torch.zeros(3, 62)) == \
        _abi.KDA_E_UNSUPPORTED
    assert chk(null_block_id=-1) == _abi.KDA_E_ARG
    with pytest.raises(TypeError):
        chk(slot_mapping=ok["slot_mapping"].int())
    with pytest.raises(ValueError):
        chk(slot_mapping=ok["slot_mapping"][:2])
    assert _abi.load().kda_check_latent_write(None) == _abi.KDA_E_ARG
