"""Sampling and draft acceptance against the row-by-row oracle: every filter
alone and together, vocabularies around the groups and the list's size, ties,
masked and non-finite logits, rows with nothing left, strides, the paths for
few and for very many kept logits, windows of ragged lengths, graph replays;
and the refusals (CPU)."""
import numpy as np
import pytest
import torch

import linear_attention_speculative_amd as kda
import oracle
from linear_attention_speculative_amd import _abi
from tests.layer_check import TORCH, f64, i32

DEV = "cuda"


def f32(a, device=DEV):
    return torch.as_tensor(np.asarray(a, np.float32)).to(device)


def run(x, u, T=None, k=None, p=None, mp=None, qsl=None, draft=None, **more):
    M, V = x.shape
    B = M if qsl is None else len(qsl) - 1
    out = dict(tokens=torch.full((M,), -9, dtype=torch.int32, device=DEV))
    if draft is not None:
        out.update(num_accepted=i32(np.full(B, -9), DEV),
                   next_tokens=i32(np.full(B, -9), DEV))
    args = dict(
        logits=x, uniform=f32(u),
        temperature=None if T is None else f32(T),
        top_k=None if k is None else i32(k, DEV),
        top_p=None if p is None else f32(p),
        min_p=None if mp is None else f32(mp),
        query_start_loc=None if qsl is None else i32(qsl, DEV),
        draft_tokens=None if draft is None else i32(draft, DEV),
        workspace=torch.full((kda.sample_workspace_size(M, V),), 0xff,
                             dtype=torch.uint8, device=DEV), **out, **more)
    kda.sample(**args)
    torch.cuda.synchronize()
    return {n: v.cpu().numpy() for n, v in out.items()}


def expect(x, u, T=None, k=None, p=None, mp=None):
    """The oracle on every row; parameters as float32 holds them."""
    h = f64(x)
    at = lambda a, m, d: d if a is None else float(np.float32(a[m]))  # noqa: E731
    return np.array([
        oracle.sample_row(h[m], float(np.float32(u[m])), at(T, m, 1.0),
                          0 if k is None else int(k[m]), at(p, m, 1.0),
                          at(mp, m, 0.0)) for m in range(len(h))])


def logits(M, V, act="f32", seed=0, std=2.0, pad=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((M, V + pad), generator=g) * std
    return x.to(TORCH[act]).to(DEV)[:, :V]


SIZES = [1, 2, 63, 64, 511, 512, 513, 1000, 4097, 20000]


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("V", SIZES)
def test_filters_match_oracle(V, act):
    """Every combination of filters on rows of their own."""
    rng = np.random.RandomState(V)
    rows = [(T, k, p, mp) for T in (0.0, 0.7, 1.5) for k in (0, 1, 5, 700)
            for p in (1.0, 0.9, 0.3) for mp in (0.0, 0.2)]
    M = len(rows)
    T, k, p, mp = (np.array(c) for c in zip(*rows))
    x = logits(M, V, act, seed=V, pad=5 if V % 2 else 0)
    u = rng.rand(M)
    got = run(x, u, T, k, p, mp)["tokens"]
    want = expect(x, u, T, k, p, mp)
    assert np.array_equal(got, want), np.nonzero(got != want)


@pytest.mark.gpu
@pytest.mark.parametrize("p", [None, 0.999, 0.5])
@pytest.mark.parametrize("k", [None, 6000, 19999])
def test_more_kept_than_the_list_holds(k, p):
    """Flat rows: thousands are kept, the thresholds come from the radix
    search."""
    M, V = 6, 20000
    x = logits(M, V, "f32", seed=3, std=0.3)
    x[3:] = x[3:].bfloat16().float()              # with ties
    u = np.linspace(0, 0.999, M)
    ks = None if k is None else np.full(M, k)
    ps = None if p is None else np.full(M, p)
    mp = np.array([0.0, 0.1, 0.3] * 2)
    for mins in (None, mp):
        got = run(x, u, None, ks, ps, mins)["tokens"]
        want = expect(x, u, None, ks, ps, mins)
        assert np.array_equal(got, want)


@pytest.mark.gpu
def test_ties_go_to_the_lowest_index():
    """All logits equal: the kept prefix is the first indexes, exactly."""
    V = 9000
    x = torch.zeros((5, V), device=DEV)
    u = np.array([0.0, 0.5, 0.999, 0.25, 0.75])
    k = np.array([1, 10, 8000, 0, 4])
    p = np.array([1.0, 1.0, 1.0, 0.5, 0.5])
    got = run(x, u, None, k, p)["tokens"]
    assert np.array_equal(got, expect(x, u, None, k, p))
    assert got.tolist() == [0, 5, 7992, 1125, 1]


@pytest.mark.gpu
def test_masked_and_non_finite_logits():
    """-inf, the type's lowest value, NaN and +inf among the logits; a row
    with nothing left."""
    V = 1500
    x = logits(8, V, "f32", seed=5)
    low = torch.finfo(torch.float32).min
    x[0, ::2] = -float("inf")
    x[1, 1:] = low
    x[2] = -float("inf")
    x[3, 5::3] = float("nan")
    x[4, 77] = x[4, 900] = float("inf")
    x[5] = float("nan")
    x[6] = low
    x[7] = -float("inf")
    x[7, 1499] = low
    u = np.array([0.3, 0.9, 0.5, 0.8, 0.7, 0.1, 0.6, 0.2])
    for T in (0.0, 1.0):
        for k, p, mp in ((0, 1.0, 0.0), (3, 1.0, 0.0), (0, 0.9, 0.0),
                         (50, 0.9, 0.05)):
            full = [np.full(8, v) for v in (T, k, p, mp)]
            got = run(x, u, *full)["tokens"]
            want = expect(x, u, *full)
            assert np.array_equal(got, want), (T, k, p, mp)
            assert got[2] == got[5] == -1 and got[7] == 1499


@pytest.mark.gpu
def test_odd_parameters():
    """NaN parameters, negative ones, infinite and tiny temperatures, u at
    and outside its bounds."""
    nan, inf = float("nan"), float("inf")
    T = np.array([nan, inf, 1e-30, -1.0, 1.0, 1.0, 1.0, 1.0, 1.0])
    k = np.array([0, 3, 0, 5, -4, 2000, 0, 0, 0])
    p = np.array([1.0, 1.0, 1.0, 1.0, nan, 2.0, 0.0, -1.0, 1.0])
    mp = np.array([0.0, 0.0, 0.0, 0.0, nan, -1.0, 0.0, 0.0, 7.0])
    u = np.array([0.4, 0.9, 0.9, 0.9, 1.5, -2.0, 0.5, 0.5, 0.99])
    x = logits(9, 800, seed=8)
    got = run(x, u, T, k, p, mp)["tokens"]
    want = expect(x, np.minimum(u, 1 - 2.0 ** -24), T, k, p, np.where(
        np.isnan(mp), 0, mp))
    assert np.array_equal(got, want)


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_windows_and_acceptance(act):
    """Ragged windows (one empty), parameters by request, drafts that match
    for a while; rows outside the requests stay as they were."""
    qsl = np.array([2, 6, 6, 7, 11, 12])
    M, V, B = 15, 3000, 5
    rng = np.random.RandomState(2)
    x = logits(M, V, act, seed=9)
    T = np.array([0.0, 1.0, 0.8, 1.0, 0.0])
    k, p = np.array([0, 4, 20, 3, 0]), np.array([1, 0.5, 0.9, 1.0, 1.0])
    u = rng.rand(M)
    req = np.searchsorted(qsl[1:], np.arange(M), side="right").clip(0, B - 1)
    want = expect(x, u, T[req], k[req], p[req])
    inside = (np.arange(M) >= qsl[0]) & (np.arange(M) < qsl[-1])
    want = np.where(inside, want, -9)
    draft = np.roll(want, 1)
    draft[5] += 1                         # the first window fails at its end
    draft[9] = -1
    got = run(x, u, T, k, p, qsl=qsl, draft=draft)
    assert np.array_equal(got["tokens"], want)
    acc, nxt = oracle.accept_drafts(want, draft, qsl)
    assert np.array_equal(got["num_accepted"], acc)
    assert np.array_equal(got["next_tokens"], nxt)
    assert acc.tolist() == [3, 0, 1, 2, 1]


@pytest.mark.gpu
def test_large_vocabulary_and_many_requests():
    V = 1 << 20
    x = logits(2, V, "bf16", seed=1)
    u = np.array([0.37, 0.81])
    k, p = np.array([0, 3000]), np.array([0.6, 1.0])
    got = run(x, u, None, k, p)["tokens"]
    assert np.array_equal(got, expect(x, u, None, k, p))
    B = 5000                              # the request search, two levels
    qsl = np.arange(B + 1)
    x = logits(B, 40, seed=2)
    u = np.random.RandomState(0).rand(B)
    T = np.random.RandomState(1).choice([0.0, 1.0], size=B)
    assert np.array_equal(run(x, u, T, qsl=qsl)["tokens"], expect(x, u, T))


@pytest.mark.gpu
@pytest.mark.parametrize("k", [1, 3, 4, 5, 60, 700, 2500])
@pytest.mark.parametrize("mp", [0.0, 1e-9, 0.3])
def test_few_groups_hold_logits(k, mp):
    """A masked vocabulary (as a grammar leaves it): only some stretches hold
    logits above -inf, more or fewer than k of them."""
    V = 20000
    rows = []
    for seed, spans in enumerate([[(7000, 7003)], [(0, 40), (9000, 9100)],
                                  [(100, 2000)], [(i, i + 1) for i in
                                                  range(5, V, 600)],
                                  [(512, 6200), (19999, 20000)]]):
        x = logits(1, V, seed=40 + seed)[0].cpu()
        keep = torch.zeros(V, dtype=torch.bool)
        for s, e in spans:
            keep[s:e] = True
        rows.append(torch.where(keep, x, torch.tensor(-float("inf"))))
    x = torch.stack(rows).to(DEV)
    M = len(rows)
    u = np.linspace(0.05, 0.95, M)
    for p in (1.0, 0.7):
        full = [np.full(M, v) for v in (0.9, k, p, mp)]
        got = run(x, u, *full)["tokens"]
        assert np.array_equal(got, expect(x, u, *full)), p


@pytest.mark.gpu
def test_counts_that_end_before_k():
    """Every group's maximum far above its other logits: the counted bins hold
    fewer than k, and the rest lies behind them."""
    V, M = 131072, 4
    x = logits(M, V, seed=50) - 60.0
    x[:, ::512] = 10.0 + logits(M, V // 512, seed=51, std=0.1)
    u = np.array([0.1, 0.5, 0.9, 0.999])
    k = np.array([900, 1000, 257, 300])
    for T, mp in ((1.0, None), (30.0, None), (30.0, np.full(M, 0.05))):
        full = [np.full(M, T), k, np.full(M, 0.99), mp]
        got = run(x, u, *full)["tokens"]
        assert np.array_equal(got, expect(x, u, *full)), T


@pytest.mark.gpu
def test_top_k_among_two_thousand_groups():
    """The k-th of up to 2048 group maxima, and k just past them."""
    V, M = 1 << 20, 5
    x = logits(M, V, "bf16", seed=52)
    u = np.array([0.2, 0.4, 0.6, 0.8, 0.95])
    k = np.array([2, 64, 1500, 2048, 2049])
    got = run(x, u, None, k)["tokens"]
    assert np.array_equal(got, expect(x, u, None, k))


@pytest.mark.gpu
def test_many_rows_share_the_sums_differently():
    """From 128 rows on a workgroup takes more groups: the same tokens."""
    V, M = 9000, 130
    x = logits(M, V, seed=53)
    rng = np.random.RandomState(5)
    u, T = rng.rand(M), rng.choice([0.7, 1.0], size=M)
    k = rng.choice([0, 30, 400], size=M)
    p, mp = rng.choice([1.0, 0.8], size=M), rng.choice([0.0, 0.05], size=M)
    got = run(x, u, T, k, p, mp)["tokens"]
    assert np.array_equal(got, expect(x, u, T, k, p, mp))
    few = run(x[:5], u[:5], T[:5], k[:5], p[:5], mp[:5])["tokens"]
    assert np.array_equal(few, got[:5])


@pytest.mark.gpu
def test_backward_offsets_stay_inside():
    """Offsets that run backwards: nothing outside the outputs is touched, no
    token leaves the vocabulary."""
    x = logits(12, 3000, seed=54)
    out = run(x, np.full(12, 0.5), np.full(4, 1.0), np.array([0, 5, 300, 40]),
              np.array([0.9, 1.0, 0.9, 1.0]), None, qsl=[8, 3, 20, 5, 10],
              draft=np.zeros(12))
    assert np.all((out["tokens"] == -9) |
                  ((out["tokens"] >= 0) & (out["tokens"] < 3000)))


@pytest.mark.gpu
def test_no_rows():
    got = run(torch.zeros((0, 50), device=DEV), np.zeros(0))
    assert got["tokens"].size == 0


@pytest.mark.gpu
def test_graph_replays():
    M, V = 8, 5000
    x = logits(M, V, seed=4)
    u = torch.rand(M, device=DEV)
    tokens = torch.zeros(M, dtype=torch.int32, device=DEV)
    args = dict(logits=x, uniform=u, tokens=tokens,
                top_k=i32([50] * 4 + [0] * 4, DEV), top_p=f32([0.9] * M),
                workspace=torch.empty(kda.sample_workspace_size(M, V),
                                      dtype=torch.uint8, device=DEV))
    kda.sample(**args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.sample(**args)
    for i in range(3):
        x.copy_(torch.randn_like(x) * 2)
        u.copy_(torch.rand_like(u))
        graph.replay()
        torch.cuda.synchronize()
        got = tokens.cpu().numpy().copy()
        kda.sample(**args)
        torch.cuda.synchronize()
        assert np.array_equal(got, tokens.cpu().numpy())
        want = expect(x, u.cpu().numpy(), None,
                      np.array([50] * 4 + [0] * 4), np.full(M, 0.9))
        assert np.array_equal(got, want), i


def _cpu():
    M, V = 4, 100
    i = lambda n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    return dict(logits=torch.zeros(M, V), uniform=torch.zeros(M),
                tokens=i(M), temperature=torch.ones(2), top_k=i(2),
                top_p=torch.ones(2), min_p=torch.zeros(2),
                query_start_loc=torch.tensor([0, 2, 4], dtype=torch.int32),
                draft_tokens=i(M), num_accepted=i(2), next_tokens=i(2),
                workspace=torch.empty(kda.sample_workspace_size(M, V),
                                      dtype=torch.uint8))


def test_sample_checks():
    ok = _cpu()
    assert kda.check_sample(**ok) == _abi.KDA_OK
    bad = [
        (dict(logits=ok["logits"].half()), _abi.KDA_E_DTYPE),
        (dict(logits=torch.zeros(100, 4).t()), _abi.KDA_E_LAYOUT),
        (dict(logits=torch.zeros(4, 0)), _abi.KDA_E_SHAPE),
        (dict(logits=torch.zeros(1, 1).expand(4, (1 << 20) + 1)),
         _abi.KDA_E_UNSUPPORTED),
        (dict(workspace=ok["workspace"][:64]), _abi.KDA_E_CAPACITY),
        (dict(num_accepted=None), _abi.KDA_E_ARG),
        (dict(draft_tokens=None), _abi.KDA_E_ARG),
    ]
    for over, code in bad:
        assert kda.check_sample(**dict(ok, **over)) == code, over.keys()
    alone = dict(ok, query_start_loc=None, draft_tokens=None,
                 num_accepted=None, next_tokens=None, temperature=None,
                 top_k=None, top_p=None, min_p=None)
    assert kda.check_sample(**alone) == _abi.KDA_OK
    lib = _abi.load()
    assert lib.kda_check_sample(None) == _abi.KDA_E_ARG
    a = kda.sample_args(**alone)
    a.batch = 3
    assert lib.kda_check_sample(a) == _abi.KDA_E_SHAPE
    a = kda.sample_args(**ok)
    a.uniform = None
    assert lib.kda_check_sample(a) == _abi.KDA_E_ARG


def test_sample_binding_refusals():
    ok = _cpu()
    with pytest.raises(ValueError, match="GPU"):
        kda.sample(**ok)
    with pytest.raises(TypeError):
        kda.check_sample(**dict(ok, top_k=torch.zeros(2)))
    with pytest.raises(TypeError):
        kda.check_sample(**dict(ok, uniform=torch.zeros(4).double()))
    with pytest.raises(ValueError, match="top_p"):
        kda.check_sample(**dict(ok, top_p=torch.zeros(1)))
    with pytest.raises(ValueError):
        kda.sample_workspace_size(4, (1 << 20) + 1)
    with pytest.raises(ValueError):       # work items of a launch past 2^32
        kda.sample_workspace_size(1 << 23, 40)


def test_oracle_sampling_closed_forms():
    """The oracle itself, on rows whose answer is plain."""
    x = np.log(np.array([1.0, 2.0, 4.0, 1.0]))
    assert [oracle.sample_row(x, u) for u in (0.0, 0.12, 0.13, 0.37, 0.38,
                                              0.87, 0.88)] == \
        [0, 0, 1, 1, 2, 2, 3]
    assert oracle.sample_row(x, 0.99, top_k=2) == 2
    assert oracle.sample_row(x, 0.01, top_p=0.5) == 2
    assert oracle.sample_row(x, 0.01, top_p=0.51) == 1
    assert oracle.sample_row(x, 0.01, min_p=0.4) == 1
    assert oracle.sample_row(x, 0.5, temperature=0) == 2
    assert oracle.sample_row(np.full(3, -np.inf), 0.5) == -1
