"""Changes of logits in place against the fp64 oracle: types, vocabulary sizes
around the slices, unaligned rows, draft windows, empty windows and
histories, tokens out of range, biases named twice, masks that allow
nothing, parameters that leave their change out, graphs; and the refusals
(CPU)."""
import numpy as np
import pytest
import torch

import linear_attention_speculative_amd as kda
import oracle
from linear_attention_speculative_amd import _abi
from tests.latent_check import ACT, f64

DEV = "cuda"
I32 = torch.int32


def make(lens, V, *, act="f32", hist=30, seed=0, pad=0, shift=0, tail=0,
         window=True, masks=3, device=DEV):
    rng = np.random.RandomState(seed)
    g = torch.Generator().manual_seed(seed)
    B, M = len(lens), int(np.sum(lens)) + tail
    rows, L = B + 2, hist + 5
    to = lambda a, t=I32: torch.as_tensor(np.asarray(a)).to(t).to(device)  # noqa: E731
    full = torch.randn((M, V + pad + shift), generator=g) * 3
    nb = rng.randint(0, 9, size=B)
    tok = rng.randint(0, V, size=(rows, L)) if V > 50 else \
        rng.randint(-2, V + 2, size=(rows, L))
    # some tokens over and over, some out of range
    tok[:, ::3] = rng.randint(0, min(V, 7), size=tok[:, ::3].shape)
    tok[:, 1] = [-1, V, 2 ** 31 - 1, -2 ** 31][seed % 4]
    known = rng.randint(0, L + 4, size=rows)
    bt = rng.randint(0, min(V, 40), size=max(int(nb.sum()), 1))
    bt[::5] = -7
    W = (V + 31) // 32
    words = rng.randint(-2 ** 31, 2 ** 31, size=(masks, W + 1))
    if masks:
        words[0] = 0                     # a mask that allows nothing
    kw = dict(logits=full.to(ACT[act]).to(device)[:, shift:shift + V],
              request_indices=to(rng.permutation(rows)[:B]),
              token_ids=to(tok), prompt_lens=to(rng.randint(-1, L, size=rows)),
              token_lens=to(known),
              repetition_penalty=to(rng.choice([1.0, 1.2, 0.7], size=B),
                                    torch.float32),
              frequency_penalty=to(rng.choice([0.0, 0.5, -0.25], size=B),
                                   torch.float32),
              presence_penalty=to(rng.choice([0.0, 0.3], size=B),
                                  torch.float32),
              bias_start=to(np.concatenate([[0], np.cumsum(nb)])),
              bias_tokens=to(bt),
              bias_values=to(rng.randn(len(bt)) * 4, torch.float32),
              mask=to(words), mask_rows=to(rng.randint(-1, masks + 1,
                                                       size=M)))
    if window:
        kw["query_start_loc"] = to(np.concatenate([[0], np.cumsum(lens)]))
        kw["draft_tokens"] = to(rng.randint(0, min(V, 9), size=M))
    return kw


def expect(kw):
    host = {k: v.cpu().numpy() if v.dtype != torch.bfloat16 else f64(v)
            for k, v in kw.items()}
    return oracle.adjust_logits(**host)


def check(kw, before, ref, size):
    """Four fp32 steps (bias, penalty, two subtractions) of half a unit each
    of the magnitudes, two more for the product f * count, one rounding."""
    got, u = f64(kw["logits"]), 2.0 ** -24
    half = 2.0 ** -8 if kw["logits"].dtype == torch.bfloat16 else u
    fin = np.isfinite(ref)
    assert np.array_equal(got[~fin], ref[~fin])
    off = 6 * u * size[fin]
    assert (np.abs(got[fin] - ref[fin]) <=
            off + half * (np.abs(ref[fin]) + off)).all()
    same = ref == before                     # nothing changes these
    assert np.array_equal(got[same], before[same])


CASES = [
    dict(lens=[1], V=1, act="f32", window=False),
    dict(lens=[1] * 5, V=33, act="bf16", window=False),
    dict(lens=[1, 0, 4, 2, 0], V=300, act="f32", tail=3),
    dict(lens=[4, 4, 1], V=8192, act="bf16"),
    dict(lens=[2, 3], V=8193, act="bf16", pad=3),
    dict(lens=[3, 1], V=16385 + 8, act="f32", pad=1),
    dict(lens=[2, 2], V=20001, act="bf16", shift=3),
    dict(lens=[1, 1], V=50021, act="f32", shift=1, window=False),
    dict(lens=[16, 1, 9], V=1000, act="bf16", hist=400),
    dict(lens=[100, 3], V=500, act="f32", hist=90),     # windows shared
    dict(lens=[0, 0], V=100, act="f32", tail=2),
    dict(lens=[2, 1], V=131072, act="bf16", hist=5000),
    # histories around what the table takes, and longer
    dict(lens=[3, 0, 1, 2], V=20001, act="bf16", hist=6130, pad=1),
    dict(lens=[80, 5], V=9001, act="f32", hist=7000),
    dict(lens=[70, 66], V=400, act="bf16", hist=40),
    dict(lens=[2] * 9, V=140000, act="f32", hist=9000),
]


@pytest.mark.gpu
@pytest.mark.parametrize("ci", range(len(CASES)))
def test_changes_match_oracle(ci):
    kw = make(seed=ci, **CASES[ci])
    before = f64(kw["logits"])
    ref, size = expect(kw)
    kda.adjust_logits(**kw)
    torch.cuda.synchronize()
    check(kw, before, ref, size)


@pytest.mark.gpu
@pytest.mark.parametrize("left_out", [
    ("mask", "mask_rows"), ("mask_rows",), ("draft_tokens",),
    ("bias_start", "bias_tokens", "bias_values"),
    ("token_ids", "prompt_lens", "token_lens", "request_indices"),
    ("repetition_penalty",), ("frequency_penalty", "presence_penalty"),
    ("repetition_penalty", "frequency_penalty", "presence_penalty"),
    ("repetition_penalty", "frequency_penalty", "presence_penalty", "mask",
     "mask_rows"),
    ("request_indices",)])
def test_changes_left_out(left_out):
    kw = make([3, 1, 2], 700, act="bf16", seed=3, masks=6)
    for n in left_out:
        del kw[n]
    before = f64(kw["logits"])
    ref, size = expect(kw)
    kda.adjust_logits(**kw)
    torch.cuda.synchronize()
    check(kw, before, ref, size)


@pytest.mark.gpu
def test_parameters_that_leave_their_change_out():
    kw = make([1] * 6, 200, seed=5)
    nan, inf = float("nan"), float("inf")
    kw["repetition_penalty"] = torch.tensor([0., -2., nan, 1., 2., inf],
                                            device=DEV)
    kw["frequency_penalty"] = torch.tensor([nan, .5, 0., 0., nan, 0.],
                                           device=DEV)
    kw["presence_penalty"] = torch.tensor([.5, nan, 0., nan, 0., 0.],
                                          device=DEV)
    kw["request_indices"][3] = -1
    kw["request_indices"][1] = 10 ** 6
    before = f64(kw["logits"])
    with np.errstate(divide="ignore"):
        ref, size = expect(kw)
    kda.adjust_logits(**kw)
    torch.cuda.synchronize()
    ok = np.isfinite(size)
    size[~ok] = 0
    check(kw, before, ref, size)


@pytest.mark.gpu
def test_infinite_and_nan_logits():
    kw = make([2, 1], 100, seed=2, masks=0)
    del kw["mask"], kw["mask_rows"]
    x = kw["logits"]
    x[:, :6] = torch.tensor([float("inf"), -float("inf"), float("nan")] * 2,
                            device=DEV)
    ref, _ = expect(kw)
    kda.adjust_logits(**kw)
    torch.cuda.synchronize()
    assert np.array_equal(f64(x)[:, :6], ref[:, :6], equal_nan=True)


@pytest.mark.gpu
def test_counts_past_an_eighth_of_a_million_and_long_lists():
    """One token produced 150000 times; 3000 biases of one request."""
    kw = make([2], 90, seed=1, hist=150000)
    kw["token_ids"][:] = 11
    kw["prompt_lens"][:] = 3
    kw["token_lens"][:] = 150005
    n = 3000
    kw["bias_start"] = torch.tensor([0, n], dtype=I32, device=DEV)
    kw["bias_tokens"] = (torch.arange(n, device=DEV) % 60).to(I32)
    kw["bias_values"] = torch.randn(n, device=DEV)
    kw["frequency_penalty"][:] = 0.125
    before = f64(kw["logits"])
    ref, size = expect(kw)
    kda.adjust_logits(**kw)
    torch.cuda.synchronize()
    check(kw, before, ref, size)


@pytest.mark.gpu
def test_graph_replays_with_growing_histories():
    kw = make([2, 1, 3], 5000, act="bf16", hist=100, seed=4)
    raw = kw["logits"].clone()
    kda.adjust_logits(**kw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.adjust_logits(**kw)
    for step in range(3):
        kw["token_lens"] += 2 * step
        kw["logits"].copy_(raw)
        before = f64(raw)
        ref, size = expect(kw)
        graph.replay()
        torch.randn(100, device=DEV).sum().item()
        check(kw, before, ref, size)


@pytest.mark.gpu
def test_logits_then_sampling():
    """The sampling sees what the mask leaves: allowed tokens only, and -1 for
    a row whose mask allows nothing."""
    V, M = 1000, 8
    kw = make([1] * M, V, act="bf16", seed=6, window=False)
    words = torch.zeros((M, 32), dtype=I32, device=DEV)
    allowed = [5, 40, 999, 0, 31, 32, 640]
    for m, t in enumerate(allowed):
        words[m, t // 32] = (1 << (t % 32)) - (1 << 32 if t % 32 == 31 else 0)
    kw["mask"], kw["mask_rows"] = words, None
    del kw["bias_start"]
    kda.adjust_logits(**kw)
    tokens = torch.zeros(M, dtype=I32, device=DEV)
    kda.sample(logits=kw["logits"], uniform=torch.rand(M, device=DEV),
               tokens=tokens, workspace=torch.empty(
                   kda.sample_workspace_size(M, V), dtype=torch.uint8,
                   device=DEV))
    torch.cuda.synchronize()
    assert tokens.tolist() == allowed + [-1]


def test_refusals():
    ok = make([2, 1], 100, device="cpu")
    chk = lambda **d: kda.check_adjust_logits(**dict(ok, **d))  # noqa: E731
    assert chk() == _abi.KDA_OK
    with pytest.raises(ValueError, match="GPU"):
        kda.adjust_logits(**ok)
    x = ok["logits"]
    assert chk(logits=x.half()) == _abi.KDA_E_DTYPE
    assert chk(logits=x[:1].expand(3, -1)) == _abi.KDA_E_LAYOUT
    assert chk(logits=x.t().contiguous().t()) == _abi.KDA_E_LAYOUT
    assert chk(logits=x[:, :0]) == _abi.KDA_E_SHAPE
    assert chk(query_start_loc=None, draft_tokens=None,
               repetition_penalty=torch.ones(3),
               frequency_penalty=torch.ones(3),
               presence_penalty=torch.ones(3), request_indices=torch.zeros(
                   3, dtype=I32), bias_start=None) == _abi.KDA_OK
    with pytest.raises(ValueError, match="entries"):
        chk(query_start_loc=None)
    with pytest.raises(TypeError):
        chk(repetition_penalty=ok["repetition_penalty"].double())
    with pytest.raises(ValueError, match="bit for every"):
        chk(mask=ok["mask"][:, :3].contiguous())
    with pytest.raises(ValueError, match="mask per row"):
        chk(mask=ok["mask"][:2], mask_rows=None)
    with pytest.raises(ValueError, match="bias_tokens"):
        chk(bias_values=None)
    with pytest.raises(ValueError, match="token_lens"):
        chk(token_lens=None)
    with pytest.raises(ValueError, match="row per"):
        chk(request_indices=None, token_ids=ok["token_ids"][:1])
    lib = _abi.load()
    assert lib.kda_check_adjust_logits(None) == _abi.KDA_E_ARG
    for name, value, want in (
            ("batch", -1, _abi.KDA_E_ARG), ("max_len", -1, _abi.KDA_E_ARG),
            ("prompt_lens", None, _abi.KDA_E_ARG),
            ("bias_values", None, _abi.KDA_E_ARG),
            ("mask_stride", 1, _abi.KDA_E_LAYOUT),
            ("token_ids_stride", 3, _abi.KDA_E_LAYOUT),
            ("query_start_loc", None, _abi.KDA_E_SHAPE),
            ("batch", 70000, _abi.KDA_E_CAPACITY)):
        a = kda.logits_args(**ok)
        setattr(a, name, value)
        assert lib.kda_check_adjust_logits(a) == want, name
