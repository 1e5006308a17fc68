"""The serving operators where offsets pass 32 bits: state pools, logits and
workspaces of more than 4 GiB; calls at once on two streams; and two captured
graphs that share a workspace."""
import numpy as np
import pytest
import torch

import linear_attention_speculative_amd as kda
from tests.layer_check import F32_TOL, OPERAND_TOL, i32, make_layer

DEV = "cuda"



@pytest.mark.gpu
def test_state_slots_past_32_bits():
    """The last slots of a pool of 2^31 fp32 elements and more give what the
    first ones give."""
    H, D, N = 32, 128, 4100                  # 2^19 elements a slot
    kw = make_layer(8, 5, H, D, 1, act="bf16", seed=71)
    far = dict(kw, out=kw["out"].clone(),
               state=torch.empty((N, H, D, D), device=DEV),
               conv_state=torch.empty((N, *kw["conv_state"].shape[1:]),
                                      dtype=torch.bfloat16, device=DEV))
    for name in ("state", "conv_state"):
        far[name][N - 4:] = kw[name][1:]
    for args, first in ((kw, 1), (far, N - 4)):
        rows = {k: args[k][:2] for k in ("mixed_qkv", "raw_gate", "raw_beta",
                                         "out")}
        kda.conv_update_decode(
            **dict(args, **rows), state_indices=i32([first, first + 1], DEV),
            final_state_indices=i32([first, first + 2], DEV))
        rows = {k: args[k][2:] for k in ("mixed_qkv", "raw_gate", "raw_beta",
                                         "out")}
        kda.conv_prefill(
            **dict(args, **rows), query_start_loc=i32([0, 6], DEV),
            state_indices=i32([first + 3], DEV),
            initial_state_indices=i32([first + 2], DEV),
            workspace=torch.empty(kda.prefill_workspace_size(
                6, 1, H, D, torch.bfloat16), dtype=torch.uint8, device=DEV))
    torch.cuda.synchronize()
    assert torch.equal(kw["out"], far["out"])
    for name in ("state", "conv_state"):
        assert torch.equal(kw[name][1:], far[name][N - 4:]), name


@pytest.mark.gpu
def test_prompt_with_a_workspace_past_32_bits():
    """One prompt whose operands take more than 4 GiB, against the same prompt
    in pieces that take less."""
    T, H, D, cut = 70016, 32, 128, 35000
    kw = make_layer(T, 3, H, D, 1, act="bf16", seed=72)
    size = kda.prefill_workspace_size(T, 1, H, D, torch.bfloat16)
    assert size > 1 << 32
    work = torch.empty(size, dtype=torch.uint8, device=DEV)
    one, two = i32([1], DEV), i32([2], DEV)
    kda.conv_prefill(**kw, query_start_loc=i32([0, T], DEV),
                     state_indices=one, workspace=work)
    whole = kw["out"].clone()
    for s, e in ((0, cut), (cut, T)):
        rows = {k: kw[k][s:e] for k in ("mixed_qkv", "raw_gate", "raw_beta",
                                        "out")}
        kda.conv_prefill(**dict(kw, **rows),
                         query_start_loc=i32([0, e - s], DEV),
                         state_indices=two,
                         initial_state_indices=two if s else None,
                         workspace=work)
    torch.cuda.synchronize()
    # each side within its bound of the exact result, and a bf16 step apart
    # where they round to neighbours
    a, b = whole[-40000:].float(), kw["out"][-40000:].float()
    assert bool(((a - b).abs() <= 2 * OPERAND_TOL * a.abs().max() +
                 2.0 ** -7 * a.abs()).all())
    a, b = kw["state"][1], kw["state"][2]
    assert float((a - b).abs().max() / a.abs().max()) <= 2 * F32_TOL
    assert torch.equal(kw["conv_state"][1][:, :3], kw["conv_state"][2][:, :3])


@pytest.mark.gpu
def test_logits_past_32_bits():
    """Rows beyond 4 GiB of logits give what the same rows give alone."""
    M, V, last = 17000, 131072, 6
    assert M * V * 2 > 1 << 32
    x = torch.zeros((M, V), dtype=torch.bfloat16, device=DEV)
    g = torch.Generator().manual_seed(73)
    x[-last:] = (2 * torch.randn((last, V), generator=g)).to(DEV)
    u = torch.rand(M, generator=g).to(DEV)
    B = 17000
    T = torch.zeros(B, device=DEV)
    k, p = i32(np.zeros(B), DEV), torch.ones(B, device=DEV)
    T[-last:] = 1.0
    k[-last:] = i32([0, 20, 1000, 0, 3000, 0], DEV)
    p[-last:] = torch.tensor([0.9, 1.0, 0.8, 1.0, 1.0, 0.5], device=DEV)
    out = []
    for s in (0, M - last):
        m = M - s
        tokens = torch.full((m,), -9, dtype=torch.int32, device=DEV)
        kda.sample(logits=x[s:], uniform=u[s:], tokens=tokens,
                   temperature=T[s:], top_k=k[s:], top_p=p[s:],
                   workspace=torch.empty(kda.sample_workspace_size(m, V),
                                         dtype=torch.uint8, device=DEV))
        out.append(tokens)
    torch.cuda.synchronize()
    assert torch.equal(out[0][-last:], out[1])
    assert bool((out[0][:-last] == 0).all())


@pytest.mark.gpu
def test_sampling_at_once_on_two_streams_and_shared_workspaces():
    """Two samplings in flight together, each with its own workspace; and two
    graphs with one workspace, replayed in turn with other work between."""
    V, M = 30000, 40
    sets = []
    for i in range(2):
        g = torch.Generator().manual_seed(80 + i)
        sets.append(dict(
            logits=(2 * torch.randn((M, V), generator=g)).to(DEV),
            uniform=torch.rand(M, generator=g).to(DEV),
            temperature=torch.full((M,), 0.8, device=DEV),
            top_k=i32(np.resize([0, 20, 900], M), DEV),
            top_p=torch.full((M,), 0.9, device=DEV)))
    size = kda.sample_workspace_size(M, V)

    def fresh():
        return torch.full((M,), -9, dtype=torch.int32, device=DEV)

    work = [torch.full((size,), 0xff, dtype=torch.uint8, device=DEV)
            for _ in range(2)]
    alone = [fresh(), fresh()]
    for s, t in zip(sets, alone):
        kda.sample(**s, tokens=t, workspace=work[0])
    streams = [torch.cuda.Stream() for _ in range(2)]
    both = [fresh(), fresh()]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, t, w, st in zip(sets, both, work, streams):
            kda.sample(**s, tokens=t, workspace=w, stream=st)
    torch.cuda.synchronize()
    graphs, outs = [], [fresh(), fresh()]
    for s, t in zip(sets, outs):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            kda.sample(**s, tokens=t, workspace=work[0])
    for i in range(3):
        for t in outs:
            t.fill_(-9)
        for gr in graphs[::1 if i % 2 else -1]:
            gr.replay()
            kda.sample(**sets[0], tokens=both[0], workspace=work[0])
        torch.cuda.synchronize()
        for a, b, c in zip(alone, both, outs):
            assert torch.equal(a, b) and torch.equal(a, c), i
