"""Edges of the block operators: calls without forks."""
import pytest
import torch

import linear_attention_speculative_amd as kda
from tests.test_gpu_blocks import fork_case


@pytest.mark.gpu
def test_no_forks_take_no_blocks():
    """num_allocated is an output of such a call, too."""
    kw, _ = fork_case(20, 30, 6, 4, seed=3)
    kda.fork_blocks(**kw)
    torch.cuda.synchronize()
    assert int(kw["num_allocated"]) > 0
    before = {n: kw[n].clone() for n in ("block_table", "num_blocks",
                                         "num_computed_tokens")}
    none = dict(kw, **{n: kw[n][:0] for n in ("parent_rows", "child_rows",
                                              "copy_pairs")})
    kda.fork_blocks(**none)
    torch.cuda.synchronize()
    assert int(kw["num_allocated"]) == 0
    for n, t in before.items():
        assert torch.equal(kw[n], t), n
    # captured, behind a call with forks
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.fork_blocks(**none)
    for _ in range(2):
        kw["num_allocated"].fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert int(kw["num_allocated"]) == 0
