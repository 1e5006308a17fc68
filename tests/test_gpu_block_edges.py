"""Edges of the block operators: calls without forks, forks at the end of the
table, blocks that a holder outside the table pins, and sizes past what one
launch takes (CPU)."""
import numpy as np
import pytest
import torch

import linear_attention_speculative_amd as kda
import oracle
from linear_attention_speculative_amd import _abi
from tests.latent_check import ints
from tests.test_gpu_blocks import (compaction, fork_case, held_case, i32,
                                   same)

DEV = "cuda"
I32 = torch.int32


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


def full_rows(F, device=DEV):
    """Forks of which every third parent holds its table's whole width, with
    a free block for each of the others."""
    width, block, rows = 4, 8, 2 * F
    rng = np.random.RandomState(F)
    comp = np.zeros(rows, np.int64)
    comp[:F] = rng.randint(0, width * block, size=F)
    comp[:F:3] = width * block + rng.randint(0, 3, size=len(comp[:F:3]))
    table = 1 + np.arange(rows * width).reshape(rows, width)
    fits = comp[:F] // block < width
    host = dict(parent_rows=np.arange(F), child_rows=F + np.arange(F),
                num_computed_tokens=comp,
                num_blocks=np.minimum(comp // block + 1, width),
                block_table=table, free_blocks=900 + np.arange(fits.sum()),
                block_size=block, null_block_id=0)
    return host, fits


@pytest.mark.parametrize("F", [1, 7, 300])
def test_oracle_forks_past_the_table_take_no_block(F):
    host, fits = full_rows(F)
    ref = oracle.fork_blocks(**host)
    assert ref["num_allocated"] == fits.sum()
    got, k = 900, host["num_computed_tokens"][:F] // 8
    for f in range(F):
        child = ref["block_table"][F + f]
        assert ref["num_blocks"][F + f] == min(k[f] + 1, 4)
        assert np.array_equal(child[:k[f]], host["block_table"][f, :k[f]])
        if fits[f]:
            assert child[k[f]] == got
            assert list(ref["copy_pairs"][f]) == [
                host["block_table"][f, k[f]], got]
            got += 1
        else:
            assert list(ref["copy_pairs"][f]) == [0, 0]


@pytest.mark.gpu
@pytest.mark.parametrize("F", [1, 7, 300])
def test_forks_past_the_table_take_no_block(F):
    host, fits = full_rows(F)
    kw = {k: i32(v) if isinstance(v, np.ndarray) else v
          for k, v in host.items()}
    kw.update(copy_pairs=torch.full((F, 2), -9, dtype=I32, device=DEV),
              num_allocated=torch.full((1,), -9, dtype=I32, device=DEV))
    kda.fork_blocks(**kw)
    torch.cuda.synchronize()
    assert int(kw["num_allocated"]) == fits.sum()
    same(kw, oracle.fork_blocks(**host))


@pytest.mark.gpu
@pytest.mark.parametrize("N", [64, 20000])
def test_pinned_blocks_follow_the_moves(N):
    """A prefix holder's blocks move with the others: it applies the pairs to
    its ids and its pins, and the next recount finds them held."""
    kw, _ = held_case(6, 5, N, seed=2, fill=1.0, released=0.5, pinned=True)
    ids = torch.tensor([N - 1, N - 3, N - 4], device=DEV)
    kw["pinned"][ids] = 1
    pool = torch.arange(N, device=DEV).view(-1, 1).repeat(1, 5).contiguous()
    text = pool[ids].clone()
    kda.free_blocks(**kw)
    kc = compaction(kw, N // 2)
    kda.compact_blocks(**kc)
    kda.BlockPools([pool]).copy(kc["copy_pairs"], kc["num_pairs"])
    # the holder: old id -> new id, pins at their new places
    src, dst = kc["copy_pairs"][:int(kc["num_pairs"])].long().t()
    to = torch.arange(N, device=DEV)
    to[src] = dst
    ids, pins = to[ids], kw["pinned"].clone()
    pins[dst], pins[src] = kw["pinned"][src], 0
    assert torch.equal(pool[ids], text)
    again = dict(kw, released_rows=kw["released_rows"][:0], pinned=pins,
                 block_table=kc["new_block_table"],
                 num_blocks=kw["new_num_blocks"],
                 new_num_blocks=kw["new_num_blocks"].clone(),
                 ref_counts=torch.empty_like(kw["ref_counts"]))
    kda.free_blocks(**again)
    torch.cuda.synchronize()
    assert torch.equal(again["ref_counts"].clamp(min=0),
                       kc["new_ref_counts"].clamp(min=0))
    free = ints(kw["free_blocks"])[:int(kw["num_free"])]
    assert not set(ints(ids)) & set(free)


def test_more_rows_than_a_launch_are_refused():
    """A workgroup of 256 a row, a fork, at most 2^32 work items."""
    n = 1 << 24
    ok, _ = fork_case(3, 8, 4, 4, device="cpu")
    lib = _abi.load()
    a = kda.fork_args(**ok)
    a.num_forks = n - 1
    assert lib.kda_check_fork_blocks(a) == _abi.KDA_OK
    a.num_forks = n
    assert lib.kda_check_fork_blocks(a) == _abi.KDA_E_CAPACITY

    ok, _ = held_case(6, 4, 30, device="cpu")
    a = kda.free_args(**ok)
    a.num_request_rows = n - 1
    assert lib.kda_check_free_blocks(a) == _abi.KDA_OK
    a.num_request_rows = n
    assert lib.kda_check_free_blocks(a) == _abi.KDA_E_CAPACITY

    z = lambda *s: torch.zeros(s, dtype=I32)  # noqa: E731
    a = kda.compact_blocks_args(
        ref_counts=ok["ref_counts"], block_table=ok["block_table"],
        num_blocks=ok["num_blocks"], new_block_table=z(6, 4),
        new_ref_counts=z(30), copy_pairs=z(15, 2), num_pairs=z(1),
        workspace=ok["workspace"])
    a.num_request_rows = n - 1
    assert lib.kda_check_compact_blocks(a) == _abi.KDA_OK
    a.num_request_rows = n
    assert lib.kda_check_compact_blocks(a) == _abi.KDA_E_CAPACITY


@pytest.mark.gpu
@pytest.mark.parametrize("rows,width,N", [
    # around what one workgroup reads of a table at a time
    (128, 64, 3000), (129, 64, 3000), (128, 65, 16384), (100, 256, 9000),
    (512, 64, 5000), (513, 3, 5000), (512, 65, 16384), (3000, 1, 700),
    (600, 0, 50), (0, 5, 50)])
def test_tables_around_a_round(rows, width, N):
    kw, host = held_case(max(rows, 1), max(width, 1), N, seed=rows + width,
                         fill=0.4, pinned=True)
    for n in ("num_blocks", "new_num_blocks"):
        kw[n] = kw[n][:rows]
    kw["block_table"] = kw["block_table"][:rows, :width]
    host.update(num_blocks=host["num_blocks"][:rows],
                block_table=host["block_table"][:rows, :width])
    ref = oracle.free_blocks(**host)
    kda.free_blocks(**kw)
    torch.cuda.synchronize()
    same(kw, ref)
    for place in (False, True):
        kc = compaction(kw, N // 2)
        if place:
            kc.update(new_block_table=kw["block_table"].clone())
            kc.update(block_table=kc["new_block_table"])
        kda.compact_blocks(**kc)
        torch.cuda.synchronize()
        same(kc, oracle.compact_blocks(
            ref_counts=ref["ref_counts"], block_table=host["block_table"],
            num_blocks=ref["new_num_blocks"], max_pairs=N // 2))
