"""A step's index tables against the request-by-request oracle: exact
integers over batch sizes around the kernels' tiles, ragged and empty
requests, exhausted free blocks, narrow tables, rows outside the table,
capacity short of the tokens, in-place block counts, and graph replays; and
the refusals (CPU)."""
import numpy as np
import pytest
import torch

import linear_attention_speculative_amd as kda
import oracle
from linear_attention_speculative_amd import _abi

DEV = "cuda"
I32 = torch.int32


def make(B, rows, width, block, qmax, seed=0, cmax=None, free=None, cap=None,
         req=True, empty=0.2, bad_rows=0, null=0, device=DEV):
    rng = np.random.RandomState(seed)
    q = rng.randint(0, qmax + 1, size=B)
    q[rng.rand(B) < empty] = 0
    computed = rng.randint(0, (cmax or width * block) + 1, size=rows)
    computed[rng.rand(rows) < 0.3] = 0
    held = np.where(computed > 0, np.minimum(computed // block + 1, width), 0)
    perm = null + 1 + rng.permutation(rows * width)
    table = perm.reshape(rows, width).copy()
    ids = rng.permutation(rows)[:B] if req else np.arange(B)
    for i in range(bad_rows):
        ids[i * 3 % B] = [-1, rows, 10 ** 6][i % 3]
    total = int(q.sum())
    cap = total + 5 if cap is None else cap
    nfree = rows * width if free is None else free
    host = dict(query_lens=q, num_computed_tokens=computed, num_blocks=held,
                block_table=table,
                free_blocks=null + 1 + rows * width + rng.permutation(nfree),
                block_size=block, null_block_id=null,
                request_indices=ids if req else None)
    to = lambda a: torch.as_tensor(a, dtype=I32).to(device)  # noqa: E731
    kw = {k: to(v) if isinstance(v, np.ndarray) else v
          for k, v in host.items()}
    kw.update(
        query_start_loc=torch.full((B + 1,), -9, dtype=I32, device=device),
        new_num_blocks=kw["num_blocks"].clone(),
        positions=torch.full((cap,), -9, dtype=I32, device=device),
        slot_mapping=torch.full((cap,), -9, dtype=torch.int64, device=device),
        num_allocated=torch.full((1,), -9, dtype=I32, device=device))
    for name in ("state", "initial_state", "final_state"):
        kw[name + "_indices"] = torch.full((B,), -9, dtype=I32, device=device)
    return kw, dict(host, max_tokens=cap)


def check(kw, ref):
    for name, want in ref.items():
        got = kw[name].cpu().numpy()
        assert np.array_equal(got, want), (name, got, want)


CASES = [
    dict(B=1, rows=1, width=3, block=4, qmax=5),
    dict(B=7, rows=9, width=6, block=16, qmax=30),
    dict(B=63, rows=64, width=5, block=1, qmax=3),
    dict(B=64, rows=64, width=9, block=100, qmax=700, req=False),
    dict(B=1023, rows=1100, width=4, block=16, qmax=4),
    dict(B=1024, rows=1024, width=4, block=16, qmax=4, req=False),
    dict(B=1025, rows=1030, width=4, block=7, qmax=30, bad_rows=3),
    dict(B=9000, rows=9000, width=3, block=8, qmax=3),
    dict(B=33, rows=40, width=8, block=16, qmax=60, free=11),
    dict(B=12, rows=12, width=8, block=16, qmax=60, free=0),
    dict(B=20, rows=20, width=2, block=16, qmax=200),
    dict(B=20, rows=25, width=8, block=16, qmax=40, cap=100),
    dict(B=20, rows=25, width=8, block=16, qmax=40, cap=0),
    dict(B=30, rows=30, width=4, block=32, qmax=9, empty=1.0, cap=70),
    dict(B=16, rows=20, width=6, block=64, qmax=90, null=5, bad_rows=4),
]


@pytest.mark.gpu
@pytest.mark.parametrize("ci", range(len(CASES)))
def test_step_tables_match_oracle(ci):
    kw, host = make(seed=ci, **CASES[ci])
    ref = oracle.step_tables(**host)
    kda.step_tables(**kw)
    torch.cuda.synchronize()
    check(kw, ref)


@pytest.mark.gpu
@pytest.mark.parametrize("free", [None, 1500])
@pytest.mark.parametrize("B", [255, 256, 257, 511, 2047, 2048, 2049, 4097])
def test_batches_around_the_tiles(B, free):
    """Batches at the borders of the request kernel's variants and tiles,
    with many new blocks a request, some requests without any."""
    kw, host = make(B=B, rows=B + 3, width=7, block=5, qmax=33, seed=B,
                    free=free)
    ref = oracle.step_tables(**host)
    kda.step_tables(**kw)
    torch.cuda.synchronize()
    check(kw, ref)


@pytest.mark.gpu
def test_empty_batch():
    kw, host = make(1, 2, 2, 4, 3, cap=6)
    for n in ("query_lens", "request_indices", "state_indices",
              "initial_state_indices", "final_state_indices"):
        kw[n] = kw[n][:0]
    kda.step_tables(**kw)
    torch.cuda.synchronize()
    assert kw["query_start_loc"][0].item() == 0
    assert kw["num_allocated"].item() == 0
    assert (kw["slot_mapping"] == -1).all() and (kw["positions"] == 0).all()


@pytest.mark.gpu
def test_block_counts_in_place_over_steps_in_a_graph():
    """Requests grow over replays of one captured step: held counts updated
    in place, computed tokens advanced between the replays, each replay
    against the oracle on the same state."""
    kw, host = make(5, 6, 12, 4, 6, cmax=8, free=60, cap=40, seed=2)
    kw["new_num_blocks"] = kw["num_blocks"]
    state = {k: kw[k].clone() for k in ("block_table", "num_blocks")}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.step_tables(**kw)
    for k, v in state.items():
        kw[k].copy_(v)
    free = host["free_blocks"]
    for step in range(4):
        ref = oracle.step_tables(**host)
        graph.replay()
        torch.cuda.synchronize()
        check(kw, ref)
        # the scheduler's part between steps: advance, drop used free blocks
        host["num_computed_tokens"] = host["num_computed_tokens"].copy()
        host["num_computed_tokens"][host["request_indices"]] += \
            host["query_lens"]
        host["num_blocks"] = ref["new_num_blocks"]
        host["block_table"] = ref["block_table"]
        used = int(ref["num_allocated"][0])
        host["free_blocks"] = np.roll(host["free_blocks"], -used)
        kw["num_computed_tokens"].copy_(
            torch.as_tensor(host["num_computed_tokens"]))
        kw["free_blocks"].copy_(torch.as_tensor(host["free_blocks"]))
        torch.randn(100, device=DEV).sum().item()
    assert free.size == 60


@pytest.mark.gpu
def test_slots_pass_32_bits():
    kw, host = make(3, 3, 2, 1 << 20, 4, cmax=100, seed=1)
    kw["block_table"] += 100_000
    host["block_table"] = host["block_table"] + 100_000
    ref = oracle.step_tables(**host)
    assert ref["slot_mapping"].max() > 1 << 32
    kda.step_tables(**kw)
    torch.cuda.synchronize()
    check(kw, ref)


@pytest.mark.gpu
def test_strided_table_rows():
    kw, host = make(6, 8, 5, 16, 40, seed=6)
    wide = torch.full((8, 9), -3, dtype=I32, device=DEV)
    wide[:, :5] = kw["block_table"]
    kw["block_table"] = wide[:, :5]
    ref = oracle.step_tables(**host)
    kda.step_tables(**kw)
    torch.cuda.synchronize()
    check(kw, ref)
    assert (wide[:, 5:] == -3).all()


def test_step_tables_refusals():
    ok, _ = make(4, 5, 3, 8, 6, device="cpu")
    assert kda.check_step_tables(**ok) == _abi.KDA_OK
    with pytest.raises(ValueError, match="GPU"):
        kda.step_tables(**ok)
    with pytest.raises(TypeError):
        kda.check_step_tables(**dict(ok, query_lens=ok["query_lens"].long()))
    with pytest.raises(TypeError):
        kda.check_step_tables(**dict(ok,
                                     slot_mapping=ok["slot_mapping"].int()))
    with pytest.raises(ValueError):
        kda.check_step_tables(**dict(ok, positions=ok["positions"][:-1]))
    with pytest.raises(ValueError, match="entries"):
        kda.check_step_tables(**dict(ok, num_blocks=ok["num_blocks"][:4]))
    with pytest.raises(ValueError, match="row per request"):
        kda.check_step_tables(**dict(ok, request_indices=None,
                                     block_table=ok["block_table"][:3]))
    assert kda.check_step_tables(**dict(ok, block_size=0)) == _abi.KDA_E_ARG
    assert kda.check_step_tables(**dict(ok, null_block_id=-1)) == \
        _abi.KDA_E_ARG
    shared = ok["block_table"][:1].expand(5, -1)
    assert kda.check_step_tables(**dict(ok, block_table=shared)) == \
        _abi.KDA_E_LAYOUT
    lib = _abi.load()
    assert lib.kda_check_step_tables(None) == _abi.KDA_E_ARG
    a = kda.tables_args(**ok)
    a.num_allocated = None
    assert lib.kda_check_step_tables(a) == _abi.KDA_E_ARG
    a = kda.tables_args(**ok)
    a.max_tokens = -1
    assert lib.kda_check_step_tables(a) == _abi.KDA_E_ARG
