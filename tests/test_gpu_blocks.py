"""Copies, forks, releases and compaction of cache blocks against the
request-by-request oracle: exact integers and bits over odd sizes, pools of
several kinds in pages, shared blocks, exhausted free blocks, rows and ids out
of range, in-place outputs, graphs; and the refusals (CPU)."""
import numpy as np
import pytest
import torch

import linear_attention_speculative_amd as kda
import oracle
from linear_attention_speculative_amd import _abi
from tests.latent_check import ints

DEV = "cuda"
I32 = torch.int32


def i32(a, device=DEV):
    return torch.as_tensor(np.asarray(a), dtype=I32).to(device)


def bits(t):
    return t.contiguous().view(torch.uint8).cpu().numpy().reshape(
        t.shape[0], -1)


# ---- copies -------------------------------------------------------------------

def pools(N, seed=0, device=DEV):
    """A state and a conv state in one page, a cache, odd bytes."""
    g = torch.Generator().manual_seed(seed)
    page = torch.randn((N, 4 * 16 * 16 + 96 * 6 + 20), generator=g).to(device)
    state = page[:, :1024].view(N, 4, 16, 16)
    conv = page[:, 1024:1024 + 576].view(N, 96, 6)
    cache = torch.randn((N, 80, 576), generator=g).bfloat16().to(device)
    odd = torch.randint(0, 256, (N, 7, 5), generator=g,
                        dtype=torch.uint8).to(device)
    half = torch.randn((N, 3, 9), generator=g).bfloat16().to(device)
    return page, [state, conv.transpose(1, 2), cache, odd, half]


@pytest.mark.gpu
@pytest.mark.parametrize("count", [None, 3, 0, 100, -4])
def test_copies(count):
    N = 40
    page, ps = pools(N)
    before = [bits(p) for p in ps]
    rest = page[:, 1600:].clone()
    pairs = np.array([[3, 7], [39, 1], [5, 5], [0, 9], [8, 0], [10 ** 6, 2],
                      [4, -3], [3, 12], [20, 30]])
    num = None if count is None else i32([count])
    kda.BlockPools(ps).copy(i32(pairs), num)
    torch.cuda.synchronize()
    want = oracle.copy_blocks(before, pairs, count)
    for p, w in zip(ps, want):
        assert np.array_equal(bits(p), w)
    assert torch.equal(page[:, 1600:], rest)


@pytest.mark.gpu
def test_copies_of_large_pools():
    """Pools past 4 GiB, blocks of several pieces, many pairs."""
    big = torch.empty((1200, 2 ** 20), dtype=torch.float32, device=DEV)
    small = torch.arange(1200, device=DEV).view(-1, 1).repeat(1, 3).contiguous()
    big[:600] = torch.arange(600, device=DEV).view(-1, 1)
    big[:, -1] = torch.arange(1200, device=DEV) * 2
    big[:, 7] = torch.arange(1200, device=DEV) * 3
    src = np.random.RandomState(0).permutation(np.arange(1, 600))
    pairs = np.stack([src, 600 + np.arange(599)], 1)
    kda.BlockPools([big, small]).copy(i32(pairs))
    torch.cuda.synchronize()
    at = torch.as_tensor(src).to(DEV)
    assert torch.equal(big[600:1199], big[at])
    assert torch.equal(small[600:1199], small[at])
    assert torch.equal(small[1:600, 0], torch.arange(1, 600, device=DEV))


@pytest.mark.gpu
def test_copies_in_a_graph():
    _, ps = pools(20)
    pools_of = kda.BlockPools(ps)
    pairs, num = i32([[1, 2], [3, 4]]), i32([2])
    graph = torch.cuda.CUDAGraph()
    pools_of.copy(pairs, num)
    with torch.cuda.graph(graph):
        pools_of.copy(pairs, num)
    for step in range(3):
        pairs.copy_(i32([[5 + step, 10 + step], [6, 15 + step]]))
        num.fill_(1 + step % 2)
        before = [bits(p) for p in ps]
        graph.replay()
        torch.cuda.synchronize()
        want = oracle.copy_blocks(before, ints(pairs), int(num))
        for p, w in zip(ps, want):
            assert np.array_equal(bits(p), w)


# ---- forks ----------------------------------------------------------------------

def fork_case(F, rows, width, block, seed=0, free=None, null=0, bad=0,
              device=DEV):
    rng = np.random.RandomState(seed)
    n = rows - F
    order = rng.permutation(rows)
    comp = rng.randint(-2, width * block + 3, size=rows)
    held = np.clip(comp // block + 1 - (rng.rand(rows) < 0.2), 0, width)
    table = null + 1 + rng.permutation(rows * width).reshape(rows, width)
    table[rng.rand(rows, width) < 0.05] = null
    parents = order[rng.randint(0, max(n, 1), size=F)]
    children = order[n:n + F]
    for i in range(bad):
        (parents if i % 2 else children)[i * 3 % F] = [-1, rows, 10 ** 8][i % 3]
    nfree = F if free is None else free
    host = dict(parent_rows=parents, child_rows=children,
                num_computed_tokens=comp, num_blocks=held, block_table=table,
                free_blocks=10 ** 6 + rng.permutation(nfree),
                block_size=block, null_block_id=null)
    kw = {k: i32(v, device) if isinstance(v, np.ndarray) else v
          for k, v in host.items()}
    kw.update(copy_pairs=torch.full((F, 2), -9, dtype=I32, device=device),
              num_allocated=torch.full((1,), -9, dtype=I32, device=device))
    return kw, host


def same(kw, ref):
    for name, want in ref.items():
        got = ints(kw[name])
        assert np.array_equal(got, want), (name, got, want)


FORKS = [
    dict(F=1, rows=2, width=1, block=1),
    dict(F=2, rows=5, width=4, block=16),
    dict(F=300, rows=700, width=9, block=7),
    dict(F=40, rows=60, width=5, block=4, free=11),
    dict(F=40, rows=60, width=5, block=4, free=0),
    dict(F=64, rows=100, width=700, block=3, null=4, bad=9),
]


@pytest.mark.gpu
@pytest.mark.parametrize("ci", range(len(FORKS)))
def test_forks(ci):
    kw, host = fork_case(seed=ci, **FORKS[ci])
    ref = oracle.fork_blocks(**host)
    kda.fork_blocks(**kw)
    torch.cuda.synchronize()
    same(kw, ref)


@pytest.mark.gpu
def test_forks_strided_table_and_no_forks():
    kw, host = fork_case(20, 30, 6, 4, seed=3)
    wide = torch.full((30, 14), -5, dtype=I32, device=DEV)
    wide[:, :12:2] = kw["block_table"]
    kw["block_table"] = wide[:, :12:2]
    ref = oracle.fork_blocks(**host)
    kda.fork_blocks(**kw)
    torch.cuda.synchronize()
    same(kw, ref)
    assert (wide[:, 1::2] == -5).all() and (wide[:, 12:] == -5).all()
    before = wide.clone()
    for n in ("parent_rows", "child_rows", "copy_pairs"):
        kw[n] = kw[n][:0]
    kda.fork_blocks(**kw)
    torch.cuda.synchronize()
    assert torch.equal(wide, before)


# ---- releases, compaction ------------------------------------------------------

def held_case(rows, width, N, seed=0, null=0, fill=0.6, released=0.3,
              pinned=False, device=DEV):
    rng = np.random.RandomState(seed)
    held = rng.randint(-1, width + 2, size=rows)
    pool = null + 1 + rng.permutation(max(N - null - 1, 1))[
        :max(1, int(fill * (N - null - 1)))]
    table = rng.choice(pool, size=(rows, width))       # shared at will
    table[rng.rand(rows, width) < 0.05] = null
    table[rng.rand(rows, width) < 0.02] = N + 3
    out = np.flatnonzero(rng.rand(rows) < released)
    out = np.concatenate([out, out[:2], [-1, rows]])   # twice, out of range
    pin = np.where(rng.rand(N) < 0.1, rng.randint(-2, 4, size=N), 0)
    host = dict(released_rows=out, block_table=table, num_blocks=held,
                null_block_id=null)
    if pinned:
        host["pinned"] = pin
    kw = {k: i32(v, device) if isinstance(v, np.ndarray) else v
          for k, v in host.items()}
    z = lambda *n: torch.full(n, -9, dtype=I32, device=device)  # noqa: E731
    kw.update(new_num_blocks=z(rows), ref_counts=z(N), free_blocks=z(N),
              num_free=z(1), workspace=torch.full(
                  (kda.blocks_workspace_size(N),), 255, dtype=torch.uint8,
                  device=device))
    return kw, dict(host, total_blocks=N)


HELD = [
    dict(rows=1, width=1, N=2),
    dict(rows=3, width=4, N=1),
    dict(rows=9, width=6, N=64, pinned=True),
    dict(rows=5, width=300, N=4095, null=3),
    dict(rows=50, width=30, N=4096, fill=0.1),
    dict(rows=400, width=33, N=4097 + 8192, pinned=True),
    dict(rows=30, width=7, N=9000, released=1.0),
    dict(rows=30, width=7, N=40, released=0.0, fill=1.0),
    dict(rows=600, width=40, N=100000, fill=0.9),
    # around what one workgroup takes
    dict(rows=40, width=9, N=16384, fill=0.02),
    dict(rows=40, width=9, N=16385, fill=0.02, null=3),
    dict(rows=4097, width=2, N=300, pinned=True),
    dict(rows=256, width=256, N=5000),
    dict(rows=257, width=256, N=5000, released=0.9),
]


def compaction(kw, max_pairs):
    N = kw["ref_counts"].shape[0]
    z = lambda *n: torch.full(n, -9, dtype=I32, device=DEV)  # noqa: E731
    return dict(ref_counts=kw["ref_counts"], block_table=kw["block_table"],
                num_blocks=kw["new_num_blocks"],
                new_block_table=z(*kw["block_table"].shape),
                new_ref_counts=z(N), copy_pairs=z(max_pairs, 2),
                num_pairs=z(1), workspace=kw["workspace"],
                null_block_id=kw["null_block_id"])


@pytest.mark.gpu
@pytest.mark.parametrize("ci", range(len(HELD)))
def test_release_then_compaction(ci):
    kw, host = held_case(seed=ci, **HELD[ci])
    ref = oracle.free_blocks(**host)
    kda.free_blocks(**kw)
    torch.cuda.synchronize()
    same(kw, ref)
    N = host["total_blocks"]
    for most in (N // 2, 5, 0, N + 30):
        kc = compaction(kw, most)
        want = oracle.compact_blocks(
            ref_counts=ref["ref_counts"], block_table=host["block_table"],
            num_blocks=ref["new_num_blocks"], max_pairs=most,
            null_block_id=host["null_block_id"])
        kda.compact_blocks(**kc)
        torch.cuda.synchronize()
        same(kc, want)
    n = int((ref["ref_counts"] > 0).sum())
    first = host["null_block_id"] + 1
    live = np.flatnonzero(want["new_ref_counts"][first:] > 0)
    assert np.array_equal(live, np.arange(n))


@pytest.mark.gpu
def test_outputs_in_place():
    kw, host = held_case(70, 9, 500, seed=8)
    ref = oracle.free_blocks(**host)
    kw["new_num_blocks"] = kw["num_blocks"]
    kda.free_blocks(**kw)
    torch.cuda.synchronize()
    same(kw, ref)
    kc = compaction(kw, 250)
    kc["new_block_table"] = kc["block_table"]
    kc["new_ref_counts"] = kc["ref_counts"]
    want = oracle.compact_blocks(
        ref_counts=ref["ref_counts"], block_table=host["block_table"],
        num_blocks=ref["new_num_blocks"], max_pairs=250)
    kda.compact_blocks(**kc)
    torch.cuda.synchronize()
    same(kc, want)


@pytest.mark.gpu
def test_counts_that_miss_references_move_nothing_wrong():
    """Held blocks that ref_counts does not know stay where they are."""
    kw, host = held_case(20, 9, 300, seed=4)
    refs = oracle.free_blocks(**host)["ref_counts"]
    refs[np.flatnonzero(refs)[::2]] = 0
    kw["ref_counts"] = i32(refs)
    kw["new_num_blocks"] = kw["num_blocks"]
    kc = compaction(kw, 150)
    want = oracle.compact_blocks(ref_counts=refs,
                                 block_table=host["block_table"],
                                 num_blocks=host["num_blocks"], max_pairs=150)
    kda.compact_blocks(**kc)
    torch.cuda.synchronize()
    same(kc, want)


@pytest.mark.gpu
def test_graph_of_release_compaction_and_copies():
    """The three as a server runs them, replayed while requests end."""
    N, rows, width = 300, 24, 8
    rng = np.random.RandomState(2)
    pool = torch.randn((N, 33), device=DEV)
    copier = kda.BlockPools([pool])
    ids = rng.permutation(np.arange(1, N))[:rows * width].reshape(rows, width)
    table, held = i32(ids), i32(rng.randint(1, width + 1, size=rows))
    text = {r: pool[table[r, :int(held[r])].long()].clone()
            for r in range(rows)}
    kw, _ = held_case(rows, width, N)
    kw.update(block_table=table, num_blocks=held, new_num_blocks=held,
              released_rows=i32([-1, -1]))
    kc = compaction(kw, N // 2)
    kc.update(new_block_table=table)

    def step():
        kda.free_blocks(**kw)
        kda.compact_blocks(**kc)
        copier.copy(kc["copy_pairs"], kc["num_pairs"])

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for k in range(4):
        out = [2 * k, 2 * k + 9]
        kw["released_rows"].copy_(i32(out))
        graph.replay()
        torch.cuda.synchronize()
        for r in out:
            text.pop(r, None)
        n = int((kc["new_ref_counts"] > 0).sum())
        for r, want in text.items():
            at = table[r, :int(held[r])].long()
            assert int(at.max()) <= n
            assert torch.equal(pool[at], want)


# ---- refusals -------------------------------------------------------------------

def test_copy_refusals():
    page, ps = pools(8, device="cpu")
    ok = i32([[1, 2]], "cpu")
    bp = kda.BlockPools(ps)
    assert bp.check(ok) == _abi.KDA_OK
    with pytest.raises(ValueError, match="GPU"):
        bp.copy(ok)
    with pytest.raises(TypeError):
        bp.check(ok.long())
    with pytest.raises(ValueError):
        bp.check(ok[0])
    with pytest.raises(ValueError, match="one piece"):
        kda.BlockPools([page[:, ::2]])
    with pytest.raises(ValueError, match="as the first"):
        kda.BlockPools([ps[0], ps[1][:4]])
    with pytest.raises(ValueError):
        kda.BlockPools([])
    shared = kda.BlockPools([page[:1].expand(8, -1)])
    assert shared.check(ok) == _abi.KDA_E_LAYOUT
    lib = _abi.load()
    assert lib.kda_check_copy_blocks(None) == _abi.KDA_E_ARG
    for name, value in (("tables", None), ("copy_pairs", None),
                        ("num_pools", 0), ("max_pairs", -1),
                        ("null_block_id", -1)):
        a = bp.args(ok)
        setattr(a, name, value)
        assert lib.kda_check_copy_blocks(a) == _abi.KDA_E_ARG, name


def test_fork_refusals():
    ok, _ = fork_case(3, 8, 4, 4, device="cpu")
    chk = lambda **d: kda.check_fork_blocks(**dict(ok, **d))  # noqa: E731
    assert chk() == _abi.KDA_OK
    with pytest.raises(ValueError, match="GPU"):
        kda.fork_blocks(**ok)
    assert chk(block_size=0) == _abi.KDA_E_ARG
    assert chk(null_block_id=-1) == _abi.KDA_E_ARG
    assert chk(block_table=ok["block_table"][:1].expand(8, -1)) == \
        _abi.KDA_E_LAYOUT
    with pytest.raises(ValueError, match="pair per fork"):
        chk(copy_pairs=ok["copy_pairs"][:2])
    with pytest.raises(ValueError, match="entries"):
        chk(child_rows=ok["child_rows"][:2])
    with pytest.raises(ValueError, match="entries"):
        chk(num_blocks=ok["num_blocks"][:7])
    lib = _abi.load()
    assert lib.kda_check_fork_blocks(None) == _abi.KDA_E_ARG
    for name in ("parent_rows", "num_blocks", "block_table", "free_blocks",
                 "num_allocated"):
        a = kda.fork_args(**ok)
        setattr(a, name, None)
        assert lib.kda_check_fork_blocks(a) == _abi.KDA_E_ARG, name


def test_free_and_compact_refusals(monkeypatch):
    ok, _ = held_case(6, 4, 30, device="cpu")
    chk = lambda **d: kda.check_free_blocks(**dict(ok, **d))  # noqa: E731
    assert chk() == _abi.KDA_OK
    with pytest.raises(ValueError, match="GPU"):
        kda.free_blocks(**ok)
    assert chk(workspace=ok["workspace"][:-4]) == _abi.KDA_E_CAPACITY
    assert chk(null_block_id=-1) == _abi.KDA_E_ARG
    with pytest.raises(ValueError, match="entries"):
        chk(free_blocks=ok["free_blocks"][:29])
    with pytest.raises(ValueError, match="entries"):
        chk(pinned=ok["free_blocks"][:29])
    with pytest.raises(ValueError):
        kda.blocks_workspace_size(1 << 40)
    lib = _abi.load()
    assert lib.kda_check_free_blocks(None) == _abi.KDA_E_ARG
    for name in ("num_blocks", "ref_counts", "num_free", "workspace",
                 "new_num_blocks", "block_table"):
        a = kda.free_args(**ok)
        setattr(a, name, None)
        assert lib.kda_check_free_blocks(a) == _abi.KDA_E_ARG, name

    monkeypatch.setattr("tests.test_gpu_blocks.DEV", "cpu")
    kc = compaction(ok, 15)
    chk = lambda **d: kda.check_compact_blocks(**dict(kc, **d))  # noqa: E731
    assert chk() == _abi.KDA_OK
    with pytest.raises(ValueError, match="GPU"):
        kda.compact_blocks(**kc)
    assert chk(workspace=ok["workspace"][:8]) == _abi.KDA_E_CAPACITY
    assert chk(new_block_table=kc["new_block_table"][:1].expand(6, -1)) == \
        _abi.KDA_E_LAYOUT
    with pytest.raises(ValueError, match="one size"):
        chk(new_block_table=kc["new_block_table"][:, :3])
    assert lib.kda_check_compact_blocks(None) == _abi.KDA_E_ARG
    for name in ("ref_counts", "new_ref_counts", "num_pairs", "copy_pairs",
                 "workspace", "new_block_table"):
        a = kda.compact_blocks_args(**kc)
        setattr(a, name, None)
        assert lib.kda_check_compact_blocks(a) == _abi.KDA_E_ARG, name
