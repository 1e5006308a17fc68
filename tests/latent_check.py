"""Inputs of the latent attention tests, and their tolerances."""
import numpy as np
import torch

ACT = {"f32": torch.float32, "bf16": torch.bfloat16}
I32 = torch.int32


def f64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def ints(t):
    return t.cpu().numpy().astype(np.int64)


def paged(lens, computed, *, rows=None, block, spare=3, null=0, seed=0,
          device="cuda", rows_of=None):
    """Offsets, rows and a block table for windows of `lens` tokens behind
    `computed` ones; ids scattered over N blocks."""
    rng = np.random.RandomState(seed)
    B = len(lens)
    rows = rows or B + 2
    total = np.asarray(lens) + np.asarray(computed)
    need = -(-total // block)
    N = null + 1 + int(need.sum()) + spare
    ids = null + 1 + rng.permutation(N - null - 1)
    req = rng.permutation(rows)[:B]
    table = np.full((rows, max(int(need.max(initial=0)), 1) + 1), null)
    comp = rng.randint(0, 5, size=rows)
    at = 0
    for b in range(B):
        table[req[b], :need[b]] = ids[at:at + need[b]]
        comp[req[b]] = computed[b]
        at += need[b]
    to = lambda a: torch.as_tensor(np.asarray(a), dtype=I32).to(device)  # noqa: E731
    return dict(query_start_loc=to(np.concatenate([[0], np.cumsum(lens)])),
                num_computed_tokens=to(comp), request_indices=to(req),
                block_table=to(table)), N


def make(lens, computed, *, H, R, P, block, act, seed=0, null=0, tail=0,
         device="cuda", gap=0):
    """Arguments of a latent attention, lse included and the workspace left
    out; `tail` rows behind the last sequence, `gap` unused bytes around rows
    of q, cache and out; unused cache places hold NaN."""
    kw, N = paged(lens, computed, block=block, null=null, seed=seed,
                  device=device)
    g = torch.Generator().manual_seed(seed)
    dt, T, W = ACT[act], int(np.sum(lens)) + tail, R + P

    def randn(*shape):
        if not gap:
            return torch.randn(shape, generator=g).to(dt).to(device)
        wide = torch.randn(*shape[:-2], shape[-2] + 1, shape[-1] + 16 * gap,
                           generator=g).to(dt).to(device)
        return wide[..., :shape[-2], :shape[-1]]

    kw["q"] = randn(T, H, W)
    kw["cache"] = randn(N, block, W)
    kw["out"] = randn(T, H, R)
    kw["lse"] = torch.full((T, H), 7.0, device=device)
    kw.update(softmax_scale=W ** -0.5, null_block_id=null)
    used = torch.zeros(N, block, dtype=torch.bool)
    table, req = ints(kw["block_table"]), ints(kw["request_indices"])
    for b in range(len(lens)):
        for j in range(lens[b] + computed[b]):
            used[table[req[b], j // block], j % block] = True
    kw["cache"].masked_fill_(~used[..., None].to(device), float("nan"))
    return kw


def bounds(ref, act, dims):
    """Largest errors of (out, lse) by arithmetic.  A score is an fp32 sum of
    `dims` products: off by dims steps of 2^-24 of the sum of magnitudes
    behind it (`size`; two more for the scale and its product with log2 e),
    and its weight by that much relatively, as is the sum of the weights.
    exp2 and its argument take 4 steps, the sums over the keys one each.  With
    bf16, weights and outputs are rounded to half a step, 2^-8."""
    u = 2.0 ** -24
    score = (dims + 4) * u * ref["size"]
    # weights reach 2^-126 relative to the largest: below, they are nothing
    rel = 2 * (np.expm1(score) + (ref["keys"] + 8) * u)
    if act == "bf16":
        rel = rel + 2.0 ** -8
    out = rel[..., None] * ref["weight"] + 1e-30
    out = out + (2.0 ** -8 if act == "bf16" else 2 * u) * (
        np.abs(ref["out"]) + out)
    lse = score + (ref["keys"] + 8) * u + 4 * u * np.abs(
        np.where(np.isfinite(ref["lse"]), ref["lse"], 0.0))
    return out, lse


def hold(got, want, bound, what):
    fin = np.isfinite(want)
    assert np.array_equal(got[~fin], want[~fin], equal_nan=True), what
    off = np.abs(got[fin] - want[fin])
    assert (off <= bound[fin]).all(), (
        what, float((off / np.maximum(bound[fin], 1e-300)).max()))
