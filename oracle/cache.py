"""fp64 reference for the operators on token caches.  TEST INFRASTRUCTURE ONLY
(see the package docstring); written request by request from the definitions.
"""
from __future__ import annotations

import numpy as np


def latent_write(*, latent, rope_key, cache, slot_mapping, null_block_id=0):
    """Updated copy of the cache [N, block_size, R + P] (any dtype)."""
    new = np.array(cache)
    N, bs = new.shape[:2]
    for t in range(len(latent)):
        blk, at = divmod(int(slot_mapping[t]), bs)
        if null_block_id < blk < N:
            row = [latent[t]] if rope_key is None else [latent[t],
                                                        rope_key[t]]
            new[blk, at] = np.concatenate(row)
    return new


def places(*, row, length, block_table, block_size, num_blocks,
           null_block_id=0):
    """(block, slot) of a request row's first `length` positions, None for
    those of null blocks or past the table."""
    rows, width = block_table.shape
    got = []
    for j in range(length):
        e, at = divmod(j, block_size)
        blk = int(block_table[row, e]) if 0 <= row < rows and e < width \
            else null_block_id
        got.append((blk, at) if null_block_id < blk < num_blocks else None)
    return got


def softmax_sum(q, k, v, see, scale):
    """One head: q [t, w], k [n, w], v [n, d], see [t, n].  Returns out [t, d],
    lse [t], the weighted magnitudes sum_j p_j |v_j| [t, d], and the largest
    sum of magnitudes behind a score, scale * sum_k |q_k k_jk| [t]."""
    s = np.where(see, (q @ k.T) * scale, -np.inf)
    top = s.max(axis=1, initial=-np.inf)
    safe = np.where(np.isfinite(top), top, 0.0)
    p = np.where(see, np.exp(s - safe[:, None]), 0.0)
    total = p.sum(axis=1)
    p /= np.where(total > 0, total, 1.0)[:, None]
    with np.errstate(divide="ignore"):
        lse = np.log(total) + safe
    size = np.where(see, (np.abs(q) @ np.abs(k).T) * abs(scale), 0.0)
    return p @ v, lse, p @ np.abs(v), size.max(axis=1, initial=0.0)


def latent_attention(*, q, cache, out, lse, query_start_loc,
                     num_computed_tokens, block_table, softmax_scale,
                     latent_dim, request_indices=None, null_block_id=0):
    """Absorbed attention over the paged cache.  Returns dict(out, lse) of
    updated copies, and for bounds on errors `weight` (like out), `size` and
    `keys` (like lse)."""
    T, H, _ = q.shape
    R, (N, bs) = latent_dim, cache.shape[:2]
    out, lse = np.array(out, np.float64), np.array(lse, np.float64)
    weight, size, keys = (np.zeros_like(out), np.zeros_like(lse),
                          np.zeros_like(lse))
    rows = block_table.shape[0]
    for b in range(len(query_start_loc) - 1):
        bos = min(max(int(query_start_loc[b]), 0), T)
        eos = min(max(int(query_start_loc[b + 1]), bos), T)
        row = b if request_indices is None else int(request_indices[b])
        ok = 0 <= row < rows
        c = max(int(num_computed_tokens[row]), 0) if ok else 0
        at = places(row=row, length=c + eos - bos, block_table=block_table,
                    block_size=bs, num_blocks=N,
                    null_block_id=null_block_id) if ok else []
        pos = np.array([j for j, p in enumerate(at) if p], np.int64)
        e = np.array([cache[at[j]] for j in pos], np.float64).reshape(
            len(pos), cache.shape[2])
        see = pos[None] <= (c + np.arange(eos - bos))[:, None]
        for h in range(H):
            r = softmax_sum(q[bos:eos, h].astype(np.float64), e, e[:, :R],
                            see, softmax_scale)
            out[bos:eos, h], lse[bos:eos, h] = r[0], r[1]
            weight[bos:eos, h], size[bos:eos, h] = r[2], r[3]
            keys[bos:eos, h] = see.sum(axis=1)
    return dict(out=out, lse=lse, weight=weight, size=size, keys=keys)


def latent_expand(*, cache, weight, key, rope_key, value, key_start_loc,
                  block_table, request_indices=None, null_block_id=0):
    """Updated copies of key, value, rope_key (or None), and for bounds the
    sums of magnitudes behind keys and values (`key_size`, `value_size`)."""
    key, value = np.array(key, np.float64), np.array(value, np.float64)
    rope = None if rope_key is None else np.array(rope_key, np.float64)
    S, H, D = key.shape
    R = weight.shape[2]
    N, bs = cache.shape[:2]
    ks, vs = np.zeros_like(key), np.zeros_like(value)
    for b in range(len(key_start_loc) - 1):
        bos = min(max(int(key_start_loc[b]), 0), S)
        eos = min(max(int(key_start_loc[b + 1]), bos), S)
        row = b if request_indices is None else int(request_indices[b])
        at = places(row=row, length=eos - bos, block_table=block_table,
                    block_size=bs, num_blocks=N, null_block_id=null_block_id)
        for j, p in enumerate(at):
            e = np.zeros(cache.shape[2]) if p is None \
                else np.asarray(cache[p], np.float64)
            kv = weight @ e[:R]
            size = np.abs(weight) @ np.abs(e[:R])
            key[bos + j], value[bos + j] = kv[:, :D], kv[:, D:]
            ks[bos + j], vs[bos + j] = size[:, :D], size[:, D:]
            if rope is not None:
                rope[bos + j] = e[R:]
    return dict(key=key, value=value, rope_key=rope, key_size=ks,
                value_size=vs)


def latent_prefill(*, q, key, value, out, lse, query_start_loc,
                   key_start_loc, softmax_scale, rope_key=None):
    """As `latent_attention`, over expanded keys and values."""
    T, H, _ = q.shape
    S = key.shape[0]
    out, lse = np.array(out, np.float64), np.array(lse, np.float64)
    weight, size, keys = (np.zeros_like(out), np.zeros_like(lse),
                          np.zeros_like(lse))
    for b in range(len(query_start_loc) - 1):
        bos = min(max(int(query_start_loc[b]), 0), T)
        eos = min(max(int(query_start_loc[b + 1]), bos), T)
        ka = min(max(int(key_start_loc[b]), 0), S)
        ke = min(max(int(key_start_loc[b + 1]), ka), S)
        n, t = ke - ka, eos - bos
        see = np.arange(n)[None] <= (n - t + np.arange(t))[:, None]
        for h in range(H):
            k = np.asarray(key[ka:ke, h], np.float64)
            if rope_key is not None:
                k = np.concatenate([k, rope_key[ka:ke]], axis=1)
            r = softmax_sum(np.asarray(q[bos:eos, h], np.float64), k,
                            np.asarray(value[ka:ke, h], np.float64), see,
                            softmax_scale)
            out[bos:eos, h], lse[bos:eos, h] = r[0], r[1]
            weight[bos:eos, h], size[bos:eos, h] = r[2], r[3]
            keys[bos:eos, h] = see.sum(axis=1)
    return dict(out=out, lse=lse, weight=weight, size=size, keys=keys)


def adjust_logits(*, logits, query_start_loc=None, draft_tokens=None,
                  request_indices=None, token_ids=None, prompt_lens=None,
                  token_lens=None, repetition_penalty=None,
                  frequency_penalty=None, presence_penalty=None,
                  bias_start=None, bias_tokens=None, bias_values=None,
                  mask=None, mask_rows=None):
    """Changed copy of the logits [M, V], and the sums of magnitudes behind
    its entries (for bounds)."""
    y = np.array(logits, np.float64)
    size = np.abs(y)
    M, V = y.shape
    B = M if query_start_loc is None else len(query_start_loc) - 1

    def param(a, b, none):
        return none if a is None or np.isnan(a[b]) else float(a[b])

    for b in range(B):
        s, e = (b, b + 1) if query_start_loc is None else (
            min(max(int(query_start_loc[b]), 0), M),
            min(max(int(query_start_loc[b + 1]), 0), M))
        r = param(repetition_penalty, b, 1.0)
        r = r if r > 0 else 1.0
        f, p = (param(a, b, 0.0) for a in (frequency_penalty,
                                           presence_penalty))
        count, seen = np.zeros(V, np.int64), np.zeros(V, bool)
        if token_ids is not None:
            row = b if request_indices is None else int(request_indices[b])
            if 0 <= row < len(token_ids):
                n = min(max(int(token_lens[row]), 0), token_ids.shape[1])
                for i in range(n):
                    t = int(token_ids[row, i])
                    if 0 <= t < V:
                        seen[t] = True
                        count[t] += i >= prompt_lens[row]
        bias = {}
        if bias_start is not None:
            lo = max(int(bias_start[b]), 0)
            hi = min(int(bias_start[b + 1]), len(bias_tokens))
            for i in range(lo, hi):
                bias[int(bias_tokens[i])] = float(bias_values[i])
        for m in range(s, e):
            if m > s and draft_tokens is not None:
                t = int(draft_tokens[m])
                if 0 <= t < V:
                    seen[t] = True
                    count[t] += 1
            for t, v in bias.items():
                if 0 <= t < V:
                    y[m, t] += v
                    size[m, t] += abs(v)
            for t in np.flatnonzero(seen):
                by = 1 / r if y[m, t] > 0 else r
                y[m, t] *= by
                size[m, t] *= by
                if count[t]:
                    y[m, t] -= f * count[t] + p
                    size[m, t] += abs(f) * count[t] + abs(p)
            mr = -1 if mask is None else m if mask_rows is None \
                else int(mask_rows[m])
            if mask is not None and 0 <= mr < len(mask):
                words = np.asarray(mask[mr]).astype(np.int64)
                bits = (words[np.arange(V) // 32] >> (np.arange(V) % 32)) & 1
                y[m, bits == 0] = -np.inf
    return y, size


def copy_blocks(pools, pairs, num_pairs=None, null_block_id=0):
    """Updated copies of the pools [N, ..]."""
    new = [np.array(p) for p in pools]
    n = len(pairs) if num_pairs is None else min(max(int(num_pairs), 0),
                                                 len(pairs))
    for src, dst in np.asarray(pairs)[:n]:
        for old, pool in zip(pools, new):
            if null_block_id < src < len(old) and \
                    null_block_id < dst < len(old):
                pool[dst] = old[src]
    return new


def fork_blocks(*, parent_rows, child_rows, num_computed_tokens, num_blocks,
                block_table, free_blocks, block_size, null_block_id=0):
    table, held, comp = (np.array(a) for a in (block_table, num_blocks,
                                               num_computed_tokens))
    rows, width = table.shape
    pairs = np.full((len(parent_rows), 2), null_block_id)
    free, asked = list(free_blocks), 0
    for f, (a, b) in enumerate(zip(parent_rows, child_rows)):
        if not (0 <= a < rows and 0 <= b < rows) or a == b or width == 0:
            continue
        c = max(int(num_computed_tokens[a]), 0)
        k = c // block_size
        table[b, :k] = block_table[a, :k]
        if k < width:
            new = int(free[asked]) if asked < len(free) else null_block_id
            asked += 1
            table[b, k] = new
            if k < num_blocks[a] and new > null_block_id and \
                    block_table[a, k] > null_block_id:
                pairs[f] = block_table[a, k], new
        comp[b], held[b] = c, min(k + 1, width)
    return dict(block_table=table, num_blocks=held, num_computed_tokens=comp,
                copy_pairs=pairs, num_allocated=np.array([asked]))


def free_blocks(*, released_rows, block_table, num_blocks, total_blocks,
                pinned=None, null_block_id=0):
    rows, width = block_table.shape
    held = np.clip(num_blocks, 0, width)
    for r in released_rows:
        if 0 <= r < rows:
            held[r] = 0
    refs = np.zeros(total_blocks, np.int64) if pinned is None \
        else np.maximum(pinned, 0)
    for r in range(rows):
        for b in block_table[r, :held[r]]:
            if null_block_id < b < total_blocks:
                refs[b] += 1
    free = [i for i in range(null_block_id + 1, total_blocks) if refs[i] == 0]
    listed = np.full(total_blocks, null_block_id)
    listed[:len(free)] = free
    return dict(new_num_blocks=held, ref_counts=refs, free_blocks=listed,
                num_free=np.array([len(free)]))


def compact_blocks(*, ref_counts, block_table, num_blocks, max_pairs,
                   null_block_id=0):
    N = len(ref_counts)
    live = [i for i in range(null_block_id + 1, N) if ref_counts[i] > 0]
    end = null_block_id + 1 + len(live)
    src = [i for i in live if i >= end]
    dst = [i for i in range(null_block_id + 1, min(end, N))
           if ref_counts[i] <= 0]
    moves = list(zip(src, dst))[:max_pairs]
    to = dict(moves)
    refs, table = np.array(ref_counts), np.array(block_table)
    for a, b in moves:
        refs[b], refs[a] = ref_counts[a], 0
    for r in range(len(table)):
        for j in range(min(max(int(num_blocks[r]), 0), table.shape[1])):
            table[r, j] = to.get(int(table[r, j]), table[r, j])
    pairs = np.full((max_pairs, 2), null_block_id)
    if moves:
        pairs[:len(moves)] = moves
    return dict(new_ref_counts=refs, new_block_table=table, copy_pairs=pairs,
                num_pairs=np.array([len(moves)]))
