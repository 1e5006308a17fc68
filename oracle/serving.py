"""fp64 reference for the operators around the verify in a serving step: the
KDA layer over prompts and single tokens, the step's index tables, and
sampling with draft acceptance.  TEST INFRASTRUCTURE ONLY (see the package
docstring); written token by token and request by request from the
definitions, out of the pieces in `oracle.kda`.
"""
from __future__ import annotations

import numpy as np

from .kda import (conv_update, delta_step, kda_gate, normalize_query)


def _live(slot, null_block_id, N):
    return null_block_id < slot < N


def layer_tokens(*, mixed_qkv, raw_gate, raw_beta, A_log, dt_bias, state,
                 out, query_start_loc, state_indices, initial_state_indices,
                 conv_state=None, conv_weight=None, num_accepted_tokens=None,
                 use_lower_bound=False, lower_bound=0.0, null_block_id=0):
    """The KDA layer over each request's tokens, from its initial slot (zeros
    when null) to its state slot.

    Arrays are float64 (exact widenings); `conv_state` is the dim-first view
    [N, 3HK, Lc], or None for convolved q | k | v.  Returns dict(out, state,
    conv_state) of updated copies.  A request without tokens changes nothing;
    one whose state slot is null gets zero outputs.
    """
    N, H, V, K = state.shape
    HK = H * K
    dt_bias = np.asarray(dt_bias, np.float64).reshape(H, K)
    A = np.exp(np.asarray(A_log, np.float64))[:, None]
    out, new = np.array(out, np.float64), np.array(state, np.float64)
    conv = None if conv_state is None else np.array(conv_state)
    T = out.shape[0]
    for b in range(len(state_indices)):
        bos = min(max(int(query_start_loc[b]), 0), T)
        eos = min(max(int(query_start_loc[b + 1]), bos), T)
        if eos == bos:
            continue
        dst = int(state_indices[b])
        if not _live(dst, null_block_id, N):
            out[bos:eos] = 0.0
            continue
        src = null_block_id if initial_state_indices is None \
            else int(initial_state_indices[b])
        live = _live(src, null_block_id, N)
        x = np.asarray(mixed_qkv[bos:eos], np.float64)
        if conv is not None:
            Lc = conv.shape[2]
            a = 1 if num_accepted_tokens is None \
                else min(max(int(num_accepted_tokens[b]), 1), Lc - 2)
            # a slot wide enough for the whole prompt, its history in front
            wide = np.zeros((3 * HK, (eos - bos) + 2 + Lc))
            if live:
                wide[:, :3] = conv_state[src][:, a - 1:a + 2]
            raw = np.concatenate([wide[:, :3], x.T], axis=1)
            x, _ = conv_update(wide, x, conv_weight, 1)
            conv[dst][:, :3] = raw[:, -3:]
        S = np.asarray(state[src], np.float64) if live \
            else np.zeros((H, V, K))
        for t in range(eos - bos):
            q, k, v = (x[t, i * HK:(i + 1) * HK].reshape(H, K)
                       for i in range(3))
            g = kda_gate(raw_gate[bos + t].reshape(H, K), dt_bias, A,
                         use_lower_bound, lower_bound)
            S, _ = delta_step(S, k, v, g, raw_beta[bos + t])
            out[bos + t] = np.einsum("hvk,hk->hv", S,
                                     normalize_query(q)).reshape(-1)
        new[dst] = S
    return dict(out=out, state=new, conv_state=conv)


def step_tables(*, query_lens, num_computed_tokens, num_blocks, block_table,
                free_blocks, block_size, max_tokens, request_indices=None,
                null_block_id=0):
    """A step's index arrays, request by request.  Returns a dict of int64
    arrays named as the library's outputs, `block_table` among them."""
    table = np.array(block_table, np.int64)
    held = np.array(num_blocks, np.int64)
    rows, width = table.shape
    B, used, tok = len(query_lens), 0, 0
    r = dict(query_start_loc=np.zeros(B + 1, np.int64),
             state_indices=np.full(B, null_block_id, np.int64),
             initial_state_indices=np.full(B, null_block_id, np.int64),
             final_state_indices=np.full(B, null_block_id, np.int64),
             positions=np.zeros(max_tokens, np.int64),
             slot_mapping=np.full(max_tokens, -1, np.int64))
    for b in range(B):
        row = b if request_indices is None else int(request_indices[b])
        q = max(int(query_lens[b]), 0)
        ok = 0 <= row < rows
        c = max(int(num_computed_tokens[row]), 0) if ok else 0

        def block(position):
            i = position // block_size
            return int(table[row, i]) if ok and i < width else null_block_id

        if ok:
            have = min(max(int(held[row]), 0), width)
            held[row] = have
            for i in range(have, min((c + q) // block_size + 1, width)):
                table[row, i] = null_block_id
                if used < len(free_blocks):
                    table[row, i] = free_blocks[used]
                    held[row] += 1
                used += 1
        r["state_indices"][b] = block(c)
        if c > 0:
            r["initial_state_indices"][b] = block(c)
        r["final_state_indices"][b] = block(c + q)
        for t in range(q):
            if tok + t < max_tokens:
                r["positions"][tok + t] = c + t
                if block(c + t) > null_block_id:
                    r["slot_mapping"][tok + t] = \
                        block(c + t) * block_size + (c + t) % block_size
        tok += q
        r["query_start_loc"][b + 1] = min(tok, max_tokens)
    r.update(block_table=table, new_num_blocks=held,
             num_allocated=np.array([used]))
    return r


def sample_row(x, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """Token of one row of logits [V] (float64), from the definition: weights
    e^((x - max) / T) rounded to the documented binary places and summed as
    Python integers, the order by falling value and rising index, the three
    prefixes, and the running sum by index."""
    x = np.where(np.isnan(x), -np.inf, np.asarray(x, np.float64))
    V, top = len(x), np.max(x)
    if top == -np.inf:
        return -1
    T = 1.0 if np.isnan(temperature) else float(temperature)
    if T <= 0:
        return int(np.argmax(x))
    places = min(46, 62 - max(0, (V - 1).bit_length()))
    with np.errstate(invalid="ignore", over="ignore"):
        w = np.where(x == top, 1.0, np.exp((x - top) / T))
    w[(x == -np.inf) | np.isnan(w)] = 0.0
    order = np.argsort(-x, kind="stable")
    kept = [i for i in order if x[i] > -np.inf and w[i] > 0]
    if min_p > 0:
        kept = [i for i in kept if w[i] >= min(min_p, 1.0)]
    if top_k > 0:
        kept = kept[:top_k]
    whole = {i: int(np.rint(np.ldexp(w[i], places))) for i in kept}
    if top_p < 1:
        need, have, n = float(top_p) * float(sum(whole.values())), 0, 0
        while n == 0 or have < need:
            have += whole[kept[n]]
            n += 1
        kept = kept[:n]
    kept = sorted(kept)
    limit = float(max(u, 0.0)) * float(sum(whole[i] for i in kept))
    have = 0
    for i in kept:
        have += whole[i]
        if have > limit:
            return int(i)
    return int(kept[-1])


def accept_drafts(tokens, draft_tokens, query_start_loc):
    """(accepted counts, next tokens) of draft windows, row by row."""
    accepted, following = [], []
    for s, e in zip(query_start_loc[:-1], query_start_loc[1:]):
        if e <= s:
            accepted.append(0)
            following.append(-1)
            continue
        t = s
        while t + 1 < e and tokens[t] == draft_tokens[t + 1]:
            t += 1
        accepted.append(t - s + 1)
        following.append(tokens[t])
    return np.array(accepted), np.array(following)
