"""A serving loop over one pool of blocks that a KDA layer's states and a latent
attention layer's cache share: prompts, forks of a request, single tokens and a
draft window, requests that end, compaction, a new prompt on the freed blocks,
and decode steps from a captured graph; against one fp64 pass over each
request's tokens.  The logits' changes and the sampling run on every step."""
import numpy as np
import pytest
import torch

import linear_attention_speculative_amd as kda
import oracle
from tests.gpu_check import TOL
from tests.latent_check import bounds
from tests.layer_check import f64, i32, make_layer, reference

DEV = "cuda"
ROWS, BLOCK, N, WIDTH = 6, 8, 40, 9
H, D, HL, R, P, DL, VOCAB = 2, 32, 5, 128, 64, 64, 97
ONES = dict(dtype=torch.int32, device=DEV)


class Server:
    """Request rows, block tables, the pools of both layers."""

    def __init__(self):
        self.kda = make_layer(1, N, H, D, 1, act="f32", seed=5)
        for n in ("mixed_qkv", "raw_gate", "raw_beta", "out"):
            del self.kda[n]
        self.cache = torch.full((N, BLOCK, R + P), float("nan"), device=DEV)
        self.weight = torch.randn((HL, 2 * DL, R), device=DEV) * R ** -0.5
        self.copier = kda.BlockPools([self.kda["state"],
                                      self.kda["conv_state"], self.cache])
        z = lambda *n: torch.zeros(n, **ONES)  # noqa: E731
        self.computed, self.held, self.table = z(ROWS), z(ROWS), z(ROWS, WIDTH)
        self.refs, self.free, self.num_free = z(N), z(N), z(1)
        self.pairs, self.num_pairs = z(N // 2, 2), z(1)
        self.work = torch.empty(kda.blocks_workspace_size(N),
                                dtype=torch.uint8, device=DEV)
        self.draw = torch.Generator().manual_seed(11)
        self.tokens = z(ROWS, 64)
        self.text = {}                       # row -> that request's tokens
        self.seen = {}                       # row -> its sampled tokens
        self.release([])

    def release(self, rows):
        kda.free_blocks(released_rows=i32(rows, DEV), block_table=self.table,
                        num_blocks=self.held, new_num_blocks=self.held,
                        ref_counts=self.refs, free_blocks=self.free,
                        num_free=self.num_free, workspace=self.work)
        for r in rows:
            self.computed[r] = 0
            del self.text[r], self.seen[r]

    def compact(self):
        kda.compact_blocks(ref_counts=self.refs, new_ref_counts=self.refs,
                           block_table=self.table, num_blocks=self.held,
                           new_block_table=self.table, copy_pairs=self.pairs,
                           num_pairs=self.num_pairs, workspace=self.work)
        self.copier.copy(self.pairs, self.num_pairs)
        self.release([])                     # the free list anew

    def fork(self, parent, children):
        n = int(self.num_free)
        pairs = torch.zeros((len(children), 2), **ONES)
        kda.fork_blocks(
            parent_rows=i32([parent] * len(children), DEV),
            child_rows=i32(children, DEV), num_computed_tokens=self.computed,
            num_blocks=self.held, block_table=self.table,
            free_blocks=self.free[:n], block_size=BLOCK, copy_pairs=pairs,
            num_allocated=torch.zeros(1, **ONES))
        self.copier.copy(pairs)
        self.release([])
        for c in children:
            self.text[c] = [dict(t) for t in self.text[parent]]
            self.seen[c] = list(self.seen[parent])

    def inputs(self, T):
        def randn(*n):
            return torch.randn(n, generator=self.draw).to(DEV)
        return dict(mixed_qkv=randn(T, 3 * H * D), raw_gate=randn(T, H * D),
                    raw_beta=randn(T, H), latent=randn(T, R),
                    rope_key=randn(T, P), q_cat=randn(T, HL, R + P),
                    q_exp=randn(T, HL, DL + P),
                    logits=randn(T, VOCAB), uniform=torch.rand(
                        T, generator=self.draw).to(DEV))

    def tables(self, rows, lens):
        B, T = len(rows), sum(lens)
        z = lambda n, t=torch.int32: torch.zeros(n, dtype=t, device=DEV)  # noqa: E731
        t = dict(query_lens=i32(lens, DEV), num_computed_tokens=self.computed,
                 num_blocks=self.held, new_num_blocks=self.held,
                 block_table=self.table,
                 free_blocks=self.free[:int(self.num_free)],
                 block_size=BLOCK, request_indices=i32(rows, DEV),
                 query_start_loc=z(B + 1), state_indices=z(B),
                 initial_state_indices=z(B), final_state_indices=z(B),
                 positions=z(T), slot_mapping=z(T, torch.int64),
                 num_allocated=z(1))
        return t

    def layers(self, t, x, lens, prompt):
        """Both layers on a step's tokens; outputs by layer."""
        T, B = x["latent"].shape[0], len(lens)
        y = dict(kda=torch.zeros((T, H * D), device=DEV),
                 lat=torch.zeros((T, HL, DL if prompt else R), device=DEV),
                 lse=torch.zeros((T, HL), device=DEV))
        act = {k: x[k] for k in ("mixed_qkv", "raw_gate", "raw_beta")}
        kda.latent_write(latent=x["latent"], rope_key=x["rope_key"],
                         cache=self.cache, slot_mapping=t["slot_mapping"])
        if prompt:
            kda.conv_prefill(
                **self.kda, **act, out=y["kda"],
                query_start_loc=t["query_start_loc"],
                state_indices=t["final_state_indices"],
                initial_state_indices=t["initial_state_indices"],
                workspace=torch.empty(kda.prefill_workspace_size(
                    T, B, H, D, torch.float32), dtype=torch.uint8,
                    device=DEV))
            before = self.computed[t["request_indices"].long()]
            ends = torch.cumsum(before + t["query_lens"], 0)
            kloc = torch.cat([ends[:1] * 0, ends]).to(torch.int32)
            S = int(kloc[-1])
            key = torch.zeros((S, HL, DL), device=DEV)
            value, rope = torch.zeros_like(key), torch.zeros((S, P),
                                                             device=DEV)
            kda.latent_expand(cache=self.cache, weight=self.weight, key=key,
                              value=value, rope_key=rope, key_start_loc=kloc,
                              block_table=self.table,
                              request_indices=t["request_indices"])
            kda.latent_prefill(q=x["q_exp"], key=key, value=value,
                               rope_key=rope, out=y["lat"], lse=y["lse"],
                               query_start_loc=t["query_start_loc"],
                               key_start_loc=kloc, softmax_scale=0.1)
        else:
            if max(lens) == 1:
                kda.conv_update_decode(
                    **self.kda, **act, out=y["kda"],
                    state_indices=t["state_indices"],
                    final_state_indices=t["final_state_indices"])
            kda.latent_attention(
                q=x["q_cat"], cache=self.cache, out=y["lat"], lse=y["lse"],
                query_start_loc=t["query_start_loc"],
                num_computed_tokens=self.computed,
                block_table=self.table,
                request_indices=t["request_indices"], softmax_scale=0.1,
                workspace=torch.empty(kda.latent_attention_workspace_size(
                    T, B, HL, R, P, torch.float32), dtype=torch.uint8,
                    device=DEV))
        return y

    def sample(self, t, x, rows, lens):
        """Penalties from each request's own tokens, then the sampling; the
        last row's token of a request is kept."""
        B, T = len(rows), sum(lens)
        for r in rows:
            self.tokens[r, :len(self.seen[r])] = i32(self.seen[r], DEV)
        known = i32([len(self.seen.get(r, [])) for r in range(ROWS)], DEV)
        before = f64(x["logits"])
        drafts = i32(np.arange(T) % 7, DEV)
        kw = dict(query_start_loc=t["query_start_loc"], draft_tokens=drafts,
                  request_indices=t["request_indices"], token_ids=self.tokens,
                  prompt_lens=torch.zeros(ROWS, **ONES), token_lens=known,
                  repetition_penalty=torch.full((B,), 1.3, device=DEV),
                  frequency_penalty=torch.full((B,), 0.5, device=DEV))
        kda.adjust_logits(logits=x["logits"], **kw)
        got = torch.zeros(T, **ONES)
        kda.sample(logits=x["logits"], uniform=x["uniform"], tokens=got,
                   workspace=torch.empty(kda.sample_workspace_size(T, VOCAB),
                                         dtype=torch.uint8, device=DEV))
        ref, size = oracle.adjust_logits(
            logits=before, **{k: v.cpu().numpy() for k, v in kw.items()})
        off = np.abs(f64(x["logits"]) - ref)
        assert (off <= 8 * 2.0 ** -24 * size).all()
        got = got.tolist()
        assert got == [oracle.sample_row(f64(x["logits"][m]),
                                         float(x["uniform"][m]), 1.0, 0, 1.0)
                       for m in range(T)]
        at = np.cumsum(lens) - 1
        for r, m in zip(rows, at):
            self.seen[r].append(got[m])

    def step(self, rows, lens, prompt=False, keep=True):
        for r in rows:
            self.text.setdefault(r, [])
            self.seen.setdefault(r, [])
        t, x = self.tables(rows, lens), self.inputs(sum(lens))
        kda.step_tables(**t)
        y = self.layers(t, x, lens, prompt)
        self.record(rows, lens, x, y, prompt)
        self.sample(t, x, rows, lens)
        if keep:
            self.computed[t["request_indices"].long()] += t["query_lens"]
        else:
            self.text = {r: v[:-lens[rows.index(r)]] if r in rows else v
                         for r, v in self.text.items()}
        self.release([])

    def record(self, rows, lens, x, y, prompt):
        """Checks the latent layer on each request's tokens so far, and keeps
        the KDA layer's outputs for the end."""
        at = 0
        for r, n in zip(rows, lens):
            for i in range(at, at + n):
                tok = {k: f64(v[i]) for k, v in x.items() if k[0] != "u"}
                tok["out"] = f64(y["kda"][i])
                self.text[r].append(tok)
            all_lat = np.stack([t["latent"] for t in self.text[r]])
            all_rope = np.stack([t["rope_key"] for t in self.text[r]])
            L = len(all_lat)
            see = np.arange(L)[None] <= (L - n + np.arange(n))[:, None]
            for h in range(HL):
                if prompt:
                    w = f64(self.weight[h])
                    k = np.concatenate([all_lat @ w[:DL].T, all_rope], 1)
                    v = all_lat @ w[DL:].T
                    q = f64(x["q_exp"][at:at + n, h])
                else:
                    k = np.concatenate([all_lat, all_rope], 1)
                    v, q = all_lat, f64(x["q_cat"][at:at + n, h])
                o, lse, weight, size = oracle.cache.softmax_sum(q, k, v, see,
                                                                0.1)
                ref = dict(out=o, lse=lse, weight=weight, size=size,
                           keys=see.sum(axis=1))
                b_out, b_lse = bounds(ref, "f32", R + P)
                if prompt:
                    # keys and values are sums of R products of their own
                    u = 2.0 ** -24
                    big = np.abs(all_lat) @ np.abs(w).T
                    s = 0.1 * (np.abs(q[:, :DL]) @ big[:, :DL].T).max(axis=1)
                    b_lse = b_lse + R * u * s
                    b_out = b_out + R * u * (2 * s[:, None] * weight
                                             + big[:, DL:].max(axis=0))
                assert (np.abs(f64(y["lat"][at:at + n, h]) - o)
                        <= b_out).all()
                assert (np.abs(f64(y["lse"][at:at + n, h]) - lse)
                        <= b_lse).all()
            at += n

    def check_states(self):
        """Every live request's KDA outputs, state and conv history against
        one pass over its tokens."""
        for r, toks in self.text.items():
            x = {k: torch.as_tensor(np.stack([t[k] for t in toks]),
                                    dtype=torch.float32)
                 for k in ("mixed_qkv", "raw_gate", "raw_beta", "out")}
            ref = reference(dict(self.kda, **x), [0, len(toks)], [1], None)
            top = np.max(np.abs(ref["out"]))
            assert np.max(np.abs(f64(x["out"]) - ref["out"])) <= \
                TOL["f32"] * top, r
            c = int(self.computed[r])
            assert c == len(toks)
            slot = int(self.table[r, c // BLOCK])
            want = ref["state"][1]
            assert np.max(np.abs(f64(self.kda["state"][slot]) - want)) <= \
                TOL["f32"] * np.max(np.abs(want)), r
            assert np.array_equal(f64(self.kda["conv_state"][slot][:, :3]),
                                  ref["conv_state"][1][:, :3])

    def check_blocks(self):
        """No block of two requests but whole ones, none both free and held."""
        held, table = self.held.cpu(), self.table.cpu()
        own = [int(table[r, int(self.computed[r]) // BLOCK])
               for r in self.text]
        assert len(set(own)) == len(own)
        used = {int(b) for r in self.text for b in table[r, :int(held[r])]}
        assert 0 not in used
        free = self.free[:int(self.num_free)].tolist()
        assert used.isdisjoint(free) and len(used) + len(free) == N - 1


@pytest.mark.gpu
def test_prompts_forks_windows_release_compaction():
    s = Server()
    s.step([0, 1], [11, 20], prompt=True)
    s.step([1, 0], [3, 9], prompt=True)          # pieces behind computed ones
    s.fork(0, [2, 4])
    s.check_blocks()
    for _ in range(5):                           # each on its own, past a block
        s.step([2, 0, 1, 4], [1, 1, 1, 1])
    s.check_states()
    # a draft window that nothing is kept of (the attention layer alone)
    s.step([4, 1], [4, 2], keep=False)
    s.release([0, 1])                            # the forks' parent ends
    s.check_blocks()
    s.compact()
    s.check_blocks()
    live = {int(b) for r in s.text for b in s.table[r, :int(s.held[r])]}
    assert live == set(range(1, len(live) + 1))
    for _ in range(4):
        s.step([4, 2], [1, 1])
    s.step([0, 3], [13, 2], prompt=True)         # on blocks given back
    s.fork(4, [1])
    for _ in range(9):
        s.step([0, 1, 2, 3, 4], [1] * 5)
    s.check_states()
    s.check_blocks()


@pytest.mark.gpu
def test_decode_steps_from_a_graph():
    """Tables, cache write, both layers and the sampling captured once, and
    replayed while the requests grow past a block."""
    s = Server()
    s.step([0, 1, 2], [6, 1, 13], prompt=True)
    rows, B = [2, 0, 1], 3
    t, x = s.tables(rows, [1] * B), s.inputs(B)
    t["free_blocks"] = s.free[:12].clone()
    y = dict(kda=torch.zeros((B, H * D), device=DEV),
             lat=torch.zeros((B, HL, R), device=DEV),
             lse=torch.zeros((B, HL), device=DEV))
    got = torch.zeros(B, **ONES)
    work = torch.empty(kda.latent_attention_workspace_size(
        B, B, HL, R, P, torch.float32), dtype=torch.uint8, device=DEV)
    scratch = torch.empty(kda.sample_workspace_size(B, VOCAB),
                          dtype=torch.uint8, device=DEV)

    def one_token():
        kda.step_tables(**t)
        kda.latent_write(latent=x["latent"], rope_key=x["rope_key"],
                         cache=s.cache, slot_mapping=t["slot_mapping"])
        kda.conv_update_decode(
            **s.kda, mixed_qkv=x["mixed_qkv"], raw_gate=x["raw_gate"],
            raw_beta=x["raw_beta"], out=y["kda"],
            state_indices=t["state_indices"],
            final_state_indices=t["final_state_indices"])
        kda.latent_attention(
            q=x["q_cat"], cache=s.cache, out=y["lat"], lse=y["lse"],
            query_start_loc=t["query_start_loc"],
            num_computed_tokens=s.computed, block_table=s.table,
            request_indices=t["request_indices"], softmax_scale=0.1,
            workspace=work)
        kda.adjust_logits(logits=x["logits"], token_ids=s.tokens,
                          prompt_lens=zeros, token_lens=s.computed,
                          request_indices=t["request_indices"],
                          presence_penalty=ones)
        kda.sample(logits=x["logits"], uniform=x["uniform"], tokens=got,
                   workspace=scratch)
        s.computed.index_add_(0, t["request_indices"].long(), t["query_lens"])

    zeros, ones = torch.zeros(ROWS, **ONES), torch.ones(B, device=DEV)
    s.tokens.random_(0, VOCAB)

    def after():
        s.record(rows, [1] * B, x, y, False)
        s.release([])
        t["free_blocks"].copy_(s.free[:12])

    one_token()
    after()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        one_token()
    for _ in range(12):
        for k, v in s.inputs(B).items():
            x[k].copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        after()
    s.check_states()
    s.check_blocks()
