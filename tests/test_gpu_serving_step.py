"""The operators of a serving step run together, over paged state slots: step
tables, the prefill of prompts in two pieces, single-token decode, the
speculative verify with sampling and draft acceptance, the commit, and decode
steps from a captured graph; against one fp64 pass over each request's
committed tokens."""
import numpy as np
import pytest
import torch

import linear_attention_speculative_amd as kda
import oracle
from tests.gpu_check import TOL
from tests.layer_check import f64, i32, make_layer, reference

DEV = "cuda"
ROWS, Q, BLOCK, SLOTS, VOCAB = 4, 4, 16, 24, 301


class Server:
    """Request rows, block tables and one layer's tensors, as a serving loop
    keeps them."""

    def __init__(self, H, D, lb, order, max_tokens):
        self.kw = make_layer(1, SLOTS, H, D, Q, act="f32", lb=lb, seed=5)
        del self.kw["mixed_qkv"], self.kw["raw_gate"], self.kw["raw_beta"], \
            self.kw["out"]
        self.H, self.D, self.max_tokens = H, D, max_tokens
        self.order = i32(order, DEV)
        B = len(order)

        def ints(*shape, dtype=torch.int32):
            return torch.zeros(shape, dtype=dtype, device=DEV)

        self.free = list(np.random.default_rng(3).permutation(SLOTS - 1) + 1)
        self.tables = dict(
            query_lens=ints(B), num_computed_tokens=ints(ROWS),
            num_blocks=ints(ROWS), block_table=ints(ROWS, 6),
            free_blocks=ints(8), block_size=BLOCK, query_start_loc=ints(B + 1),
            state_indices=ints(B), initial_state_indices=ints(B),
            final_state_indices=ints(B), positions=ints(max_tokens),
            slot_mapping=ints(max_tokens, dtype=torch.int64),
            num_allocated=ints(1), request_indices=self.order)
        self.tables["new_num_blocks"] = self.tables["num_blocks"]
        self.work = torch.empty(
            kda.prefill_workspace_size(max_tokens, B, H, D, torch.float32),
            dtype=torch.uint8, device=DEV)
        self.draw = torch.Generator().manual_seed(11)

    def rows(self, n):
        HD = self.H * self.D

        def randn(cols):
            return torch.randn((n, cols), generator=self.draw).to(DEV)

        return dict(mixed_qkv=randn(3 * HD), raw_gate=randn(HD),
                    raw_beta=randn(self.H),
                    out=torch.full((n, HD), 7.0, device=DEV))

    def give_blocks(self):
        """Free blocks for the next step; the ones it takes go with `took`."""
        self.tables["free_blocks"].copy_(i32(self.free[:8], DEV))

    def took(self):
        n = int(self.tables["num_allocated"].item())
        assert n <= 8
        del self.free[:n]

    def step(self, lens):
        self.give_blocks()
        self.tables["query_lens"].copy_(i32(lens, DEV))
        kda.step_tables(**self.tables)
        self.took()
        return self.tables


@pytest.mark.gpu
@pytest.mark.parametrize("H,D,lb", [(2, 64, None), (3, 128, -5.0)])
def test_prompts_decode_verify_sample_commit(H, D, lb):
    order = [2, 0, 3]                       # row 1 holds no request
    B = len(order)
    s = Server(H, D, lb, order, 48)
    stream = [[] for _ in range(B)]         # each request's committed rows

    def keep(x, lens, taken):
        at = 0
        for b in range(B):
            stream[b].append({k: v[at:at + taken[b]].clone()
                              for k, v in x.items()})
            at += lens[b]

    def advance(taken):
        s.tables["num_computed_tokens"][s.order.long()] += i32(taken, DEV)

    # prompts, in two pieces; rows behind the last one stay as they were
    for lens in ([21, 1, 15], [0, 12, 33]):
        t, x = s.step(lens), s.rows(48)
        kda.conv_prefill(**s.kw, **x, query_start_loc=t["query_start_loc"],
                         state_indices=t["final_state_indices"],
                         initial_state_indices=t["initial_state_indices"],
                         workspace=s.work)
        assert bool((x["out"][sum(lens):] == 7.0).all())
        keep(x, lens, lens)
        advance(lens)

    # one decoded token each
    t, x = s.step([1] * B), s.rows(B)
    kda.conv_update_decode(**s.kw, **x, state_indices=t["state_indices"],
                           final_state_indices=t["final_state_indices"])
    keep(x, [1] * B, [1] * B)
    advance([1] * B)

    # windows with drafts: verify, sample and accept, commit
    corr = torch.zeros((SLOTS, H, Q, D), device=DEV)
    keys = torch.zeros((SLOTS, H, Q, 2 * D), device=DEV)
    counter = torch.zeros(1, dtype=torch.int32, device=DEV)
    ctx = kda.CommitContext(
        [dict(state=s.kw["state"], correction=corr, key_gate=keys,
              A_log=s.kw["A_log"], dt_bias=s.kw["dt_bias"], lower_bound=lb,
              conv_state=s.kw["conv_state"])], spec_query_len=Q)
    head = torch.randn((H * D, VOCAB), generator=s.draw).to(DEV)
    temps, top_k, top_p = [0.7, 0.0, 1.3], [20, 0, 0], [1.0, 1.0, 0.9]
    sampling = dict(
        temperature=torch.tensor(temps, device=DEV), top_k=i32(top_k, DEV),
        top_p=torch.tensor(top_p, device=DEV))
    scratch = torch.empty(kda.sample_workspace_size(Q * B, VOCAB),
                          dtype=torch.uint8, device=DEV)
    for lens, want in (([4, 2, 3], [4, 1, 2]), ([1, 4, 4], [1, 4, 3])):
        t, T = s.step(lens), sum(lens)
        x = s.rows(T)
        kda.conv_update_verify(
            **s.kw, **x, correction=corr, key_gate=keys,
            query_start_loc=t["query_start_loc"],
            state_indices=t["state_indices"],
            num_accepted_tokens=i32([1] * B, DEV), work_counter=counter)
        logits = x["out"] @ head
        uniform = torch.rand(T, generator=s.draw)
        drafts, tokens, at = [], [], 0
        for b in range(B):
            mine = [oracle.sample_row(f64(logits[at + i]),
                                      float(uniform[at + i]), temps[b],
                                      top_k[b], top_p[b])
                    for i in range(lens[b])]
            # `want` leading tokens of the window match, the next one does not
            drafts += [5] + [mine[i] if i + 1 < want[b] else
                             (mine[i] + 1) % VOCAB
                             for i in range(lens[b] - 1)]
            tokens.append(mine)
            at += lens[b]
        got, count, following = (torch.full((n,), -7, dtype=torch.int32,
                                            device=DEV) for n in (T, B, B))
        kda.sample(logits=logits, uniform=uniform.to(DEV), tokens=got,
                   query_start_loc=t["query_start_loc"],
                   draft_tokens=i32(drafts, DEV), num_accepted=count,
                   next_tokens=following, workspace=scratch, **sampling)
        assert got.tolist() == sum(tokens, [])
        assert count.tolist() == want
        assert following.tolist() == [m[w - 1] for m, w in zip(tokens, want)]
        accepted = torch.zeros(ROWS, dtype=torch.int32, device=DEV)
        accepted[s.order.long()] = count      # commit reads it by row
        ctx.commit_step(accepted, t["state_indices"], t["query_start_loc"],
                        request_indices=s.order,
                        block_table=s.tables["block_table"],
                        num_computed_tokens=s.tables["num_computed_tokens"],
                        mamba_block_size=BLOCK)
        keep(x, lens, want)
        advance(want)

    # decode steps replayed from a graph: tables, layer, sampling, counting
    x = s.rows(B)
    uniform = torch.rand(B, generator=s.draw).to(DEV)
    got = torch.full((B,), -7, dtype=torch.int32, device=DEV)
    s.tables["query_lens"].fill_(1)
    index = s.order.long()
    ones = i32([1] * B, DEV)
    logits = torch.empty((B, VOCAB), device=DEV)

    def one_token():
        kda.step_tables(**s.tables)
        kda.conv_update_decode(
            **s.kw, **x, state_indices=s.tables["state_indices"],
            final_state_indices=s.tables["final_state_indices"])
        kda.sample(logits=logits, uniform=uniform, tokens=got,
                   workspace=scratch, **sampling)
        s.tables["num_computed_tokens"].index_add_(0, index, ones)

    s.give_blocks()
    one_token()
    s.took()
    keep(x, [1] * B, [1] * B)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        one_token()
    for _ in range(20):                       # across a block's end
        for name, v in s.rows(B).items():
            x[name].copy_(v)
        logits.copy_(torch.randn((B, VOCAB), generator=s.draw))
        s.give_blocks()
        graph.replay()
        s.took()
        assert got.tolist() == [
            oracle.sample_row(f64(logits[b]), float(uniform[b].item()),
                              temps[b], top_k[b], top_p[b])
            for b in range(B)]
        keep(x, [1] * B, [1] * B)

    # everything against one pass over the committed tokens
    joined = [{k: torch.cat([p[k] for p in parts]) for k in parts[0]}
              for parts in stream]
    lens = [j["out"].shape[0] for j in joined]
    assert s.tables["num_computed_tokens"].tolist() == \
        [lens[1], 0, lens[0], lens[2]]
    qsl = np.concatenate([[0], np.cumsum(lens)])
    kw = dict(s.kw, **{k: torch.cat([j[k] for j in joined])
                       for k in joined[0]})
    ref = reference(kw, qsl, [1, 2, 3], None)
    top = np.max(np.abs(ref["out"]))
    assert np.max(np.abs(f64(kw["out"]) - ref["out"])) <= TOL["f32"] * top
    final = s.tables["final_state_indices"].tolist()
    for b, slot in enumerate(final):
        want = ref["state"][b + 1]
        err = np.max(np.abs(f64(s.kw["state"][slot]) - want))
        assert err <= TOL["f32"] * np.max(np.abs(want)), (b, err)
        assert np.array_equal(f64(s.kw["conv_state"][slot][:, :3]),
                              ref["conv_state"][b + 1][:, :3])


@pytest.mark.gpu
def test_tensors_on_the_host_are_refused():
    """A tensor left on the host is refused before any launch."""
    kw = make_layer(2, 3, 1, 32, 4, act="f32", seed=1)
    args = dict(kw, state_indices=i32([1, 2], DEV))
    kda.conv_update_decode(**args)
    for name in ("mixed_qkv", "state", "state_indices", "conv_weight"):
        with pytest.raises(ValueError, match="device"):
            kda.conv_update_decode(**dict(args, **{name: args[name].cpu()}))
    with pytest.raises(ValueError, match="GPU"):
        kda.conv_update_decode(**{k: v.cpu() if isinstance(v, torch.Tensor)
                                  else v for k, v in args.items()})
