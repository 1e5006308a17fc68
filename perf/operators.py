"""What a serving step of KDA layers needs around the speculative verify and
commit, as measured operators: prefill of prompts, single-token decode, the
step's block tables and slot maps, and sampling with draft acceptance.

`run` computes an operator in its plain form (elementary torch operations in
32 bits, 64 where 32 lose what matters) when `own` is false, and calls the
library's entry points when it is true.  `exact` is the definition in 64 bits,
token by token.
"""
import math

import numpy as np
import torch

own = False

ACT = {"f32": torch.float32, "bf16": torch.bfloat16}
NULL = 0            # null block id
TAPS = 4            # taps of the short convolution
CHUNK = 32          # tokens per chunk of the plain chunked form


# ---- cases ------------------------------------------------------------------

def _prefill(name, B, mean, H, D, act, conv=True, lb=0.0, dim_first=True,
             resumed=0.0, even=False):
    """B prompts of `mean` tokens on average (`even`: exactly); `lb` the gate's
    lower bound (0: softplus); `resumed`: share that continues a state."""
    return dict(name=name, op="prefill", B=B, mean=mean, H=H, D=D, act=act,
                conv=conv, lb=lb, dim_first=dim_first, resumed=resumed,
                even=even)


def _decode(name, B, H, D, act, conv=True, lb=0.0, dim_first=True, null=0.0):
    return dict(name=name, op="decode", B=B, H=H, D=D, act=act, conv=conv,
                lb=lb, dim_first=dim_first, null=null)


def _tables(name, B, mean, block, rows):
    return dict(name=name, op="tables", B=B, mean=mean, block=block,
                rows=rows)


def _sample(name, B, Q, V, act, pad=0):
    """B requests, a window of Q rows each; Q = 1: plain sampling."""
    return dict(name=name, op="sample", B=B, Q=Q, V=V, act=act, pad=pad)


def listed():
    return [
        # a few short prompts on the smallest heads: latency
        _prefill("prefill_tiny", 3, 21, 2, 16, "f32"),
        # one long prompt at the full head shape: the recurrence is serial
        _prefill("prefill_long", 1, 8192, 32, 128, "bf16", even=True),
        # a batch of ragged prompts, half of them continued from a cached
        # state, bounded gates
        _prefill("prefill_ragged", 16, 1000, 32, 128, "bf16", lb=-5.0,
                 dim_first=False, resumed=0.5),
        # fp32 activations, already convolved, a small layer
        _prefill("prefill_qkv_f32", 5, 301, 8, 64, "f32", conv=False,
                 resumed=0.5),
        # one request generating: latency
        _decode("decode_one", 1, 32, 128, "bf16", dim_first=False),
        # the throughput batch, and a small odd fp32 one
        _decode("decode_batch", 256, 32, 128, "bf16", lb=-5.0, null=0.02),
        _decode("decode_qkv_f32", 37, 6, 64, "f32", conv=False, null=0.1),
        # a handful of requests; a large mixed step of prompts and decodes
        _tables("tables_small", 7, 4, 16, 7),
        _tables("tables_large", 2000, 33, 64, 4096),
        # one request's next token; a draft window for a whole batch; odd
        # sizes with padded rows
        _sample("sample_one", 1, 1, 131072, "f32"),
        _sample("sample_window", 256, 4, 131072, "bf16"),
        _sample("sample_odd", 33, 1, 50021, "f32", pad=3),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "decode", "tables", "sample"])
    act = rng.choice(["bf16", "bf16", "f32"])
    D = rng.choice([16, 32, 64, 128, 128])
    H = rng.choice([1, 3, 8, 32])
    lb = rng.choice([0.0, -5.0])
    if op == "prefill":
        B = _spread(rng, 1, 24)
        total = _spread(rng, max(B, 2), 16000)
        case = _prefill("", B, max(1, total // B), H, D, act,
                        rng.random() < 0.6, lb, rng.random() < 0.5,
                        rng.choice([0.0, 0.5, 1.0]))
    elif op == "decode":
        case = _decode("", _spread(rng, 1, 250), H, D, act,
                       rng.random() < 0.6, lb, rng.random() < 0.5,
                       rng.choice([0.0, 0.1]))
    elif op == "tables":
        B = _spread(rng, 1, 2000)
        case = _tables("", B, _spread(rng, 1, 33), rng.choice([16, 64, 100]),
                       B + rng.randrange(0, 50))
    else:
        case = _sample("", _spread(rng, 1, 120), rng.choice([1, 1, 2, 4]),
                       _spread(rng, 40, 131072), act, rng.choice([0, 0, 5]))
    del case["name"]
    return case


def _lengths(case):
    """Prompt lengths of a prefill case (host; from the case alone)."""
    B, mean = case["B"], case["mean"]
    if case["even"]:
        return np.full(B, mean)
    r = np.random.RandomState(B * 131 + mean)
    return r.randint(1, 2 * mean + 1, size=B)


# ---- inputs -----------------------------------------------------------------

def _device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


def _gen(seed):
    g = torch.Generator(device=_device())
    g.manual_seed(int(seed) * 7919 + 11)
    return g


def _randn(shape, g, std=1.0, dtype=torch.float32):
    return (torch.randn(shape, generator=g, device=_device()) * std).to(dtype)


def _i32(a):
    return torch.as_tensor(np.ascontiguousarray(a).astype(np.int32)) \
        .to(_device())


def _layer(case, g, T, N, Q):
    """One KDA layer's parameters, state pool and activations."""
    H, D = case["H"], case["D"]
    dt, dev = ACT[case["act"]], _device()
    s = dict(H=H, D=D, Q=Q, dim_first=case["dim_first"], conv=case["conv"],
             lb=case["lb"] if case["lb"] else None)
    s["A_log"] = torch.log(1 + 15 * torch.rand(H, generator=g, device=dev))
    if case["lb"]:
        s["dt_bias"] = _randn((H, D), g, 0.1)
    else:   # inverse softplus of steps spread over 1e-3 .. 1e-1
        step = torch.exp(torch.rand((H, D), generator=g, device=dev)
                         * math.log(100.0) + math.log(1e-3))
        s["dt_bias"] = torch.log(torch.expm1(step))
    s["mixed_qkv"] = _randn((T, 3 * H * D), g, 1.0, dt)
    s["raw_gate"] = _randn((T, H * D), g, 1.0 if case["lb"] else 0.3, dt)
    s["raw_beta"] = _randn((T, H), g, 1.0, dt)
    s["state"] = _randn((N, H, D, D), g, 0.1)
    s["out"] = torch.zeros((T, H * D), device=dev, dtype=dt)
    s["conv_state"] = s["conv_weight"] = None
    if case["conv"]:
        shape = (N, 3 * H * D, Q + 2) if case["dim_first"] \
            else (N, Q + 2, 3 * H * D)
        s["conv_state"] = _randn(shape, g, 1.0, dt)
        s["conv_weight"] = _randn((3 * H * D, TAPS), g, 0.5, dt)
    return s


def prepare(case, seed):
    return {"prefill": _prepare_prefill, "decode": _prepare_decode,
            "tables": _prepare_tables, "sample": _prepare_sample
            }[case["op"]](case, seed)


def _prepare_prefill(case, seed):
    g, rng = _gen(seed), np.random.RandomState(seed % (1 << 31))
    lens = _lengths(case)
    B, T = case["B"], int(lens.sum())
    # slots 1..B receive the results, B+1..2B hold states to continue from
    s = _layer(case, g, T, 2 * B + 1, 4)
    initial = np.where(rng.rand(B) < case["resumed"],
                       B + 1 + rng.permutation(B), NULL)
    s.update(op="prefill", B=B, T=T, longest=int(lens.max()),
             query_start_loc=_i32(np.concatenate([[0], np.cumsum(lens)])),
             state_indices=_i32(1 + rng.permutation(B)),
             initial_state_indices=_i32(initial))
    if own:
        import linear_attention_speculative_amd as kda
        s["workspace"] = torch.empty(
            kda.prefill_workspace_size(T, B, case["H"], case["D"],
                                       ACT[case["act"]]),
            dtype=torch.uint8, device=_device())
    return s


def _prepare_decode(case, seed):
    g, rng = _gen(seed), np.random.RandomState(seed % (1 << 31))
    B = case["B"]
    # sources 1..B, results B+1..2B (the next state block under caching)
    s = _layer(case, g, B, 2 * B + 1, 4)
    src = 1 + rng.permutation(B)
    src[rng.rand(B) < case["null"]] = NULL
    s.update(op="decode", B=B, state_indices=_i32(src),
             final_state_indices=_i32(B + 1 + rng.permutation(B)),
             num_accepted_tokens=_i32(rng.randint(1, 5, size=B)))
    return s


def _query_lens(case):
    """Tokens of each request's step (from the case alone): nine in ten
    decode a window of 1..4, the others run a prompt chunk."""
    B = case["B"]
    r = np.random.RandomState(B * 17 + case["mean"])
    prompt = r.rand(B) < 0.1
    return prompt, np.where(
        prompt, r.randint(1, 20 * case["mean"] + 1, size=B),
        r.randint(1, 5, size=B))


def _prepare_tables(case, seed):
    rng = np.random.RandomState(seed % (1 << 31))
    B, rows, bs = case["B"], case["rows"], case["block"]
    prompt, q = _query_lens(case)
    order = rng.permutation(B)
    prompt, q = prompt[order], q[order]
    computed = np.zeros(rows, np.int64)
    req = rng.permutation(rows)[:B]
    computed[req] = np.where(prompt, 0, rng.randint(1, 40 * bs, size=B))
    held = np.where(computed > 0, computed // bs + 1, 0)
    need = (computed[req] + q) // bs + 1
    width = (40 * bs + 20 * case["mean"] + 4) // bs + 1
    free = 1 + rng.permutation(rows * width)
    table = np.zeros((rows, width), np.int64)
    for r in req:
        n = int(held[r])
        table[r, :n], free = free[:n], free[n:]
    # the step's capacity in tokens, as a captured graph would have it
    cap = -(-int(q.sum()) // 256) * 256
    dev = _device()
    return dict(
        op="tables", B=B, block=bs, cap=cap, query_lens=_i32(q),
        request_indices=_i32(req), num_computed_tokens=_i32(computed),
        num_blocks=_i32(held), block_table=_i32(table),
        free_blocks=_i32(free[:int(np.maximum(need - held[req], 0).sum())
                              + 5]),
        out=dict(
            query_start_loc=torch.empty(B + 1, dtype=torch.int32, device=dev),
            new_num_blocks=_i32(held),
            state_indices=torch.empty(B, dtype=torch.int32, device=dev),
            initial_state_indices=torch.empty(B, dtype=torch.int32,
                                              device=dev),
            final_state_indices=torch.empty(B, dtype=torch.int32, device=dev),
            positions=torch.empty(cap, dtype=torch.int32, device=dev),
            slot_mapping=torch.empty(cap, dtype=torch.int64, device=dev),
            num_allocated=torch.empty(1, dtype=torch.int32, device=dev)))


def _prepare_sample(case, seed):
    g, rng = _gen(seed), np.random.RandomState(seed % (1 << 31))
    B, Q, V = case["B"], case["Q"], case["V"]
    lens = np.full(B, Q) if Q == 1 else rng.randint(1, Q + 1, size=B)
    if Q > 1:
        lens[0] = Q
    # rows are as many for every seed; those behind the last request stay
    M = B * Q
    dev, dt = _device(), ACT[case["act"]]
    full = torch.randn((M, V + case["pad"]), generator=g, device=dev) * 2.0
    # a few likely tokens in each row, as a trained model has them
    top = torch.randint(0, V, (M, min(8, V)), generator=g, device=dev)
    full.scatter_add_(1, top, 4 + 8 * torch.rand(top.shape, generator=g,
                                                 device=dev))
    logits = full.to(dt)[:, :V]
    del full
    pick = lambda v: torch.tensor(v, device=dev, dtype=torch.float32)[  # noqa: E731
        torch.as_tensor(rng.randint(0, len(v), size=B), device=dev)]
    s = dict(op="sample", B=B, Q=Q, logits=logits,
             uniform=torch.rand(M, generator=g, device=dev),
             temperature=pick([0.0, 0.6, 0.8, 1.0, 1.0, 1.3]),
             top_k=pick([0, 20, 50, 1000]).to(torch.int32),
             top_p=pick([1.0, 0.8, 0.9, 0.95]),
             min_p=pick([0.0, 0.0, 0.02, 0.1]),
             query_start_loc=_i32(np.concatenate([[0], np.cumsum(lens)])),
             tokens=torch.full((M,), -7, dtype=torch.int32, device=dev),
             draft_tokens=None, num_accepted=None, next_tokens=None)
    if Q > 1:
        # window token t + 1 is the draft for the row of token t: mostly the
        # row's likeliest token
        best = torch.argmax(logits.float(), dim=1).to(torch.int32)
        other = torch.randint(0, V, (M,), generator=g, device=dev,
                              dtype=torch.int32)
        hit = torch.rand(M, generator=g, device=dev) < 0.8
        s["draft_tokens"] = torch.roll(torch.where(hit, best, other), 1)
        s["num_accepted"] = torch.empty(B, dtype=torch.int32, device=dev)
        s["next_tokens"] = torch.empty(B, dtype=torch.int32, device=dev)
    if own:
        import linear_attention_speculative_amd as kda
        s["workspace"] = torch.empty(kda.sample_workspace_size(M, V),
                                     dtype=torch.uint8, device=dev)
    return s


# ---- one pass ---------------------------------------------------------------

def run(s):
    if own:
        return {"prefill": _own_prefill, "decode": _own_decode,
                "tables": _own_tables, "sample": _own_sample}[s["op"]](s)
    return {"prefill": _plain_prefill, "decode": _plain_decode,
            "tables": _plain_tables, "sample": _plain_sample}[s["op"]](s)


def _layer_kwargs(s):
    names = ["mixed_qkv", "raw_gate", "raw_beta", "A_log", "dt_bias",
             "state", "out", "state_indices"]
    kw = {n: s[n] for n in names}
    kw["lower_bound"] = s["lb"]
    if s["conv"]:
        kw.update(conv_state=s["conv_state"], conv_weight=s["conv_weight"],
                  conv_dim_first=s["dim_first"], spec_query_len=s["Q"])
    return kw


def _layer_outputs(s, lo, hi):
    """Outputs, the written state slots and their conv histories."""
    conv = ()
    if s["conv"]:
        cs = s["conv_state"][lo:hi]
        conv = (cs[:, :, :TAPS - 1] if s["dim_first"] else cs[:, :TAPS - 1],)
    return (s["out"], s["state"][lo:hi]) + conv


def _own_prefill(s):
    import linear_attention_speculative_amd as kda
    call = kda.conv_prefill if s["conv"] else kda.prefill_qkv
    call(query_start_loc=s["query_start_loc"],
         initial_state_indices=s["initial_state_indices"],
         workspace=s["workspace"], **_layer_kwargs(s))
    return _layer_outputs(s, 1, s["B"] + 1)


def _own_decode(s):
    import linear_attention_speculative_amd as kda
    kw = _layer_kwargs(s)
    if s["conv"]:
        kda.conv_update_decode(final_state_indices=s["final_state_indices"],
                               num_accepted_tokens=s["num_accepted_tokens"],
                               **kw)
    else:
        kda.decode_qkv(final_state_indices=s["final_state_indices"], **kw)
    return _layer_outputs(s, s["B"] + 1, 2 * s["B"] + 1)


def _own_tables(s):
    import linear_attention_speculative_amd as kda
    kda.step_tables(
        query_lens=s["query_lens"], num_computed_tokens=s["num_computed_tokens"],
        num_blocks=s["num_blocks"], block_table=s["block_table"],
        free_blocks=s["free_blocks"], block_size=s["block"],
        request_indices=s["request_indices"], null_block_id=NULL, **s["out"])
    return (s["out"], s["block_table"])


def _own_sample(s):
    import linear_attention_speculative_amd as kda
    kda.sample(logits=s["logits"], uniform=s["uniform"], tokens=s["tokens"],
               temperature=s["temperature"], top_k=s["top_k"],
               top_p=s["top_p"], min_p=s["min_p"],
               query_start_loc=s["query_start_loc"],
               draft_tokens=s["draft_tokens"],
               num_accepted=s["num_accepted"], next_tokens=s["next_tokens"],
               workspace=s["workspace"])
    return tuple(t for t in (s["tokens"], s["num_accepted"],
                             s["next_tokens"]) if t is not None)


# ---- plain forms ------------------------------------------------------------

def _sigmoid(x):
    return 1 / (1 + torch.exp(-x))


def _gate(x, s):
    """Log-decay from the raw gate [..., H, D]."""
    x = x + s["dt_bias"].to(x.dtype)
    A = torch.exp(s["A_log"].to(x.dtype))[:, None]
    if s["lb"] is not None:
        return s["lb"] * _sigmoid(A * x)
    return -A * torch.where(x > 20, x, torch.log1p(torch.exp(x)))


def _unit(x):
    return x * torch.rsqrt((x * x).sum(-1, keepdim=True) + 1e-6)


def _taps(seq, w):
    """SiLU of the width-4 causal convolution of seq [..., TAPS - 1 + L, C]."""
    L = seq.shape[-2] - (TAPS - 1)
    y = sum(seq[..., i:i + L, :] * w[:, i] for i in range(TAPS))
    return y * _sigmoid(y)


def _history(s, slots, accepted, dtype):
    """Conv histories [B, TAPS - 1, C]; zero for a null slot."""
    cs = s["conv_state"] if s["dim_first"] \
        else s["conv_state"].transpose(1, 2)
    at = (accepted[:, None] - 1 + torch.arange(TAPS - 1, device=cs.device)) \
        .long()
    h = cs[slots.clamp(min=0).long()]
    h = torch.gather(h, 2, at[:, None, :].expand(-1, h.shape[1], -1))
    h = torch.where((slots > NULL)[:, None, None], h, torch.zeros_like(h))
    return h.transpose(1, 2).to(dtype)


def _store_history(s, slots, live, h):
    """Entries [0, TAPS - 1) of the live slots' conv state."""
    cs = s["conv_state"] if s["dim_first"] \
        else s["conv_state"].transpose(1, 2)
    old = cs[slots.long(), :, :TAPS - 1]
    cs[slots.long(), :, :TAPS - 1] = torch.where(
        live[:, None, None], h.transpose(1, 2).to(cs.dtype), old)


def _padded(s, name, dtype):
    """Rows of each prompt padded to whole chunks: [B, N, ...], 0 behind."""
    qsl = s["query_start_loc"].long()
    n = -(-s["longest"] // CHUNK) * CHUNK
    t = torch.arange(n, device=qsl.device)
    inside = t[None] < (qsl[1:] - qsl[:-1])[:, None]
    at = torch.where(inside, qsl[:-1, None] + t[None], 0)
    x = s[name][at].to(dtype)
    return torch.where(inside[..., None], x, torch.zeros_like(x)), inside, at


def _heads(x, H):
    """[B, N, H*D] -> [B, H, N, D]."""
    return x.unflatten(-1, (H, -1)).transpose(1, 2)


def _plain_prefill(s):
    f, H, D, B = torch.float32, s["H"], s["D"], s["B"]
    x, inside, at = _padded(s, "mixed_qkv", f)
    initial, slots = s["initial_state_indices"], s["state_indices"]
    if s["conv"]:
        hist = _history(s, initial, torch.ones_like(initial), f)
        seq = torch.cat([hist, x], 1)
        x = _taps(seq, s["conv_weight"].to(f))
        lens = inside.sum(1)
        tail = torch.gather(seq, 1, (lens[:, None] + torch.arange(
            TAPS - 1, device=x.device))[..., None].expand(
                -1, -1, seq.shape[2]))
    q, k, v = (_heads(t, H) for t in x.split(H * D, -1))
    q, k = _unit(q) * D ** -0.5, _unit(k)
    # gates and their running sums inside a chunk in 64 bits: differences of
    # long sums are what the decays are made of
    g = _gate(_padded(s, "raw_gate", torch.float64)[0].unflatten(-1, (H, D)),
              s).transpose(1, 2)
    keep = inside[:, None, :, None]
    g = torch.where(keep, g, torch.zeros_like(g))
    beta = _sigmoid(_padded(s, "raw_beta", f)[0]).transpose(1, 2)
    beta = torch.where(inside[:, None], beta, torch.zeros_like(beta))
    q, k, v, g, beta = (t.unflatten(2, (-1, CHUNK))
                        for t in (q, k, v, g, beta))
    G = g.cumsum(3)
    low = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=G.device).tril()
    NC = G.shape[2]
    A = torch.empty(B, H, NC, CHUNK, CHUNK, device=G.device)
    P = torch.empty_like(A)
    for j in range(CHUNK):      # one key of every chunk at a time
        w = k[..., j:j + 1, :] * torch.exp(
            (G - G[..., j:j + 1, :]).clamp(max=0)).to(f)
        A[..., j] = (k * w).sum(-1)
        P[..., j] = (q * w).sum(-1)
    A = torch.where(low.tril(-1), A * beta[..., None], torch.zeros_like(A))
    P = torch.where(low, P, torch.zeros_like(P))
    # (I + A)^-1 of a strictly lower A, by squaring
    eye = torch.eye(CHUNK, device=G.device)
    inv, power = eye - A, A
    for _ in range(int(math.log2(CHUNK)) - 1):
        power = power @ power
        inv = inv @ (eye + power)
    inv = inv * beta[..., None, :]
    decay = torch.exp(G).to(f)
    kd, qd = k * decay, q * decay
    ke = k * torch.exp(G[..., -1:, :] - G).to(f)
    last = decay[..., -1, :]
    live0 = (initial > NULL)[:, None, None, None]
    S = s["state"][initial.clamp(min=0).long()]
    S = torch.where(live0, S, torch.zeros_like(S)).transpose(-1, -2)
    S = S.contiguous()                                   # [B, H, K, V]
    outs = []
    for n in range(NC):
        c = inv[:, :, n] @ (v[:, :, n] - kd[:, :, n] @ S)
        outs.append(qd[:, :, n] @ S + P[:, :, n] @ c)
        S = S * last[:, :, n, :, None] \
            + ke[:, :, n].transpose(-1, -2).contiguous() @ c
    o = torch.stack(outs, 2).flatten(2, 3).transpose(1, 2).flatten(2)
    s["out"][at[inside]] = o[inside].to(s["out"].dtype)
    s["state"][slots.long()] = S.transpose(-1, -2)
    if s["conv"]:
        _store_history(s, slots, slots > NULL, tail)
    return _layer_outputs(s, 1, B + 1)


def _step(s, x, raw_gate, raw_beta, S, dtype):
    """One recurrence step from S [B, H, V, K]: (out, new state)."""
    H, D = s["H"], s["D"]
    q, k, v = (t.unflatten(-1, (H, D)) for t in x.split(H * D, -1))
    q, k = _unit(q) * D ** -0.5, _unit(k)
    g = _gate(raw_gate.to(dtype).unflatten(-1, (H, D)), s)
    S = S * torch.exp(g)[..., None, :]
    c = _sigmoid(raw_beta.to(dtype))[..., None] \
        * (v - (S * k[..., None, :]).sum(-1))
    S = S + c[..., :, None] * k[..., None, :]
    return (S * q[..., None, :]).sum(-1).flatten(1), S


def _decode_with(s, dtype):
    src, dst = s["state_indices"], s["final_state_indices"]
    live = src > NULL
    x = s["mixed_qkv"].to(dtype)
    tail = None
    if s["conv"]:
        hist = _history(s, src, s["num_accepted_tokens"], dtype)
        seq = torch.cat([hist, x[:, None]], 1)
        x, tail = _taps(seq, s["conv_weight"].to(dtype))[:, 0], seq[:, 1:]
    o, S = _step(s, x, s["raw_gate"], s["raw_beta"],
                 s["state"][src.long()].to(dtype), dtype)
    o = torch.where(live[:, None], o, torch.zeros_like(o))
    S = torch.where(live[:, None, None, None], S,
                    s["state"][dst.long()].to(dtype))
    return o, S, live, tail


def _plain_decode(s):
    o, S, live, tail = _decode_with(s, torch.float32)
    dst = s["final_state_indices"]
    s["out"].copy_(o)
    s["state"][dst.long()] = S
    if s["conv"]:
        _store_history(s, dst, live, tail)
    return _layer_outputs(s, s["B"] + 1, 2 * s["B"] + 1)


def _plain_tables(s):
    o, bs, cap = s["out"], s["block"], s["cap"]
    row = s["request_indices"].long()
    q = s["query_lens"].long().clamp(min=0)
    c = s["num_computed_tokens"].long()[row]
    have = s["num_blocks"].long()[row]
    table, free = s["block_table"], s["free_blocks"]
    width, F = table.shape[1], free.shape[0]
    end = q.cumsum(0)
    need = ((c + q) // bs + 1).clamp(max=width)
    new = (need - have).clamp(min=0)
    to = new.cumsum(0)
    off = to - new
    j = torch.arange(width, device=row.device)[None]
    pos = off[:, None] + j - have[:, None]
    fresh = (j >= have[:, None]) & (j < need[:, None])
    got = torch.where(pos < F, free[pos.clamp(0, F - 1)], NULL)
    rows = torch.where(fresh, got, table[row])
    table[row] = rows.to(table.dtype)
    o["new_num_blocks"].copy_(s["num_blocks"])
    o["new_num_blocks"][row] = (have + torch.minimum(
        new, (F - off).clamp(min=0))).to(torch.int32)
    o["num_allocated"][0] = to[-1]
    o["query_start_loc"][0] = 0
    o["query_start_loc"][1:] = end

    def block(p):
        at = p // bs
        b = torch.gather(rows, 1, at.clamp(max=width - 1)[:, None])[:, 0]
        return torch.where(at < width, b, NULL)

    o["state_indices"].copy_(block(c))
    o["initial_state_indices"].copy_(torch.where(c > 0, block(c), NULL))
    o["final_state_indices"].copy_(block(c + q))
    t = torch.arange(cap, device=row.device)
    b = torch.searchsorted(end, t, right=True)
    inside = b < s["B"]
    b = b.clamp(max=s["B"] - 1)
    p = c[b] + t - (end - q)[b]
    blk = rows[b, (p // bs).clamp(max=width - 1)].long()
    ok = inside & (p // bs < width) & (blk > NULL)
    o["positions"].copy_(torch.where(inside, p, 0))
    o["slot_mapping"].copy_(torch.where(ok, blk * bs + p % bs, -1))
    return (o, table)


def _per_row(s, M):
    """The request of each row (B behind the last)."""
    t = torch.arange(M, device=s["logits"].device)
    return torch.searchsorted(s["query_start_loc"][1:].long(), t, right=True)


def _plain_sample(s):
    x, f = s["logits"].float(), torch.float64
    M, V = x.shape
    req = _per_row(s, M)
    inside = req < s["B"]
    req = req.clamp(max=s["B"] - 1)
    T, k = s["temperature"][req], s["top_k"][req]
    greedy = T <= 0
    T = torch.where(greedy, torch.ones_like(T), T)
    k = torch.where(greedy, 1, torch.where(k <= 0, V, k))
    # weights and their sums in 64 bits: a token is chosen at the border of
    # two long sums
    w = torch.exp((x.to(f) - x.amax(1, keepdim=True).to(f))
                  / T.to(f)[:, None])
    order = torch.sort(x, dim=1, descending=True, stable=True)[1]
    ws = torch.gather(w, 1, order)
    keep = (ws >= s["min_p"][req].to(f)[:, None]) \
        & (torch.arange(V, device=x.device)[None] < k[:, None])
    ws = torch.where(keep, ws, torch.zeros_like(ws))
    cum = ws.cumsum(1)
    p = s["top_p"][req].to(f)[:, None]
    keep &= (p >= 1) | (cum - ws < p * cum[:, -1:])
    chosen = torch.zeros_like(keep).scatter_(1, order, keep)
    cum = torch.where(chosen, w, torch.zeros_like(w)).cumsum(1)
    u = s["uniform"].to(f)[:, None] * cum[:, -1:]
    token = (cum <= u).sum(1).clamp(max=V - 1).to(torch.int32)
    s["tokens"].copy_(torch.where(inside, token, s["tokens"]))
    if s["draft_tokens"] is None:
        return (s["tokens"],)
    qsl = s["query_start_loc"].long()
    n = torch.zeros(s["B"], dtype=torch.long, device=x.device)
    going = torch.ones_like(n, dtype=torch.bool)
    for t in range(s["Q"] - 1):
        at = (qsl[:-1] + t).clamp(max=M - 2)
        going &= (qsl[:-1] + t + 1 < qsl[1:]) \
            & (s["tokens"][at] == s["draft_tokens"][at + 1])
        n += going
    s["num_accepted"].copy_(n + 1)
    s["next_tokens"].copy_(s["tokens"][qsl[:-1] + n])
    return (s["tokens"], s["num_accepted"], s["next_tokens"])


# ---- work -------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op in ("prefill", "decode"):
        B, H, D = case["B"], case["H"], case["D"]
        e = 4 if case["act"] == "f32" else 2
        T = int(_lengths(case).sum()) if op == "prefill" else B
        live = case["resumed"] * B if op == "prefill" \
            else (1 - case["null"]) * B
        done = B if op == "prefill" else live
        byts = T * H * (5 * D + 1) * e + (live + done) * H * D * D * 4
        if case["conv"]:
            byts += (live + done) * 3 * H * D * (TAPS - 1) * e \
                + 3 * H * D * TAPS * e
        return {"bytes": byts, "flops": T * H * (7 * D * D)}
    if op == "tables":
        B = case["B"]
        T = int(_query_lens(case)[1].sum())
        return {"bytes": T * 12 + B * 4 * 10 + T / case["block"] * 8,
                "flops": 0}
    M = case["B"] * case["Q"]
    e = 4 if case["act"] == "f32" else 2
    rows = M if case["Q"] == 1 else M * (case["Q"] + 1) / (2 * case["Q"])
    return {"bytes": rows * case["V"] * e + M * 8, "flops": 0}


# ---- the definitions in 64 bits -----------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"prefill": _exact_prefill, "decode": _exact_decode,
            "tables": _exact_tables, "sample": _exact_sample}[s["op"]](s)


def _exact_token(s, S, x, gate, beta):
    """The recurrence for one token of n requests, S [n, H, V, K] in 64 bits,
    as matrix products."""
    H, D, n = s["H"], s["D"], S.shape[0]
    q, k, v = (x[:, i * H * D:(i + 1) * H * D].reshape(n, H, D)
               for i in range(3))
    q = q / torch.sqrt((q ** 2).sum(-1, keepdim=True) + 1e-6) / math.sqrt(D)
    k = k / torch.sqrt((k ** 2).sum(-1, keepdim=True) + 1e-6)
    z = gate.reshape(n, H, D) + s["dt_bias"].double()
    A = s["A_log"].double().exp()[None, :, None]
    if s["lb"] is not None:
        g = s["lb"] * torch.sigmoid(A * z)
    else:
        g = -A * torch.nn.functional.softplus(z, threshold=20.0)
    S = S * g.exp()[:, :, None, :]
    read = torch.matmul(S, k[..., None])[..., 0]
    c = torch.sigmoid(beta)[..., None] * (v - read)
    S = torch.addcmul(S, c[..., None], k[:, :, None, :])
    return torch.matmul(S, q[..., None])[..., 0].reshape(n, H * D), S


def _exact_conv(s, window):
    """window [n, TAPS, C] -> the convolved and activated newest input."""
    y = torch.einsum("ntc,ct->nc", window, s["conv_weight"].double())
    return y * torch.sigmoid(y)


def _exact_prefill(s):
    d = torch.float64
    qsl = s["query_start_loc"].cpu().numpy()
    lens = qsl[1:] - qsl[:-1]
    by_length = np.argsort(-lens, kind="stable")     # the longest first
    dev = s["out"].device
    init = s["initial_state_indices"].cpu().numpy()[by_length]
    src = torch.as_tensor(init, device=dev).long()
    S = s["state"].to(d)[src] * (src > NULL)[:, None, None, None]
    starts = torch.as_tensor(qsl[:-1][by_length], device=dev).long()
    dst = s["state_indices"][torch.as_tensor(by_length, device=dev)].long()
    out, state = s["out"].to(d), s["state"].to(d)
    if s["conv"]:
        cs = s["conv_state"].to(d)
        cs = cs if s["dim_first"] else cs.transpose(1, 2)
        hist = cs[src, :, :TAPS - 1].transpose(1, 2) \
            * (src > NULL)[:, None, None]
        ends = cs.clone()
    for t in range(int(lens.max())):
        n = int((lens > t).sum())       # requests still running
        S, at = S[:n], starts[:n] + t
        x = s["mixed_qkv"][at].to(d)
        if s["conv"]:
            window = torch.cat([hist[:n], x[:, None]], 1)
            x, hist = _exact_conv(s, window), window[:, 1:]
        o, S = _exact_token(s, S, x, s["raw_gate"][at].to(d),
                            s["raw_beta"][at].to(d))
        out[at] = o
        m = int((lens > t + 1).sum())   # those that end with this token
        if m < n:
            state[dst[m:n]] = S[m:n]
            if s["conv"]:
                ends[dst[m:n], :, :TAPS - 1] = hist[m:n].transpose(1, 2)
    B = s["B"]
    r = (out, state[1:B + 1])
    if s["conv"]:
        e = ends[1:B + 1, :, :TAPS - 1]
        r += (e if s["dim_first"] else e.transpose(1, 2).contiguous(),)
    return r


def _exact_decode(s):
    d = torch.float64
    B, dst = s["B"], s["final_state_indices"].long()
    live = s["state_indices"] > NULL
    src = s["state_indices"][live].long()
    x = s["mixed_qkv"][live].to(d)
    state = s["state"].to(d)
    if s["conv"]:
        cs = s["conv_state"].to(d)
        cs = cs if s["dim_first"] else cs.transpose(1, 2)
        at = s["num_accepted_tokens"][live].long() - 1
        each = torch.arange(len(src), device=x.device)
        hist = torch.stack([cs[src].transpose(1, 2)[each, at + i]
                            for i in range(TAPS - 1)], 1)
        window = torch.cat([hist, x[:, None]], 1)
        x = _exact_conv(s, window)
        ends = cs.clone()
        ends[dst[live], :, :TAPS - 1] = window[:, 1:].transpose(1, 2)
    o, S = _exact_token(s, state[src], x, s["raw_gate"][live].to(d),
                        s["raw_beta"][live].to(d))
    out = torch.zeros(s["out"].shape, dtype=d, device=x.device)
    out[live] = o
    state[dst[live]] = S
    r = (out, state[B + 1:2 * B + 1])
    if s["conv"]:
        e = ends[B + 1:2 * B + 1, :, :TAPS - 1]
        r += (e if s["dim_first"] else e.transpose(1, 2).contiguous(),)
    return r


def _exact_tables(s):
    """Request by request, on the host."""
    h = {k: v.cpu().numpy().astype(np.int64) for k, v in s.items()
         if isinstance(v, torch.Tensor)}
    bs, cap, table = s["block"], s["cap"], h["block_table"].copy()
    B, width = s["B"], table.shape[1]
    free, used = h["free_blocks"], 0
    nb = h["num_blocks"].copy()
    o = dict(query_start_loc=np.zeros(B + 1, np.int64), new_num_blocks=nb,
             state_indices=np.zeros(B, np.int64),
             initial_state_indices=np.zeros(B, np.int64),
             final_state_indices=np.zeros(B, np.int64),
             positions=np.zeros(cap, np.int64),
             slot_mapping=np.full(cap, -1, np.int64))
    t = 0
    for b in range(B):
        r, q = h["request_indices"][b], max(int(h["query_lens"][b]), 0)
        c, have = int(h["num_computed_tokens"][r]), int(nb[r])
        need = min((c + q) // bs + 1, width)
        for j in range(have, need):
            table[r, j] = free[used] if used < len(free) else NULL
            nb[r] += used < len(free)
            used += 1
        at = lambda p: table[r, p // bs] if p // bs < width else NULL  # noqa: E731
        o["state_indices"][b] = at(c)
        o["initial_state_indices"][b] = at(c) if c > 0 else NULL
        o["final_state_indices"][b] = at(c + q)
        for i in range(q):
            o["positions"][t] = c + i
            if at(c + i) > NULL:
                o["slot_mapping"][t] = at(c + i) * bs + (c + i) % bs
            t += 1
        o["query_start_loc"][b + 1] = t
    o["num_allocated"] = np.array([used])
    o = {k: torch.as_tensor(v.astype(
        np.int64 if k == "slot_mapping" else np.int32)) for k, v in o.items()}
    return (o, torch.as_tensor(table.astype(np.int32)))


def _exact_sample(s):
    """Row by row, by the threshold pair (value, index) that ends the kept
    prefix."""
    qsl = s["query_start_loc"].cpu().numpy()
    x_all = s["logits"]
    M, V = x_all.shape
    tokens = s["tokens"].cpu().numpy().copy()
    host = {k: s[k].cpu().numpy() for k in ("temperature", "top_k", "top_p",
                                            "min_p", "uniform")}
    for b in range(s["B"]):
        T, k = float(host["temperature"][b]), int(host["top_k"][b])
        p, mp = float(host["top_p"][b]), float(host["min_p"][b])
        for m in range(qsl[b], qsl[b + 1]):
            x = x_all[m].double()
            if T <= 0:
                tokens[m] = int((x == x.max()).nonzero()[0])
                continue
            w = ((x - x.max()) / T).exp()
            idx = (w >= mp).nonzero()[:, 0] if mp > 0 \
                else torch.arange(V, device=x.device)
            ranked = idx[torch.sort(-x[idx], stable=True)[1]]
            if 0 < k < len(ranked):
                ranked = ranked[:k]
            if p < 1:
                mass = w[ranked].cumsum(0)
                n = int((mass < p * mass[-1]).sum()) + 1
                ranked = ranked[:n]
            kept = torch.sort(ranked)[0]
            mass = w[kept].cumsum(0)
            u = float(host["uniform"][m])
            n = int((mass <= u * mass[-1]).sum())
            tokens[m] = int(kept[min(n, len(kept) - 1)])
    r = (torch.as_tensor(tokens),)
    if s["draft_tokens"] is not None:
        d = s["draft_tokens"].cpu().numpy()
        acc = np.ones(s["B"], np.int32)
        nxt = np.zeros(s["B"], np.int32)
        for b in range(s["B"]):
            at = qsl[b]
            while at + 1 < qsl[b + 1] and tokens[at] == d[at + 1]:
                at += 1
            acc[b], nxt[b] = at - qsl[b] + 1, tokens[at]
        r += (torch.as_tensor(acc), torch.as_tensor(nxt))
    return r
