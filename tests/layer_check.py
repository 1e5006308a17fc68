"""Inputs of a KDA layer for the prefill and decode tests, the library's calls
on them and the comparison with the fp64 oracle."""
import numpy as np
import torch

import oracle

TORCH = {"f32": torch.float32, "bf16": torch.bfloat16}

# An output or state element is a few dot products over at most 128 channels
# in fp32 with lane trees (under 40 roundings on the way to it), of terms that
# sum to at most about 8 times the largest result: 40 * 2^-24 * 8.  A decode
# step ends there; a prefill's states feed the next chunk, but decay or are
# overwritten as fast (the delta rule forgets what it replaces), which the
# same factor 8 covers for the lengths tested.
F32_TOL = 2e-5
# A prefill's bf16 outputs (not its states) are sums of products whose two
# operands are rounded to fp16: each term is off by at most 2 * 2^-11 of
# itself, the sum of n independent such errors has a standard deviation of at
# most 2 * 2^-11 / sqrt(3) of the terms' 2-norm, which is that of the output,
# and the largest output is at least three times the typical one: 2^-10 of the
# largest is over five standard deviations.
OPERAND_TOL = 2.0 ** -10
HALF_STEP = {"f32": 0.0, "bf16": float(torch.finfo(torch.bfloat16).eps) / 2}


def f64(t):
    return t.detach().to("cpu").to(torch.float64).numpy()


def i32(a, device):
    return torch.as_tensor(np.asarray(a), dtype=torch.int32).to(device)


def make_layer(T, N, H, D, Q, act="bf16", weight=None, out="act", lb=None,
               conv=True, dim_first=True, seed=0, device="cuda", row_pad=0,
               slot_pad=0, gentle=True):
    """Seeded tensors of one layer.  `gentle`: steps as trained gates have
    them (decays near 1); otherwise strong random decays."""
    g = torch.Generator().manual_seed(seed * 7919 + 5)

    def randn(*shape, std=1.0):
        return torch.randn(shape, generator=g) * std

    dt, wdt = TORCH[act], TORCH[weight or act]
    C = 3 * H * D

    def act_rows(cols):
        return randn(T, cols + row_pad).to(dt).to(device)[:, :cols]

    bias = randn(H, D, std=0.1)
    if gentle and lb is None:
        bias = torch.log(torch.expm1(torch.exp(
            torch.rand((H, D), generator=g) * np.log(100.0) + np.log(1e-3))))
    pool = randn(N, H * D * D + slot_pad, std=0.1).to(device)
    kw = dict(
        mixed_qkv=act_rows(C), raw_gate=act_rows(H * D),
        raw_beta=act_rows(H),
        A_log=torch.log(1 + 15 * torch.rand(H, generator=g)).to(device),
        dt_bias=bias.to(device), lower_bound=lb,
        state=pool[:, :H * D * D].unflatten(1, (H, D, D)),
        out=torch.full((T, H * D), 7.0, device=device,
                       dtype=dt if out == "act" else TORCH[out]))
    if conv:
        shape = (N, C, Q + 2) if dim_first else (N, Q + 2, C)
        kw.update(conv_state=randn(*shape).to(dt).to(device),
                  conv_weight=randn(C, 4, std=0.5).to(wdt).to(device),
                  spec_query_len=Q, conv_dim_first=dim_first)
    return kw


def reference(kw, qsl, slots, initial, accepted=None, null=0):
    """The oracle's results on these inputs (call before the library's)."""
    cs = kw.get("conv_state")
    if cs is not None and not kw["conv_dim_first"]:
        cs = cs.transpose(1, 2)
    return oracle.layer_tokens(
        mixed_qkv=f64(kw["mixed_qkv"]), raw_gate=f64(kw["raw_gate"]),
        raw_beta=f64(kw["raw_beta"]), A_log=f64(kw["A_log"]),
        dt_bias=f64(kw["dt_bias"]), state=f64(kw["state"]),
        out=f64(kw["out"]), query_start_loc=qsl, state_indices=slots,
        initial_state_indices=initial,
        conv_state=None if cs is None else f64(cs),
        conv_weight=None if cs is None else f64(kw["conv_weight"]),
        num_accepted_tokens=accepted,
        use_lower_bound=kw["lower_bound"] is not None,
        lower_bound=kw["lower_bound"] or 0.0, null_block_id=null)


def compare(kw, ref, written, tol=F32_TOL, pairs=False):
    """Outputs and states within the tolerances; slots outside `written` and
    every conv-state entry bit for bit.  `pairs`: the outputs of a prefill,
    whose bf16 ones come from fp16 operands."""
    o, r = f64(kw["out"]), ref["out"]
    act = "bf16" if kw["out"].dtype == torch.bfloat16 else "f32"
    top = np.max(np.abs(r), initial=1e-30)
    near = OPERAND_TOL if pairs and act == "bf16" else tol
    assert np.all(np.abs(o - r) <= HALF_STEP[act] * np.abs(r) + near * top), \
        np.max(np.abs(o - r)) / top
    s, r = f64(kw["state"]), ref["state"]
    keep = np.ones(s.shape[0], bool)
    keep[written] = False
    assert np.array_equal(s[keep], r[keep])
    for i in written:
        top = np.max(np.abs(r[i]), initial=1e-30)
        err = np.max(np.abs(s[i] - r[i])) / top
        assert err <= tol, (i, err)
    if ref["conv_state"] is not None:
        cs = kw["conv_state"] if kw["conv_dim_first"] \
            else kw["conv_state"].transpose(1, 2)
        assert np.array_equal(f64(cs), ref["conv_state"])
