"""Every path of the chunked prefill against the token-by-token fp64 oracle:
state kernels of two, four and eight waves on both sides of the rule that
chooses them, decays that need the row-by-row form of the chunk kernel at every
head dim, in one sub-block or both, and products of decays on both sides of
its border; and malformed offsets between guarded buffers."""
import numpy as np
import pytest
import torch

import linear_attention_speculative_amd as kda
from tests.layer_check import F32_TOL, HALF_STEP, f64, i32, make_layer, \
    reference
from tests.test_gpu_prefill import DEV, check, run, workspace

BORDER = 1e-37         # product of a sub-block's decays below which it is used


def close(kw, ref, written, tol=F32_TOL):
    """As the layer's own comparison, with the bound of fp32 outputs for bf16
    ones too (beside the rounding to bf16)."""
    o, r = f64(kw["out"]), ref["out"]
    act = "bf16" if kw["out"].dtype == torch.bfloat16 else "f32"
    top = np.abs(r).max()
    assert np.all(np.abs(o - r) <= HALF_STEP[act] * np.abs(r) + tol * top)
    s, r = f64(kw["state"]), ref["state"]
    for i in range(len(s)):
        if i in written:
            err = np.abs(s[i] - r[i]).max() / np.abs(r[i]).max()
            assert err <= tol, (i, err)
        else:
            assert np.array_equal(s[i], r[i]), i


# ---- waves of a state kernel: few (request, head) pairs, more, many ----------

def waves(B, H, D, out_f32):
    """Waves of a workgroup by the rule on pairs and state row tiles."""
    tiles = D // 16
    if tiles > 4 and not out_f32 and B * H * (tiles // 4) > 256:
        return 8
    if tiles > 2 and B * H * (tiles // 2) > 256:
        return 4
    return min(tiles, 2)


@pytest.mark.gpu
@pytest.mark.parametrize("B,H,D,out,want", [
    (4, 16, 128, "act", 2), (5, 13, 128, "act", 4), (8, 16, 128, "act", 4),
    (3, 43, 128, "act", 8), (11, 12, 128, "act", 8),
    (4, 16, 128, "f32", 2), (5, 13, 128, "f32", 4), (7, 20, 128, "f32", 4),
    (8, 16, 64, "act", 2), (3, 43, 64, "act", 4), (10, 13, 64, "f32", 4),
    (40, 13, 32, "act", 2), (130, 2, 16, "act", 1)])
def test_waves_of_the_state_kernel(B, H, D, out, want):
    """Ragged prompts of up to four chunks, an empty one, a null slot, fresh
    and continued states."""
    assert waves(B, H, D, out == "f32") == want
    rng = np.random.RandomState(B * H + D)
    lens = rng.randint(1, 50 if B > 20 else 115, size=B)
    lens[0] = 107
    if B > 3:
        lens[2] = 0
        lens[3] = 96
    perm = 1 + rng.permutation(2 * B)
    slots, initial = perm[:B].copy(), perm[B:].copy()
    initial[::3] = 0
    if B > 3:
        slots[1] = 0
    kw = make_layer(int(lens.sum()) + 2, 2 * B + 2, H, D, 4, act="bf16",
                    out=out, seed=B + H, dim_first=H % 2 == 0)
    qsl = np.concatenate([[0], np.cumsum(lens)])
    ref = reference(kw, qsl, slots, initial)
    run(kw, qsl, slots, initial)
    close(kw, ref, [s for s, n in zip(slots, lens) if s > 0 and n > 0])
    cs = kw["conv_state"] if kw["conv_dim_first"] \
        else kw["conv_state"].transpose(1, 2)
    assert np.array_equal(f64(cs), ref["conv_state"])


# ---- decays that leave fp32's range inside a sub-block -----------------------

def log_decays(kw):
    """The gates in float64 (lower bound or softplus form)."""
    x = f64(kw["raw_gate"]).reshape(-1, *kw["dt_bias"].shape) + \
        f64(kw["dt_bias"])
    A = np.exp(f64(kw["A_log"]))[:, None]
    if kw["lower_bound"] is not None:
        return kw["lower_bound"] / (1 + np.exp(-A * x))
    return -A * np.logaddexp(0, x)


def deep_blocks(kw):
    """Per 16 tokens, whether some channel's decays multiply up to less than
    the border."""
    g = log_decays(kw)
    return [bool((g[s:s + 16].sum(axis=0) < np.log(BORDER)).any())
            for s in range(0, len(g), 16)]


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("D", [16, 32, 64, 128])
@pytest.mark.parametrize("strong", [40.0, 2000.0])
def test_strong_decays_at_every_head_dim(strong, D, act):
    """Every tenth gate or so empties its channel, others keep all; the last
    chunk is partial."""
    L, H = 90, 2
    kw = make_layer(L, 4, H, D, 4, act=act, conv=False, seed=21 + D)
    g = torch.Generator().manual_seed(D)
    gate = torch.randn(L, H * D, generator=g)
    gate[torch.rand(L, H * D, generator=g) < 0.1] = strong
    gate[torch.rand(L, H * D, generator=g) < 0.3] = -60.0
    kw["raw_gate"] = gate.to(kw["raw_gate"].dtype).to(DEV)
    kw["dt_bias"].zero_()
    assert sum(deep_blocks(kw)) >= 4
    ref = reference(kw, [0, L], [1], [2])
    run(kw, [0, L], [1], [2])
    close(kw, ref, [1])


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("D", [16, 32, 64, 128])
@pytest.mark.parametrize("where", [(0, 16), (16, 32), (32, 48), (48, 61)])
def test_one_deep_sub_block(where, D, act):
    """One of the two sub-blocks of a chunk decays past the border, in a few
    channels of one head, the other does not."""
    L, H = 61, 3
    kw = make_layer(L, 4, H, D, 4, act=act, conv=False, seed=31 + D)
    s, e = where
    kw["raw_gate"][s:e:3, D + 2:D + 9:2] = 300.0
    assert deep_blocks(kw) == [s == t for t in range(0, L, 16)]
    ref = reference(kw, [0, L], [1], [2])
    run(kw, [0, L], [1], [2])
    close(kw, ref, [1])


@pytest.mark.gpu
@pytest.mark.parametrize("D", [16, 32, 64, 128])
@pytest.mark.parametrize("total", [-60.0, -84.9, -85.1, -85.3, -87.5, -100.0])
def test_products_of_decays_around_the_border(total, D):
    """Sub-blocks whose decays multiply up to e^-60 .. e^-100 (the border lies
    at e^-85.2), spread over the tokens or all in one, first or last; keys
    and queries with channels of 1e-3 and less."""
    L, H = 64, 4
    kw = make_layer(L, 4, H, D, 4, act="f32", conv=False, seed=41 + D,
                    lb=-100.0)
    kw["A_log"].zero_()
    kw["dt_bias"].zero_()
    gate = torch.full((L, H, D), -40.0)           # 100 e^-40: none
    logit = lambda g: float(np.log(g / (100.0 - g)))  # noqa: E731
    gate[:, 0] = logit(-total / 16)
    for h, t in ((1, 0), (2, 15), (3, 7)):
        gate[t::16, h] = logit(min(-total, 99.99))
    kw["raw_gate"] = gate.reshape(L, H * D).to(DEV)
    kw["mixed_qkv"][:, :2 * H * D:3] *= 1e-3
    kw["mixed_qkv"][:, 1:2 * H * D:5] *= 1e-6
    want = total < np.log(BORDER)
    assert deep_blocks(kw) == [want] * 4
    ref = reference(kw, [0, L], [1], [2])
    run(kw, [0, L], [1], [2])
    close(kw, ref, [1])


# ---- malformed offsets -------------------------------------------------------

def guarded(t, margin=4096):
    """A contiguous copy of a tensor inside a larger allocation: (the copy,
    the allocation's bytes, the copy's place in them)."""
    n = t.numel() * t.element_size()
    raw = torch.full((n + 2 * margin,), 0x5a, dtype=torch.uint8, device=DEV)
    view = raw[margin:margin + n].view(t.dtype).view(t.shape)
    view.copy_(t)
    return view, raw, margin, n


@pytest.mark.gpu
@pytest.mark.parametrize("conv", [True, False])
@pytest.mark.parametrize("qsl", [
    [-5, 90, 20, 10 ** 9], [33, 0, 70, 0], [40, 5, 5, 39], [40, 30, 20, 10],
    [0, 40, 0, 40], [-(2 ** 31), 2 ** 31 - 1, 0, 2 ** 31 - 1],
    [7, 7, 3, 3]])
def test_malformed_offsets_between_guards(qsl, conv):
    """Offsets that run backwards, overlap or leave the rows: nothing outside
    the tensors is written, and of the slots only those named."""
    kw = make_layer(40, 7, 3, 32, 4, act="f32", conv=conv, seed=3)
    kw["workspace"] = workspace(kw, 3)
    names = ["out", "state", "workspace"] + ["conv_state"] * conv
    raws = {}
    for n in names:
        kw[n], raw, at, size = guarded(kw[n])
        raws[n] = (raw, at, size)
    inputs = {n: v.clone() for n, v in kw.items()
              if isinstance(v, torch.Tensor) and n not in names}
    before = {n: kw[n].clone() for n in ("state", "conv_state") if n in kw}
    args = dict(kw, query_start_loc=i32(qsl, DEV),
                state_indices=i32([1, 4, 6], DEV),
                initial_state_indices=i32([2, 0, 3], DEV))
    (kda.conv_prefill if conv else kda.prefill_qkv)(**args)
    torch.cuda.synchronize()
    for n, (raw, at, size) in raws.items():
        assert bool((raw[:at] == 0x5a).all()), n
        assert bool((raw[at + size:] == 0x5a).all()), n
    for n, old in before.items():
        for slot in (0, 2, 3, 5):
            assert torch.equal(kw[n][slot], old[slot]), (n, slot)
    for n, old in inputs.items():
        assert torch.equal(kw[n], old), n


@pytest.mark.gpu
@pytest.mark.parametrize("D,H,B", [(16, 2, 3), (128, 43, 3)])
def test_ordinary_call_between_guards(D, H, B):
    """The same guards around a call with results, partial last chunks and
    rows behind the last request."""
    lens = [70, 1, 33]
    qsl = np.concatenate([[0], np.cumsum(lens)])
    kw = make_layer(int(qsl[-1]) + 5, 7, H, D, 4, act="bf16", seed=4)
    ref = reference(kw, qsl, [1, 4, 6], [2, 0, 3])
    kw["workspace"] = workspace(kw, B)
    raws = {}
    for n in ("out", "state", "conv_state", "workspace"):
        kw[n], raw, at, size = guarded(kw[n])
        raws[n] = (raw, at, size)
    kda.conv_prefill(**kw, query_start_loc=i32(qsl, DEV),
                     state_indices=i32([1, 4, 6], DEV),
                     initial_state_indices=i32([2, 0, 3], DEV))
    torch.cuda.synchronize()
    close(kw, ref, [1, 4, 6])
    for n, (raw, at, size) in raws.items():
        assert bool((raw[:at] == 0x5a).all()), n
        assert bool((raw[at + size:] == 0x5a).all()), n


@pytest.mark.gpu
def test_prompts_of_every_length_to_three_chunks():
    """All lengths from 0 to 97 in one batch."""
    lens = np.random.RandomState(5).permutation(98)
    kw = make_layer(int(lens.sum()), 99, 2, 32, 4, act="bf16", seed=6)
    check(kw, lens, 1 + np.arange(98), None)
