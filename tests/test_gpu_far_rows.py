"""Operators on caches and logits whose rows lie past 32-bit offsets, in bytes
and in elements: every tensor of a call with rows 64 MiB and more apart."""
import pytest
import torch

import linear_attention_speculative_amd as kda
from tests import test_gpu_latent as latent
from tests import test_gpu_latent_prompt as prompt
from tests import test_gpu_logits as logits

DEV = "cuda"


@pytest.fixture(scope="module")
def memory():
    return torch.empty(7 << 30, dtype=torch.uint8, device=DEV)


def far(t, memory, shift):
    """t with its first dimension spread over the memory, its rows `shift`
    bytes behind a multiple of the step."""
    flat = memory.view(t.dtype)
    step = flat.numel() // t.shape[0] // 256 * 256
    shift //= t.element_size()
    wide = flat.as_strided(t.shape, (step, *t[0].contiguous().stride()), shift)
    assert shift + t[0].numel() <= step
    assert (t.shape[0] - 1) * step * t.element_size() > 1 << 32
    wide.copy_(t)
    return wide


def spread(kw, names, memory):
    at = 0
    for n in names:
        kw[n] = far(kw[n], memory, at)
        at += 1 << 18


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_latent_attention(memory, act):
    kw = latent.make([4, 9, 27], [40, 3, 65], H=4, R=128, P=64, block=16,
                     act=act, seed=3)
    kw["out"].zero_()
    spread(kw, ("q", "out", "lse", "cache"), memory)
    ref = latent.expect(kw)
    latent.run(kw)
    torch.cuda.synchronize()
    latent.check(kw, ref, act)


@pytest.mark.gpu
def test_latent_write(memory):
    g = torch.Generator().manual_seed(1)
    rows = torch.randn((50, 128), generator=g).to(DEV)
    cache = torch.zeros((60, 1, 128), device=DEV)
    kw = dict(latent=rows, cache=cache)
    spread(kw, ("latent", "cache"), memory)
    slots = torch.arange(59, 9, -1, device=DEV)
    kda.latent_write(**kw, slot_mapping=slots)
    torch.cuda.synchronize()
    assert torch.equal(kw["cache"][slots, 0], rows)
    assert (kw["cache"][:10] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_prefill(memory, act):
    kw = prompt.prompt([33, 64], [50, 64], H=2, D=64, P=64, act=act, seed=4)
    kw["out"].zero_()
    spread(kw, ("q", "key", "value", "rope_key", "out", "lse"), memory)
    ref = prompt.expect(kw)
    kda.latent_prefill(**kw)
    torch.cuda.synchronize()
    prompt.check(kw, ref, act)


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_expand(memory, act):
    kw = prompt.expansion([40, 30], H=3, D=64, R=128, P=64, block=16, act=act,
                          seed=5)
    names = ("key", "value", "rope_key")
    for n in names:
        kw[n].zero_()
    spread(kw, names, memory)
    ref = prompt.expand_expect(kw)
    kda.latent_expand(**kw)
    torch.cuda.synchronize()
    prompt.expand_check(kw, ref, act)


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_logits(memory, act):
    kw = logits.make([4, 1, 0, 20], 9000, act=act, seed=6)
    spread(kw, ("logits",), memory)
    before = logits.f64(kw["logits"])
    ref, size = logits.expect(kw)
    kda.adjust_logits(**kw)
    torch.cuda.synchronize()
    logits.check(kw, before, ref, size)
