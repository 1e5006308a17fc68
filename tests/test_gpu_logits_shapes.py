"""Changes of logits over shapes of a launch: token histories with more columns
than any request fills, many requests of which a few exceed the table, and
more rows than a grid takes."""
import numpy as np
import pytest
import torch

import linear_attention_speculative_amd as kda
from tests.latent_check import f64
from tests.test_gpu_blocks import i32
from tests.test_gpu_logits import check, expect, make

DEV = "cuda"


@pytest.mark.gpu
@pytest.mark.parametrize("B,V,known", [
    (300, 700, {7: 7000, 90: 20000, 299: 6500}),      # a few long ones
    (300, 700, {}),                                   # none
    (3, 9001, {0: 6145, 1: 6144, 2: 20000}),
    (40, 131072, {3: 9000, 17: 12000}),
    (1100, 64, {0: 6200, 1023: 6300, 1024: 6400, 1099: 6500}),
])
def test_more_columns_than_tokens(B, V, known):
    rng = np.random.RandomState(B)
    kw = make(list(rng.randint(0, 4, size=B)), V, act="bf16", hist=20000,
              seed=B)
    lens = rng.randint(0, 20, size=B + 2)
    rows = kw["request_indices"].cpu().numpy()
    for b, n in known.items():
        lens[rows[b]] = n
        kw["frequency_penalty"][b] = 0.5
    kw["token_lens"] = i32(lens)
    kw["prompt_lens"] = i32(lens // 3)
    before = f64(kw["logits"])
    ref, size = expect(kw)
    kda.adjust_logits(**kw)
    torch.cuda.synchronize()
    check(kw, before, ref, size)


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_more_rows_than_a_grid(act):
    """Masks of rows on both sides of the 65535th."""
    kw = make([30000, 35000, 1, 5100], 41, act=act, seed=2, tail=7, masks=5)
    for n in ("draft_tokens", "token_ids", "prompt_lens", "token_lens",
              "request_indices", "repetition_penalty", "frequency_penalty",
              "presence_penalty"):
        del kw[n]
    assert kw["logits"].shape[0] > 65535 + 4000
    before = f64(kw["logits"])
    ref, size = expect(kw)
    assert np.isinf(ref[65500:65535]).any() and np.isinf(ref[65536:]).any()
    kda.adjust_logits(**kw)
    torch.cuda.synchronize()
    check(kw, before, ref, size)
