"""GPU checks of gdn_paged_attention_kv8 for batches padded with requests that
have no new tokens (a capacity of slots kept for a captured graph): a prompt
whose tokens are fewer than the slots goes through the few-rows kernel, with
several row tiles per request.  Bounds as in test_gpu_serving_attention."""
import numpy as np
import pytest
import torch

from test_gpu_serving_attention import Case
from test_gpu_serving_attention_splits import check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,hq,hk", [(64, 4, 2), (128, 40, 1), (256, 8, 4)])
@pytest.mark.parametrize("slots", [129, 130, 131, 700])
def test_prompts_among_empty_slots(d, hq, hk, slots):
    """130 new tokens in two prompts and a decode row; equal to bounds on both sides of as many slots."""
    r = np.random.default_rng(slots)
    lens = [(0, 0)] * slots
    for at, one in zip(sorted(r.choice(slots, 5, replace=False)), [(90, 40), (33, 1), (100, 89), (50, 0), (7, 0)]):
        lens[at] = one
    c = Case(slots, lens, hq, hk, d, 16)
    check(c)
    check(c, window=25)
    check(c, causal=False)


@pytest.mark.parametrize("d", [64, 256])
def test_a_long_prompt_among_empty_slots(d):
    """Parts of the keys in the few-rows kernel, most row tiles not their request's first."""
    c = Case(7, [(0, 0)] * 60 + [(3000, 50)] + [(20, 0)] * 40, 4, 1, d, 16, spread=2.0)
    for longest in (3000, 2 ** 31 - 1):
        check(c, longest=longest)
    assert torch.equal(check(c, window=9), check(c, window=9))
