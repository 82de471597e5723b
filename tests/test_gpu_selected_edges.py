"""Selected-block attention on the GPU where masks, ranges and calls at once could make it go wrong.

Tolerances as counted in test_gpu_selected.py, from which the helpers come.
"""

import pytest
import torch

import free_block_sparse_response_b200 as spr
import selected_reference as R
from test_gpu_selected import _built, DEV, gen_of, rnd  # noqa: F401

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------- causal: nothing of a later key

@pytest.mark.parametrize("first,top", [(0, 2), (1, 2), (0, 1)])
def test_causal_selection_without_local_blocks_sees_no_later_key(first, top):
    """A query's own block holds later keys, so its mean must not decide: it is always selected."""
    gen = gen_of(70)
    n, at = 256, 220
    q, k = rnd(gen, 1, 4, n, 64), rnd(gen, 1, 2, n, 64)
    cfg = spr.SelectConfig(block=64, top=top, causal=True, n_first=first)
    lens = torch.tensor([n], device=DEV)
    res = []
    for later in (False, True):
        if later:
            k[:, :, at:] = 5 * rnd(gen, 1, 2, n - at, 64)
        ws = spr.selected_workspace(q, k, cfg)
        mean = spr.key_means(k, 64)
        sel = spr.select_blocks(q, mean, n, cfg, ws)
        # all first blocks and no room beside them: the own block is not scored either
        own = 1 if first < top else 0
        assert torch.equal(sel, R.select(q, mean, n, 64, top, lens, torch.zeros_like(lens), True, first, own))
        spr.check(ws)
        res.append(sel[:, :, :at])
    assert torch.equal(*res)


def test_a_cache_and_a_prompt_select_the_same_without_local_blocks():
    """Token by token over a cache (the means of what is there) against the prompt's means."""
    gen = gen_of(71)
    n = 700
    q, k = rnd(gen, 1, 2, n, 64), rnd(gen, 1, 1, n, 64)
    cfg = spr.SelectConfig(block=64, top=3, causal=True)
    ws = spr.selected_workspace(q, k, cfg)
    prompt = spr.select_blocks(q, spr.key_means(k, 64), n, cfg, ws)
    means = torch.zeros(1, 1, 11, 64, device=DEV)
    for t in range(n):
        lens = torch.tensor([t + 1], dtype=torch.int32, device=DEV)
        spr.key_means(k, 64, kv_len=lens, kv_start=lens - 1, max_new=1, out=means)
        one = spr.select_blocks(q[:, :, t:t + 1], means, n, cfg, ws, kv_len=lens, q_start=lens - 1)
        assert torch.equal(one, prompt[:, :, t:t + 1]), t
    spr.check(ws)


def test_a_selection_of_first_blocks_alone_takes_nothing_else():
    """n_first = top: the first blocks, and no score of a block with later keys."""
    gen = gen_of(72)
    n = 900
    q, k = rnd(gen, 1, 2, n, 64), rnd(gen, 1, 2, n, 64)
    cfg = spr.SelectConfig(block=64, top=2, causal=True, n_first=2)
    ws = spr.selected_workspace(q, k, cfg)
    sel = spr.select_blocks(q, spr.key_means(k, 64), n, cfg, ws)
    want = torch.tensor([0, 1], dtype=torch.int32, device=DEV).expand(1, 2, n, 2).clone()
    want[:, :, :64, 1] = -1
    assert torch.equal(sel, want)
