"""Selected-block attention on the GPU where masks, ranges and calls at once could make it go wrong.

Tolerances as counted in test_gpu_selected.py, from which the helpers come.
"""
import math
import threading

import pytest
import torch

import free_block_sparse_response_b200 as spr
import selected_reference as R
from test_gpu_selected import _built, BF, close, DEV, E, F, gen_of, problem, rnd, U  # noqa: F401

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


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("times", [0.1, 3.0, 100.0])
def test_causal_rows_are_the_same_to_the_bit_whatever_comes_later(times, dtype):
    """The whole call on two inputs that differ from a key on: the rows before it."""
    gen = gen_of(83)
    n, at = 500, 333
    q, k, v = (rnd(gen, 2, h, n, 128, dtype=dtype) for h in (4, 2, 2))
    cfg = spr.SelectConfig(block=128, top=3, causal=True)
    res = []
    for later in (False, True):
        if later:
            k[:, :, at:], v[:, :, at:] = (times * rnd(gen, 2, 2, n - at, 128, dtype=dtype) for _ in range(2))
        res.append(spr.block_attention(q, k, v, cfg)[:, :, :at].clone())
    assert torch.equal(*res)


HIDDEN = [(1e30, BF), (-1e38, BF), (math.nan, BF), (math.inf, BF), (1e30, F), (math.nan, F), (-math.inf, F)]


@pytest.mark.parametrize("d,block", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("what", ["k", "v"])
@pytest.mark.parametrize("value,dtype", HIDDEN, ids=str)
def test_hidden_keys_of_the_own_block_do_not_reach_a_query(d, block, what, value, dtype):
    """Rows before the keys that hold `value` are as without them: output, log-sum-exp and dq, through
    the lists; to the bit where the value is finite."""
    n, at = 300, 200
    q, k, v, lens, starts, cfg = problem((1, 4, 2, n, n, d, block, 2, True, 0, 1, None, dtype), 73)
    dout = rnd(gen_of(74), *q.shape, dtype=dtype)
    ws = spr.selected_workspace(q, k, cfg, backward=True)
    sel = spr.select_blocks(q, spr.key_means(k, block), n, cfg, ws)
    bad = {"k": k.clone(), "v": v.clone()}
    bad[what][:, :, at:] = value
    res = []
    for kk, vv in ((k, v), (bad["k"], bad["v"])):
        out, lse = spr.selected_attn(q, kk, vv, sel, cfg, ws)
        dq = spr.selected_attn_backward(dout, q, kk, vv, out, lse, sel, cfg, ws)[0]
        res.append([t[:, :, :at].clone() for t in (out, lse, dq)])
    spr.check(ws)
    if math.isfinite(value):
        assert all(torch.equal(a, b) for a, b in zip(*res))
    ok = R.mask(sel, n, n, block, lens, starts, True)
    want, wlse, p = R.attention(q, k, v, ok, d ** -0.5)
    size = p @ v.double().abs().repeat_interleave(2, 1)
    out, lse, dq = res[1]
    close(out, want[:, :, :at], (U[dtype] * want.abs() + (U[dtype] + E) * size)[:, :, :at], "out")
    close(lse, wlse[:, :, :at], 1e-5 * (1 + wlse[:, :, :at].abs()), "lse")
    whole = torch.cat([out, want[:, :, at:].to(dtype)], 2)
    grads, sizes, noise = R.backward(dout, q, k, v, ok, d ** -0.5, out=whole)
    bound = U[dtype] * grads[0].abs() + U[dtype] * sizes[0] * 1.01 + E * noise[0]
    close(dq, grads[0][:, :, :at], bound[:, :, :at], "dq")


@pytest.mark.parametrize("n", [1, 3, 11])
@pytest.mark.parametrize("value", [1e30, math.nan, -math.inf])
def test_hidden_keys_do_not_reach_a_query_of_a_few_tokens(n, value):
    """The same for a few tokens inside a longer cache: keys past a token's own position."""
    q, k, v, lens, starts, cfg = problem((1, 4, 2, n, 300, 128, 64, 2, True, 0, 1, None, BF), 75)
    starts = torch.full_like(starts, 200 - n)
    bad = {"k": k.clone(), "v": v.clone()}
    bad["k"][:, :, 200:], bad["v"][:, :, 200:] = value, value
    ws = spr.selected_workspace(q, k, cfg)
    sel = spr.select_blocks(q, spr.key_means(k, 64, kv_len=starts + n), 300, cfg, ws, q_start=starts)
    want = spr.selected_attn(q, k, v, sel, cfg, ws, q_start=starts)
    got = spr.selected_attn(q, bad["k"], bad["v"], sel, cfg, ws, q_start=starts)
    spr.check(ws)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


# ------------------------------------------------------------------- ranges

@pytest.mark.parametrize("n,d,block", [(3, 128, 64), (200, 128, 64), (300, 128, 128), (200, 64, 64), (333, 64, 128)])
@pytest.mark.parametrize("size", [1e3, 1e8, 1e30])
def test_one_large_column_leaves_the_others(size, n, d, block):
    """Columns of very different sizes: each is as exact as its own values allow."""
    q, k, v, lens, starts, cfg = problem((1, 4, 2, n, 640, d, block, 4, False, 0, 0, None, BF), 76)
    v[..., 7] = (v[..., 7].float() * size).to(BF)
    v[..., 9] = (v[..., 9].float() / size).to(BF)
    v[..., 11] = 0
    ws = spr.selected_workspace(q, k, cfg)
    sel = spr.select_blocks(q, spr.key_means(k, block), 640, cfg, ws)
    rest = torch.empty_like(q)
    out, _ = spr.selected_attn(q, k, v, sel, cfg, ws, rest=rest)
    spr.check(ws)
    want, _, p = R.attention(q, k, v, R.mask(sel, n, 640, block, lens, starts, False), d ** -0.5)
    wide = p @ v.double().abs().repeat_interleave(2, 1)
    close(out, want, U[BF] * want.abs() + (U[BF] + E) * wide + 1e-37, "out")
    close(out.double() + rest.double(), want, U[BF] ** 2 * want.abs() + (U[BF] + E) * wide + 1e-37, "out + rest")
    assert (out[..., 11] == 0).all()


@pytest.mark.parametrize("n", [3, 200])
@pytest.mark.parametrize("size", [1e6, 1e20, 1e38])
def test_a_value_of_no_weight_leaves_the_others(size, n):
    """A key whose weight is exp(-250) and less, beside which its value is very large."""
    q, k, v, lens, starts, cfg = problem((1, 2, 2, n, 512, 128, 128, 3, False, 0, 0, None, BF), 84)
    q = q.abs()
    k[:, :, 70], v[:, :, 70] = -40, size
    ws = spr.selected_workspace(q, k, cfg)
    sel = torch.tensor([0, 1, 3], dtype=torch.int32, device=DEV).expand(1, 2, n, 3).contiguous()
    out, _ = spr.selected_attn(q, k, v, sel, cfg, ws)
    want, _, p = R.attention(q, k, v, R.mask(sel, n, 512, 128, lens, starts, False), 128 ** -0.5)
    assert float(p[..., 70].max()) < 1e-100
    wide = p @ v.double().abs()
    close(out, want, U[BF] * want.abs() + (U[BF] + E) * wide, "out")


@pytest.mark.parametrize("d,block", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("size", [1e-33, 1e-20, 1e16, 1e25])
def test_causal_values_of_any_size(size, d, block):
    """Rows that see a part of a block beside rows that see all of it, for values whose power of two the weights
    take and for some past that; the first keys smaller than the others by up to 10^5."""
    n = 300
    q, k, v, lens, starts, cfg = problem((1, 4, 2, n, n, d, block, 3, True, 0, 1, None, BF), 98)
    v = v.float() * size
    v[:, :, :150] *= torch.logspace(-5, 0, 150, device=DEV)[:, None]
    v = v.to(BF)
    ws = spr.selected_workspace(q, k, cfg)
    sel = spr.select_blocks(q, spr.key_means(k, block), n, cfg, ws)
    out, lse = spr.selected_attn(q, k, v, sel, cfg, ws)
    spr.check(ws)
    want, wlse, p = R.attention(q, k, v, R.mask(sel, n, n, block, lens, starts, True), d ** -0.5)
    wide = p @ v.double().abs().repeat_interleave(2, 1)
    close(out, want, U[BF] * want.abs() + (U[BF] + E) * wide + 1e-38, "out")
    close(lse, wlse, 1e-5 * (1 + wlse.abs()), "lse")


@pytest.mark.parametrize("d,block", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("size", [1e3, 1e8, 1e30])
def test_one_large_key_column_leaves_the_gradients_of_others(size, d, block):
    """dq in the columns beside one of very large keys (where the queries hold zeros)."""
    q, k, v, lens, starts, cfg = problem((1, 2, 2, 200, 640, d, block, 3, False, 0, 0, None, BF), 77)
    q[..., 7] = 0
    k[..., 7] = (k[..., 7].float() * size).to(BF)
    dout = rnd(gen_of(78), *q.shape)
    ws = spr.selected_workspace(q, k, cfg, backward=True)
    sel = spr.select_blocks(q, spr.key_means(k, block), 640, cfg, ws)
    out, lse = spr.selected_attn(q, k, v, sel, cfg, ws)
    got = spr.selected_attn_backward(dout, q, k, v, out, lse, sel, cfg, ws)
    spr.check(ws)
    ok = R.mask(sel, 200, 640, block, lens, starts, False)
    grads, sizes, noise = R.backward(dout, q, k, v, ok, d ** -0.5, out=out)
    for name, g, w, s, e in zip(("dq", "dk", "dv"), got, grads, sizes, noise):
        close(g, w, U[BF] * w.abs() + U[BF] * s * 1.01 + E * e + 1e-30, name)


# ------------------------------------------------------------------- selection

@pytest.mark.parametrize("n", [4, 700])
@pytest.mark.parametrize("top", [3, 6, 9])
@pytest.mark.parametrize("where", ["query", "mean"])
def test_nan_scores_are_reported_by_every_path(n, top, where):
    """A NaN score of any row is reported, also where the row takes all of its blocks."""
    gen = gen_of(79)
    q, mean = rnd(gen, 1, 2, n, 64), rnd(gen, 1, 2, 6, 64, dtype=F)
    if where == "query":
        q[0, 1, n // 2, 5] = math.nan
    else:
        mean[0, 1, 4, 5] = math.nan
    cfg = spr.SelectConfig(block=64, top=top)
    ws = spr.selected_workspace(q, torch.zeros(1, 2, 384, 64, device=DEV, dtype=BF), cfg)
    sel = spr.select_blocks(q, mean, 384, cfg, ws)
    with pytest.raises(spr.SparsePRError) as e:
        spr.check(ws)
    assert e.value.code == spr.ERR_NONFINITE
    if where == "mean" and top < 6:
        assert not (sel[0, 1] == 4).any()
    # a forced block's score decides nothing and is not one
    cfg = spr.SelectConfig(block=64, top=6, n_first=6)
    ws = spr.selected_workspace(q, torch.zeros(1, 2, 384, 64, device=DEV, dtype=BF), cfg)
    spr.select_blocks(q, mean, 384, cfg, ws)
    spr.check(ws)


def test_the_sum_of_a_large_group_is_decided_in_64_bits():
    """2,049 heads, the first 2^24 times the others, whose sum in 32 bits is lost beside it: the exact
    difference of the two blocks' scores is +2048, without them -2048, and 2^-16 |q| |m| is 512."""
    n, group, d = 600, 2049, 64
    q = torch.zeros(1, group, n, d, dtype=BF, device=DEV)
    q[:, 0, :, 0] = q[:, 0, :, 1] = 2.0 ** 24
    q[:, 1:, :, 0], q[:, 1:, :, 1] = 1.0, -1.0
    mean = torch.zeros(1, 1, 2, d, device=DEV)
    mean[0, 0, 0, :2] = torch.tensor([-1.0, 1.0])
    mean[0, 0, 1, :2] = torch.tensor([1.0, -1.0 - 6144 * 2.0 ** -24])
    cfg = spr.SelectConfig(block=64, top=1)
    ws = spr.selected_workspace(q, torch.zeros(1, 1, 128, d, dtype=BF, device=DEV), cfg)
    sel = spr.select_blocks(q, mean, 128, cfg, ws)
    lens = torch.tensor([128], device=DEV)
    assert torch.equal(sel, R.select(q, mean, 128, 64, 1, lens, torch.zeros_like(lens), False, 0, 0))
    assert (sel == 1).all()


@pytest.mark.parametrize("group,d", [(1, 128), (3, 128), (1, 64)])
def test_ties_of_a_dominating_dim_are_decided_by_the_rest(group, d):
    """One dim a thousand times the others and equal in all blocks: what is left differs in the last bits
    of a 32-bit sum."""
    n, nb, top = 700, 96, 7
    gen = gen_of(80)
    q, mean = rnd(gen, 1, group, n, d), rnd(gen, 1, 1, nb, d, dtype=F) * 1e-2
    q[..., 3] = 1000 + q[..., 3]
    mean[..., 3] = 10
    cfg = spr.SelectConfig(block=64, top=top)
    ws = spr.selected_workspace(q, torch.zeros(1, 1, nb * 64, d, dtype=BF, device=DEV), cfg)
    sel = spr.select_blocks(q, mean, nb * 64, cfg, ws)
    spr.check(ws)
    lens = torch.tensor([nb * 64], device=DEV)
    assert torch.equal(sel, R.select(q, mean, nb * 64, 64, top, lens, torch.zeros_like(lens), False, 0, 0))


def test_two_threads_select_among_different_numbers_of_blocks():
    """Host threads with workspaces and streams of their own: neither sees the other's sizes."""
    errors, results = [], {}

    def work(i, nb):
        try:
            gen = gen_of(81 + i)
            q, mean = rnd(gen, 1, 2, 640, 64), rnd(gen, 1, 2, nb, 64, dtype=F)
            cfg = spr.SelectConfig(block=64, top=5)
            stream = torch.cuda.Stream()
            stream.wait_stream(torch.cuda.default_stream())
            with torch.cuda.stream(stream):
                ws = spr.selected_workspace(q, torch.zeros(1, 2, nb * 64, 64, device=DEV, dtype=BF), cfg)
                for _ in range(3000):
                    sel = spr.select_blocks(q, mean, nb * 64, cfg, ws)
            stream.synchronize()
            spr.check(ws)
            results[i] = (q, mean, nb, sel)
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=a) for a in ((0, 20), (1, 128), (2, 64))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for q, mean, nb, sel in results.values():
        lens = torch.tensor([nb * 64], device=DEV)
        assert torch.equal(sel, R.select(q, mean, nb * 64, 64, 5, lens, torch.zeros_like(lens), False, 0, 0))


@pytest.mark.parametrize("n", [1, 2, 3])
@pytest.mark.parametrize("top", [4, 40])
def test_bad_entries_of_a_few_tokens(n, top):
    """The direct form skips and reports what the lists skip and report, and stops at a negative entry."""
    q, k, v, lens, starts, cfg = problem((1, 4, 2, n, 64 * 50, 64, 64, top, False, 0, 0, None, BF), 82)

    def rows(*entries):
        r = torch.full((1, 2, n, top), -1, dtype=torch.int32, device=DEV)
        pad = list(range(10, 10 + top - 4)) if top > 4 else []
        line = pad + list(entries)
        r[..., :len(line)] = torch.tensor(line, dtype=torch.int32, device=DEV)
        return r

    last = 10 + top - 4 if top > 4 else 1
    ws = spr.selected_workspace(q, k, cfg)
    want = spr.selected_attn(q, k, v, rows(last, last + 2), cfg, ws)
    spr.check(ws)
    for bad in ((last, last, last + 2, last + 1), (last, last + 2, 50, 1 << 30), (last, last - 1, last + 2, 0)):
        got = spr.selected_attn(q, k, v, rows(*bad), cfg, ws)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), bad
        with pytest.raises(spr.SparsePRError) as e:
            spr.check(ws)
        assert e.value.code == spr.ERR_INVALID_ARG
        spr.sparsepr.reset_workspace(ws)
    got = spr.selected_attn(q, k, v, rows(last, last + 2, -7, last + 3), cfg, ws)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    spr.check(ws)


# ------------------------------------------------------------------- rotary

def test_a_plan_with_other_frequencies_is_checked():
    """A plan is a plain tuple: its frequencies are held to its sizes, type and layout in every call."""
    q = rnd(gen_of(85), 1, 2, 10, 64)
    pos = torch.arange(10, dtype=torch.int32, device=DEV)[None]
    plan = spr.rotary_plan(64, DEV)
    want = spr.rotary(plan, pos, q)
    wide = torch.zeros(64, dtype=torch.float64, device=DEV)
    for bad in (plan.freqs[:31], plan.freqs.float(), wide[::2], plan.freqs.cpu(), torch.zeros(32, 2, dtype=torch.float64, device=DEV)):
        with pytest.raises(ValueError):
            spr.rotary(plan._replace(freqs=bad), pos, q)
    assert torch.equal(spr.rotary(plan._replace(freqs=plan.freqs.clone()), pos, q), want)


# ------------------------------------------------------------------- large calls

def by_head(q, k, v, sel, dout, out, cfg, lens, starts):
    """64-bit gradients and what bounds them (u |.| of bf16 and noise), query head by query head."""
    hq, hk, n, keys = q.shape[1], k.shape[1], q.shape[2], k.shape[2]
    grp, d = hq // hk, q.shape[3]
    dq, bq = torch.empty(q.shape, dtype=torch.float64, device=DEV), torch.empty(q.shape, dtype=torch.float64, device=DEV)
    dk, bk, dv, bv = (torch.zeros(k.shape, dtype=torch.float64, device=DEV) for _ in range(4))
    for h in range(hq):
        one, at = slice(h, h + 1), slice(h // grp, h // grp + 1)
        ok = R.mask(sel[:, at], n, keys, cfg.block, lens, starts, cfg.causal)
        grads, sizes, noise = R.backward(dout[:, one], q[:, one], k[:, at], v[:, at], ok, d ** -0.5, out=out[:, one])
        u = U[q.dtype]
        dq[:, one], bq[:, one] = grads[0], u * grads[0].abs() + u * sizes[0] * 1.01 + E * noise[0]
        for total, bound, i in ((dk, bk, 1), (dv, bv, 2)):
            total[:, at] += grads[i]
            bound[:, at] += u * sizes[i] * 1.01 + E * noise[i]
    return (dq, dk, dv), (bq, bk + U[q.dtype] * dk.abs(), bv + U[q.dtype] * dv.abs())


def test_gradients_of_several_chunks_of_heads():
    """Heads whose partial rows together pass the workspace's chunk: worked off in two."""
    gen = gen_of(86)
    n, h, d, top = 8192, 8, 128, 64
    q, k, v = rnd(gen, 1, h, n, d), rnd(gen, 1, h, n, d), rnd(gen, 1, h, n, d)
    dout = rnd(gen, 1, h, n, d)
    cfg = spr.SelectConfig(block=64, top=top)
    ws = spr.selected_workspace(q, k, cfg, backward=True)
    sel = spr.select_blocks(q, spr.key_means(k, 64), n, cfg, ws)
    out, lse = spr.selected_attn(q, k, v, sel, cfg, ws)
    got = spr.selected_attn_backward(dout, q, k, v, out, lse, sel, cfg, ws)
    spr.check(ws)
    lens = torch.tensor([n], device=DEV)
    grads, bounds = by_head(q, k, v, sel, dout, out, cfg, lens, torch.zeros_like(lens))
    for name, g, w, b in zip(("dq", "dk", "dv"), got, grads, bounds):
        close(g, w, b + 1e-30, name)


@pytest.mark.parametrize("dtype,causal", [(BF, False), (BF, True), (F, False)])
def test_gradients_of_a_head_cut_into_token_slices(dtype, causal):
    """A head whose partial rows alone pass the chunk: its tokens in slices, a key's gradient over all of them;
    rows and keys of a ragged length, blocks that some slices do not select, the same in every run."""
    gen = gen_of(87)
    n, keys, grp, top, d = 33000, 4096, 16, 16, 64
    q, k, v = rnd(gen, 1, grp, n, d, dtype=dtype), rnd(gen, 1, 1, keys, d, dtype=dtype), rnd(gen, 1, 1, keys, d, dtype=dtype)
    dout = rnd(gen, 1, grp, n, d, dtype=dtype)
    lens = torch.tensor([keys - 100], dtype=torch.int32, device=DEV)
    starts = torch.tensor([-n + keys if causal else 0], dtype=torch.int32, device=DEV)
    cfg = spr.SelectConfig(block=64, top=top, causal=causal)
    ws = spr.selected_workspace(q, k, cfg, backward=True)
    assert ws.numel() < 2 << 30
    sel = spr.select_blocks(q, spr.key_means(k, 64, kv_len=lens), keys, cfg, ws, kv_len=lens, q_start=starts)
    sel[:, :, 20000:][sel[:, :, 20000:] < 8] = -1  # (a row's first entries: its selection ends there)
    sel[:, :, :9000][sel[:, :, :9000] > 40] = -1
    out, lse = spr.selected_attn(q, k, v, sel, cfg, ws, kv_len=lens, q_start=starts)
    runs = [spr.selected_attn_backward(dout, q, k, v, out, lse, sel, cfg, ws, kv_len=lens, q_start=starts) for _ in range(2)]
    spr.check(ws)
    for a, b in zip(*runs):
        assert torch.equal(a, b)
    first = (sel < 0).int().argmax(-1, keepdim=True)
    ends = torch.where((sel < 0).any(-1, keepdim=True), first, top)
    live = torch.where(torch.arange(top, device=DEV) < ends, sel, -1)
    grads, bounds = by_head(q, k, v, live, dout, out, cfg, lens, starts)
    for name, g, w, b in zip(("dq", "dk", "dv"), runs[0], grads, bounds):
        close(g, w, b + 1e-30, name)
    assert (runs[0][1][:, :, keys - 100:] == 0).all() and (runs[0][2][:, :, keys - 100:] == 0).all()


# ------------------------------------------------------------------- autograd

def leaves(*ts):
    return [t.detach().clone().requires_grad_() for t in ts]


@pytest.mark.parametrize("dtype", [BF, F])
def test_autograd_gives_the_gradients_of_the_calls(dtype):
    """Rotation, selection and attention on tensors that need gradients: what the explicit calls give."""
    q, k, v, lens, starts, cfg = problem((2, 4, 2, 300, 300, 128, 64, 3, True, 1, 1, (300, 77), dtype), 90)
    k, v = k.nan_to_num(0), v.nan_to_num(0, 0, 0)
    plan = spr.rotary_plan(128, DEV, rot_dim=64)
    pos = torch.arange(300, dtype=torch.int32, device=DEV)[None]
    dout = rnd(gen_of(91), *q.shape, dtype=dtype)
    a, b, c = leaves(q, k, v)
    out = spr.block_attention(*spr.rotary(plan, pos, a, b), c, cfg, kv_len=lens, q_start=starts)
    got = torch.autograd.grad(out, (a, b, c), dout)
    qr, kr = spr.rotary(plan, pos, q, k)
    ws = spr.selected_workspace(q, k, cfg, backward=True)
    sel = spr.select_blocks(qr, spr.key_means(kr, 64, kv_len=lens), 300, cfg, ws, kv_len=lens, q_start=starts)
    rest = torch.empty_like(q) if dtype is BF else None
    o, lse = spr.selected_attn(qr, kr, v, sel, cfg, ws, kv_len=lens, q_start=starts, rest=rest)
    dq, dk, dv = spr.selected_attn_backward(dout, qr, kr, v, o, lse, sel, cfg, ws, kv_len=lens, q_start=starts, rest=rest)
    want = spr.rotary(plan, pos, dq, dk, inverse=True) + (dv,)
    assert torch.equal(out, o)
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    # one tensor alone, and a gradient that is an expanded, a strided or an odd-offset tensor
    x, = leaves(q)
    assert torch.equal(torch.autograd.grad(spr.rotary(plan, pos, x, inverse=True), x, dout)[0], spr.rotary(plan, pos, dout))
    for g in (torch.ones((), dtype=dtype, device=DEV).expand(q.shape), dout.transpose(1, 2).contiguous().transpose(1, 2),
              torch.cat([dout.flatten(), dout.flatten()[:1]])[1:].view(q.shape)):
        x, y, z = leaves(qr, kr, v)
        out, lse = spr.selected_attn(x, y, z, sel, cfg, ws, kv_len=lens, q_start=starts)
        assert not lse.requires_grad
        got = torch.autograd.grad(out, (x, y, z), g)
        want = spr.selected_attn_backward(g.contiguous().clone(), qr, kr, v, o, lse, sel, cfg, ws, kv_len=lens, q_start=starts,
                                          rest=rest)
        assert all(torch.equal(s, t) for s, t in zip(got, want))
    spr.check(ws)


def test_autograd_adds_over_repeated_inputs_and_branches():
    """Expanded keys get the sum over their repeats; two uses of a tensor add up; a frozen one gets nothing."""
    gen = gen_of(92)
    q, k, v = rnd(gen, 2, 4, 150, 64, dtype=F), rnd(gen, 1, 1, 300, 64, dtype=F), rnd(gen, 1, 1, 300, 64, dtype=F)
    cfg = spr.SelectConfig(block=64, top=3)
    a, b, c = leaves(q, k, v)
    out = spr.block_attention(a, b.expand(2, 2, 300, 64), c.expand(2, 2, 300, 64), cfg)
    got = torch.autograd.grad(out.square().sum(), (b, c))
    y, z = leaves(k.expand(2, 2, 300, 64), v.expand(2, 2, 300, 64))
    want = torch.autograd.grad(spr.block_attention(q, y, z, cfg).square().sum(), (y, z))
    for s, t in zip(got, want):  # four terms added in fp32, in another order
        t = t.double()
        close(s, t.sum((0, 1), keepdim=True), 4 * U[F] * t.abs().sum((0, 1), keepdim=True) + 1e-30, "expanded")
    x, = leaves(q)
    twice = spr.block_attention(x, b.detach().expand(2, 2, 300, 64), c.detach().expand(2, 2, 300, 64), cfg)
    g1, = torch.autograd.grad(twice.sum() + (2 * x).sum(), x, retain_graph=True)
    g2, = torch.autograd.grad(twice.sum(), x)
    assert torch.equal(g1, g2 + 2)


def test_calls_that_autograd_records_are_checked():
    q, k, v, lens, starts, cfg = problem((1, 2, 2, 40, 200, 64, 64, 2, False, 0, 0, None, BF), 93)
    plan = spr.rotary_plan(64, DEV)
    pos = torch.arange(40, dtype=torch.int32, device=DEV)[None]
    ws = spr.selected_workspace(q, k, cfg)
    sel = spr.select_blocks(q, spr.key_means(k, 64), 200, cfg, ws)
    a, = leaves(q)
    buf, lse = torch.empty_like(q), torch.empty(1, 2, 40, device=DEV)
    for call in (lambda: spr.selected_attn(a, k, v, sel, cfg, ws, out=buf), lambda: spr.selected_attn(a, k, v, sel, cfg, ws, lse=lse),
                 lambda: spr.selected_attn(a, k, v, sel, cfg, ws, rest=buf), lambda: spr.block_attention(a, k, v, cfg, out=buf),
                 lambda: spr.rotary(plan, pos, a, out=buf)):
        with pytest.raises(ValueError, match="autograd"):
            call()
        with torch.no_grad():
            call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(ValueError, match="captured"):
            spr.selected_attn(a, k, v, sel, cfg, ws)
        with torch.no_grad():
            out, _ = spr.selected_attn(a, k, v, sel, cfg, ws)
    graph.replay()
    assert torch.equal(out, spr.selected_attn(q, k, v, sel, cfg, ws)[0])
    with torch.inference_mode():
        assert torch.equal(spr.selected_attn(a, k, v, sel, cfg, ws, out=torch.empty_like(q))[0], out)
    # no second derivative
    got, = torch.autograd.grad(spr.selected_attn(a, k, v, sel, cfg, ws)[0].float().square().sum(), a, create_graph=True)
    with pytest.raises(RuntimeError):
        got.sum().backward()
    spr.check(ws)


def test_what_a_recorded_call_keeps_is_not_overwritten_unseen():
    """A selection, a length or an output written again before the backward pass: an error, not other gradients."""
    q, k, v, lens, starts, cfg = problem((1, 2, 2, 40, 200, 64, 64, 2, False, 0, 0, None, BF), 94)
    ws = spr.selected_workspace(q, k, cfg)
    means = spr.key_means(k, 64)
    plan = spr.rotary_plan(64, DEV)
    pos = torch.arange(40, dtype=torch.int32, device=DEV)[None]
    for change in (lambda t: spr.select_blocks(q, means, 200, cfg, ws, out=t["sel"]), lambda t: t["lens"].sub_(1),
                   lambda t: spr.rotary(plan, pos, q, out=t["q"])):
        t = {"sel": spr.select_blocks(q, means, 200, cfg, ws), "lens": lens.clone(), "q": q.clone()}
        c, = leaves(v)
        out, _ = spr.selected_attn(t["q"], k, c, t["sel"], cfg, ws, kv_len=t["lens"])
        change(t)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            out.sum().backward()


def test_errors_of_a_recorded_backward_pass_reach_the_callers_workspace():
    """Bad entries seen by the backward pass alone (the status of the forward call was reset)."""
    q, k, v, lens, starts, cfg = problem((1, 2, 2, 40, 400, 64, 64, 3, False, 0, 0, None, BF), 95)
    sel = torch.tensor([1, 3, 2], dtype=torch.int32, device=DEV).expand(1, 2, 40, 3).contiguous()
    ws = spr.selected_workspace(q, k, cfg)
    a, = leaves(q)
    out, _ = spr.selected_attn(a, k, v, sel, cfg, ws)
    with pytest.raises(spr.SparsePRError):
        spr.check(ws)
    spr.sparsepr.reset_workspace(ws)
    out.sum().backward()
    with pytest.raises(spr.SparsePRError) as e:
        spr.check(ws)
    assert e.value.code == spr.ERR_INVALID_ARG


def test_a_recorded_pass_on_another_stream():
    """Forward and backward on a stream that is not the default one, gradients read on the default one."""
    q, k, v, lens, starts, cfg = problem((1, 4, 2, 700, 700, 128, 64, 4, True, 0, 1, None, BF), 96)
    dout = rnd(gen_of(97), *q.shape)
    a, b, c = leaves(q, k, v)
    spr.block_attention(a, b, c, cfg).backward(dout)
    want = [t.grad.clone() for t in (a, b, c)]
    side = torch.cuda.Stream()
    a, b, c = leaves(q, k, v)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out = spr.block_attention(a, b, c, cfg)
        out.backward(dout)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(t.grad, w) for t, w in zip((a, b, c), want))
