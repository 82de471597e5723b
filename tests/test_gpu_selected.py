"""Rotary positions and selected-block attention on the GPU against their 64-bit definitions.

Tolerances, counted before any run.  With u = 2^-8 (bf16) or 2^-24 (fp32) the largest relative
error of one rounding, every element of a result is held to

  out  u |out| + u sum_j P_j |v_j| + e sum_j P_j |v_j|
       (the result's rounding, the softmax weights' rounding to the operand type, and fp32
       sums and exponentials: e = 2e-5 covers 128-term fp32 sums, 128 * 2^-24 = 8e-6, and the
       exponential of a logit of magnitude 50 off by 2^-24 relative, 3e-6)
  dv   the same with sum_i P_ij |dO_i|
  dq   u |dq| + u sum_j |dS_ij| |k_j| + e sum_j W_ij |k_j|, W_ij = P_ij tau (|dO_i|.|v_j| +
       sum |dO_i out_i|): dS is rounded to the operand type, and dP - delta may cancel
  dk   the same with |q_i|
  lse  1e-5 absolute per unit of 1 + |lse|;  rotary  u |y| + 1e-6 (|a| + |b|) f
"""
import math

import pytest
import torch

import free_block_sparse_response_b200 as spr
import selected_reference as R

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")
U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
E = 2e-5


@pytest.fixture(scope="module", autouse=True)
def _built():
    from free_block_sparse_response_b200.build import build
    build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def rnd(gen, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=gen, device=DEV).to(dtype)


def gen_of(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def close(got, want, bound, what):
    got = got.double()
    assert torch.isfinite(got).all(), f"{what}: not finite"
    over = (got - want).abs() - bound
    assert (over <= 0).all(), f"{what}: {int((over > 0).sum())} of {over.numel()} past the bound by up to " \
                              f"{float(over.max()):.3e} (values up to {float(want.abs().max()):.3e})"


# (batch, heads, key heads, queries, keys, d, block, top, causal, n_first, n_local, lens, dtype)
BF, F = torch.bfloat16, torch.float32
SHAPES = [
    (1, 2, 2, 300, 300, 128, 128, 2, False, 0, 0, None, BF),
    (1, 2, 2, 257, 257, 64, 64, 3, False, 0, 0, None, F),
    (2, 4, 2, 513, 513, 128, 128, 3, True, 1, 1, (513, 130), BF),
    (1, 6, 2, 200, 200, 64, 64, 2, True, 0, 1, None, BF),
    (2, 4, 4, 190, 190, 128, 64, 3, True, 0, 2, (190, 0), F),
    (1, 5, 1, 1, 1, 128, 128, 4, True, 0, 1, None, BF),
    (3, 8, 2, 1, 700, 128, 64, 4, True, 1, 1, (1, 700, 333), BF),
    (2, 7, 7, 1, 500, 64, 128, 2, True, 0, 1, (500, 129), F),
    (2, 16, 2, 3, 1000, 64, 128, 3, True, 0, 1, (1000, 65), BF),
    (1, 2, 1, 1100, 640, 128, 128, 5, False, 2, 0, None, BF),
    (1, 1, 1, 64, 1024, 128, 64, 16, False, 0, 0, (1000,), F),
    (1, 2, 2, 1500, 1500, 64, 128, 12, True, 0, 1, None, BF),
    (1, 3, 3, 129, 129, 128, 64, 8, False, 0, 0, (3,), BF),
]


def problem(shape, seed, token_major=False):
    bt, hq, hk, n, keys, d, block, top, causal, first, local, lens, dt = shape
    gen = gen_of(seed)

    def make(h, rows):
        x = rnd(gen, bt, rows, h, d, dtype=dt)
        return x.transpose(1, 2) if token_major else x.transpose(1, 2).contiguous()

    q, k, v = make(hq, n), make(hk, keys), make(hk, keys)
    length = torch.tensor(lens if lens else [keys] * bt, dtype=torch.int32, device=DEV)
    start = (length - n if n < keys else torch.zeros_like(length)).int()
    for i in range(bt):  # rows past a sequence's end may hold anything
        k[i, :, int(length[i]):] = math.nan
        v[i, :, int(length[i]):] = math.inf
    cfg = spr.SelectConfig(block=block, top=top, causal=causal, n_first=first, n_local=local)
    return q, k, v, length, start, cfg


@pytest.mark.parametrize("token_major", [False, True])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(str(x) for x in s[:9]))
def test_selection_and_attention_match_the_definitions(shape, token_major):
    q, k, v, lens, starts, cfg = problem(shape, 3, token_major)
    bt, hq, n, d = q.shape
    keys, dt = k.shape[2], q.dtype
    ws = spr.selected_workspace(q, k, cfg)
    mean = spr.key_means(k, cfg.block, kv_len=lens)
    assert torch.equal(mean, R.means(k, cfg.block, lens))
    sel = spr.select_blocks(q, mean, keys, cfg, ws, kv_len=lens, q_start=starts)
    spr.check(ws)
    assert torch.equal(sel, R.select(q, mean, keys, cfg.block, cfg.top, lens, starts, cfg.causal, cfg.n_first, cfg.n_local))
    out, lse = spr.selected_attn(q, k, v, sel, cfg, ws, kv_len=lens, q_start=starts)
    spr.check(ws)
    assert out.stride() == q.stride()
    ok = R.mask(sel, n, keys, cfg.block, lens, starts, cfg.causal)
    want, wlse, p = R.attention(q, k, v, ok, d ** -0.5)
    size = p @ torch.where(ok.any(2)[..., None], v.double(), 0.0).abs().repeat_interleave(hq // k.shape[1], 1)
    close(out, want, U[dt] * want.abs() + (U[dt] + E) * size + 1e-30, "out")
    live = wlse > -math.inf
    assert torch.equal(lse == -math.inf, ~live)
    close(lse[live], wlse[live], 1e-5 * (1 + wlse[live].abs()), "lse")
    assert (out[~live] == 0).all()


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(str(x) for x in s[:9]))
def test_backward_matches_the_formula(shape):
    q, k, v, lens, starts, cfg = problem(shape, 5)
    bt, hq, n, d = q.shape
    keys, dt = k.shape[2], q.dtype
    dout = rnd(gen_of(6), *q.shape, dtype=dt)
    ws = spr.selected_workspace(q, k, cfg, backward=True)
    sel = spr.select_blocks(q, spr.key_means(k, cfg.block, kv_len=lens), keys, cfg, ws, kv_len=lens, q_start=starts)
    out, lse = spr.selected_attn(q, k, v, sel, cfg, ws, kv_len=lens, q_start=starts)
    got = spr.selected_attn_backward(dout, q, k, v, out, lse, sel, cfg, ws, kv_len=lens, q_start=starts)
    spr.check(ws)
    ok = R.mask(sel, n, keys, cfg.block, lens, starts, cfg.causal)
    grads, sizes, noise = R.backward(dout, q, k, v, ok, d ** -0.5, out=out)
    for name, g, w, s, e in zip(("dq", "dk", "dv"), got, grads, sizes, noise):
        close(g, w, U[dt] * w.abs() + U[dt] * s * 1.01 + E * e + 1e-30, name)


@pytest.mark.parametrize("shape", [s for s in SHAPES if s[-1] is BF], ids=lambda s: "-".join(str(x) for x in s[:9]))
def test_backward_with_the_rest_of_out(shape):
    """out + rest holds the result past its rounding, and dq and dk lose that rounding: with delta from
    out + rest the reference's delta is that of the exact out, off by u^2 + (u + e) of sum P |v| |dout|
    (the rest's own rounding; the weights' rounding and fp32 sums of the forward pass)."""
    q, k, v, lens, starts, cfg = problem(shape, 5)
    bt, hq, n, d = q.shape
    keys = k.shape[2]
    dout = rnd(gen_of(6), *q.shape)
    ws = spr.selected_workspace(q, k, cfg, backward=True)
    sel = spr.select_blocks(q, spr.key_means(k, cfg.block, kv_len=lens), keys, cfg, ws, kv_len=lens, q_start=starts)
    plain, _ = spr.selected_attn(q, k, v, sel, cfg, ws, kv_len=lens, q_start=starts)
    rest = torch.full(q.shape, math.nan, dtype=BF, device=DEV)
    out, lse = spr.selected_attn(q, k, v, sel, cfg, ws, kv_len=lens, q_start=starts, rest=rest)
    got = spr.selected_attn_backward(dout, q, k, v, out, lse, sel, cfg, ws, kv_len=lens, q_start=starts, rest=rest)
    spr.check(ws)
    assert torch.equal(out, plain)
    ok = R.mask(sel, n, keys, cfg.block, lens, starts, cfg.causal)
    whole = out.double() + rest.double()
    # at most half a step of out, itself rounded
    assert (rest.double().abs() <= U[BF] * (1 + U[BF]) * out.double().abs() + 1e-38).all()
    want, _, p = R.attention(q, k, v, ok, d ** -0.5)
    size = p @ torch.where(ok.any(2)[..., None], v.double(), 0.0).abs().repeat_interleave(hq // k.shape[1], 1)
    close(whole, want, U[BF] ** 2 * want.abs() + (U[BF] + E) * size + 1e-30, "out + rest")
    # the rows that the backward pass forms delta from are these
    grads, sizes, noise = R.backward(dout, q, k, v, ok, d ** -0.5, out=whole)
    for name, g, w, s, e in zip(("dq", "dk", "dv"), got, grads, sizes, noise):
        close(g, w, U[BF] * w.abs() + U[BF] * s * 1.01 + E * e + 1e-30, name)


def test_the_rest_of_out_takes_its_rounding_from_dq():
    """Rows whose values share a large part: delta of the rounded out is off by up to u |dout . out|, for
    every key alike.  Here out is near 4, its rounding 0.009 rms, delta's error 0.009 sqrt(128) = 0.1, dq's
    0.1 tau |sum P k| = 0.1 * 0.088 * 2 = 0.018 an element; with the rest what is left is the weights' rounding
    in out (4.1 / 22 * 1.1e-3 = 2e-4, so 4e-4 of dq) and dS's (1e-4): a factor of 40, of which 10 are asked."""
    q, k, v, lens, starts, cfg = problem((1, 2, 2, 600, 1024, 128, 128, 4, False, 0, 0, None, BF), 23)
    v, k = (v.float() + 4).to(BF), (k.float() + 2).to(BF)
    dout = rnd(gen_of(24), *q.shape)
    ws = spr.selected_workspace(q, k, cfg, backward=True)
    sel = spr.select_blocks(q, spr.key_means(k, 128), 1024, cfg, ws)
    rest = torch.empty(q.shape, dtype=BF, device=DEV)
    out, lse = spr.selected_attn(q, k, v, sel, cfg, ws, rest=rest)
    want = R.backward(dout, q, k, v, R.mask(sel, 600, 1024, 128, lens, starts, False), 128 ** -0.5)[0][0]
    dqs = (spr.selected_attn_backward(dout, q, k, v, out, lse, sel, cfg, ws, rest=r)[0] for r in (rest, None))
    with_rest, without = (float((dq.double() - want).norm()) for dq in dqs)
    assert with_rest < without / 10


def test_the_rest_is_checked():
    q, k, v, lens, starts, cfg = problem((1, 2, 2, 40, 200, 64, 64, 2, False, 0, 0, None, BF), 25)
    ws = spr.selected_workspace(q, k, cfg)
    sel = spr.select_blocks(q, spr.key_means(k, 64), 200, cfg, ws)
    for bad in (torch.empty(1, 2, 40, 64, device=DEV), torch.empty(1, 2, 39, 64, dtype=BF, device=DEV),
                torch.empty(1, 40, 2, 64, dtype=BF, device=DEV).transpose(1, 2)):
        with pytest.raises(ValueError, match="rest"):
            spr.selected_attn(q, k, v, sel, cfg, ws, rest=bad)
    with pytest.raises(spr.SparsePRError, match="out_rest"):
        spr.selected_attn(q, k, v, sel, cfg, ws, rest=torch.empty(2 * 40 * 64 + 1, dtype=BF, device=DEV)[1:].view(1, 2, 40, 64))
    with pytest.raises(ValueError, match="bf16"):
        spr.selected_attn(q.float(), k.float(), v.float(), sel, cfg, ws, rest=torch.empty(1, 2, 40, 64, device=DEV))


def test_gradients_match_differences():
    """Central differences of the 64-bit loss along random directions, selection fixed."""
    q, k, v, lens, starts, cfg = problem((1, 4, 2, 200, 200, 64, 64, 2, True, 0, 1, None, F), 8)
    gen = gen_of(9)
    dout = rnd(gen, *q.shape, dtype=F)
    ws = spr.selected_workspace(q, k, cfg, backward=True)
    sel = spr.select_blocks(q, spr.key_means(k, cfg.block), 200, cfg, ws, q_start=starts)
    out, lse = spr.selected_attn(q, k, v, sel, cfg, ws, q_start=starts)
    got = spr.selected_attn_backward(dout, q, k, v, out, lse, sel, cfg, ws, q_start=starts)
    ok = R.mask(sel, 200, 200, 64, lens, starts, True)

    def loss(*x):
        return float((R.attention(*x, ok, 64 ** -0.5)[0] * dout.double()).sum())

    for i in range(3):
        u = torch.randn(got[i].shape, generator=gen, device=DEV, dtype=torch.float64)
        hi, lo = ([t.double() + (s * u if j == i else 0) for j, t in enumerate((q, k, v))] for s in (1e-5, -1e-5))
        diff = (loss(*hi) - loss(*lo)) / 2e-5
        want = float((got[i].double() * u).sum())
        # the difference's own error: third derivative * h^2 and 2^-53 |loss| / h, both below 1e-6 of the scale
        assert abs(diff - want) <= 1e-4 * (abs(want) + float(got[i].double().norm())), (i, diff, want)


def test_selection_breaks_ties_to_the_lower_block():
    """Equal blocks score equally: keys that repeat block after block, and zero queries."""
    q = rnd(gen_of(1), 1, 2, 70, 64)
    q[:, :, ::2] = 0
    k = rnd(gen_of(2), 1, 2, 64, 64).repeat(1, 1, 7, 1)
    cfg = spr.SelectConfig(block=64, top=3)
    ws = spr.selected_workspace(q, k, cfg)
    sel = spr.select_blocks(q, spr.key_means(k, 64), k.shape[2], cfg, ws)
    assert torch.equal(sel, torch.tensor([0, 1, 2], dtype=torch.int32, device=DEV).expand(1, 2, 70, 3))


def test_near_ties_are_decided_in_64_bits():
    """Blocks whose means differ in the last bits of 32-bit sums."""
    n, d, nb, top = 700, 128, 96, 7
    gen = gen_of(4)
    base = rnd(gen, 1, 1, 1, d, dtype=F)
    mean = base + 1e-6 * rnd(gen, 1, 1, nb, d, dtype=F)
    q = rnd(gen, 1, 1, n, d)
    cfg = spr.SelectConfig(block=64, top=top)
    ws = spr.selected_workspace(q, rnd(gen, 1, 1, nb * 64, d), cfg)
    sel = spr.select_blocks(q, mean.contiguous(), nb * 64, cfg, ws)
    spr.check(ws)
    lens = torch.tensor([nb * 64], device=DEV)
    assert torch.equal(sel, R.select(q, mean, nb * 64, 64, top, lens, torch.zeros_like(lens), False, 0, 0))


@pytest.mark.parametrize("qs,ms,group", [(1e-23, 1.0, 1), (1.0, 1e-23, 1), (1e-30, 1e-18, 2), (1e-22, 1e22, 4), (1e30, 1e-30, 2)])
def test_near_ties_of_very_small_and_large_values(qs, ms, group):
    """Sizes whose squares leave the range of 32 bits."""
    n, d, nb, top = 700, 128, 96, 7
    gen = gen_of(61)
    mean = (rnd(gen, 1, 1, 1, d, dtype=F) + 1e-6 * rnd(gen, 1, 1, nb, d, dtype=F)) * ms
    q = (rnd(gen, 1, group, n, d).float() * qs).to(BF)
    cfg = spr.SelectConfig(block=64, top=top)
    ws = spr.selected_workspace(q, torch.zeros(1, 1, nb * 64, d, dtype=BF, device=DEV), cfg)
    sel = spr.select_blocks(q, mean.contiguous(), nb * 64, cfg, ws)
    spr.check(ws)
    lens = torch.tensor([nb * 64], device=DEV)
    assert torch.equal(sel, R.select(q, mean, nb * 64, 64, top, lens, torch.zeros_like(lens), False, 0, 0))


def test_nan_scores_rank_lowest_and_are_reported():
    q = torch.ones(1, 1, 4, 64, device=DEV, dtype=BF)
    mean = torch.arange(6, device=DEV, dtype=F).view(1, 1, 6, 1).expand(1, 1, 6, 64).contiguous()
    mean[0, 0, 5, 3] = math.nan
    mean[0, 0, 1, 3] = math.inf
    mean[0, 0, 2, 3] = -math.inf
    cfg = spr.SelectConfig(block=64, top=5)
    ws = spr.selected_workspace(q, torch.zeros(1, 1, 384, 64, device=DEV, dtype=BF), cfg)
    sel = spr.select_blocks(q, mean, 384, cfg, ws)
    assert sel[0, 0].tolist() == [[0, 1, 2, 3, 4]] * 4
    with pytest.raises(spr.SparsePRError) as e:
        spr.check(ws)
    assert e.value.code == spr.ERR_NONFINITE


def test_bad_selection_entries_are_skipped_and_reported():
    """Repeated, descending and out-of-range blocks: the row's valid entries are attended to."""
    q, k, v, lens, starts, cfg = problem((1, 2, 2, 130, 400, 64, 64, 4, False, 0, 0, None, BF), 11)
    good = torch.tensor([1, 3, -1, -1], dtype=torch.int32, device=DEV).expand(1, 2, 130, 4).contiguous()
    bad = good.clone()
    bad[:, :, 1::2] = torch.tensor([1, 1, 3, 2], dtype=torch.int32, device=DEV)
    bad[:, :, 2::4] = torch.tensor([1, 3, 7, 1 << 30], dtype=torch.int32, device=DEV)
    ws = spr.selected_workspace(q, k, cfg)
    want = spr.selected_attn(q, k, v, good, cfg, ws)
    spr.check(ws)
    got = spr.selected_attn(q, k, v, bad, cfg, ws)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    with pytest.raises(spr.SparsePRError) as e:
        spr.check(ws)
    assert e.value.code == spr.ERR_INVALID_ARG
    spr.sparsepr.reset_workspace(ws)
    spr.check(ws)


def test_entries_past_a_negative_one_are_not_read():
    q, k, v, lens, starts, cfg = problem((1, 1, 1, 40, 256, 128, 64, 3, False, 0, 0, None, BF), 12)
    a = torch.tensor([2, -1, -1], dtype=torch.int32, device=DEV).expand(1, 1, 40, 3).contiguous()
    b = torch.tensor([2, -5, 3], dtype=torch.int32, device=DEV).expand(1, 1, 40, 3).contiguous()
    ws = spr.selected_workspace(q, k, cfg)
    assert torch.equal(spr.selected_attn(q, k, v, a, cfg, ws)[0], spr.selected_attn(q, k, v, b, cfg, ws)[0])
    spr.check(ws)


def test_results_repeat_bit_for_bit_and_leave_the_inputs():
    q, k, v, lens, starts, cfg = problem((2, 8, 2, 900, 900, 128, 64, 5, True, 1, 1, (900, 300), BF), 13)
    keep = [t.clone() for t in (q, k, v)]
    dout = rnd(gen_of(14), *q.shape)
    runs = []
    for _ in range(2):
        ws = spr.selected_workspace(q, k, cfg, backward=True)
        ws[256:] = 255  # nothing in a new workspace is read
        sel = spr.select_blocks(q, spr.key_means(k, cfg.block, kv_len=lens), 900, cfg, ws, kv_len=lens, q_start=starts)
        out, lse = spr.selected_attn(q, k, v, sel, cfg, ws, kv_len=lens, q_start=starts)
        runs.append((sel, out, lse) + spr.selected_attn_backward(dout, q, k, v, out, lse, sel, cfg, ws, kv_len=lens,
                                                                 q_start=starts))
    for a, b in zip(*runs):
        assert torch.equal(a, b)
    for a, b in zip(keep, (q, k, v)):
        assert torch.equal(torch.nan_to_num(a.float()), torch.nan_to_num(b.float()))


def test_a_captured_step_replays_on_new_inputs_and_another_stream():
    """Rotation, selection, attention and gradients captured once, replayed on other values."""
    q, k, v, lens, starts, cfg = problem((1, 4, 2, 300, 300, 128, 64, 3, True, 0, 1, None, BF), 15)
    plan = spr.rotary_plan(128, DEV)
    pos = torch.arange(300, dtype=torch.int32, device=DEV)[None, :, None].contiguous()
    dout = rnd(gen_of(16), *q.shape)
    ws = spr.selected_workspace(q, k, cfg, backward=True)

    def step():
        qr, kr = spr.rotary(plan, pos, q, k)
        sel = spr.select_blocks(qr, spr.key_means(kr, 64), 300, cfg, ws, q_start=starts)
        out, lse = spr.selected_attn(qr, kr, v, sel, cfg, ws, q_start=starts)
        dq, dk, dv = spr.selected_attn_backward(dout, qr, kr, v, out, lse, sel, cfg, ws, q_start=starts)
        dq, dk = spr.rotary(plan, pos, dq, dk, inverse=True)
        return out, lse, dq, dk, dv

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            res = step()
    torch.cuda.current_stream().wait_stream(side)
    for seed in (17, 18):
        fresh = problem((1, 4, 2, 300, 300, 128, 64, 3, True, 0, 1, None, BF), seed)
        for a, b in zip((q, k, v), fresh):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in res]
        for a, b in zip(got, step()):
            assert torch.equal(a, b)
    spr.check(ws)


def test_decode_over_a_growing_cache_matches_the_prompt():
    """Token after token over a cache with kept means equals the causal prompt's last rows."""
    bt, hq, hk, d, block, keys = 2, 8, 2, 128, 64, 330
    gen = gen_of(20)
    q, k, v = rnd(gen, bt, hq, keys, d), rnd(gen, bt, hk, keys, d), rnd(gen, bt, hk, keys, d)
    cfg = spr.SelectConfig(block=block, top=3, causal=True, n_first=1, n_local=1)
    zero = torch.zeros(bt, dtype=torch.int32, device=DEV)
    ws = spr.selected_workspace(q, k, cfg)
    full = spr.key_means(k, block)
    cache_k, cache_v = torch.full((2, bt, hk, 400, d), math.nan, dtype=BF, device=DEV)
    m0 = 250
    cache_k[:, :, :m0], cache_v[:, :, :m0] = k[:, :, :m0], v[:, :, :m0]
    lens = torch.full((bt,), m0, dtype=torch.int32, device=DEV)
    means = spr.key_means(cache_k, block, kv_len=lens)
    one = spr.selected_workspace(q[:, :, :1], cache_k, cfg)
    for t in range(m0, keys):
        # the selection of token t sees the means of whole later blocks in a prompt: take them as of now
        cache_k[:, :, t], cache_v[:, :, t] = k[:, :, t], v[:, :, t]
        lens = torch.full((bt,), t + 1, dtype=torch.int32, device=DEV)
        spr.key_means(cache_k, block, kv_len=lens, kv_start=lens - 1, max_new=1, out=means)
        g = t // block
        assert torch.equal(means[:, :, :g], full[:, :, :g])
        qt = q[:, :, t:t + 1]
        sel = spr.select_blocks(qt, means, 400, cfg, one, kv_len=lens, q_start=lens - 1)
        out, lse = spr.selected_attn(qt, cache_k, cache_v, sel, cfg, one, kv_len=lens, q_start=lens - 1)
        ok = R.mask(sel, 1, 400, block, lens, lens - 1, True)
        want, wlse, p = R.attention(qt, cache_k, cache_v, ok, d ** -0.5)
        size = p[..., :keys] @ v.double().abs().repeat_interleave(hq // hk, 1)
        close(out, want, U[BF] * want.abs() + (U[BF] + E) * size, f"token {t}")
    spr.check(one)
    prompt = spr.block_attention(q, k, v, cfg, ws=ws, q_start=zero)
    spr.check(ws)
    # the last token sees only whole blocks and its own, forced one: the prompt's selection is the same
    close(out, prompt[:, :, -1:].double(), 2 * U[BF] * want.abs() + 2 * (U[BF] + E) * size, "last token")


@pytest.mark.parametrize("max_new", [150, 10 ** 6, 2 ** 31 - 1])
def test_means_of_appended_keys_with_any_bound_on_them(max_new):
    """max_new is an upper bound: one far past the cache renews the same blocks and no others."""
    k = rnd(gen_of(22), 2, 3, 400, 64)
    lens = torch.tensor([400, 210], dtype=torch.int32, device=DEV)
    start = torch.tensor([250, 209], dtype=torch.int32, device=DEV)
    means = torch.full((2, 3, 7, 64), 5.0, device=DEV)
    spr.key_means(k, 64, kv_len=lens, kv_start=start, max_new=max_new, out=means)
    want = torch.full_like(means, 5.0)
    full = spr.key_means(k, 64, kv_len=lens)
    want[0, :, 3:], want[1, :, 3] = full[0, :, 3:], full[1, :, 3]
    assert torch.equal(means, want)


def test_long_offsets_past_32_bits():
    """A cache view whose last rows lie past 2^32 elements of its start (strides of a wider buffer)."""
    rows, d = 1024, 128
    step = (1 << 32) // rows + 4096
    wide = torch.empty(step * rows, dtype=BF, device=DEV)
    gen = gen_of(21)
    k, v = (torch.as_strided(wide, (1, 1, rows, d), (0, 0, step, 1), off) for off in (0, 256))
    k.copy_(rnd(gen, 1, 1, rows, d))
    v.copy_(rnd(gen, 1, 1, rows, d))
    q = rnd(gen, 1, 1, 200, d)
    cfg = spr.SelectConfig(block=128, top=3)
    got = spr.block_attention(q, k, v, cfg)
    assert torch.equal(got, spr.block_attention(q, k.contiguous(), v.contiguous(), cfg))


# ------------------------------------------------------------------------------- rotary

ROT = [
    # d, rot, first, layout, sections, dtype, far, token_major
    (128, 128, 0, spr.ROTARY_HALF, (64,), BF, 131071, False),
    (128, 128, 0, spr.ROTARY_INTERLEAVED, (24, 20, 20), BF, 0, True),
    (128, 64, 64, spr.ROTARY_HALF, (32,), BF, 0, True),
    (64, 48, 0, spr.ROTARY_INTERLEAVED, (12, 12), F, 1 << 30, False),
    (64, 48, 0, spr.ROTARY_HALF, (24,), F, 5000, True),
    (64, 20, 2, spr.ROTARY_HALF, (10,), BF, 0, False),
    (128, 2, 5, spr.ROTARY_INTERLEAVED, (1,), F, 7, False),
]


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("bt,hq,hk,n", [(1, 3, 1, 1), (2, 9, 2, 77), (1, 24, 0, 1000)])
@pytest.mark.parametrize("case", ROT, ids=str)
def test_rotary_matches_the_definition(case, bt, hq, hk, n, inverse):
    d, rot, first, layout, sections, dt, far, token_major = case
    gen = gen_of(30)
    xs = []
    for h in (hq, hk):
        x = rnd(gen, bt, n, h, d, dtype=dt) if token_major else rnd(gen, bt, h, n, d, dtype=dt)
        xs.append(x.transpose(1, 2) if token_major else x)
    plan = spr.rotary_plan(d, DEV, rot_dim=rot, first=first, layout=layout, sections=sections, base=5e5,
                           scaling="ramp", scaling_factor=4.0, trained_length=4096)
    pos = (torch.randint(0, 999, (bt, n, len(sections)), generator=gen, device=DEV) + far).int()
    got = spr.rotary(plan, pos, xs[0], xs[1] if hk else None, inverse=inverse)
    for x, y in zip(xs, got if hk else (got,)):
        want = R.rotary(x, pos, plan.freqs, sections, rot, first, layout == spr.ROTARY_HALF, plan.factor, inverse)
        # 1e-6: the angle's rounding to 32 bits (2^-24 pi), sincos and two products
        size = torch.linalg.vector_norm(x.double(), ord=math.inf, dim=-1, keepdim=True)
        close(y, want, U[dt] * want.abs() + 2e-6 * plan.factor * size, "rotary")
    z = xs[0].clone()
    assert torch.equal(spr.rotary(plan, pos, z, inverse=inverse, out=z), got[0] if hk else got)


def test_rotary_writes_only_its_rows_of_a_cache():
    gen = gen_of(31)
    cache = rnd(gen, 2, 3, 50, 64)
    keep = cache.clone()
    k = rnd(gen, 2, 3, 4, 64)
    plan = spr.rotary_plan(64, DEV)
    pos = torch.arange(20, 24, dtype=torch.int32, device=DEV)[None]
    spr.rotary(plan, pos, k, out=cache[:, :, 20:24])
    keep[:, :, 20:24] = spr.rotary(plan, pos, k)
    assert torch.equal(cache, keep)


def test_rotation_back_restores_and_is_the_gradient():
    gen = gen_of(32)
    x, g = rnd(gen, 1, 2, 33, 128, dtype=F), rnd(gen, 1, 2, 33, 128, dtype=F)
    plan = spr.rotary_plan(128, DEV, layout=spr.ROTARY_INTERLEAVED)
    pos = torch.arange(33, dtype=torch.int32, device=DEV)[None]
    y = spr.rotary(plan, pos, x)
    assert float((spr.rotary(plan, pos, y, inverse=True) - x).abs().max()) <= 8e-6  # two rotations of |x| <= 5
    # <g, R x> = <R^T g, x>: 8448 products of fp32-rounded terms
    a, b = (y.double() * g.double()).sum(), (spr.rotary(plan, pos, g, inverse=True).double() * x.double()).sum()
    assert abs(float(a - b)) <= 1e-6 * float((y.double().abs() * g.double().abs()).sum())


def test_sparsepr_attention_with_rotary_positions():
    """The SparsePR call rotates q and k first where it is given a plan and positions."""
    from synthetic import CONFIGS, make_inputs
    w = CONFIGS["small"].with_(grid=(4, 16, 16), heads=2)
    q, k, v = (t.to(DEV) for t in make_inputs(w, seed=0))
    cfg = spr.SparsePRConfig(block=w.block, n_sampled=w.n_sampled, n_probe=w.n_probe, kmeans_iters=w.kmeans_iters,
                             rank=w.rank, density=w.density, ridge_lambda=w.ridge_lambda)
    grid = torch.stack(torch.meshgrid(*(torch.arange(s, device=DEV) for s in w.grid), indexing="ij"), -1)
    pos = grid.reshape(1, -1, 3).int().contiguous()
    plan = spr.rotary_plan(128, DEV, layout=spr.ROTARY_INTERLEAVED, sections=(24, 20, 20))
    keep = q.clone()
    got = spr.attention(q, k, v, cfg, rotary=(plan, pos))
    qr, kr = spr.rotary(plan, pos, q, k)
    assert torch.equal(got, spr.attention(qr, kr, v, cfg))
    assert torch.equal(got, spr.attention_call(q, k, v, cfg, rotary=(plan, pos)))
    assert torch.equal(q, keep)


# ------------------------------------------------------------------- sizes where paths change

WIDE = [
    # rows of more than 32 slots, groups past one 16-row step, every block selected
    (1, 2, 1, 300, 4096, 64, 64, 40, False, 0, 0, None, BF),
    (2, 24, 1, 1, 900, 128, 64, 9, True, 1, 1, (900, 77), BF),
    (1, 40, 2, 2, 2600, 64, 64, 41, True, 2, 3, None, BF),
    (1, 3, 1, 40, 500, 128, 128, 100, False, 0, 0, (450,), F),
    (1, 2, 2, 1, 260, 128, 64, 70, True, 0, 1, None, F),
    (4, 2, 1, 140, 140, 64, 128, 1, True, 0, 1, (1, 0, 140, 129), BF),
]


@pytest.mark.parametrize("shape", WIDE, ids=lambda s: "-".join(str(x) for x in s[:9]))
def test_wide_rows_and_groups(shape):
    test_selection_and_attention_match_the_definitions(shape, False)
    test_backward_matches_the_formula(shape)


@pytest.mark.parametrize("nb,d,n", [(130, 128, 70), (130, 128, 333), (300, 64, 300), (600, 128, 297), (700, 64, 299), (1500, 128, 301),
                                    (2048, 64, 300), (2048, 128, 3)])
def test_selection_over_many_blocks(nb, d, n):
    """The tile heights and key registers of the selection, causal and forced blocks among them."""
    gen = gen_of(nb + d)
    bt, hq, hk, top = 1, 4, 2, 11  # (up to 592 rows go to the row kernel: both kernels below)
    q, mean = rnd(gen, bt, hq, n, d), rnd(gen, bt, hk, nb, d, dtype=F)
    mean[:, :, 5] = mean[:, :, 3]
    keys = nb * 64 - 13
    lens = torch.tensor([keys - 200], dtype=torch.int32, device=DEV)
    for causal, first, local in ((False, 1, 0), (True, 2, 2)):
        cfg = spr.SelectConfig(block=64, top=top, causal=causal, n_first=first, n_local=local)
        start = torch.tensor([keys // 2 if causal else 0], dtype=torch.int32, device=DEV)
        k = torch.zeros(1, 1, 1, d, dtype=BF, device=DEV).expand(bt, hk, keys, d)
        ws = spr.selected_workspace(q, k, cfg)
        sel = spr.select_blocks(q, mean, keys, cfg, ws, kv_len=lens, q_start=start)
        spr.check(ws)
        assert torch.equal(sel, R.select(q, mean, keys, 64, top, lens, start, causal, first, local))


def test_rows_that_leave_many_blocks_open_are_decided_exactly():
    """Equal scores far past 32 blocks (zero queries, equal means) among ordinary rows."""
    gen = gen_of(41)
    n, nb, d, top = 700, 150, 64, 20
    q, mean = rnd(gen, 1, 2, n, d), rnd(gen, 1, 1, nb, d, dtype=F)
    q[:, :, 7::9] = 0
    mean[:, :, 40:110] = mean[:, :, 40:41]
    cfg = spr.SelectConfig(block=64, top=top)
    ws = spr.selected_workspace(q, torch.zeros(1, 1, nb * 64, d, dtype=BF, device=DEV), cfg)
    lens = torch.tensor([nb * 64], device=DEV)
    for _ in range(2):  # the list of left-over rows starts empty in every call
        sel = spr.select_blocks(q, mean, nb * 64, cfg, ws)
        assert torch.equal(sel, R.select(q, mean, nb * 64, 64, top, lens, torch.zeros_like(lens), False, 0, 0))
    spr.check(ws)


@pytest.mark.parametrize("size", [1e-30, 1e-4, 3e4, 1e30])
def test_values_of_any_size(size):
    """Parts travel in 16 bits: values far outside that range, and blocks of very different sizes."""
    q, k, v, lens, starts, cfg = problem((1, 2, 2, 200, 640, 128, 64, 4, False, 0, 0, None, BF), 42)
    v = (v.float() * size).to(BF)
    v[:, :, 64:128] = (v[:, :, 64:128].float() * 1e-5).to(BF)
    ws = spr.selected_workspace(q, k, cfg)
    sel = spr.select_blocks(q, spr.key_means(k, 64), 640, cfg, ws)
    out, _ = spr.selected_attn(q, k, v, sel, cfg, ws)
    ok = R.mask(sel, 200, 640, 64, lens, starts, False)
    want, _, p = R.attention(q, k, v, ok, 128 ** -0.5)
    close(out, want, U[BF] * want.abs() + (U[BF] + E) * (p @ v.double().abs()) + 1e-38, "out")


def test_an_infinite_value_reaches_its_queries_and_columns_only():
    q, k, v, lens, starts, cfg = problem((1, 1, 1, 130, 256, 128, 64, 2, False, 0, 0, None, BF), 43)
    v[0, 0, 70, 5] = math.inf   # block 1
    sel = torch.tensor([0, 3], dtype=torch.int32, device=DEV).expand(1, 1, 130, 2).contiguous()
    sel[:, :, ::3] = torch.tensor([1, 2], dtype=torch.int32, device=DEV)
    ws = spr.selected_workspace(q, k, cfg)
    out, _ = spr.selected_attn(q, k, v, sel, cfg, ws)
    bad = ~torch.isfinite(out[0, 0])
    want = torch.zeros_like(bad)
    want[::3, 5] = True
    assert torch.equal(bad, want)
    clean = v.clone()
    clean[0, 0, 70, 5] = 0
    ref, _ = spr.selected_attn(q, k, clean, sel, cfg, ws)
    assert torch.equal(out[0, 0][~bad], ref[0, 0][~bad])


def test_repeated_heads_and_batches_by_stride_zero():
    """K and V expanded over heads and batch (one cache read by all)."""
    gen = gen_of(44)
    q = rnd(gen, 2, 4, 150, 64)
    k, v = (rnd(gen, 1, 1, 300, 64).expand(2, 2, 300, 64) for _ in range(2))
    cfg = spr.SelectConfig(block=64, top=3)
    a = spr.block_attention(q, k, v, cfg)
    assert torch.equal(a, spr.block_attention(q, k.contiguous(), v.contiguous(), cfg))
    one = spr.block_attention(q[:, :, :1], k, v, cfg)
    assert torch.equal(one, spr.block_attention(q[:, :, :1], k.contiguous(), v.contiguous(), cfg))


def test_gradients_of_repeated_inputs():
    """Queries, keys and output gradients that repeat in memory: what their copies give."""
    gen = gen_of(48)
    q = rnd(gen, 1, 4, 1, 64).expand(2, 4, 150, 64)
    k, v = (rnd(gen, 1, 1, 300, 64).expand(2, 2, 300, 64) for _ in range(2))
    dout = rnd(gen, 2, 1, 1, 64).expand(2, 4, 150, 64)
    cfg = spr.SelectConfig(block=64, top=3)
    res = []
    for ins in ((q, k, v, dout), [t.contiguous() for t in (q, k, v, dout)]):
        a, b, c, g = ins
        ws = spr.selected_workspace(a, b, cfg, backward=True)
        sel = spr.select_blocks(a, spr.key_means(b, 64), 300, cfg, ws)
        out, lse = spr.selected_attn(a, b, c, sel, cfg, ws)
        res.append((sel, out, lse) + spr.selected_attn_backward(g, a, b, c, out, lse, sel, cfg, ws))
        spr.check(ws)
    for x, y in zip(*res):
        assert torch.equal(x, y)


def test_given_outputs_are_written_whole_and_nothing_beside_them():
    """out, lse, rest and the gradients into parts of wider buffers, selection and means in place."""
    q, k, v, lens, starts, cfg = problem((2, 4, 2, 140, 300, 64, 64, 3, True, 0, 1, (300, 200), BF), 49)
    dout = rnd(gen_of(50), *q.shape)
    ws = spr.selected_workspace(q, k, cfg, backward=True)
    means = spr.key_means(k, 64, kv_len=lens)
    sel = spr.select_blocks(q, means, 300, cfg, ws, kv_len=lens, q_start=starts)
    out, lse = spr.selected_attn(q, k, v, sel, cfg, ws, kv_len=lens, q_start=starts)
    want = (out,) + spr.selected_attn_backward(dout, q, k, v, out, lse, sel, cfg, ws, kv_len=lens, q_start=starts)
    sel2, means2 = torch.full_like(sel, 77), torch.full_like(means, 7.0)
    spr.key_means(k, 64, kv_len=lens, out=means2)
    spr.select_blocks(q, means2, 300, cfg, ws, kv_len=lens, q_start=starts, out=sel2)
    assert torch.equal(means2, means) and torch.equal(sel2, sel)
    wide = [torch.full((t.shape[0], t.shape[2] + 2, t.shape[1], 80), 3.0, dtype=BF, device=DEV) for t in want]
    parts = [w[:, 1:-1, :, 8:72].transpose(1, 2) for w in wide]
    lse2 = torch.full_like(lse, 7.0)
    spr.selected_attn(q, k, v, sel, cfg, ws, kv_len=lens, q_start=starts, out=parts[0], lse=lse2)
    spr.selected_attn_backward(dout, q, k, v, parts[0], lse2, sel, cfg, ws, kv_len=lens, q_start=starts, dq=parts[1],
                               dk=parts[2], dv=parts[3])
    spr.check(ws)
    assert torch.equal(lse2, lse)
    for t, p, w in zip(want, parts, wide):
        assert torch.equal(t, p)
        p.fill_(3.0)
        assert (w == 3.0).all()


def test_token_slices_of_a_large_call():
    """A head whose partial rows pass the workspace's chunk is worked off slice by slice: the same as
    calls on parts of the tokens."""
    gen = gen_of(60)
    n, keys, grp, top, d = 33000, 4096, 16, 16, 64
    q, k, v = rnd(gen, 1, grp, n, d), rnd(gen, 1, 1, keys, d), rnd(gen, 1, 1, keys, d)
    cfg = spr.SelectConfig(block=64, top=top)
    ws = spr.selected_workspace(q, k, cfg)
    sel = spr.select_blocks(q, spr.key_means(k, 64), keys, cfg, ws)
    out, lse = spr.selected_attn(q, k, v, sel, cfg, ws)
    spr.check(ws)
    for a, b in ((0, 1000), (1000, 20000), (20000, n)):
        o, l = spr.selected_attn(q[:, :, a:b], k, v, sel[:, :, a:b].contiguous(), cfg, ws)
        assert torch.equal(o, out[:, :, a:b]) and torch.equal(l, lse[:, :, a:b])


def test_two_calls_at_once_on_two_streams():
    """Overlapping calls with workspaces of their own give what they give alone."""
    cases = [problem((1, 8, 2, 3000, 3000, 128, 64, 8, True, 1, 1, None, BF), s) for s in (45, 46)]
    dout = [rnd(gen_of(47 + i), *c[0].shape) for i, c in enumerate(cases)]

    def step(i, ws):
        q, k, v, lens, starts, cfg = cases[i]
        sel = spr.select_blocks(q, spr.key_means(k, 64), 3000, cfg, ws, q_start=starts)
        out, lse = spr.selected_attn(q, k, v, sel, cfg, ws, q_start=starts)
        return (sel, out, lse) + spr.selected_attn_backward(dout[i], q, k, v, out, lse, sel, cfg, ws, q_start=starts)

    wss = [spr.selected_workspace(c[0], c[1], c[5], backward=True) for c in cases]
    alone = [[t.clone() for t in step(i, wss[i])] for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(3):
        got = []
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got.append(step(i, wss[i]))
        torch.cuda.synchronize()
    for i in range(2):
        spr.check(wss[i])
        for a, b in zip(alone[i], got[i]):
            assert torch.equal(a, b)


def test_refusals_on_the_gpu():
    q = rnd(gen_of(50), 1, 2, 40, 64)
    k = rnd(gen_of(51), 1, 2, 200, 64)
    cfg = spr.SelectConfig(block=64, top=2)
    ws = spr.selected_workspace(q, k, cfg)
    mean = spr.key_means(k, 64)
    sel = spr.select_blocks(q, mean, 200, cfg, ws)
    with pytest.raises(ValueError):
        spr.selected_attn(q, k, k[:, :, :100], sel, cfg, ws)
    with pytest.raises(ValueError):
        spr.selected_attn(q, k, k, sel.long(), cfg, ws)
    with pytest.raises(ValueError):
        spr.selected_attn(q, k, k.float(), sel, cfg, ws)
    with pytest.raises(ValueError):
        spr.selected_attn(q, k, k, sel, cfg, ws[:256])
    with pytest.raises(ValueError):
        spr.selected_attn(q, k, k, sel, cfg, ws, out=q[:, :, :1].expand(1, 2, 40, 64))
    with pytest.raises(ValueError):
        spr.select_blocks(q, mean, 400, cfg, ws)
    with pytest.raises(ValueError):
        spr.selected_attn(q, k, k, sel, cfg, ws, kv_len=torch.tensor([200], device=DEV))
    with pytest.raises(ValueError):
        spr.key_means(k, 64, kv_start=torch.zeros(1, dtype=torch.int32, device=DEV))
    with pytest.raises(spr.SparsePRError):
        spr.key_means(k, 32)
    with pytest.raises(spr.SparsePRError):
        spr.selected_workspace(q, k, spr.SelectConfig(block=64, top=0))
    with pytest.raises(spr.SparsePRError):
        wide = rnd(gen_of(52), 1, 2, 40, 65)
        spr.key_means(wide[..., 1:], 64)
    plan = spr.rotary_plan(64, DEV)
    with pytest.raises(ValueError):
        spr.rotary(plan, torch.zeros(1, 40, 1, device=DEV), q)
    with pytest.raises(ValueError):
        spr.rotary(plan, torch.zeros(1, 39, dtype=torch.int32, device=DEV), q)
    with pytest.raises(ValueError):
        spr.rotary(spr.rotary_plan(128, DEV), torch.zeros(1, 40, dtype=torch.int32, device=DEV), q)
    spr.check(ws)
