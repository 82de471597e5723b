"""Rotary and selected-block attention without a GPU: argument checks of the C entry points
(nothing is launched; the pointers are never dereferenced), the Python wrappers' refusals and
the host arithmetic of the frequency ladders."""
import ctypes
import math

import pytest
import torch

import free_block_sparse_response_b200 as spr
from free_block_sparse_response_b200 import selected as S


@pytest.fixture(scope="module")
def L():
    from free_block_sparse_response_b200.build import build
    build()
    return spr.lib()


def view(data=4096, b=0, h=0, n=128):
    return ctypes.byref(S._CView(data, b, h, n))


def problem(**kw):
    base = dict(dtype=spr.BF16, Bt=1, Hq=4, Hkv=2, Nq=100, Nk=300, d=128, block=64, top=4, causal=0, n_first=0, n_local=0,
                scale=0.0, kv_len=None, q_start=None)
    base.update(kw)
    return ctypes.byref(S._CSelected(**base))


FAKE = ctypes.c_void_p(4096)

BAD_PROBLEMS = [
    (dict(dtype=7), spr.ERR_INVALID_ARG, b"dtype"),
    (dict(Hq=5), spr.ERR_INVALID_ARG, b"multiple"),
    (dict(Nq=0), spr.ERR_INVALID_ARG, b">= 1"),
    (dict(Nk=0), spr.ERR_INVALID_ARG, b">= 1"),
    (dict(d=96), spr.ERR_UNSUPPORTED, b"head dim"),
    (dict(block=32), spr.ERR_UNSUPPORTED, b"block"),
    (dict(top=0), spr.ERR_INVALID_ARG, b"top"),
    (dict(top=1025), spr.ERR_UNSUPPORTED, b"top"),
    (dict(causal=2), spr.ERR_INVALID_ARG, b"causal"),
    (dict(n_first=-1), spr.ERR_INVALID_ARG, b"n_first"),
    (dict(n_first=5), spr.ERR_INVALID_ARG, b"exceed"),
    (dict(causal=1, n_first=2, n_local=3), spr.ERR_INVALID_ARG, b"exceed"),
    (dict(n_local=1), spr.ERR_INVALID_ARG, b"causal"),
    (dict(scale=math.nan), spr.ERR_INVALID_ARG, b"scale"),
    (dict(Nk=64 * 2048 + 1), spr.ERR_UNSUPPORTED, b"2048"),
    (dict(Bt=1 << 15, Hq=4, Nq=1 << 14), spr.ERR_UNSUPPORTED, b"2^30"),
    (dict(Bt=1 << 15, Hkv=4), spr.ERR_UNSUPPORTED, b"65535"),
    (dict(Nq=1 << 24, top=64), spr.ERR_UNSUPPORTED, b"2^30"),
]


@pytest.mark.parametrize("kw,code,word", BAD_PROBLEMS, ids=lambda x: str(x))
def test_bad_problems_are_refused_by_every_call(L, kw, code, word):
    p = problem(**kw)
    assert L.sparsepr_selected_workspace_size(p, 1) == 0
    assert word in L.sparsepr_last_error()
    v = view()
    assert L.sparsepr_key_means(p, v, None, 0, FAKE, None) == code
    assert L.sparsepr_select_blocks(p, v, FAKE, FAKE, FAKE, None) == code
    assert L.sparsepr_selected_attn(p, v, v, v, FAKE, v, FAKE, FAKE, None) == code
    assert L.sparsepr_selected_attn_backward(p, v, v, v, v, v, FAKE, FAKE, v, v, v, FAKE, None) == code
    assert word in L.sparsepr_last_error()


def test_null_and_misaligned_tensors_are_refused(L):
    p, ok = problem(), view()
    for bad in (view(data=None), view(data=4096 + 8), view(n=132), view(h=4), view(b=-8)):
        assert L.sparsepr_key_means(p, bad, None, 0, FAKE, None) == spr.ERR_INVALID_ARG
        assert L.sparsepr_select_blocks(p, bad, FAKE, FAKE, FAKE, None) == spr.ERR_INVALID_ARG
        for at in range(4):
            vs = [bad if i == at else ok for i in range(4)]
            assert L.sparsepr_selected_attn(p, vs[0], vs[1], vs[2], FAKE, vs[3], FAKE, FAKE, None) == spr.ERR_INVALID_ARG
        for at in range(8):
            vs = [bad if i == at else ok for i in range(8)]
            assert L.sparsepr_selected_attn_backward(p, *vs[:5], FAKE, FAKE, *vs[5:], FAKE, None) == spr.ERR_INVALID_ARG
    assert L.sparsepr_key_means(p, ok, None, 0, None, None) == spr.ERR_INVALID_ARG
    assert L.sparsepr_key_means(p, ok, FAKE, 0, FAKE, None) == spr.ERR_INVALID_ARG and b"max_new" in L.sparsepr_last_error()
    assert L.sparsepr_select_blocks(p, ok, ctypes.c_void_p(4100), FAKE, FAKE, None) == spr.ERR_INVALID_ARG
    assert L.sparsepr_selected_attn(p, ok, ok, ok, None, ok, FAKE, FAKE, None) == spr.ERR_INVALID_ARG
    assert L.sparsepr_selected_attn(p, ok, ok, ok, FAKE, ok, FAKE, None, None) == spr.ERR_INVALID_ARG


def test_the_rest_of_out_is_checked(L):
    v = view()
    for kw, word in ((dict(dtype=spr.F32), b"bf16"), (dict(out_rest=4096 + 8), b"16-byte")):
        p = problem(**{"out_rest": 4096, **kw})
        assert L.sparsepr_selected_attn(p, v, v, v, FAKE, v, FAKE, FAKE, None) == spr.ERR_INVALID_ARG
        assert word in L.sparsepr_last_error()
        assert L.sparsepr_selected_attn_backward(p, v, v, v, v, v, FAKE, FAKE, v, v, v, FAKE, None) == spr.ERR_INVALID_ARG
        assert word in L.sparsepr_last_error()


def test_rows_that_repeat_are_refused_where_they_cannot_be(L):
    p, ok, flat = problem(Bt=2, Nq=10, Nk=300), view(b=1 << 20, h=1 << 16), view(b=1 << 20, h=1 << 16, n=0)
    one = view(b=0, h=1 << 16)
    for bad in ((ok, flat, ok, ok), (ok, ok, flat, ok), (ok, ok, ok, flat), (ok, ok, ok, one)):
        assert L.sparsepr_selected_attn(p, bad[0], bad[1], bad[2], FAKE, bad[3], FAKE, FAKE, None) == spr.ERR_INVALID_ARG
        assert b"repeat" in L.sparsepr_last_error()
    for at in (5, 6, 7):
        vs = [one if i == at else ok for i in range(8)]
        assert L.sparsepr_selected_attn_backward(p, *vs[:5], FAKE, FAKE, *vs[5:], FAKE, None) == spr.ERR_INVALID_ARG
        assert b"repeat" in L.sparsepr_last_error()
    assert rotary_rc(L, y=view(data=8192, h=128, n=0)) == spr.ERR_INVALID_ARG


def rotary_rc(L, par=None, x=None, y=None, x2=None, y2=None, h2=0, d=128, h1=2, dtype=spr.BF16, **kw):
    base = dict(rot_dim=64, first=0, layout=0, axes=1, pairs=(ctypes.c_int32 * 4)(32, 0, 0, 0), inverse=0, factor=1.0)
    base.update(kw)
    return L.sparsepr_rotary(ctypes.byref(S._CRotary(**base)), FAKE, FAKE, 0, 1, dtype, 1, 10, d, h1, x or view(h=2048),
                             y or view(data=8192, h=2048), h2, x2, y2, None)


@pytest.mark.parametrize("kw", [dict(rot_dim=0), dict(rot_dim=63), dict(rot_dim=130), dict(first=65), dict(first=-1),
                                dict(layout=2), dict(axes=0), dict(axes=5), dict(inverse=3), dict(factor=math.inf),
                                dict(pairs=(ctypes.c_int32 * 4)(31, 0, 0, 0)), dict(axes=2, pairs=(ctypes.c_int32 * 4)(40, -8, 0, 0)),
                                dict(h1=0), dict(dtype=9), dict(h2=1), dict(x=view(data=4097))], ids=str)
def test_rotary_refuses_bad_arguments(L, kw):
    assert rotary_rc(L, **kw) == spr.ERR_INVALID_ARG
    assert rotary_rc(L, d=80) == spr.ERR_UNSUPPORTED


def test_rotary_in_place_needs_the_same_strides(L):
    assert rotary_rc(L, x=view(h=4096, n=128), y=view(h=4096, n=256)) == spr.ERR_INVALID_ARG
    assert b"in place" in L.sparsepr_last_error()


def test_workspace_grows_with_the_backward_pass_and_stays_bounded(L):
    p = problem(Hq=16, Hkv=16, Nq=32760, Nk=32760, block=128, top=16)
    fwd, both = (int(L.sparsepr_selected_workspace_size(p, b)) for b in (0, 1))
    assert 0 < fwd <= both < 2 << 30   # partial rows are worked off in chunks of at most 1 GiB


def test_wrappers_refuse_what_the_kernels_do_not_take():
    q = torch.zeros(1, 2, 8, 64)
    cfg = spr.SelectConfig(block=64, top=2)
    with pytest.raises(ValueError, match="CUDA"):
        spr.selected_workspace(q, q, cfg)
    with pytest.raises(ValueError, match="CUDA"):
        spr.key_means(q, 64)
    plan = spr.rotary_plan(64, "cpu")
    with pytest.raises(ValueError, match="CUDA"):
        spr.rotary(plan, torch.zeros(1, 8, 1, dtype=torch.int32), q)


@pytest.mark.parametrize("kw", [dict(rot_dim=3), dict(rot_dim=66), dict(first=10), dict(layout=5), dict(sections=(10, 10)),
                                dict(sections=(8, 8, 8, 4, 4)), dict(freqs=[1.0]), dict(scaling="other"), dict(base=-1.0),
                                dict(scaling="ramp", scaling_factor=2.0), dict(scaling="linear", scaling_factor=0.0),
                                dict(freqs=[1.0] * 32, base=2.0)], ids=str)
def test_rotary_plans_are_checked(kw):
    if kw.get("first") == 10:
        kw = dict(first=10, rot_dim=60)
    with pytest.raises(ValueError):
        spr.rotary_plan(64, "cpu", **kw)


def test_frequency_ladders():
    f, factor = spr.rotary_frequencies((4,), base=16.0)
    assert factor == 1.0 and f == pytest.approx([1.0, 0.5, 0.25, 0.125])
    assert spr.rotary_frequencies((4,), base=16.0, scaling="linear", scaling_factor=4.0)[0] == pytest.approx([x / 4 for x in f])
    # the base ladder keeps the first frequency and divides the last by the factor
    g, _ = spr.rotary_frequencies((32,), scaling="base", scaling_factor=8.0)
    f, _ = spr.rotary_frequencies((32,))
    assert g[0] == f[0] and g[-1] == pytest.approx(f[-1] / 8)
    # the ramp: many turns kept, few interpolated, the factor of the paper's rule
    g, factor = spr.rotary_frequencies((32,), scaling="ramp", scaling_factor=8.0, trained_length=4096)
    assert g[0] == f[0] and g[-1] == pytest.approx(f[-1] / 8) and factor == pytest.approx(0.1 * math.log(8) + 1)
    turns = [4096 * x / (2 * math.pi) for x in f]
    for a, b, r in zip(f, g, turns):
        keep = min(1.0, max(0.0, (r - 1) / 31))
        assert b == pytest.approx(a * keep + a / 8 * (1 - keep))
    # axes are ladders of their own
    assert spr.rotary_frequencies((2, 3))[0] == spr.rotary_frequencies((2,))[0] + spr.rotary_frequencies((3,))[0]
