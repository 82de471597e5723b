"""Selected-block attention without a GPU: what its workspaces take, and what the Python calls refuse."""
import ctypes

import pytest

import free_block_sparse_response_b200 as spr
from free_block_sparse_response_b200 import selected as S


@pytest.fixture(scope="module")
def L():
    from free_block_sparse_response_b200.build import build
    build()
    return spr.lib()


@pytest.mark.parametrize("dtype", [spr.BF16, spr.F32])
@pytest.mark.parametrize("hq,hk,top", [(32, 4, 16), (32, 4, 32), (64, 8, 64), (32, 1, 16), (128, 1, 64), (16, 16, 16)])
def test_workspaces_of_long_contexts_stay_bounded(L, hq, hk, top, dtype):
    """131,072 tokens: partial rows of 1 GiB at a time in both directions, or of the smallest slice, 512 tokens
    (128 heads to a key head and 64 blocks: 4.2 million rows of 272 or 520 bytes); beside them what grows
    with the call: lists and their inverse (the selection's size each) with their counts, a record of 48 bytes
    for 128 rows (2^30 rows: 0.4 GB), the row sums, and the fp32 sums of one head's dK and dV where its
    tokens are cut."""
    n, d, block = 131072, 128, 64
    p = S._CSelected(dtype=dtype, Bt=1, Hq=hq, Hkv=hk, Nq=n, Nk=n, d=d, block=block, top=top)
    sel, row = 4 * hk * n * top, 4 * hq * n
    parts = max(1 << 30, 512 * top * (hq // hk) * (2 * d + 16 if dtype == spr.BF16 else 4 * d + 8))
    for backward in (0, 1):
        size = int(L.sparsepr_selected_workspace_size(ctypes.byref(p), backward))
        assert 0 < size < parts + 48 * n * top * hq // 128 + 3 * sel + 2 * row + (1 << 28) + backward * 2 * 4 * n * d
