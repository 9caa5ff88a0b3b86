"""Pins of the block-sparse oracle, and what the library's block-sparse calls
refuse before any CUDA call (no GPU)."""
import ctypes as C

import numpy as np
import pytest

from oracle import attention as oa
from oracle import sparse as osp


@pytest.fixture(scope="module")
def pkv():
    import __graft_entry__ as g
    g.build()
    import paged_kv_cache_153_gb300 as m
    return m


def test_a_score_bounds_every_logit_of_its_block():
    rng = np.random.default_rng(0)
    for rows in (1, 7, 16):
        k, q = rng.standard_normal((16, 64)), rng.standard_normal((4, 64))
        s = osp.block_score(q, *osp.block_bounds(k, rows), 0.125)
        assert s >= (q @ k[:rows].T).max() * 0.125 - 1e-13      # (equal for one row, up to rounding)
        # one row: the bound is the logit
        one = osp.block_score(q, *osp.block_bounds(k, 1), 1.0)
        assert one == pytest.approx((q @ k[0]).max())


def test_selection_by_hand():
    s = [5.0, 1.0, 9.0, 9.0, float("nan"), 2.0, 0.0, float("-inf")]
    assert osp.select_blocks(s, 8, 1, 1, 4) == [0, 2, 4, 7]
    assert osp.select_blocks(s, 8, 0, 0, 3) == [2, 3, 4]
    assert osp.select_blocks(s, 8, 0, 0, 2) == [2, 4]          # the tie goes to the lower index
    assert osp.select_blocks(s, 8, 2, 2, 4) == [0, 1, 6, 7]
    assert osp.select_blocks(s, 3, 1, 1, 5) == [0, 1, 2]


def test_listing_every_block_is_dense_attention():
    rng = np.random.default_rng(1)
    k, v, q = rng.standard_normal((37, 32)), rng.standard_normal((37, 32)), rng.standard_normal(32)
    pos = osp.token_positions([2, 0, -1, 1], 37)
    assert sorted(pos) == list(range(37))
    assert np.allclose(oa.attend(q, k[pos], v[pos], 0.2), oa.attend(q, k, v, 0.2))


def test_refusals_before_any_cuda_call(pkv):
    lib, a, odd = pkv.lib, C.c_void_p(4096), C.c_void_p(4096 + 8)

    def bounds(kc=a, tab=a, lens=a, new=None, mx=5, b=2, hkv=2, d=128, bs=16, mb=4, nb=8, out=a, dt=1,
               fn="pkv_kv_block_bounds"):
        return getattr(lib, fn)(kc, tab, lens, new, mx, b, hkv, d, bs, mb, nb, out, dt, None, None)
    for fn in ("pkv_kv_block_bounds", "pkv_kv_block_bounds_fp8", "pkv_kv_block_bounds_e5m2"):
        for bad in (dict(kc=None), dict(tab=None), dict(lens=None), dict(out=None), dict(kc=odd), dict(out=odd),
                    dict(b=-1), dict(hkv=0), dict(mb=0), dict(nb=-1), dict(mx=-1), dict(dt=7)):
            assert bounds(fn=fn, **bad) == 1, bad
        assert bounds(fn=fn, d=96) == 2 and bounds(fn=fn, bs=32) == 2
        assert bounds(fn=fn, b=0) == 0 and bounds(fn=fn, mx=0) == 0

    def scores(q=a, bd=a, tab=a, lens=a, b=2, hq=8, hkv=2, d=128, bs=16, mb=4, nb=8, mx=64, scale=0.1, out=a, dt=1):
        return lib.pkv_block_scores(q, bd, tab, lens, None, b, hq, hkv, d, bs, mb, nb, mx, scale, out, dt, None, None)
    for bad in (dict(q=None), dict(bd=None), dict(tab=None), dict(lens=None), dict(out=None), dict(q=odd), dict(bd=odd),
                dict(b=-1), dict(hq=7), dict(hkv=0), dict(mb=0), dict(nb=-1), dict(mx=-1), dict(scale=-1.0),
                dict(scale=float("nan")), dict(dt=3)):
        assert scores(**bad) == 1, bad
    assert scores(hq=6) == 2 and scores(d=32) == 2 and scores(bs=8) == 2
    assert scores(b=0) == 0 and scores(mx=0) == 0

    def select(sc=a, lens=a, b=2, hkv=2, bs=16, mb=4, f=1, last=1, budget=4, out=a):
        return lib.pkv_select_blocks(sc, lens, b, hkv, bs, mb, f, last, budget, out, None, None)
    for bad in (dict(sc=None), dict(lens=None), dict(out=None), dict(b=-1), dict(hkv=0), dict(mb=0), dict(f=-1),
                dict(last=-1), dict(budget=0), dict(f=3, last=2), dict(f=2 ** 31 - 1, last=2 ** 31 - 1)):
        assert select(**bad) == 1, bad
    assert select(bs=32) == 2 and select(b=0) == 0

    def sparse(q=a, kc=a, vc=a, tab=a, lens=a, sel=a, budget=4, b=2, hq=8, hkv=2, d=128, bs=16, mb=4, nb=8, scale=0.1,
               out=a, dt=1, ws=a, wsb=1 << 24, fn="pkv_paged_decode_attention_sparse", scales=()):
        return getattr(lib, fn)(q, kc, vc, *scales, tab, lens, sel, budget, b, hq, hkv, d, bs, mb, nb, scale, out, dt,
                                ws, wsb, None, None)
    for fn, sc in (("pkv_paged_decode_attention_sparse", ()), ("pkv_paged_decode_attention_sparse_fp8", (a, a)),
                   ("pkv_paged_decode_attention_sparse_e5m2", (a, a))):
        for bad in (dict(q=None), dict(kc=None), dict(vc=None), dict(tab=None), dict(lens=None), dict(sel=None),
                    dict(out=None), dict(ws=None), dict(q=odd), dict(kc=odd), dict(out=odd), dict(budget=0),
                    dict(budget=-3), dict(budget=2 ** 31 - 1), dict(b=-1), dict(hq=7), dict(scale=float("inf")),
                    dict(dt=9)):
            assert sparse(fn=fn, scales=sc, **bad) == 1, (fn, bad)
        assert sparse(fn=fn, scales=sc, hq=6) == 2 and sparse(fn=fn, scales=sc, d=96) == 2
        assert sparse(fn=fn, scales=sc, b=0, sel=None) == 0
        if sc:
            assert sparse(fn=fn, scales=(None, a)) == 1 and sparse(fn=fn, scales=(a, None)) == 1
