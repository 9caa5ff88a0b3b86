"""What the shared-prefix decode refuses before any CUDA call (no GPU)."""
import ctypes as C

import pytest


@pytest.fixture(scope="module")
def pkv():
    import __graft_entry__ as g
    g.build()
    import paged_kv_cache_153_gb300 as m
    return m


def test_refusals_before_any_cuda_call(pkv):
    a, odd = C.c_void_p(4096), C.c_void_p(4096 + 8)

    def call(q=a, kc=a, vc=a, tab=a, lens=a, starts=a, pre=a, ng=2, b=4, hq=8, hkv=2, d=128, bs=16, mb=8, nb=16, mx=64,
             mp=32, scale=0.1, out=a, dt=1, ws=a, wsb=1 << 30):
        return pkv.lib.pkv_paged_decode_attention_prefix(q, kc, vc, tab, lens, starts, pre, ng, b, hq, hkv, d, bs, mb, nb,
                                                         mx, mp, scale, out, dt, ws, wsb, None, None)
    for bad in (dict(q=None), dict(kc=None), dict(vc=None), dict(tab=None), dict(lens=None), dict(starts=None),
                dict(pre=None), dict(out=None), dict(ws=None), dict(q=odd), dict(kc=odd), dict(vc=odd), dict(out=odd),
                dict(ws=odd), dict(ng=-1), dict(ng=0), dict(b=-1), dict(hq=7), dict(hq=0), dict(hkv=0), dict(mb=0),
                dict(nb=-1), dict(mx=-1), dict(mp=-1), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
                dict(dt=2)):
        assert call(**bad) == 1, bad
    for bad in (dict(hq=6), dict(d=96), dict(bs=32), dict(ng=1025)):
        assert call(**bad) == 2, bad
    assert call(b=0, ng=0) == 0
    assert pkv.lib.pkv_prefix_workspace_bytes(4, 2, 7, 2, 128, 8, 64, 32) == 0
    assert pkv.lib.pkv_prefix_workspace_bytes(-1, 2, 8, 2, 128, 8, 64, 32) == 0
