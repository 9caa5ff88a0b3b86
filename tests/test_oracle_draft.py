"""Pins of the drafted-token and window oracle, and what the library's calls for
them refuse before any CUDA call (no GPU)."""
import ctypes as C

import numpy as np
import pytest
import torch

from oracle import attention as oa
from oracle import draft as od


@pytest.fixture(scope="module")
def pkv():
    import __graft_entry__ as g
    g.build()
    import paged_kv_cache_153_gb300 as m
    return m


def test_ancestors_by_hand():
    #        0
    #      1   2        3 (a second root)
    #      4           5
    seen = od.ancestors([-1, 0, 0, -1, 1, 3])
    assert [list(np.flatnonzero(r)) for r in seen] == [[0], [0, 1], [0, 2], [3], [0, 1, 4], [3, 5]]
    assert (od.ancestors([-1, 0, 1, 2]) == np.tril(np.ones((4, 4), bool))).all()
    assert (od.ancestors([-1] * 5) == np.eye(5, dtype=bool)).all()


def test_mask_words_by_hand():
    seen = np.zeros((2, 130), dtype=bool)
    seen[0, [0, 63, 64, 129]] = True
    w = od.mask_words(seen, 3).view(np.uint64)
    assert [int(x) for x in w[0]] == [1 | 1 << 63, 1, 2] and not w[1].any()


def test_a_chain_is_causal_attention():
    rng = np.random.default_rng(0)
    k, v, q = rng.standard_normal((20, 8)), rng.standard_normal((20, 8)), rng.standard_normal((5, 8))
    got = od.masked_attend(q, k, v, od.tree_seen(15, od.ancestors([-1, 0, 1, 2, 3])), 0.3)
    for i in range(5):
        assert np.allclose(got[i], oa.attend(q[i], k[:16 + i], v[:16 + i], 0.3))


def test_what_is_not_seen_takes_no_part():
    rng = np.random.default_rng(1)
    k, v, q = rng.standard_normal((6, 4)), rng.standard_normal((6, 4)), rng.standard_normal((2, 4))
    seen = np.array([[1, 0, 1, 0, 1, 1], [0, 0, 0, 0, 0, 0]], dtype=bool)
    want = od.masked_attend(q, k, v, seen, 1.0)
    k[[1, 3]], v[[1, 3]] = np.nan, np.inf
    assert (od.masked_attend(q, k, v, seen, 1.0) == want).all() and not want[1].any()


def test_window_by_hand():
    seen = od.window_seen([6, 1], 8, 3, 2)
    assert list(np.flatnonzero(seen[0])) == [0, 1, 4, 5, 6] and list(np.flatnonzero(seen[1])) == [0, 1]
    assert (od.window_seen(range(8), 8, 8, 0) == np.tril(np.ones((8, 8), bool))).all()
    assert (od.window_seen(range(8), 8, 1, 0) == np.eye(8, dtype=bool)).all()


def test_commit_by_hand():
    rows = np.arange(10)
    assert list(od.commit(rows, 4, [0, 2, 5])) == [0, 1, 2, 3, 4, 6, 9, 7, 8, 9]
    assert list(od.commit(rows, 4, [])) == list(rows)


A, ODD = C.c_void_p(4096), C.c_void_p(4096 + 8)
KINDS = ["", "_fp8", "_e5m2"]


@pytest.mark.parametrize("kind", KINDS)
def test_window_decode_refusals(pkv, kind):
    def call(q=A, kc=A, vc=A, ks=A, vs=A, tab=A, lens=A, b=2, hq=8, hkv=2, d=128, bs=16, mb=4, nb=8, w=5, s=1,
             scale=0.1, out=A, dt=1, ws=A, wsb=1 << 30):
        scales = (ks, vs) if kind else ()
        return getattr(pkv.lib, "pkv_paged_decode_attention_window" + kind)(
            q, kc, vc, *scales, tab, lens, b, hq, hkv, d, bs, mb, nb, w, s, scale, out, dt, ws, wsb, None, None)
    for bad in (dict(q=None), dict(kc=None), dict(vc=None), dict(tab=None), dict(lens=None), dict(out=None),
                dict(ws=None), dict(q=ODD), dict(kc=ODD), dict(vc=ODD), dict(out=ODD), dict(ws=ODD), dict(b=-1),
                dict(hq=7), dict(hkv=0), dict(mb=0), dict(nb=-1), dict(w=0), dict(w=-3), dict(s=-1),
                dict(scale=float("nan")), dict(dt=2)) + ((dict(ks=None), dict(vs=None)) if kind else ()):
        assert call(**bad) == 1, bad
    for bad in (dict(hq=6), dict(d=96), dict(bs=32)):
        assert call(**bad) == 2, bad
    assert call(b=0) == 0


@pytest.mark.parametrize("kind", KINDS)
def test_tree_attention_refusals(pkv, kind):
    def call(q=A, kc=A, vc=A, ks=A, vs=A, tab=A, lens=A, cu=A, mask=A, words=1, mn=8, t=20, b=2, hq=8, hkv=2, d=128,
             bs=16, mb=4, nb=8, mx=64, scale=0.1, out=A, dt=1, ws=A, wsb=1 << 30):
        scales = (ks, vs) if kind else ()
        return getattr(pkv.lib, "pkv_paged_tree_attention" + kind)(
            q, kc, vc, *scales, tab, lens, cu, mask, words, mn, t, b, hq, hkv, d, bs, mb, nb, mx, scale, out, dt, ws,
            wsb, None, None)
    for bad in (dict(q=None), dict(kc=None), dict(vc=None), dict(tab=None), dict(lens=None), dict(cu=None),
                dict(mask=None), dict(out=None), dict(ws=None), dict(q=ODD), dict(kc=ODD), dict(vc=ODD), dict(out=ODD),
                dict(ws=ODD), dict(b=-1), dict(t=-1), dict(hq=7), dict(hkv=0), dict(mb=0), dict(nb=-1), dict(nb=0),
                dict(mx=-1), dict(mn=-1), dict(mn=65), dict(words=0), dict(scale=0.0), dict(scale=-1.0),
                dict(scale=float("inf")), dict(dt=2)) + ((dict(ks=None), dict(vs=None)) if kind else ()):
        assert call(**bad) == 1, bad
    for bad in (dict(hq=6), dict(d=96), dict(bs=32), dict(words=5), dict(b=1025), dict(nb=1 << 30), dict(t=1 << 31)):
        assert call(**bad) == 2, bad
    assert call(b=0) == 0 and call(t=0) == 0 and call(mn=0) == 0


def test_tree_workspace_of_bad_sizes(pkv):
    f = pkv.lib.pkv_tree_workspace_bytes
    for bad in ((-1, 4, 8, 2, 128, 4), (2, -4, 8, 2, 128, 4), (2, 4, 7, 2, 128, 4), (2, 4, 8, 0, 128, 4),
                (2, 4, 8, 2, 0, 4), (2, 4, 8, 2, 128, -1), (2, 4, 8, 2, 128, 257)):
        assert f(*bad) == 0, bad


def test_plan_refusals(pkv):
    def call(par=A, cu=A, tab=A, lens=A, b=2, t=9, words=1, bs=16, mb=4, nb=8, mask=A, pos=A, slots=A):
        return pkv.lib.pkv_tree_plan(par, cu, tab, lens, b, t, words, bs, mb, nb, mask, pos, slots, None, None)
    for bad in (dict(par=None), dict(cu=None), dict(tab=None), dict(lens=None), dict(mask=None), dict(b=-1),
                dict(t=-1), dict(words=0), dict(nb=-1), dict(mb=0)):
        assert call(**bad) == 1, bad
    assert call(words=5) == 2 and call(bs=32) == 2
    assert call(b=0) == 0 and call(t=0) == 0


def test_commit_refusals(pkv):
    other = C.c_void_p(8192)

    def call(kc=A, vc=A, tab=A, lens=A, cu=A, acc=A, most=4, b=2, h=2, d=128, bs=16, mb=4, nb=8, e=2, new=other):
        return pkv.lib.pkv_tree_commit(kc, vc, tab, lens, cu, acc, most, b, h, d, bs, mb, nb, e, new, None, None)
    for bad in (dict(kc=None), dict(vc=None), dict(tab=None), dict(lens=None), dict(cu=None), dict(acc=None),
                dict(kc=ODD), dict(vc=ODD), dict(most=-1), dict(b=-1), dict(h=0), dict(mb=0), dict(nb=-1), dict(e=4),
                dict(new=A)):
        assert call(**bad) == 1, bad
    for bad in (dict(d=96), dict(bs=32), dict(most=1025), dict(b=65536)):
        assert call(**bad) == 2, bad
    assert call(b=0) == 0


def test_new_lengths_within_the_old_ones_are_refused(pkv):
    for shift in (-4, 0, 4):
        assert pkv.lib.pkv_tree_commit(A, A, A, A, A, A, 4, 2, 2, 128, 16, 4, 8, 2, C.c_void_p(A.value + shift), None,
                                       None) == 1, shift


def test_window_prefill_refusals(pkv):
    def call(q=A, kc=A, vc=A, tab=A, lens=A, cu=A, t=20, b=2, hq=8, hkv=2, d=128, bs=16, mb=4, nb=8, ml=10, w=5, s=1,
             scale=0.1, out=A, dt=1):
        return pkv.lib.pkv_paged_prefill_attention_window(q, kc, vc, tab, lens, cu, t, b, hq, hkv, d, bs, mb, nb, ml, w,
                                                          s, scale, out, dt, None, None)
    for bad in (dict(q=None), dict(kc=None), dict(vc=None), dict(tab=None), dict(lens=None), dict(cu=None),
                dict(out=None), dict(q=ODD), dict(kc=ODD), dict(vc=ODD), dict(out=ODD), dict(b=-1), dict(t=-1),
                dict(hq=7), dict(hkv=0), dict(mb=0), dict(nb=-1), dict(nb=0), dict(ml=-1), dict(w=0), dict(s=-1),
                dict(scale=0.0), dict(scale=float("nan")), dict(dt=2)):
        assert call(**bad) == 1, bad
    for bad in (dict(hq=6), dict(d=96), dict(bs=32), dict(b=65536), dict(nb=1 << 30)):
        assert call(**bad) == 2, bad
    assert call(b=0) == 0 and call(t=0) == 0 and call(ml=0) == 0


# ---- what the binding refuses (tensors on the host: a call that fits is refused for its device) ----
B, T, HQ, HKV, D, NB, W = 3, 7, 8, 2, 64, 10, 4
BF = torch.bfloat16


def args(**over):
    z = torch.zeros
    a = dict(q=z((T, HQ, D), dtype=BF), out=z((T, HQ, D), dtype=BF), k=z((NB, HKV, 16, D), dtype=BF),
             v=z((NB, HKV, 16, D), dtype=BF), k8=z((NB, HKV, 16, D), dtype=torch.uint8),
             v8=z((NB, HKV, 16, D), dtype=torch.uint8), ks=z(HKV), vs=z(HKV), tab=z((B, W), dtype=torch.int32),
             lens=z(B, dtype=torch.int32), cu=z(B + 1, dtype=torch.int32), mask=z((T, 1), dtype=torch.int64),
             par=z(T, dtype=torch.int32), pos=z(T, dtype=torch.int32), slots=z(T, dtype=torch.int64),
             acc=z((B, 2), dtype=torch.int32), new=z(B, dtype=torch.int32), ws=z(64, dtype=torch.uint8),
             qd=z((B, HQ, D), dtype=BF), outd=z((B, HQ, D), dtype=BF), err=z(1, dtype=torch.int32))
    a.update(over)
    return a


def plan(pkv, a):
    pkv.pkv_tree_plan(a["par"], a["cu"], a["tab"], a["lens"], a["mask"], a["pos"], a["slots"], num_blocks=NB,
                      err_flag=a["err"], stream=0)


def tree(pkv, a):
    pkv.pkv_paged_tree_attention(a["q"], a["k"], a["v"], a["tab"], a["lens"], a["cu"], a["mask"], a["out"], scale=1.0,
                                 max_context_len=64, max_nodes=8, workspace=a["ws"], err_flag=a["err"], stream=0)


def tree_fp8(pkv, a):
    pkv.pkv_paged_tree_attention_fp8(a["q"], a["k8"], a["v8"], a["ks"], a["vs"], a["tab"], a["lens"], a["cu"],
                                     a["mask"], a["out"], scale=1.0, max_context_len=64, max_nodes=8,
                                     workspace=a["ws"], err_flag=a["err"], stream=0)


def commit(pkv, a):
    pkv.pkv_tree_commit(a["k"], a["v"], a["tab"], a["lens"], a["cu"], a["acc"], new_lens=a["new"], err_flag=a["err"],
                        stream=0)


def window(pkv, a):
    pkv.pkv_paged_decode_attention_window(a["qd"], a["k"], a["v"], a["tab"], a["lens"], a["outd"], scale=1.0, window=4,
                                          num_sinks=1, workspace=a["ws"], err_flag=a["err"], stream=0)


def window_e5m2(pkv, a):
    pkv.pkv_paged_decode_attention_window_e5m2(a["qd"], a["k8"], a["v8"], a["ks"], a["vs"], a["tab"], a["lens"],
                                               a["outd"], scale=1.0, window=4, workspace=a["ws"], err_flag=a["err"],
                                               stream=0)


def chunk(pkv, a):
    pkv.pkv_paged_prefill_attention_window(a["q"], a["k"], a["v"], a["tab"], a["lens"], a["cu"], a["out"], scale=1.0,
                                           max_query_len=8, window=4, num_sinks=1, err_flag=a["err"], stream=0)


READS = {plan: "par cu tab lens pos", tree: "tab lens cu", tree_fp8: "tab lens cu", commit: "tab lens cu acc new",
         window: "tab lens", window_e5m2: "tab lens", chunk: "tab lens cu"}


@pytest.mark.parametrize("call", READS, ids=lambda f: f.__name__)
def test_calls_that_fit_get_as_far_as_the_device(pkv, call):
    with pytest.raises(ValueError, match="device"):
        call(pkv, args())


def refused(pkv, call, **over):
    with pytest.raises((TypeError, ValueError)) as e:
        call(pkv, args(**over))
    assert "device" not in str(e.value), (over, e.value)


@pytest.mark.parametrize("call", READS, ids=lambda f: f.__name__)
def test_index_tensors_of_other_types_and_strides_are_refused(pkv, call):
    for name in READS[call].split():
        t = args()[name]
        refused(pkv, call, **{name: t.long()})
        refused(pkv, call, **{name: torch.zeros((*t.shape[:-1], 2 * t.shape[-1]), dtype=torch.int32)[..., ::2]})
    refused(pkv, call, err=torch.zeros(1))


def test_shapes_and_types_that_do_not_fit_are_refused(pkv):
    z = torch.zeros
    for call in (tree, tree_fp8, plan):
        refused(pkv, call, mask=z((T, 1), dtype=torch.int32))
        refused(pkv, call, mask=z((T + 1, 1), dtype=torch.int64))
        refused(pkv, call, mask=z(T, dtype=torch.int64))
    for call in (tree, tree_fp8, plan, commit, chunk):
        refused(pkv, call, cu=z(B, dtype=torch.int32))
    for call in (tree, chunk):
        refused(pkv, call, out=z((T, HQ, D)))
        refused(pkv, call, out=z((T + 1, HQ, D), dtype=BF))
        refused(pkv, call, q=z((T, HQ, 2 * D), dtype=BF)[..., ::2])
        refused(pkv, call, k=z((NB, HKV, 16, D), dtype=torch.float16), v=z((NB, HKV, 16, D), dtype=torch.float16))
        refused(pkv, call, v=z((NB + 1, HKV, 16, D), dtype=BF))
        refused(pkv, call, tab=z((B + 1, W), dtype=torch.int32))
    for call in (tree_fp8, window_e5m2):
        refused(pkv, call, ks=z(HKV + 1))
        refused(pkv, call, vs=z(HKV, dtype=torch.float64))
        refused(pkv, call, k8=z((NB, HKV, 16, D), dtype=BF), v8=z((NB, HKV, 16, D), dtype=BF))
    other = {tree_fp8: torch.float8_e5m2, window_e5m2: torch.float8_e4m3fn}
    for call, t in other.items():
        refused(pkv, call, k8=z((NB, HKV, 16, D), dtype=torch.uint8).view(t),
                v8=z((NB, HKV, 16, D), dtype=torch.uint8).view(t))
    refused(pkv, plan, slots=z(T, dtype=torch.int32))
    refused(pkv, plan, slots=z(T + 1, dtype=torch.int64))
    refused(pkv, plan, pos=z(T + 1, dtype=torch.int32))
    refused(pkv, commit, acc=z((B + 1, 2), dtype=torch.int32))
    refused(pkv, commit, new=z(B + 1, dtype=torch.int32))
    refused(pkv, commit, k=z((NB, HKV, 16, D)), v=z((NB, HKV, 16, D)))
    refused(pkv, commit, k=z((NB, 16, D), dtype=BF), v=z((NB, 16, D), dtype=BF))
