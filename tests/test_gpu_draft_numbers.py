"""Numbers of the drafted tokens' attention that plain random inputs do not reach."""
import numpy as np
import pytest
import torch

from tests import attn_limits
from tests.test_gpu_draft import OOB, Case
from tests.test_gpu_window import chunk_case, prefill

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    import __graft_entry__ as g
    g.build()
    import paged_kv_cache_153_gb300 as m
    return m


@pytest.mark.parametrize("kv", ["e4m3", "e5m2"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("d,new", [(64, 9), (128, 70)])
def test_scales_of_zero_and_below_and_rows_of_zeros(pkv, kv, dtype, d, new):
    # (the dense decode over FP8 caches asks nothing of the scales either)
    c = Case([0, 5, 300], [new, 3, new // 2], hq=16, hkv=8, d=d, dtype=dtype, kv=kv, seed=d)
    c.ks[:8] = torch.tensor([0.0, -0.7, 1e-9, 0.8, -1e-9, -1.2, -0.0, 2.0 ** -120])
    c.vs[:4] = torch.tensor([0.5, 0.0, -0.6, 1.0])
    c.q_h[1:4] = 0
    c.q_h[:, 6] = 0
    out = c.attend(pkv)
    assert int(c.err.item()) == 0
    c.check(out)


def test_a_scale_that_is_not_a_number_stays_in_its_head(pkv):
    c = Case([0, 200], [5, 9], hq=8, hkv=4, d=64, kv="e4m3", seed=2)
    c.ks[1] = float("nan")
    seen = [np.tril(np.ones((n, n), bool)) for n in (5, 9)]
    seen[0][2] = False                                         # no key at all: 0, whatever the scale
    c2 = Case([0, 200], [5, 9], hq=8, hkv=4, d=64, kv="e4m3", seed=2, seen=seen)
    c2.ks[1] = float("nan")
    for case in (c, c2):
        out = case.attend(pkv).float()
        fine = torch.isfinite(out).all(2)
        want = torch.ones_like(fine)
        want[:, 2:4] = False
        if case is c2:
            want[2] = True
            assert not out[2].any()
        assert torch.equal(fine, want)


@pytest.mark.parametrize("dtype,kv", [("f16", None), ("f16", "e4m3"), ("bf16", "e4m3"), ("f16", "e5m2"),
                                      ("bf16", "e5m2")])
@pytest.mark.parametrize("d", [64, 128])
def test_one_query_head_per_kv_head_keeps_the_weights_in_two_parts(pkv, dtype, kv, d):
    """The dense decode holds such weights in fp32.  Two fp16 parts of a weight are off by
    2^-22 of it; attn_limits' two-part limit (bf16 parts, 2^-15) covers them.  Pairs of
    opposite values make outputs near 0, whose own rounding is small beside one
    rounding of the weights to fp16 (2^-12)."""
    n = [2, 3, 5, 9, 150]
    c = Case([0, 1, 4, 7, 140], n, hq=4, hkv=4, d=d, dtype=dtype, kv=kv, seed=7,
             seen=[np.tril(np.ones((x, x), bool)) for x in n])
    for b in range(len(n)):
        for p in range(1, int(c.ctx[b]), 2):
            here, there = ((int(c.tab[b, x // 16]), x % 16) for x in (p, p - 1))
            c.vc_h[here[0], :, here[1]] = c.vc_h[there[0], :, there[1]] ^ 0x80 if kv else -c.vc_h[there[0], :, there[1]]
    c.q_h *= 0.25                                              # (logits near each other)
    got = c.attend(pkv).double().cpu().numpy()
    assert int(c.err.item()) == 0
    for b in range(len(n)):
        for g in range(4):
            k, v = c.rows(b, g)
            for i in range(0, n[b], 1 if n[b] < 10 else 31):
                m = int(c.base[b]) + i + 1
                ref, lim = attn_limits.attend(c.q_h[c.cu[b] + i, g].double().numpy(), k[:m], v[:m], c.scale, dtype,
                                              "bf16")
                x = got[c.cu[b] + i, g]
                assert (np.abs(x - ref) <= lim).all(), (b, g, i, float((np.abs(x - ref) / lim).max()))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("kv", ["e4m3", "e5m2"])
@pytest.mark.parametrize("outlier,where", [(2.0 ** 10, ...), (2.0 ** 12, ...), (2.0 ** 12, 3), (1.5 * 2.0 ** 14, ...)])
def test_an_outlier_of_q_leaves_the_other_elements_their_bits(pkv, dtype, kv, outlier, where):
    """One element of each row of q (or of one row) is far larger than the others, and K
    is 0 there.  The others are exact as parts down to 2^-13 of the row's largest, and off
    by 2^-21 (bf16, two parts) or 2^-24 (fp16, three) of it below."""
    c = Case([300, 20], [12, 5], hq=8, hkv=2, d=64, dtype=dtype, kv=kv, seed=3)
    c.q_h.clamp_(-2, 2)
    c.q_h[where, :, 5] = outlier if dtype == "bf16" else min(outlier, 2.0 ** 14)
    dead = c.kc_h == 0x7F
    c.kc_h[..., 5] = 0
    c.kc_h[dead] = 0x7F
    c.ks[:] = torch.tensor([4.0, 2.0])                         # (logits of tens)
    part = 2.0 ** -21 if dtype == "bf16" else 2.0 ** -24
    got = c.attend(pkv).double().cpu().numpy()
    assert int(c.err.item()) == 0
    for b in range(2):
        for g in range(2):
            k, v = c.rows(b, g)
            for i in range(int(c.new[b])):
                at = np.concatenate([np.arange(int(c.base[b])), int(c.base[b]) + np.flatnonzero(c.seen[b][i])])
                for h in range(4 * g, 4 * g + 4):
                    q = c.q_h[c.cu[b] + i, h].double().numpy()
                    ref, lim = attn_limits.attend(q, k[at], v[at], c.scale, dtype, "f16")
                    logit = k[at] @ q * c.scale
                    w = np.exp(logit - logit.max())
                    # a logit off by delta moves weight and normaliser by a factor of e^delta each
                    delta = c.scale * part * np.abs(q).max() * np.abs(k[at]).sum(1).max()
                    lim = lim + np.expm1(2 * delta) * (w / w.sum()) @ np.abs(v[at])
                    x = got[c.cu[b] + i, h]
                    assert (np.abs(x - ref) <= lim).all(), (b, i, h, float((np.abs(x - ref) / lim).max()))


@pytest.mark.parametrize("dtype,kv", [("bf16", None), ("f16", "e4m3"), ("bf16", "e5m2")])
def test_rows_behind_the_last_sequence_change_nothing(pkv, dtype, kv):
    # a batch padded to a fixed number of tokens, whatever the padding holds
    c = Case([20, 5, 130], [6, 0, 40], hq=8, hkv=2, dtype=dtype, kv=kv, extra=40)
    want = c.attend(pkv).clone()
    c.check(want)
    for bad in (float("nan"), float("inf"), 6e4):
        c.q_h[46:] = bad
        out = c.attend(pkv)
        assert torch.equal(out[:46], want[:46]) and bool((out[46:] == 7.0).all()) and int(c.err.item()) == 0, bad


@pytest.mark.parametrize("kv", [None, "e4m3"])
def test_a_bound_of_no_drafted_tokens_is_too_small_for_some(pkv, kv):
    c = Case([20, 5], [6, 2], hq=8, hkv=2, kv=kv)
    out = c.attend(pkv, max_nodes=0)
    assert int(c.err.item()) == OOB and bool((out == 7.0).all())
    c = Case([20, 5], [0, 0], hq=8, hkv=2, kv=kv, extra=3)     # nothing but padding
    out = c.attend(pkv, max_nodes=0)
    assert int(c.err.item()) == 0 and bool((out == 7.0).all())
    c = Case([20, 5], [6, 2], hq=8, hkv=2, kv=kv)
    out = c.attend(pkv, max_nodes=0, err_flag=None)            # (nobody to tell)
    assert bool((out == 7.0).all())


def test_a_bound_of_no_new_tokens_is_too_small_for_some(pkv):
    c = chunk_case([40, 40], [5, 60], hq=8, hkv=2)
    out = prefill(pkv, c, 30, 2, max_query_len=0)
    assert int(c.err.item()) == OOB and bool((out == 7.0).all())
    c = chunk_case([40, 40], [0, 0], hq=8, hkv=2, extra=3)
    out = prefill(pkv, c, 30, 2, max_query_len=0)
    assert int(c.err.item()) == 0 and bool((out == 7.0).all())
