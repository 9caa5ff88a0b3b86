"""The weights of the shared-prefix decode: as exact as the dense decode's."""
import math

import numpy as np
import pytest
import torch

from tests import attn_limits
from tests.test_gpu_prefix import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    import __graft_entry__ as g
    g.build()
    import paged_kv_cache_153_gb300 as m
    return m


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("h,d", [(3, 128), (8, 64)])
@pytest.mark.parametrize("shared,own", [(512, [0, 1, 3]), (32, [300, 200, 77]), (2000, [500, 40]), (400, [5] * 140)])
def test_one_query_head_per_kv_head(pkv, dtype, h, d, shared, own):
    # The dense decode keeps the weights in fp32 there; here they are products of
    # two 16-bit parts: for fp16, p less its 11 bits is 2^-12 p at most, and that
    # rounds by 2^-12 of itself or half of fp16's smallest step, 2^-25 of the largest
    # weight; for bf16 2^-15 of p.  One non-zero element per row keeps the logits'
    # own limit far below one rounding of p to fp16.
    case = Case([(shared, own)], hq=h, hkv=h, d=d, dtype=dtype, seed=shared + d)
    case.kc[..., 1:] = 0
    case.q[..., 1:] = 0
    case.kc[..., 0] *= 4
    case.q[..., 0] *= 6
    got = case.run(pkv).double().cpu().numpy()
    q = case.q.double().cpu().numpy()
    for b in range(0, len(own), max(1, len(own) // 8)):
        n = int(case.lens_h[b])
        ids = torch.from_numpy(case.tab_h[b, :-(-n // 16)]).long().cuda()
        for g in range(h):
            k = case.kc[ids, g].reshape(-1, d)[:n].double().cpu().numpy()
            v = case.vc[ids, g].reshape(-1, d)[:n].double().cpu().numpy()
            ref, lim = attn_limits.attend(q[b, g], k, v, case.scale, dtype, p16="bf16")
            lim += 2.0 ** -25 * np.abs(v).sum(0)
            bad = ~(np.abs(got[b, g] - ref) <= lim)
            assert not bad.any(), (b, g, n, got[b, g][bad][:4], ref[bad][:4], lim[bad][:4])
    assert int(case.err.item()) == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("shared,own", [(1024, [0] * 20), (16, [500] * 20), (1024, [200] * 20)])
def test_errors_of_one_query_head_are_the_dense_decodes(pkv, d, shared, own):
    # Over all outputs.  The dense decode's error is the rounding of its outputs, 2^-12.3
    # of them on average; 2^-15 more, in quadrature, is 1.2 %.
    case = Case([(shared, own)], hq=8, hkv=8, d=d, dtype="f16", seed=d)
    out = case.run(pkv)
    dense = torch.empty_like(out)
    ws = torch.empty(pkv.pkv_decode_workspace_bytes(len(own), 8, 8, d, case.width, case.max_ctx), dtype=torch.uint8,
                     device="cuda")
    pkv.pkv_paged_decode_attention(case.q, case.kc, case.vc, case.tab, case.lens, dense, scale=case.scale,
                                   max_context_len=case.max_ctx, workspace=ws, err_flag=case.err)
    torch.cuda.synchronize()
    assert int(case.err.item()) == 0
    exact = torch.empty(out.shape, dtype=torch.float64, device="cuda")
    for b in range(len(own)):
        n = int(case.lens_h[b])
        ids = torch.from_numpy(case.tab_h[b, :-(-n // 16)]).long().cuda()
        k, v = (x[ids].transpose(0, 1).reshape(8, -1, d)[:, :n].double() for x in (case.kc, case.vc))
        w = torch.softmax(torch.einsum("hd,hnd->hn", case.q[b].double(), k) * case.scale, 1)
        exact[b] = torch.einsum("hn,hnd->hd", w, v)
    err, err_dense = ((x.double() - exact).norm().item() for x in (out, dense))
    assert err <= 1.02 * err_dense, (err, err_dense)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("hq,hkv,d", [(2, 1, 128), (8, 2, 64), (8, 1, 128), (3, 3, 128)])
@pytest.mark.parametrize("n", [3, 140])
def test_a_constant_value_is_its_own_mean(pkv, dtype, hq, hkv, d, n):
    # The normaliser sums the weights that are multiplied: 127 equal ones whose
    # rounding to fp16 takes nearly half a step would else move the mean by 2^-11.
    case = Case([(128, [0] * n)], hq=hq, hkv=hkv, d=d, dtype=dtype, seed=5)
    case.kc.zero_()
    case.q.zero_()
    case.q[..., 0] = 1
    case.kc[int(case.tab_h[0, 0]), :, 0, 0] = 1             # the first key's logit is scale, the others' 0
    case.scale = -math.log(0.5 + 0.98 * 2.0 ** -12)
    c = 1 - torch.finfo(case.q.dtype).eps / 2               # the largest value below 1
    case.vc.fill_(c)
    out = case.run(pkv)
    assert int(case.err.item()) == 0
    assert bool((out == c).all()), out.unique()
