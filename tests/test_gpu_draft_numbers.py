"""Numbers of the drafted tokens' attention that plain random inputs do not reach."""
import numpy as np
import pytest
import torch

from tests.test_gpu_draft import Case

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
