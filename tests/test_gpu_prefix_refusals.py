"""Refusals of the shared-prefix decode come before its first launch."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    import __graft_entry__ as g
    g.build()
    import paged_kv_cache_153_gb300 as m
    return m


def call(pkv, batch, hq, hkv, d):
    """batch sequences of one shared block and one token: (status, workspace, out, err)."""
    dev = "cuda"
    kc = torch.ones((2, hkv, 16, d), dtype=torch.bfloat16, device=dev)
    q = torch.ones((batch, hq, d), dtype=torch.bfloat16, device=dev)
    tab = torch.tensor([[0, 1]], dtype=torch.int32, device=dev).repeat(batch, 1)
    lens = torch.full((batch,), 17, dtype=torch.int32, device=dev)
    starts = torch.tensor([0, batch], dtype=torch.int32, device=dev)
    pre = torch.tensor([16], dtype=torch.int32, device=dev)
    out = torch.full_like(q, 7.0)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    ws = torch.full((pkv.pkv_prefix_workspace_bytes(batch, 1, hq, hkv, d, 2, 17, 16),), 0xA5, dtype=torch.uint8,
                    device=dev)
    torch.cuda.synchronize()
    status = 0
    try:
        pkv.pkv_paged_decode_attention_prefix(q, kc, kc, tab, lens, starts, pre, out, scale=1.0, max_context_len=17,
                                              max_prefix_len=16, workspace=ws, err_flag=err)
    except pkv.PkvError as e:
        status = e.status
    torch.cuda.synchronize()
    return status, ws, out, int(err.item())


@pytest.mark.parametrize("hq,hkv,d", [(1, 1, 64), (8, 1, 128)])
def test_a_batch_that_does_not_fit_launches_nothing(pkv, hq, hkv, d):
    status, ws, out, err = call(pkv, 20000, hq, hkv, d)
    assert status == 2 and err == 0
    assert bool((ws == 0xA5).all()) and bool((out == 7.0).all())


@pytest.mark.parametrize("hq,hkv,d", [(1, 1, 64), (8, 1, 128), (8, 8, 128)])
def test_ten_thousand_sequences_fit(pkv, hq, hkv, d):
    # (every value row is ones, and so is every output)
    status, _, out, err = call(pkv, 10000, hq, hkv, d)
    assert status == 0 and err == 0
    assert bool((out == 1.0).all())
