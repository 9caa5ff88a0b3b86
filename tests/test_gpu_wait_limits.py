"""The bounded waits of the shared-prefix decode, the block scores and the sparse
decode, made to run out on purpose.

PKV_WAIT_LIMIT_NS shortens the limit of every pipeline wait.  With a nanosecond,
waits give up before their copies land; with a few microseconds, somewhere in the
middle.  The kernels then record PKV_ERR_TIMEOUT, stop, wait (with the full limit)
for their own copies and products in flight and return; the next call in the same
context has the same bits as one before."""
import numpy as np
import pytest
import torch

from tests import gpu_util as gu

pytestmark = pytest.mark.gpu

PKV_ERR_TIMEOUT = 7
LIMITS_NS = [1, 1, 300, 1000, 2000, 4000, 8000, 16000]


@pytest.fixture(scope="module")
def pkv():
    import __graft_entry__ as g
    g.build()
    import paged_kv_cache_153_gb300 as m
    return m


def expire(monkeypatch, call, out, err, ws=None):
    """call() under short limits, then as usual; the first limits have to expire
    (and with ws, whose states of the call before are cleared, to be seen in out)."""
    out.zero_()
    call()
    torch.cuda.synchronize()
    want = out.clone()
    assert int(err.item()) == 0
    for k, limit in enumerate(LIMITS_NS):
        if ws is not None:
            ws.fill_(0xFF)
        monkeypatch.setenv("PKV_WAIT_LIMIT_NS", str(limit))
        call()
        torch.cuda.synchronize()
        monkeypatch.delenv("PKV_WAIT_LIMIT_NS")
        code = int(err.item())
        assert code == PKV_ERR_TIMEOUT if k < 2 else code in (0, PKV_ERR_TIMEOUT), limit
        assert ws is None or k >= 2 or not torch.equal(out, want), limit
        err.zero_()
        out.zero_()
        call()
        torch.cuda.synchronize()
        assert int(err.item()) == 0 and torch.equal(out, want), limit


def pool(seed, nb, hkv, d, dtype):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn((nb, hkv, 16, d), generator=g, device="cuda", dtype=gu.TORCH_16[dtype]) for _ in range(2)], g


# (one row tile of two key streams; two row tiles, several units; several pieces of a range)
@pytest.mark.parametrize("dtype,hq,hkv,d,groups,blocks", [
    ("bf16", 8, 2, 128, [8], 512), ("f16", 8, 2, 128, [100], 256), ("bf16", 4, 4, 64, [200], 300),
    ("f16", 16, 2, 64, [5], 700), ("bf16", 8, 2, 128, [3, 50, 1, 90, 7], 100)])
def test_shared_prefix(pkv, monkeypatch, dtype, hq, hkv, d, groups, blocks):
    # (nothing but the prefixes: the decode beside the prefix kernel has no work and no waits)
    n = sum(groups)
    (kc, vc), g = pool(3, blocks * len(groups), hkv, d, dtype)
    q = torch.randn((n, hq, d), generator=g, device="cuda", dtype=kc.dtype)
    rows = np.concatenate([np.tile(np.arange(blocks) + j * blocks, (m, 1)) for j, m in enumerate(groups)])
    tab = torch.from_numpy(rows.astype(np.int32)).cuda()
    lens = torch.full((n,), 16 * blocks, dtype=torch.int32, device="cuda")
    starts = torch.tensor(np.cumsum([0, *groups]), dtype=torch.int32, device="cuda")
    pre = torch.full((len(groups),), 16 * blocks, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    ws = torch.empty(pkv.pkv_prefix_workspace_bytes(n, len(groups), hq, hkv, d, blocks, 16 * blocks, 16 * blocks),
                     dtype=torch.uint8, device="cuda")
    expire(monkeypatch, lambda: pkv.pkv_paged_decode_attention_prefix(
        q, kc, vc, tab, lens, starts, pre, out, scale=d ** -0.5, max_context_len=16 * blocks,
        max_prefix_len=16 * blocks, workspace=ws, err_flag=err), out, err, ws)


@pytest.mark.parametrize("dtype,hq,hkv,d", [("bf16", 32, 8, 128), ("f16", 8, 8, 64)])
def test_own_blocks_beside_a_prefix(pkv, monkeypatch, dtype, hq, hkv, d):
    # long blocks of their own behind a short prefix
    n, shared, own = 24, 4, 150
    (kc, vc), g = pool(4, shared + n * own, hkv, d, dtype)
    q = torch.randn((n, hq, d), generator=g, device="cuda", dtype=kc.dtype)
    rows = np.stack([np.concatenate([np.arange(shared), shared + b * own + np.arange(own)]) for b in range(n)])
    tab = torch.from_numpy(rows.astype(np.int32)).cuda()
    top = 16 * (shared + own)
    lens = torch.full((n,), top - 3, dtype=torch.int32, device="cuda")
    starts = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    pre = torch.tensor([16 * shared], dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    ws = torch.empty(pkv.pkv_prefix_workspace_bytes(n, 1, hq, hkv, d, shared + own, top, 16 * shared),
                     dtype=torch.uint8, device="cuda")
    expire(monkeypatch, lambda: pkv.pkv_paged_decode_attention_prefix(
        q, kc, vc, tab, lens, starts, pre, out, scale=d ** -0.5, max_context_len=top, max_prefix_len=16 * shared,
        workspace=ws, err_flag=err), out, err)


@pytest.mark.parametrize("dtype,hq,hkv,d", [("bf16", 32, 8, 128), ("f16", 8, 8, 64)])
@pytest.mark.parametrize("n_blocks", [600, 2048])
def test_flat_scores(pkv, monkeypatch, dtype, hq, hkv, d, n_blocks):
    # 64 sequences: the flat form, with few units to a thread block and with many
    n = 64
    g = torch.Generator(device="cuda").manual_seed(5)
    bounds = torch.randn((n_blocks, hkv, 2, d), generator=g, device="cuda", dtype=gu.TORCH_16[dtype])
    q = torch.randn((n, hq, d), generator=g, device="cuda", dtype=bounds.dtype)
    tab = torch.randint(0, n_blocks, (n, n_blocks), generator=g, device="cuda", dtype=torch.int32)
    lens = torch.full((n,), 16 * n_blocks, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.empty((n, hkv, n_blocks), device="cuda")
    expire(monkeypatch, lambda: pkv.pkv_block_scores(q, bounds, tab, lens, out, scale=d ** -0.5,
                                                     max_context_len=16 * n_blocks, err_flag=err), out, err)


@pytest.mark.parametrize("kv,hq,hkv,d", [("bf16", 32, 8, 128), ("f16", 8, 8, 64), ("e4m3", 8, 4, 128),
                                         ("e5m2", 16, 4, 128)])
def test_sparse_decode(pkv, monkeypatch, kv, hq, hkv, d):
    # tensor-core and CUDA-core consumers; every other block of each context listed
    n, blocks, budget = 16, 300, 150
    dtype = kv if kv in gu.TORCH_16 else "bf16"
    (kc, vc), g = pool(6, n * blocks, hkv, d, dtype)
    q = torch.randn((n, hq, d), generator=g, device="cuda", dtype=kc.dtype)
    tab = torch.randperm(n * blocks, generator=g, device="cuda").to(torch.int32).view(n, blocks)
    lens = torch.full((n,), 16 * blocks - 5, dtype=torch.int32, device="cuda")
    lists = (2 * torch.arange(budget, device="cuda", dtype=torch.int32)).expand(n, hkv, budget).contiguous()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    ws = torch.empty(pkv.pkv_decode_workspace_bytes(n, hq, hkv, d, budget, 16 * budget), dtype=torch.uint8,
                     device="cuda")
    kw = dict(scale=d ** -0.5, workspace=ws, err_flag=err)
    if kv in gu.TORCH_16:
        def call():
            pkv.pkv_paged_decode_attention_sparse(q, kc, vc, tab, lens, lists, out, **kw)
    else:
        fmt = torch.float8_e4m3fn if kv == "e4m3" else torch.float8_e5m2
        kc, vc = (x.to(fmt).view(torch.uint8) for x in (kc, vc))
        one = torch.ones(hkv, device="cuda")
        fn = getattr(pkv, "pkv_paged_decode_attention_sparse_" + ("fp8" if kv == "e4m3" else "e5m2"))

        def call():
            fn(q, kc, vc, one, one, tab, lens, lists, out, **kw)
    expire(monkeypatch, call, out, err)
