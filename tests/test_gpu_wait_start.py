"""The limit of a pipeline wait counts from the end of the previous kernel on the
stream, not from an early launch beside it."""
import pytest
import torch

from tests import gpu_util as gu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    import __graft_entry__ as g
    g.build()
    import paged_kv_cache_153_gb300 as m
    return m


@pytest.fixture(scope="module")
def slow(pkv):
    """A call that releases the next launch at its start and then runs for
    milliseconds: the choice among 2^24 blocks by one thread block."""
    n = 1 << 24
    scores = torch.randn((1, 1, n), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    lens = torch.tensor([16 * n], dtype=torch.int32, device="cuda")
    lists = torch.empty((1, 1, 4000), dtype=torch.int32, device="cuda")

    def call():
        pkv.pkv_select_blocks(scores, lens, lists)
    call()
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    call()
    end.record()
    torch.cuda.synchronize()
    assert start.elapsed_time(end) > 2.0            # ms
    return call


LIMIT_NS = 400000       # far above a wait of these small calls, far below the slow one


def check(monkeypatch, slow, call, out, err):
    out.zero_()
    call()
    torch.cuda.synchronize()
    want = out.clone()
    assert int(err.item()) == 0
    for _ in range(3):
        out.zero_()
        monkeypatch.setenv("PKV_WAIT_LIMIT_NS", str(LIMIT_NS))
        slow()
        call()
        torch.cuda.synchronize()
        monkeypatch.delenv("PKV_WAIT_LIMIT_NS")
        assert int(err.item()) == 0 and torch.equal(out, want)


@pytest.mark.parametrize("dtype,hq,hkv,d,n", [("bf16", 8, 2, 128, 8), ("f16", 8, 8, 64, 150)])
def test_shared_prefix(pkv, slow, monkeypatch, dtype, hq, hkv, d, n):
    blocks, own = 64, 3
    g = torch.Generator(device="cuda").manual_seed(2)
    kc, vc = (torch.randn((blocks + n * own, hkv, 16, d), generator=g, device="cuda", dtype=gu.TORCH_16[dtype])
              for _ in range(2))
    q = torch.randn((n, hq, d), generator=g, device="cuda", dtype=kc.dtype)
    tab = torch.empty((n, blocks + own), dtype=torch.int32, device="cuda")
    tab[:, :blocks] = torch.arange(blocks, device="cuda")
    tab[:, blocks:] = blocks + torch.arange(n * own, device="cuda").view(n, own)
    top = 16 * (blocks + own)
    lens = torch.full((n,), top, dtype=torch.int32, device="cuda")
    starts = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    pre = torch.tensor([16 * blocks], dtype=torch.int32, device="cuda")
    err, out = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.empty_like(q)
    ws = torch.empty(pkv.pkv_prefix_workspace_bytes(n, 1, hq, hkv, d, blocks + own, top, 16 * blocks),
                     dtype=torch.uint8, device="cuda")
    check(monkeypatch, slow, lambda: pkv.pkv_paged_decode_attention_prefix(
        q, kc, vc, tab, lens, starts, pre, out, scale=d ** -0.5, max_context_len=top, max_prefix_len=16 * blocks,
        workspace=ws, err_flag=err), out, err)


@pytest.mark.parametrize("kv,hq,hkv,d", [("f16", 4, 4, 128), ("bf16", 2, 2, 64), ("e4m3", 8, 4, 64), ("e5m2", 3, 3, 128),
                                         ("bf16", 16, 4, 128)])
def test_sparse_decode(pkv, slow, monkeypatch, kv, hq, hkv, d):
    # CUDA-core consumers (one query head per KV head, or FP8 rows of 64 bytes), and a tensor-core one
    n, blocks, budget = 3, 40, 20
    dtype = gu.TORCH_16.get(kv, torch.bfloat16)
    g = torch.Generator(device="cuda").manual_seed(3)
    kc, vc = (torch.randn((n * blocks, hkv, 16, d), generator=g, device="cuda", dtype=dtype) for _ in range(2))
    q = torch.randn((n, hq, d), generator=g, device="cuda", dtype=dtype)
    tab = torch.arange(n * blocks, device="cuda", dtype=torch.int32).view(n, blocks)
    lens = torch.full((n,), 16 * blocks, dtype=torch.int32, device="cuda")
    lists = (2 * torch.arange(budget, device="cuda", dtype=torch.int32)).expand(n, hkv, budget).contiguous()
    err, out = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.empty_like(q)
    ws = torch.empty(pkv.pkv_decode_workspace_bytes(n, hq, hkv, d, budget, 16 * budget), dtype=torch.uint8,
                     device="cuda")
    kw = dict(scale=d ** -0.5, workspace=ws, err_flag=err)
    if kv in gu.TORCH_16:
        def call():
            pkv.pkv_paged_decode_attention_sparse(q, kc, vc, tab, lens, lists, out, **kw)
    else:
        fmt = torch.float8_e4m3fn if kv == "e4m3" else torch.float8_e5m2
        k8, v8 = (x.to(fmt).view(torch.uint8) for x in (kc, vc))
        one = torch.ones(hkv, device="cuda")
        fn = getattr(pkv, "pkv_paged_decode_attention_sparse_" + ("fp8" if kv == "e4m3" else "e5m2"))

        def call():
            fn(q, k8, v8, one, one, tab, lens, lists, out, **kw)
    check(monkeypatch, slow, call, out, err)


def test_flat_scores(pkv, slow, monkeypatch):
    n, hkv, d, n_blocks = 64, 8, 128, 600
    g = torch.Generator(device="cuda").manual_seed(4)
    bounds = torch.randn((n_blocks, hkv, 2, d), generator=g, device="cuda", dtype=torch.bfloat16)
    q = torch.randn((n, 4 * hkv, d), generator=g, device="cuda", dtype=torch.bfloat16)
    tab = torch.randint(0, n_blocks, (n, n_blocks), generator=g, device="cuda", dtype=torch.int32)
    lens = torch.full((n,), 16 * n_blocks, dtype=torch.int32, device="cuda")
    err, out = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.empty((n, hkv, n_blocks), device="cuda")
    check(monkeypatch, slow, lambda: pkv.pkv_block_scores(q, bounds, tab, lens, out, scale=d ** -0.5,
                                                          max_context_len=16 * n_blocks, err_flag=err), out, err)
