"""16-bit data in tensors of another two-byte type, its kind given as dtype: the
same bits as from tensors of the type itself."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    import __graft_entry__ as g
    g.build()
    import paged_kv_cache_153_gb300 as m
    return m


@pytest.mark.parametrize("storage", [torch.int16, torch.uint16])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_storage_types(pkv, dtype, storage):
    n, hq, hkv, d, blocks = 5, 8, 2, 64, 6
    g = torch.Generator(device="cuda").manual_seed(1)

    def rand(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(dtype)
    q, kc, vc = rand(n, hq, d), rand(n * blocks, hkv, 16, d), rand(n * blocks, hkv, 16, d)
    new = rand(n, hkv, d)
    tab = torch.arange(n * blocks, device="cuda", dtype=torch.int32).view(n, blocks)
    lens = torch.full((n,), 16 * blocks - 3, dtype=torch.int32, device="cuda")
    pos = lens - 1
    slots = (tab[:, -1].long() * 16 + pos % 16)
    lists = torch.tensor([0, 2, 5], dtype=torch.int32, device="cuda").expand(n, hkv, 3).contiguous()
    starts, pre = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, n], [0]))
    turns, _ = pkv.pkv_rope_plan(d)
    turns = torch.from_numpy(turns).cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run(cast, tag):
        qt, kt, vt, nt = (cast(x.clone()) for x in (q, kc, vc, new))
        out, turned = (cast(torch.zeros_like(q)) for _ in range(2))
        bounds = cast(torch.zeros((n * blocks, hkv, 2, d), dtype=dtype, device="cuda"))
        scores = torch.zeros((n, hkv, blocks), device="cuda")
        kw = dict(dtype=tag, err_flag=err)
        results = []
        pkv.pkv_rope_append(qt, nt, nt, pos, slots, turns, turned, kt, vt, **kw)
        pkv.pkv_kv_block_bounds(kt, tab, lens, bounds, max_new_len=16 * blocks, **kw)
        pkv.pkv_block_scores(turned, bounds, tab, lens, scores, scale=0.125, max_context_len=16 * blocks, **kw)
        ws = torch.empty(pkv.pkv_decode_workspace_bytes(n, hq, hkv, d, 3, 48), dtype=torch.uint8, device="cuda")
        pkv.pkv_paged_decode_attention_sparse(turned, kt, vt, tab, lens, lists, out, scale=0.125, workspace=ws, **kw)
        results += [x.view(dtype).clone() for x in (turned, kt, vt, bounds, out)] + [scores]
        ws = torch.empty(pkv.pkv_prefix_workspace_bytes(n, 1, hq, hkv, d, blocks, 16 * blocks, 0), dtype=torch.uint8,
                         device="cuda")
        pkv.pkv_paged_decode_attention_prefix(turned, kt, vt, tab, lens, starts, pre, out, scale=0.125,
                                              max_context_len=16 * blocks, max_prefix_len=0, workspace=ws, **kw)
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        return results + [out.view(dtype).clone()]

    want = run(lambda x: x, None)
    got = run(lambda x: x.view(storage), pkv.PKV_F16 if dtype == torch.float16 else pkv.PKV_BF16)
    assert all(torch.equal(a, b) and bool(a.isfinite().all()) for a, b in zip(want, got))
