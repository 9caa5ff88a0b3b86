"""Windows and drafted tokens at the end of 32-bit positions: contexts of 2^31 - 17 to
2^31 - 1 tokens, whose last block ends at 2^31."""
import numpy as np
import pytest
import torch

from oracle import draft as od
from tests import attn_limits

pytestmark = pytest.mark.gpu

WIDTH = 1 << 27


@pytest.fixture(scope="module")
def pkv():
    import __graft_entry__ as g
    g.build()
    import paged_kv_cache_153_gb300 as m
    return m


@pytest.fixture(scope="module")
def table():
    return torch.full((1, WIDTH), 1 << 30, dtype=torch.int32, device="cuda")


HQ, HKV, D, NB = 8, 2, 64, 40


def caches(dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn((NB, HKV, 16, D), generator=g).to(dtype) for _ in range(2)], g


def check(out, q, kc, vc, tab, row, pos, n, window, sinks, dtype):
    # only the first and the last tokens are in the table
    seen = np.concatenate([np.arange(min(sinks, pos + 1)), np.arange(max(sinks, pos + 1 - window), pos + 1)])
    ids, off = tab[torch.from_numpy(seen // 16)].long(), torch.from_numpy(seen % 16)
    for h in range(HQ):
        k, v = (x[ids, h // (HQ // HKV), off].double().numpy() for x in (kc, vc))
        ref, lim = attn_limits.attend(q[row, h].double().numpy(), k, v, D ** -0.5, dtype)
        assert (np.abs(out[row, h].double().cpu().numpy() - ref) <= lim).all(), (n, pos, h)


@pytest.mark.parametrize("n", [2 ** 31 - 1, 2 ** 31 - 15, 2 ** 31 - 16, 2 ** 31 - 17])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("window,sinks", [(100, 20), (1, 0), (160, 300)])
def test_windows(pkv, table, n, dtype, window, sinks):
    t = {"f16": torch.float16, "bf16": torch.bfloat16}[dtype]
    (kc, vc), g = caches(t, 1)
    last = -(-n // 16)
    ids = torch.randperm(NB, generator=g)[:36].to(torch.int32)
    table.fill_(1 << 30)
    table[0, :20] = ids[:20].cuda()
    table[0, last - 16:last] = ids[20:].cuda()
    tab = _Sparse(ids, last)
    new = 20
    q = torch.randn((new, HQ, D), generator=g).to(t)
    lens, err = torch.tensor([n], dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    # (what is not seen changes nothing: a NaN behind the context)
    if n % 16:
        for x in (kc, vc):
            x[int(ids[35]), :, n % 16:] = float("nan")
    out = torch.zeros((1, HQ, D), dtype=t, device="cuda")
    ws = torch.empty(pkv.pkv_decode_workspace_bytes(1, HQ, HKV, D, WIDTH, 64), dtype=torch.uint8, device="cuda")
    kw = dict(scale=D ** -0.5, window=window, num_sinks=sinks, err_flag=err)
    pkv.pkv_paged_decode_attention_window(q[:1].cuda(), kc.cuda(), vc.cuda(), table, lens, out, workspace=ws, **kw)
    assert int(err.item()) == 0
    check(out, q, kc, vc, tab, 0, n - 1, n, window, sinks, dtype)
    out = torch.zeros((new, HQ, D), dtype=t, device="cuda")
    cu = torch.tensor([0, new], dtype=torch.int32, device="cuda")
    pkv.pkv_paged_prefill_attention_window(q.cuda(), kc.cuda(), vc.cuda(), table, lens, cu, out, max_query_len=new,
                                           **kw)
    assert int(err.item()) == 0
    for i in range(new):
        check(out, q, kc, vc, tab, i, n - new + i, n, window, sinks, dtype)


class _Sparse:
    """The table's entries that exist: the first 20 blocks and the last 16."""

    def __init__(self, ids, last):
        self.ids, self.last = ids, last

    def __getitem__(self, blk):
        return self.ids[torch.where(blk < 20, blk, blk - self.last + 36)]


@pytest.mark.parametrize("kv", [None, "e4m3"])
def test_drafted_tokens(pkv, table, kv):
    """Context keys of 0 with values of 1; drafted token j has a logit of 30 + 10 j nats and
    a value of 2 + j, so that a token's output is its most preferred visible one's."""
    n, nb, d = 2 ** 31 - 1, 20000, 64
    torch.arange(WIDTH, out=table[0])
    table.remainder_(nb)
    table[0, -1] = nb
    kc, vc = torch.zeros((nb + 1, 1, 16, d), device="cuda"), torch.ones((nb + 1, 1, 16, d), device="cuda")
    for j in range(3):
        kc[nb, 0, 12 + j] = (30 + 10 * j) / 8
        vc[nb, 0, 12 + j] = 2 + j
    scales = []
    if kv:
        scales = [torch.ones(1, device="cuda")] * 2
        kc, vc = (x.to(torch.float8_e4m3fn).view(torch.uint8) for x in (kc, vc))
        kc[nb, 0, 15], vc[nb, 0, 15] = 0x7F, 0x7F
    else:
        kc, vc = kc.half(), vc.half()
        kc[nb, 0, 15], vc[nb, 0, 15] = float("nan"), float("nan")
    seen = np.array([[1, 0, 0], [0, 1, 0], [1, 0, 1]], bool)
    mask = torch.from_numpy(od.mask_words(seen, 1)).cuda()
    i32 = dict(dtype=torch.int32, device="cuda")
    q = torch.ones((3, 1, d), dtype=torch.float16, device="cuda")
    out, err = torch.zeros_like(q), torch.zeros(1, **i32)
    ws = torch.empty(pkv.pkv_tree_workspace_bytes(1, 3, 1, 1, d, 3), dtype=torch.uint8, device="cuda")
    getattr(pkv, "pkv_paged_tree_attention" + ("_fp8" if kv else ""))(
        q, kc, vc, *scales, table, torch.tensor([n], **i32), torch.tensor([0, 3], **i32), mask, out, scale=0.125,
        max_context_len=n, max_nodes=3, workspace=ws, err_flag=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    keys = kc[nb, 0, 12:15, 0].contiguous()
    logit = 8 * (keys.view(torch.float8_e4m3fn) if kv else keys).double().cpu()
    for i, (top, value) in enumerate([(logit[0], 2.0), (logit[1], 3.0), (logit[2], 4.0)]):
        rest = (n - 3) * torch.exp(-top) + (torch.exp(logit[0] - top) if i == 2 else 0)
        low = 1.0 if i != 2 else 2.0                           # (token 2 sees token 0 as well)
        want = value - rest * (value - low)                    # to first order, rest < 2e-3
        # fp16's step at 2 to 4, twice (weights and output), and the second order
        assert float((out[i].double().cpu() - want).abs().max()) <= 2 * 2.0 ** -9 + 4 * float(rest) ** 2, i
