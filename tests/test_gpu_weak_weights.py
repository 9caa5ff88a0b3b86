"""Attention whose weights span many orders of magnitude: one strongly preferred key
over a long context, whose own V is 0, so that the output is what the others leave.

Weights rounded to fp16 have a smallest step, 2^-24.  The kernels multiply them by a
power of two first (below 2^16, fp16's largest), so a weight of w times the row's
largest is rounded to 2^-11 of itself at most (half of that to nearest) or, where it is
small, to half a step: 2^-25 / 2^7 = 2^-32 of the largest for drafted tokens and chunks
(their reference may lie 2^8 below the largest weight), 2^-25 / 2^15 = 2^-40 for single
tokens.  n such errors, times |V|, join the limits of attn_limits."""
import numpy as np
import pytest
import torch

from oracle import draft as od
from tests import attn_limits
from tests.test_gpu_draft import FP8, Case
from tests.test_gpu_window import decode, prefill

pytestmark = pytest.mark.gpu

GAPS = [15.0, 16.0, 17.0, 18.0]          # nats between the preferred key and the others


@pytest.fixture(scope="module")
def pkv():
    import __graft_entry__ as g
    g.build()
    import paged_kv_cache_153_gb300 as m
    return m


def preferred(base, new, at, *, spread=0.3, **kw):
    """A case whose sequence b prefers the key at position at[b]; the other logits have
    a standard deviation of `spread`."""
    masks = [np.eye(n, dtype=bool) for n in new]
    c = Case(base, new, seen=masks, **kw)
    g = torch.Generator().manual_seed(99)
    sign = torch.where(torch.rand((len(base), c.d), generator=g) < 0.5, -1.0, 1.0)
    for b in range(len(base)):
        c.q_h[int(c.cu[b]):int(c.cu[b + 1])] = sign[b].to(c.q_h.dtype)
        p = np.arange(int(c.ctx[b]))
        ids, off = torch.from_numpy(c.tab[b][p // 16].astype(np.int64)), torch.from_numpy(p % 16)
        ks = c.ks if c.kv else torch.ones(c.hkv)
        vs = c.vs if c.kv else torch.ones(c.hkv)
        # scale <q, k> = d^-1/2 <sign, k>: normal elements of deviation s give logits of deviation s
        k = torch.randn((len(p), c.hkv, c.d), generator=g) * spread / ks[:, None]
        v = (1 + 0.25 * torch.rand((len(p), c.hkv, c.d), generator=g)) / vs[:, None]
        k[at[b]] = GAPS[b % len(GAPS)] * c.d ** -0.5 * sign[b] / ks[:, None]
        v[at[b]] = 0
        for dst, x in ((c.kc_h, k), (c.vc_h, v)):
            dst[ids, :, off] = x.to(FP8[c.kv]).view(torch.uint8) if c.kv else x.to(dst.dtype)
    return c


def check(c, got, b, row, seen, floor):
    got = got.double().cpu().numpy()
    per, at = c.hq // c.hkv, np.flatnonzero(seen)
    for g in range(c.hkv):
        k, v = (x[at] for x in c.rows(b, g))
        for h in range(g * per, (g + 1) * per):
            ref, lim = attn_limits.attend(c.q_h[row, h].double().numpy(), k, v, c.scale, c.dtype,
                                          "f16" if c.kv else None)
            lim = lim + len(at) * floor * np.abs(v).max()
            assert (np.abs(got[row, h] - ref) <= lim).all(), (b, h, float((np.abs(got[row, h] - ref) / ref).max()))


@pytest.mark.parametrize("dtype,kv", [("f16", None), ("bf16", None), ("f16", "e4m3"), ("bf16", "e5m2")])
@pytest.mark.parametrize("hq,d", [(8, 64), (4, 128)])
def test_drafted_tokens(pkv, dtype, kv, hq, d):
    # the last cached key, which is met first; 160 units, most of a context in one thread block
    n = 40
    base = [3000 + 17 * b for b in range(n)]
    c = preferred(base, [1] * n, [x - 1 for x in base], hq=hq, hkv=4, d=d, dtype=dtype, kv=kv, seed=1)
    out = c.attend(pkv)
    assert int(c.err.item()) == 0
    for b in range(0, n, 3):
        check(c, out, b, b, np.ones(base[b] + 1, bool), 2.0 ** -32)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("hq,hkv,new", [(2, 2, 3), (8, 2, 40)])
def test_prompt_chunks(pkv, dtype, hq, hkv, new):
    base = [4000, 2500, 3300, 2900]
    c = preferred(base, [new] * 4, [x - 1 for x in base], hq=hq, hkv=hkv, d=64, dtype=dtype, seed=2)
    out = prefill(pkv, c, 3500, 4)
    assert int(c.err.item()) == 0
    for b in range(4):
        for i in (0, new - 1):
            check(c, out, b, int(c.cu[b]) + i, od.window_seen([base[b] + i], base[b] + new, 3500, 4)[0], 2.0 ** -32)


def dense(pkv, c):
    c.upload()
    q = c.q[:len(c.ctx)].contiguous()
    out = torch.full_like(q, 7.0)
    ws = torch.full((pkv.pkv_decode_workspace_bytes(len(c.ctx), c.hq, c.hkv, c.d, c.width, int(c.ctx.max())),), 0xFF,
                    dtype=torch.uint8, device="cuda")
    kw = dict(scale=c.scale, max_context_len=int(c.ctx.max()), workspace=ws, err_flag=c.err)
    if c.kv:
        call = pkv.pkv_paged_decode_attention_fp8 if c.kv == "e4m3" else pkv.pkv_paged_decode_attention_e5m2
        call(q, c.kc, c.vc, c.ks.cuda(), c.vs.cuda(), c.tables, c.lens, out, **kw)
    else:
        pkv.pkv_paged_decode_attention(q, c.kc, c.vc, c.tables, c.lens, out, **kw)
    torch.cuda.synchronize()
    return out


@pytest.mark.parametrize("dtype,kv", [("f16", None), ("bf16", None), ("f16", "e4m3"), ("bf16", "e5m2")])
@pytest.mark.parametrize("hq,hkv,d", [(8, 4, 64), (16, 4, 128), (32, 4, 128), (4, 4, 64)])
def test_single_tokens(pkv, dtype, kv, hq, hkv, d):
    # the first token, as many models prefer it
    n = 40
    base = [3000 + 17 * b for b in range(n)]
    c = preferred(base, [1] * n, [0] * n, hq=hq, hkv=hkv, d=d, dtype=dtype, kv=kv, seed=3)
    outs = {0: dense(pkv, c), 4096: decode(pkv, c, 4096, 4), 1500: decode(pkv, c, 1500, 4)}
    assert int(c.err.item()) == 0
    for window, out in outs.items():
        for b in range(0, n, 3):
            seen = od.window_seen([base[b]], base[b] + 1, window, 4)[0] if window else np.ones(base[b] + 1, bool)
            check(c, out, b, b, seen, 2.0 ** -40)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("hq", [2, 8])
@pytest.mark.parametrize("where", ["first", "middle", "last"])
def test_prefill(pkv, dtype, hq, where):
    base, new = [4000, 2500, 3300, 2900], 40
    at = [{"first": 0, "middle": x // 2, "last": x - 1}[where] for x in base]
    c = preferred(base, [new] * 4, at, hq=hq, hkv=2, d=128, dtype=dtype, seed=2).upload()
    pkv.pkv_paged_prefill_attention(c.q, c.kc, c.vc, c.tables, c.lens, c.cu_d, c.out, scale=c.scale, max_query_len=new,
                                    err_flag=c.err)
    torch.cuda.synchronize()
    assert int(c.err.item()) == 0
    for b in range(4):
        for i in (0, new - 1):
            check(c, c.out, b, int(c.cu[b]) + i, np.arange(base[b] + new) <= base[b] + i, 2.0 ** -32)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("hq", [16, 4])
@pytest.mark.parametrize("members,where", [(5, "first"), (5, "last"), (100, "first"), (100, "last")])
def test_shared_prefixes(pkv, dtype, hq, members, where):
    # 40 groups x 4 KV heads: a thread block takes most of a prefix.  One and two row tiles.
    groups, hkv, n = 40, 4, 2992
    c = preferred([n - 1] * groups, [1] * groups, [{"first": 0, "last": n - 1}[where]] * groups, hq=hq, hkv=hkv, d=64,
                  dtype=dtype, seed=4).upload()
    rows = torch.arange(groups, device="cuda").repeat_interleave(members)
    q, tab, lens = c.q[rows].contiguous(), c.tables[rows].contiguous(), c.lens[rows].contiguous()
    starts = torch.arange(0, members * groups + 1, members, dtype=torch.int32, device="cuda")
    pre = torch.full((groups,), n, dtype=torch.int32, device="cuda")
    out = torch.full_like(q, 7.0)
    ws = torch.full((pkv.pkv_prefix_workspace_bytes(len(rows), groups, hq, hkv, 64, c.width, n, n),), 0xFF,
                    dtype=torch.uint8, device="cuda")
    pkv.pkv_paged_decode_attention_prefix(q, c.kc, c.vc, tab, lens, starts, pre, out, scale=c.scale, max_context_len=n,
                                          max_prefix_len=n, workspace=ws, err_flag=c.err)
    torch.cuda.synchronize()
    assert int(c.err.item()) == 0
    for b in range(0, groups, 3):
        for i in (0, members - 1):
            check(c, out.view(groups, members, hq, 64)[:, i], b, b, np.ones(n, bool), 2.0 ** -32)
