"""Attention to the first tokens and a window on the GPU against float64: single
tokens over 16-bit and FP8 caches, and prompt chunks."""
import numpy as np
import pytest
import torch

from oracle import draft as od
from tests import attn_limits
from tests import gpu_util as gu
from tests.test_gpu_draft import FP8, Case

pytestmark = pytest.mark.gpu
OOB = 4


@pytest.fixture(scope="module")
def pkv():
    import __graft_entry__ as g
    g.build()
    import paged_kv_cache_153_gb300 as m
    return m


def drop(c, window, sinks, b, first_query):
    """Table entries of blocks that nobody sees become bad ids, rows that nobody
    sees NaN."""
    n = int(c.ctx[b])
    seen = od.window_seen(range(first_query, n), n, window, sinks).any(0)
    nan = 0x7F if c.kv else float("nan")
    for i in range(-(-n // 16)):
        rows = seen[16 * i:16 * i + 16]
        blk = int(c.tab[b, i])
        for off in np.flatnonzero(~rows):
            c.kc_h[blk, :, off], c.vc_h[blk, :, off] = nan, nan
        if not rows.any():
            c.tab[b, i] = 1 << 30


def decode(pkv, c, window, sinks, **over):
    c.upload()
    q = c.q[:len(c.ctx)].contiguous()
    out = torch.full_like(q, 7.0)
    ws = torch.full((pkv.pkv_decode_workspace_bytes(len(c.ctx), c.hq, c.hkv, c.d, c.width, 64),), 0xFF,
                    dtype=torch.uint8, device="cuda")
    kw = dict(scale=c.scale, window=window, num_sinks=sinks, workspace=ws, err_flag=c.err)
    kw.update(over)
    if c.kv:
        call = (pkv.pkv_paged_decode_attention_window_fp8 if c.kv == "e4m3"
                else pkv.pkv_paged_decode_attention_window_e5m2)
        call(q, c.kc, c.vc, c.ks.cuda(), c.vs.cuda(), c.tables, c.lens, out, **kw)
    else:
        pkv.pkv_paged_decode_attention_window(q, c.kc, c.vc, c.tables, c.lens, out, **kw)
    torch.cuda.synchronize()
    return out


def check_rows(c, got, b, positions, rows, window, sinks, tab):
    got = got.double().cpu().numpy()
    n, per = int(c.ctx[b]), c.hq // c.hkv
    seen = od.window_seen(positions, n, window, sinks)
    keep, c.tab = c.tab, tab
    for g in range(c.hkv):
        k, v = c.rows(b, g)
        for i, row in enumerate(rows):
            at = np.flatnonzero(seen[i])
            for h in range(g * per, (g + 1) * per):
                ref, lim = attn_limits.attend(c.q_h[row, h].double().numpy(), k[at], v[at], c.scale, c.dtype,
                                              "f16" if c.kv else None)
                bad = ~(np.abs(got[row, h] - ref) <= lim)
                assert not bad.any(), (b, i, h, float(np.abs(got[row, h] - ref).max()))
    c.tab = keep


LENS = [1, 15, 16, 17, 40, 127, 128, 129, 500, 777]


@pytest.mark.parametrize("dtype,kv", [("f16", None), ("bf16", None), ("bf16", "e4m3"), ("f16", "e5m2")])
@pytest.mark.parametrize("hq,hkv,d", [(2, 2, 64), (2, 2, 128), (8, 2, 64), (16, 2, 128)])
def test_decode_windows(pkv, dtype, kv, hq, hkv, d):
    for window, sinks in ((1, 0), (16, 4), (33, 17), (100, 0), (128, 130), (2000, 3)):
        c = Case([n - 1 for n in LENS], [1] * len(LENS), hq=hq, hkv=hkv, d=d, dtype=dtype, kv=kv, seed=window)
        tab = c.tab.copy()
        for b, n in enumerate(LENS):
            drop(c, window, sinks, b, n - 1)
        out = decode(pkv, c, window, sinks)
        assert int(c.err.item()) == 0, (window, sinks)
        for b, n in enumerate(LENS):
            check_rows(c, out, b, [n - 1], [b], window, sinks, tab)


def test_a_window_of_everything_is_the_dense_decode(pkv):
    c = Case([n - 1 for n in LENS], [1] * len(LENS), hq=8, hkv=2)
    for window, sinks in ((777, 0), (1 << 30, 5), (100, 700), (2 ** 31 - 1, 2 ** 31 - 1)):
        out = decode(pkv, c, window, sinks)
        for b, n in enumerate(LENS):
            check_rows(c, out, b, [n - 1], [b], window, sinks, c.tab)


def test_empty_long_and_broken_contexts(pkv):
    c = Case([30, 30, 30, 30], [1, 1, 1, 1], hq=8, hkv=2)
    c.ctx[1] = 0
    out = decode(pkv, c, 8, 2)
    assert int(c.err.item()) == 0 and not out[1].any()
    check_rows(c, out, 0, [30], [0], 8, 2, c.tab)
    c.ctx[2] = 16 * c.width + 5                                # cut to the table, and reported
    out = decode(pkv, c, 8, 2)
    assert int(c.err.item()) == OOB
    check_rows(c, out, 3, [30], [3], 8, 2, c.tab)
    c.ctx[2] = -4
    assert not decode(pkv, c, 8, 2)[2].any() and int(c.err.item()) == OOB
    c.ctx[2] = 31
    c.tab[2, 0] = -1                                           # the first tokens' block
    decode(pkv, c, 8, 2)
    assert int(c.err.item()) == OOB
    decode(pkv, c, 8, 0)                                       # without them it is not looked at
    assert int(c.err.item()) == 0


def test_many_sequences_take_the_workspace_path(pkv):
    lens = np.random.default_rng(0).integers(1, 200, size=300)
    c = Case(lens - 1, np.ones(300, int), hq=4, hkv=2, d=64)
    out = decode(pkv, c, 40, 4)
    assert int(c.err.item()) == 0
    for b in range(0, 300, 23):
        check_rows(c, out, b, [int(lens[b]) - 1], [b], 40, 4, c.tab)


def test_long_contexts_between_runs_of_blocks(pkv):
    lens = [20000, 5, 4097, 9000]
    c = Case([n - 1 for n in lens], [1] * 4, hq=8, hkv=2, seed=1)
    tab = c.tab.copy()
    for b, n in enumerate(lens):
        drop(c, 4096, 4, b, n - 1)
    out = decode(pkv, c, 4096, 4)
    assert int(c.err.item()) == 0
    for b, n in enumerate(lens):
        check_rows(c, out, b, [n - 1], [b], 4096, 4, tab)


# ---- prompt chunks ----
def prefill(pkv, c, window, sinks, **over):
    c.upload()
    kw = dict(scale=c.scale, max_query_len=int(c.new.max()), window=window, num_sinks=sinks, err_flag=c.err)
    kw.update(over)
    pkv.pkv_paged_prefill_attention_window(c.q, c.kc, c.vc, c.tables, c.lens, c.cu_d, c.out, **kw)
    torch.cuda.synchronize()
    return c.out


def chunk_case(base, new, **kw):
    # (Case's masks are not used; its trees would be too large)
    return Case(base, new, seen=[np.zeros((n, 1), bool) for n in new], **kw)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("hq,hkv,d", [(1, 1, 64), (2, 1, 128), (8, 2, 128), (8, 1, 64)])
def test_chunks(pkv, dtype, hq, hkv, d):
    base, new = [0, 5, 127, 300, 640, 9], [130, 1, 40, 17, 70, 0]
    for window, sinks in ((1, 0), (16, 4), (100, 33), (128, 0), (300, 200), (5000, 3)):
        c = chunk_case(base, new, hq=hq, hkv=hkv, d=d, dtype=dtype, seed=window, extra=3)
        tab = c.tab.copy()
        for b in range(len(base)):
            drop(c, window, sinks, b, base[b])
        out = prefill(pkv, c, window, sinks)
        assert int(c.err.item()) == 0, (window, sinks)
        for b in range(len(base)):
            rows = [i for i in range(new[b]) if i % 5 == 0 or i in (new[b] - 1, 31, 32, 63, 64, 127, 128)]
            check_rows(c, out, b, [base[b] + i for i in rows], [int(c.cu[b]) + i for i in rows], window, sinks, tab)
        assert bool((out[-3:] == 7.0).all())


@pytest.mark.parametrize("dtype,hq,hkv,d", [("bf16", 32, 8, 128), ("f16", 32, 4, 128), ("f16", 32, 16, 64)])
def test_many_rows_share_the_keys_in_pairs_of_tiles(pkv, dtype, hq, hkv, d):
    base, new = [0, 130, 77, 1000], [700, 33, 1, 800]
    for window, sinks in ((100, 4), (1, 0), (600, 200), (5000, 0)):
        c = chunk_case(base, new, hq=hq, hkv=hkv, d=d, dtype=dtype, seed=window, extra=3)
        tab = c.tab.copy()
        for b in range(len(base)):
            drop(c, window, sinks, b, base[b])
        out = prefill(pkv, c, window, sinks)
        assert int(c.err.item()) == 0, (window, sinks)
        for b in range(len(base)):
            rows = [i for i in range(new[b]) if i % 97 == 0 or i in (31, 32, 63, 64, 127, 128, new[b] - 1)]
            check_rows(c, out, b, [base[b] + i for i in rows], [int(c.cu[b]) + i for i in rows], window, sinks, tab)
        assert bool((out[-3:] == 7.0).all())


@pytest.mark.parametrize("dtype,bad", [("bf16", float("nan")), ("f16", float("inf"))])
def test_chunk_rows_that_are_not_seen_change_nothing(pkv, dtype, bad):
    # not finite: a key that leaves the window within the chunk, and one of the chunk's own
    base, n, window, sinks = 200, 90, 64, 2
    c = chunk_case([base], [n], hq=4, hkv=1, d=128, dtype=dtype, seed=2)
    for p in (170, 240):
        c.vc_h[int(c.tab[0, p // 16]), :, p % 16, 5] = bad
    out = prefill(pkv, c, window, sinks)
    assert int(c.err.item()) == 0
    hit = ~torch.isfinite(out[:, :, 5].float()).all(1).cpu().numpy()
    seen = od.window_seen(range(base, base + n), base + n, window, sinks)
    assert (hit == (seen[:, 170] | seen[:, 240])).all()
    got = out.double().cpu().numpy()
    k, v = c.rows(0, 0)
    for i in range(n):
        at = np.flatnonzero(seen[i])
        for h in range(4):
            ref, lim = attn_limits.attend(c.q_h[i, h].double().numpy(), k[at], v[at], c.scale, dtype)
            cols = np.arange(128) != 5 if hit[i] else slice(None)
            assert (np.abs(got[i, h] - ref)[cols] <= lim[cols]).all(), (i, h)


def test_a_chunk_agrees_with_the_decode_of_its_last_token(pkv):
    c = chunk_case([300, 77], [33, 129], hq=16, hkv=2, dtype="bf16", seed=4)
    out = prefill(pkv, c, 100, 4)
    last = [int(x) - 1 for x in c.cu[1:]]
    q = c.q[last].contiguous()
    dec = torch.empty_like(q)
    ws = torch.empty(pkv.pkv_decode_workspace_bytes(2, 16, 2, 128, c.width, 104), dtype=torch.uint8, device="cuda")
    pkv.pkv_paged_decode_attention_window(q, c.kc, c.vc, c.tables, c.lens, dec, scale=c.scale, window=100, num_sinks=4,
                                          workspace=ws)
    # (a rounding of each output to bf16, half a step of 2^-8 each, and their sums' last bits)
    assert bool(((out[last].float() - dec.float()).abs() <= 2.0 ** -7 * dec.float().abs() + 1e-4).all())


def test_broken_chunks_are_skipped_and_flagged(pkv):
    for kind in ("ctx", "table", "query"):
        c = chunk_case([40, 40, 40], [5, 60, 7], hq=8, hkv=2)
        over = {}
        if kind == "ctx":
            c.ctx[1] = 59
        elif kind == "table":
            c.ctx[1] = 16 * c.width + 1
        else:
            over["max_query_len"] = 50
        out = prefill(pkv, c, 30, 2, **over)
        assert int(c.err.item()) == OOB and bool((out[5:65] == 7.0).all()), kind
        check_rows(c, out, 0, range(40, 45), range(5), 30, 2, c.tab)
        check_rows(c, out, 2, range(40, 47), range(65, 72), 30, 2, c.tab)
    c = chunk_case([40], [5], hq=8, hkv=2)
    c.cu = np.array([0, 9], np.int32)
    prefill(pkv, c, 30, 2)
    assert int(c.err.item()) == OOB
    c = chunk_case([40], [20], hq=8, hkv=2)
    c.tab[0, 2] = c.nb
    prefill(pkv, c, 30, 2)
    assert int(c.err.item()) == OOB


def test_chunks_captured_and_replayed(pkv):
    c = chunk_case([200], [150], hq=8, hkv=2, seed=3)
    want = prefill(pkv, c, 90, 4).clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pkv.pkv_paged_prefill_attention_window(c.q, c.kc, c.vc, c.tables, c.lens, c.cu_d, c.out, scale=c.scale,
                                               max_query_len=150, window=90, num_sinks=4, err_flag=c.err)
    for _ in range(3):
        c.out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(c.out, want)


def test_not_finite_rows_in_pairs_of_tiles(pkv):
    # as above with row tiles in pairs: the same rows behind many others
    base, n, window, sinks = 200, 90, 64, 2
    c = chunk_case([0, base], [1400, n], hq=32, hkv=8, d=128, dtype="bf16", seed=2)
    for p in (170, 240):
        c.vc_h[int(c.tab[1, p // 16]), :, p % 16, 5] = float("inf")
    out = prefill(pkv, c, window, sinks)
    assert int(c.err.item()) == 0
    assert bool(torch.isfinite(out[:1400].float()).all())
    got = out[1400:].double().cpu().numpy()
    seen = od.window_seen(range(base, base + n), base + n, window, sinks)
    assert (np.isfinite(got[:, :, 5]) == ~(seen[:, 170] | seen[:, 240])[:, None]).all()
    for h in (0, 5, 31):
        k, v = c.rows(1, h // 4)
        for i in range(0, n, 3):
            at = np.flatnonzero(seen[i])
            ref, lim = attn_limits.attend(c.q_h[1400 + i, h].double().numpy(), k[at], v[at], c.scale, "bf16")
            cols = np.arange(128) != 5
            assert (np.abs(got[i, h] - ref)[cols] <= lim[cols]).all(), (i, h)


def test_the_largest_windows_and_first_tokens(pkv):
    most = 2 ** 31 - 1
    c = Case([300, 17, 0], [1, 1, 1], hq=8, hkv=2, d=64, seed=6)
    want = decode(pkv, c, 400, 0).clone()
    for window, sinks in ((most, 0), (most, most), (1, most), (400, 400)):
        assert torch.equal(decode(pkv, c, window, sinks), want), (window, sinks)
    c = chunk_case([300, 17], [40, 130], hq=8, hkv=2, d=64, seed=6)
    want = prefill(pkv, c, 400, 0).clone()
    for window, sinks in ((most, 0), (most, most), (1, most), (400, 400)):
        assert torch.equal(prefill(pkv, c, window, sinks), want), (window, sinks)
    assert int(c.err.item()) == 0
