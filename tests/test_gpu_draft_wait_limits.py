"""The bounded waits of the drafted tokens' attention and of the windowed prompt chunks,
made to run out on purpose, and where their limit counts from.

With short limits the kernel's warps give up somewhere in the pipeline, record
PKV_ERR_TIMEOUT, tell the others, wait (with the full limit) for their own copies and
products in flight and return; the next call has the same bits as one before."""
import pytest
import torch

from tests.test_gpu_draft import Case
from tests.test_gpu_wait_limits import expire
from tests.test_gpu_wait_start import check, slow   # noqa: F401  (slow: a fixture)
from tests.test_gpu_window import chunk_case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    import __graft_entry__ as g
    g.build()
    import paged_kv_cache_153_gb300 as m
    return m


def tree_call(pkv, c):
    c.upload()
    ws = torch.empty(pkv.pkv_tree_workspace_bytes(len(c.ctx), c.tokens, c.hq, c.hkv, c.d, c.max_nodes),
                     dtype=torch.uint8, device="cuda")
    scales = [x.cuda() for x in (c.ks, c.vs)] if c.kv else []
    fn = getattr(pkv, "pkv_paged_tree_attention" + {None: "", "e4m3": "_fp8", "e5m2": "_e5m2"}[c.kv])
    kw = dict(scale=c.scale, max_context_len=int(c.ctx.max()), max_nodes=c.max_nodes, workspace=ws, err_flag=c.err)
    return lambda: fn(c.q, c.kc, c.vc, *scales, c.tables, c.lens, c.cu_d, c.mask, c.out, **kw), ws


def chunk_call(pkv, c, window, sinks):
    c.upload()
    kw = dict(scale=c.scale, max_query_len=int(c.new.max()), window=window, num_sinks=sinks, err_flag=c.err)
    return lambda: pkv.pkv_paged_prefill_attention_window(c.q, c.kc, c.vc, c.tables, c.lens, c.cu_d, c.out, **kw)


# (one row tile, two, several units of two; several pieces of a thread block, and units that none holds alone)
@pytest.mark.parametrize("dtype,kv", [("bf16", None), ("f16", None), ("bf16", "e4m3"), ("f16", "e5m2")])
@pytest.mark.parametrize("hq,hkv,d,base,new", [(8, 2, 128, [9000], [9]), (8, 2, 64, [5000, 3000], [60, 50]),
                                               (16, 2, 128, [2000, 700, 1200, 3000], [100, 3, 16, 40]),
                                               (2, 2, 128, [6000, 400], [7, 150]),
                                               (8, 8, 64, [700 + 90 * b for b in range(40)], [5] * 40)])
def test_drafted_tokens(pkv, monkeypatch, dtype, kv, hq, hkv, d, base, new):
    c = Case(base, new, hq=hq, hkv=hkv, d=d, dtype=dtype, kv=kv, seed=1)
    call, ws = tree_call(pkv, c)
    expire(monkeypatch, call, c.out, c.err, ws)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("hq,hkv,d,base,new", [(8, 2, 128, [6000], [40]), (8, 1, 64, [3000, 4000], [300, 20]),
                                               (32, 8, 128, [2000, 5000], [600, 800])])
def test_prompt_chunks(pkv, monkeypatch, dtype, hq, hkv, d, base, new):
    c = chunk_case(base, new, hq=hq, hkv=hkv, d=d, dtype=dtype, seed=1)
    expire(monkeypatch, chunk_call(pkv, c, 4096, 4), c.out, c.err)


@pytest.mark.parametrize("dtype,kv,hq,hkv,new", [
    ("bf16", None, 8, 2, 9), ("f16", None, 8, 2, 60), ("f16", None, 2, 2, 9), ("bf16", "e4m3", 8, 2, 9),
    ("f16", "e5m2", 8, 2, 60)])
def test_the_limit_counts_from_the_end_of_the_previous_kernel(pkv, slow, monkeypatch, dtype, kv, hq, hkv,   # noqa: F811
                                                              new):
    c = Case([300, 40], [new, 3], hq=hq, hkv=hkv, d=64, dtype=dtype, kv=kv, seed=2)
    call, _ = tree_call(pkv, c)
    check(monkeypatch, slow, call, c.out, c.err)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_the_limit_of_chunks_counts_from_the_end_of_the_previous_kernel(pkv, slow, monkeypatch, dtype):   # noqa: F811
    c = chunk_case([300, 40], [30, 200], hq=8, hkv=2, d=64, dtype=dtype, seed=2)
    check(monkeypatch, slow, chunk_call(pkv, c, 100, 4), c.out, c.err)
