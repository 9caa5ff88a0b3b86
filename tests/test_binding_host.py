"""What the Python binding refuses before it calls the library: caches of
another element type or shape than the call reads and writes, lengths and tables
that do not have a row per sequence.  (Tensors on the host: nothing is launched.)"""
import pytest
import torch


@pytest.fixture(scope="module")
def pkv():
    import __graft_entry__ as g
    g.build()
    import paged_kv_cache_153_gb300 as m
    return m


B, HQ, HKV, D, NB, W = 3, 8, 2, 64, 10, 4
Q = torch.zeros((B, HQ, D), dtype=torch.bfloat16)
K16 = torch.zeros((NB, HKV, 16, D), dtype=torch.bfloat16)
K8 = torch.zeros((NB, HKV, 16, D), dtype=torch.uint8)
TAB = torch.zeros((B, W), dtype=torch.int32)
LENS = torch.ones(B, dtype=torch.int32)
SCALE = torch.ones(HKV)
BOUNDS = torch.zeros((NB, HKV, 2, D), dtype=torch.bfloat16)
SCORES = torch.zeros((B, HKV, W))
LISTS = torch.zeros((B, HKV, 2), dtype=torch.int32)
WS = torch.zeros(16, dtype=torch.uint8)
STARTS, PRE = torch.tensor([0, B], dtype=torch.int32), torch.tensor([16], dtype=torch.int32)
NEW = torch.zeros((B, HKV, D), dtype=torch.bfloat16)
SLOTS = torch.zeros(B, dtype=torch.int64)
TURNS = torch.zeros(D // 2, dtype=torch.int64)


def sparse(pkv, k=K16, v=K16, tab=TAB, lens=LENS, out=Q):
    pkv.pkv_paged_decode_attention_sparse(Q, k, v, tab, lens, LISTS, out, scale=1.0, workspace=WS, stream=0)


def sparse_fp8(pkv, k=K8, v=K8, tab=TAB, lens=LENS, out=Q):
    pkv.pkv_paged_decode_attention_sparse_fp8(Q, k, v, SCALE, SCALE, tab, lens, LISTS, out, scale=1.0, workspace=WS,
                                              stream=0)


def prefix(pkv, k=K16, v=K16, tab=TAB, lens=LENS, out=Q):
    pkv.pkv_paged_decode_attention_prefix(Q, k, v, tab, lens, STARTS, PRE, out, scale=1.0, max_context_len=64,
                                          max_prefix_len=16, workspace=WS, stream=0)


@pytest.mark.parametrize("call", [sparse, prefix])
def test_attention_over_16_bit_caches(pkv, call):
    for bad in (dict(k=K8, v=K8), dict(v=K8), dict(v=K16[:5]), dict(k=K16.transpose(0, 1)), dict(k=K16.float()),
                dict(tab=TAB[:2]), dict(lens=LENS[:2]), dict(out=Q[:2])):
        with pytest.raises(ValueError):
            call(pkv, **bad)


def test_attention_over_fp8_caches(pkv):
    for bad in (dict(k=K16, v=K16), dict(v=K8[:5]), dict(tab=TAB[:2]), dict(lens=LENS[:2])):
        with pytest.raises(ValueError):
            sparse_fp8(pkv, **bad)


def test_tensors_of_another_device(pkv):
    # (all that these calls get is on the host)
    for call in (sparse, sparse_fp8, prefix):
        with pytest.raises(ValueError, match="device"):
            call(pkv)
    with pytest.raises(ValueError, match="device"):
        pkv.pkv_block_scores(Q, BOUNDS, TAB, LENS, SCORES, scale=1.0, max_context_len=64, stream=0)
    with pytest.raises(ValueError, match="device"):
        pkv.pkv_select_blocks(SCORES, LENS, LISTS, stream=0)
    with pytest.raises(ValueError, match="device"):
        pkv.pkv_rope_append(Q, NEW, NEW, LENS, SLOTS, TURNS, Q, K16, K16, stream=0)
    with pytest.raises(ValueError, match="device"):
        pkv.pkv_kv_block_bounds(K16, TAB, LENS, BOUNDS, max_new_len=1, stream=0)


def test_block_index(pkv):
    def bounds(k, new=None, tab=TAB, fn="pkv_kv_block_bounds"):
        getattr(pkv, fn)(k, tab, LENS, BOUNDS, max_new_len=1, new_lens=new, stream=0)
    for bad in (dict(k=K8), dict(k=K16, tab=TAB[:2]), dict(k=K16, new=LENS[:2]), dict(k=K16, fn="pkv_kv_block_bounds_fp8"),
                dict(k=K16, fn="pkv_kv_block_bounds_e5m2")):
        with pytest.raises(ValueError):
            bounds(**bad)
    with pytest.raises(ValueError):
        pkv.pkv_block_scores(Q, BOUNDS, TAB[:2], LENS, SCORES, scale=1.0, max_context_len=64, stream=0)
    with pytest.raises(TypeError):
        pkv.pkv_block_scores(Q, BOUNDS, TAB, LENS, SCORES.half(), scale=1.0, max_context_len=64, stream=0)
    with pytest.raises(ValueError):
        pkv.pkv_select_blocks(SCORES.half(), LENS, LISTS, stream=0)
    with pytest.raises(ValueError):
        pkv.pkv_select_blocks(SCORES, LENS[:2], LISTS, stream=0)


def test_rope_append(pkv):
    def rope(k=K16, v=K16, turns=TURNS):
        pkv.pkv_rope_append(Q, NEW, NEW, LENS, SLOTS, turns, Q, k, v, stream=0)
    for bad in (dict(k=K8, v=K8), dict(v=K16[:5]), dict(v=K16.half())):
        with pytest.raises(ValueError):
            rope(**bad)
    for turns in (TURNS.double(), TURNS.int()):
        with pytest.raises(TypeError):
            rope(turns=turns)
    with pytest.raises(ValueError):
        pkv.pkv_rope_append_fp8(Q, NEW, NEW, LENS, SLOTS, TURNS, Q, K16, K16, SCALE, SCALE, stream=0)
