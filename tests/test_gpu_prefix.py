"""Shared-prefix decode on the GPU against float64, within limits taken from
the arithmetic; and its refusals."""
import ctypes as C

import numpy as np
import pytest
import torch

from tests import attn_limits
from tests import gpu_util as gu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    import __graft_entry__ as g
    g.build()
    import paged_kv_cache_153_gb300 as m
    return m


class Case:
    """groups: a list of (shared tokens, own tokens of each sequence); own None
    is a padding sequence of length 0 whose table row is -1.  Every cache row
    that no context covers is NaN."""

    def __init__(self, groups, *, hq=8, hkv=2, d=128, dtype="bf16", seed=0, declared=None, bias=0.0):
        g = torch.Generator().manual_seed(seed)
        t = gu.TORCH_16[dtype]
        self.hq, self.hkv, self.d, self.dtype, self.scale = hq, hkv, d, dtype, d ** -0.5
        lens, rows, starts = [], [], [0]
        nxt, live = 0, {}

        def take(n):
            nonlocal nxt
            nxt += n
            return list(range(nxt - n, nxt))
        for shared, own in groups:
            common = take(shared // 16)
            for x in own:
                n = 0 if x is None else shared + x
                row = [] if x is None else (common + take(max(0, -(-n // 16) - len(common))))[:-(-n // 16)]
                lens.append(n)
                rows.append(row)
                for i, blk in enumerate(row):
                    live[blk] = max(live.get(blk, 0), min(16, n - 16 * i))
            starts.append(len(lens))
        self.nb = nxt + 3
        perm = torch.randperm(self.nb, generator=g).tolist()
        self.width = max(1, max(len(r) for r in rows)) + 1
        tab = np.full((len(rows), self.width), -1, np.int32)
        for b, r in enumerate(rows):
            tab[b, :len(r)] = [perm[i] for i in r]
        kc = torch.randn((self.nb, hkv, 16, d), generator=g) + bias
        vc = torch.randn((self.nb, hkv, 16, d), generator=g)
        dead = torch.ones((self.nb, 16), dtype=torch.bool)
        for blk, n in live.items():
            dead[perm[blk], :n] = False
        dead = dead[:, None, :, None].expand(kc.shape)
        kc[dead] = vc[dead] = float("nan")
        self.kc, self.vc = kc.to(t).cuda(), vc.to(t).cuda()
        self.q = (torch.randn((len(lens), hq, d), generator=g) + bias).to(t).cuda()
        self.tab_h, self.lens_h = tab, np.array(lens, np.int32)
        self.tab, self.lens = torch.from_numpy(tab).cuda(), torch.from_numpy(self.lens_h).cuda()
        self.starts = torch.tensor(starts, dtype=torch.int32).cuda()
        pre = [s for s, _ in groups] if declared is None else declared
        self.pre = torch.tensor(pre, dtype=torch.int32).cuda()
        self.max_pre, self.max_ctx = max(pre + [0]), max(lens + [1])
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def workspace(self, pkv):
        n = pkv.pkv_prefix_workspace_bytes(len(self.lens_h), self.pre.numel(), self.hq, self.hkv, self.d, self.width,
                                           self.max_ctx, self.max_pre)
        return torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")

    def call(self, pkv, out, ws, stream=None):
        pkv.pkv_paged_decode_attention_prefix(self.q, self.kc, self.vc, self.tab, self.lens, self.starts, self.pre, out,
                                              scale=self.scale, max_context_len=self.max_ctx, max_prefix_len=self.max_pre,
                                              workspace=ws, err_flag=self.err, stream=stream)

    def run(self, pkv, ws=None):
        out = torch.full_like(self.q, float("nan"))
        self.call(pkv, out, self.workspace(pkv) if ws is None else ws)
        torch.cuda.synchronize()
        return out

    def check(self, out, seqs=None):
        q, got = self.q.double().cpu().numpy(), out.double().cpu().numpy()
        per = self.hq // self.hkv
        for b in range(len(self.lens_h)) if seqs is None else seqs:
            n = int(self.lens_h[b])
            ids = torch.from_numpy(self.tab_h[b, :-(-n // 16)]).long().cuda()
            for g in range(self.hkv):
                k = self.kc[ids, g].reshape(-1, self.d)[:n].double().cpu().numpy()
                v = self.vc[ids, g].reshape(-1, self.d)[:n].double().cpu().numpy()
                for h in range(g * per, (g + 1) * per):
                    ref, lim = attn_limits.attend(q[b, h], k, v, self.scale, self.dtype)
                    bad = ~(np.abs(got[b, h] - ref) <= lim)
                    assert not bad.any(), (b, h, n, got[b, h][bad][:4], ref[bad][:4], lim[bad][:4])


SHAPES = [(3, 3, 128), (4, 2, 64), (8, 2, 128), (8, 1, 64), (16, 2, 128), (4, 4, 64)]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("hq,hkv,d", SHAPES)
def test_one_group(pkv, dtype, hq, hkv, d):
    case = Case([(512, [1, 16, 100, 37, 300])], hq=hq, hkv=hkv, d=d, dtype=dtype, seed=hq + d)
    case.check(case.run(pkv))
    assert int(case.err.item()) == 0


@pytest.mark.parametrize("dtype,hq,hkv,d", [("bf16", 8, 2, 128), ("f16", 8, 1, 64), ("f16", 2, 2, 128)])
@pytest.mark.parametrize("shared", [16, 112, 128, 144, 1008, 1024, 2064])
def test_prefix_lengths_around_the_tiles(pkv, dtype, hq, hkv, d, shared):
    case = Case([(shared, [5, 0, 40])], hq=hq, hkv=hkv, d=d, dtype=dtype, seed=shared)
    case.check(case.run(pkv))
    assert int(case.err.item()) == 0


@pytest.mark.parametrize("n", [1, 31, 32, 33, 63, 64, 65, 130, 200])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_row_counts_around_the_tiles(pkv, n, dtype):
    # n sequences x 4 query heads: one row tile, two against the same keys, several units
    case = Case([(656, [(7 * i) % 50 for i in range(n)])], hq=8, hkv=2, dtype=dtype, seed=n)
    case.check(case.run(pkv), range(0, n, max(1, n // 9)))
    assert int(case.err.item()) == 0


@pytest.mark.parametrize("hq,hkv,d,n", [(2, 2, 64, 200), (2, 2, 128, 300), (16, 2, 64, 40), (4, 2, 64, 129)])
def test_row_tiles_of_other_groups_and_dims(pkv, hq, hkv, d, n):
    case = Case([(1040, [(11 * i) % 70 for i in range(n)])], hq=hq, hkv=hkv, d=d, dtype="bf16", seed=n)
    case.check(case.run(pkv), range(0, n, max(1, n // 7)))
    assert int(case.err.item()) == 0


@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (8, 8, 64), (8, 1, 128)])
def test_many_groups(pkv, hq, hkv, d):
    groups = [(1500, [10, 20, 1]), (0, [100, 7]), (48, []), (16, [3]), (4000, [1] * 40), (33, [64, 2]), (640, [0] * 5)]
    case = Case(groups, hq=hq, hkv=hkv, d=d, dtype="f16", seed=5)
    case.check(case.run(pkv))
    assert int(case.err.item()) == 0


def test_hundreds_of_groups(pkv):
    rng = np.random.default_rng(0)
    groups = [(int(rng.integers(0, 90)), [int(x) for x in rng.integers(0, 40, size=rng.integers(0, 4))])
              for _ in range(700)]
    case = Case(groups, hq=4, hkv=2, d=64, seed=6)
    case.check(case.run(pkv), range(0, len(case.lens_h), 37))
    assert int(case.err.item()) == 0


def test_lengths_that_are_no_whole_blocks(pkv):
    # the declared prefix ends inside a block: that block is each sequence's own
    case = Case([(512, [30, 9, 250])], seed=7, declared=[519])
    case.check(case.run(pkv))
    # a declaration shorter than what is shared
    case = Case([(512, [30, 9, 250])], seed=8, declared=[100])
    case.check(case.run(pkv))
    # nothing declared, or a negative length
    for declared in ([0], [15], [-5]):
        case = Case([(512, [30, 9, 250])], seed=9, declared=declared)
        case.check(case.run(pkv))
    assert int(case.err.item()) == 0


def test_padding_and_short_sequences(pkv):
    # sequences without tokens, first and last of a group, and a group of them alone
    case = Case([(300, [None, 20, 5, None]), (256, [None, None]), (128, [1, None, 2])], seed=10)
    out = case.run(pkv)
    case.check(out)
    assert torch.all(out[case.lens == 0] == 0) and int(case.err.item()) == 0
    # a sequence that ends inside the shared blocks; NaN behind its own end must not reach it
    case = Case([(512, [40, 3])], seed=11)
    case.lens_h[1] = 100
    case.lens.copy_(torch.from_numpy(case.lens_h))
    case.check(case.run(pkv))
    short = Case([(512, [-412, -500])], seed=12, declared=[512])     # the whole group is shorter than declared
    short.check(short.run(pkv))
    assert int(short.err.item()) == 0


def test_large_logits(pkv):
    # a common offset makes logits of several hundred: the reference must follow them
    case = Case([(1200, [77, 3, 12])], hq=4, hkv=1, dtype="f16", seed=13, bias=3.0)
    case.check(case.run(pkv))


def test_result_agrees_with_dense_decode_and_repeats(pkv):
    case = Case([(2048, [16 + 31 * i for i in range(16)])], hq=32, hkv=8, seed=14)
    out = case.run(pkv)
    dense = torch.empty_like(case.q)
    ws = torch.empty(pkv.pkv_decode_workspace_bytes(16, 32, 8, 128, case.width, case.max_ctx), dtype=torch.uint8,
                     device="cuda")
    pkv.pkv_paged_decode_attention(case.q, case.kc, case.vc, case.tab, case.lens, dense, scale=case.scale,
                                   max_context_len=case.max_ctx, workspace=ws)
    torch.cuda.synchronize()
    assert (out.float() - dense.float()).abs().max() <= 2 * 2.0 ** -8 * dense.float().abs().max()
    case.check(out, [0, 15])
    for _ in range(20):                               # the same bits each time
        assert torch.equal(case.run(pkv), out)


def test_long_prefix(pkv):
    case = Case([(20000, [3, 500, 16, 1])], hq=8, hkv=2, seed=15)
    case.check(case.run(pkv))
    case = Case([(6000, [(5 * i) % 90 for i in range(70)])], hq=8, hkv=1, dtype="f16", seed=16)
    case.check(case.run(pkv), [0, 31, 32, 63, 64, 69])


def test_streams_graphs_and_workspaces(pkv):
    a = Case([(900, [16, 33, 50]), (200, [1, 2])], seed=17)
    b = Case([(1700, [9] * 40)], seed=18)
    ra, rb = a.run(pkv), b.run(pkv)
    # an unaligned workspace (16 bytes) is enough
    ws = a.workspace(pkv)
    big = torch.empty(ws.numel() + 16, dtype=torch.uint8, device="cuda")
    assert torch.equal(a.run(pkv, big[16:]), ra)
    # two streams at a time, each with its workspace
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    oa, ob = torch.empty_like(ra), torch.empty_like(rb)
    wa, wb = a.workspace(pkv), b.workspace(pkv)
    torch.cuda.synchronize()
    for _ in range(10):
        a.call(pkv, oa, wa, sa)
        b.call(pkv, ob, wb, sb)
    torch.cuda.synchronize()
    assert torch.equal(oa, ra) and torch.equal(ob, rb)
    # captured, then replayed with other data in the same buffers; one workspace, one after the other
    graph = torch.cuda.CUDAGraph()
    ws = a.workspace(pkv) if a.workspace(pkv).numel() > b.workspace(pkv).numel() else b.workspace(pkv)
    with torch.cuda.graph(graph):
        a.call(pkv, oa, ws)
        b.call(pkv, ob, ws)
    oa.fill_(float("nan")), ob.fill_(float("nan"))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(oa, ra) and torch.equal(ob, rb)
    a.q.copy_(torch.randn(a.q.shape, device="cuda"))
    a.lens_h[0] -= 13
    a.lens.copy_(torch.from_numpy(a.lens_h))
    graph.replay()
    torch.cuda.synchronize()
    a.check(oa)


def test_device_errors(pkv):
    def broken(f, seed=19):
        case = Case([(512, [30, 9]), (256, [4])], seed=seed)
        f(case)
        case.run(pkv)
        return int(case.err.item())
    assert broken(lambda c: None) == 0
    assert broken(lambda c: c.tab.__setitem__((0, 3), c.nb)) == 4         # a shared block's id
    assert broken(lambda c: c.tab.__setitem__((1, 32), -7)) == 4          # a private one's
    assert broken(lambda c: c.lens.__setitem__(2, 16 * c.width + 1)) == 4
    assert broken(lambda c: c.lens.__setitem__(2, -1)) == 4
    for starts in ([0, 3, 2], [0, 2, 4], [-1, 2, 3], [1, 2, 3], [0, 5, 3], [0, 1, 2]):
        assert broken(lambda c: c.starts.copy_(torch.tensor(starts))) == 4, starts


def test_group_starts_far_behind_the_first_sequence(pkv):
    # no group starts at or before most of the sequences: reported, and what the
    # others' states would be is not read
    case = Case([(512, [30] * 130)], seed=24)
    case.starts.copy_(torch.tensor([100, 130]))
    case.run(pkv)
    assert int(case.err.item()) == 4


def test_lengths_at_the_end_of_int32(pkv):
    # a bound that promises nothing changes no result
    case = Case([(512, [30, 9]), (64, [100])], seed=25)
    want = case.run(pkv)
    case.max_ctx = case.max_pre = 2 ** 31 - 1
    assert torch.equal(case.run(pkv), want) and int(case.err.item()) == 0
    dense = torch.empty_like(case.q)
    ws = torch.empty(pkv.pkv_decode_workspace_bytes(3, 8, 2, 128, case.width, case.max_ctx), dtype=torch.uint8,
                     device="cuda")
    pkv.pkv_paged_decode_attention(case.q, case.kc, case.vc, case.tab, case.lens, dense, scale=case.scale,
                                   max_context_len=case.max_ctx, workspace=ws, err_flag=case.err)
    torch.cuda.synchronize()
    case.check(dense)
    assert int(case.err.item()) == 0
    # a context as long: clamped and reported (both forms of the merge), the others as they were
    for groups in ([(512, [30, 9]), (64, [100])], [(512, [30] * 300), (64, [100])]):
        case = Case(groups, seed=26)
        want = case.run(pkv)
        for n in (2 ** 31 - 1, 2 ** 31 - 16):
            case.lens[0] = n
            out = case.run(pkv)
            assert int(case.err.item()) == 4
            case.check(out, [1, len(case.lens_h) - 1])
            case.err.zero_()


def test_contexts_past_the_declared_bound(pkv):
    # as in the dense decode: clamped to the bound and reported
    case = Case([(512, [30, 9]), (64, [400])], seed=21)
    case.max_ctx = 523
    out = case.run(pkv)
    assert int(case.err.item()) == 4
    case.check(out, [1, 2])
    case = Case([(512, [30, 9]), (64, [100])], seed=22)
    case.max_ctx = 170                               # shorter than the first group's prefix
    out = case.run(pkv)
    assert int(case.err.item()) == 4
    case.check(out, [2])


def test_far_blocks_of_a_large_pool(pkv):
    # blocks past 4 GiB of the cache
    case = Case([(256, [20, 33])], hq=16, hkv=8, seed=23)
    near = case.run(pkv)
    nb = 140000
    move = {int(i): nb - 1 - k for k, i in enumerate(np.unique(case.tab_h[case.tab_h >= 0]))}
    for name in ("kc", "vc"):
        big = torch.zeros((nb, 8, 16, 128), dtype=torch.bfloat16, device="cuda")
        small = getattr(case, name)
        for i, j in move.items():
            big[j] = small[i]
        setattr(case, name, big)
    case.tab_h = np.vectorize(lambda i: move.get(int(i), -1))(case.tab_h).astype(np.int32)
    case.tab.copy_(torch.from_numpy(case.tab_h))
    assert torch.equal(case.run(pkv), near) and int(case.err.item()) == 0


def test_refusals(pkv):
    case = Case([(512, [30, 9])], seed=20)
    ws = case.workspace(pkv)
    for name in ("lens", "tab", "pre", "starts"):
        keep = getattr(case, name)
        setattr(case, name, keep.long())
        with pytest.raises(TypeError):
            case.run(pkv, ws)
        setattr(case, name, keep)
    with pytest.raises(pkv.PkvError) as e:
        case.run(pkv, ws[:-1])
    assert e.value.status == 6
    with pytest.raises(ValueError):
        case.pre = case.pre.repeat(2)
        case.run(pkv, ws)
