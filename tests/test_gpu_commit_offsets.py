"""The commit's device errors for offsets, and lists longer than a thread block."""
import numpy as np
import pytest
import torch

from oracle import draft as od
from tests.test_gpu_draft import OOB, Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    import __graft_entry__ as g
    g.build()
    import paged_kv_cache_153_gb300 as m
    return m


@pytest.mark.parametrize("cu,moved", [([-1, 5, 11], [1]), ([-3, -1, 5], []), ([0, 5, 3], [0]), ([5, 0, 6], [1]),
                                      ([-2 ** 31, 2 ** 31 - 1, 2 ** 31 - 1], [1])])
def test_bad_offsets_move_nothing(pkv, cu, moved):
    c = Case([20, 20], [6, 6], hq=1, hkv=2, d=64)
    c.cu = np.asarray(cu, np.int32)
    c.upload()
    before = [x.clone() for x in (c.kc, c.vc)]
    lists = torch.tensor([[1, 2, -1], [0, 3, -1]] if cu[-1] != cu[-2] else [[1, 2, -1], [-1, 0, 0]], dtype=torch.int32,
                         device="cuda")
    new = torch.full((2,), -5, dtype=torch.int32, device="cuda")
    pkv.pkv_tree_commit(c.kc, c.vc, c.tables, c.lens, c.cu_d, lists, new_lens=new, err_flag=c.err)
    torch.cuda.synchronize()
    assert int(c.err.item()) == OOB
    for b in range(2):
        if b in moved:
            assert int(new[b]) >= 0, b
            continue
        assert int(new[b]) == -5, b
        ids = torch.from_numpy(c.tab[b][c.tab[b] >= 0].astype(np.int64)).cuda()
        for x, y in zip((c.kc, c.vc), before):
            assert torch.equal(x[ids].view(torch.int16), y[ids].view(torch.int16)), b


@pytest.mark.parametrize("most", [300, 1024])
def test_long_lists(pkv, most):
    # more entries than a thread block has threads, in one and in several turns of the loops
    rng = np.random.default_rng(most)
    new = np.array([1500, most, 700])
    base = np.array([9, 100, 0])
    c = Case(base, np.minimum(new, 60), hq=1, hkv=1, d=64)     # (its masks hold 256 tokens at most)
    ctx = base + new
    width = int(-(-ctx.max() // 16))
    tab = rng.permutation(3 * width).reshape(3, width).astype(np.int32)
    acc = [sorted(rng.choice(1500, most, replace=False).tolist()), list(range(most)),
           sorted(rng.choice(700, 257, replace=False).tolist())]
    lists = np.full((3, most), -1, np.int32)
    for b, a in enumerate(acc):
        lists[b, :len(a)] = a
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a).astype(np.int32)).cuda()   # noqa: E731
    raw = [torch.randint(0, 256, (3 * width, 2, 16, 64), dtype=torch.uint8) for _ in range(2)]
    kc, vc = (x.cuda() for x in raw)
    c.upload()
    out = torch.zeros(3, dtype=torch.int32, device="cuda")
    pkv.pkv_tree_commit(kc, vc, up(tab), up(ctx), up(np.concatenate([[0], np.cumsum(new)])), up(lists), new_lens=out,
                        err_flag=c.err)
    torch.cuda.synchronize()
    assert int(c.err.item()) == 0 and out.tolist() == [int(x) + len(a) for x, a in zip(base, acc)]
    for got, x in zip((kc, vc), raw):
        want = x.numpy().copy()
        for b, a in enumerate(acc):
            p = np.arange(int(ctx[b]))
            want[tab[b][p // 16], :, p % 16] = od.commit(want[tab[b][p // 16], :, p % 16], int(base[b]), a)
        assert (got.cpu().numpy() == want).all()


def test_a_bad_entry_late_in_a_long_list_moves_nothing(pkv):
    n, most = 900, 800
    tab = np.arange(60, dtype=np.int32)[None]
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a).astype(np.int32)).cuda()   # noqa: E731
    raw = torch.randint(0, 256, (60, 1, 16, 64), dtype=torch.uint8)
    for bad in ((700, 650), (799, 900)):
        lists = 50 + np.arange(most)[None].astype(np.int32)
        lists[0, bad[0]] = bad[1]
        kc, vc, err = raw.cuda(), raw.cuda(), torch.zeros(1, dtype=torch.int32, device="cuda")
        new = torch.full((1,), -5, dtype=torch.int32, device="cuda")
        pkv.pkv_tree_commit(kc, vc, up(tab), up([10 + n]), up([0, n]), up(lists), new_lens=new, err_flag=err)
        torch.cuda.synchronize()
        assert int(err.item()) == OOB and int(new.item()) == -5
        assert torch.equal(kc.cpu(), raw) and torch.equal(vc.cpu(), raw)
