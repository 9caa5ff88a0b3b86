"""Block-sparse decode on the GPU against float64: bounds and lists exactly,
scores and attention within limits taken from the arithmetic."""
import numpy as np
import pytest
import torch

from oracle import sparse as osp
from tests import attn_limits
from tests import gpu_util as gu

pytestmark = pytest.mark.gpu

FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


@pytest.fixture(scope="module")
def pkv():
    import __graft_entry__ as g
    g.build()
    import paged_kv_cache_153_gb300 as m
    return m


class Case:
    """Random pool, tables and queries; every row no context covers is NaN."""

    def __init__(self, lens, *, hq=8, hkv=2, d=128, dtype="bf16", kv=None, seed=0, wide=0, poison=True):
        self.lens_h, self.hq, self.hkv, self.d, self.dtype, self.kv = np.asarray(lens, np.int32), hq, hkv, d, dtype, kv
        g = torch.Generator().manual_seed(seed)
        t = gu.TORCH_16[dtype]
        nblk = [-(-int(n) // 16) for n in lens]
        self.nb = sum(nblk) + 2
        self.width = max(1, max(nblk, default=0)) + wide
        perm = torch.randperm(self.nb, generator=g).to(torch.int32)
        tab = torch.full((len(lens), self.width), -1, dtype=torch.int32)
        at = 0
        kc = torch.randn((self.nb, hkv, 16, d), generator=g)
        vc = torch.randn((self.nb, hkv, 16, d), generator=g)
        live = torch.zeros((self.nb, 16), dtype=torch.bool)
        for b, n in enumerate(nblk):
            tab[b, :n] = perm[at:at + n]
            at += n
            for i in range(n):
                live[tab[b, i].long(), :min(16, int(lens[b]) - 16 * i)] = True
        dead = ~live[:, None, :, None].expand(kc.shape)
        if kv:
            self.scales = (torch.rand((2, hkv), generator=g) + 0.5).cuda()
            kc, vc = (x.to(FP8[kv]).view(torch.uint8) for x in (kc, vc))
            if poison:
                kc[dead], vc[dead] = 0x7F, 0x7F          # a NaN code of both formats
        else:
            kc, vc = kc.to(t), vc.to(t)
            if poison:
                kc[dead], vc[dead] = float("nan"), float("nan")
        self.q = torch.randn((len(lens), hq, d), generator=g).to(t).cuda()
        self.kc, self.vc, self.tab, self.tab_h = kc.cuda(), vc.cuda(), tab.cuda(), tab.numpy()
        self.lens = torch.from_numpy(self.lens_h).cuda()
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.scale = d ** -0.5
        self.gen = g

    def values(self, which, scaled=True):
        c = self.kc if which == 0 else self.vc
        x = c.view(FP8[self.kv]).float() if self.kv else c
        x = x.double().cpu().numpy()
        return x * self.scales[which].double().cpu().numpy()[:, None, None] if self.kv and scaled else x

    def attention(self, pkv, selected, ws=None, stream=None):
        budget = selected.shape[2]
        n = pkv.pkv_decode_workspace_bytes(len(self.lens_h), self.hq, self.hkv, self.d, budget, 16 * budget)
        ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") if ws is None else ws
        out = torch.full_like(self.q, float("nan"))
        fn = {"e4m3": pkv.pkv_paged_decode_attention_sparse_fp8,
              "e5m2": pkv.pkv_paged_decode_attention_sparse_e5m2}.get(self.kv, pkv.pkv_paged_decode_attention_sparse)
        fn(self.q, self.kc, self.vc, *(tuple(self.scales) if self.kv else ()), self.tab, self.lens, selected, out,
           scale=self.scale, workspace=ws, err_flag=self.err, stream=stream)
        torch.cuda.synchronize()
        return out

    def check_attention(self, out, selected):
        k, v = self.values(0), self.values(1)
        q = self.q.double().cpu().numpy()
        got = out.double().cpu().numpy()
        sel = selected.cpu().numpy()
        per = self.hq // self.hkv
        for b, n in enumerate(self.lens_h):
            nblk = -(-int(n) // 16)
            for g in range(self.hkv):
                pos = osp.token_positions([i for i in sel[b, g, :min(sel.shape[2], nblk)] if i < nblk], int(n))
                ids = self.tab_h[b][pos // 16]
                for h in range(g * per, (g + 1) * per):
                    ref, lim = attn_limits.attend(q[b, h], k[ids, g, pos % 16], v[ids, g, pos % 16], self.scale,
                                                  self.dtype, "f16" if self.kv else None)
                    bad = ~(np.abs(got[b, h] - ref) <= lim)
                    assert not bad.any(), (b, h, int(n), got[b, h][bad][:4], ref[bad][:4], lim[bad][:4])


def random_lists(case, budget, seed=0, ragged=False):
    """Ascending random lists with the last block, -1 behind (and, ragged, at
    random places)."""
    rng = np.random.default_rng(seed)
    out = np.full((len(case.lens_h), case.hkv, budget), -1, dtype=np.int32)
    for b, n in enumerate(case.lens_h):
        nblk = -(-int(n) // 16)
        for g in range(case.hkv):
            m = min(nblk, budget)
            if m:
                x = np.sort(np.append(rng.permutation(nblk - 1)[:m - 1], nblk - 1))
                out[b, g, :m] = np.where(rng.random(m) < 0.3, -1, x) if ragged else x
    return torch.from_numpy(out).cuda()


# ---------------------------------------------------------------------------
# bounds
# ---------------------------------------------------------------------------
def expected_bounds(case, before, new=None):
    want = before.double().cpu().numpy().copy()
    k = case.values(0, scaled=False)
    for b, n in enumerate(case.lens_h):
        n = int(n)
        m = n if new is None else int(new[b])
        if m == 0:
            continue
        for i in range((n - m) // 16, -(-n // 16)):
            for g in range(case.hkv):
                lo, hi = osp.block_bounds(k[case.tab_h[b, i], g], min(16, n - 16 * i))
                want[case.tab_h[b, i], g] = lo, hi
    return want


def run_bounds(pkv, case, bounds, new=None, max_new=None):
    fn = {"e4m3": pkv.pkv_kv_block_bounds_fp8, "e5m2": pkv.pkv_kv_block_bounds_e5m2}.get(
        case.kv, pkv.pkv_kv_block_bounds)
    new_t = None if new is None else torch.tensor(new, dtype=torch.int32, device="cuda")
    top = max(case.lens_h.tolist() if new is None else new) if max_new is None else max_new
    fn(case.kc, case.tab, case.lens, bounds, new_lens=new_t, max_new_len=int(top), err_flag=case.err)
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype,kv", [("f16", None), ("bf16", None), ("f16", "e4m3"), ("bf16", "e4m3"), ("bf16", "e5m2"),
                                      ("f16", "e5m2")])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hkv", [1, 3])
def test_bounds(pkv, dtype, kv, d, hkv):
    case = Case([0, 1, 15, 16, 17, 100, 333], hkv=hkv, hq=hkv, d=d, dtype=dtype, kv=kv, seed=d + hkv)
    for new in (None, [0, 1, 15, 1, 2, 37, 333], [0, 1, 1, 1, 1, 1, 1]):
        bounds = torch.full((case.nb, hkv, 2, d), 7.0, dtype=gu.TORCH_16[dtype], device="cuda")
        want = expected_bounds(case, bounds, new)
        run_bounds(pkv, case, bounds, new)
        assert np.array_equal(bounds.double().cpu().numpy(), want)
    assert int(case.err.item()) == 0


def device_bounds(case):
    """Bounds of every block of every context, on the GPU in the keys' type."""
    k = case.kc.view(FP8[case.kv]).float() if case.kv else case.kc.float()
    want = torch.full((case.nb, case.hkv, 2, case.d), 7.0, device="cuda")
    row = torch.arange(16, device="cuda")
    for b, n in enumerate(case.lens_h):
        ids = case.tab[b, :-(-int(n) // 16)].long()
        past = (torch.arange(len(ids), device="cuda")[:, None] * 16 + row >= int(n))[:, None, :, None]
        want[ids, :, 0] = k[ids].masked_fill(past, float("inf")).amin(2)
        want[ids, :, 1] = k[ids].masked_fill(past, float("-inf")).amax(2)
    return want


@pytest.mark.parametrize("dtype,kv,hkv,d", [("bf16", None, 3, 128), ("f16", None, 1, 64), ("bf16", "e4m3", 8, 128),
                                            ("f16", "e5m2", 5, 64)])
def test_bounds_of_large_mixed_batches(pkv, dtype, kv, hkv, d):
    # enough slabs that the work is dealt flat over the sequences
    rng = np.random.default_rng(hkv)
    lens = [0, 1, 40000, 17, 0] + [int(x) for x in rng.integers(0, 9000, size=60)] + [0, 16]
    case = Case(lens, hkv=hkv, hq=hkv, d=d, dtype=dtype, kv=kv, seed=hkv)
    bounds = torch.full((case.nb, hkv, 2, d), 7.0, dtype=gu.TORCH_16[dtype], device="cuda")
    run_bounds(pkv, case, bounds)
    assert torch.equal(bounds.float(), device_bounds(case)) and int(case.err.item()) == 0
    # the newest tokens only: as many, up to the whole context
    new = [min(n, 5000) for n in lens]
    part = torch.full_like(bounds, 7.0)
    run_bounds(pkv, case, part, new)
    kept = torch.ones(case.nb, dtype=torch.bool)
    for b, (n, m) in enumerate(zip(lens, new)):
        if m:
            kept[case.tab_h[b, (n - m) // 16:-(-n // 16)]] = False
    kept = kept.cuda()
    assert torch.all(part[kept] == 7.0) and torch.equal(part[~kept], bounds[~kept]) and int(case.err.item()) == 0
    # a bad id and a context past its table are reported, the rest is done
    case.tab[2, 100] = case.nb
    case.lens[4] = 16 * case.width + 1
    case.tab[4] = case.tab[2, 0]
    again = torch.full_like(bounds, 7.0)
    run_bounds(pkv, case, again)
    assert int(case.err.item()) == 4
    ids = case.tab[5, :-(-lens[5] // 16)].long()
    assert torch.equal(again[ids], bounds[ids])


def test_bounds_keep_a_nan_and_infinities(pkv):
    case = Case([40], hkv=1, hq=1, d=64, dtype="f16", seed=3)
    ids = case.tab_h[0]
    case.kc[ids[0], 0, 3, 5] = float("nan")
    case.kc[ids[1], 0, 3, 6] = float("-inf")
    bounds = torch.zeros((case.nb, 1, 2, 64), dtype=torch.float16, device="cuda")
    run_bounds(pkv, case, bounds)
    assert torch.isnan(bounds[ids[0], 0, :, 5]).all() and int(torch.isnan(bounds).sum()) == 2
    assert bounds[ids[1], 0, 0, 6] == float("-inf") and torch.isfinite(bounds[ids[1], 0, 1, 6])


def test_bounds_device_errors(pkv):
    case = Case([100, 40], seed=4)
    full = torch.zeros((case.nb, 2, 2, 128), dtype=torch.bfloat16, device="cuda")
    for break_it in (lambda c: c.tab.__setitem__((0, 2), c.nb), lambda c: c.tab.__setitem__((0, 2), -5),
                     lambda c: c.lens.__setitem__(1, 16 * c.width + 1), lambda c: c.lens.__setitem__(1, -1)):
        c = Case([100, 40], seed=4)
        break_it(c)
        run_bounds(pkv, c, full)
        assert int(c.err.item()) == 4
    c = Case([100, 40], seed=4)
    run_bounds(pkv, c, full, new=[101, 1])
    assert int(c.err.item()) == 4
    c = Case([100, 40], seed=4)
    full.fill_(9)
    run_bounds(pkv, c, full, new=[100, 1], max_new=20)   # more new tokens than the bound
    assert int(c.err.item()) == 4
    assert torch.all(full[c.tab_h[0, 4]] == 9)           # past it: left as they were


# ---------------------------------------------------------------------------
# scores
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (6, 3), (8, 2), (16, 2)])
def test_scores(pkv, dtype, d, hq, hkv):
    case = Case([0, 1, 16, 17, 255, 256, 257, 1030, 4000], hq=hq, hkv=hkv, d=d, dtype=dtype, seed=d + hq, wide=3)
    bounds = torch.full((case.nb, hkv, 2, d), float("nan"), dtype=gu.TORCH_16[dtype], device="cuda")
    run_bounds(pkv, case, bounds)
    k_scale = torch.rand(hkv).cuda() + 0.5
    scores = torch.full((9, hkv, case.width), -7.0, device="cuda")
    for ks in (None, k_scale):
        pkv.pkv_block_scores(case.q, bounds, case.tab, case.lens, scores, scale=case.scale, max_context_len=4000,
                             k_scale=ks, err_flag=case.err)
        torch.cuda.synchronize()
        got = scores.double().cpu().numpy()
        bd, q = bounds.double().cpu().numpy(), case.q.double().cpu().numpy()
        factor = np.full(hkv, case.scale) * (1.0 if ks is None else ks.double().cpu().numpy())
        per = hq // hkv
        for b, n in enumerate(case.lens_h):
            nblk = -(-int(n) // 16)
            assert np.all(got[b, :, nblk:] == -7.0)
            for g in range(hkv):
                lo_hi = bd[case.tab_h[b, :nblk], g]
                for i in range(nblk):
                    qg = q[b, g * per:(g + 1) * per]
                    ref = osp.block_score(qg, lo_hi[i, 0], lo_hi[i, 1], factor[g])
                    # 2 D exact products, each addition off by at most 2^-23 of the sum of magnitudes;
                    # the two factors round three times
                    mass = (np.abs(qg) * np.abs(lo_hi[i]).max(0)).sum(1).max() * factor[g]
                    assert abs(got[b, g, i] - ref) <= mass * (2 * d + 4) * 2.0 ** -23
    assert int(case.err.item()) == 0


@pytest.mark.parametrize("dtype,hq,hkv,d", [("bf16", 32, 8, 128), ("f16", 8, 1, 64), ("bf16", 5, 5, 128),
                                            ("f16", 64, 8, 128), ("bf16", 40, 20, 64), ("f16", 3, 3, 64)])
def test_scores_of_large_mixed_batches(pkv, dtype, hq, hkv, d):
    # enough blocks that persistent thread blocks take them from one list
    rng = np.random.default_rng(hq)
    lens = [0, 1, 60000, 17, 0] + [int(x) for x in rng.integers(0, 20000, size=90)] + [0, 16]
    g = torch.Generator(device="cuda").manual_seed(hq)
    t = gu.TORCH_16[dtype]
    nblk = [-(-n // 16) for n in lens]
    width, nb, per = max(nblk) + 2, sum(nblk) + 5, hq // hkv
    ids = torch.randperm(nb, generator=g, device="cuda", dtype=torch.int32)
    tab = torch.full((len(lens), width), -1, dtype=torch.int32, device="cuda")
    for b, n in enumerate(nblk):
        tab[b, :n] = ids[sum(nblk[:b]):sum(nblk[:b]) + n]
    x = torch.randn((nb, hkv, 2, d), generator=g, device="cuda").to(t)
    bounds = torch.stack([x.amin(2), x.amax(2)], 2).contiguous()
    bounds[ids[sum(nblk):].long()] = float("nan")
    q = torch.randn((len(lens), hq, d), generator=g, device="cuda").to(t)
    scores = torch.full((len(lens), hkv, width), -7.0, device="cuda")
    lens_t = torch.tensor(lens, dtype=torch.int32, device="cuda")
    k_scale = torch.rand(hkv, generator=g, device="cuda") + 0.5
    err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def call():
        pkv.pkv_block_scores(q, bounds, tab, lens_t, scores, scale=0.1, max_context_len=60000, k_scale=k_scale,
                             err_flag=err)
        torch.cuda.synchronize()
    call()
    assert int(err.item()) == 0
    factor = 0.1 * k_scale.double()[:, None]
    for b in [0, 1, 2, 3, 4, 5, 30, 60, 94, 95, 96]:
        n = nblk[b]
        assert torch.all(scores[b, :, n:] == -7.0)
        if n == 0:
            continue
        bd = bounds[tab[b, :n].long()].double()
        best, mass = None, None
        for h in range(per):
            qh = q[b].view(hkv, per, d)[:, h].double()
            s = torch.maximum(qh[:, None] * bd[:, :, 0].transpose(0, 1), qh[:, None] * bd[:, :, 1].transpose(0, 1)).sum(-1)
            m = (qh.abs()[:, None] * bd.abs().amax(2).transpose(0, 1)).sum(-1)
            best, mass = (s, m) if best is None else (torch.maximum(best, s), torch.maximum(mass, m))
        # (the limit of test_scores: 2 D products summed, the factors' roundings)
        assert torch.all((scores[b, :, :n].double() - best * factor).abs() <= mass * factor * (2 * d + 4) * 2.0 ** -23)
    # bad ids score -infinity, their neighbours as before
    before = scores.clone()
    tab[2, 77], tab[2, 78] = nb, -3
    call()
    assert int(err.item()) == 4 and torch.all(scores[2, :, 77:79] == float("-inf"))
    scores[2, :, 77:79] = before[2, :, 77:79]
    assert torch.equal(scores, before)


def test_scores_bound_the_logits(pkv):
    case = Case([3000], hq=8, hkv=1, seed=5)
    bounds = torch.zeros((case.nb, 1, 2, 128), dtype=torch.bfloat16, device="cuda")
    run_bounds(pkv, case, bounds)
    scores = torch.zeros((1, 1, case.width), device="cuda")
    pkv.pkv_block_scores(case.q, bounds, case.tab, case.lens, scores, scale=case.scale, max_context_len=3000)
    k = case.values(0)[case.tab_h[0], 0].reshape(-1, 128)[:3000]
    logits = (case.q[0].double().cpu().numpy() @ k.T).max(0) * case.scale
    top = np.array([logits[i:i + 16].max() for i in range(0, 3000, 16)])
    assert np.all(scores[0, 0].cpu().numpy() >= top - 1e-4)


def test_scores_device_errors(pkv):
    for what in ("id", "len", "negative"):
        case = Case([100, 40], seed=6)
        bounds = torch.ones((case.nb, 2, 2, 128), dtype=torch.bfloat16, device="cuda")
        scores = torch.zeros((2, 2, case.width), device="cuda")
        if what == "id":
            case.tab[0, 3] = case.nb
        else:
            case.lens[1] = 101 if what == "len" else -4
        pkv.pkv_block_scores(case.q, bounds, case.tab, case.lens, scores, scale=1.0, max_context_len=100,
                             err_flag=case.err)
        torch.cuda.synchronize()
        assert int(case.err.item()) == 4
        if what == "id":
            assert torch.all(scores[0, :, 3] == float("-inf")) and torch.isfinite(scores[0, :, 4]).all()


# ---------------------------------------------------------------------------
# selection
# ---------------------------------------------------------------------------
def run_select(pkv, scores, lens, budget, first, last):
    b, h, _ = scores.shape
    out = torch.full((b, h, budget), -9, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pkv.pkv_select_blocks(scores, torch.tensor(lens, dtype=torch.int32, device="cuda"), out, num_first=first,
                          num_last=last, err_flag=err)
    torch.cuda.synchronize()
    return out.cpu().numpy(), int(err.item())


KINDS = ["normal", "coarse", "equal", "special", "spread", "signs"]


def make_scores(kind, shape, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g)
    if kind == "coarse":
        x = (x * 2).round() / 2
    elif kind == "equal":
        x = torch.full(shape, 1.25)
    elif kind == "special":
        x[torch.rand(shape, generator=g) < 0.2] = float("-inf")
        x[torch.rand(shape, generator=g) < 0.05] = float("inf")
        x[torch.rand(shape, generator=g) < 0.02] = float("nan")
    elif kind == "spread":
        x = x * torch.exp2(torch.randint(-140, 120, shape, generator=g).float())
    elif kind == "signs":
        x = torch.where(torch.rand(shape, generator=g) < 0.5, 0.0, -0.0) * torch.ones(shape)
        x[torch.rand(shape, generator=g) < 0.1] = 1e-45
    return x


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("budget,first,last", [(1, 0, 0), (1, 0, 1), (7, 1, 2), (64, 4, 8), (300, 0, 0), (5, 3, 2)])
def test_select(pkv, kind, budget, first, last):
    lens = [0, 1, 16 * budget, 16 * budget + 1, 16 * budget + 40, 5000, 9999, 40000]
    width = 2501
    scores = make_scores(kind, (len(lens), 3, width), budget)
    got, err = run_select(pkv, scores.cuda(), lens, budget, first, last)
    assert err == 0
    for b, n in enumerate(lens):
        for g in range(3):
            want = osp.select_blocks(scores[b, g].numpy(), -(-n // 16), first, last, budget)
            want = want + [-1] * (budget - len(want))
            assert got[b, g].tolist() == want, (b, g, n)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("budget", [1, 60, 255, 256, 700, 4096])
def test_select_among_thousands(pkv, kind, budget):
    lens = [16 * 4098, 16 * 6001 - 5, 16 * 8197, 16 * 8210, 16 * 17000]
    scores = make_scores(kind, (len(lens), 2, 17003), budget)
    got, err = run_select(pkv, scores.cuda(), lens, budget + 3, 1, 2)
    assert err == 0
    for b, n in enumerate(lens):
        for g in range(2):
            want = osp.select_blocks(scores[b, g].numpy(), -(-n // 16), 1, 2, budget + 3)
            assert got[b, g].tolist() == want + [-1] * (budget + 3 - len(want)), (b, g)


def test_select_many_blocks_and_units(pkv):
    # more blocks than one pass's threads hold, by a wide margin; and many pairs
    n = 16 * 70000 + 3
    scores = make_scores("coarse", (1, 2, 70005), 1)
    got, err = run_select(pkv, scores.cuda(), [n], 1000, 1, 1)
    assert err == 0
    for g in range(2):
        assert got[0, g].tolist() == osp.select_blocks(scores[0, g].numpy(), 70001, 1, 1, 1000)
    scores = make_scores("normal", (700, 5, 40), 2)
    lens = [(37 * b) % 640 + 1 for b in range(700)]
    got, err = run_select(pkv, scores.cuda(), lens, 9, 1, 1)
    for b in range(0, 700, 31):
        want = osp.select_blocks(scores[b, 4].numpy(), -(-lens[b] // 16), 1, 1, 9)
        assert got[b, 4].tolist() == want + [-1] * (9 - len(want))


def test_select_device_errors(pkv):
    scores = make_scores("normal", (2, 1, 30), 3).cuda()
    got, err = run_select(pkv, scores, [481, 100], 4, 0, 1)
    assert err == 4 and got[0, 0, -1] == 29           # the context is clamped to the table
    got, err = run_select(pkv, scores, [-1, 100], 4, 0, 1)
    assert err == 4 and got[0, 0].tolist() == [-1] * 4


# ---------------------------------------------------------------------------
# attention over lists
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype,kv", [("f16", None), ("bf16", None), ("bf16", "e4m3"), ("f16", "e5m2")])
@pytest.mark.parametrize("hq,hkv,d", [(3, 3, 128), (4, 2, 64), (8, 2, 128), (8, 1, 64), (16, 2, 128)])
@pytest.mark.parametrize("budget", [1, 5, 40])
def test_sparse_attention(pkv, dtype, kv, hq, hkv, d, budget):
    case = Case([0, 1, 16, 31, 64, 65, 500, 1601], hq=hq, hkv=hkv, d=d, dtype=dtype, kv=kv, seed=budget + d, wide=1)
    sel = random_lists(case, budget, seed=budget)
    out = case.attention(pkv, sel)
    assert int(case.err.item()) == 0
    case.check_attention(out, sel)


@pytest.mark.parametrize("hq,hkv,d,kv", [(4, 4, 128, None), (8, 2, 128, None), (8, 2, 64, "e4m3"), (8, 2, 128, "e4m3")])
def test_skipped_unordered_and_repeated_entries(pkv, hq, hkv, d, kv):
    case = Case([1000, 700, 90, 3], hq=hq, hkv=hkv, d=d, kv=kv, seed=11)
    sel = random_lists(case, 24, seed=1, ragged=True)
    sel[1] = sel[1].flip(-1)                          # any order, -1 in front
    sel[0, 0, :4] = 62                                # the same block (a partial one) four times
    sel[0, hkv - 1] = -1                              # a pair with nothing listed
    sel[2, :, 6:] = 12345                             # behind the counted entries: never read
    out = case.attention(pkv, sel)
    assert int(case.err.item()) == 0
    per = hq // hkv
    assert torch.all(out[0, -per:] == 0)
    case.check_attention(out, sel)


def test_every_block_listed_equals_dense_decode(pkv):
    case = Case([777, 16, 0, 2048], seed=12)
    sel = random_lists(case, case.width, seed=2)
    out = case.attention(pkv, sel)
    dense = torch.empty_like(case.q)
    ws = torch.empty(pkv.pkv_decode_workspace_bytes(4, 8, 2, 128, case.width, 2048), dtype=torch.uint8, device="cuda")
    pkv.pkv_paged_decode_attention(case.q, case.kc, case.vc, case.tab, case.lens, dense, scale=case.scale,
                                   max_context_len=2048, workspace=ws)
    torch.cuda.synchronize()
    assert torch.equal(out, dense)                    # the same split, the same order


def test_attention_device_errors(pkv):
    case = Case([1000, 700], seed=13)
    sel = random_lists(case, 10, seed=3)
    sel[0, 0, 2] = 63                                 # behind the context's 63 blocks
    out = case.attention(pkv, sel)
    assert int(case.err.item()) == 4 and torch.isfinite(out).all()
    sel[0, 0, 2] = -1
    case.err.zero_()
    case.check_attention(out, sel)                    # skipped
    case.tab[0, 62] = case.nb                         # a bad id
    out = case.attention(pkv, sel)
    assert int(case.err.item()) == 4
    small = torch.empty(64, dtype=torch.uint8, device="cuda")
    with pytest.raises(pkv.PkvError) as e:
        case.attention(pkv, sel, ws=small)
    assert e.value.status == 6
    case = Case([1000, 700], seed=13)
    case.lens[1] = 16 * case.width + 1                # a context longer than its table
    out = case.attention(pkv, random_lists(case, 10, seed=3))
    assert int(case.err.item()) == 4


@pytest.mark.parametrize("n", [2 ** 31 - 1, 2 ** 31 - 16])
def test_lengths_at_the_end_of_int32(pkv, n):
    # a context as long is clamped to its table and reported, in every step
    case = Case([1000, 700], seed=14)
    bounds = torch.zeros((case.nb, 2, 2, 128), dtype=torch.bfloat16, device="cuda")
    case.lens[1] = n
    run_bounds(pkv, case, bounds)
    assert int(case.err.item()) == 4
    scores = torch.zeros((2, 2, case.width), device="cuda")
    case.err.zero_()
    pkv.pkv_block_scores(case.q, bounds, case.tab, case.lens, scores, scale=1.0, max_context_len=2 ** 31 - 1,
                         err_flag=case.err)
    torch.cuda.synchronize()
    assert int(case.err.item()) == 4 and torch.isfinite(scores[0]).all()
    got, err = run_select(pkv, scores, [1000, n], 4, 1, 1)
    assert err == 4 and got[1, 0, 0] == 0 and got[1, 0, -1] == case.width - 1
    sel = random_lists(case, 10, seed=3)
    case.err.zero_()
    case.attention(pkv, sel)
    assert int(case.err.item()) == 4


def test_binding_refuses_shapes_that_do_not_fit(pkv):
    case = Case([100], seed=14)
    sel = torch.zeros((1, 3, 4), dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        case.attention(pkv, sel)
    with pytest.raises(ValueError):
        pkv.pkv_select_blocks(torch.zeros((1, 2, 7), device="cuda"), case.lens, sel)
    with pytest.raises(ValueError):
        run_bounds(pkv, case, torch.zeros((case.nb, 2, 128), dtype=torch.bfloat16, device="cuda"))
    bounds = torch.zeros((case.nb, 2, 2, 128), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        pkv.pkv_block_scores(case.q, bounds, case.tab, case.lens, torch.zeros((1, 2, 9), device="cuda"), scale=1.0,
                             max_context_len=100)
    lists = torch.zeros((1, 2, 4), dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError):       # index types and strides
        case.attention(pkv, lists.long())
    with pytest.raises(TypeError):
        case.attention(pkv, torch.zeros((1, 2, 8), dtype=torch.int32, device="cuda")[..., ::2])
    with pytest.raises(ValueError):
        pkv.pkv_select_blocks(torch.zeros((1, 2, 14), device="cuda")[..., ::2], case.lens, lists)
    with pytest.raises(TypeError):
        pkv.pkv_select_blocks(torch.zeros((1, 2, 7), device="cuda"), case.lens.long(), lists)
    q = case.q
    case.q = torch.zeros((1, 8, 256), dtype=q.dtype, device="cuda")[..., ::2]
    with pytest.raises(ValueError):
        case.attention(pkv, lists)
    case.q = q
    with pytest.raises(TypeError):
        pkv.pkv_block_scores(case.q, bounds.half(), case.tab, case.lens, torch.zeros((1, 2, 7), device="cuda"),
                             scale=1.0, max_context_len=100)


# ---------------------------------------------------------------------------
# the operators together, as a decode step runs them
# ---------------------------------------------------------------------------
def step_buffers(pkv, case, budget):
    b = len(case.lens_h)
    return dict(
        bounds=torch.zeros((case.nb, case.hkv, 2, case.d), dtype=case.q.dtype, device="cuda"),
        scores=torch.zeros((b, case.hkv, case.width), device="cuda"),
        sel=torch.zeros((b, case.hkv, budget), dtype=torch.int32, device="cuda"),
        out=torch.zeros_like(case.q), pos=case.lens - 1, slots=torch.zeros(b, dtype=torch.int64, device="cuda"),
        one=torch.ones(b, dtype=torch.int32, device="cuda"),
        ws=torch.empty(pkv.pkv_decode_workspace_bytes(b, case.hq, case.hkv, case.d, budget, 16 * budget),
                       dtype=torch.uint8, device="cuda"))


def sparse_step(pkv, case, buf, q, k, v, turns, q_out):
    """rope and append of the newest token, its block's bounds, scores,
    selection, attention."""
    top = int(case.lens_h.max())
    pkv.pkv_slot_mapping(case.tab, case.lens, buf["slots"], num_blocks=case.nb, position_offset=-1)
    pkv.pkv_rope_append(q, k, v, buf["pos"], buf["slots"], turns, q_out, case.kc, case.vc)
    pkv.pkv_kv_block_bounds(case.kc, case.tab, case.lens, buf["bounds"], new_lens=buf["one"], max_new_len=1)
    pkv.pkv_block_scores(q_out, buf["bounds"], case.tab, case.lens, buf["scores"], scale=case.scale, max_context_len=top)
    pkv.pkv_select_blocks(buf["scores"], case.lens, buf["sel"], num_first=1, num_last=2)
    pkv.pkv_paged_decode_attention_sparse(q_out, case.kc, case.vc, case.tab, case.lens, buf["sel"], buf["out"],
                                          scale=case.scale, workspace=buf["ws"])


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_a_decode_step_end_to_end(pkv, dtype):
    case = Case([2000, 17, 900, 513], hq=8, hkv=2, dtype=dtype, seed=15)
    g = torch.Generator().manual_seed(1)
    qkv = torch.randn((4, 12, 128), generator=g).to(gu.TORCH_16[dtype]).cuda()
    q, k, v = qkv[:, :8], qkv[:, 8:10], qkv[:, 10:]
    buf = step_buffers(pkv, case, 12)
    turns = torch.from_numpy(pkv.pkv_rope_plan(128)[0]).cuda()
    # the cache before the step holds all but the newest token
    older = torch.from_numpy(case.lens_h - 1).cuda()
    pkv.pkv_kv_block_bounds(case.kc, case.tab, older, buf["bounds"], max_new_len=2000)
    q_out = torch.empty_like(case.q)
    sparse_step(pkv, case, buf, q, k, v, turns, q_out)
    torch.cuda.synchronize()
    # the bounds now are those of the cache as it is, whole
    assert np.array_equal(buf["bounds"].double().cpu().numpy(),
                          expected_bounds(case, torch.zeros_like(buf["bounds"])))
    # the lists are those of the scores, and the attention is over the lists
    sc = buf["scores"].cpu().numpy()
    for b, n in enumerate(case.lens_h):
        for h in range(2):
            want = osp.select_blocks(sc[b, h], -(-int(n) // 16), 1, 2, 12)
            assert buf["sel"][b, h].tolist() == want + [-1] * (12 - len(want))
    case.q = q_out
    case.check_attention(buf["out"], buf["sel"])
    # the same step captured and replayed, and on another stream: the same bits
    ref = {n: buf[n].clone() for n in ("bounds", "scores", "sel", "out")}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sparse_step(pkv, case, buf, q, k, v, turns, q_out)
    side = torch.cuda.Stream()
    for run in (graph.replay, lambda: sparse_step(pkv, case, buf, q, k, v, turns, q_out)):
        for n in ("scores", "out"):
            buf[n].fill_(float("nan"))
        buf["sel"].fill_(99)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            run()
        torch.cuda.synchronize()
        for n, t in ref.items():
            live = ~torch.isnan(buf[n].float())
            assert torch.equal(buf[n][live], t[live]) and (n == "scores" or bool(live.all()))


@pytest.mark.parametrize("b,hkv", [(3, 2), (64, 8)])
def test_bounds_right_behind_fused_steps(pkv, b, hkv):
    # launches that start early, one behind the other: a step appends, the bounds read its rows
    steps, d, hq = 24, 128, 4 * hkv
    rng = np.random.default_rng(33)
    start = rng.integers(1, 700, size=b).astype(np.int32)
    width = (int(start.max()) + steps + 15) // 16
    nb = b * width
    g = torch.Generator(device="cuda").manual_seed(33)
    kc, vc = (torch.randn((nb, hkv, 16, d), generator=g, device="cuda").bfloat16() for _ in range(2))
    tab = torch.randperm(nb, generator=g, device="cuda").to(torch.int32).view(b, width)
    lens = [torch.from_numpy(start + i).cuda() for i in range(steps + 1)]
    q = torch.randn((b, hq, d), generator=g, device="cuda").bfloat16()
    new = torch.randn((2, steps, b, hkv, d), generator=g, device="cuda").bfloat16()
    bounds = torch.zeros((nb, hkv, 2, d), dtype=torch.bfloat16, device="cuda")
    one, out = torch.ones(b, dtype=torch.int32, device="cuda"), torch.empty_like(q)
    top = int(start.max()) + steps
    ws = torch.empty(pkv.pkv_decode_workspace_bytes(b, hq, hkv, d, width, top), dtype=torch.uint8, device="cuda")
    pkv.pkv_kv_block_bounds(kc, tab, lens[0], bounds, max_new_len=top)
    torch.cuda.synchronize()
    for i in range(steps):
        pkv.pkv_paged_decode_step(q, new[0, i], new[1, i], kc, vc, tab, lens[i + 1], out, scale=d ** -0.5,
                                  max_context_len=top, workspace=ws)
        pkv.pkv_kv_block_bounds(kc, tab, lens[i + 1], bounds, new_lens=one, max_new_len=1)
    torch.cuda.synchronize()
    k, got, ids = kc.double().cpu().numpy(), bounds.double().cpu().numpy(), tab.cpu().numpy()
    for s in range(b):
        n = int(start[s]) + steps
        for i in range(-(-n // 16)):
            rows = k[ids[s, i], :, :min(16, n - 16 * i)]
            assert np.array_equal(got[ids[s, i], :, 0], rows.min(1)) and np.array_equal(got[ids[s, i], :, 1], rows.max(1))


def test_scores_from_two_threads(pkv):
    # two shapes of the flat form at a time: neither call takes the other's shared-memory limit
    import threading
    g = torch.Generator(device="cuda").manual_seed(31)

    def make(b, hq, hkv, d, width, nb=500):
        q = torch.randn((b, hq, d), generator=g, device="cuda").bfloat16()
        bounds = torch.randn((nb, hkv, 2, d), generator=g, device="cuda").bfloat16()
        tab = torch.randint(0, nb, (b, width), generator=g, device="cuda", dtype=torch.int32)
        lens = torch.randint(1, 16 * width + 1, (b,), generator=g, device="cuda", dtype=torch.int32)
        return (q, bounds, tab, lens), *(torch.zeros((b, hkv, width), device="cuda") for _ in range(2))
    work = [make(40, 32, 8, 128, 1024), make(800, 4, 1, 64, 600)]

    def call(item, out, stream=None):
        pkv.pkv_block_scores(*item[0], out, scale=0.1, max_context_len=16 * out.shape[2], stream=stream)
    failures = []

    def loop(item, stream):
        try:
            for _ in range(200):
                call(item, item[2], stream)
        except Exception as e:   # noqa: BLE001 (reported below)
            failures.append(e)
    for item in work:
        call(item, item[1])
    torch.cuda.synchronize()
    threads = [threading.Thread(target=loop, args=(item, torch.cuda.Stream())) for item in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failures, failures[0]
    assert all(torch.equal(want, got) for _, want, got in work)


def test_two_streams_each_with_its_workspace(pkv):
    a, b = Case([4000, 1300, 20], seed=20), Case([900] * 9, hq=16, hkv=4, dtype="f16", seed=21)
    jobs = []
    for case in (a, b):
        sel = random_lists(case, 30, seed=4)
        n = pkv.pkv_decode_workspace_bytes(len(case.lens_h), case.hq, case.hkv, case.d, 30, 480)
        jobs.append((case, sel, case.attention(pkv, sel), torch.empty_like(case.q),
                     torch.empty(n, dtype=torch.uint8, device="cuda"), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for case, sel, _, out, ws, stream in jobs:
            pkv.pkv_paged_decode_attention_sparse(case.q, case.kc, case.vc, case.tab, case.lens, sel, out,
                                                  scale=case.scale, workspace=ws, stream=stream)
    torch.cuda.synchronize()
    for _, _, ref, out, _, _ in jobs:
        assert torch.equal(out, ref)


def test_far_blocks_of_a_large_pool(pkv):
    # slabs past 4 GiB of the cache: byte offsets need 64 bits
    hkv, d, nb = 8, 128, 140000                       # 32 KiB a block: 4.6 GB
    kc = torch.zeros((nb, hkv, 16, d), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    ids = torch.tensor([[nb - 1, 3, nb - 7]], dtype=torch.int32)
    g = torch.Generator().manual_seed(2)
    rows = torch.randn((2, 3, hkv, 16, d), generator=g).to(torch.bfloat16).cuda()
    kc[ids[0].long()], vc[ids[0].long()] = rows[0], rows[1]
    case = Case([41], hq=16, hkv=hkv, seed=16)
    case.kc, case.vc, case.tab, case.tab_h, case.nb = kc, vc, ids.cuda(), ids.numpy(), nb
    bounds = torch.zeros((nb, hkv, 2, d), dtype=torch.bfloat16, device="cuda")
    run_bounds(pkv, case, bounds)
    assert torch.equal(bounds[ids[0, 0].long(), :, 1], rows[0, 0].amax(1))
    assert torch.equal(bounds[ids[0, 2].long(), :, 0], rows[0, 2][:, :9].amin(1))
    scores = torch.zeros((1, hkv, 3), device="cuda")
    pkv.pkv_block_scores(case.q, bounds, case.tab, case.lens, scores, scale=case.scale, max_context_len=41)
    assert (scores != 0).all()
    sel = torch.tensor([0, 2], dtype=torch.int32, device="cuda").expand(1, hkv, 2).contiguous()
    out = case.attention(pkv, sel)
    per = 2
    for h in range(16):
        pos = osp.token_positions([0, 2], 41)
        k = rows[0][pos // 16, h // per, pos % 16].double().cpu().numpy()
        v = rows[1][pos // 16, h // per, pos % 16].double().cpu().numpy()
        ref, lim = attn_limits.attend(case.q[0, h].double().cpu().numpy(), k, v, case.scale, "bf16")
        assert np.all(np.abs(out[0, h].double().cpu().numpy() - ref) <= lim)
