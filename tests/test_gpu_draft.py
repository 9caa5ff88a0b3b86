"""Drafted tokens on the GPU against float64: the plan and the commit exactly,
attention within limits taken from the arithmetic."""
import numpy as np
import pytest
import torch

from oracle import draft as od
from tests import attn_limits
from tests import gpu_util as gu

pytestmark = pytest.mark.gpu

FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
OOB = 4


@pytest.fixture(scope="module")
def pkv():
    import __graft_entry__ as g
    g.build()
    import paged_kv_cache_153_gb300 as m
    return m


def rand_tree(rng, n, back=9):
    i = np.arange(n)
    return np.maximum(i - rng.integers(1, back + 1, size=n), -1).astype(np.int32)


class Case:
    """Contexts of base[b] tokens and new[b] drafted ones; cached rows behind a
    context are NaN."""

    def __init__(self, base, new, *, hq=8, hkv=2, d=128, dtype="bf16", kv=None, seed=0, seen=None, extra=0, wide=0,
                 spare=2):
        rng = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        self.base, self.new = np.asarray(base), np.asarray(new)
        self.hq, self.hkv, self.d, self.dtype, self.kv = hq, hkv, d, dtype, kv
        ctx = self.base + self.new
        self.cu = np.concatenate([[0], np.cumsum(self.new)]).astype(np.int32)
        self.tokens = int(self.cu[-1]) + extra
        self.max_nodes = max(1, int(self.new.max()))
        self.words = -(-self.max_nodes // 64)
        nblk = -(-ctx // 16)
        self.nb, self.width = int(nblk.sum()) + spare, max(1, int(nblk.max())) + wide
        ids = rng.permutation(self.nb).astype(np.int32)
        self.tab = np.full((len(ctx), self.width), -1, dtype=np.int32)
        at = 0
        for b, n in enumerate(nblk):
            self.tab[b, :n] = ids[at:at + n]
            at += n
        self.parents = [rand_tree(rng, int(n)) for n in self.new]
        self.seen = [od.ancestors(p) for p in self.parents] if seen is None else seen
        mask = np.full((self.tokens, self.words), -1, dtype=np.int64)          # (behind the last one: not read)
        for b, s in enumerate(self.seen):
            mask[self.cu[b]:self.cu[b + 1]] = od.mask_words(s, self.words)
        t = gu.TORCH_16[dtype]
        kc, vc = (torch.randn((self.nb, hkv, 16, d), generator=g) for _ in range(2))
        dead = torch.ones((self.nb, 16), dtype=torch.bool)
        for b, n in enumerate(ctx):
            for p in range(int(n)):
                dead[int(self.tab[b, p // 16]), p % 16] = False
        if kv:
            self.ks, self.vs = (torch.rand(hkv, generator=g) + 0.5 for _ in range(2))
            kc, vc = (x.to(FP8[kv]).view(torch.uint8) for x in (kc, vc))
            nan = 0x7F
        else:
            kc, vc, nan = kc.to(t), vc.to(t), float("nan")
        for x in (kc, vc):
            x.transpose(1, 2)[dead] = nan
        self.kc_h, self.vc_h = kc, vc
        self.q_h = torch.randn((self.tokens, hq, d), generator=g).to(t)
        self.ctx, self.scale, self.mask_h = ctx.astype(np.int32), d ** -0.5, mask

    def upload(self):
        c = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()   # noqa: E731
        self.kc, self.vc, self.q = self.kc_h.cuda(), self.vc_h.cuda(), self.q_h.cuda()
        self.lens, self.tables, self.cu_d, self.mask = c(self.ctx), c(self.tab), c(self.cu), c(self.mask_h)
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.out = torch.full_like(self.q, 7.0)
        return self

    def attend(self, pkv, **over):
        self.upload()
        n = pkv.pkv_tree_workspace_bytes(len(self.ctx), self.tokens, self.hq, self.hkv, self.d, self.max_nodes)
        ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")            # (NaN states)
        kw = dict(scale=self.scale, max_context_len=int(self.ctx.max()), max_nodes=self.max_nodes, workspace=ws,
                  err_flag=self.err)
        kw.update(over)
        if self.kv:
            call = pkv.pkv_paged_tree_attention_fp8 if self.kv == "e4m3" else pkv.pkv_paged_tree_attention_e5m2
            call(self.q, self.kc, self.vc, self.ks.cuda(), self.vs.cuda(), self.tables, self.lens, self.cu_d,
                 self.mask, self.out, **kw)
        else:
            pkv.pkv_paged_tree_attention(self.q, self.kc, self.vc, self.tables, self.lens, self.cu_d, self.mask,
                                         self.out, **kw)
        torch.cuda.synchronize()
        return self.out

    def rows(self, b, g):
        """K and V [ctx, d] of a KV head in float64."""
        p = np.arange(int(self.ctx[b]))
        ids, off = torch.from_numpy(self.tab[b][p // 16].astype(np.int64)), torch.from_numpy(p % 16)
        out = []
        for x, sc in ((self.kc_h, "ks"), (self.vc_h, "vs")):
            r = x[ids, g, off]
            r = r.view(FP8[self.kv]).double() * getattr(self, sc)[g].double() if self.kv else r.double()
            out.append(r.numpy())
        return out

    def check(self, got, seqs=None, columns=None):
        got = got.double().cpu().numpy()
        per, worst = self.hq // self.hkv, 0.0
        for b in (range(len(self.ctx)) if seqs is None else seqs):
            if self.new[b] == 0:
                continue
            full = od.tree_seen(int(self.base[b]), self.seen[b])
            for g in range(self.hkv):
                k, v = self.rows(b, g)
                for i in range(int(self.new[b])):
                    at = np.flatnonzero(full[i])
                    for h in range(g * per, (g + 1) * per):
                        q = self.q_h[self.cu[b] + i, h].double().numpy()
                        ref, lim = attn_limits.attend(q, k[at], v[at], self.scale, self.dtype, "f16" if self.kv else None)
                        x = got[self.cu[b] + i, h]
                        if columns is not None:
                            ref, lim, x = ref[columns], lim[columns], x[columns]
                        bad = ~(np.abs(x - ref) <= lim)
                        assert not bad.any(), (b, i, h, float(np.abs(x - ref).max()), float(lim.min()))
                        worst = max(worst, float((np.abs(x - ref) / np.maximum(lim, 1e-30)).max()))
        return worst


# ---- attention ----
@pytest.mark.parametrize("dtype,kv", [("f16", None), ("bf16", None), ("f16", "e4m3"), ("bf16", "e4m3"),
                                      ("f16", "e5m2"), ("bf16", "e5m2")])
@pytest.mark.parametrize("hq,hkv,d", [(2, 2, 64), (4, 2, 128), (8, 2, 64), (8, 1, 128)])
def test_contexts_and_trees_of_every_edge(pkv, dtype, kv, hq, hkv, d):
    base = [0, 1, 15, 16, 100, 127, 128, 129, 250, 600, 40]
    new = [5, 1, 2, 16, 33, 1, 8, 30, 7, 17, 0]
    c = Case(base, new, hq=hq, hkv=hkv, d=d, dtype=dtype, kv=kv, seed=hq + d)
    c.check(c.attend(pkv))
    assert int(c.err.item()) == 0


@pytest.mark.parametrize("dtype,kv", [("f16", None), ("bf16", None), ("bf16", "e4m3")])
@pytest.mark.parametrize("hq,d,new", [(1, 64, 256), (2, 128, 129), (8, 128, 70), (4, 64, 200), (8, 64, 256)])
def test_many_drafted_tokens(pkv, dtype, kv, hq, d, new):
    # units of two row tiles, and several of them; masks of one to four words
    c = Case([37, 0, 300], [new, new // 2, 3], hq=hq, hkv=1, d=d, dtype=dtype, kv=kv, seed=new)
    c.check(c.attend(pkv))
    assert int(c.err.item()) == 0


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_one_long_context_is_split(pkv, dtype):
    c = Case([5000], [6], hq=2, hkv=1, d=64, dtype=dtype, seed=3)
    c.check(c.attend(pkv))


@pytest.mark.parametrize("kv", [None, "e4m3", "e5m2"])
def test_any_set_of_drafted_tokens_and_none(pkv, kv):
    # rows that see themselves or not, later tokens or not, nothing at all
    rng = np.random.default_rng(0)
    seen = [rng.random((n, n)) < 0.5 for n in (9, 70, 130)]
    seen[0][3] = False
    seen[1][::7] = False
    c = Case([0, 20, 128], [9, 70, 130], hq=2, hkv=2, d=64, kv=kv, seed=1, seen=seen)
    out = c.attend(pkv)
    c.check(out)
    assert not out[3].any()                                    # no context, no drafted token: 0


@pytest.mark.parametrize("dtype,kv,bad", [("bf16", None, float("nan")), ("bf16", None, float("inf")),
                                          ("f16", None, float("-inf")), ("bf16", "e4m3", 0x7F), ("f16", "e5m2", 0xFC)])
@pytest.mark.parametrize("base", [0, 115])
def test_rows_that_are_not_seen_change_nothing(pkv, dtype, kv, bad, base):
    # token 4 is seen by itself alone, token 7 by none, token 20 by some
    n = 24
    seen = np.tril(np.ones((n, n), bool))
    seen[:, [4, 7]] = False
    seen[4, 4] = True
    seen[22:, 20] = False
    c = Case([base, 300], [n, 2], hq=8, hkv=2, d=128, dtype=dtype, kv=kv, seed=5, seen=[seen, np.eye(2, dtype=bool)])
    columns = [3, 64, 127]
    for j in (4, 7, 20):
        p = base + j
        blk, off = int(c.tab[0, p // 16]), p % 16
        c.vc_h[blk, :, off, columns] = bad
        if j == 7:
            c.kc_h[blk, :, off, :] = bad
    out = c.attend(pkv)
    assert int(c.err.item()) == 0
    free = [x for x in range(c.d) if x not in columns]
    c.check(out, columns=free)
    hit = ~torch.isfinite(out[:n][:, :, columns].float()).all(2).all(1).cpu().numpy()
    assert list(np.flatnonzero(hit)) == [4, 20, 21]
    clean = np.array([i for i in range(n) if i not in (4, 20, 21)])
    got = out.double().cpu().numpy()[clean][:, :, columns]
    for b_i, i in enumerate(clean):                            # the columns themselves, where the tokens are not seen
        for g in range(2):
            k, v = c.rows(0, g)
            at = np.flatnonzero(od.tree_seen(base, seen)[i])
            for h in range(4 * g, 4 * g + 4):
                ref, lim = attn_limits.attend(c.q_h[i, h].double().numpy(), k[at], v[at], c.scale, dtype,
                                              "f16" if kv else None)
                assert (np.abs(got[b_i, h] - ref[columns]) <= lim[columns]).all()


@pytest.mark.parametrize("dtype,kv", [("bf16", None), ("f16", None), ("bf16", "e5m2")])
def test_rows_that_are_not_finite_in_many_short_sequences(pkv, dtype, kv):
    # tens of one-tile units a thread block, each with a token that is not finite
    new = [2 + b % 3 for b in range(400)]
    c = Case([10 + b % 50 for b in range(400)], new, hq=8, hkv=8, d=64, dtype=dtype, kv=kv, seed=9)
    for b in range(0, 400, 2):
        p = int(c.ctx[b]) - 1 - (b // 2) % 2
        c.vc_h[int(c.tab[b, p // 16]), :, p % 16] = 0x7C if kv else float("inf")
    for _ in range(20):
        fine = torch.isfinite(c.attend(pkv).float()).cpu().numpy()
        for b in range(400):
            want = np.ones(new[b], bool)
            if b % 2 == 0:
                want &= ~c.seen[b][:, new[b] - 1 - (b // 2) % 2]
            assert (fine[c.cu[b]:c.cu[b + 1]] == want[:, None, None]).all(), b
    assert int(c.err.item()) == 0


def test_every_fp8_code(pkv):
    # every finite code of both formats as K and as V, denormals among them
    for kv in FP8:
        c = Case([250], [6], hq=4, hkv=1, d=64, dtype="f16", kv=kv, seed=8)
        codes = torch.arange(256, dtype=torch.int16).to(torch.uint8)
        codes = codes[torch.isfinite(codes.view(FP8[kv]).float())]
        if kv == "e5m2":
            codes = codes[codes.view(FP8[kv]).float().abs() < 16]
        for p in range(256):
            blk, off = int(c.tab[0, p // 16]), p % 16
            roll = torch.roll(codes, 5 * p)
            c.kc_h[blk, 0, off], c.vc_h[blk, 0, off] = roll[:64], roll[64:128]
        c.ks[0], c.vs[0] = 2.0 ** -6, 0.5
        c.check(c.attend(pkv))


def test_tokens_behind_the_last_sequence_stay(pkv):
    c = Case([20, 5], [6, 0], extra=9)
    out = c.attend(pkv)
    c.check(out)
    assert bool((out[6:] == 7.0).all()) and int(c.err.item()) == 0


def test_the_launch_size_does_not_matter(pkv):
    c = Case([700, 30], [5, 9], hq=8, hkv=2)
    a = c.attend(pkv).clone()
    for mx in (0, 1, 700, 1 << 20):
        c.check(c.attend(pkv, max_context_len=mx))
    assert torch.equal(a, c.attend(pkv))                       # the same call, the same bits


def test_bad_sequences_are_skipped_and_flagged(pkv):
    base, new = [40, 40, 40], [5, 6, 7]
    for kind in ("ctx", "table", "nodes", "negative"):
        c = Case(base, new, hq=8, hkv=2)
        over = {}
        if kind == "ctx":
            c.ctx[1] = 5
        elif kind == "table":
            c.ctx[1] = 16 * c.width + 1
        elif kind == "negative":
            c.ctx[1] = -3
        else:
            over["max_nodes"] = 5
        out = c.attend(pkv, **over)
        assert int(c.err.item()) == OOB, kind
        c.base, c.ctx = np.asarray(base), (np.asarray(base) + np.asarray(new)).astype(np.int32)
        left = [0] if kind == "nodes" else [0, 2]
        c.check(out, seqs=left)
        assert bool((out[5:11] == 7.0).all()), kind


@pytest.mark.parametrize("cu", [[0, 5, 3, 9], [0, 5, 11, 40], [-1, 5, 11, 18]])
def test_bad_offsets_are_flagged(pkv, cu):
    c = Case([40, 40, 40], [5, 6, 7], hq=8, hkv=2)
    c.cu = np.asarray(cu, np.int32)
    c.attend(pkv)
    assert int(c.err.item()) == OOB


@pytest.mark.parametrize("kv", [None, "e4m3"])
def test_a_bad_table_entry_reads_as_zeros(pkv, kv):
    c = Case([40, 40], [5, 6], hq=8, hkv=2, kv=kv)
    good = int(c.tab[0, 1])
    c.tab[0, 1] = c.nb + 3
    out = c.attend(pkv)
    assert int(c.err.item()) == OOB
    c.tab[0, 1] = good
    c.kc_h[good], c.vc_h[good] = 0, 0
    c.check(out)


def test_a_pool_beyond_32_bit_offsets(pkv):
    hkv, d, nb = 8, 128, 140000                                # 4.6 GB of K
    c = Case([30], [4], hq=8, hkv=hkv, d=d)
    c.upload()
    kc, vc = (torch.zeros((nb, hkv, 16, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ids = torch.arange(c.width, device="cuda") * 7 + nb - 40
    kc[ids], vc[ids] = c.kc[c.tables[0].long()], c.vc[c.tables[0].long()]
    ws = torch.empty(pkv.pkv_tree_workspace_bytes(1, 4, 8, hkv, d, 4), dtype=torch.uint8, device="cuda")
    pkv.pkv_paged_tree_attention(c.q, kc, vc, ids[None].to(torch.int32), c.lens, c.cu_d, c.mask, c.out, scale=c.scale,
                                 max_context_len=34, max_nodes=4, workspace=ws, err_flag=c.err)
    torch.cuda.synchronize()
    assert int(c.err.item()) == 0
    c.check(c.out)
    acc = torch.tensor([[1, 3]], dtype=torch.int32, device="cuda")
    want = vc[ids[33 // 16], :, 33 % 16].clone()
    pkv.pkv_tree_commit(kc, vc, ids[None].to(torch.int32), c.lens, c.cu_d, acc, err_flag=c.err)
    assert int(c.err.item()) == 0 and torch.equal(vc[ids[31 // 16], :, 31 % 16], want)


def test_workspaces_that_are_too_small_are_refused(pkv):
    c = Case([40], [5])
    n = pkv.pkv_tree_workspace_bytes(1, c.tokens, c.hq, c.hkv, c.d, c.max_nodes)
    with pytest.raises(pkv.PkvError) as e:
        c.attend(pkv, workspace=torch.empty(n - 1, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 6
    c.check(c.attend(pkv, workspace=torch.empty(n, dtype=torch.uint8, device="cuda")))


@pytest.mark.parametrize("base,new,hq,hkv,d,seqs", [
    ([20 + 37 * (i % 17) for i in range(700)], [1 + i % 2 for i in range(700)], 2, 2, 64, (0, 1, 16, 333, 699)),
    ([50 * i for i in range(12)], [130, 256, 5, 64, 1, 256, 200, 0, 129, 128, 100, 99], 8, 2, 128, (2, 4, 8, 11)),
])
def test_states_of_many_and_of_few_rows_are_joined(pkv, base, new, hq, hkv, d, seqs):
    # more thread blocks of the merge than the GPU holds at once; four rows a warp
    c = Case(base, new, hq=hq, hkv=hkv, d=d, seed=5)
    c.check(c.attend(pkv), seqs=seqs)
    assert int(c.err.item()) == 0


def test_many_sequences(pkv):
    # the most that one call takes, some without drafted tokens
    rng = np.random.default_rng(4)
    new = rng.integers(0, 4, size=1024)
    c = Case(rng.integers(0, 40, size=1024), new, hq=1, hkv=1, d=64, seed=6)
    out = c.attend(pkv)
    assert int(c.err.item()) == 0
    c.check(out, seqs=list(range(0, 1024, 37)) + [1023])


# ---- plan ----
def run_plan(pkv, parents, cu, tab, ctx, words, nb, tokens):
    c = lambda a, t=torch.int32: torch.from_numpy(np.ascontiguousarray(a)).to(t).cuda()   # noqa: E731
    mask = torch.full((tokens, words), 7, dtype=torch.int64, device="cuda")
    pos = torch.full((tokens,), -9, dtype=torch.int32, device="cuda")
    slots = torch.full((tokens,), -9, dtype=torch.int64, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pkv.pkv_tree_plan(c(parents), c(cu), c(tab), c(ctx), mask, pos, slots, num_blocks=nb, err_flag=err)
    torch.cuda.synchronize()
    return mask.cpu().numpy(), pos.cpu().numpy(), slots.cpu().numpy(), int(err.item())


@pytest.mark.parametrize("back", [1, 3, 300])
@pytest.mark.parametrize("words", [1, 2, 3, 4])
def test_plan(pkv, words, back):
    rng = np.random.default_rng(10 * words + back)
    new = np.array([0, 1, 64 * words, 5, 33, 64 * words - 1, 2])
    base = np.array([10, 0, 100, 15, 16, 31, 1000])
    c = Case(base, new, hq=1, hkv=1, d=64, seed=words, extra=4)
    par = [rand_tree(rng, int(n), back) for n in new]
    mask, pos, slots, err = run_plan(pkv, np.concatenate([*par, [0] * 4]), c.cu, c.tab, c.ctx, words, c.nb, c.tokens)
    assert err == 0
    for b, p in enumerate(par):
        s = od.ancestors(p)
        at = slice(c.cu[b], c.cu[b + 1])
        assert (mask[at] == od.mask_words(s, words)).all()
        assert (pos[at] == base[b] + s.sum(1) - 1).all()
        p = base[b] + np.arange(len(p))
        assert (slots[at] == c.tab[b][p // 16].astype(np.int64) * 16 + p % 16).all()
    assert (mask[-4:] == 7).all() and (pos[-4:] == -9).all() and (slots[-4:] == -9).all()


def test_plan_flags_what_does_not_fit(pkv):
    c = Case([10, 10, 10], [3, 4, 5], hq=1, hkv=1, d=64)
    par = np.concatenate([[-1, 0, 1], [-1, 0, 2, 9], [-1, 0, 0, 1, 1]])
    mask, pos, slots, err = run_plan(pkv, par, c.cu, c.tab, c.ctx, 1, c.nb, 12)
    assert err == OOB and list(mask[3:7, 0]) == [1, 3, 4, 8] and list(pos[3:7]) == [10, 11, 10, 10]
    good = np.concatenate([[-1, 0, 1], [-1, 0, 0, 1], [-1, 0, 0, 1, 1]])
    ctx = c.ctx.copy()
    ctx[1] = 3                                                 # fewer than its drafted tokens
    mask, pos, slots, err = run_plan(pkv, good, c.cu, c.tab, ctx, 1, c.nb, 12)
    assert err == OOB and not mask[3:7].any() and (pos[3:7] == -1).all() and (slots[3:7] == -1).all()
    assert list(mask[:3, 0]) == [1, 3, 7] and (slots[7:] >= 0).all()
    tab = c.tab.copy()
    tab[2, 0] = c.nb
    _, _, slots, err = run_plan(pkv, good, c.cu, tab, c.ctx, 1, c.nb, 12)
    assert err == OOB and (slots[7:] == -1).all() and (slots[:7] >= 0).all()
    for cu in ([0, 3, 2, 12], [0, 3, 7, 13], [-1, 3, 7, 12]):
        assert run_plan(pkv, good, np.array(cu), c.tab, c.ctx, 1, c.nb, 12)[3] == OOB


def test_plan_without_positions_or_slots(pkv):
    cu, lens = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, 3], [9]))
    par = torch.tensor([-1, 0, 0], dtype=torch.int32, device="cuda")
    mask = torch.zeros((3, 1), dtype=torch.int64, device="cuda")
    pkv.pkv_tree_plan(par, cu, None, lens, mask, None, None, num_blocks=0)
    assert mask.flatten().tolist() == [1, 3, 5]


# ---- commit ----
@pytest.mark.parametrize("dtype,layers,d", [("bf16", 0, 128), ("f16", 3, 64), ("u8", 0, 64), ("u8", 2, 128)])
def test_commit(pkv, dtype, layers, d):
    rng = np.random.default_rng(3)
    new = np.array([4, 1, 40, 0, 17, 30])
    base = np.array([0, 15, 100, 8, 31, 1])
    acc = [[0, 1, 2, 3], [], list(range(1, 40, 2)), [], [16], sorted(rng.choice(30, 12, replace=False).tolist())]
    c = Case(base, new, hq=1, hkv=1, d=64, seed=2)
    shape = (c.nb, layers, 2, 16, d) if layers else (c.nb, 2, 16, d)
    raw = [torch.randint(0, 256, (*shape[:-1], d * (1 if dtype == "u8" else 2)), dtype=torch.uint8) for _ in range(2)]
    kc, vc = (x.cuda() if dtype == "u8" else x.cuda().view(gu.TORCH_16[dtype]) for x in raw)
    most = max(len(a) for a in acc) + 1
    lists = np.full((6, most), -1, dtype=np.int32)
    for b, a in enumerate(acc):
        lists[b, :len(a)] = a
        lists[b, len(a) + 1:] = 3                              # (behind the first negative entry: not read)
    c.upload()
    new_lens = torch.zeros(6, dtype=torch.int32, device="cuda")
    pkv.pkv_tree_commit(kc, vc, c.tables, c.lens, c.cu_d, torch.from_numpy(lists).cuda(), new_lens=new_lens,
                        err_flag=c.err)
    torch.cuda.synchronize()
    assert int(c.err.item()) == 0
    assert new_lens.tolist() == [int(x) + len(a) for x, a in zip(base, acc)]
    for got, x in zip((kc, vc), raw):
        want = x.numpy().reshape(c.nb, -1, 16, x.shape[-1]).copy()
        for b, a in enumerate(acc):
            p = np.arange(int(c.ctx[b]))
            rows = want[c.tab[b][p // 16], :, p % 16]
            want[c.tab[b][p // 16], :, p % 16] = od.commit(rows, int(base[b]), a)
        assert (got.view(torch.uint8).cpu().numpy().reshape(want.shape) == want).all()


def test_commit_of_bad_lists_moves_nothing(pkv):
    c = Case([10, 10, 10, 10], [6, 6, 6, 6], hq=1, hkv=2, d=64).upload()
    before = c.vc.clone()
    lists = torch.tensor([[1, 3, -1], [3, 2, -1], [2, 2, -1], [1, 6, -1]], dtype=torch.int32, device="cuda")
    new = torch.full((4,), -5, dtype=torch.int32, device="cuda")
    pkv.pkv_tree_commit(c.kc, c.vc, c.tables, c.lens, c.cu_d, lists, new_lens=new, err_flag=c.err)
    assert int(c.err.item()) == OOB and new.tolist() == [12, -5, -5, -5]
    rows = torch.from_numpy(c.tab[1:].reshape(-1)[c.tab[1:].reshape(-1) >= 0].astype(np.int64)).cuda()
    assert torch.equal(c.vc[rows].view(torch.int16), before[rows].view(torch.int16))
    c = Case([10], [6], hq=1, hkv=2, d=64)
    c.tab[0, 0] = -1
    c.upload()
    pkv.pkv_tree_commit(c.kc, c.vc, c.tables, c.lens, c.cu_d, lists[:1], err_flag=c.err)
    assert int(c.err.item()) == OOB


def test_commit_of_nothing(pkv):
    c = Case([10], [6], hq=1, hkv=2, d=64).upload()
    before, new = c.vc.clone(), torch.zeros(1, dtype=torch.int32, device="cuda")
    pkv.pkv_tree_commit(c.kc, c.vc, c.tables, c.lens, c.cu_d, torch.zeros((1, 0), dtype=torch.int32, device="cuda"),
                        new_lens=new, err_flag=c.err)
    assert int(c.err.item()) == 0 and new.tolist() == [10]
    assert torch.equal(c.vc.view(torch.int16), before.view(torch.int16))


# ---- together ----
@pytest.mark.parametrize("kv", [None, "e4m3"])
def test_a_speculative_step_is_the_steps_it_replaces(pkv, kv):
    """Plan, rotary append, attention and commit of a drafted tree leave the cache
    and the outputs of plain steps over the accepted path; the same captured into
    a graph and replayed with other drafts."""
    hq, hkv, d, base = 8, 2, 64, [21, 130]
    g = torch.Generator().manual_seed(0)
    fmt = {None: "", "e4m3": "_fp8"}[kv]
    dev = dict(device="cuda")
    n, width, nb = 6, 12, 30
    parents = [[-1, 0, 0, 1, 1, 3], [-1, -1, 1, 2, 2, 4]]
    paths = [[0, 1, 3, 5], [1, 2, 4, 5]]
    tab = torch.randperm(nb, generator=g)[:2 * width].view(2, width).to(torch.int32).cuda()
    cu = torch.tensor([0, n, 2 * n], dtype=torch.int32, **dev)
    lens = torch.tensor([x + n for x in base], dtype=torch.int32, **dev)
    scales = [torch.rand(hkv, generator=g).cuda() + 0.1 for _ in range(2)] if kv else []
    pool = [torch.randn((nb, hkv, 16, d), generator=g) for _ in range(2)]
    pool = [x.to(FP8[kv]).view(torch.uint8).cuda() if kv else x.to(torch.bfloat16).cuda() for x in pool]
    qkv = torch.randn((2 * n, hq + 2 * hkv, d), generator=g).to(torch.bfloat16).cuda()
    turns, amp = pkv.pkv_rope_plan(d)
    turns = torch.from_numpy(turns).cuda()
    par = torch.tensor(parents, dtype=torch.int32, **dev).flatten()
    mask = torch.zeros((2 * n, 1), dtype=torch.int64, **dev)
    pos, slots = torch.zeros(2 * n, dtype=torch.int32, **dev), torch.zeros(2 * n, dtype=torch.int64, **dev)
    q, out = (torch.zeros((2 * n, hq, d), dtype=torch.bfloat16, **dev) for _ in range(2))
    acc = torch.tensor(paths, dtype=torch.int32, **dev)
    new_lens, err = torch.zeros(2, dtype=torch.int32, **dev), torch.zeros(1, dtype=torch.int32, **dev)
    ws = torch.empty(pkv.pkv_tree_workspace_bytes(2, 2 * n, hq, hkv, d, n), dtype=torch.uint8, **dev)
    kc, vc = (x.clone() for x in pool)

    def rope(qi, ki, vi, p, s, qo, k, v):
        getattr(pkv, "pkv_rope_append" + fmt)(qi, ki, vi, p, s, turns, qo, k, v, *scales, amplitude=amp, err_flag=err)

    def step():
        pkv.pkv_tree_plan(par, cu, tab, lens, mask, pos, slots, num_blocks=nb, err_flag=err)
        rope(qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], pos, slots, q, kc, vc)
        getattr(pkv, "pkv_paged_tree_attention" + fmt)(
            q, kc, vc, *scales, tab, lens, cu, mask, out, scale=d ** -0.5, max_context_len=200, max_nodes=n,
            workspace=ws, err_flag=err)
        pkv.pkv_tree_commit(kc, vc, tab, lens, cu, acc, new_lens=new_lens, err_flag=err)

    def plain(paths):
        k, v = (x.clone() for x in pool)
        outs = torch.zeros_like(out)
        dws = torch.empty(pkv.pkv_decode_workspace_bytes(1, hq, hkv, d, width, 200), dtype=torch.uint8, **dev)
        for b, path in enumerate(paths):
            for i, node in enumerate(path):
                t = b * n + node
                p = torch.tensor([base[b] + i], dtype=torch.int32, **dev)
                s = (tab[b, (base[b] + i) // 16].long() * 16 + (base[b] + i) % 16)[None]
                qi = torch.zeros((1, hq, d), dtype=torch.bfloat16, **dev)
                rope(qkv[t:t + 1, :hq], qkv[t:t + 1, hq:hq + hkv], qkv[t:t + 1, hq + hkv:], p, s, qi, k, v)
                getattr(pkv, "pkv_paged_decode_attention" + fmt)(
                    qi, k, v, *scales, tab[b:b + 1], p + 1, outs[t:t + 1], scale=d ** -0.5, max_context_len=200,
                    workspace=dws, err_flag=err)
        torch.cuda.synchronize()
        return k, v, outs

    def compare(paths):
        torch.cuda.synchronize()
        assert int(err.item()) == 0 and new_lens.tolist() == [x + len(p) for x, p in zip(base, paths)]
        k, v, outs = plain(paths)
        for b, path in enumerate(paths):
            p = torch.arange(base[b] + len(path), device="cuda")
            ids, off = tab[b][p // 16].long(), p % 16
            for x, y in ((kc, k), (vc, v)):
                assert torch.equal(x[ids, :, off].view(torch.uint8), y[ids, :, off].view(torch.uint8))
            t = [b * n + node for node in path]
            # both are within attn_limits of the same values; their sum covers a rounding each
            diff = (out[t].float() - outs[t].float()).abs()
            assert bool((diff <= 2.0 ** -7 * outs[t].float().abs() + 4e-3).all())

    step()
    compare(paths)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    for x, y in zip((kc, vc), pool):
        x.copy_(y)
    with torch.cuda.graph(graph, stream=side):
        step()
    for seed in (1, 2):
        gen = torch.Generator().manual_seed(seed)
        qkv.copy_(torch.randn(qkv.shape, generator=gen).to(torch.bfloat16))
        for x, y in zip((kc, vc), pool):
            x.copy_(y)
        out.zero_()
        graph.replay()
        compare(paths)


def test_two_streams_at_once(pkv):
    cases = [Case([900, 40, 333], [5, 60, 17], hq=8, hkv=2, seed=s) for s in range(2)]
    want = [c.attend(pkv).clone() for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    ws = [torch.empty(pkv.pkv_tree_workspace_bytes(3, c.tokens, 8, 2, 128, 60), dtype=torch.uint8, device="cuda")
          for c in cases]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, s, w in zip(cases, streams, ws):
            with torch.cuda.stream(s):
                pkv.pkv_paged_tree_attention(c.q, c.kc, c.vc, c.tables, c.lens, c.cu_d, c.mask, c.out, scale=c.scale,
                                             max_context_len=917, max_nodes=60, workspace=w, err_flag=c.err)
    torch.cuda.synchronize()
    for c, w in zip(cases, want):
        assert torch.equal(c.out, w) and int(c.err.item()) == 0


def test_many_runs_give_the_same_bits(pkv):
    # ragged rows (some warps of a tile without any), several pieces a thread block
    c = Case([700, 1500, 90, 260, 2000, 10], [3, 25, 20, 9, 31, 14], hq=16, hkv=4, seed=12)
    want = c.attend(pkv).clone()
    ws = torch.empty(pkv.pkv_tree_workspace_bytes(6, c.tokens, 16, 4, 128, 31), dtype=torch.uint8, device="cuda")
    for i in range(300):
        c.out.zero_()
        pkv.pkv_paged_tree_attention(c.q, c.kc, c.vc, c.tables, c.lens, c.cu_d, c.mask, c.out, scale=c.scale,
                                     max_context_len=2031, max_nodes=31, workspace=ws, err_flag=c.err)
        assert torch.equal(c.out, want), i
    assert int(c.err.item()) == 0
