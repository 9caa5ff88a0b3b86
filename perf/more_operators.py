"""Real work for drafted tokens and bounded contexts over the paged cache:
cases, their inputs, one pass each, and what a pass cannot do without.

Operators (the ``op`` of a case)
  plan      parents of drafted tokens -> which of them each sees, positions, slots
  tree      attention of drafted tokens over the cached context and their own tree
  commit    the accepted tokens' cached rows move up behind the context
  window    decode attention to the first few and the last tokens of a context
  chunk     the same for the tokens of a prompt chunk

Shapes follow the package: caches [blocks, KV heads, 16, head_dim], block
tables int32 [batch, blocks per sequence], q [tokens, query heads, head_dim].
A drafted token i of sequence b is cached at position base + i, base = context
length - number of drafted tokens.
"""
import math

import numpy as np
import torch

own = False

BS = 16                                   # tokens per cache block
T16 = {"f16": torch.float16, "bf16": torch.bfloat16}
FP8 = {"e4m3": (torch.float8_e4m3fn, 448.0), "e5m2": (torch.float8_e5m2, 57344.0)}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # four chats with a handful of drafted tokens each: launch latency
        dict(name="plan_small", op="plan", seqs=4, nlo=3, nhi=12, lo=100, hi=900, tree="wide"),
        # a full server, up to 256 drafted tokens a sequence
        dict(name="plan_batch", op="plan", seqs=256, nlo=100, nhi=256, lo=500, hi=8000, tree="wide"),
        # four short chats of a small model, a few drafted tokens each: latency
        dict(name="tree_small", op="tree", seqs=4, nlo=3, nhi=9, lo=50, hi=600, hq=4, hkv=4, d=64, dtype="f16",
             kv="f16", tree="chain"),
        # a batch of mixed contexts, up to 32 drafted tokens each (128 query rows a KV head)
        dict(name="tree_batch", op="tree", seqs=32, nlo=20, nhi=32, lo=1024, hi=16384, hq=32, hkv=8, d=128,
             dtype="bf16", kv="bf16", tree="wide"),
        # one very long document, 64 drafted tokens
        dict(name="tree_long", op="tree", seqs=1, nlo=64, nhi=64, lo=131072, hi=131072, hq=32, hkv=8, d=128,
             dtype="f16", kv="f16", tree="wide"),
        # long contexts in an 8-bit cache
        dict(name="tree_e4m3", op="tree", seqs=16, nlo=10, nhi=31, lo=4096, hi=32768, hq=32, hkv=8, d=128,
             dtype="bf16", kv="e4m3", tree="wide"),
        # four chats, one layer of a small model
        dict(name="commit_small", op="commit", seqs=4, nlo=3, nhi=9, lo=50, hi=600, heads=4, d=64, kv="f16",
             tree="wide"),
        # a batch, all 32 layers of 8 heads in one layer-major cache
        dict(name="commit_model", op="commit", seqs=64, nlo=32, nhi=64, lo=1024, hi=16384, heads=256, d=128,
             kv="bf16", tree="deep"),
        # four chats of a small model: latency
        dict(name="window_small", op="window", seqs=4, lo=100, hi=3000, window=256, sinks=4, hq=4, hkv=4, d=64,
             dtype="f16", kv="f16"),
        # long conversations, 4096 tokens of each kept; the rest of the cache is gone
        dict(name="window_batch", op="window", seqs=64, lo=3000, hi=131072, window=4096, sinks=4, hq=32, hkv=8,
             d=128, dtype="bf16", kv="bf16"),
        # a short prompt, longer than the window
        dict(name="chunk_small", op="chunk", seqs=1, new=300, lo=1, hi=1, window=128, sinks=4, hq=8, hkv=2, d=128,
             dtype="f16", kv="f16"),
        # a chunk of four prompts deep in long documents
        dict(name="chunk_batch", op="chunk", seqs=4, new=2048, lo=8000, hi=40000, window=4096, sinks=4, hq=32, hkv=8,
             d=128, dtype="bf16", kv="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "tree", "tree", "tree", "commit", "window", "window", "chunk"])
    dtype = rng.choice(["f16", "bf16"])
    hkv, d = rng.choice([1, 2, 3, 4, 5, 8]), rng.choice([64, 128])
    hq = hkv * (rng.choice([1, 2, 4, 8]) if hkv <= 4 else rng.choice([1, 2, 4]))
    kv = rng.choice([dtype, dtype, "e4m3", "e5m2"])
    tree = rng.choice(["wide", "deep", "chain"])
    nhi = _log(rng, 1, 128)
    nlo = rng.randint(1, nhi)
    lo = _log(rng, 1, 4096)
    hi = lo + _log(rng, 1, 16384)
    if op == "plan":
        nhi = min(2 * nhi, 256)
        return dict(op=op, seqs=_log(rng, 1, 256), nlo=nlo, nhi=nhi, lo=lo, hi=hi, tree=tree)
    if op == "commit":
        return dict(op=op, seqs=_log(rng, 1, 48), nlo=nlo, nhi=nhi, lo=lo, hi=hi, heads=hkv * _log(rng, 1, 28), d=d,
                    kv=kv, tree=tree)
    if op == "tree":
        seqs = _log(rng, 1, 24) if hi < 16384 else _log(rng, 1, 8)
        return dict(op=op, seqs=seqs, nlo=nlo, nhi=nhi, lo=lo, hi=hi, hq=hq, hkv=hkv, d=d, dtype=dtype, kv=kv,
                    tree=tree)
    window, sinks = _log(rng, 1, 4096), rng.choice([0, 1, 4, rng.randint(2, 70)])
    if op == "window":
        return dict(op=op, seqs=_log(rng, 1, 48), lo=lo, hi=hi, window=window, sinks=sinks, hq=hq, hkv=hkv, d=d,
                    dtype=dtype, kv=kv)
    return dict(op=op, seqs=rng.randint(1, 3), new=_log(rng, 1, 2048), lo=lo, hi=hi, window=window, sinks=sinks,
                hq=hq, hkv=hkv, d=128, dtype=dtype, kv=dtype)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _lens_of(case):
    """Context lengths (without new tokens) and counts of new tokens: the same
    for every seed, so that shapes are too."""
    rng = np.random.Generator(np.random.PCG64([case["seqs"], case["lo"], case["hi"]]))
    u = rng.uniform(math.log(case["lo"]), math.log(case["hi"]), size=case["seqs"])
    base = np.clip(np.rint(np.exp(u)), case["lo"], case["hi"]).astype(np.int64)
    if case["op"] == "window":
        return base, np.zeros_like(base)
    if case["op"] == "chunk":
        new = rng.integers(max(1, case["new"] // 2), case["new"] + 1, size=case["seqs"])
        new[0] = case["new"]
        return base - case["lo"] if case["lo"] == 1 else base, new
    return base, rng.integers(case["nlo"], case["nhi"] + 1, size=case["seqs"])


def _parents(rng, n, kind):
    """Parents of n drafted tokens, each before its children, -1 at the root."""
    i = np.arange(n)
    if kind == "chain":
        return (i - 1).astype(np.int32)
    back = rng.uniform(size=n)
    p = i - 1 - np.floor((back ** 3 if kind == "deep" else back) * np.minimum(i + 1, 6 if kind == "deep" else 16))
    return np.maximum(p, -1).astype(np.int32)


def _nblk(n):
    return (n + BS - 1) // BS


def _tables(rng, live):
    """Block tables over one random permutation of the pool; live bool [batch,
    width] says which entries exist (the others are -1)."""
    ids = rng.permutation(int(live.sum()) + 3).astype(np.int32)
    out = np.full(live.shape, -1, dtype=np.int32)
    out[live] = ids[:int(live.sum())]
    return out, len(ids)


def _cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _pools(gen, shape, kv, dtype, s):
    """K and V caches of random values; 8-bit ones as codes, with a scale per head."""
    for name, sc in (("kc", "ks"), ("vc", "vs")):
        x = torch.randn(shape, generator=gen, device="cuda", dtype=T16[dtype])
        if kv in FP8:
            t, top = FP8[kv]
            s[sc] = x.abs().amax(dim=(0, 2, 3)).float() / top
            codes = torch.empty(shape, dtype=torch.uint8, device="cuda")
            for h in range(shape[1]):     # a head at a time bounds the 32-bit copy
                codes[:, h] = (x[:, h].float() / s[sc][h]).to(t).view(torch.uint8)
            x = codes
        s[name] = x


def _closure(parents):
    """Which drafted tokens each sees: itself and its ancestors."""
    n = len(parents)
    vis = np.zeros((n, n), dtype=bool)
    for i in range(n):
        if parents[i] >= 0:
            vis[i] = vis[parents[i]]
        vis[i, i] = True
    return vis


def _words(vis, words):
    """Bits of bool [n, m] as int64 [n, words], bit j of word j // 64."""
    bits = np.zeros((vis.shape[0], words * 64), dtype=np.uint8)
    bits[:, :vis.shape[1]] = vis
    return np.packbits(bits, axis=1, bitorder="little").view(np.int64)


def prepare(case, seed):
    base, new = _lens_of(case)
    rng = np.random.Generator(np.random.PCG64([seed, 23]))
    gen = torch.Generator(device="cuda").manual_seed(1000003 * seed + 29)
    op, n = case["op"], case["seqs"]
    ctx = base + new
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    width = int(_nblk(ctx.max()))
    col = np.arange(width)[None]
    live = col < _nblk(ctx)[:, None]
    if op == "commit":                                # only the blocks that hold drafted tokens
        live &= col >= (base // BS)[:, None]
    if op in ("window", "chunk"):                     # blocks between the first and the last tokens are gone
        first_query = ctx - 1 if op == "window" else base
        low = np.maximum(first_query - case["window"] + 1, 0)
        live &= (col < _nblk(case["sinks"])) | (col >= (low // BS)[:, None])
    tables, nb = _tables(rng, live)
    s = dict(case=case, lens=_cuda(ctx.astype(np.int32)), tables=_cuda(tables), cu=_cuda(cu))
    if op in ("plan", "tree", "commit"):
        nmax = int(new.max())
        words = -(-nmax // 64)
        par = [_parents(rng, int(m), case["tree"]) for m in new]
        s["nmax"] = nmax
        if op == "plan":
            s["parents"] = _cuda(np.concatenate(par))
            t = int(cu[-1])
            s.update(nb=nb, mask=torch.zeros((t, words), dtype=torch.int64, device="cuda"),
                     pos=torch.zeros(t, dtype=torch.int32, device="cuda"),
                     slots=torch.zeros(t, dtype=torch.int64, device="cuda"))
            return s
        vis = [_closure(p) for p in par]
        if op == "commit":
            # a path from a root to one of the tokens, cut where the model disagreed
            paths = [np.flatnonzero(v[rng.integers(0, len(v))]) for v in vis]
            paths = [p[:rng.integers(1, len(p) + 1)] for p in paths]
            acc = np.full((n, nmax), -1, dtype=np.int32)
            for b, p in enumerate(paths):
                acc[b, :len(p)] = p
            s["accepted"] = _cuda(acc)
            _pools(gen, (nb, case["heads"], BS, case["d"]), case["kv"], "f16" if case["kv"] in FP8 else case["kv"], s)
            s["new_lens"] = torch.zeros(n, dtype=torch.int32, device="cuda")
            return s
        s["mask"] = _cuda(np.concatenate([_words(v, words) for v in vis]))
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    _pools(gen, (nb, hkv, BS, d), case["kv"], case["dtype"], s)
    tokens = n if op == "window" else int(cu[-1])
    s["q"] = torch.randn((tokens, hq, d), generator=gen, device="cuda", dtype=T16[case["dtype"]])
    s.update(out=torch.empty_like(s["q"]), scale=d ** -0.5, max_ctx=int(ctx.max()), max_new=int(new.max()))
    if own and op != "chunk":
        import paged_kv_cache_153_gb300 as pkv
        size = (pkv.pkv_decode_workspace_bytes(n, hq, hkv, d, width, case["window"] + case["sinks"])
                if op == "window" else pkv.pkv_tree_workspace_bytes(n, tokens, hq, hkv, d, s["nmax"]))
        s["ws"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    return (_run_own if own else _run_plain)(s)


def _values(s):
    """Both caches as what they stand for (8-bit codes before their scale)."""
    kv = s["case"]["kv"]
    return [s[name].view(FP8[kv][0]) if kv in FP8 else s[name] for name in ("kc", "vc")]


def _run_own(s):
    import paged_kv_cache_153_gb300 as pkv
    case = s["case"]
    op = case["op"]
    if op == "plan":
        pkv.pkv_tree_plan(s["parents"], s["cu"], s["tables"], s["lens"], s["mask"], s["pos"], s["slots"],
                          num_blocks=s["nb"])
        return s["mask"], s["pos"], s["slots"]
    if op == "commit":
        pkv.pkv_tree_commit(s["kc"], s["vc"], s["tables"], s["lens"], s["cu"], s["accepted"], new_lens=s["new_lens"])
        return _values(s), s["new_lens"]
    fmt = {"e4m3": "_fp8", "e5m2": "_e5m2"}.get(case["kv"], "")
    caches = (s["kc"], s["vc"]) + ((s["ks"], s["vs"]) if fmt else ())
    if op == "tree":
        call = getattr(pkv, "pkv_paged_tree_attention" + fmt)
        call(s["q"], *caches, s["tables"], s["lens"], s["cu"], s["mask"], s["out"], scale=s["scale"],
             max_context_len=s["max_ctx"], max_nodes=s["nmax"], workspace=s["ws"])
    elif op == "window":
        call = getattr(pkv, "pkv_paged_decode_attention_window" + fmt)
        call(s["q"], *caches, s["tables"], s["lens"], s["out"], scale=s["scale"], window=case["window"],
             num_sinks=case["sinks"], workspace=s["ws"])
    else:
        pkv.pkv_paged_prefill_attention_window(s["q"], *caches, s["tables"], s["lens"], s["cu"], s["out"],
                                               scale=s["scale"], max_query_len=s["max_new"], window=case["window"],
                                               num_sinks=case["sinks"])
    return s["out"]


def _rows(s, name, blocks, off):
    """Rows (block, offset) of a cache for every head, in 32 bits: [..., heads, d]."""
    x = s[name][blocks, :, off]
    sc = s.get(name[0] + "s")
    return x.float() if sc is None else x.view(FP8[s["case"]["kv"]][0]).float() * sc[:, None]


def _attend(s, q, blocks, off, keep):
    """q [batch, m, heads, d]; keys [batch, n] by block and offset; keep bool
    [batch, m, n]; a query that keeps none gives 0."""
    b, m, hq, d = q.shape
    k, v = (_rows(s, name, blocks, off).transpose(1, 2) for name in ("kc", "vc"))      # [batch, hkv, n, d]
    hkv = k.shape[1]
    x = q.float().view(b, m, hkv, -1, d).permute(0, 2, 1, 3, 4).reshape(b, hkv, -1, d)
    p = torch.matmul(x, k.transpose(2, 3)).mul_(s["scale"]).view(b, hkv, m, -1, k.shape[2])
    p.masked_fill_(~keep[:, None, :, None, :], float("-inf"))
    p = p.sub_(p.amax(-1, keepdim=True).clamp_min(-3e38)).exp_()
    p /= p.sum(-1, keepdim=True).clamp_min(1e-38)
    o = torch.matmul(p.view(b, hkv, -1, k.shape[2]), v)
    return o.view(b, hkv, m, -1, d).permute(0, 2, 1, 3, 4).reshape(b, m, hq, d)


def _padded(s):
    """Token index [batch, m] of every sequence's new tokens, and which exist."""
    new = (s["cu"][1:] - s["cu"][:-1]).long()
    i = torch.arange(s["nmax"] if "nmax" in s else s["max_new"], device="cuda")
    return (s["cu"][:-1, None] + i).clamp_max(int(s["q"].shape[0] if "q" in s else s["parents"].shape[0]) - 1), \
        i < new[:, None], new


def _run_plain(s):
    case, dev = s["case"], "cuda"
    op, lens, tab = case["op"], s["lens"].long(), s["tables"].long()
    if op == "plan":
        tok, live, new = _padded(s)
        b, i = live.nonzero(as_tuple=True)
        m = s["nmax"]
        par = torch.where(live, s["parents"][tok].long(), -1)
        step = (par[..., None] == torch.arange(m, device=dev)).float()
        vis = torch.eye(m, device=dev) + step
        for _ in range(max(m - 1, 1).bit_length()):   # paths of up to 2, 4, 8, ... edges
            vis = (torch.matmul(vis, vis) > 0).float()
        bits = torch.nn.functional.pad(vis[b, i].long(), (0, 64 * s["mask"].shape[1] - m))
        s["mask"].copy_((bits.view(len(b), -1, 64) << torch.arange(64, device=dev)).sum(2))
        base = (lens - new)[b]
        s["pos"].copy_(base + vis[b, i].long().sum(1) - 1)
        at = base + i
        s["slots"].copy_(tab[b, at // BS] * BS + at % BS)
        return s["mask"], s["pos"], s["slots"]
    if op == "commit":
        new = (s["cu"][1:] - s["cu"][:-1]).long()
        acc = s["accepted"].long()
        b, k = (acc >= 0).nonzero(as_tuple=True)
        base = (lens - new)[b]
        src, dst = base + acc[b, k], base + k
        for c in (s["kc"], s["vc"]):
            c[tab[b, dst // BS], :, dst % BS] = c[tab[b, src // BS], :, src % BS]
        s["new_lens"].copy_(lens - new + (acc >= 0).sum(1))
        return _values(s), s["new_lens"]
    if op == "tree":
        tok, live, new = _padded(s)
        key = torch.arange(s["max_ctx"], device=dev)
        node = key - (lens - new)[:, None]                                        # [batch, n]
        j = torch.arange(s["nmax"], device=dev)
        bit = (s["mask"][tok][..., j // 64] >> (j % 64)) & 1                      # [batch, m, m]
        at = node.clamp(0, s["nmax"] - 1)[:, None].expand(-1, s["nmax"], -1)
        keep = ((node < 0)[:, None] | (bit.gather(2, at) > 0)) & (key < lens[:, None])[:, None]
        o = _attend(s, s["q"][tok], tab[:, key // BS].clamp_min(0), (key % BS).expand(len(lens), -1), keep)
        s["out"].copy_(o[live])
        return s["out"]
    # the first tokens, then the last ones
    tok, live, new = _padded(s) if op == "chunk" else (torch.arange(len(lens), device=dev)[:, None], None, 1)
    m = tok.shape[1]
    low = (lens - new - case["window"] + 1).clamp_min(0)                          # first key of the first query
    c = torch.arange(case["sinks"] + min(case["window"] + m - 1, s["max_ctx"]), device=dev)
    last = low[:, None] + c - case["sinks"]
    key = torch.where(c < case["sinks"], c, last)
    ok = torch.where(c < case["sinks"], c < low[:, None], last < lens[:, None])
    pos = (lens - new)[:, None] + torch.arange(m, device=dev)
    key, pos = key[:, None], pos[..., None]
    keep = ok[:, None] & (key <= pos) & ((key < case["sinks"]) | (key > pos - case["window"]))
    key = key[:, 0].clamp_max(s["max_ctx"] - 1)
    o = _attend(s, s["q"][tok], tab.gather(1, key // BS).clamp_min(0), key % BS, keep)
    s["out"].copy_(o[:, 0] if live is None else o[live])
    return s["out"]


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    op = case["op"]
    base, new = _lens_of(case)
    ctx, t = base + new, int(new.sum())
    e = 1 if case.get("kv") in FP8 else 2
    if op in ("plan", "tree"):
        words = -(-int(new.max()) // 64)
    if op == "plan":
        return {"bytes": t * (4 + 8 * words + 4 + 8 + 4) + 8 * len(new), "flops": int((new * new).sum())}
    if op == "commit":
        moved = _moved(case)
        return {"bytes": moved * case["heads"] * case["d"] * e * 4, "flops": moved * case["heads"] * case["d"]}
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if op == "tree":
        return {"bytes": int(ctx.sum()) * hkv * d * 2 * e + t * (hq * d * 4 + 8 * words),
                "flops": 4 * hq * d * int((new * base + new).sum())}
    if op == "window":
        seen = np.minimum(ctx, case["window"]) + np.minimum(np.maximum(ctx - case["window"], 0), case["sinks"])
        return {"bytes": int(seen.sum()) * hkv * d * 2 * e + len(ctx) * hq * d * 4, "flops": 4 * hq * d * int(seen.sum())}
    pos = np.concatenate([np.arange(b, b + n) for b, n in zip(base, new)]) + 1
    seen = np.minimum(pos, case["window"]) + np.minimum(np.maximum(pos - case["window"], 0), case["sinks"])
    low = np.maximum(base - case["window"] + 1, 0)
    keys = ctx - low + np.minimum(low, case["sinks"])
    return {"bytes": int(keys.sum()) * hkv * d * 4 + t * hq * d * 4, "flops": 4 * hq * d * int(seen.sum())}


def _moved(case):
    """About the rows that change their place (paths differ by seed): half of a typical depth."""
    _, new = _lens_of(case)
    rng = np.random.Generator(np.random.PCG64([7]))
    depth = [_closure(_parents(rng, int(n), case["tree"])).sum(1).mean() for n in new]
    return max(1, int(sum(depth) / 2))


# ---------------------------------------------------------------------------
# from the definitions, in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    if case["op"] == "plan":
        return None
    s = prepare(case, seed)
    base, new = _lens_of(case)
    if case["op"] == "commit":
        caches = [x.double() for x in _values(s)]
        for b, accepted in enumerate(s["accepted"].tolist()):
            for k, i in enumerate(a for a in accepted if a >= 0):      # ascending: a row is read before it is written
                to, at = int(base[b]) + k, int(base[b]) + i
                for x in caches:
                    x[int(s["tables"][b, to // BS]), :, to % BS] = x[int(s["tables"][b, at // BS]), :, at % BS]
        return caches, None
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    per = case["hq"] // case["hkv"]
    at = 0
    for b in range(case["seqs"]):
        if case["op"] == "window":
            rows, pos = torch.arange(b, b + 1), [int(base[b]) - 1]
        else:
            rows = torch.arange(at, at + int(new[b]))
            pos = list(range(int(base[b]), int(base[b] + new[b])))
            at += int(new[b])
        n = int(base[b] + new[b])
        pos = torch.tensor(pos, device="cuda")[:, None]
        key = torch.arange(n, device="cuda")
        if case["op"] == "tree":
            need = key
            words = s["mask"][rows.cuda()].cpu().numpy().view(np.uint64)
            seen = torch.ones((len(rows), n), dtype=torch.bool)
            for i in range(len(rows)):
                value = sum(int(w) << (64 * x) for x, w in enumerate(words[i]))
                for j in range(int(new[b])):
                    seen[i, int(base[b]) + j] = bool(value >> j & 1)
            seen = seen.cuda()
        else:
            first = max(0, int(pos[0, 0]) + 1 - case["window"])
            need = key[(key < case["sinks"]) | (key >= first)]
            seen = (need <= pos) & ((need < case["sinks"]) | (pos - need < case["window"]))
        ids = s["tables"][b].long()[need // BS]
        for g in range(case["hkv"]):
            kv = []
            for name, sc in (("kc", "ks"), ("vc", "vs")):
                x = s[name][ids, g, need % BS]
                kv.append(x.view(FP8[case["kv"]][0]).double() * s[sc][g].double() if sc in s else x.double())
            for h in range(g * per, (g + 1) * per):
                logit = s["q"][rows.cuda(), h].double() @ kv[0].T * s["scale"]
                logit = torch.where(seen, logit, float("-inf"))
                out[rows.cuda(), h] = torch.softmax(logit, 1) @ kv[1]
    return out
