"""Real work for the cache's rotary append, block-sparse decode and
shared-prefix decode: cases, their inputs, one pass each, and what a pass
cannot do without.

Operators (the ``op`` of a case)
  rope      rotary positions of q and k, with the append of k and v
  bounds    per-block minimum and maximum of the cached keys
  scores    upper bound of every block's logits, from those bounds
  select    the highest-scoring blocks of each (sequence, KV head)
  sparse    decode attention over selected blocks
  prefix    decode attention of sequences that share a prefix

Shapes follow the package: caches [blocks, KV heads, 16, head_dim], block
tables int32 [batch, blocks per sequence], q [batch, query heads, head_dim].
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
        # four short sequences of a small model decode one token each: launch latency
        dict(name="rope_step_small", op="rope", seqs=4, new=1, lo=1, hi=256, hq=4, hkv=4, d=64, rot=32,
             dtype="f16", kv="f16", layout="interleaved", scaling="none", factor=1.0, base=10000.0),
        # one prefill chunk of 4 x 2048 tokens behind a long prompt, positions scaled to a longer context
        dict(name="rope_prefill_chunk", op="rope", seqs=4, new=2048, lo=4096, hi=98304, hq=32, hkv=8, d=128,
             rot=128, dtype="bf16", kv="bf16", layout="half", scaling="wavelength", factor=8.0, base=500000.0),
        # after a decode step: each of 64 sequences refreshes the block of its newest token
        dict(name="bounds_step", op="bounds", seqs=64, new=1, lo=128, hi=8192, hkv=8, d=128, dtype="bf16",
             kv="bf16"),
        # after prefill: every block of 32 long contexts over an 8-bit cache
        dict(name="bounds_prefill_e4m3", op="bounds", seqs=32, new=0, lo=2048, hi=32768, hkv=8, d=128,
             dtype="bf16", kv="e4m3"),
        # one long conversation, eight query heads per KV head
        dict(name="scores_one_long", op="scores", seqs=1, lo=16384, hi=16384, hq=32, hkv=4, d=128, dtype="f16"),
        # a batch of mixed long contexts
        dict(name="scores_batch", op="scores", seqs=64, lo=1024, hi=32768, hq=32, hkv=8, d=128, dtype="bf16"),
        # a few middling contexts
        dict(name="select_small", op="select", seqs=4, lo=1000, hi=8000, hkv=8, budget=32, first=1, last=2),
        # a batch of contexts up to 131072 tokens, 2048 of them kept
        dict(name="select_batch", op="select", seqs=64, lo=8192, hi=131072, hkv=8, budget=128, first=4, last=8),
        # one query head per KV head, head_dim 64, few sequences: latency
        dict(name="sparse_small", op="sparse", seqs=4, lo=500, hi=6000, hq=4, hkv=4, d=64, dtype="f16", kv="f16",
             budget=16),
        # a batch of long contexts, 2048 tokens of each attended
        dict(name="sparse_batch", op="sparse", seqs=64, lo=1500, hi=32768, hq=32, hkv=8, d=128, dtype="bf16",
             kv="bf16", budget=128),
        # 16 requests behind one system prompt of 2048 tokens
        dict(name="prefix_prompt", op="prefix", groups=1, seqs=16, prefix=2048, lo=16, hi=512, hq=32, hkv=8, d=128,
             dtype="bf16"),
        # 64 questions about one long document
        dict(name="prefix_document", op="prefix", groups=1, seqs=64, prefix=32768, lo=16, hi=2048, hq=32, hkv=8,
             d=128, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "bounds", "scores", "select", "sparse", "prefix"])
    dtype = rng.choice(["f16", "bf16"])
    hkv, d = rng.choice([1, 2, 3, 4, 5, 8]), rng.choice([64, 128])
    group = rng.choice([1, 2, 4, 8]) if hkv <= 4 else rng.choice([1, 2, 4])
    hq = hkv * group
    kv = rng.choice([dtype, dtype, "e4m3", "e5m2"])
    if op == "rope":
        new = rng.choice([1, 1, _log(rng, 2, 2048)])
        seqs = _log(rng, 1, 64) if new == 1 else rng.randint(1, 4)
        lo = _log(rng, 1, 16384)
        return dict(op=op, seqs=seqs, new=new, lo=lo, hi=lo + _log(rng, 1, 65536), hq=hq, hkv=hkv, d=d,
                    rot=16 * rng.randint(1, d // 16), dtype=dtype, kv=kv,
                    layout=rng.choice(["half", "interleaved"]),
                    scaling=rng.choice(["none", "linear", "base", "ramp", "wavelength"]),
                    factor=rng.choice([2.0, 4.0, 8.0, 16.0]), base=rng.choice([10000.0, 500000.0]))
    lo = _log(rng, 1, 4096)
    hi = lo + _log(rng, 1, 16384)
    if op == "bounds":
        return dict(op=op, seqs=_log(rng, 1, 48), new=rng.choice([0, 1, _log(rng, 2, 512)]), lo=lo, hi=hi, hkv=hkv,
                    d=d, dtype=dtype, kv=kv)
    if op == "scores":
        return dict(op=op, seqs=_log(rng, 1, 64), lo=lo, hi=hi, hq=hq, hkv=hkv, d=d, dtype=dtype)
    if op == "select":
        first, last = rng.randint(0, 4), rng.randint(1, 8)
        return dict(op=op, seqs=_log(rng, 1, 64), lo=lo, hi=hi + _log(rng, 1, 65536), hkv=hkv,
                    budget=first + last + _log(rng, 1, 256), first=first, last=last)
    if op == "sparse":
        return dict(op=op, seqs=_log(rng, 1, 48), lo=lo, hi=hi, hq=hq, hkv=hkv, d=d, dtype=dtype, kv=kv,
                    budget=_log(rng, 1, 128))
    groups = rng.choice([1, 1, 2, rng.randint(3, 8)])
    seqs = _log(rng, 1, 96) if groups == 1 else rng.randint(1, 16)
    return dict(op=op, groups=groups, seqs=seqs, prefix=_log(rng, 1, 16384 // groups),
                lo=rng.randint(0, 64), hi=rng.randint(64, 1024), hq=hq, hkv=hkv, d=d, dtype=dtype)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _lengths(rng, lo, hi, n):
    """n context lengths, log-uniform in [lo, hi]."""
    u = rng.uniform(math.log(max(lo, 1)), math.log(max(hi, 1)), size=n)
    return np.clip(np.rint(np.exp(u)), max(lo, 1), max(hi, 1)).astype(np.int32)


def _nblk(n):
    return (n + BS - 1) // BS


def _tables(rng, counts, spare=3):
    """Block tables over one random permutation of the pool, -1 past each end."""
    total = int(sum(counts))
    ids = rng.permutation(total + spare).astype(np.int32)
    out = np.full((len(counts), max(1, max(counts))), -1, dtype=np.int32)
    pos = 0
    for b, n in enumerate(counts):
        out[b, :n] = ids[pos:pos + n]
        pos += n
    return out, total + spare


def _pool(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device="cuda", dtype=T16[dtype])


def _coded(x, kv):
    """8-bit codes of x [..., heads at 1] with one scale per head, and the scales."""
    t, top = FP8[kv]
    amax = x.abs().amax(dim=(0, 2, 3)).float()
    scale = amax / top
    codes = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    for h in range(x.shape[1]):           # a head at a time bounds the 32-bit copy
        codes[:, h] = (x[:, h].float() / scale[h]).to(t).view(torch.uint8)
    return codes, scale


def _cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _lens_of(case):
    """The case's lengths: the same for every seed, so that shapes are too."""
    n = case["seqs"] * case.get("groups", 1)
    return _lengths(np.random.Generator(np.random.PCG64([n, case["lo"], case["hi"]])), case["lo"], case["hi"], n)


def prepare(case, seed):
    lens, rng = _lens_of(case), np.random.Generator(np.random.PCG64([seed, 17]))
    gen = torch.Generator(device="cuda").manual_seed(1000003 * seed + 11)
    op = case["op"]
    s = dict(case=case)
    if op == "rope":
        new, n = case["new"], case["seqs"]
        hq, hkv, d = case["hq"], case["hkv"], case["d"]
        ctx = lens + new                              # the new tokens are each sequence's last ones
        # blocks of the new tokens only (the older ones are not touched)
        first = lens // BS
        counts = _nblk(ctx) - first
        tables, nb = _tables(rng, counts)
        pos = np.concatenate([np.arange(c - new, c) for c in ctx]).astype(np.int32)
        seq = np.repeat(np.arange(n), new)
        slots = tables[seq, pos // BS - first[seq]].astype(np.int64) * BS + pos % BS
        # q, k and v are slices of one projection's output
        qkv = _pool(gen, (n * new, hq + 2 * hkv, d), case["dtype"])
        s.update(q=qkv[:, :hq], k=qkv[:, hq:hq + hkv], v=qkv[:, hq + hkv:], pos=_cuda(pos), slots=_cuda(slots))
        pool = _pool(gen, (2, nb, hkv, BS, d), case["dtype"])
        if case["kv"] in FP8:
            s["kc"], s["ks"] = _coded(pool[0], case["kv"])
            s["vc"], s["vs"] = _coded(pool[1], case["kv"])
        else:
            s["kc"], s["vc"] = pool[0].clone(), pool[1].clone()
        s["q_out"] = torch.empty((n * new, hq, d), dtype=T16[case["dtype"]], device="cuda")
        if own:
            import paged_kv_cache_153_gb300 as pkv
            turns, amp = pkv.pkv_rope_plan(case["rot"], base=case["base"], scaling=case["scaling"],
                                           factor=case["factor"], original_context=8192)
            s.update(turns=torch.from_numpy(turns).cuda(), amp=amp)
        else:
            inv, amp = _inverse_frequencies(case)
            s.update(inv=_cuda(inv), amp=amp)
        return s
    if op == "select":
        width = int(_nblk(lens.max()))
        s["lens"] = _cuda(lens)
        s["scores"] = 60 + 8 * torch.randn((case["seqs"], case["hkv"], width), generator=gen, device="cuda")
        s["selected"] = torch.empty((case["seqs"], case["hkv"], case["budget"]), dtype=torch.int32, device="cuda")
        return s
    if op == "prefix":
        return _prepare_prefix(case, lens, rng, gen, s)
    counts = _nblk(lens)
    tables, nb = _tables(rng, counts)
    s.update(lens=_cuda(lens), tables=_cuda(tables))
    hkv, d = case["hkv"], case["d"]
    if op == "bounds":
        kc = _pool(gen, (nb, hkv, BS, d), case["dtype"])
        s["kc"] = _coded(kc, case["kv"])[0] if case["kv"] in FP8 else kc
        s["new"] = _cuda(np.minimum(lens, case["new"]).astype(np.int32)) if case["new"] else None
        s["max_new"] = int(min(lens.max(), case["new"]) if case["new"] else lens.max())
        s["bounds"] = torch.zeros((nb, hkv, 2, d), dtype=T16[case["dtype"]], device="cuda")
        return s
    if op == "scores":
        lo_hi = _pool(gen, (nb, hkv, 2, d), case["dtype"])
        s["bounds"] = torch.stack([lo_hi.amin(2) - 1, lo_hi.amax(2) + 1], 2).contiguous()
        s["q"] = _pool(gen, (case["seqs"], case["hq"], d), case["dtype"])
        s["scale"] = d ** -0.5
        s["scores"] = torch.zeros((case["seqs"], hkv, tables.shape[1]), device="cuda")
        s["max_ctx"] = int(lens.max())
        return s
    # sparse
    kc, vc = (_pool(gen, (nb, hkv, BS, d), case["dtype"]) for _ in range(2))
    if case["kv"] in FP8:
        kc, s["ks"] = _coded(kc, case["kv"])
        vc, s["vs"] = _coded(vc, case["kv"])
    s.update(kc=kc, vc=vc, q=_pool(gen, (case["seqs"], case["hq"], d), case["dtype"]), scale=d ** -0.5)
    # the lists a selection returns: ascending, the newest block among them, -1 past each end
    nblk = s["lens"].add(BS - 1).div(BS, rounding_mode="floor").view(-1, 1, 1)
    width, budget = tables.shape[1], case["budget"]
    rank = torch.rand((case["seqs"], hkv, width), generator=gen, device="cuda")
    col = torch.arange(width, device="cuda")
    rank = torch.where(col == nblk - 1, 2.0, rank.masked_fill(col >= nblk, -1.0))
    val, idx = rank.topk(min(budget, width), dim=2)
    idx = idx.masked_fill(val < 0, width).sort(dim=2).values
    idx = torch.where(idx == width, -1, idx).to(torch.int32)
    s["selected"] = torch.nn.functional.pad(idx, (0, budget - idx.shape[2]), value=-1).contiguous()
    s["out"] = torch.empty_like(s["q"])
    if own:
        import paged_kv_cache_153_gb300 as pkv
        s["ws"] = torch.empty(pkv.pkv_decode_workspace_bytes(case["seqs"], case["hq"], hkv, d, budget, BS * budget),
                              dtype=torch.uint8, device="cuda")
    return s


def _prepare_prefix(case, lens, rng, gen, s):
    g, n, hkv, d = case["groups"], case["seqs"], case["hkv"], case["d"]
    pre = [case["prefix"] if j == 0 else max(1, case["prefix"] // (j + 1)) for j in range(g)]
    pb = [p // BS for p in pre]                      # shared whole blocks
    ctx = np.array([pre[b // n] + (lens[b] if case["lo"] or b % 5 else 0) for b in range(g * n)], dtype=np.int32)
    counts = [int(_nblk(ctx[b])) - pb[b // n] for b in range(g * n)]
    priv, nb = _tables(rng, counts + pb)
    tables = np.full((g * n, max(1, int(_nblk(ctx.max())))), -1, dtype=np.int32)
    for b in range(g * n):
        j = b // n
        tables[b, :pb[j]] = priv[g * n + j, :pb[j]]
        tables[b, pb[j]:pb[j] + counts[b]] = priv[b, :counts[b]]
    s.update(tables=_cuda(tables), lens=_cuda(ctx), starts=_cuda(np.arange(g + 1, dtype=np.int32) * n),
             pre=_cuda(np.array(pre, dtype=np.int32)), max_ctx=int(ctx.max()), max_pre=int(max(pre)),
             host=dict(ctx=ctx, pb=pb), scale=d ** -0.5,
             kc=_pool(gen, (nb, hkv, BS, d), case["dtype"]), vc=_pool(gen, (nb, hkv, BS, d), case["dtype"]),
             q=_pool(gen, (g * n, case["hq"], d), case["dtype"]))
    s["out"] = torch.empty_like(s["q"])
    if own:
        import paged_kv_cache_153_gb300 as pkv
        s["ws"] = torch.empty(pkv.pkv_prefix_workspace_bytes(g * n, g, case["hq"], hkv, d, tables.shape[1],
                                                             s["max_ctx"], s["max_pre"]),
                              dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    return (_run_own if own else _run_plain)(s)


def _values(codes, kv):
    """What 8-bit codes stand for, before their scale."""
    return codes.view(FP8[kv][0]).float()


def _run_own(s):
    import paged_kv_cache_153_gb300 as pkv
    case = s["case"]
    op = case["op"]
    if op == "rope":
        kw = dict(amplitude=s["amp"], layout=case["layout"])
        if case["kv"] in FP8:
            call = pkv.pkv_rope_append_fp8 if case["kv"] == "e4m3" else pkv.pkv_rope_append_e5m2
            call(s["q"], s["k"], s["v"], s["pos"], s["slots"], s["turns"], s["q_out"], s["kc"], s["vc"], s["ks"],
                 s["vs"], **kw)
            return s["q_out"], s["kc"].view(FP8[case["kv"]][0]), s["vc"].view(FP8[case["kv"]][0])
        pkv.pkv_rope_append(s["q"], s["k"], s["v"], s["pos"], s["slots"], s["turns"], s["q_out"], s["kc"], s["vc"],
                            **kw)
        return s["q_out"], s["kc"], s["vc"]
    if op == "bounds":
        call = {"e4m3": pkv.pkv_kv_block_bounds_fp8, "e5m2": pkv.pkv_kv_block_bounds_e5m2}.get(
            case["kv"], pkv.pkv_kv_block_bounds)
        call(s["kc"], s["tables"], s["lens"], s["bounds"], new_lens=s["new"], max_new_len=s["max_new"])
        return s["bounds"]
    if op == "scores":
        pkv.pkv_block_scores(s["q"], s["bounds"], s["tables"], s["lens"], s["scores"], scale=s["scale"],
                             max_context_len=s["max_ctx"])
        return s["scores"]
    if op == "select":
        pkv.pkv_select_blocks(s["scores"], s["lens"], s["selected"], num_first=case["first"], num_last=case["last"])
        return s["selected"]
    if op == "sparse":
        if case["kv"] in FP8:
            call = (pkv.pkv_paged_decode_attention_sparse_fp8 if case["kv"] == "e4m3"
                    else pkv.pkv_paged_decode_attention_sparse_e5m2)
            call(s["q"], s["kc"], s["vc"], s["ks"], s["vs"], s["tables"], s["lens"], s["selected"], s["out"],
                 scale=s["scale"], workspace=s["ws"])
        else:
            pkv.pkv_paged_decode_attention_sparse(s["q"], s["kc"], s["vc"], s["tables"], s["lens"], s["selected"],
                                                  s["out"], scale=s["scale"], workspace=s["ws"])
        return s["out"]
    pkv.pkv_paged_decode_attention_prefix(s["q"], s["kc"], s["vc"], s["tables"], s["lens"], s["starts"], s["pre"],
                                          s["out"], scale=s["scale"], max_context_len=s["max_ctx"],
                                          max_prefix_len=s["max_pre"], workspace=s["ws"])
    return s["out"]


def _inverse_frequencies(case):
    """Scaled inverse frequencies (64 bits) and the amplitude of the rotation."""
    rot, base, f, orig = case["rot"], case["base"], case["factor"], 8192.0
    i = np.arange(rot // 2, dtype=np.float64)
    kind = case["scaling"]
    if kind == "base":
        return (base * f ** (rot / (rot - 2.0))) ** (-2.0 * i / rot), 1.0
    inv = base ** (-2.0 * i / rot)
    if kind == "linear":
        return inv / f, 1.0
    if kind == "ramp":
        def dim_of(turns):
            return rot * math.log(orig / (turns * 2 * math.pi)) / (2 * math.log(base))
        low, high = max(math.floor(dim_of(32.0)), 0), min(math.ceil(dim_of(1.0)), rot - 1)
        ramp = np.clip((i - low) / max(high - low, 0.001), 0, 1)
        return inv / f * ramp + inv * (1 - ramp), 0.1 * math.log(f) + 1.0
    if kind == "wavelength":
        turns = orig * inv / (2 * math.pi)
        w = np.clip((turns - 1.0) / (4.0 - 1.0), 0, 1)
        return (1 - w) * inv / f + w * inv, 1.0
    return inv, 1.0


def _rotate(x, cos, sin, layout, rot):
    """x [tokens, heads, d] in 32 bits, cos and sin [tokens, rot / 2]."""
    c, n = cos[:, None], sin[:, None]
    y = x.clone()
    if layout == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * c - b * n, a * n + b * c
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * c - b * n, a * n + b * c
    return y


def _softmax_rows(q, k, v, scale, keep=None):
    """q [..., g, d], k and v [..., n, d] in 32 bits; keep: rows that count."""
    p = torch.matmul(q, k.transpose(-1, -2)) * scale
    if keep is not None:
        p = p.masked_fill(~keep, float("-inf"))
    p = torch.exp(p - p.amax(-1, keepdim=True).clamp_min(-3e38))
    return torch.matmul(p / p.sum(-1, keepdim=True).clamp_min(1e-38), v)


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op == "rope":
        ang = s["pos"].double()[:, None] * s["inv"]
        cos, sin = (s["amp"] * torch.cos(ang)).float(), (s["amp"] * torch.sin(ang)).float()
        s["q_out"].copy_(_rotate(s["q"].float(), cos, sin, case["layout"], case["rot"]))
        k = _rotate(s["k"].float(), cos, sin, case["layout"], case["rot"])
        blk, off = s["slots"] // BS, s["slots"] % BS
        if case["kv"] in FP8:
            t, top = FP8[case["kv"]]
            for x, c, sc in ((k, s["kc"], s["ks"]), (s["v"].float(), s["vc"], s["vs"])):
                c[blk, :, off] = (x / sc[:, None]).clamp(-top, top).to(t).view(torch.uint8)
            return s["q_out"], s["kc"].view(FP8[case["kv"]][0]), s["vc"].view(FP8[case["kv"]][0])
        s["kc"][blk, :, off] = k.to(s["kc"].dtype)
        s["vc"][blk, :, off] = s["v"]
        return s["q_out"], s["kc"], s["vc"]
    if op == "bounds":
        lens, new = s["lens"].long(), (s["lens"] if s["new"] is None else s["new"]).long()
        i = torch.arange(s["tables"].shape[1], device="cuda")
        live = (i < ((lens + BS - 1) // BS)[:, None]) & (i >= ((lens - new) // BS)[:, None]) & (new > 0)[:, None]
        b, i = live.nonzero(as_tuple=True)
        for at in range(0, b.numel(), 4096):          # pieces bound the 32-bit copies
            bb, ii = b[at:at + 4096], i[at:at + 4096]
            ids = s["tables"][bb, ii].long()
            k = s["kc"][ids]
            k = _values(k, case["kv"]) if case["kv"] in FP8 else k.float()
            past = (torch.arange(BS, device="cuda") >= (lens[bb] - BS * ii)[:, None])[:, None, :, None]
            s["bounds"][ids, :, 0] = k.masked_fill(past, float("inf")).amin(2).to(s["bounds"].dtype)
            s["bounds"][ids, :, 1] = k.masked_fill(past, float("-inf")).amax(2).to(s["bounds"].dtype)
        return s["bounds"]
    if op == "scores":
        for b in range(case["seqs"]):
            n = (s["lens"][b] + BS - 1) // BS
            ids = s["tables"][b].long().clamp_min(0)
            bd = s["bounds"][ids].float()                                        # [blocks, hkv, 2, d]
            q = s["q"][b].float().view(case["hkv"], -1, 1, case["d"])            # [hkv, group, 1, d]
            top = torch.maximum(q * bd[:, :, 0].transpose(0, 1)[:, None], q * bd[:, :, 1].transpose(0, 1)[:, None])
            sc = top.sum(-1).amax(1) * s["scale"]
            live = torch.arange(sc.shape[1], device="cuda") < n
            s["scores"][b] = torch.where(live, sc, s["scores"][b])
        return s["scores"]
    if op == "select":
        sc = s["scores"]
        nblk = ((s["lens"] + BS - 1) // BS).long().view(-1, 1, 1)
        i = torch.arange(sc.shape[2], device="cuda")
        key = sc.masked_fill((i < case["first"]) | (i >= nblk - case["last"]), float("inf"))
        key = key.masked_fill(i >= nblk, float("-inf"))
        order = key.sort(dim=2, descending=True, stable=True).indices[..., :case["budget"]]
        order = order.masked_fill(order >= nblk, sc.shape[2]).sort(dim=2).values
        order = torch.where(order == sc.shape[2], -1, order).to(torch.int32)
        s["selected"].fill_(-1)
        s["selected"][..., :order.shape[2]] = order
        return s["selected"]
    hkv, d = case["hkv"], case["d"]
    if op == "sparse":
        for b in range(case["seqs"]):
            sel = s["selected"][b].long()                                        # [hkv, budget]
            ids = s["tables"][b].long()[sel.clamp_min(0)].clamp_min(0)
            pos = sel[..., None] * BS + torch.arange(BS, device="cuda")
            keep = ((sel[..., None] >= 0) & (pos < s["lens"][b])).view(hkv, 1, -1)
            h = torch.arange(hkv, device="cuda")[:, None]
            k, v = s["kc"][ids, h], s["vc"][ids, h]                              # [hkv, budget, 16, d]
            if case["kv"] in FP8:
                k = _values(k, case["kv"]) * s["ks"].view(-1, 1, 1, 1)
                v = _values(v, case["kv"]) * s["vs"].view(-1, 1, 1, 1)
            o = _softmax_rows(s["q"][b].float().view(hkv, -1, d), k.float().reshape(hkv, -1, d),
                              v.float().reshape(hkv, -1, d), s["scale"], keep)
            s["out"][b] = o.reshape(-1, d).to(s["out"].dtype)
        return s["out"]
    ctx = s["host"]["ctx"]
    for b in range(len(ctx)):
        n = int(ctx[b])
        ids = s["tables"][b, :_nblk(n)].long()
        k = s["kc"][ids].transpose(0, 1).reshape(hkv, -1, d)[:, :n].float()
        v = s["vc"][ids].transpose(0, 1).reshape(hkv, -1, d)[:, :n].float()
        if n == 0:
            s["out"][b] = 0
            continue
        o = _softmax_rows(s["q"][b].float().view(hkv, -1, d), k, v, s["scale"])
        s["out"][b] = o.reshape(-1, d).to(s["out"].dtype)
    return s["out"]


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    op = case["op"]
    lens = _lens_of(case)
    e = 1 if case.get("kv") in FP8 else 2
    hkv, d, hq = case["hkv"], case.get("d", 0), case.get("hq", 0)
    n = case["seqs"]
    blocks = int(_nblk(lens.astype(np.int64)).sum())
    if op == "rope":
        t = n * case["new"]
        return {"bytes": t * (2 * (2 * hq + 2 * hkv) * d + 2 * hkv * d * e + 12),
                "flops": t * (hq + hkv) * case["rot"] * 3}
    if op == "bounds":
        if case["new"]:
            first = np.maximum(lens - case["new"], 0) // BS
            blocks = int((_nblk(lens) - first).sum())
            rows = int((lens - first * BS).sum())
        else:
            rows = int(lens.astype(np.int64).sum())
        return {"bytes": rows * hkv * d * e + blocks * hkv * d * 4, "flops": 2 * rows * hkv * d}
    if op == "scores":
        return {"bytes": blocks * (hkv * (4 * d + 4) + 4) + n * hq * d * 2, "flops": 4 * blocks * hq * d}
    if op == "select":
        return {"bytes": blocks * hkv * 4 + n * hkv * case["budget"] * 4, "flops": blocks * hkv}
    if op == "sparse":
        listed_blocks = int(np.minimum(_nblk(lens), case["budget"]).sum())
        return {"bytes": listed_blocks * BS * hkv * d * 2 * e + n * (4 * hq * d + 4 * hkv * case["budget"]),
                "flops": 4 * listed_blocks * BS * hq * d}
    g = case["groups"]
    pre = [case["prefix"] if j == 0 else max(1, case["prefix"] // (j + 1)) for j in range(g)]
    tail = int(lens.sum())
    shared = sum(p // BS * BS for p in pre)
    every = sum(p * n for p in pre) + tail
    private = every - sum(p // BS * BS * n for p in pre)
    return {"bytes": (shared + private) * hkv * d * 4 + 4 * g * n * hq * d, "flops": 4 * every * hq * d}


# ---------------------------------------------------------------------------
# from the definitions, in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rope":
        return _exact_rope(case, s)
    if op == "bounds":
        return _exact_bounds(case, s)
    if op == "scores":
        out = s["scores"].double()
        for b in range(case["seqs"]):
            m = -(-int(s["lens"][b]) // BS)
            for g in range(case["hkv"]):
                per = case["hq"] // case["hkv"]
                bd = s["bounds"][s["tables"][b, :m].long(), g].double()
                qs = s["q"][b, g * per:(g + 1) * per].double()
                up = torch.where(qs[:, None] >= 0, qs[:, None] * bd[None, :, 1], qs[:, None] * bd[None, :, 0])
                out[b, g, :m] = up.sum(2).max(0).values * s["scale"]
        return out
    if op == "select":
        return None
    hkv, d = case["hkv"], case["d"]
    per = case["hq"] // hkv
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    tok = torch.arange(BS, device="cuda")
    for b in range(s["q"].shape[0]):
        n = int(s["lens"][b])
        if n == 0:
            continue
        for g in range(hkv):
            if op == "sparse":
                sel = s["selected"][b, g]
                sel = sel[sel >= 0].long()
            else:
                sel = torch.arange(-(-n // BS), device="cuda")
            at = (sel[:, None] * BS + tok).reshape(-1)
            rows = []
            for name, sc in (("kc", "ks"), ("vc", "vs")):
                x = s[name][s["tables"][b].long()[sel], g].reshape(-1, d)[at < n]
                x = x.view(FP8[case["kv"]][0]).double() * s[sc][g].double() if sc in s else x.double()
                rows.append(x)
            logit = s["q"][b, g * per:(g + 1) * per].double() @ rows[0].T * s["scale"]
            out[b, g * per:(g + 1) * per] = torch.softmax(logit, 1) @ rows[1]
    return out


def _exact_rope(case, s):
    """A rotation is a product of complex numbers."""
    rot, base, f = case["rot"], case["base"], case["factor"]
    freq, amp = [], 1.0
    for i in range(rot // 2):
        b = base * f ** (rot / (rot - 2)) if case["scaling"] == "base" else base
        w = math.exp(-2 * i / rot * math.log(b))
        turns = 8192 * w / (2 * math.pi)             # full turns over the original context
        if case["scaling"] == "linear":
            w /= f
        elif case["scaling"] == "wavelength":
            share = 0.0 if turns < 1 else 1.0 if turns > 4 else (turns - 1) / 3
            w = w * (share + (1 - share) / f)
        elif case["scaling"] == "ramp":
            edge = [rot * math.log(8192 / (r * 2 * math.pi)) / (2 * math.log(base)) for r in (32, 1)]
            lo, hi = max(math.floor(edge[0]), 0), min(math.ceil(edge[1]), rot - 1)
            share = min(max((i - lo) / max(hi - lo, 0.001), 0), 1)
            w = w * (1 - share) + w / f * share
            amp = 1 + math.log(f) / 10
        freq.append(w)
    phase = s["pos"].double()[:, None] * torch.tensor(freq, dtype=torch.float64, device="cuda")
    turn = torch.polar(torch.full_like(phase, amp), phase)[:, None]

    def turned(x):
        x = x.double()
        if case["layout"] == "half":
            z = torch.complex(x[..., :rot // 2], x[..., rot // 2:rot]) * turn
            return torch.cat([z.real, z.imag, x[..., rot:]], -1)
        z = torch.complex(x[..., 0:rot:2], x[..., 1:rot:2]) * turn
        return torch.cat([torch.view_as_real(z).flatten(-2), x[..., rot:]], -1)

    outs = [turned(s["q"])]
    for rows, cache, scale in ((turned(s["k"]), "kc", "ks"), (s["v"].double(), "vc", "vs")):
        if scale in s:
            top = FP8[case["kv"]][1]
            rows = (rows / s[scale].double()[:, None]).clamp(-top, top)
            full = s[cache].view(FP8[case["kv"]][0]).double()
        else:
            full = s[cache].double()
        full[s["slots"] // BS, :, s["slots"] % BS] = rows
        outs.append(full)
    return tuple(outs)


def _exact_bounds(case, s):
    out = s["bounds"].double()
    for b in range(case["seqs"]):
        n = int(s["lens"][b])
        new = n if s["new"] is None else int(s["new"][b])
        if new == 0:
            continue
        lo, hi = (n - new) // BS, -(-n // BS)
        ids = s["tables"][b, lo:hi].long()
        k = s["kc"][ids]
        k = (k.view(FP8[case["kv"]][0]) if case["kv"] in FP8 else k).double()
        out[ids, :, 0], out[ids, :, 1] = k.min(2).values, k.max(2).values
        used = n - (hi - 1) * BS                     # the last block may be part full
        out[ids[-1], :, 0] = k[-1, :, :used].min(1).values
        out[ids[-1], :, 1] = k[-1, :, :used].max(1).values
    return out
