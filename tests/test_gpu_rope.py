"""Rotary append on the GPU against the float64 rotation.

Tolerances, from the arithmetic: the angle's fraction of a turn is rounded to
fp32 (2^-25 half turns of at most one: 1e-7 rad), sincospi is within 2 units of
2^-24, the products and their sum round three times, so a turned element is
within (|x| + |y|) a 8e-7 of the exact one before its one rounding to the
output type (half a step: eps / 2 relative, or half the type's smallest step).
"""
import numpy as np
import pytest
import torch

from oracle import rope as orp
from tests import gpu_util as gu

pytestmark = pytest.mark.gpu

FP8 = {"e4m3": (torch.float8_e4m3fn, 448.0, 2.0 ** -4, 2.0 ** -10), "e5m2": (torch.float8_e5m2, 57344.0, 2.0 ** -3, 2.0 ** -17)}


@pytest.fixture(scope="module")
def pkv():
    import __graft_entry__ as g
    g.build()
    import paged_kv_cache_153_gb300 as m
    return m


class Case:
    def __init__(self, pkv, *, tokens, hq, hkv, d, rot, dtype, kv=None, layout="half", scaling="none", pos=None, seed=0,
                 strided=True, blocks=None):
        self.__dict__.update(locals())
        g = torch.Generator().manual_seed(seed)
        t = gu.TORCH_16[dtype]
        extra = 2 if strided else 0     # a gap of two heads behind each token's heads
        self.qkv = torch.randn((tokens, hq + 2 * hkv + extra, d), generator=g).to(t).cuda()
        self.q, self.k, self.v = self.qkv[:, :hq], self.qkv[:, hq:hq + hkv], self.qkv[:, hq + hkv:hq + 2 * hkv]
        self.nb = blocks or tokens // 8 + 3
        self.pos = torch.randint(0, 1 << 20, (tokens,), generator=g, dtype=torch.int32) if pos is None else \
            torch.tensor(pos, dtype=torch.int32)
        self.slots = torch.randperm(self.nb * 16, generator=g)[:tokens].to(torch.int64)
        shape = (2, self.nb, hkv, 16, d)
        if kv in FP8:
            self.caches = torch.randint(0, 120, shape, generator=g, dtype=torch.uint8).cuda()
            self.scales = (torch.rand((2, hkv), generator=g) * 0.02 + 0.002).cuda()
        else:
            self.caches = torch.randn(shape, generator=g).to(t).cuda()
        self.before = self.caches.clone()
        self.q_out = torch.full((tokens, hq, d), float("nan"), dtype=t, device="cuda")
        turns, self.amp = pkv.pkv_rope_plan(rot, scaling=scaling, factor=4.0)
        self.freq, ref_amp = orp.frequencies(rot, scaling=scaling, factor=4.0)
        assert abs(self.amp - ref_amp) < 1e-6
        self.turns = torch.from_numpy(turns).cuda()
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run(self, stream=None, q=True, kv=True, q_out=None):
        fn = {"e4m3": self.pkv.pkv_rope_append_fp8, "e5m2": self.pkv.pkv_rope_append_e5m2}.get(
            self.kv, self.pkv.pkv_rope_append)
        scales = tuple(self.scales) if self.kv in FP8 else ()
        fn(self.q if q else None, self.k if kv else None, self.v if kv else None, self.pos.cuda(),
           self.slots.cuda() if kv else None, self.turns, (self.q_out if q_out is None else q_out) if q else None,
           *(self.caches if kv else (None, None)), *scales, layout=self.layout, amplitude=self.amp,
           err_flag=self.err, stream=stream)
        torch.cuda.synchronize()

    def want(self, x):
        x = x.double().cpu().numpy()
        out = orp.rotate(x, self.pos.clamp_min(0).numpy(), self.freq, self.amp, self.layout)
        half, r = self.rot // 2, np.abs(x)
        size = r.copy()
        if self.layout == "half":
            size[..., :half] = size[..., half:2 * half] = r[..., :half] + r[..., half:2 * half]
        else:
            size[..., 0:2 * half:2] = size[..., 1:2 * half:2] = r[..., 0:2 * half:2] + r[..., 1:2 * half:2]
        slack = size * self.amp * 8e-7
        slack[..., self.rot:] = 0
        return out, slack

    def close16(self, got, x):
        ref, slack = self.want(x)
        t = gu.TORCH_16[self.dtype]
        fi = torch.finfo(t)
        lim = slack + (np.abs(ref) + slack) * fi.eps / 2 + fi.smallest_normal * fi.eps / 2
        diff = np.abs(got.double().cpu().numpy() - ref)
        assert np.all(diff <= lim), float((diff - lim).max())

    def check(self, q=True, kv=True, live=None):
        live = np.ones(self.tokens, dtype=bool) if live is None else np.asarray(live)
        if q:
            self.close16(self.q_out, self.q)
        touched = torch.zeros((self.nb, 16), dtype=torch.bool)
        blk, off = self.slots // 16, self.slots % 16
        touched[blk[live], off[live]] = kv
        keep = ~touched.view(self.nb, 1, 16, 1).expand(self.before[0].shape).cuda()
        for i in range(2):
            assert torch.equal(self.caches[i][keep], self.before[i][keep])
        if not kv:
            return
        rows = [c[blk[live], :, off[live]] for c in self.caches]
        if self.kv in FP8:
            t, top, half, tiny = FP8[self.kv]
            for got, x, sc, turned in ((rows[0], self.k, self.scales[0], True), (rows[1], self.v, self.scales[1], False)):
                ref, slack = self.want(x) if turned else (x.double().cpu().numpy(), 0.0)
                s = sc.double().cpu().numpy()[None, :, None]
                ref, slack = (ref / s)[live], (np.broadcast_to(slack, ref.shape) / s)[live]
                # the fp32 quotient rounds once (2^-24) before the code's half step
                lim = slack + (np.abs(ref) + slack) * (half + 2.0 ** -23) + tiny
                clip = np.clip(ref, -top, top)
                got = got.view(t).double().cpu().numpy()
                assert np.all(np.abs(got - clip) <= lim)
        else:
            ref = self.k[torch.from_numpy(live)]
            full = torch.zeros_like(self.k, memory_format=torch.contiguous_format)
            full[torch.from_numpy(live)] = rows[0]
            if live.all():
                self.close16(full, self.k)
            assert ref.shape == rows[0].shape
            assert torch.equal(rows[1], self.v[torch.from_numpy(live)])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("d,rot", [(64, 16), (64, 64), (128, 48), (128, 128)])
@pytest.mark.parametrize("dtype,kv", [("f16", None), ("bf16", None), ("bf16", "e4m3"), ("f16", "e5m2")])
def test_rope_append(pkv, layout, d, rot, dtype, kv):
    c = Case(pkv, tokens=37, hq=6, hkv=3, d=d, rot=rot, dtype=dtype, kv=kv, layout=layout, seed=d + rot)
    c.run()
    c.check()
    assert int(c.err.item()) == 0


@pytest.mark.parametrize("scaling", ["linear", "base", "ramp", "wavelength"])
def test_scaled_frequencies_at_far_positions(pkv, scaling):
    # the last positions an int32 holds, and their neighbours
    pos = [0, 1, 2, 131071, 131072, (1 << 20) - 1, (1 << 24) + 1, (1 << 31) - 2, (1 << 31) - 1]
    # a frequency's own rounding (about 40 units of 2^-53) times 2^31: 1e-5 rad at the far end,
    # so the far tail is checked against the plan's own turns, the rest against the formula
    c = Case(pkv, tokens=len(pos), hq=4, hkv=1, d=128, rot=128, dtype="bf16", scaling=scaling, pos=pos, seed=9)
    u = c.turns.cpu().numpy().view(np.uint64)
    p = c.pos.numpy().astype(np.uint64)[:, None]
    with np.errstate(over="ignore"):
        frac = (p * u).astype(np.float64) / 2.0 ** 64
    near = c.pos.numpy() <= (1 << 20)
    exact = np.mod(c.pos.numpy()[:, None] * c.freq / (2 * np.pi), 1.0)
    gap = np.abs(frac - exact)[near]
    assert np.minimum(gap, 1 - gap).max() < 1e-9
    c.run()
    q = c.q.double().cpu().numpy()
    turn = c.amp * np.exp(2j * np.pi * frac)[:, None]
    z = (q[..., :64] + 1j * q[..., 64:]) * turn
    ref = np.concatenate([z.real, z.imag], -1)
    size = np.tile(np.abs(q[..., :64]) + np.abs(q[..., 64:]), 2) * c.amp
    diff = np.abs(c.q_out.double().cpu().numpy() - ref)
    assert np.all(diff <= size * 8e-7 + (np.abs(ref) + size * 8e-7) * 2.0 ** -8)


@pytest.mark.parametrize("tokens,hq,hkv", [(1, 1, 1), (1, 64, 8), (3, 128, 1), (515, 2, 2)])
def test_token_and_head_counts(pkv, tokens, hq, hkv):
    # one token, one head; more items than a block's threads hold in flight; many blocks
    c = Case(pkv, tokens=tokens, hq=hq, hkv=hkv, d=128, rot=64, dtype="bf16", seed=tokens + hq,
             layout="interleaved", strided=tokens > 1)
    c.run()
    c.check()


def test_in_place_and_parts(pkv):
    c = Case(pkv, tokens=21, hq=4, hkv=2, d=128, rot=96, dtype="f16", seed=3)
    c.run(kv=False)                      # q alone: the caches stay
    c.check(kv=False)
    first = c.q_out.clone()
    c.run(q=False)                       # append alone
    c.check(q=False)
    keep = c.qkv.clone()
    c.run(kv=False, q_out=c.q)           # q turned where it lies, heads behind it untouched
    assert torch.equal(c.q, first) and torch.equal(c.qkv[:, 4:], keep[:, 4:])


def test_padding_and_slots_out_of_range(pkv):
    c = Case(pkv, tokens=12, hq=4, hkv=2, d=64, rot=32, dtype="bf16", seed=4)
    c.pos[3] = -1                        # padding: nothing is written for it
    c.slots[5] = -1                      # turned, not appended
    good = c.slots.clone()
    c.run()
    assert int(c.err.item()) == 0
    live = np.ones(12, dtype=bool)
    live[[3, 5]] = False
    assert torch.isnan(c.q_out[3]).all() and not torch.isnan(c.q_out[[5]]).any()
    c.check(q=False, live=live)
    c.slots = good
    c.slots[7] = c.nb * 16               # one past the pool
    c.run()
    assert int(c.err.item()) == 4
    assert not torch.isnan(c.q_out[7]).any()
    touched = c.caches.clone()
    c.slots[7] = -1
    c.run()
    assert torch.equal(touched, c.caches)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("kv", ["fp8", "e5m2"])
def test_every_16_bit_value_under_many_scales(pkv, dtype, kv):
    # v rows get the codes of the plain append (an IEEE division): ordinary scales, powers of two, scales
    # whose quotients are often exact or ties, and scales at the ends of the range or outside it
    scales = [1.0, 0.5, 2.0 ** -9, 0.0234567, 1.5, 0.75, 3.0, 1.1, 0.9999999, 448.0, 1e-30, 1e-38, 1e-44, 3e38, 0.0,
              -0.7, float("inf"), float("nan"), 2.0 ** 100, 2.0 ** -100, 7.3e29, 1.3e-29, 5.0, 1 / 3]
    h = len(scales)
    x = torch.arange(65536, dtype=torch.int32).to(torch.uint16).view(gu.TORCH_16[dtype]).view(512, 1, 128)
    v = x.expand(512, h, 128).contiguous().cuda()
    s = torch.tensor(scales, dtype=torch.float32, device="cuda")
    caches = [torch.zeros((32, h, 16, 128), dtype=torch.uint8, device="cuda") for _ in range(4)]
    slots = torch.arange(512, dtype=torch.int64, device="cuda")
    pos = torch.zeros(512, dtype=torch.int32, device="cuda")
    turns = torch.from_numpy(pkv.pkv_rope_plan(128)[0]).cuda()
    getattr(pkv, f"pkv_rope_append_{kv}")(None, v, v, pos, slots, turns, None, caches[0], caches[1], s, s)
    getattr(pkv, f"pkv_kv_append_{kv}")(v, v, slots, caches[2], caches[3], s, s)
    torch.cuda.synchronize()
    assert torch.equal(caches[1], caches[3])
    # and k rows at position 0, where the rotation is x 1 - y 0: the same but for what 0 times infinity and the
    # sign of a zero change
    y = torch.roll(x.double(), 64, 2)
    plain = (torch.isfinite(x.double()) & torch.isfinite(y) & (x.double() != 0)).expand(512, h, 128)
    plain = plain.reshape(32, 16, h, 128).transpose(1, 2).cuda()
    assert torch.equal(caches[0][plain], caches[2][plain])


def test_nonfinite_values_stay_in_their_pair(pkv):
    c = Case(pkv, tokens=4, hq=2, hkv=1, d=64, rot=64, dtype="bf16", seed=5)
    c.q[1, 0, 3] = float("inf")
    c.q[2, 1, 35] = float("nan")
    c.run()
    bad = ~torch.isfinite(c.q_out)
    want = torch.zeros_like(bad)
    want[1, 0, 3] = want[1, 0, 35] = want[2, 1, 3] = want[2, 1, 35] = True
    assert torch.equal(bad, want)


def test_matches_turning_first_and_appending_after(pkv):
    # the turned k rounded to 16 bits and appended by pkv_kv_append: the same bits
    c = Case(pkv, tokens=50, hq=4, hkv=4, d=128, rot=128, dtype="bf16", seed=6)
    c.run()
    turned = torch.empty((50, 4, 128), dtype=torch.bfloat16, device="cuda")
    pkv.pkv_rope_append(c.k, None, None, c.pos.cuda(), None, c.turns, turned, None, None, layout=c.layout,
                        amplitude=c.amp)
    other = c.before.clone()
    pkv.pkv_kv_append(turned, c.v.contiguous(), c.slots.cuda(), other[0], other[1])
    torch.cuda.synchronize()
    assert torch.equal(other, c.caches)


def test_other_stream_and_graph(pkv):
    c = Case(pkv, tokens=9, hq=4, hkv=2, d=128, rot=128, dtype="f16", seed=7)
    c.run()
    ref, caches = c.q_out.clone(), c.caches.clone()
    c.q_out.fill_(float("nan"))
    pos, slots = c.pos.cuda(), c.slots.cuda()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()

    def call():
        pkv.pkv_rope_append(c.q, c.k, c.v, pos, slots, c.turns, c.q_out, *c.caches, layout=c.layout, amplitude=c.amp)
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    assert torch.equal(c.q_out, ref) and torch.equal(c.caches, caches)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    c.q_out.fill_(float("nan"))
    c.caches.copy_(c.before)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(c.q_out, ref) and torch.equal(c.caches, caches)


def test_binding_refuses_shapes_that_do_not_fit(pkv):
    c = Case(pkv, tokens=5, hq=4, hkv=2, d=64, rot=32, dtype="f16", seed=8)
    pos, slots = c.pos.cuda(), c.slots.cuda()
    with pytest.raises(ValueError):      # heads not contiguous
        pkv.pkv_rope_append(c.qkv.transpose(0, 1), None, None, pos, None, c.turns, c.qkv.transpose(0, 1), None, None)
    with pytest.raises(ValueError):
        pkv.pkv_rope_append(c.q, c.k, c.v, pos, slots[:4], c.turns, c.q_out, *c.caches)
    with pytest.raises(ValueError):
        pkv.pkv_rope_append(c.q, None, None, pos, None, c.turns, c.q_out[:3], None, None)
    with pytest.raises(ValueError):
        pkv.pkv_rope_append(c.q, None, None, pos, None, c.turns, c.q_out, None, None, layout="other")
    with pytest.raises(TypeError):
        pkv.pkv_rope_append(c.q, None, None, pos.long(), None, c.turns, c.q_out, None, None)
    with pytest.raises(ValueError):
        pkv.pkv_rope_append(c.q, c.k, c.v, pos, slots.int(), c.turns, c.q_out, *c.caches)
    with pytest.raises(pkv.PkvError) as e:   # one row of q for every token
        pkv.pkv_rope_append(c.q[:1].expand(5, 4, 64), None, None, pos, None, c.turns, c.q_out, None, None)
    assert e.value.status == 1
    pkv.pkv_rope_append(c.q[:0], None, None, pos[:0], None, c.turns, c.q_out[:0], None, None)   # no tokens
    with pytest.raises(pkv.PkvError) as e:   # 24 turned elements
        pkv.pkv_rope_append(c.q, None, None, pos, None, c.turns[:12], c.q_out, None, None)
    assert e.value.status == 2


def test_far_slots_of_a_large_pool(pkv):
    # slots past 4 GiB of the cache: byte offsets need 64 bits
    nb = 140000                          # 32 KiB a block: 4.6 GB
    c = Case(pkv, tokens=6, hq=8, hkv=8, d=128, rot=128, dtype="bf16", seed=10)
    far = torch.zeros((2, nb, 8, 16, 128), dtype=torch.bfloat16, device="cuda")
    slots = torch.tensor([16 * nb - 1, 0, 16 * nb - 40, 17, 16 * (nb - 9) + 3, 16 * 131072], device="cuda")
    pkv.pkv_rope_append(c.q, c.k, c.v, c.pos.cuda(), slots, c.turns, c.q_out, far[0], far[1], layout=c.layout,
                        amplitude=c.amp, err_flag=c.err)
    c.run()                              # the same rows, near
    for i in range(2):
        near = c.caches[i][c.slots // 16, :, c.slots % 16]
        assert torch.equal(far[i][slots // 16, :, slots % 16], near)
        assert int((far[i] != 0).any(-1).any(1).sum()) == 6
    assert int(c.err.item()) == 0
