"""Pins of the rotary oracle, and the library's frequency plan against it
(host code: no GPU)."""
import ctypes as C

import numpy as np
import pytest

from oracle import rope as orp

SCALINGS = ["none", "linear", "base", "ramp", "wavelength"]


@pytest.fixture(scope="module")
def pkv():
    import __graft_entry__ as g
    g.build()
    import paged_kv_cache_153_gb300 as m
    return m


def test_rotation_keeps_norms_and_scores_depend_on_the_distance():
    rng = np.random.default_rng(0)
    for layout in ("half", "interleaved"):
        f, amp = orp.frequencies(32)
        q, k = rng.standard_normal((1, 3, 64)), rng.standard_normal((1, 3, 64))
        q2 = orp.rotate(q, [1234], f, amp, layout)
        assert np.allclose(np.linalg.norm(q2, axis=-1), np.linalg.norm(q, axis=-1))
        assert np.array_equal(q2[..., 32:], q[..., 32:])
        assert np.array_equal(orp.rotate(q, [0], f, amp, layout), q)
        near = (orp.rotate(q, [17], f, amp, layout) * orp.rotate(k, [5], f, amp, layout)).sum(-1)
        far = (orp.rotate(q, [100012], f, amp, layout) * orp.rotate(k, [100000], f, amp, layout)).sum(-1)
        assert np.allclose(near, far)


def test_layouts_are_permutations_of_each_other():
    rng = np.random.default_rng(1)
    f, amp = orp.frequencies(64)
    x = rng.standard_normal((2, 1, 64))
    perm = np.concatenate([np.arange(0, 64, 2), np.arange(1, 64, 2)])
    a = orp.rotate(x[..., perm], [3, 9], f, amp, "half")
    b = orp.rotate(x, [3, 9], f, amp, "interleaved")
    assert np.allclose(a, b[..., perm])


def test_first_pair_by_hand():
    f, amp = orp.frequencies(16)
    assert f[0] == 1.0 and amp == 1.0
    x = np.zeros((1, 1, 64))
    x[..., 0] = 1.0
    out = orp.rotate(x, [2], f, amp, "half")
    assert out[0, 0, 0] == pytest.approx(np.cos(2.0)) and out[0, 0, 8] == pytest.approx(np.sin(2.0))


@pytest.mark.parametrize("scaling", SCALINGS)
@pytest.mark.parametrize("rot,base", [(16, 10000.0), (64, 500000.0), (128, 10000.0)])
def test_plan_matches_the_frequencies(pkv, scaling, rot, base):
    turns, amp = pkv.pkv_rope_plan(rot, base=base, scaling=scaling, factor=8.0, original_context=4096)
    f, ref_amp = orp.frequencies(rot, base, scaling, 8.0, 4096.0)
    assert turns.dtype == np.int64 and turns.shape == (rot // 2,)
    got = turns.view(np.uint64).astype(np.float64) / 2.0 ** 64
    # pow, log and one division in float64 on both sides: a few units of 2^-53
    # (the exponent's rounding, 2^-53 * ln(base) relative, is the largest),
    # and the fixed point's own step, half of 2^-64 turns
    assert np.all(np.abs(got - f / (2 * np.pi)) <= 64 * 2.0 ** -53 * f / (2 * np.pi) + 0.5 * 2.0 ** -64)
    assert amp == pytest.approx(ref_amp, rel=1e-7)


def test_scalings_leave_the_fast_pairs_and_divide_the_slow_ones(pkv):
    plain = pkv.pkv_rope_plan(128)[0].astype(np.float64)
    for scaling in ("ramp", "wavelength"):
        r = pkv.pkv_rope_plan(128, scaling=scaling, factor=8.0)[0] / plain
        # (the slowest plain pair has 3e14 steps of 2^-64: a ratio is good to 1e-13)
        assert r[0] == 1.0 and abs(r[-1] - 0.125) < 1e-12 and np.all(np.diff(r) <= 1e-12)
    # a factor of one changes nothing
    for scaling in SCALINGS:
        assert np.allclose(pkv.pkv_rope_plan(128, scaling=scaling, factor=1.0)[0], plain, rtol=1e-12)


def test_plan_refusals(pkv):
    buf, amp = (C.c_uint64 * 64)(), C.c_float()

    def plan(rot=64, base=1e4, kind=0, factor=2.0, orig=8192.0, low=1.0, high=4.0, out=buf, a=amp):
        return pkv.lib.pkv_rope_plan(rot, base, kind, factor, orig, low, high, out, None if a is None else C.byref(a))
    assert plan() == 0
    for bad in (dict(rot=0), dict(rot=-2), dict(rot=33), dict(base=1.0), dict(base=float("nan")), dict(base=float("inf")),
                dict(kind=5), dict(kind=-1), dict(kind=1, factor=0.5), dict(kind=2, factor=float("nan")),
                dict(kind=2, rot=2), dict(kind=3, orig=0.0), dict(kind=3, low=0.0), dict(kind=4, low=4.0),
                dict(kind=4, high=float("inf")), dict(out=None), dict(a=None)):
        assert plan(**bad) == 1, bad
    with pytest.raises(ValueError):
        pkv.pkv_rope_plan(64, scaling="other")


def test_append_refusals_before_any_cuda_call(pkv):
    a, odd = C.c_void_p(4096), C.c_void_p(4096 + 8)

    def call(q=a, qs=512, k=a, ks=256, v=a, vs=256, pos=a, slots=a, n=3, turns=a, rot=64, layout=0, amp=1.0, qo=a,
             qos=512, kc=a, vc=a, nb=8, hq=4, hkv=2, d=128, bs=16, dt=1, fn="pkv_rope_append", scales=()):
        return getattr(pkv.lib, fn)(q, qs, k, ks, v, vs, pos, slots, n, turns, rot, layout, amp, qo, qos, kc, vc, nb,
                                    *scales, hq, hkv, d, bs, dt, None, None)
    for bad in (dict(n=-1), dict(nb=-1), dict(amp=float("nan")), dict(dt=2), dict(layout=2), dict(rot=0), dict(rot=144),
                dict(q=None), dict(qo=None), dict(k=None), dict(v=None), dict(pos=None), dict(slots=None),
                dict(turns=None), dict(q=None, qo=None, k=None, v=None), dict(kc=None), dict(vc=None),
                dict(qs=504), dict(qos=511), dict(qs=516), dict(ks=248), dict(vs=260), dict(q=odd), dict(qo=odd),
                dict(k=odd), dict(v=odd), dict(kc=odd), dict(vc=odd), dict(hq=0), dict(hkv=0)):
        assert call(**bad) == 1, bad
    for bad in (dict(rot=24), dict(d=96, rot=32), dict(bs=32)):
        assert call(**bad) == 2, bad
    assert call(n=0) == 0
    for fn in ("pkv_rope_append_fp8", "pkv_rope_append_e5m2"):
        assert call(fn=fn, scales=(None, a)) == 1 and call(fn=fn, scales=(a, None)) == 1
