"""Rotary positions with the cache write (pa_rope_init, pa_rope_write, pa_rope_write_fp8) against
the formula in 64 bits.

Tolerances.  A turned value is m (a cos t - b sin t) in fp32: the angle is off by at most
pi 2^-25 (its 24-bit half turn) + 2 pi 2^-32, cos and sin by 2 units in the last place (2^-22), the
products and the sum by 2^-24 each: below 2^-20 (|a| + |b|) m together.  bf16 then rounds by half a
step, 2^-8 of the value; e4m3 by 2^-4 of it, or half its smallest step (2^-10 of the scale).
"""
import ctypes
import math

import numpy as np
import pytest
import torch

from paged_kv_decode_cache_gb300 import build as B
from paged_kv_decode_cache_gb300 import pa

YARN = dict(factor=4.0, original_positions=4096.0, low=1.0, high=32.0)
BANDED = dict(factor=8.0, original_positions=8192.0, low=1.0, high=4.0)
SCALINGS = {"none": {}, "linear": dict(factor=3.0), "ntk": dict(factor=4.0), "yarn": YARN, "banded": BANDED}


@pytest.fixture(scope="module", autouse=True)
def _built():
    B.build()


def frequencies(rot, base, scaling):
    """Radians per position of each pair, and the factor on cos and sin, in 64 bits."""
    p, out = SCALINGS[scaling], []
    for i in range(rot // 2):
        f = base ** (-2.0 * i / rot)
        if scaling == "linear":
            f /= p["factor"]
        elif scaling == "ntk":
            f = (base * p["factor"] ** (rot / (rot - 2))) ** (-2.0 * i / rot)
        elif scaling == "yarn":
            edge = [rot * math.log(p["original_positions"] / (2 * math.pi * n)) / (2 * math.log(base))
                    for n in (p["high"], p["low"])]
            lo, hi = max(math.floor(edge[0]), 0), min(math.ceil(edge[1]), rot - 1)
            r = min(max((i - lo) / max(hi - lo, 0.001), 0), 1)
            f = f / p["factor"] * r + f * (1 - r)
        elif scaling == "banded":
            turns = p["original_positions"] * f / (2 * math.pi)
            keep = min(max((turns - p["low"]) / (p["high"] - p["low"]), 0), 1)
            f = f / p["factor"] * (1 - keep) + f * keep
        out.append(f)
    return np.array(out), 0.1 * math.log(p["factor"]) + 1 if scaling == "yarn" else 1.0


def turned(x, positions, rot, layout, f, m):
    """x [N, H, D] turned in 64 bits, and the bound on its fp32 error."""
    x = x.double().cpu().numpy()
    a = positions.double().cpu().numpy()[:, None, None] * f
    cos, sin = m * np.cos(a), m * np.sin(a)
    even, odd = (slice(0, rot, 2), slice(1, rot, 2)) if layout == "interleaved" else \
        (slice(0, rot // 2), slice(rot // 2, rot))
    y, slack = x.copy(), np.zeros_like(x)
    y[..., even] = x[..., even] * cos - x[..., odd] * sin
    y[..., odd] = x[..., even] * sin + x[..., odd] * cos
    slack[..., even] = slack[..., odd] = 2.0 ** -20 * m * (abs(x[..., even]) + abs(x[..., odd]))
    return y, slack


# ---- the plan (host only) --------------------------------------------------------------------


@pytest.mark.parametrize("scaling", SCALINGS)
@pytest.mark.parametrize("rot,base", [(16, 10000.0), (64, 1e6), (128, 500000.0)])
def test_plan_holds_the_frequencies(scaling, rot, base):
    rope = pa.pa_rope_init(rot, base, scaling=scaling, **SCALINGS[scaling])
    f, m = frequencies(rot, base, scaling)
    got = np.array([t / 2.0 ** 64 for t in rope.turn[:rot // 2]]) * 2 * math.pi
    # pow and the divisions differ by a few units of 2^-53
    np.testing.assert_allclose(got, f, rtol=2.0 ** -48, atol=2.0 ** -58)
    assert rope.magnitude == np.float32(m) and rope.rot_dim == rot
    assert not any(rope.turn[rot // 2:])


def test_plan_magnitude_can_be_given():
    assert pa.pa_rope_init(64, 1e4, scaling="yarn", magnitude=1.25, **YARN).magnitude == 1.25


@pytest.mark.parametrize("kw,code", [
    (dict(rot_dim=0), pa.PA_EINVAL), (dict(rot_dim=24), pa.PA_EUNSUPPORTED), (dict(rot_dim=144), pa.PA_EUNSUPPORTED),
    (dict(base=1.0), pa.PA_EINVAL), (dict(base=math.inf), pa.PA_EINVAL), (dict(base=math.nan), pa.PA_EINVAL),
    (dict(scaling="linear", factor=0.0), pa.PA_EINVAL), (dict(scaling="ntk", factor=math.inf), pa.PA_EINVAL),
    (dict(scaling="yarn", **{**YARN, "factor": 0.5}), pa.PA_EINVAL),
    (dict(scaling="yarn", **{**YARN, "original_positions": 0.0}), pa.PA_EINVAL),
    (dict(scaling="banded", **{**BANDED, "low": 4.0}), pa.PA_EINVAL),
    (dict(magnitude=-1.0), pa.PA_EINVAL), (dict(magnitude=math.nan), pa.PA_EINVAL),
])
def test_plan_refusals(kw, code):
    with pytest.raises(pa.PAError) as e:
        pa.pa_rope_init(**{"rot_dim": 64, "base": 1e4, **kw})
    assert e.value.code == code


def test_plan_refuses_unknown_names():
    with pytest.raises(ValueError):
        pa.pa_rope_init(64, 1e4, layout="diagonal")
    with pytest.raises(ValueError):
        pa.pa_rope_init(64, 1e4, scaling="magic")
    rope = pa.Rope()
    assert pa.lib().pa_rope_init(ctypes.byref(rope), 64, 2, 1e4, None) == pa.PA_EINVAL
    assert pa.lib().pa_rope_init(ctypes.byref(rope), 64, 0, 1e4,
                                 ctypes.byref(pa.RopeScaling(9, 1, 1, 1, 2, 0))) == pa.PA_EINVAL
    assert pa.lib().pa_rope_init(None, 64, 0, 1e4, None) == pa.PA_EINVAL


FAKE = ctypes.c_void_p(1 << 20)  # aligned, never dereferenced: these calls fail validation first


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), pa.PA_EINVAL), (dict(q_out=None), pa.PA_EINVAL), (dict(k=None), pa.PA_EINVAL),
    (dict(pos=None), pa.PA_EINVAL), (dict(slots=None), pa.PA_EINVAL), (dict(kc=None), pa.PA_EINVAL),
    (dict(n=-1), pa.PA_EINVAL), (dict(n=1 << 40), pa.PA_EUNSUPPORTED), (dict(Hq=0), pa.PA_EINVAL),
    (dict(q_stride=511), pa.PA_EINVAL), (dict(q_stride=516), pa.PA_EINVAL), (dict(k_stride=128), pa.PA_EINVAL),
    (dict(v_stride=0), pa.PA_EINVAL), (dict(q_out_stride=256), pa.PA_EINVAL),
    (dict(q=ctypes.c_void_p((1 << 20) + 8)), pa.PA_EINVAL), (dict(slots=ctypes.c_void_p((1 << 20) + 4)), pa.PA_EINVAL),
    (dict(desc=pa.CacheDesc(64, 16, 2, 96)), pa.PA_EUNSUPPORTED), (dict(desc=pa.CacheDesc(64, 8, 2, 128)), pa.PA_EUNSUPPORTED),
    (dict(desc=pa.CacheDesc(0, 16, 2, 128)), pa.PA_EINVAL),
    (dict(desc=pa.CacheDesc(64, 16, 2, 64)), pa.PA_EINVAL),        # rot_dim 128 > head_dim
    (dict(rope=None), pa.PA_EINVAL),
])
def test_write_refusals(kw, code):
    rope = pa.pa_rope_init(128, 1e4)
    a = dict(q_out=FAKE, q_out_stride=512, q=FAKE, q_stride=512, k=FAKE, k_stride=256, v=FAKE, v_stride=256, pos=FAKE,
             slots=FAKE, n=3, Hq=4, kc=FAKE, vc=FAKE, desc=pa.CacheDesc(64, 16, 2, 128), rope=ctypes.byref(rope))
    a.update(kw)
    args = [a[x] for x in ("q_out", "q_out_stride", "q", "q_stride", "k", "k_stride", "v", "v_stride", "pos", "slots",
                           "n", "Hq", "kc", "vc", "desc")]
    assert pa.lib().pa_rope_write(*args, a["rope"], None, None) == code
    assert pa.lib().pa_rope_write_fp8(*args, 1.0, 1.0, a["rope"], None, None) == code


def test_write_fp8_refuses_bad_scales_and_takes_no_tokens():
    rope = pa.pa_rope_init(128, 1e4)
    d = pa.CacheDesc(64, 16, 2, 128)
    args = [FAKE, 512, FAKE, 512, FAKE, 256, FAKE, 256, FAKE, FAKE]
    for ks, vs in ((0.0, 1.0), (1.0, -1.0), (math.nan, 1.0), (1.0, math.inf)):
        assert pa.lib().pa_rope_write_fp8(*args, 3, 4, FAKE, FAKE, d, ks, vs, ctypes.byref(rope), None, None) == \
            pa.PA_EINVAL
    assert pa.lib().pa_rope_write(*args, 0, 4, FAKE, FAKE, d, ctypes.byref(rope), None, None) == pa.PA_OK


# ---- on the GPU ------------------------------------------------------------------------------


def inputs(n, hq, hkv, d, bs, packed, seed, far):
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn(n, (hq + 2 * hkv) * d, generator=g).to(torch.bfloat16).cuda()
    q, k, v = (t.view(n, -1, d) for t in qkv.split([hq * d, hkv * d, hkv * d], dim=1))
    if not packed:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    nb = n // bs + 2
    pos = torch.randint(0, far, (n,), generator=g, dtype=torch.int32)
    slots = torch.randperm(nb * bs, generator=g)[:n].contiguous()
    return q, k, v, pos, slots, nb


CASES = [  # n, Hq, Hkv, D, block, rot, layout, scaling, packed, far
    (1, 1, 1, 64, 16, 16, "half", "none", False, 10),
    (1, 28, 4, 128, 16, 128, "half", "none", True, 1 << 20),
    (8, 12, 2, 128, 16, 64, "interleaved", "yarn", True, 2_000_000),
    (7, 3, 3, 64, 32, 48, "interleaved", "banded", False, 100_000),
    (33, 16, 8, 128, 16, 112, "half", "linear", False, 2**31 - 1),
    (257, 8, 1, 64, 256, 64, "half", "ntk", True, 4096),
    (5, 70, 1, 128, 16, 128, "interleaved", "none", True, 50_000),   # more units than a CTA has threads
]


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n,hq,hkv,d,bs,rot,layout,scaling,packed,far", CASES)
def test_matches_the_formula(n, hq, hkv, d, bs, rot, layout, scaling, packed, far, fp8):
    q, k, v, pos, slots, nb = inputs(n, hq, hkv, d, bs, packed, n + hq, far)
    if n > 4:
        slots[1], slots[3] = -1, -7          # padding
        pos[2] = -5                          # a position before the first one turns back
    rope = pa.pa_rope_init(rot, 10000.0, layout=layout, scaling=scaling, **SCALINGS[scaling])
    f, m = frequencies(rot, 10000.0, scaling)
    dtype = torch.uint8 if fp8 else torch.bfloat16
    kc, vc = (torch.full((nb, bs, hkv, d), 9, dtype=dtype, device="cuda") for _ in range(2))
    q_out = torch.full((n, hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ks, vs = 0.03, 0.02
    at = (q_out, q, k, v, pos.cuda(), slots.cuda(), kc, vc)
    if fp8:
        pa.pa_rope_write_fp8(*at, ks, vs, rope, status=status)
    else:
        pa.pa_rope_write(*at, rope, status=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    want, slack = turned(q, pos, rot, layout, f, m)
    got = q_out.double().cpu().numpy()
    assert (abs(got - want) <= 2.0 ** -8 * abs(want) + slack).all()
    kept = slots >= 0
    want_k, slack = turned(k, pos, rot, layout, f, m)
    for pool, want, slack, scale in ((kc, want_k, slack, ks), (vc, v.double().cpu().numpy(), 0 * slack, vs)):
        rows = pool.flatten(0, 1).cpu()
        left = torch.ones(nb * bs, dtype=torch.bool)
        left[slots[kept]] = False
        assert (rows[left] == 9).all()       # nothing else is written
        rows = rows[slots[kept]]
        want, slack = want[kept.numpy()], slack[kept.numpy()]
        if fp8:
            got = rows.view(torch.float8_e4m3fn).double().numpy() * scale
            want = np.clip(want, -448 * scale, 448 * scale)
            assert (abs(got - want) <= 2.0 ** -4 * abs(want) + scale * 2.0 ** -10 + slack + 2.0 ** -22 * abs(want)).all()
        else:
            got = rows.double().numpy()
            assert (abs(got - want) <= 2.0 ** -8 * abs(want) + slack).all()
    if not fp8:  # values that do not turn are copied
        assert torch.equal(q_out[..., rot:], q[..., rot:])
        assert torch.equal(vc.flatten(0, 1)[slots[kept].cuda()], v[kept.cuda()])


LONG_CASES = [  # prompts: CTAs that loop over groups of tokens, a last group that is not whole
    (768, 4, 1, 64, 16, 64, "half", "none", False, 10),
    (771, 70, 1, 128, 16, 96, "interleaved", "none", True, 50_000),    # heads in two parts
    (3001, 16, 8, 128, 16, 64, "interleaved", "yarn", True, 2_000_000),
    (10007, 3, 1, 64, 32, 48, "half", "banded", True, 100_000),
    (20010, 1, 2, 64, 16, 64, "half", "linear", False, 2**31 - 1),
]


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("case", LONG_CASES)
def test_prompts_match_the_formula(case, fp8):
    test_matches_the_formula(*case, fp8)


@pytest.mark.gpu
def test_prompts_in_place_with_padding_and_bad_slots():
    q, k, v, pos, slots, nb = inputs(9001, 6, 2, 64, 16, True, 8, 9000)
    slots[::7] = -1
    rope = pa.pa_rope_init(64, 10000.0)
    pools = [torch.zeros(nb, 16, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    out = torch.empty(9001, 6, 64, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.pa_rope_write(out, q, k, v, pos.cuda(), slots.cuda(), pools[0], pools[1], rope, status=status)
    assert status.item() == 0
    slots[::7] = nb * 16      # past the pools: reported, not written
    pa.pa_rope_write(q, q, k, v, pos.cuda(), slots.cuda(), pools[2], pools[3], rope, status=status)
    assert status.item() == pa.PA_STATUS_BAD_SLOT
    assert torch.equal(q, out) and torch.equal(pools[0], pools[2]) and torch.equal(pools[1], pools[3])


@pytest.mark.gpu
def test_in_place_and_on_another_stream():
    q, k, v, pos, slots, nb = inputs(19, 8, 2, 128, 16, True, 5, 9000)
    rope = pa.pa_rope_init(128, 10000.0)
    pools = [torch.zeros(nb, 16, 2, 128, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    out = torch.empty(19, 8, 128, dtype=torch.bfloat16, device="cuda")
    pos, slots = pos.cuda(), slots.cuda()
    pa.pa_rope_write(out, q, k, v, pos, slots, pools[0], pools[1], rope)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    pa.pa_rope_write(q, q, k, v, pos, slots, pools[2], pools[3], rope, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(q, out) and torch.equal(pools[0], pools[2]) and torch.equal(pools[1], pools[3])


@pytest.mark.gpu
def test_bad_slot_is_reported_and_skipped():
    q, k, v, pos, slots, nb = inputs(4, 4, 2, 64, 16, False, 6, 100)
    slots[2] = nb * 16
    kc, vc = (torch.zeros(nb, 16, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    pa.pa_rope_write(out, q, k, v, pos.cuda(), slots.cuda(), kc, vc, pa.pa_rope_init(64, 1e4), status=status)
    assert status.item() == pa.PA_STATUS_BAD_SLOT
    assert int((kc.flatten(0, 1).abs().sum((1, 2)) > 0).sum()) == 3


@pytest.mark.gpu
def test_wrapper_refuses_what_does_not_fit():
    q, k, v, pos, slots, nb = inputs(4, 4, 2, 64, 16, False, 6, 100)
    kc, vc = (torch.zeros(nb, 16, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pos, slots, rope = pos.cuda(), slots.cuda(), pa.pa_rope_init(64, 1e4)
    with pytest.raises(ValueError):
        pa.pa_rope_write(q, q, k[:3], v[:3], pos, slots, kc, vc, rope)
    with pytest.raises(ValueError):
        pa.pa_rope_write(q, q, k.transpose(0, 1), v.transpose(0, 1), pos, slots, kc, vc, rope)
    with pytest.raises(TypeError):
        pa.pa_rope_write(q.float(), q, k, v, pos, slots, kc, vc, rope)
    with pytest.raises(TypeError):
        pa.pa_rope_write(q, q, k, v, pos.long(), slots, kc, vc, rope)
    with pytest.raises(TypeError):
        pa.pa_rope_write(q, q, k, v, pos, slots, kc, vc, {"rot_dim": 64})


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [1.0, 0.03, 1.0 / 448, 3.3e-5, 7.7, 1e-37, 3e38, 0.02340001])
def test_fp8_codes_equal_the_cache_write(scale):
    """Every bf16 value: the values' codes, and the keys' where nothing turns (position 0), are
    pa_cache_write_fp8's, byte for byte."""
    every = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).view(128, 4, 128).cuda()
    finite = torch.where(torch.isfinite(every), every, torch.ones_like(every))
    slots = torch.randperm(128, generator=torch.Generator().manual_seed(1)).cuda()
    pools = [torch.zeros(8, 16, 4, 128, dtype=torch.uint8, device="cuda") for _ in range(4)]
    pa.pa_cache_write_fp8(finite, every, slots, pools[0], pools[1], scale, scale)
    q = torch.zeros(128, 4, 128, dtype=torch.bfloat16, device="cuda")
    pa.pa_rope_write_fp8(q, q, finite, every, torch.zeros(128, dtype=torch.int32, device="cuda"), slots, pools[2],
                         pools[3], scale, scale, pa.pa_rope_init(128, 1e4))
    torch.cuda.synchronize()
    assert torch.equal(pools[1], pools[3])
    # (a turned -0 may come out as +0)
    assert torch.equal(torch.where(pools[0] == 0x80, 0, pools[0]), torch.where(pools[2] == 0x80, 0, pools[2]))
