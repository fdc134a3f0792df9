"""Attention over blocks of every KV head's own (pa_decode_selected, pa_decode_selected_fp8) against a plain one in 64 bits.

Tolerances, from the roundings on the way, for scores |s| < 40 in log2 units: a score's fp32 sum and product are off by
less than 2^-14 in all, p = 2^(s - m) is held to 2^-17 (tensor cores: a hi + lo pair; CUDA cores: fp32), so a weight is
off by less than 2^-13 of itself, the output by 2^-12 max |v| (numerator and denominator), then rounded to bf16: 2^-8 of
the value, half a step at most 2^-9 more than that covers.  lse: 2^-13 + 2^-23 of itself.
"""
import ctypes
import math
import random

import pytest
import torch

from paged_kv_decode_cache_gb300 import build as B
from paged_kv_decode_cache_gb300 import pa
from paged_model import as64, attention64, encode, i32, rows_of


@pytest.fixture(scope="module", autouse=True)
def _built():
    B.build()


def lists(lens, nb, bs, seed, width):
    """A list of blocks for every (sequence, head) with lens[b][h] tokens, of blocks that other lists may name too."""
    rng = random.Random(seed)
    out = []
    for row in lens:
        out.append([])
        for n in row:
            ids = rng.sample(range(nb), -(-n // bs))
            out[-1].append(ids + [-1] * (width - len(ids)))
    return out


def case(hq, hkv, d, bs, lens, splits, fp8=False, seed=1, extra=0, stream=None, status=None):
    Bn = len(lens)
    width = max(1, max(-(-n // bs) for row in lens for n in row)) + extra
    nb = width + 5
    g = torch.Generator().manual_seed(seed)
    q = (torch.randn(Bn, hq, d, generator=g) * 3).to(torch.bfloat16)
    pools = [encode(torch.randn(nb, bs, hkv, d, generator=g), fp8) for _ in range(2)]
    sel = lists(lens, nb, bs, seed, width)
    ks, vs = (0.5, 0.75) if fp8 else (1.0, 1.0)
    scale = d ** -0.5
    used = torch.zeros(nb * bs, hkv, dtype=torch.bool)
    out, lse = torch.zeros(Bn, hq, d, dtype=torch.float64), torch.full((Bn, hq), -math.inf, dtype=torch.float64)
    G = hq // hkv
    for b in range(Bn):
        for h in range(hkv):
            at = rows_of(sel[b][h], lens[b][h], bs)
            used[at, h] = True
            k, v = (as64(p.flatten(0, 1)[at, h]) for p in pools)
            hs = slice(h * G, h * G + G)
            out[b, hs], lse[b, hs] = attention64(as64(q[b, hs]), k * ks, v * vs, scale)
    for p in pools:   # what no list names is never looked at
        p.view(nb * bs, hkv, d)[~used] = 0x7F if fp8 else math.nan
    P = splits or pa.pa_selected_num_splits(Bn, hq, hkv, d, width, bs)
    ws = torch.zeros(max(1, pa.pa_splitkv_workspace_bytes(Bn, hq, d, P)), dtype=torch.uint8, device="cuda")
    got, z = torch.full((Bn, hq, d), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((Bn, hq), 7.0, device="cuda")
    pools = [p.cuda() for p in pools]
    args = (i32(sel), i32(lens), scale)
    torch.cuda.synchronize()
    if fp8:
        pa.pa_decode_selected_fp8(got, z, q.cuda(), *pools, ks, vs, *args, num_splits=splits, workspace=ws, status=status,
                                  stream=stream)
    else:
        pa.pa_decode_selected(got, z, q.cuda(), *pools, *args, num_splits=splits, workspace=ws, status=status, stream=stream)
    torch.cuda.synchronize()
    got, z = got.double().cpu(), z.double().cpu()
    none = torch.isinf(lse)
    assert torch.equal(torch.isinf(z), none) and (got[none] == 0).all()
    assert ((z - lse)[~none].abs() <= 2.0 ** -13 + 2.0 ** -23 * lse[~none].abs()).all()
    assert ((got - out).abs() <= 2.0 ** -12 * 6 * vs + 2.0 ** -8 * out.abs()).all()


def ragged(Bn, hkv, most, seed):
    rng = random.Random(seed)
    return [[rng.choice([0, 1, 15, 16, 17, most, rng.randint(1, most)]) for _ in range(hkv)] for _ in range(Bn)]


@pytest.mark.gpu
@pytest.mark.parametrize("splits", [0, 1, 2, 7])
@pytest.mark.parametrize("hq,hkv,d,bs,most,fp8", [
    (28, 4, 128, 16, 700, False), (28, 4, 128, 16, 700, True), (16, 8, 128, 32, 300, True), (32, 1, 128, 256, 1000, False),
    (32, 1, 128, 16, 130, True), (5, 5, 128, 48, 200, False), (12, 3, 64, 16, 500, False), (8, 1, 64, 256, 600, False),
    (2, 2, 64, 32, 90, False), (34, 2, 128, 16, 400, False),
])
def test_selected(hq, hkv, d, bs, most, fp8, splits):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for Bn in (1, 3):
        case(hq, hkv, d, bs, ragged(Bn, hkv, most, Bn + splits), splits, fp8, seed=Bn, extra=Bn - 1, status=status)
    assert status.item() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True])
def test_selected_in_many_rows(fp8):
    """More rows than SMs (waves, merged by a kernel of their own) and than the merge has counters."""
    case(16, 8, 128, 16, ragged(40, 8, 900, 3), 0, fp8, seed=3)
    case(16, 8, 128, 16, ragged(140, 8, 60, 4), 2, fp8, seed=4)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_selected_without_tokens_and_on_another_stream(d):
    side = torch.cuda.Stream()
    for splits in (1, 3):
        case(8, 2, d, 16, [[0, 0]], splits, stream=side)
        case(8, 2, d, 16, [[0, 50], [33, 0]], splits, stream=side, extra=4)


@pytest.mark.gpu
def test_selected_is_plain_decode_where_every_head_reads_everything():
    """The same blocks for every head: what pa_decode_splitkv gives, to bf16's rounding."""
    g = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)   # noqa: E731
    q, k, v = rnd(2, 28, 128), rnd(40, 16, 4, 128), rnd(40, 16, 4, 128)
    t, n = torch.randperm(40, generator=torch.Generator().manual_seed(2))[:36].int().view(2, 18).cuda(), i32([288, 201])
    a, b, za, zb = torch.empty_like(q), torch.empty_like(q), torch.empty(2, 28, device="cuda"), torch.empty(2, 28, device="cuda")
    ws = torch.zeros(1 << 22, dtype=torch.uint8, device="cuda")
    pa.pa_decode_splitkv(a, za, q, k, v, t, n, 0.1, num_splits=3, workspace=ws)
    pa.pa_decode_selected(b, zb, q, k, v, t[:, None].expand(2, 4, 18).contiguous(), n[:, None].expand(2, 4).contiguous(), 0.1,
                          num_splits=3, workspace=ws)
    assert ((a.double() - b.double()).abs() <= 2.0 ** -7 * a.double().abs() + 2.0 ** -11).all()
    assert ((za - zb).abs() <= 2.0 ** -12).all()


@pytest.mark.gpu
def test_selected_takes_the_splits_that_its_workspace_holds():
    """num_splits = 0 with less workspace than the rule's count needs, or none."""
    g = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)   # noqa: E731
    q, k, v = rnd(1, 8, 128), rnd(80, 16, 2, 128), rnd(80, 16, 2, 128)
    t, n = torch.arange(80, device="cuda").int().expand(1, 2, 80).contiguous(), i32([[1280, 1111]])
    P = pa.pa_selected_num_splits(1, 8, 2, 128, 80, 16)
    assert P > 4
    outs = []
    for size in (pa.pa_splitkv_workspace_bytes(1, 8, 128, P), pa.pa_splitkv_workspace_bytes(1, 8, 128, 3), 4096, 0):
        ws = torch.zeros(size, dtype=torch.uint8, device="cuda") if size else None
        outs.append(torch.empty_like(q))
        pa.pa_decode_selected(outs[-1], None, q, k, v, t, n, 0.1, workspace=ws)
    for x in outs[1:]:
        assert ((x.double() - outs[0].double()).abs() <= 2.0 ** -7 * outs[0].double().abs() + 2.0 ** -11).all()


@pytest.mark.gpu
def test_selected_reports_bad_blocks_and_lengths():
    g = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)   # noqa: E731
    for d in (64, 128):
        q, k, v = rnd(1, 4, d), rnd(6, 16, 2, d), rnd(6, 16, 2, d)
        out = torch.empty_like(q)
        for sel, n, bit in (([[[0, 6], [1, 2]]], [[32, 20]], pa.PA_STATUS_BAD_BLOCK),
                            ([[[0, 1], [-1, 2]]], [[32, 20]], pa.PA_STATUS_BAD_BLOCK),
                            ([[[0, 1], [1, 2]]], [[33, 20]], pa.PA_STATUS_BAD_SEQLEN),
                            ([[[0, 1], [1, 2]]], [[3, -1]], pa.PA_STATUS_BAD_SEQLEN)):
            status = torch.zeros(1, dtype=torch.int32, device="cuda")
            pa.pa_decode_selected(out, None, q, k, v, i32(sel), i32(n), 0.1, num_splits=1, status=status)
            assert status.item() == bit


@pytest.mark.gpu
@pytest.mark.parametrize("splits", [1, 3])
def test_selected_on_cuda_cores_with_the_grid_merge_and_plain_launches(use_kernel, merge_path, splits):
    """The kernels and launches that the switches choose."""
    use_kernel("cuda_core")
    case(8, 2, 128, 16, ragged(3, 2, 500, 5), splits)
    use_kernel("auto")
    merge_path("grid")
    for d, fp8 in ((128, False), (128, True), (64, False)):
        case(8, 2, d, 16, ragged(3, 2, 500, 6), splits, fp8)
    prev = pa.pa_get_option(pa.PA_OPT_PDL)
    pa.pa_set_option(pa.PA_OPT_PDL, 0)
    try:
        case(8, 2, 128, 16, ragged(3, 2, 500, 7), splits)
    finally:
        pa.pa_set_option(pa.PA_OPT_PDL, prev)


FAKE = ctypes.c_void_p(1 << 20)  # aligned, never dereferenced: these calls fail validation first


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), pa.PA_EINVAL), (dict(B=-1), pa.PA_EINVAL), (dict(K=0), pa.PA_EINVAL), (dict(Hq=5), pa.PA_EINVAL),
    (dict(Hq=0), pa.PA_EINVAL), (dict(splits=-1), pa.PA_EINVAL), (dict(splits=3), pa.PA_EWORKSPACE),
    (dict(scale=math.inf), pa.PA_EINVAL), (dict(out=None), pa.PA_EINVAL), (dict(Hq=66), pa.PA_EUNSUPPORTED),
    (dict(B=70000), pa.PA_EUNSUPPORTED), (dict(desc=pa.CacheDesc(64, 16, 2, 96)), pa.PA_EUNSUPPORTED),
    (dict(desc=pa.CacheDesc(64, 16, 0, 128)), pa.PA_EINVAL), (dict(B=0), pa.PA_OK),
])
def test_selected_refusals(kw, code):
    a = dict(out=FAKE, q=FAKE, desc=pa.CacheDesc(64, 16, 2, 128), K=7, B=4, Hq=4, scale=0.1, splits=1) | kw
    tail = (FAKE, a["K"], FAKE, a["B"], a["Hq"], a["scale"], a["splits"], None, 0, None, None)
    assert pa.lib().pa_decode_selected(a["out"], None, a["q"], FAKE, FAKE, a["desc"], *tail) == code
    assert pa.lib().pa_decode_selected_fp8(a["out"], None, a["q"], FAKE, FAKE, a["desc"], 1.0, 1.0, *tail) == code
    for ks, vs in ((0.0, 1.0), (1.0, math.nan)):
        assert pa.lib().pa_decode_selected_fp8(a["out"], None, a["q"], FAKE, FAKE, a["desc"], ks, vs, *tail) == pa.PA_EINVAL


def test_selected_refuses_what_its_kernels_do_not_take():
    d64 = pa.CacheDesc(64, 16, 2, 64)
    tail = (FAKE, 7, FAKE, 4, 18, 0.1, 1, None, 0, None, None)
    assert pa.lib().pa_decode_selected(FAKE, None, FAKE, FAKE, FAKE, d64, *tail) == pa.PA_EUNSUPPORTED   # 9 heads of 64
    assert pa.lib().pa_decode_selected_fp8(FAKE, None, FAKE, FAKE, FAKE, d64, 1.0, 1.0, *tail) == pa.PA_EUNSUPPORTED


def test_selected_split_counts():
    for tiles in (1, 3, 64, 128, 1000):
        for Bn in (1, 4, 64, 1000):
            for heads in ((28, 4), (16, 8), (12, 2)):
                P = pa.pa_selected_num_splits(Bn, *heads, 128, tiles, 16, sm_count=152)
                assert 1 <= P <= min(64, tiles)
    assert pa.pa_selected_num_splits(64, 16, 8, 128, 128, 16, sm_count=152) == 2
    assert pa.pa_selected_num_splits(1, 12, 2, 128, 64, 16, sm_count=152) == 16
    assert pa.pa_selected_num_splits(8, 8, 2, 64, 64, 16, sm_count=152) == pa.pa_choose_num_splits(8, 8, 2, 64, 64, 16, 152)
    for a in ((8, 28, 4, 128, 0, 16, 152), (8, 28, 4, 128, 8, 15, 152), (8, 27, 4, 128, 8, 16, 152), (8, 28, 4, 128, 8, 16, -1)):
        with pytest.raises(pa.PAError) as e:
            pa.pa_selected_num_splits(*a[:6], sm_count=a[6])
        assert e.value.code == pa.PA_EINVAL


@pytest.mark.gpu
def test_selected_wrapper_refuses():
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")   # noqa: E731
    ok = dict(out=z(1, 4, 64), lse=None, q=z(1, 4, 64), k=z(4, 16, 2, 64), v=z(4, 16, 2, 64), t=i32([[[0], [1]]]), n=i32([[3, 4]]))
    for kw in (dict(t=i32([[0, 1]])), dict(n=i32([3])), dict(out=z(1, 4, 128)), dict(lse=torch.zeros(4, device="cuda")),
               dict(v=z(4, 16, 1, 64)), dict(q=z(1, 4, 64).float()), dict(k=ok["k"].to(torch.uint8))):
        a = ok | kw
        with pytest.raises((TypeError, ValueError)):
            pa.pa_decode_selected(a["out"], a["lse"], a["q"], a["k"], a["v"], a["t"], a["n"], 0.1, num_splits=1)
