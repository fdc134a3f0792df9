"""Bounds of the keys (pa_key_bounds) and the blocks they choose (pa_blocks_select) against plain models in 64 bits.
Bounds are some of the keys and choices are whole numbers: equality throughout."""
import ctypes
import math
import random

import pytest
import torch

from paged_kv_decode_cache_gb300 import build as B
from paged_kv_decode_cache_gb300 import pa
from paged_model import FP8, as64, encode, i32, layout, scores64, unused_rows


@pytest.fixture(scope="module", autouse=True)
def _built():
    B.build()


# ---- bounds -------------------------------------------------------------------------------------


def pool(nb, bs, hkv, d, fp8, seed, tables=None, lens=None):
    """A pool on the CPU; places of no token hold NaN."""
    g = torch.Generator().manual_seed(seed)
    k = encode(torch.randn(nb, bs, hkv, d, generator=g) * 2, fp8)
    if tables is not None:
        k.flatten(0, 1)[unused_rows(tables, lens, nb, bs)] = 0x7F if fp8 else math.nan
    return k


def same_values(a, b):
    a, b = as64(a), as64(b)
    return torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(torch.nan_to_num(a), torch.nan_to_num(b))


def plain_bounds(bounds, k, tables, lens, starts, bs, max_new=None):
    out, vals = bounds.clone(), as64(k)
    for row, n, s in zip(tables, lens, starts):
        s = max(s, n - max_new) if max_new else s
        for j in range(s // bs, -(-n // bs)):
            if j * bs < n and (j + 1) * bs > s and s < n:
                x = vals[row[j], :min(bs, n - j * bs)]
                lo, hi = x.amin(0), x.amax(0)   # (a NaN makes both one)
                out[row[j], :, 0], out[row[j], :, 1] = (encode(y.float(), out.dtype == torch.uint8) for y in (lo, hi))
    return out


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("hkv,d,bs,lens,starts,max_new", [
    (4, 128, 16, [1, 16, 17, 0, 100], None, None),
    (4, 128, 16, [1, 16, 17, 0, 100], [0, 15, 16, 0, 99], 1),
    (1, 64, 16, [33, 5], [32, 0], 5),
    (3, 64, 32, [31, 32, 33, 129], [0, 0, 31, 40], None),
    (8, 128, 256, [255, 257, 700], [254, 200, 511], 300),
    (2, 128, 48, [47, 48, 49, 200], None, 200),
    (40, 128, 16, [20, 40], None, None),       # more chunks of a token than threads
    (5, 64, 256, [256, 1], None, None),
])
def test_bounds(hkv, d, bs, lens, starts, max_new, fp8):
    tables, _, nb = layout(lens, bs, seed=len(lens))
    k = pool(nb, bs, hkv, d, fp8, 3, tables, lens)
    before = pool(nb, hkv, 2, d, fp8, 4)
    got, status = before.cuda(), torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.pa_key_bounds(got, k.cuda(), i32(tables), i32(lens), starts=None if starts is None else i32(starts), max_new=max_new,
                     status=status)
    want = plain_bounds(before, k, tables, lens, starts or [0] * len(lens), bs)
    assert status.item() == 0 and same_values(got, want)


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("hkv,d,bs,mb", [(4, 128, 16, 520), (1, 64, 16, 600), (3, 64, 48, 500)])
def test_bounds_of_many_blocks(hkv, d, bs, mb, fp8):
    """Tables that would hold enough blocks for the kernel of whole prompts."""
    rng = random.Random(mb)
    lens = [0, 1, bs, bs + 1] + [rng.randint(1, 12 * bs) for _ in range(36)]
    starts = [rng.randint(0, n) if rng.random() < 0.5 else 0 for n in lens]
    tables, _, nb = layout(lens, bs, seed=mb, extra=mb)
    k = pool(nb, bs, hkv, d, fp8, 5, tables, lens)
    before = pool(nb, hkv, 2, d, fp8, 6)
    got, status = before.cuda(), torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.pa_key_bounds(got, k.cuda(), i32(tables), i32(lens), starts=i32(starts), status=status)
    assert status.item() == 0 and same_values(got, plain_bounds(before, k, tables, lens, starts, bs))
    tables[7][0], tables[9][0] = nb, -1
    got = before.cuda()
    pa.pa_key_bounds(got, k.cuda(), i32(tables), i32(lens), status=status)
    good = [t if i not in (7, 9) else [tables[0][0] if x < 0 or x >= nb else x for x in t] for i, t in enumerate(tables)]
    want = plain_bounds(before, k, [t for i, t in enumerate(good) if i not in (7, 9)],
                        [n for i, n in enumerate(lens) if i not in (7, 9)], [0] * len(lens), bs)
    for i in (7, 9):
        want = plain_bounds(want, k, [good[i]], [lens[i]], [bs], bs)
    assert status.item() == pa.PA_STATUS_BAD_BLOCK and same_values(got, want)


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True])
def test_bounds_of_nan_infinity_and_zeros(fp8):
    k = encode(torch.zeros(3, 16, 2, 64), fp8)
    if fp8:
        k[0, 5, 0, 7], k[1, 0, 1, 3] = 0xFF, 0x80         # a NaN, a -0
        k[2] = torch.randint(0, 256, (16, 2, 64), generator=torch.Generator().manual_seed(1)).to(torch.uint8)
    else:
        k[0, 5, 0, 7], k[1, 0, 1, 3], k[1, 2, 0, 9], k[2, 0, 0, 0] = math.nan, -0.0, math.inf, -math.inf
        k[2, :, 1] = 1e-40                                 # (below bf16's normal range)
    got = torch.zeros(3, 2, 2, 64, dtype=k.dtype, device="cuda")
    pa.pa_key_bounds(got, k.cuda(), i32([[0, 1, 2]]), i32([48]))
    assert same_values(got, plain_bounds(got.cpu(), k, [[0, 1, 2]], [48], [0], 16))


@pytest.mark.gpu
def test_bounds_report_what_they_skip():
    k, b = torch.randn(4, 16, 1, 64).to(torch.bfloat16), torch.zeros(4, 1, 2, 64, dtype=torch.bfloat16, device="cuda")
    for tables, lens, starts, max_new, bit in (([[9, 1]], [32], [0], None, pa.PA_STATUS_BAD_BLOCK),
                                               ([[-1, 1]], [32], [0], None, pa.PA_STATUS_BAD_BLOCK),
                                               ([[0, 1]], [40], [0], None, pa.PA_STATUS_BAD_SEQLEN),
                                               ([[0, 1]], [-1], [0], None, pa.PA_STATUS_BAD_SEQLEN),
                                               ([[0, 1]], [20], [-3], None, pa.PA_STATUS_BAD_SEQLEN),
                                               ([[0, 1]], [32], [0], 7, pa.PA_STATUS_BAD_SEQLEN)):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = b.clone()
        pa.pa_key_bounds(got, k.cuda(), i32(tables), i32(lens), starts=i32(starts), max_new=max_new, status=status)
        assert status.item() == bit
        n = min(max(lens[0], 0), 32)
        if bit == pa.PA_STATUS_BAD_BLOCK:
            want = b.cpu().clone()
            want[1] = plain_bounds(b.cpu(), k, [[1, 1]], [32], [0], 16)[1]
        else:
            want = plain_bounds(b.cpu(), k, tables, [n], [max(0, starts[0])], 16, max_new)
        assert same_values(got, want)


# ---- selection ----------------------------------------------------------------------------------


def plain_select(q, bounds, tables, lens, bs, K, first, last):
    Bn, hq, d = q.shape
    hkv = bounds.shape[1]
    q, bounds = as64(q).view(Bn, hkv, -1, d), as64(bounds)
    out, tokens = torch.full((Bn, hkv, K), -1, dtype=torch.int32), torch.zeros(Bn, hkv, dtype=torch.int32)
    for b in range(Bn):
        n = -(-lens[b] // bs)
        ids = torch.tensor(tables[b][:n], dtype=torch.long)
        ok = (ids >= 0) & (ids < len(bounds))
        for h in range(hkv):
            x = bounds[ids.clamp(0, len(bounds) - 1), h]
            s = torch.where(ok, scores64(q[b, h], x[:, 0], x[:, 1]), -math.inf).tolist()
            forced = [j < first or j >= n - last for j in range(n)]
            took = sorted(sorted(range(n), key=lambda j: (not forced[j], -s[j], j))[:K])
            out[b, h, :len(took)] = torch.tensor([tables[b][j] for j in took], dtype=torch.int32)
            tokens[b, h] = sum(min(bs, lens[b] - j * bs) for j in took)
    return out, tokens


def select(q, bounds, tables, lens, bs, K, first, last, status=None, stream=None):
    hkv = bounds.shape[1]
    out = torch.full((len(lens), hkv, K), 77, dtype=torch.int32, device="cuda")
    tokens = torch.full((len(lens), hkv), 77, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    pa.pa_blocks_select(out, tokens, q.cuda(), bounds.cuda(), bs, i32(tables), i32(lens), first=first, last=last, status=status,
                        stream=stream)
    torch.cuda.synchronize()
    return out.cpu(), tokens.cpu()


def make_bounds(nb, hkv, d, fp8, seed, mean=1.0):
    g = torch.Generator().manual_seed(seed)
    mid = torch.randn(nb, hkv, d, generator=g) * 0.5 + mean * torch.randn(hkv, d, generator=g)
    wide = (torch.randn(nb, hkv, d, generator=g) * 0.3 + 1.7).abs()
    return encode(torch.stack((mid - wide, mid + wide), 2), fp8)


def queries(Bn, hq, d, seed):
    return (torch.randn(Bn, hq, d, generator=torch.Generator().manual_seed(seed)) * 1.5).to(torch.bfloat16)


def check(q, bounds, tables, lens, bs, K, first, last):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = select(q, bounds, tables, lens, bs, K, first, last, status)
    want = plain_select(q, bounds, tables, lens, bs, K, first, last)
    assert status.item() == 0
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("hq,hkv,d,bs,lens,K,first,last", [
    (7, 1, 128, 16, [1, 15, 16, 17, 0, 320], 4, 1, 1),
    (28, 4, 128, 16, [1000, 4097], 33, 1, 4),
    (16, 8, 64, 16, [511, 512, 513, 2000], 8, 0, 1),
    (12, 3, 64, 32, [5000], 16, 4, 8),
    (32, 1, 128, 256, [9000, 300], 5, 2, 2),
    (9, 1, 128, 16, [4000], 249, 0, 1),          # all but one
    (17, 1, 64, 16, [4000], 3, 1, 2),            # none but the forced
    (2, 2, 128, 48, [48 * 40 + 1, 47], 40, 0, 40),
    (6, 2, 128, 16, [16389], 64, 1, 2),
    (4, 4, 64, 16, [40000], 300, 4, 8),
])
def test_select(hq, hkv, d, bs, lens, K, first, last, fp8):
    tables, _, nb = layout(lens, bs, seed=K)
    check(queries(len(lens), hq, d, K), make_bounds(nb, hkv, d, fp8, K + 1), tables, lens, bs, K, first, last)


@pytest.mark.gpu
@pytest.mark.parametrize("Bn,hkv,fp8", [(300, 1, False), (259, 2, True), (40, 8, False)])
def test_select_in_many_rows(Bn, hkv, fp8):
    """More clusters than run at once: sequences are taken by length, some of them equal."""
    rng = random.Random(Bn)
    lens = [rng.choice([0, 16, 200, 200, 333, rng.randint(1, 700)]) for _ in range(Bn)]
    tables, _, nb = layout(lens, 16, seed=Bn)
    check(queries(Bn, 2 * hkv, 64, Bn), make_bounds(nb, hkv, 64, fp8, Bn + 1), tables, lens, 16, 6, 1, 1)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [40960 * 16, 40960 * 16 - 33, 16 * 16 + 1])
def test_select_of_the_most_blocks(n):
    tables, _, nb = layout([40960 * 16], 16, seed=5)
    check(queries(1, 32, 64, 5), make_bounds(nb, 1, 64, True, 6), tables, [n], 16, 500, 2, 3)


@pytest.mark.gpu
@pytest.mark.parametrize("seed", range(6))
def test_select_scores_that_fp32_does_not_tell_apart(seed):
    """Hundreds of blocks that differ in one small channel by one step: sums in 64 bits tell them apart, sums in fp32
    do not.  Some are wholly alike: the earlier one wins."""
    rng = random.Random(seed)
    n, d, K = 400, 128, 50 + 37 * seed
    g = torch.Generator().manual_seed(seed)
    one = torch.randn(2, d, generator=g).sort(0).values.mul(4).to(torch.bfloat16)
    bounds = one.expand(n, 1, 2, d).clone()
    q = (torch.randn(1, 3, d, generator=g) * 8).to(torch.bfloat16)
    small = rng.randrange(d)
    q[0, :, small] = 2.0 ** -14                                   # products near 2^-23 of the sum
    bounds[:, 0, :, small] = torch.tensor([rng.choice([0.5, 0.50390625, 0.5078125]) for _ in range(n)],
                                          dtype=torch.bfloat16)[:, None]
    tables, _, _ = layout([n * 16], 16, seed=seed, spare=0)
    check(q, bounds, tables, [n * 16], 16, K, 0, 1)


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True])
def test_select_equal_scores(fp8):
    """Zeros (a cache of a warm-up run), one score for all, and queries of zeros: the first blocks."""
    lens, K = [16 * 1500, 16 * 77, 5], 40
    tables, _, nb = layout(lens, 16, seed=1)
    same = encode(torch.full((nb, 2, 2, 64), 1.5), fp8)
    for q, bounds in ((queries(3, 4, 64, 1), encode(torch.zeros(nb, 2, 2, 64), fp8)), (queries(3, 4, 64, 2), same),
                      (torch.zeros(3, 4, 64, dtype=torch.bfloat16), make_bounds(nb, 2, 64, fp8, 3))):
        check(q, bounds, tables, lens, 16, K, 1, 1)


@pytest.mark.gpu
def test_select_extremes():
    """Products and sums past fp32's range, or below it, of finite values: the 64-bit order."""
    lens, K, d = [16 * 200], 30, 64
    tables, _, nb = layout(lens, 16, seed=2)
    for qs, bs_ in ((1e20, 1e25), (3e38, 1.0), (3e38, 3e38), (1e-25, 1e-25), (1e-20, 1e-15), (1e38, 1e-38)):
        g = torch.Generator().manual_seed(7)
        q = (torch.rand(1, 4, d, generator=g) * 2 - 1).mul(qs).to(torch.bfloat16)
        b = (torch.rand(nb, 1, 2, d, generator=g).double() * 2 - 1).mul(bs_).to(torch.bfloat16).sort(2).values
        check(q, b, tables, lens, 16, K, 1, 1)


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True])
def test_select_infinities_and_nans(fp8):
    lens, K, d = [16 * 120, 16 * 50], 20, 128
    tables, _, nb = layout(lens, 16, seed=3)
    bounds, q = make_bounds(nb, 2, d, fp8, 5), queries(2, 6, d, 5)
    bad = 0x7F if fp8 else math.nan
    for j in (7, 30, 99):
        bounds[tables[0][j], 0, j % 2, j] = bad
    if not fp8:
        bounds[tables[0][50], 1, 0, 3], bounds[tables[0][51], 1, 1, 3] = -math.inf, math.inf
        bounds[tables[1][2:45], 0, 1, 0] = math.inf      # more than can be taken
    check(q, bounds, tables, lens, 16, K, 2, 2)
    q[1, 4, 9] = math.nan                                 # KV head 1 of sequence 1
    q[0, 0, 0] = math.inf
    check(q, bounds, tables, lens, 16, K, 2, 2)


@pytest.mark.gpu
def test_select_reports_bad_blocks_and_lengths():
    lens, d = [16 * 60, 16 * 60], 64
    tables, _, nb = layout(lens, 16, seed=4)
    tables[0][5], tables[0][30], tables[0][0], tables[1][59] = -1, nb, -7, 1 << 30
    q, bounds = queries(2, 4, d, 6), make_bounds(nb, 2, d, False, 6)
    for K in (10, 58, 60, 64):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = select(q, bounds, tables, lens, 16, K, 1, 1, status)
        want = plain_select(q, bounds, tables, lens, 16, K, 1, 1)
        assert status.item() == pa.PA_STATUS_BAD_BLOCK
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    tables, _, nb = layout(lens, 16, seed=4)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = select(q, bounds, tables, [16 * 60 + 1, -2], 16, 10, 1, 1, status)
    want = plain_select(q, bounds, tables, [16 * 60, 0], 16, 10, 1, 1)
    assert status.item() == pa.PA_STATUS_BAD_SEQLEN
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.gpu
def test_select_in_a_graph_and_on_another_stream():
    lens, d = [16 * 300, 700], 128
    tables, _, nb = layout(lens, 16, seed=5)
    q, bounds = queries(2, 8, d, 8).cuda(), make_bounds(nb, 2, d, False, 8).cuda()
    t, n = i32(tables), i32(lens)
    out, tokens = torch.zeros(2, 2, 24, dtype=torch.int32, device="cuda"), torch.zeros(2, 2, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    pa.pa_blocks_select(out, tokens, q, bounds, 16, t, n, stream=side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.pa_blocks_select(out, tokens, q, bounds, 16, t, n)
        pa.pa_blocks_select(out, tokens, q, bounds, 16, t, n)
    for lens in ([16 * 300, 700], [1000, 16 * 20 + 3]):
        n.copy_(i32(lens))
        q.copy_(queries(2, 8, d, lens[0]))
        graph.replay()
        torch.cuda.synchronize()
        want = plain_select(q.cpu(), bounds.cpu(), tables, lens, 16, 24, 1, 1)
        assert torch.equal(out.cpu(), want[0]) and torch.equal(tokens.cpu(), want[1])


# ---- refusals -----------------------------------------------------------------------------------

FAKE = ctypes.c_void_p(1 << 20)  # aligned, never dereferenced: these calls fail validation first
DESC = pa.CacheDesc(64, 16, 2, 128)


@pytest.mark.parametrize("kw,code", [
    (dict(elem=3), pa.PA_EINVAL), (dict(B=-1), pa.PA_EINVAL), (dict(mb=0), pa.PA_EINVAL), (dict(max_new=-1), pa.PA_EINVAL),
    (dict(bounds=None), pa.PA_EINVAL), (dict(bounds=(1 << 20) + 8), pa.PA_EINVAL), (dict(starts=(1 << 20) + 2), pa.PA_EINVAL),
    (dict(desc=pa.CacheDesc(64, 16, 2, 96)), pa.PA_EUNSUPPORTED), (dict(desc=pa.CacheDesc(64, 8, 2, 64)), pa.PA_EUNSUPPORTED),
    (dict(mb=1 << 27), pa.PA_EUNSUPPORTED), (dict(B=70000), pa.PA_EUNSUPPORTED), (dict(B=0, bounds=None), pa.PA_OK),
])
def test_bounds_refusals(kw, code):
    a = dict(bounds=FAKE, elem=2, desc=DESC, mb=7, starts=None, max_new=0, B=4) | kw
    assert pa.lib().pa_key_bounds(a["bounds"], FAKE, a["elem"], a["desc"], FAKE, a["mb"], FAKE, a["starts"], a["max_new"],
                                  a["B"], None, None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(elem=4), pa.PA_EINVAL), (dict(B=-1), pa.PA_EINVAL), (dict(mb=0), pa.PA_EINVAL), (dict(K=0), pa.PA_EINVAL),
    (dict(first=-1), pa.PA_EINVAL), (dict(last=0), pa.PA_EINVAL), (dict(first=5, last=4), pa.PA_EINVAL),
    (dict(first=2 ** 31 - 1, last=2), pa.PA_EINVAL), (dict(q=None), pa.PA_EINVAL), (dict(q=(1 << 20) + 8), pa.PA_EINVAL),
    (dict(Hq=5), pa.PA_EINVAL), (dict(Hq=66), pa.PA_EUNSUPPORTED), (dict(desc=pa.CacheDesc(64, 16, 2, 96)), pa.PA_EUNSUPPORTED),
    (dict(mb=40961), pa.PA_EUNSUPPORTED), (dict(B=70000), pa.PA_EUNSUPPORTED), (dict(B=0, q=None), pa.PA_OK),
])
def test_select_refusals(kw, code):
    a = dict(K=8, q=FAKE, elem=2, desc=DESC, mb=7, B=4, Hq=4, first=1, last=1) | kw
    assert pa.lib().pa_blocks_select(FAKE, a["K"], FAKE, a["q"], FAKE, a["elem"], a["desc"], FAKE, a["mb"], FAKE, a["B"],
                                     a["Hq"], a["first"], a["last"], None, None) == code


@pytest.mark.gpu
def test_wrappers_refuse():
    k, t, n = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16, device="cuda"), i32([[0, 1]]), i32([20])
    b = torch.zeros(4, 2, 2, 64, dtype=torch.bfloat16, device="cuda")
    for kw in (dict(bounds=b.view(torch.int16)), dict(bounds=b[:3]), dict(n=n.long()), dict(starts=i32([1, 2])),
               dict(max_new=0), dict(k=k.cpu()), dict(k=k[:, ::2])):
        a = dict(bounds=b, k=k, n=n, starts=None, max_new=None) | kw
        with pytest.raises((TypeError, ValueError)):
            pa.pa_key_bounds(a["bounds"], a["k"], t, a["n"], starts=a["starts"], max_new=a["max_new"])
    q, st, sn = torch.zeros(1, 4, 64, dtype=torch.bfloat16, device="cuda"), i32([[[0] * 8] * 2]), i32([[0, 0]])
    for kw in (dict(q=q.float()), dict(st=st[0]), dict(sn=sn[:, :1]), dict(b=b[:, :, :, :32].contiguous()), dict(n=i32([1, 2])),
               dict(st=st.long())):
        a = dict(q=q, st=st, sn=sn, b=b, n=n) | kw
        with pytest.raises((TypeError, ValueError)):
            pa.pa_blocks_select(a["st"], a["sn"], a["q"], a["b"], 16, t, a["n"])
    with pytest.raises(pa.PAError) as e:
        pa.pa_blocks_select(st, sn, q, b, 24, t, n)
    assert e.value.code == pa.PA_EUNSUPPORTED
    with pytest.raises(pa.PAError) as e:
        pa.pa_blocks_select(st, sn, q, b, 16, t, n, first=8)
    assert e.value.code == pa.PA_EINVAL
