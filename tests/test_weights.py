"""Accumulated attention weights (pa_weights_add, pa_weights_add_fp8) against a plain sum in 64 bits.

A term exp(s - lse) is off, relative to itself, by the error of s - lse and that of the exponential: s is an fp32 sum of
exact products on tensor cores (at most 8 MMAs of 16 products, each cutting less than 17 * 2^-23 of the sum of
|products|: below 2^-15 of scale * sum |q k|), the scale's product, the subtraction and lse in log2 units round by 2^-24
of |s| + |lse| each (together 2^-22), the exponential by 2^-22, and the scale itself, rounded to fp32, by 2^-23 of |s|.
Sums of N terms and the old weight: (N + 3) 2^-24 of the total.
"""
import ctypes
import math
import random

import pytest
import torch

from paged_kv_decode_cache_gb300 import build as B
from paged_kv_decode_cache_gb300 import pa
from paged_model import as64, encode, i32, layout, rows_of, unused_rows


@pytest.fixture(scope="module", autouse=True)
def _built():
    B.build()


def case(hq, hkv, d, bs, lens, q_len=1, fp8=False, decay=1.0, ends=None, positions=True, same=False, seed=1, room=None,
         stream=None, sharp=2.0, extra=0):
    Bn, G, scale, ks = len(lens), hq // hkv, d ** -0.5, 0.5 if fp8 else 1.0
    tables, _, nb = layout(lens, bs, seed, extra=extra)
    room = room or len(tables[0]) * bs
    g = torch.Generator().manual_seed(seed)
    q = (torch.randn(Bn, q_len, hq, d, generator=g) * sharp).to(torch.bfloat16)
    k = encode(torch.randn(nb, bs, hkv, d, generator=g), fp8)
    k.flatten(0, 1)[unused_rows(tables, lens, nb, bs)] = 0x7F if fp8 else math.nan
    old = torch.randn(Bn, hkv, room, generator=g).mul(2).exp()
    new = torch.full_like(old, 5.0)
    pos = torch.full((Bn, hkv, room), 9, dtype=torch.int32)
    lse = torch.full((Bn, q_len, hq), -math.inf)
    want = (old if same else new).double()
    tol, want_pos = torch.zeros_like(want), pos.clone()
    for b, n in enumerate(lens):
        keys = as64(k.flatten(0, 1)[rows_of(tables[b], n, bs)]) * ks
        for h in range(hkv):
            total, off, terms = torch.zeros(n, dtype=torch.float64), torch.zeros(n, dtype=torch.float64), 0
            for i in range(q_len):
                see = n - q_len + i + 1
                if see <= 0:
                    continue
                for x in range(h * G, h * G + G):
                    qq = as64(q[b, i, x])
                    s = keys[:see, h] @ qq * scale
                    lse[b, i, x] = torch.logsumexp(s, 0)
                    z = lse[b, i, x].double()
                    p = torch.exp(s - z)
                    total[:see] += p
                    size = keys[:see, h].abs() @ qq.abs() * scale
                    off[:see] += p * (2.0 ** -15 * size + 2.0 ** -22 * (s.abs() + z.abs()) + 2.0 ** -23 * s.abs() + 2.0 ** -22)
                    terms += 1
            past = max(0, n - q_len)
            total[:past] += decay * old[b, h, :past].double()
            want[b, h, :n] = total
            tol[b, h, :n] = off + (terms + 3) * 2.0 ** -24 * total
            first = (ends[b] if ends else n) - n
            want_pos[b, h, past:n] = torch.arange(past, n) + first
    dev = dict(old=old.cuda(), new=new.cuda(), pos=pos.cuda(), status=torch.zeros(1, dtype=torch.int32, device="cuda"))
    if same:
        dev["new"] = dev["old"]
    if q_len == 1 and seed % 2:
        q, lse = q[:, 0].contiguous(), lse[:, 0].contiguous()
    args = (q.cuda(), lse.cuda(), k.cuda()) + ((ks,) if fp8 else ()) + (i32(tables), i32(lens), scale)
    torch.cuda.synchronize()
    (pa.pa_weights_add_fp8 if fp8 else pa.pa_weights_add)(
        dev["new"], dev["old"], dev["pos"] if positions else None, *args, ends=i32(ends) if ends else None, decay=decay,
        status=dev["status"], stream=stream)
    torch.cuda.synchronize()
    assert dev["status"].item() == 0
    got = dev["new"].double().cpu()
    assert ((got - want).abs() <= tol).all(), float(((got - want).abs() - tol).max())
    assert torch.equal(dev["pos"].cpu(), want_pos if positions else pos)


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("hq,hkv,d,bs,lens,q_len", [
    (28, 4, 128, 16, [1, 16, 17, 0, 600], 1), (2, 2, 64, 32, [31, 33, 257], 1), (32, 1, 128, 256, [255, 256, 513], 1),
    (12, 3, 64, 16, [100, 3], 5), (16, 8, 128, 16, [300, 40, 0], 17), (28, 4, 128, 16, [511, 20], 32),
    (33, 3, 128, 48, [90, 700], 12), (8, 1, 64, 16, [1000], 40), (5, 5, 64, 16, [64], 64), (1, 1, 128, 16, [2], 3),
])
def test_weights(hq, hkv, d, bs, lens, q_len, fp8):
    case(hq, hkv, d, bs, lens, q_len, fp8, seed=q_len, extra=q_len % 2)
    case(hq, hkv, d, bs, lens, q_len, fp8, decay=0.75, ends=[n + 11 * b for b, n in enumerate(lens)], same=True, seed=q_len + 1)


@pytest.mark.gpu
@pytest.mark.parametrize("q_len", [1, 200])
def test_weights_of_a_long_ragged_batch(q_len):
    rng = random.Random(q_len)
    lens = [rng.randint(0, 3000 if q_len == 1 else 400) for _ in range(9 if q_len == 1 else 3)]
    case(14, 2, 128, 16, lens, q_len, seed=3, positions=False, decay=0.0, stream=torch.cuda.Stream())


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True])
def test_weights_of_a_whole_prompt(fp8):
    """More queries than tokens in one sequence, chunks of columns that go over many tiles."""
    case(2, 1, 64, 16, [1300, 700], q_len=1000, fp8=fp8, seed=4, ends=[1400, 700])


@pytest.mark.gpu
@pytest.mark.parametrize("sharp", [0.0, 12.0])
def test_weights_of_flat_and_sharp_queries(sharp):
    case(8, 2, 128, 16, [1, 200, 333], 4, sharp=sharp, seed=5)


@pytest.mark.gpu
def test_weights_sum_to_the_queries_and_repeat_bit_for_bit():
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k = (torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16) for s in ((3, 2, 8, 128), (60, 16, 2, 128)))
    v = torch.randn(60, 16, 2, 128, generator=g, device="cuda").to(torch.bfloat16)
    lens = [300, 2, 77]
    tables, _, _ = layout(lens, 16, 1, spare=34)
    t, n = i32(tables), i32(lens)
    out, lse = torch.empty_like(q), torch.empty(3, 2, 8, device="cuda")
    pa.pa_decode_mq(out, lse, q, k, v, t, n, 0.1, num_splits=1)
    w = [torch.zeros(3, 2, t.shape[1] * 16, device="cuda") for _ in range(2)]
    for x in w:
        pa.pa_weights_add(x, x, None, q, lse, k, t, n, 0.1)
    assert torch.equal(w[0], w[1])
    # (2 queries of 4 heads; lse and the weights are each good to 2^-13)
    assert ((w[0].double().sum(-1) - 8).abs() <= 8 * 2.0 ** -12).all()


@pytest.mark.gpu
def test_weights_of_infinite_and_nan_scores_stay_with_their_token():
    g = torch.Generator(device="cuda").manual_seed(2)
    q, k = (torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16) for s in ((1, 1, 3, 64), (4, 16, 1, 64)))
    k[1, 3], k[2, 0, 0, 5], k[2, 1, 0, 5] = math.nan, math.inf, -math.inf
    lse = torch.tensor([[[1.0, -math.inf, 2.0]]], device="cuda")      # (head 1 saw nothing)
    w = torch.ones(1, 1, 64, device="cuda")
    pa.pa_weights_add(w, w, None, q, lse, k, i32([[0, 1, 2, 3]]), i32([60]), 0.125)
    keys = as64(k).reshape(64, 64)[:60]
    s = as64(q[0, 0])[[0, 2]] @ keys.t() * 0.125 - torch.tensor([[1.0], [2.0]]).double()
    want = torch.exp(s).sum(0)
    want[:59] += 1
    got = w[0, 0, :60].double().cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want)) and torch.equal(torch.isinf(got), torch.isinf(want))
    fin = torch.isfinite(want)
    assert ((got - want)[fin].abs() <= 2.0 ** -14 * want[fin]).all() and (w[0, 0, 60:] == 1).all()


@pytest.mark.gpu
def test_weights_report_bad_blocks_and_lengths():
    q = torch.randn(2, 4, 64, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").to(torch.bfloat16)
    k, lse = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(2, 4, device="cuda")
    for tables, lens, room, bit in (([[0, 4], [2, 3]], [32, 20], 32, pa.PA_STATUS_BAD_BLOCK),
                                    ([[0, -1], [2, 3]], [32, 20], 32, pa.PA_STATUS_BAD_BLOCK),
                                    ([[0, 1], [2, 3]], [33, 20], 40, pa.PA_STATUS_BAD_SEQLEN),
                                    ([[0, 1], [2, 3]], [-1, 20], 32, pa.PA_STATUS_BAD_SEQLEN),
                                    ([[0, 1], [2, 3]], [30, 20], 25, pa.PA_STATUS_BAD_SEQLEN)):
        w, status = torch.ones(2, 2, room, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
        pa.pa_weights_add(w, w, None, q, lse, k, i32(tables), i32(lens), 0.1, status=status)
        want = torch.ones(2, 2, room)
        for b in range(2):
            n = min(max(lens[b], 0), 32, room)
            for t in range(n):
                draws = 2.0 if 0 <= tables[b][t // 16] < 4 else 0.0     # (two heads, scores of 0)
                want[b, :, t] = draws + (1.0 if t < n - 1 else 0.0)
        assert status.item() == bit and torch.equal(w.cpu(), want)


@pytest.mark.gpu
def test_weights_in_a_graph():
    q, k, lse = (torch.zeros(*s, dtype=t, device="cuda") for s, t in
                 (((2, 4, 64), torch.bfloat16), ((8, 16, 2, 64), torch.bfloat16), ((2, 4), torch.float32)))
    t, n, w = i32([[0, 1, 2, 3], [4, 5, 6, 7]]), i32([20, 30]), torch.zeros(2, 2, 64, device="cuda")
    pos = torch.full((2, 2, 64), -1, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.pa_weights_add(w, w, pos, q, lse, k, t, n, 0.1)
        n.add_(1)
    for _ in range(5):
        graph.replay()
    want, p = torch.zeros(2, 2, 64), torch.full((2, 2, 64), -1, dtype=torch.int32)
    for b, first in enumerate((20, 30)):
        for s in range(5):
            want[b, :, :first + s - 1] += 2
            want[b, :, first + s - 1] = 2
            p[b, :, first + s - 1] = first + s - 1
    assert torch.equal(w.cpu(), want) and torch.equal(pos.cpu(), p)


FAKE = ctypes.c_void_p(1 << 20)  # aligned, never dereferenced: these calls fail validation first


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), pa.PA_EINVAL), (dict(w=None), pa.PA_EINVAL), (dict(q=(1 << 20) + 8), pa.PA_EINVAL), (dict(B=-1), pa.PA_EINVAL),
    (dict(q_len=0), pa.PA_EINVAL), (dict(q_len=70000), pa.PA_EINVAL), (dict(mb=0), pa.PA_EINVAL), (dict(room=0), pa.PA_EINVAL),
    (dict(Hq=5), pa.PA_EINVAL), (dict(scale=math.nan), pa.PA_EINVAL), (dict(decay=-0.5), pa.PA_EINVAL),
    (dict(decay=math.inf), pa.PA_EINVAL), (dict(decay=math.nan), pa.PA_EINVAL), (dict(pos=(1 << 20) + 1), pa.PA_EINVAL),
    (dict(Hq=66), pa.PA_EUNSUPPORTED), (dict(mb=1 << 27), pa.PA_EUNSUPPORTED), (dict(B=70000), pa.PA_EUNSUPPORTED),
    (dict(desc=pa.CacheDesc(64, 16, 2, 96)), pa.PA_EUNSUPPORTED), (dict(B=0, q=None), pa.PA_OK),
])
def test_weights_refusals(kw, code):
    a = dict(w=FAKE, q=FAKE, q_len=1, desc=pa.CacheDesc(64, 16, 2, 128), mb=7, room=100, B=4, Hq=4, scale=0.1, decay=1.0,
             pos=None) | kw
    head = (a["w"], FAKE, a["pos"], a["q"], a["q_len"], FAKE, FAKE, a["desc"])
    tail = (FAKE, a["mb"], FAKE, None, a["room"], a["B"], a["Hq"], a["scale"], a["decay"], None, None)
    assert pa.lib().pa_weights_add(*head, *tail) == code
    assert pa.lib().pa_weights_add_fp8(*head, 1.0, *tail) == code
    assert pa.lib().pa_weights_add_fp8(*head, 0.0, *tail) == pa.PA_EINVAL


@pytest.mark.gpu
def test_weights_wrapper_refuses():
    z = lambda *s, t=torch.float32: torch.zeros(*s, dtype=t, device="cuda")   # noqa: E731
    ok = dict(nw=z(1, 2, 32), w=z(1, 2, 32), pos=None, q=z(1, 4, 64, t=torch.bfloat16), lse=z(1, 4),
              k=z(4, 16, 2, 64, t=torch.bfloat16), t=i32([[0, 1]]), n=i32([3]), ends=None)
    for kw in (dict(nw=z(1, 2, 31)), dict(w=z(2, 32)), dict(pos=z(1, 2, 32)), dict(lse=z(1, 1, 4)), dict(lse=z(1, 3)),
               dict(q=z(1, 4, 128, t=torch.bfloat16)), dict(t=i32([[0], [1]])), dict(ends=i32([1, 2])), dict(n=i32([3]).long()),
               dict(w=z(1, 2, 64)[..., ::2])):
        a = ok | kw
        with pytest.raises((TypeError, ValueError)):
            pa.pa_weights_add(a["nw"], a["w"], a["pos"], a["q"], a["lse"], a["k"], a["t"], a["n"], 0.1, ends=a["ends"])
