"""Beam selection (pa_beam_select) against a plain one in 64 bits.

Tokens and parents are whole numbers and have to be equal; the inputs leave no two scores nearer
than the kernel's error.  A score's error: lse's sum of exponentials in fp32, each term off by
2^-21 or so of itself (the product's rounding, 2 units in the last place of the exponential), the sum by
2^-20 at most; the result is rounded to fp32 once (2^-24 of it).  So 2^-19 + 2^-23 |score|.
"""
import ctypes
import math

import numpy as np
import pytest
import torch

from paged_kv_decode_cache_gb300 import build as B
from paged_kv_decode_cache_gb300 import pa


@pytest.fixture(scope="module", autouse=True)
def _built():
    B.build()


def plain(logits, cum, finished, eos, K):
    """[(score, token, parent row)] of every group, K each, in 64 bits."""
    x = logits.double().cpu().numpy()
    cum = cum.double().cpu().numpy()
    groups, beams = cum.shape
    out = []
    for g in range(groups):
        found = []
        for w in range(beams):
            c = cum[g, w]
            if finished is not None and finished[g, w]:
                found.append((np.array([c]), np.array([w * x.shape[1] + eos])))
                continue
            row = x[g * beams + w]
            top = row.max()
            if not np.isfinite(top):   # (NaN, +inf, or nothing allowed)
                continue
            s = c + (row - (top + np.log(np.exp(row - top).sum())))
            found.append((s, w * x.shape[1] + np.arange(x.shape[1])))
        s = np.concatenate([f[0] for f in found]) if found else np.zeros(0)
        i = np.concatenate([f[1] for f in found]) if found else np.zeros(0, int)
        keep = s > -np.inf
        s, i = s[keep], i[keep]
        order = np.lexsort((i, -s))[:K]
        rows = [(s[j], i[j] % x.shape[1], g * beams + i[j] // x.shape[1]) for j in order]
        out.append(rows + [(-math.inf, -1, -1)] * (K - len(rows)))
    return out


def run(logits, cum, K, finished=None, eos=-1, ws=None, stream=None):
    groups, beams = cum.shape
    scores = torch.full((groups, K), 7.0, device="cuda")
    tokens, parents = (torch.full((groups, K), 77, dtype=torch.int32, device="cuda") for _ in range(2))
    if ws is None:
        ws = torch.zeros(pa.pa_beam_workspace_bytes(groups, beams, logits.shape[1], K, logits.dtype),
                         dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    pa.pa_beam_select(scores, tokens, parents, logits, cum, finished=finished, eos=eos, workspace=ws, stream=stream)
    torch.cuda.synchronize()
    return scores.cpu(), tokens.cpu(), parents.cpu()


def check(got, want):
    scores, tokens, parents = got
    assert tokens.tolist() == [[r[1] for r in rows] for rows in want]
    assert parents.tolist() == [[r[2] for r in rows] for rows in want]
    want = np.array([[r[0] for r in rows] for rows in want])
    got = scores.double().numpy()
    fin = np.isfinite(want)
    assert np.array_equal(got[~fin], want[~fin])
    assert (abs(got[fin] - want[fin]) <= 2.0 ** -19 + 2.0 ** -23 * abs(want[fin])).all()


def spread(cum_shape, seed):
    """Beams' scores whose differences keep clear of the logits' grids."""
    g = torch.Generator().manual_seed(seed)
    return (torch.rand(cum_shape, generator=g) * -5).cuda()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("groups,beams,vocab,K,pad", [
    (1, 1, 1, 1, 0), (1, 1, 5, 8, 3), (1, 4, 7, 4, 0), (3, 2, 1000, 4, 1), (2, 5, 8191, 10, 0), (1, 4, 32000, 4, 0),
    (2, 3, 50257, 6, 0), (1, 1, 16384, 64, 0), (1, 64, 300, 64, 5), (40, 4, 9001, 8, 0), (1, 8, 262147, 16, 0),
    (70, 8, 700, 3, 0),
])
def test_matches_the_definition(dtype, groups, beams, vocab, K, pad):
    g = torch.Generator().manual_seed(vocab + K)
    logits = (torch.randn(groups * beams, vocab + pad, generator=g) * 2.5).to(dtype).cuda()[:, :vocab]
    cum = spread((groups, beams), vocab)
    check(run(logits, cum, K), plain(logits, cum, None, -1, K))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("vocab", [37, 20000, 100003])
@pytest.mark.parametrize("kind", ["same", "rising", "falling", "one block", "few allowed", "two values", "steps"])
def test_orders_that_defeat_a_bound(dtype, vocab, kind):
    """Equal values, sorted rows, and rows whose large values sit together."""
    i = torch.arange(vocab, dtype=torch.float32)
    x = {"same": torch.zeros(vocab), "rising": i / vocab * 8, "falling": -i / vocab * 8,
         "one block": torch.where((i >= vocab // 3) & (i < vocab // 3 + 900), 5 + (i % 64) / 32, -3.0),
         "few allowed": torch.where(i % 9973 == 7, i / 4096, -math.inf),
         "two values": torch.where(i % 7 < 3, 1.0, 0.5), "steps": (i // 100 % 5)}[kind]
    logits = torch.stack([x, x.flip(0), x.roll(11)]).to(dtype).cuda()
    cum = torch.tensor([[-0.3, -1.7321, -2.2361]], device="cuda")
    for K in (1, 3, 64):
        check(run(logits, cum, K), plain(logits, cum, None, -1, K))


@pytest.mark.gpu
def test_equal_rows_tie_to_the_lower_beam():
    row = (torch.randn(30011, generator=torch.Generator().manual_seed(1)) * 2).to(torch.bfloat16)
    logits = row.repeat(3, 1).cuda()
    cum = torch.full((1, 3), -1.25, device="cuda")
    scores, tokens, parents = run(logits, cum, 12)
    best = torch.sort(row.float(), descending=True, stable=True).indices[:4]
    want = sorted(((-float(row[t]), w, int(t)) for t in torch.sort(row.float(), descending=True, stable=True).indices[:40]
                   for w in range(3)))[:12]
    assert parents[0].tolist() == [w for _, w, _ in want] and tokens[0].tolist() == [t for _, _, t in want]
    assert int(tokens[0, 0]) == int(best[0])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_finished_dead_and_masked_beams(dtype):
    g = torch.Generator().manual_seed(3)
    logits = (torch.randn(12, 5003, generator=g) * 2).to(dtype).cuda()
    logits[1] = -math.inf                       # nothing allowed
    logits[2, 2:] = -math.inf                   # two entries allowed
    logits[4] = math.nan                        # a finished beam's logits are not read
    logits[6, 17] = math.nan                    # leaves its beam without candidates
    logits[7, :] = -math.inf                    # so does one among entries that are not allowed
    logits[7, 4001] = math.nan
    logits[9, 5] = math.inf                     # leaves its beam without candidates
    cum = spread((4, 3), 4)
    cum[2, 0] = -math.inf                       # dead
    fin = torch.zeros(4, 3, dtype=torch.uint8, device="cuda")
    fin[1, 1] = 1
    fin[3, :] = torch.tensor([0, 1, 1])
    for K in (2, 6, 9):
        check(run(logits, cum, K, finished=fin, eos=4999), plain(logits, cum, fin.cpu().numpy(), 4999, K))


@pytest.mark.gpu
def test_nothing_left_anywhere():
    logits = torch.full((2, 999), -math.inf, dtype=torch.bfloat16, device="cuda")
    scores, tokens, parents = run(logits, torch.zeros(1, 2, device="cuda"), 5)
    assert (scores == -math.inf).all() and (tokens == -1).all() and (parents == -1).all()
    logits = torch.zeros(2, 999, dtype=torch.bfloat16, device="cuda")
    assert (run(logits, torch.full((1, 2), -math.inf, device="cuda"), 5)[1] == -1).all()


@pytest.mark.gpu
@pytest.mark.parametrize("big", [300.0, 60000.0])
def test_large_logits(big):
    g = torch.Generator().manual_seed(5)
    logits = (torch.randn(4, 12345, generator=g) + big).to(torch.float32).cuda()
    cum = spread((2, 2), 6)
    want = plain(logits, cum, None, -1, 4)
    scores, tokens, parents = run(logits, cum, 4)
    assert tokens.tolist() == [[r[1] for r in rows] for rows in want]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("groups,beams,vocab,K", [
    (1, 1, 40000, 1), (3, 1, 40001, 33), (2, 16, 20000, 12), (1, 7, 70000, 9), (60, 4, 20011, 16), (1, 33, 9000, 33),
    (2, 8, 120001, 16), (1, 64, 3000, 5), (5, 12, 150, 20), (4, 2, 1025, 64),
])
def test_joins_of_every_size(dtype, groups, beams, vocab, K):
    """Lists of a join: from one to many slices per row, few and many candidates; some beams done."""
    g = torch.Generator().manual_seed(vocab + beams)
    logits = (torch.randn(groups * beams, vocab, generator=g) * 2).to(dtype).cuda()
    cum = spread((groups, beams), vocab + K)
    fin = (torch.rand(groups, beams, generator=g) < 0.2).to(torch.uint8).cuda()
    check(run(logits, cum, K, finished=fin, eos=vocab - 1), plain(logits, cum, fin.cpu().numpy(), vocab - 1, K))


@pytest.mark.gpu
def test_negative_zero_ties_with_zero():
    logits = torch.tensor([[-0.0, 0.0, -1.0, -0.0]], dtype=torch.bfloat16, device="cuda")
    assert run(logits, torch.zeros(1, 1, device="cuda"), 3)[1].tolist() == [[0, 1, 3]]


@pytest.mark.gpu
def test_workspace_serves_many_calls_a_graph_and_a_stream():
    g = torch.Generator().manual_seed(7)
    logits = (torch.randn(24, 20011, generator=g) * 2.5).to(torch.bfloat16).cuda()
    cum = spread((6, 4), 8)
    want = plain(logits, cum, None, -1, 4)
    ws = torch.zeros(pa.pa_beam_workspace_bytes(6, 4, 20011, 4, torch.bfloat16), dtype=torch.uint8, device="cuda")
    for _ in range(3):
        check(run(logits, cum, 4, ws=ws), want)
    check(run(logits, cum, 4, ws=ws, stream=torch.cuda.Stream()), want)
    scores = torch.empty(6, 4, device="cuda")
    tokens, parents = (torch.empty(6, 4, dtype=torch.int32, device="cuda") for _ in range(2))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.pa_beam_select(scores, tokens, parents, logits, cum, workspace=ws)
    for _ in range(2):
        scores.zero_()
        graph.replay()
        torch.cuda.synchronize()
        check((scores.cpu(), tokens.cpu(), parents.cpu()), want)


@pytest.mark.gpu
def test_wrapper_refuses():
    logits = torch.zeros(4, 100, dtype=torch.bfloat16, device="cuda")
    cum = torch.zeros(2, 2, device="cuda")
    out = [torch.zeros(2, 3, device="cuda")] + [torch.zeros(2, 3, dtype=torch.int32, device="cuda")] * 2
    ws = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda")
    with pytest.raises(TypeError):
        pa.pa_beam_select(*out, logits.half(), cum, workspace=ws)
    with pytest.raises(ValueError):
        pa.pa_beam_select(*out, logits[:3], cum, workspace=ws)
    with pytest.raises(ValueError):
        pa.pa_beam_select(*out, logits.t().contiguous().t(), cum, workspace=ws)
    with pytest.raises(ValueError):
        pa.pa_beam_select(*out, logits, cum, finished=torch.zeros(2, 3, dtype=torch.uint8, device="cuda"), eos=1,
                          workspace=ws)
    with pytest.raises(pa.PAError) as e:
        pa.pa_beam_select(*out, logits, cum)
    assert e.value.code == pa.PA_EWORKSPACE
    with pytest.raises(TypeError):
        pa.pa_beam_workspace_bytes(1, 1, 10, 1, torch.float16)


FAKE = ctypes.c_void_p(1 << 20)  # aligned, never dereferenced: these calls fail validation first


@pytest.mark.parametrize("kw,code", [
    (dict(groups=-1), pa.PA_EINVAL), (dict(beams=0), pa.PA_EINVAL), (dict(vocab=0), pa.PA_EINVAL), (dict(K=0), pa.PA_EINVAL),
    (dict(beams=65), pa.PA_EUNSUPPORTED), (dict(K=65), pa.PA_EUNSUPPORTED),
    (dict(vocab=1 << 30, stride=1 << 30), pa.PA_EUNSUPPORTED), (dict(groups=1 << 21), pa.PA_EUNSUPPORTED),
    (dict(type=2), pa.PA_EINVAL), (dict(stride=999), pa.PA_EINVAL), (dict(eos=-1), pa.PA_EINVAL),
    (dict(eos=1000), pa.PA_EINVAL), (dict(logits=None), pa.PA_EINVAL), (dict(cum=None), pa.PA_EINVAL),
    (dict(parents=None), pa.PA_EINVAL), (dict(logits=ctypes.c_void_p((1 << 20) + 2)), pa.PA_EINVAL),
    (dict(scores=ctypes.c_void_p((1 << 20) + 2)), pa.PA_EINVAL), (dict(ws=None), pa.PA_EWORKSPACE),
    (dict(ws_bytes=10), pa.PA_EWORKSPACE), (dict(ws=ctypes.c_void_p((1 << 20) + 64)), pa.PA_EWORKSPACE),
])
def test_refusals(kw, code):
    a = dict(scores=FAKE, tokens=FAKE, parents=FAKE, logits=FAKE, type=0, stride=1000, cum=FAKE, finished=FAKE, eos=5,
             groups=2, beams=4, vocab=1000, K=4, ws=FAKE, ws_bytes=1 << 20)
    a.update(kw)
    assert pa.lib().pa_beam_select(*a.values(), None) == code


def test_no_groups_and_workspace_sizes():
    assert pa.lib().pa_beam_select(None, None, None, None, 0, 1000, None, None, -1, 0, 4, 1000, 4, None, 0, None) == pa.PA_OK
    assert pa.pa_beam_workspace_bytes(0, 4, 1000, 4, torch.bfloat16) == 0
    assert pa.pa_beam_workspace_bytes(1, 65, 1000, 4, torch.bfloat16) == 0
    assert pa.pa_beam_workspace_bytes(2, 4, 1000, 4, torch.float32) >= 8 * 4 * 8 + 8 * 12
