"""Attention under score rules (pa_decode_scored, pa_decode_scored_fp8) against a plain one in 64 bits.

Tolerances, from the roundings on the way.  A score (in log2 units) is off by its fp32 product's
2^-22 of itself, the cap's 2^-21 of the cap (the exponential's form) and the bias's 2^-23 of itself;
for the magnitudes here (|s| < 40, cap <= 50, biases that matter < 40) that is below 2^-14 in s.
p = 2^(s - m) is held to 2^-17 (the hi + lo pair).  So a weight is off by 2^-13 of itself at most and the
output, a weighted mean, by 2^-12 max |v| (numerator and denominator), then rounded to bf16: 2^-8 of the
value.  lse: 2^-13 + 2^-23 of itself.  FP8 pools: the queries are exact in fp16 here, the codes too.
"""
import ctypes
import math
import random

import pytest
import torch

from paged_kv_decode_cache_gb300 import build as B
from paged_kv_decode_cache_gb300 import pa

FP8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _built():
    B.build()


def plain(q, k_cache, v_cache, tables, lens, scale, softcap, slopes, window, prefix, ks=1.0, vs=1.0):
    """(out, lse) in 64 bits; q [B, Q, Hq, D].  Only tokens that a query sees are read."""
    Bn, Q, Hq, D = q.shape
    bs, Hkv = k_cache.shape[1], k_cache.shape[2]
    out = torch.zeros(Bn, Q, Hq, D, dtype=torch.float64)
    lse = torch.full((Bn, Q, Hq), -math.inf, dtype=torch.float64)
    as64 = lambda t, s: (t.view(FP8).double() * s if t.dtype == torch.uint8 else t.double())  # noqa: E731
    q = q.double().cpu()
    for b in range(Bn):
        L = int(lens[b])
        pre = 0 if prefix is None else int(prefix[b])
        for i in range(Q):
            pos = L - Q + i
            seen = [t for t in range(L) if t < pre or (t <= pos and (window == 0 or t > pos - window))]
            if not seen:
                continue
            where = torch.tensor([int(tables[b][t // bs]) * bs + t % bs for t in seen], device=k_cache.device)
            at = torch.tensor(seen).double() - pos
            k = as64(k_cache.flatten(0, 1)[where], ks).cpu()
            v = as64(v_cache.flatten(0, 1)[where], vs).cpu()
            for h in range(Hq):
                g = h // (Hq // Hkv)
                s = k[:, g] @ q[b, i, h] * scale
                if softcap:
                    s = softcap * torch.tanh(s / softcap)
                if slopes is not None:
                    s = s + float(slopes[h]) * at
                lse[b, i, h] = torch.logsumexp(s, 0)
                out[b, i, h] = torch.exp(s - lse[b, i, h]) @ v[:, g]
    return out, lse


def inputs(Bn, Q, Hq, Hkv, D, bs, lens, fp8, seed, sharp=3.0, window=0, prefix=None):
    """Pools whose unused and unseen rows hold NaN, and tables that name nothing where no query looks."""
    g = torch.Generator().manual_seed(seed)
    rng = random.Random(seed)
    mb = max(1, max(-(-n // bs) for n in lens))
    nb = sum(-(-n // bs) for n in lens) + 2
    ids = list(range(nb))
    rng.shuffle(ids)
    q = (torch.randn(Bn, Q, Hq, D, generator=g) * sharp).to(torch.bfloat16)
    pools = [torch.randn(nb, bs, Hkv, D, generator=g).to(torch.bfloat16) for _ in range(2)]
    if fp8:
        pools = [p.to(FP8).view(torch.uint8) for p in pools]
    used = torch.zeros(nb * bs, dtype=torch.bool)
    tables = torch.full((Bn, mb), -1, dtype=torch.int32)
    at = 0
    for b, L in enumerate(lens):
        row = ids[at:at + -(-L // bs)]
        at += len(row)
        pre = 0 if prefix is None else prefix[b]
        first = max(0, L - Q - window + 1) if window else 0
        for t in range(L):
            # (a query of the call before the first one's window start sees nothing older)
            if t < pre or t >= first:
                used[row[t // bs] * bs + t % bs] = True
                tables[b, t // bs] = row[t // bs]
    for p in pools:
        p.flatten(0, 1)[~used] = 0x7F if fp8 else math.nan
    return q.cuda(), [p.cuda() for p in pools], tables.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")


def run(q, pools, tables, lens, scale, splits, fp8, ks=0.5, vs=0.75, stream=None, status=None, squeeze=True, **rules):
    Bn, Q, Hq, D = q.shape
    bs, Hkv = pools[0].shape[1], pools[0].shape[2]
    x = q.view(Bn, Hq, D) if Q == 1 and squeeze else q
    out, lse = torch.full_like(x, 7.0), torch.full(x.shape[:-1], 7.0, device="cuda")
    P = splits or pa.pa_scored_num_splits(Bn, Q, Hq, Hkv, D, tables.shape[1], bs, window=rules.get("window", 0),
                                          max_prefix=(rules.get("max_prefix") or tables.shape[1] * bs)
                                          if rules.get("prefix_lens") is not None else 0)
    ws = torch.zeros(max(1, pa.pa_splitkv_workspace_bytes(Bn * Q, Hq, D, P)), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    if fp8:
        pa.pa_decode_scored_fp8(out, lse, x, *pools, ks, vs, tables, lens, scale, num_splits=splits, workspace=ws,
                                status=status, stream=stream, **rules)
    else:
        pa.pa_decode_scored(out, lse, x, *pools, tables, lens, scale, num_splits=splits, workspace=ws, status=status,
                            stream=stream, **rules)
    torch.cuda.synchronize()
    return out.view(q.shape), lse.view(q.shape[:-1])


def close(got, want, vmax):
    out, lse = got[0].double().cpu(), got[1].double().cpu()
    assert torch.equal(torch.isinf(lse), torch.isinf(want[1]))
    fin = torch.isfinite(want[1])
    assert ((lse - want[1])[fin].abs() <= 2.0 ** -13 + 2.0 ** -23 * want[1][fin].abs()).all()
    assert torch.isfinite(out).all() and (out[~fin] == 0).all()
    assert ((out - want[0]).abs() <= 2.0 ** -12 * vmax + 2.0 ** -8 * want[0].abs()).all()


def slopes_of(Hq):
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / Hq) for h in range(Hq)], device="cuda")


def case(Bn, Q, Hq, Hkv, D, bs, lens, fp8=False, splits=0, seed=0, **rules):
    prefix, window = rules.pop("prefix", None), rules.get("window", 0)
    q, pools, tables, L = inputs(Bn, Q, Hq, Hkv, D, bs, lens, fp8, seed, window=window, prefix=prefix)
    scale = 1.0 / math.sqrt(D)
    if rules.pop("alibi", False):
        rules["alibi_slopes"] = slopes_of(Hq)
    if prefix is not None:
        rules["prefix_lens"] = torch.tensor(prefix, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run(q, pools, tables, L, scale, splits, fp8, status=status, **rules)
    assert status.item() == 0
    want = plain(q, *pools, tables.cpu(), lens, scale, rules.get("softcap", 0.0), rules.get("alibi_slopes"), window,
                 prefix, *((0.5, 0.75) if fp8 else ()))
    seen = pools[1].view(FP8).double() * 0.75 if fp8 else pools[1].double()
    close(got, want, float(torch.nan_to_num(seen).abs().max()))


RULES = {
    "none": {}, "cap": dict(softcap=20.0), "tight cap": dict(softcap=1.5), "alibi": dict(alibi=True),
    "window": dict(window=37), "window of one": dict(window=1), "all": dict(softcap=50.0, alibi=True, window=100),
}


@pytest.mark.gpu
@pytest.mark.parametrize("rules", RULES)
@pytest.mark.parametrize("D,Hq,Hkv", [(128, 28, 4), (128, 3, 1), (128, 16, 8), (128, 40, 2), (64, 4, 2), (64, 8, 1)])
def test_single_tokens(D, Hq, Hkv, rules):
    lens = [1, 16, 17, 150, 333, 0]
    for splits in (1, 3, 0):
        case(len(lens), 1, Hq, Hkv, D, 16, lens, splits=splits, seed=D + Hq, **RULES[rules])


@pytest.mark.gpu
@pytest.mark.parametrize("rules", RULES)
@pytest.mark.parametrize("Hq,Hkv", [(28, 4), (16, 8), (32, 1), (2, 2)])
def test_single_tokens_over_fp8_pools(Hq, Hkv, rules):
    lens = [1, 48, 50, 311, 0]
    for splits in (1, 4, 0):
        case(len(lens), 1, Hq, Hkv, 128, 16, lens, fp8=True, splits=splits, seed=Hq, **RULES[rules])


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("bs", [16, 256])
@pytest.mark.parametrize("window,prefix", [(20, [4, 0, 33, 200, 16]), (0, [5, 1, 9, 31, 0]), (1, [1, 1, 1, 1, 1]),
                                           (64, [300, 3, 47, 48, 49]), (5000, [7, 1, 0, 2, 3])])
def test_prefix_with_and_without_a_window(window, prefix, bs, fp8):
    lens = [250, 5, 100, 400, 64]
    prefix = [min(p, n) for p, n in zip(prefix, lens)]
    for splits in (1, 5, 0):
        case(5, 1, 12, 2, 128, bs, lens, fp8=fp8, splits=splits, seed=bs, window=window, prefix=prefix, softcap=30.0)
    if not fp8:
        case(5, 1, 8, 2, 64, bs, lens, splits=3, seed=bs, window=window, prefix=prefix, alibi=True)


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("Q,Hq,Hkv", [(2, 28, 4), (5, 4, 4), (8, 8, 2), (7, 12, 2)])
def test_a_few_tokens(Q, Hq, Hkv, fp8):
    """Verification of drafted tokens: several queries per sequence, some before the first token."""
    lens = [Q, 3, 70, 129, 1]
    prefix = [0, 2, 68, 5, 1]
    for splits in (1, 3, 0):
        case(5, Q, Hq, Hkv, 128, 16, lens, fp8=fp8, splits=splits, seed=Q, softcap=25.0, alibi=True)
        case(5, Q, Hq, Hkv, 128, 16, lens, fp8=fp8, splits=splits, seed=Q, window=11, prefix=prefix, alibi=True)


@pytest.mark.gpu
@pytest.mark.parametrize("Q,Hq,Hkv,bs", [(33, 4, 4, 16), (100, 12, 2, 16), (40, 28, 4, 256), (130, 2, 1, 32)])
def test_chunks(Q, Hq, Hkv, bs):
    lens = [Q, Q + 90, 150, 20]
    prefix = [Q // 2, 0, 149, 20]
    case(4, Q, Hq, Hkv, 128, bs, lens, seed=Q, softcap=30.0, prefix=prefix)
    case(4, Q, Hq, Hkv, 128, bs, lens, seed=Q, window=29, prefix=[min(p, 9) for p in prefix], alibi=True)
    case(4, Q, Hq, Hkv, 128, bs, lens, seed=Q, splits=3, window=50)
    case(4, Q, Hq, Hkv, 128, bs, lens, seed=Q, splits=2, alibi=True)


@pytest.mark.gpu
def test_chunk_over_fp8_pools():
    case(2, 20, 8, 2, 128, 16, [20, 75], fp8=True, seed=3, softcap=30.0, window=31, prefix=[3, 0])


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True])
def test_long_cache(fp8):
    """Several chunks per partition, waves of CTAs, the grid and the combine merges."""
    for Bn, lens, rules in ((1, [9000], dict(softcap=40.0)), (2, [3000, 8191], dict(window=2500, prefix=[100, 4])),
                            (70, [700 + 13 * i for i in range(70)], dict(window=300, softcap=15.0))):
        if Bn == 70:
            case(Bn, 1, 4, 2, 128, 16, lens, fp8=fp8, seed=Bn, **rules)
        else:
            case(Bn, 1, 8, 4, 128, 16, lens, fp8=fp8, seed=Bn, alibi=True, **rules)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
def test_no_rules_equal_plain_decode(D):
    lens = [300, 17, 1, 0]
    q, pools, tables, L = inputs(4, 1, 8, 2, D, 16, lens, False, 9)
    out, lse = run(q, pools, tables, L, 0.1, 1, False)
    ref, ref_lse = torch.empty_like(q.view(4, 8, D)), torch.empty(4, 8, device="cuda")
    pa.pa_decode(ref, ref_lse, q.view(4, 8, D), *pools, tables, L, 0.1)
    torch.cuda.synchronize()
    assert torch.equal(out.view(4, 8, D), ref) and torch.equal(lse.view(4, 8), ref_lse)


@pytest.mark.gpu
def test_scores_at_the_cap_and_far_biases():
    """Scores far past the cap, and a bias that leaves the last tokens alone."""
    q, pools, tables, L = inputs(1, 1, 4, 2, 128, 16, [200], False, 4, sharp=200.0)
    for rules in (dict(softcap=5.0), dict(softcap=30.0, alibi_slopes=torch.full((4,), 3.0, device="cuda"))):
        got = run(q, pools, tables, L, 0.09, 2, False, **rules)
        want = plain(q, *pools, tables.cpu(), [200], 0.09, rules["softcap"], rules.get("alibi_slopes"), 0, None)
        close(got, want, float(torch.nan_to_num(pools[1].double()).abs().max()))


@pytest.mark.gpu
def test_bad_prefix_lengths_are_reported_and_clamped():
    lens = [40, 40]
    q, pools, tables, L = inputs(2, 1, 4, 2, 128, 16, lens, False, 4)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    bad = torch.tensor([-3, 30], dtype=torch.int32, device="cuda")
    got = run(q, pools, tables, L, 0.1, 1, False, window=5, prefix_lens=bad, max_prefix=20, status=status)
    assert status.item() == pa.PA_STATUS_BAD_SEQLEN
    want = plain(q, *pools, tables.cpu(), lens, 0.1, 0.0, None, 5, [0, 20])
    close(got, want, float(torch.nan_to_num(pools[1].double()).abs().max()))


@pytest.mark.gpu
def test_in_a_graph_and_on_another_stream():
    lens = [900, 40, 333]
    q, pools, tables, L = inputs(3, 1, 28, 4, 128, 16, lens, False, 4)
    rules = dict(softcap=30.0, window=256, alibi_slopes=slopes_of(28))
    ref = run(q, pools, tables, L, 0.1, 0, False, **rules)
    other = run(q, pools, tables, L, 0.1, 0, False, stream=torch.cuda.Stream(), **rules)
    assert torch.equal(ref[0], other[0]) and torch.equal(ref[1], other[1])
    out, lse = torch.empty(3, 28, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(3, 28, device="cuda")
    P = pa.pa_scored_num_splits(3, 1, 28, 4, 128, tables.shape[1], 16, window=256)
    ws = torch.zeros(pa.pa_splitkv_workspace_bytes(3, 28, 128, P), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.pa_decode_scored(out, lse, q.view(3, 28, 128), *pools, tables, L, 0.1, num_splits=P, workspace=ws, **rules)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out.view_as(ref[0]), ref[0]) and torch.equal(lse.view_as(ref[1]), ref[1])


@pytest.mark.gpu
@pytest.mark.parametrize("kernel", ["cuda_core"])
def test_forced_kernel(use_kernel, kernel):
    use_kernel(kernel)
    lens = [1, 100, 260]
    case(3, 1, 12, 2, 128, 16, lens, splits=2, seed=1, softcap=20.0, alibi=True, window=77, prefix=[1, 20, 3])


# ---- host only -------------------------------------------------------------------------------

FAKE = ctypes.c_void_p(1 << 20)  # aligned, never dereferenced: these calls fail validation first


@pytest.mark.parametrize("kw,code", [
    (dict(softcap=-1.0), pa.PA_EINVAL), (dict(softcap=math.nan), pa.PA_EINVAL), (dict(softcap=math.inf), pa.PA_EINVAL),
    (dict(softcap=1e-35), pa.PA_EINVAL), (dict(window=-1), pa.PA_EINVAL), (dict(prefix=1 << 20, max_prefix=-1), pa.PA_EINVAL),
    (dict(slopes=(1 << 20) + 2), pa.PA_EINVAL), (dict(prefix=(1 << 20) + 1), pa.PA_EINVAL),
    (dict(q_len=0), pa.PA_EINVAL), (dict(q_len=70000), pa.PA_EINVAL), (dict(q=None), pa.PA_EINVAL),
    (dict(Hq=5), pa.PA_EINVAL), (dict(Hq=66), pa.PA_EUNSUPPORTED), (dict(splits=-1), pa.PA_EINVAL),
    (dict(splits=3), pa.PA_EWORKSPACE), (dict(desc=pa.CacheDesc(64, 16, 2, 96)), pa.PA_EUNSUPPORTED),
    (dict(desc=pa.CacheDesc(64, 16, 2, 64), q_len=2), pa.PA_EUNSUPPORTED), (dict(scale=math.nan), pa.PA_EINVAL),
])
def test_refusals(kw, code):
    a = dict(softcap=10.0, slopes=None, window=5, prefix=None, max_prefix=0, q=FAKE, q_len=1, Hq=4, splits=1, scale=0.1,
             desc=pa.CacheDesc(64, 16, 2, 128))
    a.update(kw)
    rules = pa.ScoreRules(a["softcap"], a["slopes"], a["window"], a["prefix"], a["max_prefix"])
    tail = (FAKE, 7, FAKE, 4, a["Hq"], a["scale"], ctypes.byref(rules), a["splits"], None, 0, None, None)
    assert pa.lib().pa_decode_scored(FAKE, None, a["q"], a["q_len"], FAKE, FAKE, a["desc"], *tail) == code
    assert pa.lib().pa_decode_scored_fp8(FAKE, None, a["q"], a["q_len"], FAKE, FAKE, a["desc"], 1.0, 1.0, *tail) == code


def test_more_refusals_and_an_empty_batch():
    rules = pa.ScoreRules(0.0, None, 0, None, 0)
    d = pa.CacheDesc(64, 16, 2, 128)
    tail = (FAKE, 7, FAKE, 4, 4, 0.1, ctypes.byref(rules), 1, None, 0, None, None)
    for ks, vs in ((0.0, 1.0), (1.0, math.nan)):
        assert pa.lib().pa_decode_scored_fp8(FAKE, None, FAKE, 1, FAKE, FAKE, d, ks, vs, *tail) == pa.PA_EINVAL
    assert pa.lib().pa_decode_scored_fp8(FAKE, None, FAKE, 1, FAKE, FAKE, pa.CacheDesc(64, 16, 2, 64), 1.0, 1.0,
                                         *tail) == pa.PA_EUNSUPPORTED
    none = list(tail)
    none[6] = None
    assert pa.lib().pa_decode_scored(FAKE, None, FAKE, 1, FAKE, FAKE, d, *none) == pa.PA_EINVAL
    empty = list(tail)
    empty[3] = 0
    assert pa.lib().pa_decode_scored(FAKE, None, FAKE, 1, FAKE, FAKE, d, *empty) == pa.PA_OK


@pytest.mark.gpu
@pytest.mark.parametrize("Bn", [2, 31, 32, 33])
def test_chunks_of_many_ragged_sequences(Bn):
    """The kernel takes up to 32 sequences from the longest; equal, empty and short ones among them."""
    rng = random.Random(Bn)
    lens = [rng.choice([0, 7, 40, 40, 64, 65, rng.randint(1, 500)]) for _ in range(Bn)]
    for splits in (1, 2):
        case(Bn, 40, 4, 2, 128, 16, lens, seed=Bn, splits=splits, softcap=30.0)


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("Bn", [1, 16])
@pytest.mark.parametrize("L", [15, 48, 112, 192, 320, 512])
def test_short_calls_of_every_split(L, Bn, fp8):
    """The rule's count, and partitions of a tile each, some of them empty."""
    for Q, Hq, Hkv in ((1, 28, 4), (4, 16, 8)):
        for splits in (0, -(-L // 16), -(-L // 16) + 1):
            case(Bn, Q, Hq, Hkv, 128, 16, [max(0, L - 3 * b) for b in range(Bn)], fp8=fp8, splits=splits, seed=L,
                 softcap=30.0)


def test_split_counts_of_short_calls():
    for L, most in ((1, 1), (3, 1), (7, 7), (32, 32), (600, 64)):   # tiles of a table
        for B in (1, 4, 16, 64, 1000):
            for heads in ((28, 4), (32, 8), (16, 8), (12, 2)):
                for q_len in (1, 4, 40):
                    P = pa.pa_scored_num_splits(B, q_len, *heads, 128, L, 16, sm_count=152)
                    assert 1 <= P <= most
                    if q_len == 40 and heads[0] * q_len >= 256 * heads[1]:
                        assert P <= -(-L // 8)


def test_split_counts():
    """Without a window the plain rule; with one, the rule for what can be seen."""
    for args in ((8, 1, 28, 4, 128, 256, 16), (1, 1, 12, 2, 128, 100, 16), (3, 4, 28, 4, 128, 64, 256), (2, 1, 8, 2, 64, 50, 16)):
        assert pa.pa_scored_num_splits(*args, sm_count=152) == pa.pa_choose_num_splits_mq(*args, 152)
    assert pa.pa_scored_num_splits(8, 1, 28, 4, 128, 2048, 16, window=1024, max_prefix=4, sm_count=152) == \
        pa.pa_choose_num_splits(8, 28, 4, 128, 66, 16, 152)
    assert pa.pa_scored_num_splits(1, 1, 28, 4, 128, 2048, 16, window=1, sm_count=152) == 1
    for kw in (dict(window=-1), dict(max_prefix=-1), dict(sm_count=-1)):
        with pytest.raises(pa.PAError) as e:
            pa.pa_scored_num_splits(8, 1, 28, 4, 128, 256, 16, **{"sm_count": 152, **kw})
        assert e.value.code == pa.PA_EINVAL
    with pytest.raises(pa.PAError):
        pa.pa_scored_num_splits(8, 2, 8, 2, 64, 256, 16, sm_count=152)
