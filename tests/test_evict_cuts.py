"""Sequences that are cut again before a token was appended (pa_cache_evict): a cut leaves a row in no order, so its newest
tokens are found by their positions, not by their places.  And what a call reads stays bit for bit as it was."""
import math
import random

import pytest
import torch

import test_evict
from paged_kv_decode_cache_gb300 import build as B
from paged_kv_decode_cache_gb300 import pa
from paged_model import i32
from test_evict import Cache


@pytest.fixture(scope="module", autouse=True)
def _built():
    B.build()


def by_positions(weights, positions, n, fixed, first, recent):
    """The places of a row that stay, as a set, and the row's source of every place below n: the `recent` newest are those
    within `recent` of the largest position."""
    newest = max(positions, default=0)

    def key(t):
        safe = t < fixed or positions[t] < first or positions[t] > newest - recent
        w = math.inf if weights[t] != weights[t] else weights[t] + 0.0
        return (0, 0.0, t) if safe else (1, -w, t)
    stay = set(sorted(range(len(weights)), key=key)[:n])
    src = [t if t in stay else None for t in range(n)]
    behind = iter(t for t in range(n, len(weights)) if t in stay)
    return stay, [next(behind) if t is None else t for t in src]


def next_of(c, got):
    """The cache that a call left."""
    d = object.__new__(Cache)
    d.__dict__.update(c.__dict__)
    d.tables, d.lens, d.refs, d.weights, d.positions, d.pools = got[0], got[1], got[2], got[3], got[4], got[5]
    return d


def newest_stay(before, after, recent):
    """Of every row the tokens within `recent` of the newest are among those that stayed."""
    for b, n in enumerate(after.lens):
        for la in range(before.positions.shape[0]):
            for h in range(before.positions.shape[2]):
                had = before.positions[la, b, h, :before.lens[b]].tolist()
                has = set(after.positions[la, b, h, :n].tolist())
                assert {p for p in had if p > max(had, default=0) - recent} <= has


def cut_in_turn(monkeypatch, c, cuts):
    monkeypatch.setattr(test_evict, "evicted", by_positions)
    for budget, first, recent in cuts:
        c.check(budget, first, recent)
        after = next_of(c, c.run(budget, first, recent))
        newest_stay(c, after, recent)
        c = after
    return c


@pytest.mark.gpu
@pytest.mark.parametrize("lens,bs,hkv,d,layers,fp8,cuts", [
    ([100] * 6, 16, 3, 64, 1, False, [(60, 2, 8), (32, 2, 8)]),
    ([100, 70, 33, 0, 1], 16, 2, 128, 2, True, [(64, 4, 20), (40, 0, 20), (30, 0, 30), (29, 4, 8), (1, 0, 1)]),
    ([300, 1000], 32, 2, 64, 1, False, [(500, 0, 64), (499, 0, 64), (77, 1, 64), (64, 0, 64)]),
    ([9000], 16, 1, 64, 1, True, [(6000, 4, 300), (4500, 4, 200), (700, 4, 500)]),       # (a cluster for a row)
    ([20000, 12000], 16, 1, 64, 2, False, [(16000, 4, 128), (15000, 0, 3000), (100, 4, 90)]),
])
def test_a_row_cut_again_keeps_its_newest(monkeypatch, lens, bs, hkv, d, layers, fp8, cuts):
    cut_in_turn(monkeypatch, Cache(lens, bs, hkv, d, layers, fp8, seed=len(lens)), cuts)


@pytest.mark.gpu
@pytest.mark.parametrize("seed", range(8))
def test_cuts_of_many_random_rows(monkeypatch, seed):
    rng = random.Random(seed)
    c = Cache([rng.randint(80, 140) for _ in range(25)], 16, 2, 64, 1, fp8=seed % 2 == 1, seed=seed, again=seed % 4 > 1)
    cut_in_turn(monkeypatch, c, [(60, 2, 8), (32, 2, 8), (31, 0, 31)])


@pytest.mark.gpu
def test_the_newest_anywhere_in_a_row(monkeypatch):
    """The newest token at the first place, at the last one, next to the new length, in another CTA's share; rows of every
    head in an order of their own; positions that int32 just holds."""
    monkeypatch.setattr(test_evict, "evicted", by_positions)
    for lens, heads in (([200, 200, 200], 3), ([9000], 2)):
        c = Cache(lens, 16, heads, 64, 1, seed=7)
        for b, n in enumerate(lens):
            for h in range(heads):
                order = torch.randperm(n, generator=torch.Generator().manual_seed(10 * b + h)).int()
                spot = [0, n - 1, 59, 60, n // 2, n // 8][(2 * b + h) % 6]
                at = int((order == n - 1).nonzero())
                order[[at, spot]] = order[[spot, at]]
                c.positions[0, b, h, :n] = order + (2 ** 31 - n if (b + h) % 2 else 0)
        c.check(60, 3, 12)
        c.check(60, 0, 0)


@pytest.mark.gpu
def test_a_prefix_let_go_between_two_cuts(monkeypatch):
    """The other holder of a beginning goes: the second cut may throw its tokens out, and keeps the newest."""
    monkeypatch.setattr(test_evict, "evicted", by_positions)
    c = Cache([260, 300, 280], 16, 2, 64, 1, seed=12, shared=6)
    c.check(40, 2, 16)
    c = next_of(c, c.run(40, 2, 16))
    assert c.lens == [114] * 3
    for x in set(c.tables[0][:6]):
        c.refs[x] = 1
    c.tables, c.lens = [c.tables[0]], [c.lens[0]]     # (two of the three sequences are done)
    c.weights, c.positions = c.weights[:, :1].contiguous(), c.positions[:, :1].contiguous()
    c.check(40, 2, 16)
    newest_stay(c, next_of(c, c.run(40, 2, 16)), 16)

@pytest.mark.gpu
@pytest.mark.parametrize("again", [False, True])
def test_what_a_call_reads_stays_as_it_was(again):
    c = Cache([300, 64, 200, 7], 16, 2, 64, 2, seed=2, shared=2, again=again)
    c.weights[..., ::9], c.weights[..., 4::31] = math.nan, -0.0
    t, n, r, w, p = i32(c.tables), i32(c.lens), i32(c.refs), c.weights.cuda(), c.positions.cuda()
    pools = [x.cuda().view(torch.bfloat16) for x in c.pools]
    old = [x.clone() for x in (t, n, r, w, p)]
    new = [torch.zeros_like(x) for x in old]
    pa.pa_cache_evict(*new, t, n, r, w, p, pa.PoolSet(pools), 50, first=2, recent=9)
    for x, y in zip((t, n, r, w, p), old):
        assert torch.equal(x.view(torch.int32), y.view(torch.int32))
    assert new[1].tolist() == [50, 50, 50, 7] and int(new[2].sum()) < int(r.sum())
