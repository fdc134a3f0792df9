"""Eviction by accumulated weight (pa_cache_evict) against a plain Python model.  Everything is chosen, counted or
copied: equality throughout."""
import ctypes
import math
import random

import pytest
import torch

from paged_kv_decode_cache_gb300 import build as B
from paged_kv_decode_cache_gb300 import pa
from paged_model import evicted, i32, layout


@pytest.fixture(scope="module", autouse=True)
def _built():
    B.build()


def plain(tables, lens, refs, weights, positions, pools, bs, budget, first, recent, room, odd=()):
    """What a call leaves: (tables, lens, refs, weights, positions, pools, places written of the two in between)."""
    layers, Bn, hkv, _ = weights.shape
    mb, nb = len(tables[0]), len(refs)
    new_t, new_n, new_r = [], [], list(refs)
    w, p, pools = weights.clone(), positions.clone(), [x.clone() for x in pools]
    for b in range(Bn):
        L = lens[b]
        k = -(-L // bs)
        good = [x if 0 <= x < nb and refs[x] > 0 else -1 for x in tables[b][:k]]
        ahead = [x for x in tables[b][k:k + 1] if L % bs == 0 and 0 <= x < nb and refs[x] > 0]
        held = [j + 1 for j, x in enumerate(good) if x >= 0 and refs[x] > 1]
        fixed = min(L, max(held, default=0) * bs)
        n = min(L, max(budget, fixed + first + recent) if fixed else budget)
        if -1 in good or L > room or b in odd:
            n = L
        row = good + ahead
        if n < L:
            for x in row[n // bs + 1:]:
                new_r[x] -= 1
            row = row[:n // bs + 1]
        new_t.append(row + [-1] * (mb - len(row)))
        new_n.append(n)
        for la in range(layers):
            for h in range(hkv):
                m = min(L, room)
                if n == L:
                    src = list(range(m))
                else:
                    src = evicted(weights[la, b, h, :L].tolist(), positions[la, b, h, :L].tolist(), n, fixed, first, recent)[1]
                    for to, at in enumerate(src):
                        if to != at:
                            for x in (2 * la, 2 * la + 1):
                                pools[x][good[to // bs], to % bs, h] = pools[x][good[at // bs], at % bs, h]
                w[la, b, h, :len(src)] = weights[la, b, h][src]
                p[la, b, h, :len(src)] = positions[la, b, h][src]
    return new_t, new_n, new_r, w, p, pools


class Cache:
    def __init__(self, lens, bs, hkv, d, layers, fp8=False, seed=1, shared=0, room=None, extra=0, again=False, spread=2.0):
        g, rng = torch.Generator().manual_seed(seed), random.Random(seed)
        self.tables, self.refs, nb = layout(lens, bs, seed, shared=shared, extra=extra)
        self.lens, self.bs, self.rng = list(lens), bs, rng
        self.room = room or len(self.tables[0]) * bs
        dtype = torch.uint8 if fp8 else torch.int16   # (any bytes will do)
        self.pools = [torch.randint(0, 256 if fp8 else 30000, (nb, bs, hkv, d), generator=g).to(dtype) for _ in range(2 * layers)]
        shape = (layers, len(lens), hkv, self.room)
        self.weights = (torch.randn(*shape, generator=g) * spread).exp()
        pos = torch.arange(self.room).expand(shape).clone()
        if again:   # older tokens in no order, positions with gaps
            for x in pos.view(-1, self.room):
                x[:] = torch.cat((torch.randperm(self.room, generator=g), ))
            for b, n in enumerate(lens):
                tail = min(n, 9)
                pos[:, b, :, n - tail:n] = self.room + torch.arange(tail)
        self.positions = pos.int()
        self.fp8 = fp8

    def run(self, budget, first=0, recent=0, stream=None, twice=False):
        dev = lambda x: x.clone().cuda()   # noqa: E731
        pools = [dev(x) if self.fp8 else dev(x).view(torch.bfloat16) for x in self.pools]
        t, n, r = i32(self.tables), i32(self.lens), i32(self.refs)
        w, p = dev(self.weights), dev(self.positions)
        nt, nn, nr = torch.full_like(t, 77), torch.full_like(n, 77), torch.full_like(r, 77)
        nw, np_ = torch.full_like(w, 7.0), torch.full_like(p, 7)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()
        for _ in range(2 if twice else 1):
            pa.pa_cache_evict(nt, nn, nr, nw, np_, t, n, r, w, p, pa.PoolSet(pools), budget, first=first, recent=recent,
                              status=status, stream=stream)
        torch.cuda.synchronize()
        # the inputs are as they were
        assert torch.equal(w.cpu(), self.weights) or torch.equal(torch.isnan(w.cpu()), torch.isnan(self.weights))
        assert torch.equal(p.cpu(), self.positions) and t.tolist() == self.tables and n.tolist() == self.lens
        return nt.tolist(), nn.tolist(), nr.tolist(), nw.cpu(), np_.cpu(), \
            [x.cpu() if self.fp8 else x.view(torch.int16).cpu() for x in pools], status.item()

    def check(self, budget, first=0, recent=0, status=0, **kw):
        got = self.run(budget, first, recent, **kw)
        lens = [min(max(n, 0), len(self.tables[0]) * self.bs) for n in self.lens]
        odd = [b for b, n in enumerate(self.lens) if n != lens[b]]
        want = plain(self.tables, lens, self.refs, self.weights, self.positions, self.pools, self.bs, budget, first, recent,
                     self.room, odd)
        assert got[6] == status
        assert got[:3] == want[:3]
        for b, n in enumerate(want[1]):
            m = min(n, self.room)
            a, c = got[3][:, b, :, :m], want[3][:, b, :, :m]
            assert torch.equal(torch.isnan(a), torch.isnan(c)) and torch.equal(torch.nan_to_num(a), torch.nan_to_num(c))
            assert torch.equal(got[4][:, b, :, :m], want[4][:, b, :, :m])
            assert (got[3][:, b, :, m:] == 7.0).all() and (got[4][:, b, :, m:] == 7).all()
        for a, c in zip(got[5], want[5]):
            assert torch.equal(a, c)


@pytest.mark.gpu
@pytest.mark.parametrize("lens,bs,hkv,d,layers,fp8,budget,first,recent", [
    ([100, 64, 65, 0, 1], 16, 2, 64, 1, False, 64, 4, 8), ([100, 64, 65, 0, 1], 16, 2, 128, 2, True, 64, 0, 0),
    ([300, 1000, 77], 32, 3, 128, 1, False, 77, 0, 77), ([300, 1000, 77], 16, 1, 64, 3, True, 1, 0, 1),
    ([513], 256, 8, 128, 1, False, 300, 4, 100), ([4097, 2000], 16, 2, 64, 1, True, 1024, 4, 128),
    ([48, 48, 47], 48, 2, 128, 1, False, 47, 1, 1), ([2, 3], 16, 1, 128, 1, True, 2, 1, 1),
    ([9000], 16, 1, 64, 1, False, 8999, 0, 5), ([9000, 40], 16, 1, 64, 1, False, 3, 0, 0),
    ([20000], 16, 2, 64, 1, True, 777, 4, 32),
])
@pytest.mark.parametrize("again", [False, True])
def test_evict(lens, bs, hkv, d, layers, fp8, budget, first, recent, again):
    Cache(lens, bs, hkv, d, layers, fp8, seed=len(lens), again=again, extra=again).check(budget, first, recent)


@pytest.mark.gpu
@pytest.mark.parametrize("seed", range(4))
def test_evict_keeps_what_others_hold(seed):
    """A shared beginning, and a block in the middle that a prefix cache holds."""
    rng = random.Random(seed)
    c = Cache([rng.randint(100, 400) for _ in range(3)], 16, 2, 64, 1, seed=seed, shared=3)
    c.check(60, 2, 10)
    c.refs[c.tables[1][4 + seed]] += 1
    c.check(40, 2, 10)
    c.refs[c.tables[2][(c.lens[2] - 1) // 16]] += 1   # its last one: nothing of it goes
    c.check(40, 2, 10)


@pytest.mark.gpu
def test_evict_equal_nan_and_infinite_weights():
    for kind in range(5):
        c = Cache([500, 333, 1200], 16, 2, 64, 1, seed=kind, again=kind % 2)
        w = c.weights
        if kind == 0:
            w.zero_()
        elif kind == 1:
            w[..., ::3], w[..., 1::3], w[..., 2::3] = 0.5, 0.25, -0.0
            w[..., 5::7] = 0.0
        elif kind == 2:
            w[..., ::5] = math.nan
            w[..., 1::5] = math.inf
            w[..., 2::50] = -math.inf
        elif kind == 3:
            w[:] = 1e-42   # (below fp32's normal range)
            w[..., ::11] = 2e-42
        else:
            w.neg_()
        c.check(200, 4, 9)
        c.check(90, 0, 9)


@pytest.mark.gpu
def test_evict_next_tokens_block():
    """The block that a fork gave for the next token: kept with a sequence that stays, given back with one that is cut; a
    free block at that place is no one's."""
    c = Cache([64, 64, 64, 50], 16, 1, 64, 1, seed=3, extra=1)
    nb = len(c.refs)
    free = [x for x in range(nb) if c.refs[x] == 0]
    c.tables[0][4], c.refs[free[0]] = free[0], 1
    c.tables[1][4] = free[1]
    c.check(64, 0, 4)
    c.check(48, 0, 4)     # (48 is a multiple of the block size: entry 3 is the next token's)
    c.check(40, 0, 4)


@pytest.mark.gpu
def test_evict_leaves_rows_with_bad_blocks_and_lengths():
    c = Cache([200, 150, 180], 16, 2, 64, 1, seed=4)
    c.tables[0][3] = -1
    c.check(64, 4, 8, status=pa.PA_STATUS_BAD_BLOCK)
    c = Cache([200, 150, 180], 16, 2, 64, 1, seed=4)
    c.tables[1][2] = len(c.refs)
    c.refs[c.tables[2][0]] = 0
    c.check(64, 4, 8, status=pa.PA_STATUS_BAD_BLOCK)
    c = Cache([200, 150, 180], 16, 2, 64, 1, seed=4, room=190)
    c.check(64, 4, 8, status=pa.PA_STATUS_BAD_SEQLEN)
    c = Cache([200, 150, 208], 16, 2, 64, 1, seed=4)
    c.lens = [200, -3, 209]
    c.check(64, 4, 8, status=pa.PA_STATUS_BAD_SEQLEN)


@pytest.mark.gpu
def test_evict_twice_is_once_and_on_another_stream():
    c = Cache([300, 700], 16, 2, 128, 2, seed=5, again=True)
    c.check(128, 4, 9, twice=True)
    c.check(128, 4, 9, stream=torch.cuda.Stream())


@pytest.mark.gpu
@pytest.mark.parametrize("budget,first,recent", [(100000, 4, 30000), (50, 0, 1)])
def test_evict_from_the_most_tokens(budget, first, recent):
    Cache([196608], 256, 1, 64, 1, fp8=True, seed=8).check(budget, first, recent)


@pytest.mark.gpu
@pytest.mark.parametrize("spread", [0.0, 1e-6, 40.0])
def test_evict_weights_that_are_alike_or_far_apart(spread):
    """One value for all, a few neighbouring ones, and some that under- and overflow: the border among many keys."""
    Cache([5000, 1200, 300], 16, 2, 64, 1, seed=9, spread=spread).check(200, 2, 20)


@pytest.mark.gpu
def test_evict_with_plain_launches():
    prev = pa.pa_get_option(pa.PA_OPT_PDL)
    pa.pa_set_option(pa.PA_OPT_PDL, 0)
    try:
        Cache([300, 700, 20], 16, 2, 128, 2, seed=5, again=True).check(128, 4, 9, twice=True)
    finally:
        pa.pa_set_option(pa.PA_OPT_PDL, prev)


@pytest.mark.gpu
def test_evict_right_after_the_weights():
    """Weights and positions written by the kernel before, over and over: every call sees the last ones."""
    c = Cache([900, 500], 16, 2, 64, 1, seed=11)
    pools = [x.cuda().view(torch.bfloat16) for x in c.pools]
    t, n, r = i32(c.tables), i32(c.lens), i32(c.refs)
    w, p = torch.zeros_like(c.weights).cuda(), torch.zeros_like(c.positions).cuda()
    q, lse = torch.zeros(2, 900, 2, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(2, 900, 2, device="cuda")
    new = [torch.zeros_like(x) for x in (t, n, r, w, p)]
    got = []
    for i in range(40):
        lse.fill_(float(-i))   # (every query gives each token that it sees e^i)
        pa.pa_weights_add(w[0], w[0], p[0], q, lse, pools[0], t, n, 0.1)
        pa.pa_cache_evict(*new, t, n, r, w, p, pa.PoolSet([x.clone() for x in pools]), 100, 1, 3)
        got.append([x.clone() for x in (w, new[3], new[4])])
    torch.cuda.synchronize()
    for i, (before, weights, positions) in enumerate(got):
        for b, L in enumerate(c.lens):
            m = min(L, 100)
            # the earliest tokens are seen by the most queries: they, and the newest, stay in their order
            src = list(range(m - 3)) + list(range(L - 3, L))
            assert torch.equal(weights[0, b, :, :m], before[0, b][:, src]), i
            assert (positions[0, b, :, :m].cpu() == torch.tensor(src)).all(), i


@pytest.mark.gpu
def test_evict_many_rows():
    rng = random.Random(6)
    Cache([rng.randint(0, 300) for _ in range(70)], 16, 4, 64, 2, fp8=True, seed=6).check(100, 2, 20)


@pytest.mark.gpu
def test_evict_without_sequences():
    pool = [torch.zeros(9, 16, 1, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    z = lambda *s, t=torch.int32: torch.zeros(*s, dtype=t, device="cuda")   # noqa: E731
    refs, new = i32(list(range(9))), z(9)
    pa.pa_cache_evict(z(0, 4), z(0), new, z(1, 0, 1, 64, t=torch.float32), z(1, 0, 1, 64), z(0, 4), z(0), refs,
                      z(1, 0, 1, 64, t=torch.float32), z(1, 0, 1, 64), pa.PoolSet(pool), 4)
    assert torch.equal(new, refs)


@pytest.mark.gpu
def test_evict_in_a_graph():
    c = Cache([150, 99], 16, 2, 64, 1, seed=7)
    pools = [x.cuda().view(torch.bfloat16) for x in c.pools]
    t, n, r, w, p = i32(c.tables), i32(c.lens), i32(c.refs), c.weights.cuda(), c.positions.cuda()
    nt, nn, nr, nw, np_ = (torch.zeros_like(x) for x in (t, n, r, w, p))
    ps = pa.PoolSet(pools)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.pa_cache_evict(nt, nn, nr, nw, np_, t, n, r, w, p, ps, 64, first=2, recent=5)
    for lens in ([150, 99], [80, 64]):
        n.copy_(i32(lens))
        before = [x.view(torch.int16).cpu() for x in pools]
        graph.replay()
        torch.cuda.synchronize()
        want = plain(c.tables, lens, c.refs, c.weights, c.positions, before, 16, 64, 2, 5, c.room)
        # (blocks behind a shorter length are not the row's here: the table's rest is dropped, its counts stay)
        for b in range(2):
            assert nt[b].tolist()[:4] == want[0][b][:4] and nn[b].item() == want[1][b]
            m = want[1][b]
            assert torch.equal(nw[:, b, :, :m].cpu(), want[3][:, b, :, :m])
        for a, x in zip(pools, want[5]):
            assert torch.equal(a.view(torch.int16).cpu(), x)


FAKE = ctypes.c_void_p(1 << 20)  # aligned, never dereferenced: these calls fail validation first
OTHER = [ctypes.c_void_p((2 + i) << 20) for i in range(10)]


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), pa.PA_EINVAL), (dict(mb=0), pa.PA_EINVAL), (dict(room=0), pa.PA_EINVAL), (dict(budget=0), pa.PA_EINVAL),
    (dict(first=-1), pa.PA_EINVAL), (dict(recent=-1), pa.PA_EINVAL), (dict(first=40, recent=30), pa.PA_EINVAL),
    (dict(first=2 ** 31 - 1, recent=2 ** 31 - 1), pa.PA_EINVAL), (dict(elem=0), pa.PA_EINVAL), (dict(n_pools=1), pa.PA_EINVAL),
    (dict(n_pools=0), pa.PA_EINVAL), (dict(n_pools=258), pa.PA_EUNSUPPORTED), (dict(weights=None), pa.PA_EINVAL),
    (dict(weights=OTHER[3]), pa.PA_EINVAL), (dict(tables=OTHER[0]), pa.PA_EINVAL), (dict(refs=OTHER[2]), pa.PA_EINVAL),
    (dict(weights=(1 << 24) + 2), pa.PA_EINVAL), (dict(desc=pa.CacheDesc(64, 16, 2, 96)), pa.PA_EUNSUPPORTED),
    (dict(mb=1 << 27), pa.PA_EUNSUPPORTED), (dict(mb=1 << 14, room=1 << 18), pa.PA_EUNSUPPORTED), (dict(B=70000), pa.PA_EUNSUPPORTED),
])
def test_evict_refusals(kw, code):
    a = dict(tables=OTHER[5], refs=OTHER[7], weights=OTHER[8], room=100, B=4, mb=7, n_pools=2, elem=2,
             desc=pa.CacheDesc(64, 16, 2, 128), budget=60, first=4, recent=8) | kw
    pools = (ctypes.c_void_p * 300)(*[1 << 20] * 300)
    assert pa.lib().pa_cache_evict(*OTHER[:5], a["tables"], OTHER[6], a["refs"], a["weights"], OTHER[9], a["room"], a["B"],
                                   a["mb"], pools, a["n_pools"], a["elem"], a["desc"], a["budget"], a["first"], a["recent"],
                                   None, None) == code


@pytest.mark.gpu
def test_evict_wrapper_refuses():
    z = lambda *s, t=torch.int32: torch.zeros(*s, dtype=t, device="cuda")   # noqa: E731
    pool = [torch.zeros(9, 16, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    f = torch.float32
    ok = dict(nt=z(3, 4), nn=z(3), nr=z(9), nw=z(1, 3, 2, 64, t=f), np=z(1, 3, 2, 64), t=z(3, 4), n=z(3), r=z(9),
              w=z(1, 3, 2, 64, t=f), p=z(1, 3, 2, 64), pools=pa.PoolSet(pool))
    names = list(ok)
    for kw in (dict(nt=z(3, 5)), dict(nr=z(8)), dict(w=z(3, 2, 64, t=f)), dict(nw=z(1, 3, 2, 63, t=f)), dict(p=z(2, 3, 2, 64)),
               dict(w=z(1, 3, 1, 64, t=f)), dict(pools=pa.PoolSet(pool + pool)), dict(pools=pool), dict(n=z(4)),
               dict(w=z(1, 3, 2, 64))):
        with pytest.raises((TypeError, ValueError)):
            pa.pa_cache_evict(*[(ok | kw)[x] for x in names], 32)
    with pytest.raises(pa.PAError) as e:
        pa.pa_cache_evict(*[ok[x] for x in names], 32, first=30, recent=3)
    assert e.value.code == pa.PA_EINVAL
