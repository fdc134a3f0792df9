"""Page operators (pa_sequences_fork, pa_blocks_compact, pa_blocks_copy) against a plain Python
model of the pages.  Everything is whole numbers and copied bytes: equality throughout."""
import ctypes
import random

import pytest
import torch

from paged_kv_decode_cache_gb300 import build as B
from paged_kv_decode_cache_gb300 import pa


@pytest.fixture(scope="module", autouse=True)
def _built():
    B.build()


# ---- the plain model -------------------------------------------------------------------------


def plain_fork(tables, lens, refs, parents, bs, mb):
    """(new tables, lens, refs, slots, copies as (source, destination, rows), whether blocks ran out)."""
    refs = list(refs)
    for row, length in zip(tables, lens):
        for x in row[:-(-length // bs)]:
            refs[x] -= 1
    new = [list(tables[p][:-(-lens[p] // bs)]) if p >= 0 else None for p in parents]
    for row in new:
        for x in row or ():
            refs[x] += 1
    length = [lens[p] if p >= 0 else 0 for p in parents]
    tails = {}
    for i, row in enumerate(new):
        if row is not None and length[i] % bs:
            tails.setdefault(row[-1], []).append(i)
    free = [x for x, n in enumerate(refs) if n == 0]
    slots, copies, ran_out = [], [], False
    shared = {t: (refs[t] == len(rows), rows[0]) for t, rows in tails.items()}
    for i, row in enumerate(new):
        off = length[i] % bs
        if row is None:
            slots.append(-1)
            continue
        if off and shared[row[-1]] == (True, i):
            slots.append(row[-1] * bs + off)
            continue
        if not off and len(row) == mb:
            slots.append(-1)
            continue
        if not free:
            ran_out = True
            slots.append(-1)
            continue
        x = free.pop(0)
        refs[x] = 1
        if off:
            refs[row[-1]] -= 1
            copies.append((row[-1], x, off))
            row[-1] = x
        else:
            row.append(x)
        slots.append(x * bs + off)
    return [(row or []) + [-1] * (mb - len(row or [])) for row in new], length, refs, slots, copies, ran_out


def plain_compact(tables, lens, refs, bs):
    n = sum(x != 0 for x in refs)
    holes = iter([i for i in range(n) if refs[i] == 0])
    remap = [-1 if r == 0 else i if i < n else next(holes) for i, r in enumerate(refs)]
    now = [0] * len(refs)
    for i, r in enumerate(refs):
        if r:
            now[remap[i]] = r
    used = [-(-x // bs) for x in lens]
    return [[remap[x] for x in row[:u]] + [-1] * (len(row) - u) for row, u in zip(tables, used)], now, remap, n


def random_state(rng, rows, bs, mb, spare, prefixes=3):
    """Sequences of which some share their first blocks, some end with a full block, some are
    empty, and blocks that a prefix cache holds."""
    at, shared, tables, lens, held = 0, [], [], [], []
    for _ in range(prefixes):
        n = rng.randint(0, mb - 1)
        shared.append(list(range(at, at + n)))
        held += shared[-1] if rng.random() < 0.5 else []
        at += n
    for _ in range(rows):
        start = rng.choice(shared)
        used = rng.randint(len(start), mb)
        row = start + list(range(at, at + used - len(start)))
        at += used - len(start)
        last = rng.choice([0, 0, rng.randrange(bs)]) if used > 0 else 0
        lens.append(max(0, used * bs - last))
        tables.append(row)
    nb = max(1, at + spare)   # (a pool has a block)
    ids = list(range(nb))
    rng.shuffle(ids)
    refs = [0] * nb
    for x in [x for row in tables for x in row] + held:
        refs[ids[x]] += 1
    return [[ids[x] for x in row] + [-1] * (mb - len(row)) for row in tables], lens, refs


def dev(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device="cuda")


def make_pools(n, nb, bs, hkv, d, fp8, seed):
    g = torch.Generator().manual_seed(seed)
    out = [torch.randint(0, 256, (nb, bs, hkv, d * (1 if fp8 else 2)), generator=g, dtype=torch.uint8).cuda()
           for _ in range(n)]
    return out if fp8 else [t.view(torch.bfloat16) for t in out]


def run_fork(tables, lens, refs, parents, bs, mb, pools, stream=None, capture=False):
    nb, n = len(refs), len(parents)
    new = [torch.full((n, mb), 77, dtype=torch.int32, device="cuda"), dev([77] * n), dev([77] * nb),
           dev([77] * n, torch.int64)]
    status, ps = dev([0]), pa.PoolSet(pools)
    ws = torch.full((pa.pa_fork_workspace_bytes(len(lens), n, nb),), 255, dtype=torch.uint8, device="cuda")
    old = [dev(tables).view(len(lens), mb), dev(lens), dev(refs), dev(parents)]
    call = lambda: pa.pa_sequences_fork(*new, *old, ps, ws, status=status, stream=stream)  # noqa: E731
    if capture:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        g.replay()
    else:
        torch.cuda.synchronize()
        call()
    torch.cuda.synchronize()
    return [t.cpu().tolist() for t in new], status.item()


# ---- on the GPU ------------------------------------------------------------------------------


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("rows,new_rows,bs,mb,hkv,d,n_pools", [
    (1, 1, 16, 1, 1, 64, 1), (4, 4, 16, 9, 2, 128, 2), (5, 17, 32, 4, 3, 64, 3), (64, 40, 256, 3, 1, 128, 2),
    (300, 1100, 16, 40, 1, 64, 4),
])
def test_fork_matches_the_model(rows, new_rows, bs, mb, hkv, d, n_pools, fp8):
    rng = random.Random(rows * 1000 + mb)
    for trial in range(3):
        tables, lens, refs = random_state(rng, rows, bs, mb, spare=new_rows + 5)
        parents = [rng.choice([-1, rng.randrange(rows), rng.randrange(rows), 0]) for _ in range(new_rows)]
        if trial == 2:  # every row keeps its place
            parents = [i % rows for i in range(new_rows)]
        pools = make_pools(n_pools, len(refs), bs, hkv, d, fp8, trial)
        before = [t.clone() for t in pools]
        got, status = run_fork(tables, lens, refs, parents, bs, mb, pools)
        want = plain_fork(tables, lens, refs, parents, bs, mb)
        full = any(p >= 0 and lens[p] == mb * bs for p in parents)
        assert status == (pa.PA_STATUS_BAD_SEQLEN if full else 0)
        assert not want[5]
        assert got == [want[0], want[1], want[2], want[3]]
        for pool, old in zip(pools, before):
            for src, dst, n in want[4]:
                old[dst, :n] = old[src, :n]
            assert torch.equal(pool.view(torch.uint8), old.view(torch.uint8))


@pytest.mark.gpu
def test_fork_when_blocks_run_out():
    bs, mb = 16, 4
    tables, lens, refs = [[0, 1, -1, -1]], [20], [1, 1, 0]
    pools = make_pools(1, 3, bs, 1, 64, False, 1)
    got, status = run_fork(tables, lens, refs, [0, 0, 0], bs, mb, pools)
    want = plain_fork(tables, lens, refs, [0, 0, 0], bs, mb)
    assert want[5] and status == pa.PA_STATUS_NO_BLOCKS
    assert got == list(want[:4])
    assert got[3] == [20, 2 * 16 + 4, -1] and got[2] == [3, 2, 1]


@pytest.mark.gpu
def test_fork_frees_everything_and_takes_no_rows():
    bs, mb = 16, 3
    tables, lens, refs = random_state(random.Random(4), 6, bs, mb, 3)
    pools = make_pools(2, len(refs), bs, 1, 64, False, 1)
    for parents in ([], [-1, -5]):
        got, status = run_fork(tables, lens, refs, parents, bs, mb, pools)
        assert status == 0 and got == list(plain_fork(tables, lens, refs, parents, bs, mb)[:4])


@pytest.mark.gpu
def test_fork_shared_partial_block_that_another_row_has_filled():
    """A partial last block that a longer sequence goes on with is never written in place."""
    bs, mb = 16, 4
    tables, lens, refs = [[5, 3, -1, -1], [5, 3, 1, -1]], [20, 40], [0, 1, 0, 2, 0, 2]
    got, status = run_fork(tables, lens, refs, [0, 1], bs, mb, make_pools(1, 6, bs, 1, 64, False, 2))
    assert status == 0
    assert got[0] == [[5, 0, -1, -1], [5, 3, 1, -1]] and got[3] == [4, 1 * 16 + 8] and got[2] == [1, 1, 0, 1, 0, 2]


@pytest.mark.gpu
def test_fork_reports_bad_parents_blocks_and_lengths():
    bs, mb = 16, 3
    pools = make_pools(1, 4, bs, 1, 64, False, 3)
    got, status = run_fork([[0, 1, -1]], [20], [1, 1, 0, 0], [0, 1], bs, mb, pools)
    assert status == pa.PA_STATUS_BAD_PARENT and got[1] == [20, 0] and got[3] == [20, -1]
    got, status = run_fork([[0, 9, -1]], [20], [1, 0, 0, 0], [0, 0], bs, mb, pools)
    assert status == pa.PA_STATUS_BAD_BLOCK and got[0] == [[0, -1, -1]] * 2 and got[3] == [-1, -1]
    got, status = run_fork([[0, 1, 2]], [999], [1, 1, 1, 0], [0], bs, mb, pools)
    assert status == pa.PA_STATUS_BAD_SEQLEN and got[1] == [48] and got[3] == [-1]
    got, status = run_fork([[0, 1, 2]], [-4], [0, 0, 0, 0], [0], bs, mb, pools)
    assert status == pa.PA_STATUS_BAD_SEQLEN and got[1] == [0] and got[0] == [[0, -1, -1]] and got[3] == [0]


@pytest.mark.gpu
def test_fork_in_a_graph_and_on_another_stream():
    rng = random.Random(8)
    bs, mb = 16, 20
    tables, lens, refs = random_state(rng, 16, bs, mb, 40)
    parents = [rng.randrange(16) for _ in range(16)]
    want = list(plain_fork(tables, lens, refs, parents, bs, mb)[:4])
    pools = make_pools(2, len(refs), bs, 2, 64, False, 1)
    assert run_fork(tables, lens, refs, parents, bs, mb, pools, capture=True)[0] == want
    assert run_fork(tables, lens, refs, parents, bs, mb, pools, stream=torch.cuda.Stream())[0] == want


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("rows,bs,mb,spare,hkv,d,n_pools", [
    (1, 16, 1, 0, 1, 64, 1), (3, 16, 5, 40, 2, 64, 2), (40, 32, 9, 700, 1, 128, 3), (200, 16, 60, 9000, 1, 64, 2),
    (4, 256, 3, 30, 4, 128, 1),
])
def test_compact_matches_the_model(rows, bs, mb, spare, hkv, d, n_pools, fp8):
    rng = random.Random(rows + spare)
    for trial in range(2):
        tables, lens, refs = random_state(rng, rows, bs, mb, spare)
        nb = len(refs)
        if trial:  # nothing is live
            tables, lens, refs = [[-1] * mb] * rows, [0] * rows, [0] * nb
        pools = make_pools(n_pools, nb, bs, hkv, d, fp8, trial)
        before = [t.clone() for t in pools]
        new = [torch.full((rows, mb), 77, dtype=torch.int32, device="cuda"), dev([77] * nb), dev([77] * nb), dev([77])]
        status = dev([0])
        ws = torch.full((pa.pa_compact_workspace_bytes(nb),), 255, dtype=torch.uint8, device="cuda")
        pa.pa_blocks_compact(*new, dev(tables), dev(lens), dev(refs), pa.PoolSet(pools), ws, status=status)
        torch.cuda.synchronize()
        want = plain_compact(tables, lens, refs, bs)
        assert status.item() == 0
        assert [t.cpu().tolist() for t in new] == [want[0], want[1], want[2], [want[3]]]
        for pool, old in zip(pools, before):
            for i, to in enumerate(want[2]):
                if to >= 0 and to != i:
                    old[to] = old[i]
            assert torch.equal(pool.view(torch.uint8), old.view(torch.uint8))


@pytest.mark.gpu
@pytest.mark.parametrize("nb", [1, 2, 255, 256, 257, 2047, 2048, 2049, 5001])
@pytest.mark.parametrize("live", ["every", "odd", "upper half", "lower half", "last", "some"])
def test_compact_at_pool_sizes(nb, live):
    """Counts of every pattern, tables of single blocks that name some of the live ones."""
    rng = random.Random(nb)
    pick = {"every": lambda i: True, "odd": lambda i: i % 2, "upper half": lambda i: i >= nb // 2,
            "lower half": lambda i: i < nb // 2, "last": lambda i: i == nb - 1, "some": lambda i: rng.random() < 0.4}[live]
    refs = [rng.randint(1, 3) if pick(i) else 0 for i in range(nb)]
    ids = [i for i in range(nb) if refs[i]][-7:]
    tables, lens = [[i] for i in ids] + [[-1]], [16 - rng.randrange(16) for _ in ids] + [0]
    pools = make_pools(2, nb, 16, 1, 64, True, nb)
    before = [t.clone() for t in pools]
    new = [torch.full((len(lens), 1), 77, dtype=torch.int32, device="cuda"), dev([77] * nb), dev([77] * nb), dev([77])]
    status = dev([0])
    ws = torch.full((pa.pa_compact_workspace_bytes(nb),), 255, dtype=torch.uint8, device="cuda")
    pa.pa_blocks_compact(*new, dev(tables), dev(lens), dev(refs), pa.PoolSet(pools), ws, status=status)
    torch.cuda.synchronize()
    want = plain_compact(tables, lens, refs, 16)
    assert status.item() == 0
    assert [t.cpu().tolist() for t in new] == [want[0], want[1], want[2], [want[3]]]
    moved = [i for i, to in enumerate(want[2]) if to >= 0 and to != i]
    for pool, old in zip(pools, before):
        if moved:
            old[[want[2][i] for i in moved]] = old[moved]
        assert torch.equal(pool, old)


@pytest.mark.gpu
def test_compact_reports_entries_that_name_no_live_block():
    new = [dev([[7, 7]]), dev([7, 7, 7]), dev([7, 7, 7]), dev([7])]
    status = dev([0])
    ws = torch.empty(pa.pa_compact_workspace_bytes(3), dtype=torch.uint8, device="cuda")
    pools = pa.PoolSet(make_pools(1, 3, 16, 1, 64, False, 1))
    pa.pa_blocks_compact(*new, dev([[2, 1]]), dev([32]), dev([0, 0, 1]), pools, ws, status=status)
    torch.cuda.synchronize()
    assert status.item() == pa.PA_STATUS_BAD_BLOCK
    assert [t.cpu().tolist() for t in new] == [[[0, -1]], [1, 0, 0], [-1, -1, 0], [1]]


@pytest.mark.gpu
@pytest.mark.parametrize("bs,hkv,d,fp8", [(16, 1, 64, True), (16, 3, 128, False), (256, 8, 128, False)])
def test_copy_blocks(bs, hkv, d, fp8):
    pools = make_pools(3, 12, bs, hkv, d, fp8, 5)
    before = [t.clone() for t in pools]
    status = dev([0])
    pa.pa_blocks_copy(pa.PoolSet(pools), dev([[3, 0], [-1, 4], [3, 11], [7, 2]]), status=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    for pool, old in zip(pools, before):
        old[0], old[11], old[2] = old[3], old[3], old[7]
        assert torch.equal(pool.view(torch.uint8), old.view(torch.uint8))
    pa.pa_blocks_copy(pa.PoolSet(pools), dev([[3, 12], [12, 3], [1, -1]]), status=status)
    torch.cuda.synchronize()
    assert status.item() == pa.PA_STATUS_BAD_BLOCK
    assert all(torch.equal(p.view(torch.uint8), o.view(torch.uint8)) for p, o in zip(pools, before))


@pytest.mark.gpu
def test_pool_set_refuses():
    pools = make_pools(2, 4, 16, 1, 64, False, 1)
    with pytest.raises(ValueError):
        pa.PoolSet([])
    with pytest.raises(TypeError):
        pa.PoolSet([pools[0].float()])
    with pytest.raises(TypeError):
        pa.PoolSet([pools[0], pools[1].view(torch.uint8)])
    with pytest.raises(ValueError):
        pa.PoolSet([pools[0], pools[1][:3]])
    with pytest.raises(ValueError):
        pa.PoolSet([p.cpu() for p in pools])
    with pytest.raises(TypeError):
        pa.pa_blocks_copy(pools, dev([[0, 1]]))


# ---- refusals (host only) --------------------------------------------------------------------

FAKE = ctypes.c_void_p(1 << 20)    # aligned, never dereferenced: these calls fail validation first
OTHER = [ctypes.c_void_p((1 << 20) + 4096 * i) for i in range(1, 9)]
POOLS = (ctypes.c_void_p * 2)(1 << 21, 1 << 22)
DESC = pa.CacheDesc(64, 16, 2, 64)


@pytest.mark.parametrize("kw,code", [
    (dict(B_old=-1), pa.PA_EINVAL), (dict(B_new=-1), pa.PA_EINVAL), (dict(B_new=4097), pa.PA_EUNSUPPORTED),
    (dict(mb=0), pa.PA_EINVAL), (dict(mb=1 << 28), pa.PA_EUNSUPPORTED), (dict(tables=None), pa.PA_EINVAL),
    (dict(parents=None), pa.PA_EINVAL), (dict(slots=None), pa.PA_EINVAL), (dict(refs=None), pa.PA_EINVAL),
    (dict(new_refs=OTHER[6]), pa.PA_EINVAL), (dict(new_tables=OTHER[4]), pa.PA_EINVAL),
    (dict(slots=ctypes.c_void_p((1 << 20) + 4)), pa.PA_EINVAL), (dict(lens=ctypes.c_void_p((1 << 20) + 2)), pa.PA_EINVAL),
    (dict(n_pools=-1), pa.PA_EINVAL), (dict(n_pools=257), pa.PA_EUNSUPPORTED), (dict(pools=None), pa.PA_EINVAL),
    (dict(pools=(ctypes.c_void_p * 2)(1 << 21, (1 << 22) + 8)), pa.PA_EINVAL), (dict(elem=4), pa.PA_EINVAL),
    (dict(desc=pa.CacheDesc(64, 8, 2, 64)), pa.PA_EUNSUPPORTED), (dict(desc=pa.CacheDesc(-1, 16, 2, 64)), pa.PA_EINVAL),
    (dict(ws=None), pa.PA_EWORKSPACE), (dict(ws_bytes=100), pa.PA_EWORKSPACE),
    (dict(ws=ctypes.c_void_p((1 << 20) + 16)), pa.PA_EWORKSPACE),
])
def test_fork_refusals(kw, code):
    a = dict(new_tables=OTHER[0], new_lens=OTHER[1], new_refs=OTHER[2], slots=OTHER[3], tables=OTHER[4], lens=OTHER[5],
             refs=OTHER[6], parents=OTHER[7], B_old=3, B_new=3, mb=4, pools=POOLS, n_pools=2, elem=2, desc=DESC,
             ws=FAKE, ws_bytes=pa.pa_fork_workspace_bytes(3, 3, 64))
    a.update(kw)
    assert pa.lib().pa_sequences_fork(*a.values(), None, None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), pa.PA_EINVAL), (dict(mb=0), pa.PA_EINVAL), (dict(mb=1 << 28), pa.PA_EUNSUPPORTED),
    (dict(tables=None), pa.PA_EINVAL), (dict(remap=None), pa.PA_EINVAL), (dict(n_live=None), pa.PA_EINVAL),
    (dict(new_refs=OTHER[6]), pa.PA_EINVAL), (dict(remap=OTHER[1]), pa.PA_EINVAL), (dict(elem=0), pa.PA_EINVAL),
    (dict(n_pools=300), pa.PA_EUNSUPPORTED), (dict(ws=None), pa.PA_EWORKSPACE), (dict(ws_bytes=0), pa.PA_EWORKSPACE),
])
def test_compact_refusals(kw, code):
    a = dict(new_tables=OTHER[0], new_refs=OTHER[1], remap=OTHER[2], n_live=OTHER[3], tables=OTHER[4], lens=OTHER[5],
             refs=OTHER[6], B=3, mb=4, pools=POOLS, n_pools=2, elem=2, desc=DESC, ws=FAKE,
             ws_bytes=pa.pa_compact_workspace_bytes(64))
    a.update(kw)
    assert pa.lib().pa_blocks_compact(*a.values(), None, None) == code


def test_copy_refusals_and_workspace_sizes():
    L = pa.lib()
    assert L.pa_blocks_copy(POOLS, 2, 2, DESC, None, 3, None, None) == pa.PA_EINVAL
    assert L.pa_blocks_copy(POOLS, 2, 2, DESC, ctypes.c_void_p((1 << 20) + 4), 3, None, None) == pa.PA_EINVAL
    assert L.pa_blocks_copy(POOLS, 2, 3, DESC, FAKE, 3, None, None) == pa.PA_EINVAL
    assert L.pa_blocks_copy(POOLS, 2, 2, DESC, FAKE, -3, None, None) == pa.PA_EINVAL
    assert L.pa_blocks_copy(POOLS, 2, 2, DESC, None, 0, None, None) == pa.PA_OK
    assert pa.pa_fork_workspace_bytes(-1, 1, 1) == 0 and pa.pa_compact_workspace_bytes(0) == 0
    assert pa.pa_fork_workspace_bytes(4, 4, 1000) >= 2 * 4 * 1000 + 16 * 4
    assert pa.pa_compact_workspace_bytes(1000) >= 20 * 1000
