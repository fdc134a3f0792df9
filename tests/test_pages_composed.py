"""Page operators after one another: a fork of what a fork has just made, and tokens written in between or not.

A row whose length is a multiple of the block size holds, at entry length / bs of its table, the block
that a fork gave it for its next token.  The model counts that entry as the row's own."""
import ctypes
import random

import pytest
import torch

from paged_kv_decode_cache_gb300 import pa
from test_pages import DESC, FAKE, OTHER, POOLS, _built, dev, make_pools, run_fork  # noqa: F401


def blocks_of(row, length, refs, bs):
    """A row's blocks: those of its tokens, and the one that waits for the next token."""
    n = -(-length // bs)
    if length % bs == 0 and n < len(row) and 0 <= row[n] < len(refs) and refs[row[n]] > 0:
        n += 1
    return list(row[:n])


def plain_fork(tables, lens, refs, parents, bs, mb):
    """(new tables, lens, refs, slots, copies)."""
    old = [blocks_of(row, n, refs, bs) for row, n in zip(tables, lens)]
    refs = list(refs)
    for row in old:
        for x in row:
            refs[x] -= 1
    new = [list(old[p]) if p >= 0 else None for p in parents]
    for row in new:
        for x in row or ():
            refs[x] += 1
    length = [lens[p] if p >= 0 else 0 for p in parents]
    last = [row[n // bs] if row is not None and n // bs < len(row) else None for row, n in zip(new, length)]
    keeps = {x: refs[x] == last.count(x) and last.index(x) for x in last if x is not None}
    free = [x for x, n in enumerate(refs) if n == 0]
    slots, copies = [], []
    for i, row in enumerate(new):
        off, x = length[i] % bs, last[i]
        if row is None or (x is None and len(row) == mb):
            slots.append(-1)
            continue
        if x is None or not (keeps[x] is not False and keeps[x] == i):
            if not free:
                slots.append(-1)
                continue
            own = free.pop(0)
            refs[own] = 1
            if x is None:
                row.append(own)
            else:
                refs[x] -= 1
                row[-1] = own
                if off:
                    copies.append((x, own, off))
            x = own
        slots.append(x * bs + off)
    return [(row or []) + [-1] * (mb - len(row or [])) for row in new], length, refs, slots, copies


def counts(tables, nb, held=()):
    refs = [0] * nb
    for x in [x for row in tables for x in row if x >= 0] + list(held):
        refs[x] += 1
    return refs


@pytest.mark.gpu
def test_fork_after_fork_keeps_the_fresh_block():
    """16 tokens of 16 per block: the block of the 17th is given once, however often the row is forked."""
    bs, mb = 16, 3
    pools = make_pools(1, 4, bs, 1, 64, False, 1)
    tables, lens, refs = [[2, -1, -1]], [16], [0, 0, 1, 0]
    for _ in range(5):
        (tables, lens, refs, slots), status = run_fork(tables, lens, refs, [0], bs, mb, pools)
        assert status == 0 and tables == [[2, 0, -1]] and refs == [1, 0, 1, 0] and slots == [0] and lens == [16]
    # two children: the first keeps it, the other gets one of its own; then both are dropped
    (tables, lens, refs, slots), status = run_fork(tables, lens, refs, [0, 0], bs, mb, pools)
    assert status == 0 and tables == [[2, 0, -1], [2, 1, -1]] and refs == [1, 1, 2, 0] and slots == [0, 16]
    (tables, lens, refs, slots), status = run_fork(tables, lens, refs, [-1, -1], bs, mb, pools)
    assert status == 0 and refs == [0, 0, 0, 0] and slots == [-1, -1]


@pytest.mark.gpu
def test_fork_when_the_fresh_block_cannot_be_replaced():
    """No block left for the second child: it goes on sharing, without a slot, and nothing is lost."""
    bs, mb = 16, 2
    pools = make_pools(1, 2, bs, 1, 64, False, 1)
    (tables, lens, refs, slots), status = run_fork([[1, 0]], [16], [1, 1], [0, 0], bs, mb, pools)
    assert status == pa.PA_STATUS_NO_BLOCKS
    assert tables == [[1, 0], [1, 0]] and refs == [2, 2] and slots == [0, -1]
    (tables, lens, refs, slots), status = run_fork(tables, lens, refs, [0], bs, mb, pools)
    assert status == 0 and tables == [[1, 0]] and refs == [1, 1] and slots == [0]


@pytest.mark.gpu
def test_entries_that_name_no_held_block_are_not_taken():
    """Past its tokens a row's entry counts only where it names a block in use."""
    bs, mb = 16, 3
    pools = make_pools(1, 4, bs, 1, 64, False, 1)
    for junk in (-1, -7, 1, 4, 1 << 30):       # (1: free)
        (tables, lens, refs, slots), status = run_fork([[2, junk, 3]], [16], [0, 0, 1, 1], [0], bs, mb, pools)
        assert status == 0 and tables == [[2, 0, -1]] and refs == [1, 0, 1, 1] and slots == [0]
    (tables, lens, refs, slots), status = run_fork([[2, 1, 0]], [48], [1, 1, 1, 0], [0], bs, mb, pools)
    assert status == pa.PA_STATUS_BAD_SEQLEN and tables == [[2, 1, 0]] and refs == [1, 1, 1, 0] and slots == [-1]


@pytest.mark.gpu
@pytest.mark.parametrize("rows,bs,mb,spare", [(3, 16, 4, 20), (12, 16, 9, 40), (70, 32, 6, 300), (100, 16, 100, 1000)])
def test_chains_of_forks_lose_nothing(rows, bs, mb, spare):
    """Forks in a row, in which some tokens are written and some are not: the model's state after
    every one, counts that are the tables' own, and the sequences' contents."""
    rng = random.Random(rows)
    nb = rows * mb + spare
    pools = make_pools(1, nb, bs, 1, 64, False, rows)
    pool = pools[0]
    held = [rng.randrange(nb)]
    tables, lens, refs = [[-1] * mb for _ in range(rows)], [0] * rows, counts([], nb, held)
    texts = [[] for _ in range(rows)]
    alive = list(range(rows))
    slots = [-1] * rows
    parents = alive
    at = 0
    for step in range(24):
        want = plain_fork(tables, lens, refs, parents, bs, mb)
        (tables, lens, refs, slots), status = run_fork(tables, lens, refs, parents, bs, mb, pools)
        assert (tables, lens, refs, slots) == want[:4]
        full = any(n == mb * bs for n in lens)
        assert status == (pa.PA_STATUS_BAD_SEQLEN if full else 0)
        assert refs == counts(tables, nb, held)
        texts = [list(texts[p]) if p >= 0 else [] for p in parents]
        flat = pool.view(nb * bs, 64)
        for i in range(rows):
            if texts[i]:
                where = [tables[i][t // bs] * bs + t % bs for t in range(len(texts[i]))]
                assert flat[where][:, 0].float().tolist() == texts[i]
        for i in range(rows):       # the tokens of this step, of some rows
            if parents[i] >= 0 and slots[i] >= 0 and rng.random() < 0.7:
                for _ in range(rng.choice([1, 1, bs - 1])):   # (within the block that the slot is in)
                    if lens[i] % bs == 0 and lens[i] // bs != tables[i].index(slots[i] // bs):
                        break
                    at = at % 199 + 1
                    flat[tables[i][lens[i] // bs] * bs + lens[i] % bs] = float(at)
                    texts[i].append(float(at))
                    lens[i] += 1
                    if lens[i] % bs == 0:
                        break
        parents = [rng.choice([-1, rng.randrange(rows), i, i, i]) if step % 5 else i for i in range(rows)]


# ---- compaction between two steps ------------------------------------------------------------


def plain_compact(tables, lens, refs, slots, bs):
    """(new tables, counts, remap, live blocks, slots)."""
    n = sum(x != 0 for x in refs)
    holes = iter([i for i in range(n) if refs[i] == 0])
    remap = [-1 if r == 0 else i if i < n else next(holes) for i, r in enumerate(refs)]
    now = [0] * len(refs)
    for i, r in enumerate(refs):
        if r:
            now[remap[i]] = r
    rows = [[remap[x] for x in blocks_of(row, length, refs, bs)] for row, length in zip(tables, lens)]
    moved = [-1 if s < 0 else remap[s // bs] * bs + s % bs for s in slots]
    return [row + [-1] * (len(tables[0]) - len(row)) for row in rows], now, remap, n, moved


def run_compact(tables, lens, refs, bs, pools, slots=None):
    nb, rows = len(refs), len(lens)
    new = [torch.full((rows, len(tables[0])), 77, dtype=torch.int32, device="cuda"), dev([77] * nb), dev([77] * nb), dev([77])]
    status = dev([0])
    ws = torch.full((pa.pa_compact_workspace_bytes(nb),), 255, dtype=torch.uint8, device="cuda")
    kw = {}
    if slots is not None:
        kw = dict(slots=dev(slots, torch.int64), new_slots=dev([77] * rows, torch.int64))
    pa.pa_blocks_compact(*new, dev(tables), dev(lens), dev(refs), pa.PoolSet(pools), ws, status=status, **kw)
    torch.cuda.synchronize()
    out = [t.cpu().tolist() for t in new]
    out[3] = out[3][0]
    return out + ([kw["new_slots"].cpu().tolist()] if kw else []), status.item()


@pytest.mark.gpu
@pytest.mark.parametrize("nb", [6, 3000])
def test_compact_keeps_the_fresh_block(nb):
    """The block for the 17th token moves with its row, before that token is written."""
    bs, mb = 16, 3
    pools = make_pools(2, nb, bs, 1, 64, False, 1)
    refs = [0] * nb
    refs[2] = refs[nb - 1] = 1
    got, status = run_compact([[2, nb - 1, -1]], [16], refs, bs, pools, slots=[(nb - 1) * bs])
    assert status == 0 and got[0] == [[0, 1, -1]] and got[4] == [bs]
    assert got[1][:3] == [1, 1, 0] and got[3] == 2 and got[2][2] == 0 and got[2][nb - 1] == 1


@pytest.mark.gpu
@pytest.mark.parametrize("nb", [6, 3000])
def test_slots_of_blocks_that_are_not_held_are_reported(nb):
    bs = 16
    pools = make_pools(1, nb, bs, 1, 64, False, 1)
    refs = [0] * nb
    refs[2] = refs[4] = 1
    tables = [[4, -1], [2, -1], [2, -1], [2, -1]]
    got, status = run_compact(tables, [10, 16, 16, 16], refs, bs, pools, slots=[4 * bs + 10, -5, 5 * bs, nb * bs])
    assert status == pa.PA_STATUS_BAD_SLOT
    assert got[4] == [bs + 10, -1, -1, -1] and got[0] == [[1, -1], [0, -1], [0, -1], [0, -1]]


@pytest.mark.gpu
@pytest.mark.parametrize("rows,bs,mb,spare", [(3, 16, 4, 20), (12, 16, 9, 40), (40, 32, 6, 3000)])
def test_servers_that_tidy_between_steps(rows, bs, mb, spare):
    """Forks, compactions and writes in turn, the model's state after each, and the sequences' contents."""
    rng = random.Random(rows)
    nb = rows * mb + spare
    pools = make_pools(2, nb, bs, 1, 64, False, rows)
    tables, lens, refs = [[-1] * mb for _ in range(rows)], [0] * rows, [0] * nb
    texts, parents, at = [[] for _ in range(rows)], list(range(rows)), 0
    for step in range(16):
        (tables, lens, refs, slots), _ = run_fork(tables, lens, refs, parents, bs, mb, pools)
        texts = [list(texts[p]) if p >= 0 else [] for p in parents]
        if step % 3 != 1:
            want = plain_compact(tables, lens, refs, slots, bs)
            got, status = run_compact(tables, lens, refs, bs, pools, slots=slots)
            assert status == 0 and got == list(want)
            tables, refs, slots = got[0], got[1], got[4]
        assert refs == counts(tables, nb)
        for i in range(rows):
            if parents[i] >= 0 and slots[i] >= 0 and rng.random() < 0.8:
                at = at % 199 + 1
                for pool in pools:
                    pool.view(nb * bs, 64)[slots[i]] = float(at)
                texts[i].append(float(at))
                lens[i] += 1
        for i in range(rows):
            where = [tables[i][t // bs] * bs + t % bs for t in range(len(texts[i]))]
            for pool in pools:
                assert pool.view(nb * bs, 64)[where][:, 0].float().tolist() == texts[i]
        parents = [rng.choice([-1, rng.randrange(rows), i, i, i, i]) for i in range(rows)]
        if step % 4 == 3:    # jump near a block's end, where the fresh blocks are
            for i in range(rows):
                while 0 < len(texts[i]) < mb * bs and len(texts[i]) % bs and rng.random() < 0.95:
                    if refs[tables[i][lens[i] // bs]] != 1:   # (only a block of its own)
                        break
                    at = at % 199 + 1
                    for pool in pools:
                        pool.view(nb * bs, 64)[tables[i][lens[i] // bs] * bs + lens[i] % bs] = float(at)
                    texts[i].append(float(at))
                    lens[i] += 1


@pytest.mark.gpu
def test_wrapper_refuses_half_a_pair_of_slots():
    pools = pa.PoolSet(make_pools(1, 3, 16, 1, 64, False, 1))
    new = [dev([[7, 7]]), dev([7, 7, 7]), dev([7, 7, 7]), dev([7])]
    old = [dev([[2, 1]]), dev([32]), dev([0, 1, 1])]
    ws = torch.empty(pa.pa_compact_workspace_bytes(3), dtype=torch.uint8, device="cuda")
    for kw in (dict(slots=dev([5], torch.int64)), dict(new_slots=dev([5], torch.int64)),
               dict(slots=dev([5], torch.int64), new_slots=dev([5, 5], torch.int64))):
        with pytest.raises(ValueError):
            pa.pa_blocks_compact(*new, *old, pools, ws, **kw)
    with pytest.raises(TypeError):
        pa.pa_blocks_compact(*new, *old, pools, ws, slots=dev([5]), new_slots=dev([5]))


@pytest.mark.parametrize("slots,new_slots", [
    (None, 1 << 22), (1 << 22, None), (1 << 22, 1 << 22), ((1 << 22) + 4, 1 << 23), (1 << 22, (1 << 23) + 4)])
def test_slots_refusals(slots, new_slots):
    at = lambda x: None if x is None else ctypes.c_void_p(x)   # noqa: E731
    assert pa.lib().pa_blocks_compact_slots(OTHER[0], OTHER[1], OTHER[2], OTHER[3], at(new_slots), OTHER[4], OTHER[5], OTHER[6],
                                            at(slots), 3, 4, POOLS, 2, 2, DESC, FAKE, pa.pa_compact_workspace_bytes(64), None,
                                            None) == pa.PA_EINVAL


@pytest.mark.gpu
def test_padding_pairs_are_skipped_whatever_their_destination():
    pools = make_pools(2, 12, 16, 1, 64, False, 5)
    before = [t.clone() for t in pools]
    status = dev([0])
    pa.pa_blocks_copy(pa.PoolSet(pools), dev([[-1, 12], [-1, -1], [-7, 1 << 30], [3, 0]]), status=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    for pool, old in zip(pools, before):
        old[0] = old[3]
        assert torch.equal(pool.view(torch.uint8), old.view(torch.uint8))
