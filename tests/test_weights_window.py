"""What pa_weights_add does with bad blocks, lengths, keys and lse, for few columns (queries x heads of a group: one
kernel) and for many (another, 128 tokens and up to 256 columns at a time), against a plain sum in 64 bits.  The
tolerance is that of test_weights.py."""
import math

import pytest
import torch

from paged_kv_decode_cache_gb300 import build as B
from paged_kv_decode_cache_gb300 import pa
from paged_model import as64, encode, i32

BS = 16


@pytest.fixture(scope="module", autouse=True)
def _built():
    B.build()


SHAPES = [  # heads, KV heads, head_dim, queries: 2, 20, 80, 90 and (two and three chunks of) 400 and 600 columns
    (4, 2, 64, 1), (4, 1, 128, 5), (4, 2, 128, 40), (6, 2, 64, 30), (2, 1, 128, 200), (6, 2, 64, 200),
]


class Call:
    """Sequences of some tokens over a pool, blocks in order of nothing; `old` weights that fade."""
    def __init__(self, shape, fp8, lens, blocks, seed=1, room=None):
        self.hq, self.hkv, self.d, self.q_len = shape
        self.fp8, self.lens, self.blocks, self.scale, self.ks = fp8, lens, blocks, shape[2] ** -0.5, 0.5 if fp8 else 1.0
        g = torch.Generator().manual_seed(seed)
        self.nb = len(lens) * blocks + 1
        self.tables = torch.randperm(self.nb, generator=g)[:len(lens) * blocks].view(len(lens), blocks).tolist()
        self.q = torch.randn(len(lens), self.q_len, self.hq, self.d, generator=g).to(torch.bfloat16)
        self.k = encode(torch.randn(self.nb, BS, self.hkv, self.d, generator=g), fp8)
        self.room = room or blocks * BS
        self.old = torch.rand(len(lens), self.hkv, self.room, generator=g) + 0.5
        # near what attention gives: a query's weights sum to something near one
        self.lse = torch.rand(len(lens), self.q_len, self.hq, generator=g) + 5.0

    def spoil(self, b, t, value):
        """Token t's key of every head."""
        self.k[self.tables[b][t // BS], t % BS] = value

    def check(self, status=0, decay=0.75, same=False):
        Bn, G = len(self.lens), self.hq // self.hkv
        old = self.old.cuda()
        new = old if same else torch.full_like(old, 7.0)
        flag = torch.zeros(1, dtype=torch.int32, device="cuda")
        fp8 = (self.ks,) if self.fp8 else ()
        (pa.pa_weights_add_fp8 if self.fp8 else pa.pa_weights_add)(
            new, old, None, self.q.cuda(), self.lse.cuda(), self.k.cuda(), *fp8, i32(self.tables), i32(self.lens), self.scale,
            decay=decay, status=flag)
        torch.cuda.synchronize()
        assert flag.item() == status
        got, q, keys = new.double().cpu(), as64(self.q), as64(self.k) * self.ks
        for b in range(Bn):
            n = min(max(self.lens[b], 0), self.blocks * BS, self.room)
            ids = torch.tensor(self.tables[b])[torch.arange(n) // BS]
            good = (ids >= 0) & (ids < self.nb)
            rows = keys[torch.where(good, ids, 0), torch.arange(n) % BS]
            seen = torch.arange(n)[:, None] <= n - self.q_len + torch.arange(self.q_len)
            for h in range(self.hkv):
                hs = slice(h * G, h * G + G)
                z = self.lse[b, :, hs].double()
                s = torch.einsum("qgd,td->tqg", q[b, :, hs], rows[:, h]) * self.scale
                size = torch.einsum("qgd,td->tqg", q[b, :, hs].abs(), rows[:, h].abs()) * self.scale
                here = seen[:, :, None] & good[:, None, None] & (z != -math.inf)
                p = torch.where(here, torch.exp(s - z), 0.0)
                off = p * (2.0 ** -15 * size + 2.0 ** -22 * (s.abs() + z.abs()) + 2.0 ** -23 * s.abs() + 2.0 ** -22)
                # (a term of s = -inf or lse = inf is exp(-inf) = 0 in any arithmetic: nothing off, where 0 * inf is NaN)
                want, tol = p.sum((1, 2)), torch.where(here & (p > 0), off, 0.0).sum((1, 2))
                past = max(0, n - self.q_len)
                want[:past] += decay * self.old[b, h, :past].double()
                tol += (self.q_len * G + 3) * 2.0 ** -24 * want
                mine = got[b, h, :n]
                assert torch.equal(torch.isnan(mine), torch.isnan(want)) and torch.equal(torch.isinf(mine), torch.isinf(want))
                fine = torch.isfinite(want)
                assert ((mine - want).abs() <= tol)[fine].all(), (b, h, float(((mine - want).abs() - tol)[fine].max()))
            rest = self.old[b, :, n:].double() if same else torch.full_like(got[b, :, n:], 7.0)
            assert torch.equal(got[b, :, n:], rest)


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
def test_blocks_outside_the_pool_draw_nothing(shape, fp8):
    """One in the middle of 128 tokens, all of some 128, the first, the last, every one of a sequence."""
    c = Call(shape, fp8, [600, 470, 333, 40], 38, seed=shape[3])
    for j in (3, 12, 13, 14):
        c.tables[0][j] = (-1, c.nb, 1 << 30, -5)[j % 4]
    c.tables[1][8:16] = [-1] * 8
    c.tables[1][29] = c.nb
    c.tables[2] = [-1] * 38
    c.tables[3][0] = c.nb + 3
    c.check(pa.PA_STATUS_BAD_BLOCK)
    c.check(pa.PA_STATUS_BAD_BLOCK, same=True)
    c.tables[0][:8] = [c.nb] * 8
    c.check(pa.PA_STATUS_BAD_BLOCK, decay=0.0)


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
def test_bad_blocks_behind_a_sequence_are_nobodys(shape, fp8):
    c = Call(shape, fp8, [129, 16, 0, 256], 20, seed=shape[3])
    for b, n in enumerate(c.lens):
        k = -(-n // BS)
        c.tables[b][k:] = [(-1, c.nb + 7)[j % 2] for j in range(20 - k)]
    c.check()


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("lens,room", [([700, 609, 20], None), ([-1, 300, -2 ** 31], None), ([600, 200, 511], 510),
                                       ([2 ** 31 - 1, 1, 130], 129)])
def test_lengths_outside_the_table_or_the_room(shape, fp8, lens, room):
    Call(shape, fp8, lens, 38, seed=shape[3], room=room).check(pa.PA_STATUS_BAD_SEQLEN)


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
def test_nan_and_infinite_keys_stay_with_their_token(shape, fp8):
    """Next to finite ones, in rows of another KV head, behind the last token and in blocks that no sequence has."""
    c = Call(shape, fp8, [300, 131, 64], 19, seed=shape[3])
    bad = 0x7F if fp8 else math.nan
    for b, t in ((0, 0), (0, 17), (0, 128), (0, 299), (1, 127), (1, 130)):
        c.spoil(b, t, bad)
    c.k[c.tables[2][1], 3, 0] = bad            # (one KV head's alone)
    for b, n in enumerate(c.lens):
        for t in range(n, 19 * BS):
            c.spoil(b, t, bad)
    if not fp8:
        c.k[c.tables[0][4], 5, :, 7] = math.inf
        c.k[c.tables[0][4], 6, :, 7] = -math.inf
        c.k[c.tables[1][2], 9, :, 0] = math.inf
    c.check()
    c.check(same=True)


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
def test_a_query_that_saw_nothing_among_others(shape, fp8):
    """An lse of -inf, of one head of one query, of a whole query, of all of a sequence's; and +inf, which draws nothing."""
    c = Call(shape, fp8, [300, 131, 64], 19, seed=shape[3])
    mid = shape[3] // 2
    c.lse[0, mid, 1] = -math.inf
    c.lse[0, -1, 0] = math.inf
    c.lse[1, mid] = -math.inf
    c.lse[2] = -math.inf
    c.spoil(0, 30, 0x7F if fp8 else math.nan)
    c.check()
    c.lse[0, 0, 0] = math.nan                  # (a query whose attention was NaN: every token that it sees)
    c.check()
