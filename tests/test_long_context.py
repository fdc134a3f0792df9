"""The operators on long contexts together, as a server runs them: prompts are read in and cut down by the weight that
their last queries gave to their tokens, then steps add a token each, attend the blocks that the bounds promise, keep
the weights and cut again.  A plain model on the CPU, in 64 bits, keeps every token's row by its place; tolerances are
those of the operators' own tests."""
import math
import os
import random
import re

import pytest
import torch

from paged_kv_decode_cache_gb300 import build as B
from paged_kv_decode_cache_gb300 import pa
from paged_model import as64, attention64, evicted, i32, scores64


@pytest.fixture(scope="module", autouse=True)
def _built():
    B.build()


HQ, HKV, D, BS, LAYERS = 8, 2, 128, 16, 2
G, SCALE = HQ // HKV, D ** -0.5
BUDGET, SLACK, FIRST, RECENT, KEEP, WINDOW = 64, 12, 2, 8, 4, 16


class Server:
    def __init__(self, lens, fp8, seed):
        self.fp8, self.ks, self.vs = fp8, 0.5 if fp8 else 1.0, 0.75 if fp8 else 1.0
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        self.B, self.mb = len(lens), 20
        nb = self.B * self.mb + 3
        ids = list(range(nb))
        random.Random(seed).shuffle(ids)
        self.tables = torch.full((self.B, self.mb), -1, dtype=torch.int32, device="cuda")
        self.refs = torch.zeros(nb, dtype=torch.int32, device="cuda")
        for b, n in enumerate(lens):
            k = -(-n // BS)
            self.tables[b, :k] = i32(ids[:k])
            self.refs[self.tables[b, :k].long()] = 1
            ids = ids[k:]
        self.lens, self.ends = i32([0] * self.B), i32([0] * self.B)
        dtype = torch.uint8 if fp8 else torch.bfloat16
        # what no token has been written to is never looked at
        self.pools = [torch.full((nb, BS, HKV, D), 0x7F if fp8 else math.nan, dtype=dtype, device="cuda") for _ in range(2 * LAYERS)]
        self.bounds = [torch.full((nb, HKV, 2, D), 0x7F if fp8 else math.nan, dtype=dtype, device="cuda") for _ in range(LAYERS)]
        room = self.mb * BS
        self.weights = torch.zeros(LAYERS, self.B, HKV, room, device="cuda")
        # (a call writes the positions of its queries' tokens: those before the window's have theirs from here)
        self.positions = torch.arange(room, device="cuda").int().expand(LAYERS, self.B, HKV, room).contiguous()
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.ws = torch.zeros(1 << 22, dtype=torch.uint8, device="cuda")
        # the model: of every layer, sequence and head the K and V rows by place, and their positions
        self.text = [[[([], [], []) for _ in range(HKV)] for _ in range(self.B)] for _ in range(LAYERS)]

    def rnd(self, *shape):
        return torch.randn(*shape, generator=self.gen, device="cuda").to(torch.bfloat16)

    def write(self, counts):
        """`counts` new tokens of each sequence."""
        lens, tables = self.lens.tolist(), self.tables.tolist()
        slots = [tables[b][t // BS] * BS + t % BS for b in range(self.B) for t in range(lens[b], lens[b] + counts[b])]
        for la in range(LAYERS):
            k, v = self.rnd(len(slots), HKV, D), self.rnd(len(slots), HKV, D)
            kp, vp = self.pools[2 * la:2 * la + 2]
            at = torch.tensor(slots, device="cuda")
            if self.fp8:
                pa.pa_cache_write_fp8(k, v, at, kp, vp, self.ks, self.vs, status=self.status)
            else:
                pa.pa_cache_write(k, v, at, kp, vp, status=self.status)
            rows = [as64(p.flatten(0, 1)[at]) for p in (kp, vp)]
            i = 0
            for b in range(self.B):
                for j in range(counts[b]):
                    for h in range(HKV):
                        text = self.text[la][b][h]
                        text[0].append(rows[0][i, h])
                        text[1].append(rows[1][i, h])
                        text[2].append(int(self.ends[b]) + j)
                    i += 1
        self.lens += i32(counts)
        self.ends += i32(counts)

    def keys(self, la, b, h):
        return torch.stack(self.text[la][b][h][0])

    def add_weights(self, la, q, lse):
        """The weights after one call, against the model's from the weights before it."""
        before = self.weights[la].double().cpu()
        args = (self.weights[la], self.weights[la], self.positions[la], q, lse, self.pools[2 * la])
        rest = (self.tables, self.lens, SCALE, self.ends)
        if self.fp8:
            pa.pa_weights_add_fp8(*args, self.ks, *rest, status=self.status)
        else:
            pa.pa_weights_add(*args, *rest, status=self.status)
        got, q_len = self.weights[la].double().cpu(), q.shape[1]
        q, lse = as64(q), lse.double().cpu()
        for b, n in enumerate(self.lens.tolist()):
            for h in range(HKV):
                k = self.keys(la, b, h) * self.ks
                want, off = before[b, h, :n].clone(), torch.zeros(n, dtype=torch.float64)
                want[max(0, n - q_len):] = 0.0
                for i in range(q_len):
                    see = n - q_len + i + 1
                    if see <= 0:
                        continue
                    for x in range(h * G, h * G + G):
                        s, z = k[:see] @ q[b, i, x] * SCALE, lse[b, i, x]
                        p = torch.exp(s - z)
                        want[:see] += p
                        size = k[:see].abs() @ q[b, i, x].abs() * SCALE
                        off[:see] += p * (2.0 ** -15 * size + 2.0 ** -22 * (s.abs() + z.abs()) + 2.0 ** -23 * s.abs() + 2.0 ** -22)
                assert ((got[b, h, :n] - want).abs() <= off + (q_len * G + 3) * 2.0 ** -24 * want).all()
                assert self.positions[la, b, h, :n].tolist() == self.text[la][b][h][2]

    def evict(self):
        new = [torch.empty_like(x) for x in (self.tables, self.lens, self.refs, self.weights, self.positions)]
        pa.pa_cache_evict(*new, self.tables, self.lens, self.refs, self.weights, self.positions, pa.PoolSet(self.pools), BUDGET,
                          first=FIRST, recent=RECENT, status=self.status)
        used = self.refs.sum().item()
        for b, n in enumerate(self.lens.tolist()):
            m = min(n, BUDGET)
            assert new[1][b].item() == m
            for la in range(LAYERS):
                for h in range(HKV):
                    text = self.text[la][b][h]
                    w = self.weights[la, b, h, :n].tolist()
                    src = evicted(w, text[2], m, 0, FIRST, RECENT)[1] if n > m else range(n)
                    self.text[la][b][h] = tuple([x[i] for i in src] for x in text)
                    assert new[3][la, b, h, :m].tolist() == [w[i] for i in src]
                    assert new[4][la, b, h, :m].tolist() == self.text[la][b][h][2]
                    at = (new[0][b].long().cpu().repeat_interleave(BS) * BS + torch.arange(self.mb * BS) % BS)[:m]
                    for pool, rows in zip(self.pools[2 * la:2 * la + 2], self.text[la][b][h][:2]):
                        assert torch.equal(as64(pool.flatten(0, 1)[at.cuda(), h]), torch.stack(rows))
            if n > m:
                used -= -(-n // BS) - (m // BS + 1)
        assert new[2].sum().item() == used
        self.tables, self.lens, self.refs, self.weights, self.positions = new
        for la in range(LAYERS):
            pa.pa_key_bounds(self.bounds[la], self.pools[2 * la], self.tables, self.lens, status=self.status)

    def room_for_one(self):
        """A block for every sequence's next token."""
        lens = self.lens.tolist()
        for b, n in enumerate(lens):
            if self.tables[b, n // BS].item() < 0:
                free = int((self.refs == 0).nonzero()[0])
                self.tables[b, n // BS] = free
                self.refs[free] = 1

    def attend(self, la, q, sel, sel_lens):
        out, lse = torch.empty_like(q), torch.empty(self.B, HQ, device="cuda")
        kp, vp = self.pools[2 * la:2 * la + 2]
        if self.fp8:
            pa.pa_decode_selected_fp8(out, lse, q, kp, vp, self.ks, self.vs, sel, sel_lens, SCALE, workspace=self.ws,
                                      status=self.status)
        else:
            pa.pa_decode_selected(out, lse, q, kp, vp, sel, sel_lens, SCALE, workspace=self.ws, status=self.status)
        return out.double().cpu(), lse.double().cpu()

    def plain_attend(self, la, q):
        out, lse = torch.empty_like(q), torch.empty(self.B, HQ, device="cuda")
        kp, vp = self.pools[2 * la:2 * la + 2]
        if self.fp8:
            pa.pa_decode_splitkv_fp8(out, lse, q, kp, vp, self.ks, self.vs, self.tables, self.lens, SCALE, workspace=self.ws,
                                     status=self.status)
        else:
            pa.pa_decode_splitkv(out, lse, q, kp, vp, self.tables, self.lens, SCALE, workspace=self.ws, status=self.status)
        return lse

    def check_attention(self, la, q, sel, sel_lens, out, lse):
        sel, sel_lens, q, tables = sel.tolist(), sel_lens.tolist(), as64(q), self.tables.tolist()
        for b, n in enumerate(self.lens.tolist()):
            blocks = -(-n // BS)
            for h in range(HKV):
                k, v = (torch.stack(x) for x in self.text[la][b][h][:2])
                hs = slice(h * G, h * G + G)
                parts = [k[j * BS:(j + 1) * BS] for j in range(blocks)]
                s = scores64(q[b, hs], torch.stack([x.amin(0) for x in parts]), torch.stack([x.amax(0) for x in parts]))
                if blocks > KEEP:
                    free = sorted(range(1, blocks - 1), key=lambda j: (-s[j], j))[:KEEP - 2]
                    take = sorted([0, blocks - 1] + free)
                else:
                    take = list(range(blocks))
                assert sel[b][h] == [tables[b][j] for j in take] + [-1] * (KEEP - len(take))
                at = [t for j in take for t in range(j * BS, min(n, (j + 1) * BS))]
                assert sel_lens[b][h] == len(at)
                want, z = attention64(q[b, hs], k[at] * self.ks, v[at] * self.vs, SCALE)
                assert ((lse[b, hs] - z).abs() <= 2.0 ** -13 + 2.0 ** -23 * z.abs()).all()
                assert ((out[b, hs] - want).abs() <= 2.0 ** -12 * 6 * self.vs + 2.0 ** -8 * want.abs()).all()


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True])
def test_prompts_cut_and_continued(fp8):
    lens = [150, 63, 33, 17]
    s = Server(lens, fp8, 3)
    s.write(lens)
    for la in range(LAYERS):
        # the last queries of the prompts, with the lse that attention gives them
        q = s.rnd(s.B, WINDOW, HQ, D) * 2
        lse = torch.full((s.B, WINDOW, HQ), -math.inf, device="cuda")
        if fp8:
            for i in range(WINDOW):
                out, z = torch.empty(s.B, HQ, D, dtype=torch.bfloat16, device="cuda"), torch.empty(s.B, HQ, device="cuda")
                pa.pa_decode_splitkv_fp8(out, z, q[:, i].contiguous(), *s.pools[2 * la:2 * la + 2], s.ks, s.vs, s.tables,
                                         s.lens - (WINDOW - 1 - i), SCALE, workspace=s.ws, status=s.status)
                lse[:, i] = z
        else:
            pa.pa_decode_mq(torch.empty_like(q), lse, q, *s.pools[2 * la:2 * la + 2], s.tables, s.lens, SCALE, workspace=s.ws,
                            status=s.status)
        s.add_weights(la, q, lse)
    s.evict()
    cuts = 0
    for step in range(30):
        s.room_for_one()
        s.write([1] * s.B)
        for la in range(LAYERS):
            q = s.rnd(s.B, HQ, D) * 2
            sel, n = torch.empty(s.B, HKV, KEEP, dtype=torch.int32, device="cuda"), torch.empty(s.B, HKV, dtype=torch.int32, device="cuda")
            pa.pa_key_bounds(s.bounds[la], s.pools[2 * la], s.tables, s.lens, s.lens - 1, max_new=1, status=s.status)
            pa.pa_blocks_select(sel, n, q, s.bounds[la], BS, s.tables, s.lens, status=s.status)
            out, lse = s.attend(la, q, sel, n)
            s.check_attention(la, q, sel, n, out, lse)
            s.add_weights(la, q[:, None], s.plain_attend(la, q)[:, None])
        if s.lens.max().item() >= BUDGET + SLACK:
            s.evict()
            cuts += 1
    assert cuts >= 2 and s.status.item() == 0


@pytest.mark.gpu
def test_a_step_of_selected_attention_in_a_graph():
    """Write, bounds, selection, attention and weights captured once; every replay adds a token."""
    g = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)   # noqa: E731
    steps, mb, nb, Bn = 20, 12, 40, 3
    tables = torch.randperm(nb, generator=torch.Generator().manual_seed(2))[:Bn * mb].int().view(Bn, mb).cuda()
    start = [70, 130, 16]
    pools = [rnd(nb, BS, HKV, D), rnd(nb, BS, HKV, D)]
    qs, ks, vs = rnd(steps, Bn, HQ, D), rnd(steps, Bn, HKV, D), rnd(steps, Bn, HKV, D)

    def state():
        z = lambda *s, t=torch.int32: torch.zeros(*s, dtype=t, device="cuda")   # noqa: E731
        lens = i32(start)
        st = dict(kc=pools[0].clone(), vc=pools[1].clone(), lens=lens, q=rnd(Bn, HQ, D), k=rnd(Bn, HKV, D), v=rnd(Bn, HKV, D),
                  bounds=z(nb, HKV, 2, D, t=torch.bfloat16), sel=z(Bn, HKV, KEEP), n=z(Bn, HKV), out=rnd(Bn, HQ, D),
                  lse=z(Bn, HQ, t=torch.float32), w=z(Bn, HKV, mb * BS, t=torch.float32), pos=z(Bn, HKV, mb * BS),
                  ws=z(1 << 22, t=torch.uint8), slots=z(Bn, t=torch.int64))
        pa.pa_key_bounds(st["bounds"], st["kc"], tables, lens)
        return st

    def step(s):
        at = s["lens"].long()
        s["slots"].copy_(tables.gather(1, (at // BS)[:, None])[:, 0] * BS + at % BS)
        pa.pa_cache_write(s["k"], s["v"], s["slots"], s["kc"], s["vc"])
        s["lens"].add_(1)
        pa.pa_key_bounds(s["bounds"], s["kc"], tables, s["lens"], s["lens"] - 1, max_new=1)
        pa.pa_blocks_select(s["sel"], s["n"], s["q"], s["bounds"], BS, tables, s["lens"])
        pa.pa_decode_selected(s["out"], s["lse"], s["q"], s["kc"], s["vc"], s["sel"], s["n"], SCALE, workspace=s["ws"])
        pa.pa_weights_add(s["w"], s["w"], s["pos"], s["q"], s["lse"], s["kc"], tables, s["lens"], SCALE)

    eager, graphed = state(), state()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        warm = state()
        step(warm)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(graphed)
    for i in range(steps):
        for s in (eager, graphed):
            s["q"].copy_(qs[i]), s["k"].copy_(ks[i]), s["v"].copy_(vs[i])
        step(eager)
        graph.replay()
        for name in ("lens", "sel", "n", "out", "lse", "w", "pos", "bounds", "kc"):
            assert torch.equal(eager[name], graphed[name]), (i, name)
    assert eager["lens"].tolist() == [n + steps for n in start]


@pytest.mark.gpu
def test_the_readmes_step_runs():
    """The README's calls as they stand there: a sequence above the budget is cut, what is attended is what the lists say."""
    with open(os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "README.md")) as f:
        code = [x for x in re.findall(r"```python\n(.*?)```", f.read(), re.S) if "pa_cache_evict" in x]
    assert len(code) == 1
    g = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)   # noqa: E731
    z = lambda *s, t=torch.int32: torch.zeros(*s, dtype=t, device="cuda")   # noqa: E731
    Bn, mb, nb, lens = 2, 80, 170, [1100, 900]
    tables = torch.randperm(nb, generator=torch.Generator().manual_seed(2))[:Bn * mb].int().view(Bn, mb).cuda()
    for b, n in enumerate(lens):
        tables[b, -(-n // BS):] = -1
    refs = torch.bincount(tables[tables >= 0].long(), minlength=nb).int()
    slots = torch.tensor([int(tables[b, (n - 1) // BS]) * BS + (n - 1) % BS for b, n in enumerate(lens)], device="cuda")
    ns = dict(torch=torch, pa=pa, num_blocks=nb, Hkv=HKV, D=D, bs=BS, scale=SCALE, layer=0, k_cache=rnd(nb, BS, HKV, D),
              v_cache=rnd(nb, BS, HKV, D), block_tables=tables, seq_lens=i32(lens), ends=i32(lens), refs=refs, k_new=rnd(Bn, HKV, D),
              v_new=rnd(Bn, HKV, D), slot_mapping=slots, q=rnd(Bn, HQ, D), sel=z(Bn, HKV, 64), sel_lens=z(Bn, HKV),
              out=rnd(Bn, HQ, D), lse=z(Bn, HQ, t=torch.float32), ws=z(1 << 22, t=torch.uint8),
              weights=torch.rand(1, Bn, HKV, mb * BS, generator=g, device="cuda"),
              positions=torch.arange(mb * BS, device="cuda").int().expand(1, Bn, HKV, mb * BS).contiguous(),
              new_tables=torch.empty_like(tables), new_lens=z(Bn), new_refs=z(nb), new_weights=z(1, Bn, HKV, mb * BS, t=torch.float32),
              new_positions=z(1, Bn, HKV, mb * BS))
    ns["pools"] = pa.PoolSet([ns["k_cache"], ns["v_cache"]])
    exec(compile(code[0], "README.md", "exec"), ns)
    assert ns["new_lens"].tolist() == [1024, 900]
    assert (ns["new_tables"] >= 0).sum(1).tolist() == [65, 57] and int(ns["new_refs"].sum()) == 65 + 57
    assert ((ns["sel"] >= 0).sum(-1) == torch.tensor([[64], [57]], device="cuda")).all()
    assert torch.isfinite(ns["lse"]).all() and ns["new_positions"][0, 0, :, :1024].unique(dim=-1).shape[-1] == 1024


@pytest.mark.gpu
def test_two_streams_at_once():
    """Every operator on two streams at a time, again and again: the results are those of one call alone."""
    g = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)   # noqa: E731
    Bn, mb, nb, hq, hkv = 4, 300, 1300, 8, 2
    z = lambda *s, t=torch.int32: torch.zeros(*s, dtype=t, device="cuda")   # noqa: E731

    class Side:
        def __init__(self, seed):
            self.tables = torch.randperm(nb, generator=torch.Generator().manual_seed(seed))[:Bn * mb].int().view(Bn, mb).cuda()
            self.lens = i32([mb * BS, 2000 + seed, 77, 4000])
            self.refs = z(nb)
            self.refs[self.tables.flatten().long()] = 1
            self.kc, self.vc, self.q = rnd(nb, BS, hkv, D), rnd(nb, BS, hkv, D), rnd(Bn, hq, D)
            self.window = rnd(Bn, 12, hq, D)
            self.lse = torch.full((Bn, 12, hq), 8.0, device="cuda")
            self.bounds, self.sel, self.n = z(nb, hkv, 2, D, t=torch.bfloat16), z(Bn, hkv, 32), z(Bn, hkv)
            self.out, self.z, self.ws = rnd(Bn, hq, D), z(Bn, hq, t=torch.float32), z(1 << 23, t=torch.uint8)
            self.w, self.pos = z(1, Bn, hkv, mb * BS, t=torch.float32), z(1, Bn, hkv, mb * BS)
            self.w1 = torch.zeros_like(self.w)
            self.new = [torch.zeros_like(x) for x in (self.tables, self.lens, self.refs, self.w, self.pos)]
            self.kept = [self.kc.clone(), self.vc.clone()]

        def run(self):
            pa.pa_key_bounds(self.bounds, self.kc, self.tables, self.lens)
            pa.pa_blocks_select(self.sel, self.n, self.q, self.bounds, BS, self.tables, self.lens)
            pa.pa_decode_selected(self.out, self.z, self.q, self.kc, self.vc, self.sel, self.n, SCALE, workspace=self.ws)
            pa.pa_weights_add(self.w[0], self.w1[0], self.pos[0], self.window, self.lse, self.kc, self.tables, self.lens, SCALE)
            pa.pa_weights_add(self.w[0], self.w[0], None, self.q, self.z, self.kc, self.tables, self.lens, SCALE)
            self.kept[0].copy_(self.kc), self.kept[1].copy_(self.vc)
            pa.pa_cache_evict(*self.new, self.tables, self.lens, self.refs, self.w, self.pos, pa.PoolSet(self.kept), 1000, 4, 64)

        def results(self):
            return [x.clone() for x in [self.bounds, self.sel, self.n, self.out, self.z, self.w] + self.new[:3] + self.kept]

    sides = [Side(1), Side(2)]
    alone = []
    for s in sides:
        s.run()
        torch.cuda.synchronize()
        alone.append(s.results())
    streams = [torch.cuda.Stream() for _ in sides]
    for _ in range(4):
        for _ in range(5):
            for s, st in zip(sides, streams):
                with torch.cuda.stream(st):
                    s.run()
        torch.cuda.synchronize()
        for s, want in zip(sides, alone):
            assert all(torch.equal(a, b) for a, b in zip(s.results(), want))


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True])
def test_blocks_past_32_bits_of_a_large_pool(fp8):
    """The same blocks at the front of a small pool and behind 2^32 bytes of a large one: the same results."""
    g = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)   # noqa: E731
    z = lambda *s, t=torch.int32: torch.zeros(*s, dtype=t, device="cuda")   # noqa: E731
    Bn, hq, hkv, mb, nb = 2, 16, 8, 30, 64
    far = (2 ** 32 // (BS * hkv * D * (1 if fp8 else 2))) + 5
    code = (lambda x: x.to(torch.float8_e4m3fn).view(torch.uint8)) if fp8 else (lambda x: x)
    k, v = code(rnd(nb, BS, hkv, D)), code(rnd(nb, BS, hkv, D))
    tables = torch.randperm(nb, generator=torch.Generator().manual_seed(2))[:Bn * mb].int().view(Bn, mb).cuda()
    lens, q, window = i32([mb * BS - 3, 333]), rnd(Bn, hq, D), rnd(Bn, 40, hq, D)
    lse = torch.full((Bn, 40, hq), 7.0, device="cuda")
    results = []
    for base in (0, far):
        pools = []
        for x in (k, v):
            pool = torch.empty(base + nb, BS, hkv, D, dtype=x.dtype, device="cuda")
            pool[base:] = x
            pools.append(pool)
        t = tables + base
        refs = z(base + nb)
        refs[t.flatten().long()] = 1
        bounds = z(base + nb, hkv, 2, D, t=k.dtype)
        sel, n, out, ws = z(Bn, hkv, 9), z(Bn, hkv), torch.empty_like(q), z(1 << 22, t=torch.uint8)
        w, pos = z(1, Bn, hkv, mb * BS, t=torch.float32), z(1, Bn, hkv, mb * BS)
        pa.pa_key_bounds(bounds, pools[0], t, lens)
        pa.pa_blocks_select(sel, n, q, bounds, BS, t, lens)
        scales = (0.5, 0.5) if fp8 else ()
        (pa.pa_decode_selected_fp8 if fp8 else pa.pa_decode_selected)(out, None, q, *pools, *scales, sel, n, SCALE, workspace=ws)
        for queries, z_ in ((window, lse), (q, lse[:, 0].contiguous())):
            if fp8:
                pa.pa_weights_add_fp8(w[0], w[0], pos[0], queries, z_, pools[0], 0.5, t, lens, SCALE)
            else:
                pa.pa_weights_add(w[0], w[0], pos[0], queries, z_, pools[0], t, lens, SCALE)
        pos.copy_(torch.arange(mb * BS, device="cuda").int().expand_as(pos))
        new = [torch.zeros_like(x) for x in (t, lens, refs, w, pos)]
        pa.pa_cache_evict(*new, t, lens, refs, w, pos, pa.PoolSet(pools), 200, 4, 16)
        results.append([bounds[base:], sel - base * (sel >= 0), n, out, w, new[0] - base * (new[0] >= 0), new[1], new[2][base:]] +
                       new[3:] + [p[base:] for p in pools])
    for i, (a, b) in enumerate(zip(*results)):
        assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8)), i
