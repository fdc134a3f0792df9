"""The README's calls on long contexts as a loop runs them: step after step, each adds a token, and the next one selects and
attends what the cut has left."""
import os
import re

import pytest
import torch

from paged_kv_decode_cache_gb300 import build as B
from paged_kv_decode_cache_gb300 import pa
from paged_model import i32

HQ, HKV, D, BS = 8, 2, 128, 16
README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


def parts():
    """(what is run once, what is run every step)."""
    with open(README) as f:
        code = [x for x in re.findall(r"```python\n(.*?)```", f.read(), re.S) if "pa_cache_evict" in x]
    assert len(code) == 1
    at = code[0].index("pa.pa_cache_write(")
    return code[0][:at], code[0][at:]


@pytest.mark.gpu
def test_the_readmes_steps_as_a_loop():
    B.build()
    g = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)   # noqa: E731
    z = lambda *s, t=torch.int32: torch.zeros(*s, dtype=t, device="cuda")   # noqa: E731
    Bn, mb, nb, lens = 2, 80, 170, [1099, 1010]
    tables = torch.randperm(nb, generator=torch.Generator().manual_seed(2))[:Bn * mb].int().view(Bn, mb).cuda()
    for b, n in enumerate(lens):
        tables[b, -(-n // BS):] = -1
    ns = dict(torch=torch, pa=pa, num_blocks=nb, Hkv=HKV, D=D, bs=BS, scale=D ** -0.5, layer=0, k_cache=rnd(nb, BS, HKV, D),
              v_cache=rnd(nb, BS, HKV, D), block_tables=tables, seq_lens=i32(lens), ends=i32(lens),
              refs=torch.bincount(tables[tables >= 0].long(), minlength=nb).int(), sel=z(Bn, HKV, 64), sel_lens=z(Bn, HKV),
              out=rnd(Bn, HQ, D), lse=z(Bn, HQ, t=torch.float32), ws=z(1 << 22, t=torch.uint8),
              weights=torch.rand(1, Bn, HKV, mb * BS, generator=g, device="cuda"),
              positions=torch.arange(mb * BS, device="cuda").int().expand(1, Bn, HKV, mb * BS).contiguous(),
              new_tables=torch.empty_like(tables), new_lens=z(Bn), new_refs=z(nb), new_weights=z(1, Bn, HKV, mb * BS, t=torch.float32),
              new_positions=z(1, Bn, HKV, mb * BS))
    ns["pools"] = pa.PoolSet([ns["k_cache"], ns["v_cache"]])
    once, step = (compile(x, "README.md", "exec") for x in parts())
    exec(once, ns)
    for turn in range(1, 21):
        for b, n in enumerate(ns["seq_lens"].tolist()):     # a block for the next token
            if n % BS == 0 and ns["block_tables"][b, n // BS] < 0:
                free = int((ns["refs"] == 0).nonzero()[0])
                ns["block_tables"][b, n // BS], ns["refs"][free] = free, 1
        at = ns["seq_lens"].long()
        ns["slot_mapping"] = ns["block_tables"].gather(1, (at // BS)[:, None])[:, 0] * BS + at % BS
        ns["seq_lens"] += 1
        ns["ends"] += 1
        ns["q"], ns["k_new"], ns["v_new"] = rnd(Bn, HQ, D), rnd(Bn, HKV, D), rnd(Bn, HKV, D)
        exec(step, ns)
        assert ns["seq_lens"].tolist() == [1024, min(1024, 1010 + turn)]
        assert int(ns["refs"].sum()) == int((ns["block_tables"] >= 0).sum())
        fresh = torch.full_like(ns["bounds"], float("nan"))
        pa.pa_key_bounds(fresh, ns["k_cache"], ns["block_tables"], ns["seq_lens"])
        for b, n in enumerate(ns["seq_lens"].tolist()):
            ids = ns["block_tables"][b, :-(-n // BS)].long()
            assert torch.equal(ns["bounds"][ids], fresh[ids]), (turn, b)
            for h in range(HKV):
                has = ns["positions"][0, b, h, :n].tolist()
                end = int(ns["ends"][b])
                assert len(set(has)) == n and set(range(end - 128, end)) <= set(has) and {0, 1, 2, 3} <= set(has)
