"""The README's step of beam search, run as it stands there."""
import os
import re

import pytest
import torch

from paged_kv_decode_cache_gb300 import build as B
from paged_kv_decode_cache_gb300 import pa

README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


def snippet():
    with open(README) as f:
        blocks = re.findall(r"```python\n(.*?)```", f.read(), re.S)
    found = [b for b in blocks if "pa_sequences_fork" in b]
    assert len(found) == 1
    return found[0]


def test_the_step_is_there_and_compiles():
    compile(snippet(), "README.md", "exec")


@pytest.mark.gpu
def test_the_step_keeps_every_token():
    """Three steps of two beams (one of them near a block's end): every token's V row stays where the
    new tables look for it, and the next slots come after it."""
    B.build()
    bs, mb, nb, hq, hkv, d, vocab, rows = 16, 6, 40, 4, 2, 128, 500, 4
    g = torch.Generator(device="cuda").manual_seed(1)
    new = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)   # noqa: E731
    i32 = {"dtype": torch.int32, "device": "cuda"}
    lens = torch.tensor([14, 14, 20, 20], **i32)
    tables = torch.full((rows, mb), -1, **i32)
    tables[0, 0], tables[1, 0] = 3, 9
    tables[2, :2], tables[3, :2] = torch.tensor([7, 5], **i32), torch.tensor([7, 2], **i32)
    refs = torch.bincount(tables[tables >= 0].long(), minlength=nb).int()
    slots = torch.tensor([3 * bs + 14, 9 * bs + 14, 5 * bs + 4, 2 * bs + 4], device="cuda")
    k_cache, v_cache = new(nb, bs, hkv, d), new(nb, bs, hkv, d)
    texts = [[v_cache[tables[i, t // bs], t % bs].clone() for t in range(int(lens[i]))] for i in range(rows)]
    P = pa.pa_scored_num_splits(rows, 1, hq, hkv, d, mb, bs, window=4096, max_prefix=4)
    ns = {"pa": pa, "k_cache": k_cache, "v_cache": v_cache, "tables": tables, "lens": lens, "refs": refs, "slots": slots,
          "scale": d ** -0.5, "slopes": torch.full((hq,), 0.1, device="cuda"), "sinks": torch.full((rows,), 4, **i32), "P": P,
          "ws": torch.zeros(max(1, pa.pa_splitkv_workspace_bytes(rows, hq, d, P)), dtype=torch.uint8, device="cuda"),
          "scores": torch.zeros(2, 2, device="cuda"), "tokens": torch.zeros(2, 2, **i32), "parents": torch.zeros(2, 2, **i32),
          "done": torch.zeros(2, 2, dtype=torch.uint8, device="cuda"),
          "beam_ws": torch.zeros(pa.pa_beam_workspace_bytes(2, 2, vocab, 2, torch.bfloat16), dtype=torch.uint8, device="cuda"),
          "fork_ws": torch.empty(pa.pa_fork_workspace_bytes(rows, rows, nb), dtype=torch.uint8, device="cuda")}
    code = compile(snippet(), "README.md", "exec")
    for step in range(3):
        v_new = new(rows, hkv, d)
        ns |= {"q": new(rows, hq, d), "k_new": new(rows, hkv, d), "v_new": v_new, "out": torch.empty(rows, hq, d, dtype=torch.bfloat16, device="cuda"),
               "logits": new(rows, vocab), "cum": ns["scores"].clone(), "new_tables": torch.empty(rows, mb, **i32),
               "new_lens": torch.empty(rows, **i32), "new_refs": torch.empty(nb, **i32)}
        exec(code, ns)
        texts = [texts[p] + [v_new[p]] for p in ns["parents"].view(-1).tolist()]
        ns |= {"tables": ns["new_tables"], "lens": ns["new_lens"], "refs": ns["new_refs"]}
        assert ns["lens"].tolist() == [len(t) for t in texts]
        for i, text in enumerate(texts):
            kept = torch.stack([v_cache[ns["tables"][i, t // bs], t % bs] for t in range(len(text))])
            assert torch.equal(kept, torch.stack(text)), (step, i)
            at = int(ns["slots"][i])
            assert at % bs == len(text) % bs and at // bs == int(ns["tables"][i, len(text) // bs])
        assert len(set(ns["slots"].tolist())) == rows
