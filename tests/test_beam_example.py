"""The operators together: examples/beam_search.py's hypotheses, scored again from scratch."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_decode_cache_gb300 import build
    build.build()


def rescore(m, prompt, tokens):
    """A hypothesis's log-probability: the whole sequence through the layer at once in fp64, with the
    activations rounded to bf16 where the model holds them in bf16."""
    r = lambda t: t.to(torch.bfloat16).double()  # noqa: E731
    seq = torch.tensor(prompt + tokens[:-1], device="cuda")
    x = m.embedding[seq].double()
    y = r(x @ m.w_qkv.double())
    n, h, kv, d = len(seq), m.heads, m.kv_heads, m.head_dim
    q, k, v = (t.view(n, -1, d) for t in y.split([h * d, kv * d, kv * d], dim=1))
    angle = torch.arange(n, device="cuda").double()[:, None] * 10000.0 ** (-2.0 * torch.arange(d // 2, device="cuda") / d)
    cos, sin = angle.cos()[:, None], angle.sin()[:, None]
    turn = lambda t: r(torch.cat([t[..., :d // 2] * cos - t[..., d // 2:] * sin,   # noqa: E731
                                  t[..., :d // 2] * sin + t[..., d // 2:] * cos], -1))
    q, k = turn(q), turn(k).repeat_interleave(h // kv, 1)
    v = v.repeat_interleave(h // kv, 1)
    s = torch.einsum("qhd,thd->hqt", q, k) * m.scale
    s = m.softcap * torch.tanh(s / m.softcap)
    at = torch.arange(n, device="cuda")
    s = s + m.slopes.double()[:, None, None] * (at[None, None, :] - at[None, :, None])
    pos = torch.arange(n, device="cuda")[:, None]
    seen = (at < m.prefix) | ((at <= pos) & (at > pos - m.window))
    # (a prompt token sees the whole prefix, a later one only what is behind it, prefix included)
    s = s.masked_fill(~seen, -torch.inf)
    out = r(torch.einsum("hqt,thd->qhd", s.softmax(-1), v)).reshape(n, -1)
    logits = r(r(out @ m.w_out.double()) @ m.embedding.t().double()) * 0.5
    logp = logits.log_softmax(-1)
    first = len(prompt) - 1
    return sum(float(logp[first + i, t]) for i, t in enumerate(tokens))


@pytest.mark.parametrize("beams,length,block", [(1, 5, 16), (4, 37, 16), (3, 32, 32)])
def test_hypotheses_score_what_they_claim(beams, length, block):
    from beam_search import BeamSearch, Model
    m = Model(vocab=1009, window=24)
    prompts = torch.randint(3, m.vocab, (3, length), generator=torch.Generator().manual_seed(length)).cuda()
    search = BeamSearch(m, prompts, beams=beams, steps=25, block_size=block)
    found = search.run()
    for g, hyps in enumerate(found):
        scores = [s for s, _ in hyps]
        assert scores == sorted(scores, reverse=True)
        assert len({tuple(t) for _, t in hyps}) == beams          # hypotheses differ
        for score, tokens in hyps:
            again = rescore(m, prompts[g].tolist(), tokens)
            # A logit below 16 is off by its own bf16 half step (2^-5) and the ones of qkv, the
            # attention output and the hidden state (2^-8 of it each, 2^-4 together at 16): a
            # step's log-probability by less than twice 0.1 at the very worst, 0.1 on average
            # over the steps.
            assert abs(score - again) <= 0.1 * len(tokens)
    # the pages: what the tables name is what is counted, and every row has its own last page
    state = search.states[(search.steps - 1) % 2]
    tables, lens, refs = state.tables.cpu(), state.lens.cpu(), state.refs.cpu()
    count = torch.zeros_like(refs)
    for row, n in zip(tables, lens):
        used = n // block + 1                                      # the next token's page among them
        for b in row[:used].tolist():
            count[b] += 1
    assert torch.equal(count, refs)
    last = [int(row[n // block]) for row, n in zip(tables, lens)]
    assert len(set(last)) == len(last) and all(int(refs[b]) == 1 for b in last)
