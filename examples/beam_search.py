"""Beam search over the paged KV cache: every step of a one-layer toy model (random weights) on the
GPU, without the host looking at anything until the end.

    python examples/beam_search.py

A step turns the new queries and keys and writes K and V (pa_rope_write), attends under the model's
score rules (pa_decode_scored), selects the best continuations (pa_beam_select) and reorders the
sequences, sharing their pages (pa_sequences_fork), which also gives the slots of the next step.  The
state of the pages is double-buffered, so two captured CUDA graphs, replayed in turn, are the loop.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from paged_kv_decode_cache_gb300 import pa  # noqa: E402


class Model:
    """One attention layer between an embedding and its transpose."""

    def __init__(self, vocab=5003, width=256, heads=8, kv_heads=2, head_dim=128, softcap=30.0, window=48, prefix=4,
                 seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.vocab, self.heads, self.kv_heads, self.head_dim = vocab, heads, kv_heads, head_dim
        self.softcap, self.window, self.prefix, self.scale = softcap, window, prefix, head_dim ** -0.5
        new = lambda *shape: torch.randn(*shape, generator=g, device="cuda", dtype=torch.bfloat16)  # noqa: E731
        self.embedding = new(vocab, width)
        self.w_qkv = new(width, (heads + 2 * kv_heads) * head_dim) * width ** -0.5
        self.w_out = new(heads * head_dim, width) * (heads * head_dim) ** -0.5
        self.slopes = torch.tensor([2.0 ** (-8.0 * (h + 1) / heads) for h in range(heads)], device="cuda")
        self.rope = pa.pa_rope_init(head_dim, 10000.0)

    def qkv(self, x):
        y = x @ self.w_qkv
        sizes = [self.heads * self.head_dim] + [self.kv_heads * self.head_dim] * 2
        return [t.view(len(x), -1, self.head_dim) for t in y.split(sizes, dim=1)]

    def logits(self, attended):
        return (attended.reshape(len(attended), -1) @ self.w_out) @ self.embedding.t() * 0.5


class State:
    """The sequences' pages: block tables, lengths, reference counts and the next tokens' slots."""

    def __init__(self, rows, max_blocks, num_blocks):
        i32 = {"dtype": torch.int32, "device": "cuda"}
        self.tables = torch.full((rows, max_blocks), -1, **i32)
        self.lens = torch.zeros(rows, **i32)
        self.refs = torch.zeros(num_blocks, **i32)
        self.slots = torch.full((rows,), -1, dtype=torch.int64, device="cuda")


class BeamSearch:
    def __init__(self, model: Model, prompts: torch.Tensor, beams: int, steps: int, block_size=16, eos=2):
        m, (groups, length) = model, prompts.shape
        self.model, self.beams, self.steps, self.eos = model, beams, steps, eos
        self.groups, self.prompt_len, rows = groups, length, groups * beams
        self.max_blocks = -(-(length + steps + 1) // block_size)
        num_blocks = groups * (beams + 1) * self.max_blocks
        shape = (num_blocks, block_size, m.kv_heads, m.head_dim)
        self.k_cache, self.v_cache = (torch.zeros(shape, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.pools = pa.PoolSet([self.k_cache, self.v_cache])
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.states = [State(rows, self.max_blocks, num_blocks) for _ in range(2)]
        self.fork_space = torch.empty(pa.pa_fork_workspace_bytes(rows, rows, num_blocks), dtype=torch.uint8, device="cuda")
        self.beam_space = torch.zeros(pa.pa_beam_workspace_bytes(groups, beams, m.vocab, beams, torch.bfloat16),
                                      dtype=torch.uint8, device="cuda")
        self.prefix = torch.full((rows,), m.prefix, dtype=torch.int32, device="cuda")
        self.splits = pa.pa_scored_num_splits(rows, 1, m.heads, m.kv_heads, m.head_dim, self.max_blocks, block_size,
                                              window=m.window, max_prefix=m.prefix)
        self.space = torch.zeros(max(1, pa.pa_splitkv_workspace_bytes(rows, m.heads, m.head_dim, self.splits)),
                                 dtype=torch.uint8, device="cuda")
        self.scores = torch.zeros(groups, beams, device="cuda")
        self.tokens, self.parents = (torch.zeros(groups, beams, dtype=torch.int32, device="cuda") for _ in range(2))
        self.finished = torch.zeros(groups, beams, dtype=torch.uint8, device="cuda")
        self.history = torch.zeros(steps, 2, rows, dtype=torch.int32, device="cuda")  # token, parent
        self.at = torch.zeros(1, dtype=torch.int64, device="cuda")
        self._start(prompts, block_size)

    def _attend(self, out, q, tables, lens, prefix, splits, space):
        m = self.model
        pa.pa_decode_scored(out, None, q, self.k_cache, self.v_cache, tables, lens, m.scale, softcap=m.softcap,
                            alibi_slopes=m.slopes, window=m.window, prefix_lens=prefix, max_prefix=m.prefix,
                            num_splits=splits, workspace=space, status=self.status)

    def _record(self):
        """Note the chosen tokens and parents, and which beams have ended."""
        row = torch.stack([self.tokens.view(-1), self.parents.view(-1)])
        self.history.index_copy_(0, self.at, row[None])
        self.at += 1

    def _start(self, prompts, block_size):
        """The prompts in one chunk, their first continuations, and one table per beam."""
        m, groups, length = self.model, self.groups, self.prompt_len
        num_blocks = self.k_cache.shape[0]
        state, used = State(groups, self.max_blocks, num_blocks), -(-length // block_size)
        blocks = torch.arange(groups * used, dtype=torch.int32, device="cuda").view(groups, used)
        state.tables[:, :used] = blocks
        state.refs[:groups * used] = 1
        state.lens += length
        t = torch.arange(length, device="cuda")
        slots = (blocks[:, t // block_size].long() * block_size + t % block_size).reshape(-1)
        x = m.embedding[prompts.reshape(-1)]
        q, k, v = m.qkv(x)
        turned = torch.empty(groups, length, m.heads, m.head_dim, dtype=torch.bfloat16, device="cuda")
        pa.pa_rope_write(turned.view(groups * length, m.heads, m.head_dim), q, k, v, t.int().repeat(groups), slots,
                         self.k_cache, self.v_cache, m.rope, status=self.status)
        P = pa.pa_scored_num_splits(groups, length, m.heads, m.kv_heads, m.head_dim, self.max_blocks, block_size,
                                    window=m.window, max_prefix=m.prefix)
        space = torch.zeros(max(1, pa.pa_splitkv_workspace_bytes(groups * length, m.heads, m.head_dim, P)),
                            dtype=torch.uint8, device="cuda")
        out = torch.empty_like(turned)
        self._attend(out, turned, state.tables, state.lens, self.prefix[:groups].contiguous(), P, space)
        logits = m.logits(out[:, -1])
        first = torch.zeros(pa.pa_beam_workspace_bytes(groups, 1, m.vocab, self.beams, torch.bfloat16), dtype=torch.uint8,
                            device="cuda")
        pa.pa_beam_select(self.scores, self.tokens, self.parents, logits, torch.zeros(groups, 1, device="cuda"),
                          workspace=first)
        self.finished.copy_(self.tokens == self.eos)
        self._record()
        self._fork(state, self.states[0], self.parents.view(-1))

    def _fork(self, old, new, parents):
        pa.pa_sequences_fork(new.tables, new.lens, new.refs, new.slots, old.tables, old.lens, old.refs, parents,
                             self.pools, self.fork_space, status=self.status)

    def step(self, old: State, new: State):
        """One token for every beam, from the pages of `old` to those of `new`."""
        m, rows = self.model, self.groups * self.beams
        x = m.embedding[self.tokens.view(-1).clamp(min=0).long()]
        q, k, v = m.qkv(x)
        turned = torch.empty(rows, m.heads, m.head_dim, dtype=torch.bfloat16, device="cuda")
        pa.pa_rope_write(turned, q, k, v, old.lens, old.slots, self.k_cache, self.v_cache, m.rope, status=self.status)
        old.lens += (old.slots >= 0).int()
        out = torch.empty_like(turned)
        self._attend(out, turned, old.tables, old.lens, self.prefix, self.splits, self.space)
        logits = m.logits(out)
        done, cum = self.finished.clone(), self.scores.clone()
        pa.pa_beam_select(self.scores, self.tokens, self.parents, logits, cum, finished=done, eos=self.eos,
                          workspace=self.beam_space)
        parents = self.parents.view(-1)
        self.finished.copy_(((self.tokens == self.eos) | (self.parents < 0)).to(torch.uint8))
        self._record()
        self._fork(old, new, parents)

    def run(self):
        """All steps by replaying two graphs; [(score, tokens)] of every request, best first."""
        a, b = self.states
        graphs = []
        keep = [t.clone() for t in self._mutable()]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):  # warm up the library calls of the step, then start over
            self.step(a, b)
        torch.cuda.current_stream().wait_stream(side)
        for t, saved in zip(self._mutable(), keep):
            t.copy_(saved)
        for old, new in ((a, b), (b, a)):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                self.step(old, new)
            graphs.append(g)
        for i in range(self.steps - 1):
            graphs[i % 2].replay()
        torch.cuda.synchronize()
        return self.results()

    def _mutable(self):
        pages = [t for s in self.states for t in (s.tables, s.lens, s.refs, s.slots)]
        return [self.k_cache, self.v_cache, self.scores, self.tokens, self.parents, self.finished, self.history, self.at,
                *pages]

    def results(self):
        if self.status.item():
            raise RuntimeError(f"status {self.status.item()}")
        history, scores = self.history[:int(self.at)].cpu(), self.scores.cpu()
        out = []
        for g in range(self.groups):
            found = []
            for w in range(self.beams):
                row, tokens = g * self.beams + w, []
                for i in reversed(range(len(history))):
                    tokens.append(int(history[i, 0, row]))
                    row = int(history[i, 1, row])
                tokens.reverse()
                if self.eos in tokens:
                    tokens = tokens[:tokens.index(self.eos) + 1]
                found.append((float(scores[g, w]), tokens))
            out.append(found)
        return out


def main():
    model = Model()
    prompts = torch.randint(3, model.vocab, (4, 37), generator=torch.Generator().manual_seed(1)).cuda()
    search = BeamSearch(model, prompts, beams=4, steps=40)
    for g, found in enumerate(search.run()):
        score, tokens = found[0]
        print(f"request {g}: log-probability {score:.3f}, {len(tokens)} tokens: {tokens[:12]} ...")


if __name__ == "__main__":
    main()
