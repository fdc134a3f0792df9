"""Small paged caches and plain 64-bit models for the tests of the operators on long contexts."""
import math
import random

import torch

FP8 = torch.float8_e4m3fn


def as64(t):
    """The values of a bf16 or e4m3 tensor in 64 bits, on the CPU."""
    t = t.cpu()
    return (t.view(FP8).float() if t.dtype == torch.uint8 else t).double()


def encode(x, fp8):
    return x.to(FP8).view(torch.uint8) if fp8 else x.to(torch.bfloat16)


def layout(lens, bs, seed, spare=2, shared=0, extra=0):
    """(tables, refs, number of blocks): blocks anywhere in the pool; the first `shared` are everyone's; `extra` unused
    columns."""
    rng = random.Random(seed)
    mb = max(1, max([-(-n // bs) for n in lens] or [1])) + extra
    nb = sum(-(-n // bs) for n in lens) + spare + shared
    ids = list(range(nb))
    rng.shuffle(ids)
    tables, refs, at = [], [0] * nb, shared
    for n in lens:
        k = -(-n // bs)
        row = ids[:min(shared, k)] + ids[at:at + max(0, k - shared)]
        at += max(0, k - shared)
        for x in row:
            refs[x] += 1
        tables.append(row + [-1] * (mb - k))
    return tables, refs, nb


def rows_of(table, n, bs):
    """Places in the pool (block * bs + offset) of a sequence's n tokens."""
    return torch.tensor([table[t // bs] * bs + t % bs for t in range(n)], dtype=torch.long)


def unused_rows(tables, lens, nb, bs):
    """Mask [nb * bs] of the pool's places that no sequence's tokens have."""
    free = torch.ones(nb * bs, dtype=torch.bool)
    for row, n in zip(tables, lens):
        free[rows_of(row, n, bs)] = False
    return free


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def scores64(q, lo, hi):
    """q [G, D], lo and hi [n, D]: each block's score."""
    s = torch.maximum(q[:, None] * lo, q[:, None] * hi).sum(-1).amax(0) if len(lo) else torch.zeros(0, dtype=torch.float64)
    odd = ~(torch.isfinite(lo).all(-1) & torch.isfinite(hi).all(-1))
    return torch.where(odd | ~torch.isfinite(q).all(), math.inf, s)


def attention64(q, k, v, scale):
    """q [G, D], k and v [n, D]: (out [G, D], lse [G])."""
    if not len(k):
        return torch.zeros_like(q), torch.full((len(q),), -math.inf, dtype=torch.float64)
    s = q @ k.t() * scale
    z = torch.logsumexp(s, -1)
    return torch.exp(s - z[:, None]) @ v, z


def evicted(weights, positions, n, fixed, first, recent):
    """The places of a row that stay, as a set, and the row's source of every place below n."""
    L = len(weights)
    newest = positions[-1] if L else 0

    def key(t):
        if t < fixed or positions[t] < first or positions[t] > newest - recent:
            return (2, 0.0)
        w = weights[t]
        return (1, math.inf if w != w else w + 0.0)
    stay = set(sorted(range(L), key=lambda t: (-key(t)[0], -key(t)[1], t))[:n])
    free = [t for t in range(n) if t not in stay]
    behind = [t for t in range(n, L) if t in stay]
    assert len(free) == len(behind)
    src = list(range(n))
    for a, b in zip(free, behind):
        src[a] = b
    return stay, src
