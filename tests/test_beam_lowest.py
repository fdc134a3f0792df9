"""Beam selection over logits masked with their type's lowest value or another far one (not -inf), and over
values next to the type's largest one."""
import math

import pytest
import torch

from test_beam import _built, check, plain, run, spread  # noqa: F401


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("mask", ["lowest", -1e38, -1e30, -1e12, -1e9, -1e4])
@pytest.mark.parametrize("vocab,allowed", [(37, 5), (5003, 20), (5003, 2500), (100003, 3), (100003, 60000)])
def test_lowest_value_as_a_mask(dtype, vocab, allowed, mask):
    """The masked entries add nothing to the sums, and come after every allowed one."""
    g = torch.Generator().manual_seed(vocab + allowed)
    low = torch.finfo(dtype).min if mask == "lowest" else mask
    x = (torch.randn(6, vocab, generator=g) * 2.5).to(dtype)
    keep = torch.zeros(6, vocab, dtype=torch.bool)
    for w in range(6):   # a run of allowed entries: whole chunks before it and after it are masked
        at = (w * vocab // 6) % max(1, vocab - allowed)
        keep[w, at:at + allowed] = True
    x[~keep] = low
    cum = spread((2, 3), vocab)
    for K in (1, 4):
        check(run(x.cuda(), cum, K), plain(x, cum, None, -1, K))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("value", ["lowest", -1e38, -1e30, -1e12, -2.0 ** 31, -2.0 ** 30, -1e9, 1e9, 1e30])
@pytest.mark.parametrize("vocab", [8, 3000, 70001])
def test_a_row_of_one_far_value(dtype, vocab, value):
    """All entries are equally likely: cum - ln V (the formula; x - max first, since 64 bits cannot hold
    x - ln V next to such an x)."""
    x = torch.full((2, vocab), torch.finfo(dtype).min if value == "lowest" else value, dtype=dtype, device="cuda")
    cum = torch.tensor([[-2.0, -1.0]], device="cuda")
    scores, tokens, parents = run(x, cum, 3)
    assert tokens.tolist() == [[0, 1, 2]] and parents.tolist() == [[1, 1, 1]]
    assert (scores.double() + 1.0 + math.log(vocab)).abs().max() <= 2.0 ** -19 + 2.0 ** -23 * 13


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("vocab", [9, 20011])
def test_values_at_the_ends_of_the_range(dtype, vocab):
    """One entry far above the others, up to the largest value; rows of values far below zero with one that is
    less so: its probability is 1."""
    top, low = torch.finfo(dtype).max, torch.finfo(dtype).min
    at = vocab * 2 // 3
    cum = torch.tensor([[-0.5, -1.5, -2.5, -3.5]], device="cuda")
    x = torch.zeros(4, vocab)
    x[0], x[0, at] = low, low * 0.75
    x[1, at] = top
    x[2], x[2, at] = low * 0.25, 1.0
    x[3], x[3, at] = low, top
    x = x.to(dtype).cuda()
    scores, tokens, parents = run(x, cum, 4)
    assert tokens.tolist() == [[at] * 4] and parents.tolist() == [[0, 1, 2, 3]]
    assert (scores.double() - cum.cpu().double()).abs().max() <= 2.0 ** -19 + 2.0 ** -23 * 4
