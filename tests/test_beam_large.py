"""Beam selection over logits of every magnitude, held to the tolerance of test_beam.py: an lse is off by its
sum's rounding, not by the logits' size.

Beams' rows are one row rolled, so that their lse are the same number; their scores so far are 2^-15 apart, 16
times the tolerance: a beam whose lse is off by more than that changes its place."""
import pytest
import torch

from test_beam import _built, check, plain, run  # noqa: F401


def rolled(vocab, beams, seed, scale=1.0):
    x = torch.randn(vocab, generator=torch.Generator().manual_seed(seed)) * scale
    return torch.stack([x.roll(w * vocab // beams) for w in range(beams)])


def close_beams(groups, beams):
    step = torch.arange(beams, dtype=torch.float32) * 5 % beams   # (in no order)
    return (-1.0 - step * 2.0 ** -15).repeat(groups, 1).cuda()


@pytest.mark.gpu
@pytest.mark.parametrize("vocab", [900, 12345, 100003])
@pytest.mark.parametrize("offset", [0.0, -300.0, 300.0, 4097.0, 60000.0, -60000.0])
def test_beams_close_to_one_another(offset, vocab):
    """fp32 logits on a grid of 2^-7, so that an offset leaves their differences as they are."""
    beams = 4
    x = (rolled(vocab, beams, 3) * 128).round() / 128 + offset
    logits, cum = x.cuda(), close_beams(1, beams)
    for K in (4, 12):
        check(run(logits, cum, K), plain(logits, cum, None, -1, K))


@pytest.mark.gpu
@pytest.mark.parametrize("vocab", [5000, 120001])
@pytest.mark.parametrize("offset", [300.0, 60000.0])
def test_rising_rows(offset, vocab):
    """The running maximum moves in every chunk: each move's factor counts."""
    i = torch.arange(vocab, dtype=torch.float32)
    x = ((i * (24.0 / vocab)) * 128).round() / 128 + i % 7 / 16 + offset
    logits = torch.stack([x, x.flip(0), x.roll(vocab // 3)]).cuda()
    cum = close_beams(1, 3)
    check(run(logits, cum, 6), plain(logits, cum, None, -1, 6))
