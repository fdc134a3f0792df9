"""One workspace of pa_beam_select for calls of several shapes: nothing of one call is left where
another looks."""
import pytest
import torch

from paged_kv_decode_cache_gb300 import pa
from test_beam import _built, check, plain, run, spread  # noqa: F401


def inputs(groups, beams, vocab, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(groups * beams, vocab, generator=g) * 2.5).to(dtype).cuda(), spread((groups, beams), seed)


@pytest.mark.gpu
def test_groups_that_come_and_go():
    shapes = [(32, 4, 700, 4), (100, 4, 700, 4), (32, 4, 700, 4), (65, 2, 9000, 5), (1, 8, 40000, 16), (300, 1, 64, 2),
              (64, 4, 5000, 8), (257, 3, 100, 6)]
    for dtype in (torch.bfloat16, torch.float32):
        size = max(pa.pa_beam_workspace_bytes(*s, dtype) for s in shapes)
        ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
        for seed, (groups, beams, vocab, K) in enumerate(shapes):
            logits, cum = inputs(groups, beams, vocab, dtype, seed)
            check(run(logits, cum, K, ws=ws), plain(logits, cum, None, -1, K))


@pytest.mark.gpu
@pytest.mark.parametrize("groups", [4095, 4096, 4097, 9000])
def test_more_groups_than_one_launch_takes(groups):
    beams, vocab, K = 2, 37, 3
    logits, cum = inputs(groups, beams, vocab, torch.bfloat16, groups)
    fin = (torch.arange(groups * beams).view(groups, beams) % 5 == 0).to(torch.uint8).cuda()
    ws = torch.zeros(pa.pa_beam_workspace_bytes(groups, beams, vocab, K, torch.bfloat16), dtype=torch.uint8, device="cuda")
    want = plain(logits, cum, fin.cpu().numpy(), 7, K)
    for _ in range(2):
        check(run(logits, cum, K, finished=fin, eos=7, ws=ws), want)


def test_a_workspace_serves_fewer_groups():
    for vocab in (50, 5000, 151937):
        for beams in (1, 4, 12):
            sizes = [pa.pa_beam_workspace_bytes(g, beams, vocab, beams, torch.bfloat16) for g in range(1, 5000, 7)]
            assert sizes == sorted(sizes) and all(s % 256 == 0 for s in sizes)
    assert pa.pa_beam_workspace_bytes(5000, 2, 100, 4, torch.bfloat16) == pa.pa_beam_workspace_bytes(4096, 2, 100, 4, torch.bfloat16)
