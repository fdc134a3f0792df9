"""One workspace of the split decode calls, shared by calls of several shapes and split counts."""
import math

import pytest
import torch

from paged_kv_decode_cache_gb300 import build as B
from paged_kv_decode_cache_gb300 import pa


@pytest.fixture(scope="module", autouse=True)
def _built():
    B.build()


HQ, HKV, D, BS, MB = 28, 4, 128, 16, 512


def splits(b, window, **kw):
    return pa.pa_scored_num_splits(b, 1, HQ, HKV, D, MB, BS, window=window, **kw)


def test_windows_change_the_split_count():
    """The shapes below do meet at the counters (more than 16 partitions), with different counts."""
    for b in (1, 2, 4, 8):
        assert splits(b, 0, sm_count=152) != splits(b, 1024, sm_count=152)
        assert min(splits(b, 0, sm_count=152), splits(b, 1024, sm_count=152)) > 16


def test_counters_have_their_own_place():
    for b, hq, p in ((1, 1, 2), (8, 28, 9), (64, 32, 64)):
        rows = b * hq * p
        assert pa.pa_splitkv_workspace_bytes(b, hq, D, p) >= 4096 + rows * D * 4 + rows * 4
    # more groups than counters: never merged in the launch, whatever the GPU's size
    assert pa.pa_decode_launches(1024, 1, 16, 8, 128, 64, 16, 2, 1 << 20) == 1
    assert pa.pa_decode_launches(1025, 1, 16, 8, 128, 64, 16, 2, 1 << 20) == 2


class Call:
    """A decode call of b sequences on the given workspace, and on a new one."""

    def __init__(self, b, seed, window=0, fp8=False, plain=False, kv_heads=HKV, num_splits=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.b, self.window, self.fp8, self.plain, self.splits = b, window, fp8, plain, num_splits
        self.q = torch.randn(b, HQ, D, generator=g, device="cuda").to(torch.bfloat16)
        shape = (b * MB, BS, kv_heads, D)
        self.pools = [torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2)]
        if fp8:
            self.pools = [p.to(torch.float8_e4m3fn).view(torch.uint8) for p in self.pools]
        self.tables = torch.randperm(b * MB, generator=g, device="cuda").to(torch.int32).view(b, MB)
        self.lens = torch.tensor([MB * BS - 37 * (i % 5) for i in range(b)], dtype=torch.int32, device="cuda")
        self.size = pa.pa_splitkv_workspace_bytes(b, HQ, D, num_splits or (
            pa.pa_auto_num_splits(b, HQ, kv_heads, D, MB, BS) if plain
            else pa.pa_scored_num_splits(b, 1, HQ, kv_heads, D, MB, BS, window=window)))

    def __call__(self, ws):
        out, lse = torch.full_like(self.q, 7.0), torch.full((self.b, HQ), 7.0, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        kw = dict(num_splits=self.splits, workspace=ws, status=status)
        scale = 1.0 / math.sqrt(D)
        if self.plain and self.fp8:
            pa.pa_decode_splitkv_fp8(out, lse, self.q, *self.pools, 1.0, 1.0, self.tables, self.lens, scale, **kw)
        elif self.plain:
            pa.pa_decode_splitkv(out, lse, self.q, *self.pools, self.tables, self.lens, scale, **kw)
        elif self.fp8:
            pa.pa_decode_scored_fp8(out, lse, self.q, *self.pools, 1.0, 1.0, self.tables, self.lens, scale,
                                    window=self.window, **kw)
        else:
            pa.pa_decode_scored(out, lse, self.q, *self.pools, self.tables, self.lens, scale, window=self.window, **kw)
        torch.cuda.synchronize()
        assert status.item() == 0
        return out, lse

    def alone(self):
        return self(torch.zeros(max(1, self.size), dtype=torch.uint8, device="cuda"))


@pytest.mark.gpu
def test_layers_and_batches_share_a_workspace():
    calls = [Call(b, 10 * b + i, window=w, fp8=f, plain=p, kv_heads=h, num_splits=n) for i, (b, w, f, p, h, n) in enumerate([
        (1, 0, False, False, 4, 0), (1, 1024, False, False, 4, 0), (4, 0, False, False, 4, 0), (4, 1024, False, False, 4, 0),
        (2, 0, True, False, 4, 0), (2, 300, True, False, 4, 0), (1, 0, False, True, 4, 0), (3, 0, True, True, 2, 0),
        (8, 0, False, False, 4, 0), (8, 1024, False, False, 4, 0), (1, 0, False, True, 4, 256), (2, 0, False, True, 1, 17),
        (3, 0, False, True, 4, 300)])]
    want = [c.alone() for c in calls]
    ws = torch.zeros(max(c.size for c in calls) + 100, dtype=torch.uint8, device="cuda")
    order = list(range(len(calls)))
    for i in order + order[::-1] + [0, 1, 0, 1, 3, 2, 3, 2]:
        out, lse = calls[i](ws)
        assert torch.equal(out, want[i][0]) and torch.equal(lse, want[i][1]), i
        assert int(ws[len(ws) // 256 * 256 - 4096:].count_nonzero()) == 0, i


@pytest.mark.gpu
def test_the_counters_merge_shares_too(merge_path):
    """Small split counts through the counters instead of a cluster."""
    merge_path("grid")
    calls = [Call(b, b, window=w, num_splits=n) for b, w, n in ((2, 0, 5), (3, 100, 9), (1, 0, 16), (4, 700, 3))]
    want = [c.alone() for c in calls]
    ws = torch.zeros(max(c.size for c in calls), dtype=torch.uint8, device="cuda")
    for _ in range(2):
        for c, w in zip(calls, want):
            out, lse = c(ws)
            assert torch.equal(out, w[0]) and torch.equal(lse, w[1])
