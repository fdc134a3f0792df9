"""What no query sees leaves no trace in pa_decode_scored's results: they are a function of the seen
rows alone, to the last bit, whatever the unseen rows of the pools hold and whatever an earlier launch
left in shared memory and in the tensor memory."""
import math

import pytest
import torch

from test_scored import FP8, _built, inputs, run, slopes_of  # noqa: F401

CASES = {
    "one token": dict(Bn=3, Q=1, Hq=12, Hkv=2, D=128, lens=[509, 150, 17]),
    "one token, one sequence": dict(Bn=1, Q=1, Hq=12, Hkv=2, D=128, lens=[509]),
    "one token, a window": dict(Bn=3, Q=1, Hq=28, Hkv=4, D=128, lens=[509, 150, 17], window=41),
    "one token, fp8": dict(Bn=3, Q=1, Hq=16, Hkv=8, D=128, lens=[509, 150, 17], fp8=True),
    "one token, D 64": dict(Bn=3, Q=1, Hq=8, Hkv=2, D=64, lens=[509, 150, 17]),
    "a few tokens": dict(Bn=3, Q=4, Hq=16, Hkv=8, D=128, lens=[300, 61, 5]),
    "a few tokens, fp8": dict(Bn=3, Q=4, Hq=16, Hkv=8, D=128, lens=[300, 61, 5], fp8=True),
    "a chunk": dict(Bn=2, Q=50, Hq=12, Hkv=2, D=128, lens=[333, 77]),
    "a chunk, a window": dict(Bn=2, Q=50, Hq=12, Hkv=2, D=128, lens=[333, 77], window=30),
}


def filled(pools, rows, fp8, value):
    """The pools with every value of `rows` (never seen ones) replaced."""
    out = []
    for p in pools:
        p = p.clone()
        flat = p.flatten(0, 1)
        if fp8:
            flat[rows] = torch.tensor(value, dtype=torch.float32).to(FP8).view(torch.uint8).item()
        else:
            flat[rows] = value
        out.append(p)
    return out


@pytest.mark.gpu
@pytest.mark.parametrize("softcap", [2.0, 30.0])
@pytest.mark.parametrize("name", CASES)
def test_unseen_rows_leave_no_trace(name, softcap):
    c = dict(CASES[name])
    fp8, window = c.pop("fp8", False), c.pop("window", 0)
    q, pools, tables, L = inputs(c["Bn"], c["Q"], c["Hq"], c["Hkv"], c["D"], 16, c["lens"], fp8, 11, sharp=1.0,
                                 window=window)
    values = pools[0].view(FP8).float() if fp8 else pools[0].float()
    unseen = values.isnan().flatten(0, 1).flatten(1).all(1)
    assert unseen.any() and not unseen.all()
    scale, rules = 1.0 / math.sqrt(c["D"]), dict(softcap=softcap, window=window, alibi_slopes=slopes_of(c["Hq"]))
    for splits in (1, 3, 0):
        seen_first = None
        for value in (math.nan, 0.0, 300.0, -300.0):
            mine = filled(pools, unseen, fp8, value)
            # an earlier launch of the same kernel over full tables, which leaves other scores behind
            full = [torch.full_like(p, 0x30 if fp8 else 1.0) if value == 0.0 else filled([p], unseen, fp8, 1.0)[0]
                    for p in pools]
            run(q * (0.01 if value == 0.0 else 400.0), full, tables.clamp(min=0), L.clamp(min=tables.shape[1] * 16), scale,
                splits, fp8, softcap=0.0)
            got = run(q, mine, tables, L, scale, splits, fp8, **rules)
            seen_first = seen_first or got
            assert torch.equal(got[0], seen_first[0]) and torch.equal(got[1], seen_first[1]), (splits, value)


@pytest.mark.gpu
def test_a_score_does_not_depend_on_its_neighbours():
    """One key whose score lies past the cap's small range, beside keys of small scores: the small ones
    keep the relative error of the small range (2^-21), with a cap of 4096 far below the 2^-22 of the
    cap (2^-10) that the form for large scores has.  Head 0 meets the large score, head 1 only small ones."""
    D, n = 128, 16
    k = torch.zeros(1, n, 1, D)
    k[0, :, 0, 0] = torch.linspace(-2.0, 2.0, n)      # head 1's scores
    k[0, 5, 0, 1] = 3500.0                            # head 0's large one
    q = torch.zeros(1, 1, 2, D)
    q[0, 0, 0, 1] = 1.0
    q[0, 0, 1, 0] = 1.0
    pools = [k.to(torch.bfloat16).cuda(), torch.randn(1, n, 1, D, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()]
    tables, L = torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.tensor([n], dtype=torch.int32, device="cuda")
    out, lse = run(q.to(torch.bfloat16).cuda(), pools, tables, L, 1.0, 1, False, softcap=4096.0)
    s = 4096.0 * torch.tanh(pools[0].double().cpu()[0, :, 0, 0] / 4096.0)
    # scores below 2 with an error of 2^-21 of themselves, and lse's own 2^-21 (its sum's and its logarithm's)
    assert abs(lse.double().cpu()[0, 0, 1] - torch.logsumexp(s, 0)) <= 2.0 ** -19
