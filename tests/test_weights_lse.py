"""Which attention's lse pa_weights_add takes: with that of every call that its documentation names, a query's weights sum to
one; with one of other scores or of fewer tokens they do not."""
import re

import pytest
import torch

from paged_kv_decode_cache_gb300 import build as B
from paged_kv_decode_cache_gb300 import pa
from paged_model import i32, layout

LENS, HQ, HKV, D, BS, QLEN, SCALE = [300, 33, 77], 8, 2, 128, 16, 3, 128 ** -0.5
KS, VS = 0.5, 0.75


@pytest.fixture(scope="module", autouse=True)
def _built():
    B.build()


def named():
    """The calls whose lse fits, and those whose lse does not."""
    fits, others = re.sub(r"\s+", " ", pa.pa_weights_add.__doc__).split("not that of")
    names = [set(re.findall(r"pa_decode\w*", x)) for x in (fits, others)]
    return names[0], names[1]


CALLS = {
    "pa_decode": lambda s: pa.pa_decode(*s["one"], *s["kv"], *s["rows"], SCALE),
    "pa_decode_splitkv": lambda s: pa.pa_decode_splitkv(*s["one"], *s["kv"], *s["rows"], SCALE, workspace=s["ws"]),
    "pa_decode_step": lambda s: pa.pa_decode_step(*s["one"], *s["new"], *s["kv"], *s["rows"], SCALE, workspace=s["ws"]),
    "pa_decode_cascade": lambda s: pa.pa_decode_cascade(*s["one"], *s["kv"], 2, *s["rows"], SCALE, workspace=s["ws"]),
    "pa_decode_mq": lambda s: pa.pa_decode_mq(*s["more"], *s["kv"], *s["rows"], SCALE, workspace=s["ws"]),
    "pa_decode_splitkv_fp8": lambda s: pa.pa_decode_splitkv_fp8(*s["one"], *s["kv"], KS, VS, *s["rows"], SCALE, workspace=s["ws"]),
    "pa_decode_step_fp8": lambda s: pa.pa_decode_step_fp8(*s["one"], *s["new"], *s["kv"], KS, VS, *s["rows"], SCALE,
                                                          workspace=s["ws"]),
    "pa_decode_scored": lambda s: pa.pa_decode_scored(*s["more"], *s["kv"], *s["rows"], SCALE, workspace=s["ws"]),
    "pa_decode_scored_fp8": lambda s: pa.pa_decode_scored_fp8(*s["more"], *s["kv"], KS, VS, *s["rows"], SCALE, workspace=s["ws"]),
}


def state(fp8):
    g = torch.Generator(device="cuda").manual_seed(3)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)   # noqa: E731
    tables, _, nb = layout(LENS, BS, 1, shared=2)
    t, n = i32(tables), i32(LENS)
    kv = [rnd(nb, BS, HKV, D) for _ in range(2)]
    if fp8:
        kv = [x.to(torch.float8_e4m3fn).view(torch.uint8) for x in kv]
    slots = torch.tensor([tables[b][(x - 1) // BS] * BS + (x - 1) % BS for b, x in enumerate(LENS)], device="cuda")
    q = rnd(len(LENS), QLEN, HQ, D) * 2
    q1 = q[:, -1].contiguous()
    return dict(kv=kv, rows=[t, n], new=[rnd(len(LENS), HKV, D), rnd(len(LENS), HKV, D), slots],
                one=[torch.empty_like(q1), torch.empty(len(LENS), HQ, device="cuda"), q1],
                more=[torch.empty_like(q), torch.empty(len(LENS), QLEN, HQ, device="cuda"), q],
                ws=torch.zeros(1 << 24, dtype=torch.uint8, device="cuda"))


def sums(s, fp8, q, lse):
    """What every sequence and KV head's tokens draw in all."""
    w = torch.zeros(len(LENS), HKV, s["rows"][0].shape[1] * BS, device="cuda")
    if fp8:
        pa.pa_weights_add_fp8(w, w, None, q, lse, s["kv"][0], KS, *s["rows"], SCALE)
    else:
        pa.pa_weights_add(w, w, None, q, lse, s["kv"][0], *s["rows"], SCALE)
    return w.double().sum(-1).cpu()


def test_the_documentation_names_them():
    fits, others = named()
    assert fits == set(CALLS) and others == {"pa_decode_scored", "pa_decode_selected"}


@pytest.mark.gpu
@pytest.mark.parametrize("name", list(CALLS))
def test_weights_of_a_call_sum_to_its_queries(name):
    fp8 = name.endswith("_fp8")
    s = state(fp8)
    CALLS[name](s)
    _, lse, q = s["more" if name in ("pa_decode_mq", "pa_decode_scored", "pa_decode_scored_fp8") else "one"]
    queries = HQ // HKV * (q.shape[1] if q.dim() == 4 else 1)
    # (lse and every weight are good to 2^-13)
    assert ((sums(s, fp8, q, lse) - queries).abs() <= queries * 2.0 ** -12).all()


@pytest.mark.gpu
def test_weights_under_rules_or_lists_do_not():
    """Why those are named: nothing in the call could tell."""
    s = state(False)
    out, lse, q = s["one"]
    G = HQ // HKV
    pa.pa_decode_scored(out, lse, q, *s["kv"], *s["rows"], SCALE, softcap=1.0, workspace=s["ws"])
    assert ((sums(s, False, q, lse) - G).abs() > 0.01 * G).any()
    sel, n = i32([[row[:2].tolist()] * HKV for row in s["rows"][0]]).contiguous(), i32([[2 * BS] * HKV] * len(LENS))
    pa.pa_decode_selected(out, lse, q, *s["kv"], sel, n, SCALE, workspace=s["ws"])
    assert (sums(s, False, q, lse)[0] > 1.5 * G).all()      # (32 tokens of 300)
