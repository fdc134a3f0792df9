"""The operators around one step of beam search over the paged KV cache, as cases to measure.

  rope      rotary positions for this step's queries and keys, with the slot-mapping write of K and V
  scored    attention over the paged cache whose scores are capped by a tanh, get a bias that grows
            with distance, a sliding window, a prefix that every query sees
  beam      the best K of beams x vocabulary continuations of every request
  fork      the sequences' block tables reordered, shared, freed, their last pages copied on write
  compact   the live pages moved to the front of the pools

``run`` computes them in plain torch operations, or, with ``own`` true, through the library's entry
points.  Both work on what ``prepare`` made.
"""
import math
import random

import torch

own = False

SCALINGS = ("none", "linear", "ntk", "yarn", "banded")
FP8 = torch.float8_e4m3fn


# ---------------------------------------------------------------------------------------------
# cases


def listed():
    return [
        # one decode step of 8 sequences of the 7B-shaped layer, q, k, v as one projection's output
        {"name": "rope-step", "op": "rope", "n": 8, "heads": 28, "kv_heads": 4, "head_dim": 128, "rot": 128,
         "layout": "half", "scaling": "none", "far": 4096, "fp8": False, "packed": True, "block_size": 16},
        # 8 prompts of 2048 tokens far into a long context, half of each head rotated, FP8 pools
        {"name": "rope-prompts-fp8", "op": "rope", "n": 16384, "heads": 16, "kv_heads": 8, "head_dim": 128, "rot": 64,
         "layout": "interleaved", "scaling": "yarn", "far": 1000000, "fp8": True, "packed": True, "block_size": 16},
        # a single user's short sequence: the latency of one call
        {"name": "scored-one-short", "op": "scored", "b": 1, "q_len": 1, "heads": 12, "kv_heads": 2, "head_dim": 128,
         "min_len": 509, "max_len": 509, "block_size": 16, "softcap": 50.0, "alibi": True, "window": 0, "prefix": 0,
         "fp8": False},
        # the 7B-shaped layer as a sliding-window layer: 1024 tokens back, the first 4 always seen
        {"name": "scored-window", "op": "scored", "b": 8, "q_len": 1, "heads": 28, "kv_heads": 4, "head_dim": 128,
         "min_len": 4096, "max_len": 4096, "block_size": 16, "softcap": 50.0, "alibi": False, "window": 1024,
         "prefix": 4, "fp8": False},
        # a serving batch of ragged lengths over FP8 pools, a distance bias on every head
        {"name": "scored-ragged-fp8", "op": "scored", "b": 64, "q_len": 1, "heads": 16, "kv_heads": 8, "head_dim": 128,
         "min_len": 1, "max_len": 8192, "block_size": 16, "softcap": 0.0, "alibi": True, "window": 0, "prefix": 0,
         "fp8": True},
        # 512-token prompt chunks whose first tokens see one another in both directions
        {"name": "scored-chunk-prefix", "op": "scored", "b": 8, "q_len": 512, "heads": 12, "kv_heads": 2,
         "head_dim": 128, "min_len": 512, "max_len": 2048, "block_size": 16, "softcap": 30.0, "alibi": False,
         "window": 0, "prefix": 700, "fp8": False},
        # one request with 4 beams, a small vocabulary
        {"name": "beam-one", "op": "beam", "groups": 1, "beams": 4, "vocab": 32000, "k": 4, "dtype": "bf16",
         "finished": 0.0, "allowed": 1.0, "first": False, "pad": 0},
        # 32 requests with 8 beams each, an odd vocabulary, some beams done, twice as many candidates as beams
        {"name": "beam-batch", "op": "beam", "groups": 32, "beams": 8, "vocab": 151937, "k": 16, "dtype": "bf16",
         "finished": 0.1, "allowed": 1.0, "first": False, "pad": 0},
        # one request's 4 beams reordered, one layer
        {"name": "fork-one", "op": "fork", "groups": 1, "beams": 4, "prompt": 300, "new": 60, "block_size": 16,
         "kv_heads": 4, "head_dim": 128, "layers": 1, "spare": 64, "fp8": False},
        # 32 requests of 8 beams, the pools of 4 layers
        {"name": "fork-batch", "op": "fork", "groups": 32, "beams": 8, "prompt": 1500, "new": 400, "block_size": 16,
         "kv_heads": 8, "head_dim": 128, "layers": 4, "spare": 1000, "fp8": False},
        # a small pool tidied
        {"name": "compact-small", "op": "compact", "b": 8, "blocks": 256, "live": 0.5, "block_size": 16,
         "kv_heads": 4, "head_dim": 128, "layers": 1, "fp8": False},
        # the pools of 4 layers after most requests have left
        {"name": "compact-large", "op": "compact", "b": 64, "blocks": 16384, "live": 0.3, "block_size": 16,
         "kv_heads": 8, "head_dim": 128, "layers": 4, "fp8": False},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(("rope", "scored", "scored", "beam", "fork", "compact"))
    if op == "rope":
        d = rng.choice((64, 128, 128))
        heads = _heads(rng, 8)
        return {"op": op, "n": _log_int(rng, 1, 262144 // max(16, heads["heads"])), "head_dim": d,
                "rot": 16 * rng.randint(1, d // 16), "layout": rng.choice(("half", "interleaved")),
                "scaling": rng.choice(SCALINGS), "far": _log_int(rng, 64, 1000000), "fp8": rng.random() < 0.4,
                "packed": rng.random() < 0.6, "block_size": rng.choice((16, 32, 256))} | heads
    if op == "scored":
        d = rng.choice((64, 128, 128, 128))
        kind = "one" if d == 64 else rng.choice(("one", "one", "few", "chunk"))
        case = {"op": op, "head_dim": d, "block_size": rng.choice((16, 16, 32, 256)), "fp8": False,
                "softcap": rng.choice((0.0, 15.0, 30.0, 50.0)), "alibi": rng.random() < 0.5,
                "window": _log_int(rng, 1, 4096) if rng.random() < 0.5 else 0,
                "prefix": _log_int(rng, 1, 1500) if rng.random() < 0.4 else 0}
        if kind == "chunk":
            case |= _heads(rng, 8) | {"b": rng.randint(1, 4), "q_len": _log_int(rng, 9, 500)}
            hi = _log_int(rng, 16, max(16, min(2500, 60000000 // (case["b"] * case["q_len"] * case["heads"]))))
        else:
            case |= _heads(rng, 8 if d == 64 else 12 if kind == "one" else 4)
            case |= {"b": _log_int(rng, 1, 64), "q_len": 1 if kind == "one" else rng.randint(2, 8)}
            case["fp8"] = d == 128 and kind == "one" and rng.random() < 0.5
            hi = _log_int(rng, 1, min(32768, 262144 * 8 // (case["b"] * case["kv_heads"])))
        lo = hi if rng.random() < 0.3 else rng.randint(1, hi)
        return case | {"min_len": lo, "max_len": hi}
    if op == "beam":
        beams = rng.randint(1, 12)
        k = beams * rng.randint(1, 2)
        dtype = rng.choice(("bf16", "bf16", "f32"))
        vocab = _log_int(rng, 50, 160000)
        groups = _log_int(rng, 1, max(1, min(32, 19000000 // (vocab * beams))))
        return {"op": op, "groups": groups, "beams": beams, "vocab": vocab, "k": k, "dtype": dtype,
                "finished": rng.choice((0.0, 0.2)), "allowed": rng.choice((1.0, 1.0, 0.01)),
                "first": rng.random() < 0.2, "pad": rng.choice((0, 0, 7))}
    if op == "fork":
        return {"op": op, "groups": _log_int(rng, 1, 24), "beams": rng.randint(1, 8), "prompt": _log_int(rng, 1, 1500),
                "new": _log_int(rng, 1, 400), "block_size": rng.choice((16, 32, 256)), "kv_heads": rng.choice((1, 2, 4)),
                "head_dim": rng.choice((64, 128)), "layers": rng.randint(1, 4), "spare": _log_int(rng, 200, 1000),
                "fp8": rng.random() < 0.4}
    return {"op": "compact", "b": _log_int(rng, 1, 64), "blocks": _log_int(rng, 3, 8000), "live": rng.uniform(0.0, 1.0),
            "block_size": rng.choice((16, 32)), "kv_heads": rng.choice((1, 2, 4)), "head_dim": rng.choice((64, 128)),
            "layers": rng.randint(1, 4), "fp8": rng.random() < 0.4}


def _heads(rng, most_group):
    hkv = rng.choice((1, 2, 3, 4, 8))
    return {"kv_heads": hkv, "heads": hkv * rng.randint(1, most_group)}


# ---------------------------------------------------------------------------------------------
# inputs


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _dev(values, dtype):
    return torch.tensor(values, dtype=dtype, device="cuda")


def _pool(gen, shape, fp8):
    """A pool of ordinary values: bf16, or one-byte e4m3 codes."""
    x = torch.randn(*shape, generator=gen, device="cuda", dtype=torch.bfloat16)
    return x.to(FP8).view(torch.uint8) if fp8 else x


def prepare(case, seed):
    return {"rope": _prepare_rope, "scored": _prepare_scored, "beam": _prepare_beam, "fork": _prepare_fork,
            "compact": _prepare_compact}[case["op"]](case, seed)


def _prepare_rope(c, seed):
    g, r = _gen(seed), random.Random(seed)
    n, hq, hkv, d, bs = c["n"], c["heads"], c["kv_heads"], c["head_dim"], c["block_size"]
    if c["packed"]:
        qkv = torch.randn(n, (hq + 2 * hkv) * d, generator=g, device="cuda").to(torch.bfloat16)
        q, k, v = (x.view(n, -1, d) for x in qkv.split([hq * d, hkv * d, hkv * d], dim=1))
    else:
        q, k, v = (torch.randn(n, h, d, generator=g, device="cuda").to(torch.bfloat16) for h in (hq, hkv, hkv))
    run_len = max(1, n // 8)  # runs of neighbouring positions: one per prompt, or a token each
    blocks_per_run = -(-run_len // bs) + 1
    runs = -(-n // run_len)
    nb = runs * blocks_per_run + 3
    ids = list(range(nb))
    r.shuffle(ids)
    pos, slots = [], []
    for j in range(runs):
        at = r.randrange(c["far"])
        mine = ids[j * blocks_per_run:(j + 1) * blocks_per_run]
        for t in range(min(run_len, n - j * run_len)):
            p = at + t
            pos.append(p)
            off = at % bs + t
            slots.append(mine[off // bs] * bs + off % bs)
    for i in range(n // 50):  # padding rows
        slots[r.randrange(n)] = -1
    s = {"case": c, "q": q, "k": k, "v": v, "positions": _dev(pos, torch.int32), "slots": _dev(slots, torch.int64),
         "k_cache": _pool(g, (nb, bs, hkv, d), c["fp8"]), "v_cache": _pool(g, (nb, bs, hkv, d), c["fp8"]),
         "k_scale": 0.03125, "v_scale": 0.0234375}
    s["q_out"] = torch.empty(n, hq, d, dtype=torch.bfloat16, device="cuda")
    if own:  # the plan that a program keeps
        from paged_kv_decode_cache_gb300 import pa
        s["rope"] = pa.pa_rope_init(c["rot"], BASE, layout=c["layout"], scaling=c["scaling"], **ROPE[c["scaling"]])
    return s


BASE = 1000000.0
ROPE = {"none": {}, "linear": {"factor": 4.0}, "ntk": {"factor": 4.0},
        "yarn": {"factor": 4.0, "original_positions": 32768.0, "low": 1.0, "high": 32.0},
        "banded": {"factor": 8.0, "original_positions": 8192.0, "low": 1.0, "high": 4.0}}


def _prepare_scored(c, seed):
    g, r = _gen(seed), random.Random(seed)
    b, ql, hq, hkv, d, bs = (c[k] for k in ("b", "q_len", "heads", "kv_heads", "head_dim", "block_size"))
    lens = [r.randint(c["min_len"], c["max_len"]) for _ in range(b)]
    lens[0] = c["max_len"]
    mb = -(-c["max_len"] // bs)
    nbs = [-(-x // bs) for x in lens]
    nb = sum(nbs) + 2
    ids = list(range(nb))
    r.shuffle(ids)
    tables, at = [], 0
    for x in nbs:
        tables.append(ids[at:at + x] + [-1] * (mb - x))
        at += x
    q = torch.randn(b, ql, hq, d, generator=g, device="cuda").mul_(3.0).to(torch.bfloat16)
    s = {"case": c, "q": q if ql > 1 else q.view(b, hq, d), "k_cache": _pool(g, (nb, bs, hkv, d), c["fp8"]),
         "v_cache": _pool(g, (nb, bs, hkv, d), c["fp8"]), "tables": _dev(tables, torch.int32),
         "lens": _dev(lens, torch.int32), "scale": 1.0 / math.sqrt(d), "k_scale": 1.0, "v_scale": 0.75,
         "slopes": None, "prefix": None}
    if c["alibi"]:
        s["slopes"] = _dev([2.0 ** (-8.0 * (h + 1) / hq) for h in range(hq)], torch.float32)
    if c["prefix"]:
        s["prefix"] = _dev([r.randint(0, c["prefix"]) for _ in range(b)], torch.int32)
    s["out"], s["lse"] = torch.empty_like(s["q"]), torch.empty(s["q"].shape[:-1], dtype=torch.float32, device="cuda")
    if own:  # the workspace that a program keeps
        from paged_kv_decode_cache_gb300 import pa
        s["splits"] = pa.pa_scored_num_splits(b, ql, hq, hkv, d, mb, bs, window=c["window"], max_prefix=c["prefix"])
        size = pa.pa_splitkv_workspace_bytes(b * ql, hq, d, s["splits"])
        s["workspace"] = torch.zeros(max(1, size), dtype=torch.uint8, device="cuda")
    return s


def _prepare_beam(c, seed):
    g, r = _gen(seed), random.Random(seed)
    rows, v = c["groups"] * c["beams"], c["vocab"]
    dtype = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
    x = torch.randn(rows, v + c["pad"], generator=g, device="cuda").mul_(2.5)
    x[torch.rand(x.shape, generator=g, device="cuda") >= c["allowed"]] = -math.inf  # a grammar's mask
    cum = torch.rand(c["groups"], c["beams"], generator=g, device="cuda").mul_(-6.0)
    if c["first"]:  # the prompt's last token: only the first beam lives
        cum[:, 1:] = -math.inf
    fin = torch.rand(c["groups"], c["beams"], generator=g, device="cuda") < c["finished"]
    s = {"case": c, "logits": x.to(dtype)[:, :v], "cum": cum, "finished": fin.to(torch.uint8) if c["finished"] else None,
         "eos": r.randrange(v)}
    k = c["k"]
    s["scores"] = torch.empty(c["groups"], k, dtype=torch.float32, device="cuda")
    s["tokens"] = torch.empty(c["groups"], k, dtype=torch.int32, device="cuda")
    s["parents"] = torch.empty(c["groups"], k, dtype=torch.int32, device="cuda")
    if own:
        from paged_kv_decode_cache_gb300 import pa
        size = pa.pa_beam_workspace_bytes(c["groups"], c["beams"], v, k, dtype)
        s["workspace"] = torch.zeros(max(1, size), dtype=torch.uint8, device="cuda")
    return s


def _prepare_fork(c, seed):
    g, r = _gen(seed), random.Random(seed)
    bs, rows = c["block_size"], c["groups"] * c["beams"]
    lens, tables, at, held = [], [], 0, []
    mb = -(-(c["prompt"] + c["new"]) // bs) + 1
    for _ in range(c["groups"]):
        prompt, new = r.randint(1, c["prompt"]), r.randint(0, c["new"])
        if r.random() < 0.2:  # the last page is full
            new += -(prompt + new) % bs
        new = min(new, mb * bs - prompt)
        common = prompt // bs
        shared = list(range(at, at + common))
        at += common
        if r.random() < 0.5:
            held += shared  # a prefix cache holds the prompt's pages
        for _ in range(c["beams"]):
            mine = -(-(prompt + new) // bs) - common
            tables.append(shared + list(range(at, at + mine)))
            at += mine
            lens.append(prompt + new)
    nb = c["groups"] * (c["prompt"] // bs + c["beams"] * (c["new"] // bs + 3)) + c["spare"]
    ids = list(range(nb))
    r.shuffle(ids)
    refs = [0] * nb
    for x in [t for row in tables for t in row] + held:
        refs[ids[x]] += 1
    tables = [[ids[x] for x in row] + [-1] * (mb - len(row)) for row in tables]
    parents = []
    for j in range(c["groups"]):
        done = r.random() < 0.1  # a finished request frees its pages
        for _ in range(c["beams"]):
            parents.append(-1 if done else j * c["beams"] + min(r.randrange(c["beams"]), r.randrange(c["beams"])))
    pools = _pool(g, (2 * c["layers"], nb, bs, c["kv_heads"], c["head_dim"]), c["fp8"])
    i32 = {"dtype": torch.int32, "device": "cuda"}
    s = {"case": c, "pools": pools, "tables": _dev(tables, torch.int32), "lens": _dev(lens, torch.int32),
         "refs": _dev(refs, torch.int32), "parents": _dev(parents, torch.int32),
         "new_tables": torch.empty(rows, mb, **i32), "new_lens": torch.empty(rows, **i32),
         "new_refs": torch.empty(nb, **i32), "slots": torch.empty(rows, dtype=torch.int64, device="cuda")}
    if own:
        from paged_kv_decode_cache_gb300 import pa
        s["pool_set"] = pa.PoolSet(list(pools))
        s["workspace"] = torch.empty(pa.pa_fork_workspace_bytes(rows, rows, nb), dtype=torch.uint8, device="cuda")
    return s


def _prepare_compact(c, seed):
    g, r = _gen(seed), random.Random(seed)
    nb, bs, b = c["blocks"], c["block_size"], c["b"]
    live = r.sample(range(nb), int(c["live"] * nb))
    refs = [0] * nb
    per = max(1, len(live) // b)
    mb = per + 2
    tables, lens = [], []
    for j in range(b):
        row = live[j * per:(j + 1) * per]
        if row and j and r.random() < 0.3:  # a page shared with the sequence before
            row[0] = live[(j - 1) * per]
        tables.append(row + [-1] * (mb - len(row)))
        lens.append(max(0, len(row) * bs - r.randrange(bs)))
        for x in row:
            refs[x] += 1
    for x in live:
        refs[x] = max(refs[x], 1)  # what no table names is held by a prefix cache
    pools = _pool(g, (2 * c["layers"], nb, bs, c["kv_heads"], c["head_dim"]), c["fp8"])
    i32 = {"dtype": torch.int32, "device": "cuda"}
    s = {"case": c, "pools": pools, "tables": _dev(tables, torch.int32), "lens": _dev(lens, torch.int32),
         "refs": _dev(refs, torch.int32), "new_tables": torch.empty(b, mb, **i32), "new_refs": torch.empty(nb, **i32),
         "remap": torch.empty(nb, **i32), "n_live": torch.empty(1, **i32)}
    if own:
        from paged_kv_decode_cache_gb300 import pa
        s["pool_set"] = pa.PoolSet(list(pools))
        s["workspace"] = torch.empty(pa.pa_compact_workspace_bytes(nb), dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------------------------------------
# one pass


def run(s):
    op = s["case"]["op"]
    if own:
        return {"rope": _own_rope, "scored": _own_scored, "beam": _own_beam, "fork": _own_fork,
                "compact": _own_compact}[op](s)
    return {"rope": _rope, "scored": _scored, "beam": _beam, "fork": _fork, "compact": _compact}[op](s)


def _values(pool):
    return pool.view(FP8) if pool.dtype == torch.uint8 else pool


# -- rotary positions and the write


def _frequencies(c):
    """(radians per position of every pair in 64 bits, the factor on cos and sin)."""
    rot, p = c["rot"], ROPE[c["scaling"]]
    i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    base, factor = BASE, p.get("factor", 1.0)
    if c["scaling"] == "ntk" and rot > 2:
        base = base * factor ** (rot / (rot - 2.0))
    f = base ** (-2.0 * i / rot)
    if c["scaling"] == "linear":
        return f / factor, 1.0
    if c["scaling"] == "yarn":
        def dim(turns):
            return rot * math.log(p["original_positions"] / (turns * 2 * math.pi)) / (2 * math.log(BASE))
        lo, hi = max(math.floor(dim(p["high"])), 0), min(math.ceil(dim(p["low"])), rot - 1)
        ramp = ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        return f / factor * ramp + f * (1 - ramp), 0.1 * math.log(factor) + 1.0
    if c["scaling"] == "banded":
        turns = p["original_positions"] * f / (2 * math.pi)
        keep = ((turns - p["low"]) / (p["high"] - p["low"])).clamp(0, 1)
        return f / factor * (1 - keep) + f * keep, 1.0
    return f, 1.0


def _rotate(x, cos, sin, rot, layout):
    y = x.clone()
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if layout == "interleaved" else (x[..., :rot // 2], x[..., rot // 2:rot])
    u, w = a * cos - b * sin, a * sin + b * cos
    if layout == "interleaved":
        y[..., 0:rot:2], y[..., 1:rot:2] = u, w
    else:
        y[..., :rot // 2], y[..., rot // 2:rot] = u, w
    return y


def _rope(s):
    c = s["case"]
    f, m = _frequencies(c)
    angle = s["positions"].double()[:, None] * f
    cos, sin = ((t * m).float()[:, None, :] for t in (angle.cos(), angle.sin()))
    q = _rotate(s["q"].float(), cos, sin, c["rot"], c["layout"])
    k, v = _rotate(s["k"].float(), cos, sin, c["rot"], c["layout"]), s["v"].float()
    s["q_out"].copy_(q.to(torch.bfloat16))
    at = torch.nonzero(s["slots"] >= 0)[:, 0]
    to = s["slots"][at]
    for pool, x, scale in ((s["k_cache"], k, s["k_scale"]), (s["v_cache"], v, s["v_scale"])):
        rows = pool.view(-1, *pool.shape[2:])
        x = x[at]
        rows[to] = (x / scale).clamp(-448, 448).to(FP8).view(torch.uint8) if c["fp8"] else x.to(torch.bfloat16)
    return {"q": s["q_out"], "k_cache": _values(s["k_cache"]), "v_cache": _values(s["v_cache"])}


def _own_rope(s):
    from paged_kv_decode_cache_gb300 import pa
    if s["case"]["fp8"]:
        pa.pa_rope_write_fp8(s["q_out"], s["q"], s["k"], s["v"], s["positions"], s["slots"], s["k_cache"], s["v_cache"],
                             s["k_scale"], s["v_scale"], s["rope"])
    else:
        pa.pa_rope_write(s["q_out"], s["q"], s["k"], s["v"], s["positions"], s["slots"], s["k_cache"], s["v_cache"],
                         s["rope"])
    return {"q": s["q_out"], "k_cache": _values(s["k_cache"]), "v_cache": _values(s["v_cache"])}


# -- attention


def _attend(q, k, v, seen, at, slopes, cap, scale):
    """q [.., Q, G, D] of one KV head, k and v [.., T, D], seen [.., Q, T], at = t - position [.., Q, T]."""
    n, g, d = q.shape[-3:]
    x = (q.flatten(-3, -2) @ k.transpose(-1, -2)).unflatten(-2, (n, g)) * scale
    if cap:
        x = cap * torch.tanh(x / cap)
    if slopes is not None:
        x = x + slopes[..., None, :, None] * at.unsqueeze(-2)
    x = x.masked_fill(~seen.unsqueeze(-2), -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(x - m)
    total = p.sum(-1, keepdim=True)
    out = (p.flatten(-3, -2) @ v).unflatten(-2, (n, g)) / torch.where(total == 0, torch.ones_like(total), total)
    return out, (m + torch.log(total)).squeeze(-1)


def _seen(c, lens, prefix, t):
    """(which tokens t [T] the queries of sequences of these lengths see, t - position), both [B, Q, T]."""
    pos = (lens[:, None] - c["q_len"] + torch.arange(c["q_len"], device="cuda"))[..., None]
    seen = t <= pos
    if c["window"]:
        seen = seen & (t > pos - c["window"])
    if prefix is not None:
        seen = seen | (t < prefix[:, None, None])
    return seen & (t < lens[:, None, None]), (t - pos)


def _scored(s):
    c = s["case"]
    b, ql, hq, hkv, d = (c[k] for k in ("b", "q_len", "heads", "kv_heads", "head_dim"))
    ids = s["tables"].clamp(min=0).long()
    k, v = (_values(p)[ids].flatten(1, 2).float().transpose(1, 2) for p in (s["k_cache"], s["v_cache"]))
    if c["fp8"]:
        k, v = k * s["k_scale"], v * s["v_scale"]
    seen, at = _seen(c, s["lens"].long(), None if s["prefix"] is None else s["prefix"].long(),
                     torch.arange(k.shape[2], device="cuda"))
    q = s["q"].float().view(b, ql, hkv, hq // hkv, d).transpose(1, 2)
    slopes = None if s["slopes"] is None else s["slopes"].view(hkv, hq // hkv)
    out, lse = _attend(q, k, v, seen[:, None], at[:, None].float(), slopes, c["softcap"], s["scale"])
    out, lse = out.transpose(1, 2).reshape(s["q"].shape), lse.transpose(1, 2).reshape(s["lse"].shape)
    return {"out": out.to(torch.bfloat16), "lse": lse}


def _own_scored(s):
    from paged_kv_decode_cache_gb300 import pa
    c = s["case"]
    more = {"softcap": c["softcap"], "alibi_slopes": s["slopes"], "window": c["window"], "prefix_lens": s["prefix"],
            "max_prefix": c["prefix"], "num_splits": s["splits"], "workspace": s["workspace"]}
    if c["fp8"]:
        pa.pa_decode_scored_fp8(s["out"], s["lse"], s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"],
                                s["tables"], s["lens"], s["scale"], **more)
    else:
        pa.pa_decode_scored(s["out"], s["lse"], s["q"], s["k_cache"], s["v_cache"], s["tables"], s["lens"], s["scale"],
                            **more)
    return {"out": s["out"], "lse": s["lse"]}


# -- beams


def _beam(s):
    # in 64 bits: bf16 logits repeat, and scores of different beams come close to one another
    c = s["case"]
    n, w, v, k = c["groups"], c["beams"], c["vocab"], c["k"]
    x = s["logits"].double()
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    x = torch.where(x == -math.inf, x, x - (top + torch.log(torch.exp(x - top).sum(-1, keepdim=True))))
    x = x.view(n, w, v) + s["cum"].double()[..., None]
    if s["finished"] is not None:  # a finished beam has one continuation, itself
        done = s["finished"].bool()[..., None]
        is_eos = torch.arange(v, device="cuda") == s["eos"]
        x = torch.where(done, torch.where(is_eos, s["cum"].double()[..., None], -math.inf), x)
    best, at = torch.sort(x.view(n, w * v), dim=-1, descending=True, stable=True)
    best, at = best[:, :k], at[:, :k]
    none = best == -math.inf
    first = torch.arange(n, device="cuda")[:, None] * w
    tokens = torch.where(none, -1, at % v).to(torch.int32)
    parents = torch.where(none, -1, first + at // v).to(torch.int32)
    return {"scores": best.float(), "tokens": tokens, "parents": parents}


def _own_beam(s):
    from paged_kv_decode_cache_gb300 import pa
    pa.pa_beam_select(s["scores"], s["tokens"], s["parents"], s["logits"], s["cum"], finished=s["finished"],
                      eos=s["eos"] if s["finished"] is not None else -1, workspace=s["workspace"])
    return {"scores": s["scores"], "tokens": s["tokens"], "parents": s["parents"]}


# -- pages


def _count(ids, valid, blocks):
    return torch.zeros(blocks, dtype=torch.int64, device="cuda").index_add_(
        0, torch.where(valid, ids, 0).flatten().long(), valid.flatten().long())


def _lowest(free):
    """The ids where `free` is true, ascending, then ids past the end."""
    n = free.numel()
    return torch.sort(torch.where(free, torch.arange(n, device="cuda"), n)).values


def _fork(s):
    c = s["case"]
    tables, lens, refs, bs = s["tables"].long(), s["lens"].long(), s["refs"].long(), c["block_size"]
    rows, mb, nb = tables.shape[0], tables.shape[1], refs.numel()
    i, j = torch.arange(rows, device="cuda"), torch.arange(mb, device="cuda")
    parent = s["parents"].long()
    alive = parent >= 0
    p = parent.clamp(min=0)
    length = torch.where(alive, lens[p], 0)
    used = -(-length // bs)
    new = torch.where(j < used[:, None], tables[p], -1)
    held = refs - _count(tables, j < -(-lens[:, None] // bs), nb)  # references that no old table makes
    now = held + _count(new, new >= 0, nb)
    part = alive & (length % bs != 0)
    tail = torch.where(part, new.gather(1, (used - 1).clamp(min=0)[:, None])[:, 0], -1)
    same = (tail[:, None] == tail[None, :]) & part[:, None]
    alone = same.sum(1) == now[tail.clamp(min=0)]  # every reference to it is a tail
    keeps = part & alone & ~(same & (i[None, :] < i[:, None])).any(1)
    grow = alive & (length % bs == 0)
    need = grow | (part & ~keeps)
    ids = torch.cat([_lowest(now == 0), torch.full((rows,), nb, device="cuda")])[need.long().cumsum(0) - 1]
    at = torch.where(grow, used, used - 1).clamp(min=0, max=mb - 1)
    last = torch.where(need, ids, torch.where(alive, new.gather(1, at[:, None])[:, 0], -1))
    new = torch.where(need[:, None] & (j == at[:, None]), ids[:, None], new)
    now = now + _count(ids, need, nb) - _count(tail, part & ~keeps, nb)
    slots = torch.where(alive, last * bs + length % bs, -1)
    copies = torch.nonzero(part & ~keeps)[:, 0]
    src, dst = tail[copies], ids[copies]
    ours = (torch.arange(bs, device="cuda") < (length % bs)[copies][:, None])[None, :, :, None, None]
    s["pools"][:, dst] = torch.where(ours, s["pools"][:, src], s["pools"][:, dst])
    i32 = torch.int32
    return {"tables": new.to(i32), "lens": length.to(i32), "refs": now.to(i32), "slots": slots,
            "pools": _values(s["pools"])}


def _own_fork(s):
    from paged_kv_decode_cache_gb300 import pa
    pa.pa_sequences_fork(s["new_tables"], s["new_lens"], s["new_refs"], s["slots"], s["tables"], s["lens"], s["refs"],
                         s["parents"], s["pool_set"], s["workspace"])
    return {"tables": s["new_tables"], "lens": s["new_lens"], "refs": s["new_refs"], "slots": s["slots"],
            "pools": _values(s["pools"])}


def _compact(s):
    c = s["case"]
    tables, refs, bs = s["tables"].long(), s["refs"].long(), c["block_size"]
    nb = refs.numel()
    ids = torch.arange(nb, device="cuda")
    live = refs > 0
    n_live = live.sum()
    mover, hole = live & (ids >= n_live), ~live & (ids < n_live)
    to = _lowest(hole)[(mover.long().cumsum(0) - 1).clamp(min=0)]
    remap = torch.where(live, torch.where(mover, to, ids), -1)
    used = torch.arange(tables.shape[1], device="cuda") < -(-s["lens"].long()[:, None] // bs)
    new = torch.where(used, remap[tables.clamp(min=0)], -1)
    src = torch.nonzero(live)[:, 0]
    now = torch.zeros_like(refs)
    now[remap[src]] = refs[src]
    src = torch.nonzero(mover)[:, 0]
    s["pools"][:, remap[src]] = s["pools"][:, src]
    i32 = torch.int32
    return {"tables": new.to(i32), "refs": now.to(i32), "remap": remap.to(i32), "n_live": n_live.to(i32).view(1),
            "pools": _values(s["pools"])}


def _own_compact(s):
    from paged_kv_decode_cache_gb300 import pa
    pa.pa_blocks_compact(s["new_tables"], s["new_refs"], s["remap"], s["n_live"], s["tables"], s["lens"], s["refs"],
                         s["pool_set"], s["workspace"])
    return {"tables": s["new_tables"], "refs": s["new_refs"], "remap": s["remap"], "n_live": s["n_live"],
            "pools": _values(s["pools"])}


# ---------------------------------------------------------------------------------------------
# what a pass cannot do without, and its outputs in 64 bits


def work(c):
    if c["op"] == "rope":
        row = c["head_dim"] * (c["heads"] * 4 + 2 * c["kv_heads"] * (3 if c["fp8"] else 4)) + 12
        return {"bytes": c["n"] * row, "flops": 3 * c["n"] * c["rot"] * (c["heads"] + c["kv_heads"])}
    if c["op"] == "scored":
        mean = 0.5 * (c["min_len"] + c["max_len"])
        one = c["min_len"] == c["max_len"]
        keys = min(mean, c["window"] + (c["q_len"] - 1) + 0.5 * c["prefix"]) if c["window"] else mean
        pairs = keys * c["q_len"]
        if c["q_len"] > 1 and not c["window"]:  # causal: on average half of the new tokens are unseen
            pairs = max(mean - 0.5 * c["q_len"], 0.5 * mean) * c["q_len"]
        kv = 2 * c["kv_heads"] * c["head_dim"] * (1 if c["fp8"] else 2)
        q = c["q_len"] * c["heads"] * (4 * c["head_dim"] + 4)
        return {"bytes": int(c["b"] * (keys * kv + q)) if not one else c["b"] * (int(keys) * kv + q),
                "flops": int(4 * c["b"] * c["heads"] * c["head_dim"] * pairs)}
    if c["op"] == "beam":
        rows = c["groups"] * c["beams"]
        return {"bytes": rows * c["vocab"] * (2 if c["dtype"] == "bf16" else 4) + rows * 5 + c["groups"] * c["k"] * 12,
                "flops": 4 * rows * c["vocab"]}
    token = 2 * c["layers"] * c["kv_heads"] * c["head_dim"] * (1 if c["fp8"] else 2)
    if c["op"] == "fork":
        rows, mean = c["groups"] * c["beams"], 0.5 * (c["prompt"] + c["new"])
        entries = rows * mean / c["block_size"]
        return {"bytes": int(0.3 * rows * c["block_size"] * token + 8 * entries + 24 * rows), "flops": 0}
    moved = c["blocks"] * c["live"] * (1 - c["live"])
    return {"bytes": int(2 * moved * c["block_size"] * token + 12 * c["blocks"] + 8 * c["blocks"] * c["live"]), "flops": 0}


def exact(c, seed):
    """The computed numbers in 64 bits, from the definitions; None for the pages, which are only moved."""
    if c["op"] == "rope":
        return _exact_rope(c, seed)
    if c["op"] == "scored":
        return _exact_scored(c, seed)
    if c["op"] == "beam":
        return _exact_beam(c, seed)
    return None


def _exact_rope(c, seed):
    s = prepare(c, seed)
    f, m = _frequencies(c)
    rot, half = c["rot"], c["rot"] // 2
    # every pair as a complex number, turned by exp(i angle)
    order = torch.arange(rot, device="cuda").view(half, 2) if c["layout"] == "interleaved" else \
        torch.arange(rot, device="cuda").view(2, half).t()
    turn = m * torch.exp(1j * s["positions"].double()[:, None, None] * f)

    def turned(x):
        y = x.double()
        z = torch.complex(y[..., order[:, 0]], y[..., order[:, 1]]) * turn
        y[..., order[:, 0]], y[..., order[:, 1]] = z.real, z.imag
        return y

    out = {"q": turned(s["q"])}
    at = s["slots"] >= 0
    for name, x, scale in (("k_cache", turned(s["k"]), s["k_scale"]), ("v_cache", s["v"].double(), s["v_scale"])):
        pool = _values(s[name]).double()
        x = (x / scale).clamp(-448, 448) if c["fp8"] else x
        pool.view(-1, *pool.shape[2:])[s["slots"][at]] = x[at]
        out[name] = pool
    return out


def _exact_scored(c, seed):
    if 4 * c["b"] * c["q_len"] * c["heads"] * c["max_len"] * c["head_dim"] > 4e11:
        return None
    s = prepare(c, seed)
    hkv, bs = c["kv_heads"], c["block_size"]
    out, lse = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda"), \
        torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
    q = s["q"].double().view(c["b"], c["q_len"], hkv, -1, c["head_dim"])
    group = q.shape[3]
    slopes = torch.zeros(hkv, group, dtype=torch.float64, device="cuda") if s["slopes"] is None else \
        s["slopes"].double().view(hkv, group)
    o, z = out.view(q.shape), lse.view(q.shape[:-1])
    for b, length in enumerate(s["lens"].tolist()):
        t = torch.arange(length, device="cuda")
        where = s["tables"][b].long()[t // bs] * bs + t % bs
        k, v = (_values(s[n]).flatten(0, 1)[where].double() for n in ("k_cache", "v_cache"))
        if c["fp8"]:
            k, v = k * s["k_scale"], v * s["v_scale"]
        pos = length - c["q_len"] + torch.arange(c["q_len"], device="cuda")[:, None]
        ok = (t <= pos) & ((t > pos - c["window"]) if c["window"] else (t >= 0))
        if s["prefix"] is not None:
            ok |= t < s["prefix"][b]
        for h in range(hkv):
            x = torch.einsum("qgd,td->gqt", q[b, :, h], k[:, h]) * s["scale"]
            if c["softcap"]:
                x = c["softcap"] * torch.tanh(x / c["softcap"])
            x = x + slopes[h][:, None, None] * (t - pos)
            x = torch.where(ok, x, -math.inf)
            z[b, :, h] = torch.logsumexp(x, -1).t()
            w = torch.exp(x - torch.where(ok.any(-1), torch.logsumexp(x, -1), 0.0)[..., None])
            o[b, :, h] = torch.einsum("gqt,td->qgd", w, v[:, h])
    return {"out": out, "lse": lse}


def _exact_beam(c, seed):
    s = prepare(c, seed)
    n, w = c["groups"], c["beams"]
    scores = torch.full((n, c["k"]), -math.inf, dtype=torch.float64, device="cuda")
    for g in range(n):
        found = []
        for b in range(w):
            cum = s["cum"][g, b].double()
            if s["finished"] is not None and bool(s["finished"][g, b]):
                found.append(cum[None])
                continue
            x = s["logits"][g * w + b].double()
            x = x[x > -math.inf]
            if x.numel():
                found.append(torch.topk(x, min(c["k"], x.numel())).values - torch.logsumexp(x, 0) + cum)
        if found:
            best = torch.cat(found).sort(descending=True).values[:c["k"]]
            scores[g, :best.numel()] = best
    return {"scores": scores, "tokens": None, "parents": None}
