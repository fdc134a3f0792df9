"""What a long context costs a decode step, cut down: operators over the paged KV cache, as cases to measure.

  bounds   every channel's least and largest key of each block that new tokens were written to
  select   the blocks whose bounds promise a query the largest scores, for every sequence and KV head
  attend   attention over blocks that differ from KV head to KV head
  weights  the attention weight that every cached token has drawn, accumulated over queries
  evict    the tokens that drew the least thrown out, the rest moved together, their blocks given back

``run`` computes them in plain torch operations, or, with ``own`` true, through the library's entry
points.  Both work on what ``prepare`` made.
"""
import math
import random

import torch

own = False

FP8 = torch.float8_e4m3fn


# ---------------------------------------------------------------------------------------------
# cases


def listed():
    return [
        # one decode step of 8 sequences of the 7B-shaped layer: the one block that each has written to
        {"name": "bounds-step", "op": "bounds", "b": 8, "kv_heads": 4, "head_dim": 128, "min_len": 4000, "max_len": 4096,
         "new": 1, "block_size": 16, "fp8": False},
        # the bounds of 16 whole prompts, once after they were read in
        {"name": "bounds-prompts", "op": "bounds", "b": 16, "kv_heads": 8, "head_dim": 128, "min_len": 2048,
         "max_len": 16384, "new": 0, "block_size": 16, "fp8": False},
        # a single user's context of the 1.5B-shaped layer: the latency of one call
        {"name": "select-one", "op": "select", "b": 1, "kv_heads": 2, "heads": 12, "head_dim": 128, "min_len": 16389,
         "max_len": 16389, "block_size": 16, "keep": 64, "first": 1, "last": 2, "fp8": False},
        # 8 long contexts of the 7B-shaped layer, 2048 of 32768 tokens each
        {"name": "select-long", "op": "select", "b": 8, "kv_heads": 4, "heads": 28, "head_dim": 128, "min_len": 32000,
         "max_len": 32768, "block_size": 16, "keep": 128, "first": 1, "last": 4, "fp8": False},
        # a ragged batch up to 128k tokens, bounds of FP8 pools
        {"name": "select-ragged-fp8", "op": "select", "b": 16, "kv_heads": 8, "heads": 16, "head_dim": 128,
         "min_len": 1000, "max_len": 131072, "block_size": 16, "keep": 256, "first": 4, "last": 8, "fp8": True},
        # the attention of select-one: 64 blocks per KV head
        {"name": "attend-one", "op": "attend", "b": 1, "kv_heads": 2, "heads": 12, "head_dim": 128, "min_len": 16389,
         "max_len": 16389, "block_size": 16, "keep": 64, "fp8": False},
        # a full batch of the 0.6B-shaped layer over FP8 pools, 2048 tokens per KV head
        {"name": "attend-batch-fp8", "op": "attend", "b": 64, "kv_heads": 8, "heads": 16, "head_dim": 128,
         "min_len": 1500, "max_len": 32768, "block_size": 16, "keep": 128, "fp8": True},
        # the weights of one decode step of the 7B-shaped layer
        {"name": "weights-step", "op": "weights", "b": 8, "q_len": 1, "kv_heads": 4, "heads": 28, "head_dim": 128,
         "min_len": 4000, "max_len": 4096, "block_size": 16, "decay": 1.0, "fp8": False},
        # the same for a ragged batch over FP8 pools, older weights fading
        {"name": "weights-ragged-fp8", "op": "weights", "b": 32, "q_len": 1, "kv_heads": 8, "heads": 16, "head_dim": 128,
         "min_len": 500, "max_len": 16384, "block_size": 16, "decay": 0.9375, "fp8": True},
        # a prompt's last 32 queries over all of it, before what they do not look at is thrown out
        {"name": "weights-window", "op": "weights", "b": 4, "q_len": 32, "kv_heads": 4, "heads": 28, "head_dim": 128,
         "min_len": 32000, "max_len": 32768, "block_size": 16, "decay": 1.0, "fp8": False},
        # a layer's budget of 1024 tokens, 64 over it, in sequences that have been cut before
        {"name": "evict-step", "op": "evict", "layers": 1, "b": 8, "kv_heads": 4, "head_dim": 128, "min_len": 1088,
         "max_len": 1088, "block_size": 16, "budget": 1024, "first": 4, "recent": 128, "shared": 0, "again": True,
         "fp8": False},
        # prompts of up to 16384 tokens behind a shared instruction, cut to 2048 in 8 layers
        {"name": "evict-prompts-fp8", "op": "evict", "layers": 8, "b": 4, "kv_heads": 8, "head_dim": 128, "min_len": 8000,
         "max_len": 16384, "block_size": 16, "budget": 2048, "first": 4, "recent": 256, "shared": 4, "again": False,
         "fp8": True},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("bounds", "select", "select", "attend", "weights", "weights", "evict"))
    hkv = rng.choice((1, 2, 3, 4, 8))
    c = {"op": op, "kv_heads": hkv, "head_dim": rng.choice((64, 128, 128)), "fp8": rng.random() < 0.4,
         "block_size": rng.choice((16, 16, 32, 64, 256)), "b": _log_int(rng, 1, 32)}
    if op == "evict":
        c["layers"] = rng.randint(1, 4)
    if op == "weights":
        c["heads"] = hkv * rng.randint(1, 8)
        c["q_len"] = 1 if rng.random() < 0.5 else _log_int(rng, 2, 48)
    most = min(131072, 900000 // (c["b"] * hkv * c.get("layers", 1)))
    if op == "weights":
        most = max(1, min(most, 110000000 // (c["b"] * c["heads"] * c["q_len"])))
    hi = _log_int(rng, 1, most)
    lo = hi if rng.random() < 0.3 else rng.randint(1, hi)
    c |= {"min_len": lo, "max_len": hi}
    if op == "bounds":
        return c | {"new": rng.choice((0, 1, 1, _log_int(rng, 1, 2000)))}
    if op == "weights":
        return c | {"decay": rng.choice((1.0, 1.0, 0.875))}
    blocks = -(-hi // c["block_size"])
    if op == "select":
        c["heads"] = hkv * rng.randint(1, 12)
        first, last = rng.choice((0, 1, 4)), rng.choice((1, 2, 8))
        return c | {"first": first, "last": last, "keep": first + last + _log_int(rng, 1, max(1, blocks // 2))}
    if op == "attend":
        if c["head_dim"] == 64:
            c["fp8"] = False
        return c | {"heads": hkv * rng.randint(1, 8 if c["head_dim"] == 64 else 12), "keep": _log_int(rng, 1, max(1, blocks))}
    first, recent = rng.choice((0, 4)), _log_int(rng, 1, max(1, hi // 4))
    return c | {"first": first, "recent": recent, "budget": first + recent + _log_int(rng, 1, max(1, hi // 2)),
                "shared": rng.choice((0, 0, rng.randint(0, blocks // 4))), "again": rng.random() < 0.5}


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


def _values(pool):
    return pool.view(FP8) if pool.dtype == torch.uint8 else pool


def prepare(case, seed):
    s = _sequences(case, seed)
    return {"bounds": _prepare_bounds, "select": _prepare_select, "attend": _prepare_attend, "weights": _prepare_weights,
            "evict": _prepare_evict}[case["op"]](case, s, _gen(seed), random.Random(seed + 1))


def _sequences(c, seed):
    """Lengths, and block tables whose blocks lie anywhere in the pool; the first `shared` blocks are everyone's."""
    r = random.Random(seed)
    bs = c["block_size"]
    lens = [r.randint(c["min_len"], c["max_len"]) for _ in range(c["b"])]
    lens[0] = c["max_len"]
    if c["b"] > 4 and c["min_len"] < c["max_len"]:
        lens[r.randrange(1, c["b"])] = 0  # a padding row
    mb = -(-c["max_len"] // bs)
    shared = min(c.get("shared", 0), min(lens) // bs)
    nbs = [-(-x // bs) for x in lens]
    nb = c["b"] * mb + 2
    ids = list(range(nb))
    r.shuffle(ids)
    tables, refs, at = [], [0] * nb, shared
    for x in nbs:
        row = ids[:shared] + ids[at:at + x - shared]
        at += x - shared
        for i in row:
            refs[i] += 1
        tables.append(row + [-1] * (mb - x))
    return {"case": c, "len_list": lens, "lens": _dev(lens, torch.int32), "tables": _dev(tables, torch.int32),
            "refs": _dev(refs, torch.int32), "blocks": nb, "scale": 1.0 / math.sqrt(c["head_dim"])}


def _prepare_bounds(c, s, g, r):
    nb, hkv, d = s["blocks"], c["kv_heads"], c["head_dim"]
    s["k_cache"] = _pool(g, (nb, c["block_size"], hkv, d), c["fp8"])
    s["bounds"] = torch.zeros(nb, hkv, 2, d, dtype=s["k_cache"].dtype, device="cuda")
    s["starts"] = (s["lens"] - c["new"]).clamp(min=0) if c["new"] else None
    return s


def _prepare_select(c, s, g, r):
    nb, hkv, d, b = s["blocks"], c["kv_heads"], c["head_dim"], c["b"]
    lean = torch.randn(hkv, d, generator=g, device="cuda")  # a head's channels have their own means
    mid = torch.randn(nb, hkv, d, generator=g, device="cuda").mul_(0.5).add_(lean)
    wide = torch.randn(nb, hkv, d, generator=g, device="cuda").mul_(0.3).add_(1.7).abs_()
    x = torch.stack((mid - wide, mid + wide), dim=2)
    s["bounds"] = x.to(FP8).view(torch.uint8) if c["fp8"] else x.to(torch.bfloat16)
    s["q"] = torch.randn(b, c["heads"], d, generator=g, device="cuda").mul_(1.5).to(torch.bfloat16)
    s["sel_tables"] = torch.empty(b, hkv, c["keep"], dtype=torch.int32, device="cuda")
    s["sel_lens"] = torch.empty(b, hkv, dtype=torch.int32, device="cuda")
    return s


def _prepare_attend(c, s, g, r):
    nb, hkv, d, b, bs, keep = s["blocks"], c["kv_heads"], c["head_dim"], c["b"], c["block_size"], c["keep"]
    s["k_cache"], s["v_cache"] = (_pool(g, (nb, bs, hkv, d), c["fp8"]) for _ in range(2))
    s["k_scale"], s["v_scale"] = (1.0, 0.75) if c["fp8"] else (1.0, 1.0)
    s["q"] = torch.randn(b, c["heads"], d, generator=g, device="cuda").mul_(2.0).to(torch.bfloat16)
    lens, mb = s["lens"].long()[:, None, None], s["tables"].shape[1]
    n = -(-lens // bs)
    j = torch.arange(mb, device="cuda")
    luck = torch.rand(b, hkv, mb, generator=g, device="cuda").masked_fill_(j == n - 1, 2.0).masked_fill_(j >= n, -1.0)
    order = luck.argsort(-1, descending=True)[..., :keep]
    order = torch.where(order < n, order, mb).sort(-1).values
    order = torch.nn.functional.pad(order, (0, keep - order.shape[-1]), value=mb)
    ids = torch.nn.functional.pad(s["tables"], (0, 1), value=-1)[:, None, :].expand(b, hkv, mb + 1)
    s["sel_tables"] = ids.gather(-1, order).contiguous()
    s["sel_lens"] = torch.where(n > keep, (keep - 1) * bs + lens - (n - 1) * bs, lens)[..., 0].expand(b, hkv).int().contiguous()
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty(b, c["heads"], dtype=torch.float32, device="cuda")
    if own:  # the workspace that a program keeps
        from paged_kv_decode_cache_gb300 import pa
        p = pa.pa_selected_num_splits(b, c["heads"], hkv, d, keep, bs)
        s["workspace"] = torch.zeros(max(1, pa.pa_splitkv_workspace_bytes(b, c["heads"], d, p)), dtype=torch.uint8,
                                     device="cuda")
    return s


def _prepare_weights(c, s, g, r):
    nb, hkv, d, b, bs, hq, ql = s["blocks"], c["kv_heads"], c["head_dim"], c["b"], c["block_size"], c["heads"], c["q_len"]
    s["k_cache"] = _pool(g, (nb, bs, hkv, d), c["fp8"])
    s["k_scale"] = 1.0
    q = torch.randn(b, ql, hq, d, generator=g, device="cuda").mul_(2.0).to(torch.bfloat16)
    lse = torch.full((b, ql, hq), -math.inf, device="cuda")  # what attention gave for these queries
    for i, n in enumerate(s["len_list"]):
        if n:
            t = torch.arange(n, device="cuda")
            k = _values(s["k_cache"])[s["tables"][i].long()[t // bs], t % bs].float()
            x = torch.einsum("qhgd,thd->qhgt", q[i].float().view(ql, hkv, -1, d), k) * s["scale"]
            seen = t <= n - ql + torch.arange(ql, device="cuda")[:, None]
            lse[i] = torch.logsumexp(x.masked_fill(~seen[:, None, None], -math.inf), -1).view(ql, hq)
    s["q"], s["lse"] = (q, lse) if ql > 1 else (q[:, 0].contiguous(), lse[:, 0].contiguous())
    room = s["tables"].shape[1] * bs
    s["weights"] = torch.randn(b, hkv, room, generator=g, device="cuda").mul_(2.0).exp_()
    s["new_weights"] = torch.zeros(b, hkv, room, device="cuda")
    s["positions"] = torch.full((b, hkv, room), -1, dtype=torch.int32, device="cuda")
    s["ends"] = s["lens"] + r.randrange(1000)  # some tokens have been thrown out before
    return s


def _prepare_evict(c, s, g, r):
    nb, hkv, d, b, bs, ly = s["blocks"], c["kv_heads"], c["head_dim"], c["b"], c["block_size"], c["layers"]
    s["pools"] = torch.empty(2 * ly, nb, bs, hkv, d, dtype=torch.uint8 if c["fp8"] else torch.bfloat16, device="cuda")
    for p in s["pools"]:
        p.copy_(_pool(g, p.shape, c["fp8"]))
    room = s["tables"].shape[1] * bs
    s["weights"] = torch.randn(ly, b, hkv, room, generator=g, device="cuda").mul_(2.0).exp_()
    pos = torch.arange(room, device="cuda").expand(ly, b, hkv, room)
    if c["again"]:  # older tokens stand in no order, with gaps where others were
        old = pos < s["lens"][:, None, None] - c["recent"]
        luck = torch.rand(ly, b, hkv, room, generator=g, device="cuda")
        mixed = torch.where(old, luck, 2.0).argsort(-1)
        pos = torch.where(old, torch.where(mixed < c["first"], mixed, 2 * mixed), 2 * room + pos)
    s["positions"] = pos.int().contiguous()
    s["new_weights"], s["new_positions"] = torch.zeros_like(s["weights"]), torch.zeros_like(s["positions"])
    s["new_tables"], s["new_lens"], s["new_refs"] = (torch.empty_like(s[n]) for n in ("tables", "lens", "refs"))
    if own:  # the handle that a program keeps
        from paged_kv_decode_cache_gb300 import pa
        s["pool_set"] = pa.PoolSet(list(s["pools"]))
    return s


# ---------------------------------------------------------------------------------------------
# one pass


def run(s):
    op = s["case"]["op"]
    if own:
        return {"bounds": _own_bounds, "select": _own_select, "attend": _own_attend, "weights": _own_weights,
                "evict": _own_evict}[op](s)
    return {"bounds": _bounds, "select": _select, "attend": _attend, "weights": _weights, "evict": _evict}[op](s)


# -- bounds of the keys


def _bounds(s):
    c = s["case"]
    bs, lens = c["block_size"], s["lens"].long()[:, None]
    j = torch.arange(s["tables"].shape[1], device="cuda")
    start = lens * 0 if s["starts"] is None else s["starts"].long()[:, None]
    touched = (j * bs < lens) & ((j + 1) * bs > start)
    rows = (lens - j * bs).clamp(1, bs)[touched]
    ids = s["tables"].long()[touched]
    k = _values(s["k_cache"])[ids].float()
    past = (torch.arange(bs, device="cuda") >= rows[:, None])[:, :, None, None]
    lo, hi = k.masked_fill(past, math.inf).amin(1), k.masked_fill(past, -math.inf).amax(1)
    s["bounds"][ids] = torch.stack((lo, hi), dim=2).to(_values(s["bounds"]).dtype).view(s["bounds"].dtype)
    return _values(s["bounds"])


def _own_bounds(s):
    from paged_kv_decode_cache_gb300 import pa
    pa.pa_key_bounds(s["bounds"], s["k_cache"], s["tables"], s["lens"], starts=s["starts"], max_new=s["case"]["new"] or None)
    return _values(s["bounds"])


# -- selection of blocks


def _select(s):
    c = s["case"]
    b, hkv, bs, keep = c["b"], c["kv_heads"], c["block_size"], c["keep"]
    # sums in 64 bits: blocks next to the border must not change places
    lo, hi = _values(s["bounds"])[s["tables"].long().clamp(min=0)].double().permute(0, 2, 3, 4, 1).unbind(2)
    q = s["q"].double().view(b, hkv, -1, c["head_dim"])
    score = (q.clamp(min=0) @ hi + q.clamp(max=0) @ lo).amax(2)
    n = -(-s["lens"].long()[:, None, None] // bs)
    j = torch.arange(s["tables"].shape[1], device="cuda")
    score = score.masked_fill((j < c["first"]) | (j >= n - c["last"]), math.inf).masked_fill(j >= n, -math.inf)
    best = score.sort(dim=-1, descending=True, stable=True).indices[..., :keep]
    best = torch.where(best < n, best, j.numel()).sort(-1).values
    best = torch.nn.functional.pad(best, (0, keep - best.shape[-1]), value=j.numel())
    ids = torch.nn.functional.pad(s["tables"], (0, 1), value=-1)[:, None, :].expand(b, hkv, j.numel() + 1)
    lens = s["lens"].long()[:, None]
    tokens = torch.where(n[..., 0] > keep, (keep - 1) * bs + lens - (n[..., 0] - 1) * bs, lens)
    return {"sel_tables": ids.gather(-1, best), "sel_lens": tokens.int().expand(b, hkv)}


def _own_select(s):
    from paged_kv_decode_cache_gb300 import pa
    c = s["case"]
    pa.pa_blocks_select(s["sel_tables"], s["sel_lens"], s["q"], s["bounds"], c["block_size"], s["tables"], s["lens"],
                        first=c["first"], last=c["last"])
    return {"sel_tables": s["sel_tables"], "sel_lens": s["sel_lens"]}


# -- attention over the selected blocks


def _attend(s):
    c = s["case"]
    b, hkv, d, bs = c["b"], c["kv_heads"], c["head_dim"], c["block_size"]
    ids = s["sel_tables"].long().clamp(min=0)
    t = torch.arange(c["keep"] * bs, device="cuda")
    rows = ids[..., t // bs] * bs + t % bs
    heads = torch.arange(hkv, device="cuda")[:, None]
    k, v = (_values(s[n]).flatten(0, 1)[rows, heads].float() for n in ("k_cache", "v_cache"))
    x = (s["q"].float().view(b, hkv, -1, d) @ k.transpose(-1, -2)) * (s["scale"] * s["k_scale"])
    x = x.masked_fill((t >= s["sel_lens"][..., None])[:, :, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(x - m)
    total = p.sum(-1, keepdim=True)
    out = (p @ v) * s["v_scale"] / torch.where(total == 0, torch.ones_like(total), total)
    s["out"].copy_(out.reshape(b, -1, d))
    s["lse"].copy_((m + torch.log(total)).reshape(b, -1))
    return {"out": s["out"], "lse": s["lse"]}


def _own_attend(s):
    from paged_kv_decode_cache_gb300 import pa
    if s["case"]["fp8"]:
        pa.pa_decode_selected_fp8(s["out"], s["lse"], s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"],
                                  s["sel_tables"], s["sel_lens"], s["scale"], workspace=s["workspace"])
    else:
        pa.pa_decode_selected(s["out"], s["lse"], s["q"], s["k_cache"], s["v_cache"], s["sel_tables"], s["sel_lens"],
                              s["scale"], workspace=s["workspace"])
    return {"out": s["out"], "lse": s["lse"]}


# -- attention weights that tokens draw


def _weights(s):
    c = s["case"]
    b, hkv, d, bs, ql = c["b"], c["kv_heads"], c["head_dim"], c["block_size"], c["q_len"]
    t = torch.arange(s["weights"].shape[-1], device="cuda")
    lens = s["lens"].long()[:, None]
    k = _values(s["k_cache"])[s["tables"].long().clamp(min=0)].flatten(1, 2).float()  # [b, t, hkv, d]
    q = s["q"].float().view(b, ql, hkv, -1, d).permute(0, 2, 1, 3, 4)
    x = (q.flatten(2, 3) @ k.permute(0, 2, 3, 1)).unflatten(2, (ql, -1)) * (s["scale"] * s["k_scale"])
    lse = s["lse"].view(b, ql, hkv, -1).permute(0, 2, 1, 3)[..., None]
    seen = t <= lens[:, :, None] - ql + torch.arange(ql, device="cuda")[:, None]
    p = torch.exp(x - lse).masked_fill(~(seen[:, None, :, None] & (lse > -math.inf)), 0.0).sum((2, 3))
    old = torch.where(t < lens - ql, 1.0, 0.0)[:, None] * s["weights"] * c["decay"]  # (a new token has none)
    here = (t < lens)[:, None].expand(b, hkv, -1)
    fresh = here & (t >= lens - ql)[:, None]
    s["new_weights"].copy_(torch.where(here, old + p, s["new_weights"]))
    place = (s["ends"].long()[:, None] - lens + t)[:, None]
    s["positions"].copy_(torch.where(fresh, place.int(), s["positions"]))
    return {"weights": s["new_weights"], "positions": s["positions"]}


def _own_weights(s):
    from paged_kv_decode_cache_gb300 import pa
    c = s["case"]
    if c["fp8"]:
        pa.pa_weights_add_fp8(s["new_weights"], s["weights"], s["positions"], s["q"], s["lse"], s["k_cache"], s["k_scale"],
                              s["tables"], s["lens"], s["scale"], ends=s["ends"], decay=c["decay"])
    else:
        pa.pa_weights_add(s["new_weights"], s["weights"], s["positions"], s["q"], s["lse"], s["k_cache"], s["tables"],
                          s["lens"], s["scale"], ends=s["ends"], decay=c["decay"])
    return {"weights": s["new_weights"], "positions": s["positions"]}


# -- eviction


def _evict(s):
    c = s["case"]
    ly, b, hkv, bs, d = c["layers"], c["b"], c["kv_heads"], c["block_size"], c["head_dim"]
    tables, lens, refs = s["tables"].long(), s["lens"].long(), s["refs"].long()
    j = torch.arange(tables.shape[1], device="cuda")
    used = j < -(-lens[:, None] // bs)
    held = used & (refs[tables.clamp(min=0)] > 1)  # blocks of others too: up to the last of them nothing moves
    fixed = torch.minimum(lens, (torch.where(held, j + 1, 0).amax(1)) * bs)
    least = torch.where(fixed > 0, fixed + c["first"] + c["recent"], 0)
    now = torch.minimum(lens, least.clamp(min=c["budget"]))
    # which tokens stay
    t = torch.arange(s["weights"].shape[-1], device="cuda")
    length, n = lens[:, None, None], now[:, None, None]
    newest = s["positions"].gather(-1, (length - 1).clamp(min=0).expand(ly, b, hkv, 1))
    safe = (t < fixed[:, None, None]) | (s["positions"] < c["first"]) | (s["positions"] > newest - c["recent"])
    rank = torch.where(safe, math.inf, s["weights"]).masked_fill(t >= length, -math.inf)
    order = rank.sort(dim=-1, descending=True, stable=True).indices
    keep = torch.zeros_like(safe).scatter_(-1, order, (t < n).expand(ly, b, hkv, -1))
    # the k-th place that came free gets the k-th token that stays from behind
    room = t.numel()
    hole = torch.where(~keep & (t < n), t, room).sort(-1).values
    mover = torch.where(keep & (t >= n), t, room).sort(-1).values
    src = torch.nn.functional.pad(t.expand(ly, b, hkv, -1), (0, 1)).scatter(-1, hole, mover)[..., :room]
    here = t < n
    src = torch.where(here, src, t)
    s["new_weights"].copy_(torch.where(here, s["weights"].gather(-1, src), s["new_weights"]))
    s["new_positions"].copy_(torch.where(here, s["positions"].gather(-1, src), s["new_positions"]))
    top = min(room, int(max(c["budget"], c["shared"] * bs + c["first"] + c["recent"])))
    src, dst = src[..., :top], t[:top].expand(ly, b, hkv, -1)
    rows = [tables.clamp(min=0)[:, None].expand(b, hkv, -1).expand(ly, b, hkv, -1).gather(-1, x // bs) * bs + x % bs
            for x in (src, dst)]
    moved = (dst < n) & (src != dst)
    nowhere = s["pools"].shape[1] * bs - 1  # (the last block is no one's: what does not move is copied there to itself)
    spare = torch.where(s["refs"].long() == 0, torch.arange(refs.numel(), device="cuda"), -1).amax() * bs
    rows = [torch.where(moved, x, spare.clamp(max=nowhere)) for x in rows]
    pools = s["pools"].view(ly, 2, -1, hkv, d)
    at = (torch.arange(ly, device="cuda")[:, None, None, None, None], torch.arange(2, device="cuda")[:, None, None, None])
    head = torch.arange(hkv, device="cuda")[:, None]
    pools[(*at, rows[1][:, None], head)] = pools[(*at, rows[0][:, None], head)]
    # blocks behind the new lengths go back
    stay = torch.where(now == lens, -(-lens // bs), torch.maximum(-(-now // bs), now // bs + 1))[:, None]
    gone = used & (j >= stay)
    s["new_tables"].copy_(torch.where(used & ~gone, tables, -1))
    s["new_refs"].copy_(refs.index_add(0, tables.clamp(min=0).flatten(), -gone.long().flatten()))
    s["new_lens"].copy_(now)
    return {"tables": s["new_tables"], "lens": s["new_lens"], "refs": s["new_refs"], "weights": s["new_weights"],
            "positions": s["new_positions"], "pools": _values(s["pools"])}


def _own_evict(s):
    from paged_kv_decode_cache_gb300 import pa
    c = s["case"]
    pa.pa_cache_evict(s["new_tables"], s["new_lens"], s["new_refs"], s["new_weights"], s["new_positions"], s["tables"],
                      s["lens"], s["refs"], s["weights"], s["positions"], s["pool_set"], c["budget"], first=c["first"],
                      recent=c["recent"])
    return {"tables": s["new_tables"], "lens": s["new_lens"], "refs": s["new_refs"], "weights": s["new_weights"],
            "positions": s["new_positions"], "pools": _values(s["pools"])}


# ---------------------------------------------------------------------------------------------
# what a pass cannot do without, and its outputs in 64 bits


def work(c):
    mean = 0.5 * (c["min_len"] + c["max_len"])
    hkv, d, bs, e = c["kv_heads"], c["head_dim"], c["block_size"], 1 if c["fp8"] else 2
    if c["op"] == "bounds":
        tokens = mean if not c["new"] else min(mean, c["new"] + bs / 2)
        blocks = tokens / bs if not c["new"] else max(1.0, tokens / bs)
        return {"bytes": int(c["b"] * (tokens + 2 * blocks) * hkv * d * e), "flops": int(2 * c["b"] * tokens * hkv * d)}
    if c["op"] == "select":
        blocks = mean / bs
        return {"bytes": int(c["b"] * (hkv * (blocks * 2 * d * e + 4 * min(blocks, c["keep"]) + 4) + 4 * blocks
                                       + 2 * c["heads"] * d)),
                "flops": int(4 * c["b"] * c["heads"] * d * blocks)}
    if c["op"] == "attend":
        tokens = min(mean, c["keep"] * bs)
        return {"bytes": int(c["b"] * (hkv * (2 * tokens * d * e + 4 * tokens / bs + 4) + c["heads"] * (4 * d + 4))),
                "flops": int(4 * c["b"] * c["heads"] * d * tokens)}
    if c["op"] == "weights":
        return {"bytes": int(c["b"] * (hkv * mean * (d * e + 8) + c["q_len"] * (c["heads"] * (2 * d + 4) + 4 * hkv))),
                "flops": int(2 * c["b"] * c["q_len"] * c["heads"] * d * mean)}
    stay = min(mean, c["budget"])
    moved = stay * (1 - stay / mean)
    rows = c["layers"] * c["b"] * hkv
    return {"bytes": int(rows * (8 * mean + 8 * stay + 4 * moved * d * e) + 12 * c["b"] * mean / bs), "flops": 0}


def exact(c, seed):
    """The computed numbers in 64 bits, from the definitions; None for what is only chosen or moved."""
    if c["op"] == "bounds":
        return _exact_bounds(c, seed)
    if c["op"] == "attend":
        return _exact_attend(c, seed)
    if c["op"] == "weights":
        return _exact_weights(c, seed)
    return None


def _exact_bounds(c, seed):
    s = prepare(c, seed)
    out, keys = torch.zeros(s["bounds"].shape, dtype=torch.float64, device="cuda"), _values(s["k_cache"])
    bs = c["block_size"]
    for b, length in enumerate(s["len_list"]):
        first = max(0, length - c["new"]) // bs if c["new"] else 0
        ids = s["tables"][b, first:-(-length // bs)].long()
        if not ids.numel():
            continue
        k = keys[ids].double()
        out[ids, :, 0], out[ids, :, 1] = k.min(1).values, k.max(1).values
        tail = k[-1, :(length - 1) % bs + 1]
        out[ids[-1], :, 0], out[ids[-1], :, 1] = tail.min(0).values, tail.max(0).values
    return out


def _exact_attend(c, seed):
    s = prepare(c, seed)
    hkv, bs, d, group = c["kv_heads"], c["block_size"], c["head_dim"], c["heads"] // c["kv_heads"]
    out, lse = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda"), \
        torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
    lens = s["sel_lens"].tolist()
    for b in range(c["b"]):
        for h in range(hkv):
            n = lens[b][h]
            if not n:
                continue
            ids = s["sel_tables"][b, h, :-(-n // bs)].long()
            k, v = (_values(s[x])[ids, :, h].double().reshape(-1, d)[:n] for x in ("k_cache", "v_cache"))
            x = s["q"][b, h * group:(h + 1) * group].double() @ (k * s["k_scale"]).t() * s["scale"]
            z = torch.logsumexp(x, -1)
            lse[b, h * group:(h + 1) * group] = z
            out[b, h * group:(h + 1) * group] = torch.exp(x - z[:, None]) @ (v * s["v_scale"])
    return {"out": out, "lse": lse}


def _exact_weights(c, seed):
    if 2 * c["b"] * c["q_len"] * c["heads"] * c["max_len"] * c["head_dim"] > 2e11:
        return None
    s = prepare(c, seed)
    hkv, bs, ql = c["kv_heads"], c["block_size"], c["q_len"]
    out = s["new_weights"].double()
    q = s["q"].double().view(c["b"], ql, hkv, -1, c["head_dim"])
    lse = s["lse"].double().view(c["b"], ql, hkv, -1)
    for b, length in enumerate(s["len_list"]):
        t = torch.arange(length, device="cuda")
        k = _values(s["k_cache"]).flatten(0, 1)[s["tables"][b].long()[t // bs] * bs + t % bs].double() * s["k_scale"]
        total = torch.zeros(hkv, length, dtype=torch.float64, device="cuda")
        for i in range(ql):
            n = max(0, length - ql + i + 1)
            x = torch.einsum("hgd,thd->hgt", q[b, i], k[:n]) * s["scale"]
            total[:, :n] += torch.exp(x - lse[b, i, :, :, None]).sum(1) if n else 0.0
        past = max(0, length - ql)
        total[:, :past] += s["weights"][b, :, :past].double() * c["decay"]
        out[b, :, :length] = total
    return {"weights": out, "positions": None}
