"""What is measured of the operators around sparse attention over the paged cache.

Five operators over the device arrays of a step, each with its plain form in torch:

  tables  gp_build_tables: pages for the new tokens, the block tables, the slot
          map and the positions of the packed rows, from lengths on the GPU
  rotary  gp_append_mapped: rotary positions (half or interleaved pairs, all or
          part of a head, scaled for long contexts), rotated keys and values
          written where the slot map says
  bounds  gp_block_bounds: per block of keys and KV head, bounds of every
          dimension in 8 bits with one scale, a power of two
  select  gp_select_blocks: the blocks that each row attends to, by the bound
          that the group's queries reach over them
  attend  gp_sparse_attention: softmax attention over the listed blocks

A case: op, model shape (hq, hkv, d, kv: type of cache and queries), n requests
whose lengths are drawn between two ends by `mix` (the same for every seed), the
block's tokens, how many blocks a row takes, and `pad` rows behind the last one,
which stay as they are.
"""

import math
import random

import numpy as np
import torch

own = False

PAGE = 256
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
TOPICS = 48
NO_ROPE = dict(layout="half", part=1.0, scaling="none", theta=1.0e4, factor=1.0, original=8192)


def listed():
    llama = dict(hq=32, hkv=8, d=128, kv="bf16", pad=0, **NO_ROPE)
    blocks = dict(llama, block=64, top=32, sink=1, recent=4)
    one = dict(new=1, new_spread=0)
    return [
        # a decode step of 64 requests: what every step pays before its first layer
        dict(llama, name="tables_step", op="tables", n=64, cached=900, spread=3000, mix=1, **one),
        # a step that mixes many prompts, some behind others' cached prefixes
        dict(llama, name="tables_prompts", op="tables", n=300, cached=0, spread=2000, new=1, new_spread=280, mix=2)
        | dict(pad=77),
        # one decode step's tokens of 64 requests, one layer, positions far past the trained length
        dict(llama, name="rotary_step", op="rotary", n=64, cached=100, spread=400, mix=3, **one)
        | dict(scaling="ramp", theta=5.0e5, factor=8.0),
        # prompts of four requests, interleaved pairs in half of a head
        dict(llama, name="rotary_prompt", op="rotary", n=4, cached=0, spread=700, new=3001, new_spread=1700, mix=4)
        | dict(layout="interleaved", part=0.5, scaling="bands", factor=8.0),
        # the blocks that a decode step's tokens fall into
        dict(blocks, name="bounds_step", op="bounds", n=64, cached=100, spread=500, mix=5, **one),
        # the blocks of four prompts
        dict(blocks, name="bounds_prompt", op="bounds", n=4, cached=0, spread=700, new=3001, new_spread=1700, mix=6)
        | dict(block=32),
        # a decode step of 64 requests of 4 to 128 pages
        dict(blocks, name="select_batch", op="select", n=64, cached=1024, spread=31744, mix=7, **one),
        # the second part of a long prompt
        dict(blocks, name="select_chunk", op="select", n=1, cached=12007, spread=0, new=4001, new_spread=0, mix=8),
        # a single long request: the latency of a decode step
        dict(blocks, name="attend_one", op="attend", n=1, cached=60000, spread=0, mix=9, **one) | dict(top=64),
        # a decode step of 64 requests of 4 to 128 pages
        dict(blocks, name="attend_batch", op="attend", n=64, cached=1024, spread=31744, mix=10, **one),
        # the second part of a long prompt
        dict(blocks, name="attend_chunk", op="attend", n=1, cached=12007, spread=0, new=4001, new_spread=0, mix=11),
        # drafted tokens over a cache kept in 32 bits, small heads and blocks
        dict(blocks, name="attend_draft_f32", op="attend", n=6, cached=900, spread=3000, new=3, new_spread=2, mix=12)
        | dict(hq=4, hkv=2, d=64, kv="f32", block=16, top=24, recent=2, pad=3),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tables", "rotary", "bounds", "select", "attend"])
    d, group, kv = rng.choice([64, 128]), rng.choice([2, 4]), rng.choice(["bf16", "bf16", "bf16", "f32"])
    hkv = rng.choice([1, 2, 4, 8])
    c = dict(NO_ROPE, op=op, hq=group * hkv, hkv=hkv, d=d, kv=kv, mix=rng.randrange(1 << 20), pad=rng.choice([0, 0, 1, 37]))
    if op == "tables":
        c.update(n=_log(rng, 1, 300), cached=rng.randrange(0, 600), spread=_log(rng, 1, 4000))
        c.update(new=rng.randrange(0, 3), new_spread=_log(rng, 1, 280))
    elif op == "rotary":
        n = _log(rng, 1, 64)
        c.update(n=n, cached=rng.randrange(0, 300), spread=_log(rng, 1, 600))
        c.update(new=_log(rng, 1, 4000 // n + 1), new_spread=_log(rng, 1, 200))
        c.update(layout=rng.choice(["half", "interleaved"]), part=rng.choice([1.0, 1.0, 0.5, 0.25]),
                 scaling=rng.choice(["none", "linear", "bands", "ramp"]), theta=rng.choice([1.0e4, 5.0e5, 1.0e6]),
                 factor=rng.choice([2.0, 4.0, 8.0, 32.0]), original=rng.choice([4096, 8192, 32768]))
    else:
        block = rng.choice([16, 32, 64, 128])
        most = 4096 // block  # a row attends to 4096 tokens at most
        top = _log(rng, min(most, 4), most)
        sink = rng.choice([0, 1, 1, 2])
        c.update(block=block, top=top, sink=sink, recent=rng.randrange(1, max(2, min(top - sink, 5))))
        if op == "bounds":
            n = _log(rng, 1, 64)
            c.update(n=n, cached=rng.randrange(0, 300), spread=_log(rng, 1, 600))
            c.update(new=_log(rng, 1, 4000 // n + 1), new_spread=_log(rng, 1, 200))
        elif rng.random() < 0.5:  # a decode step, or a few drafted tokens
            c.update(n=_log(rng, 1, 64), cached=rng.randrange(0, 600), spread=_log(rng, 50, 31000))
            c.update(new=1, new_spread=rng.choice([0, 0, 3, 7]))
        else:
            n = _log(rng, 1, 8)
            c.update(n=n, cached=rng.randrange(0, 500), spread=_log(rng, 20, 12000 // n + 20))
            c.update(new=_log(rng, 1, 1500 // n + 1), new_spread=_log(rng, 1, 200))
    return c


def _lengths(case):
    """Per request: tokens in the cache before the call, and new ones."""
    rng = random.Random(case["mix"])
    cached = [case["cached"] + rng.randrange(case["spread"] + 1) for _ in range(case["n"])]
    return cached, [case["new"] + rng.randrange(case["new_spread"] + 1) for _ in range(case["n"])]


def _pages(tokens):
    return -(-tokens // PAGE)


def prepare(case, seed):
    cached, new = _lengths(case)
    n, hq, hkv, d, op = (case[k] for k in ("n", "hq", "hkv", "d", "op"))
    dt = TYPES[case["kv"]]
    total = [a + b for a, b in zip(cached, new)]
    rows, max_rows = sum(new), sum(new) + case["pad"]
    cap, pool = max(1, max(map(_pages, total))), max(1, sum(map(_pages, total)))
    rng = np.random.default_rng(seed)
    order, slots = rng.permutation(pool).astype(np.int32), rng.permutation(n + 2)[:n].astype(np.int32)
    tables = np.full((n + 2, cap), -1, dtype=np.int32)  # by request slot, as a serving process holds them
    held, free, at = np.zeros(n + 2, dtype=np.int32), [], 0
    for r, s in enumerate(slots):
        have = _pages(cached[r]) if op == "tables" else _pages(total[r])
        tables[s, :have] = order[at:at + have]
        at += have
        held[s] = have
    free = order[at:] if op == "tables" else order[:0]
    pos = [t + 5000 * (r % 3) for r, t in enumerate(cached)]  # positions count evicted tokens too

    def dev(x, dtype):
        return torch.as_tensor(np.asarray(x, dtype=dtype), device="cuda")

    s = dict(case=case, cached=cached, new=new, rows=rows, slots=dev(slots, np.int32), num_cached=dev(cached, np.int32),
             num_new=dev(new, np.int32), pos=dev(pos, np.int64), tables=dev(tables, np.int32))
    row_req, slot_map, positions = np.full(max_rows, -1, np.int32), np.full(max_rows, -1, np.int64), np.zeros(max_rows, np.int64)
    row0 = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    if op == "tables":
        s.update(held=dev(held, np.int32), num_pages=dev(held.copy(), np.int32), free=dev(free, np.int32),
                 taken=torch.zeros(1, dtype=torch.int32, device="cuda"), state=torch.full((n,), -1, dtype=torch.int32, device="cuda"))
        row0[:] = -1
    else:
        for r, sl in enumerate(slots):
            t = cached[r] + np.arange(new[r])
            at = slice(row0[r], row0[r] + new[r])
            row_req[at], positions[at] = r, pos[r] + np.arange(new[r])
            slot_map[at] = tables[sl, t // PAGE].astype(np.int64) * PAGE + t % PAGE
    s.update(row0=dev(row0, np.int32), row_req=dev(row_req, np.int32), slot_map=dev(slot_map, np.int64),
             positions=dev(positions, np.int64))
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=gen)

    if op == "rotary":
        # what a projection gives: queries, keys and values side by side in a row
        qkv = normal(max_rows, (hq + 2 * hkv) * d).to(dt)
        a, b = hq * d, (hq + hkv) * d
        s.update(q=qkv[:, :a].unflatten(1, (hq, d)), k_new=qkv[:, a:b].unflatten(1, (hkv, d)), v_new=qkv[:, b:].unflatten(1, (hkv, d)),
                 q_rot=torch.zeros(max_rows, hq, d, dtype=dt, device="cuda"))
    if op in ("rotary", "bounds", "attend"):
        s["k"], s["v"] = (torch.zeros(1, pool, hkv, PAGE, d, dtype=dt, device="cuda") for _ in range(2))
    if op in ("bounds", "select", "attend"):
        # keys look like their neighbours: a run of 64 tokens shares one of a few topics
        look = normal(hkv, TOPICS, d)
        topic = torch.randint(TOPICS, (pool, PAGE // 64), device="cuda", generator=gen)
        B, per = case["block"], PAGE // case["block"]
        s["bounds"] = torch.zeros(1, pool, hkv, per, 2, d, dtype=torch.int8, device="cuda")
        s["scales"] = torch.zeros(1, pool, hkv, per, dtype=torch.float32, device="cuda")
        for p in range(0, pool, 256):
            z = topic[p:p + 256].repeat_interleave(64, 1)  # [pages, PAGE]
            k = normal(z.shape[0], hkv, PAGE, d).add_(look[:, z].transpose(0, 1)).to(dt)
            if op != "select":
                s["k"][0, p:p + 256] = k
                s["v"][0, p:p + 256] = normal(z.shape[0], hkv, PAGE, d).to(dt)
            if op != "bounds":
                lo, hi = k.float().unflatten(2, (per, B)).aminmax(dim=3)
                s["bounds"][0, p:p + 256], s["scales"][0, p:p + 256] = _held_bounds(lo, hi)
    if op in ("select", "attend"):
        # queries ask for a few topics, others every 48 tokens of a request
        q, G = normal(max_rows, hkv, hq // hkv, d), hq // hkv
        if rows:
            r, t = _packed(s)
            asked = torch.randint(TOPICS, (len(new), max(new) // 48 + 1, 3), device="cuda", generator=gen)[r, t // 48]
            q[:rows] += 0.7 * look[:, asked].sum(2).permute(1, 0, 2)[:, :, None]
        s["q"] = q.reshape(max_rows, hq, d).to(dt)
        s["blocks"] = torch.full((max_rows, hkv, case["top"]), -1, dtype=torch.int32, device="cuda")
    if op == "attend":
        _select(s)
        s["out"] = torch.zeros_like(s["q"])
    if own:
        _engine(s)
    return s


def _engine(s):
    """The engine and the arrays of its steps, as a serving process keeps them."""
    import paged_kv_cache_step_gb300 as gp
    c, dt = s["case"], gp.GP_DTYPE_F32 if s["case"]["kv"] == "f32" else gp.GP_DTYPE_BF16
    slots, cap = s["tables"].shape
    pool = max(1, sum(_pages(a + b) for a, b in zip(s["cached"], s["new"])))
    if "k" not in s:
        s["k"], s["v"] = (torch.empty(1, pool, c["hkv"], PAGE, c["d"], dtype=TYPES[c["kv"]], device="cuda") for _ in range(2))
    cfg = gp.gp_config_default(num_layers=1, num_q_heads=c["hq"], num_kv_heads=c["hkv"], head_dim=c["d"], kv_dtype=dt,
                               q_dtype=dt, max_slots=slots, num_pages=pool, max_pages_per_req=cap)
    ctx = gp.gp_create(cfg, s["k"], s["v"], torch.cuda.current_stream())
    step = gp.Step(ctx, slots=s["slots"], num_cached=s["num_cached"], num_new=s["num_new"], pos=s["pos"], tables=s["tables"],
                   row0=s["row0"], row_req=s["row_req"], slot_map=s["slot_map"], positions=s["positions"])

    class Handle:
        def __del__(self, destroy=gp.gp_destroy, ctx=ctx):
            destroy(ctx)

    rope = None
    if c["op"] == "rotary":
        rope = gp.gp_rope_default(
            layout=gp.GP_ROPE_INTERLEAVED if c["layout"] == "interleaved" else gp.GP_ROPE_HALF, rotary_dim=int(c["part"] * c["d"]),
            theta=c["theta"], factor=c["factor"], original_length=c["original"],
            scaling={"none": gp.GP_ROPE_NONE, "linear": gp.GP_ROPE_LINEAR, "bands": gp.GP_ROPE_BANDS, "ramp": gp.GP_ROPE_RAMP}[c["scaling"]])
    s.update(gp=gp, ctx=ctx, step=step, rope=rope, handle=Handle())


def run(s):
    c, op = s["case"], s["case"]["op"]
    if own:
        gp, ctx, step = s["gp"], s["ctx"], s["step"]
        if op == "tables":
            gp.gp_build_tables(ctx, step, s["held"], s["num_pages"], s["free"], None, s["taken"], s["state"])
        elif op == "rotary":
            gp.gp_append_mapped(ctx, 0, step, s["rope"], s["q"], s["k_new"], s["v_new"], s["q_rot"])
        elif op == "bounds":
            gp.gp_block_bounds(ctx, 0, step, c["block"], s["bounds"], s["scales"])
        elif op == "select":
            gp.gp_select_blocks(ctx, 0, step, c["block"], c["top"], c["sink"], c["recent"], s["q"], s["bounds"], s["scales"],
                                s["blocks"])
        else:
            gp.gp_sparse_attention(ctx, 0, step, c["block"], c["top"], s["q"], s["blocks"], s["out"])
    else:
        {"tables": _tables, "rotary": _rotary, "bounds": _bounds, "select": _select, "attend": _attend}[op](s)
    if op == "tables":
        return {k: s[k] for k in ("tables", "num_pages", "row0", "row_req", "slot_map", "positions", "state", "taken")}
    if op == "rotary":
        return {"q_rot": s["q_rot"], "k": s["k"], "v": s["v"]}
    if op == "bounds":
        return {"bounds": s["bounds"] * s["scales"][..., None, None], "scales": s["scales"]}  # the values they stand for
    return {"blocks": s["blocks"]} if op == "select" else {"out": s["out"]}


# ---- plain forms ------------------------------------------------------------

def _packed(s):
    """Request and index within it of every packed row of new tokens."""
    new = s["num_new"].long()
    r = torch.repeat_interleave(torch.arange(len(new), device="cuda"), new, output_size=s["rows"])
    return r, torch.arange(s["rows"], device="cuda") - (torch.cumsum(new, 0) - new)[r]


def _tables(s):
    slots, cached, new, held = s["slots"].long(), s["num_cached"].long(), s["num_new"].long(), s["held"].long()[s["slots"].long()]
    max_rows, cap = len(s["row_req"]), s["tables"].shape[1]
    need = -(-(cached + new) // PAGE)
    valid = (cached >= 0) & (new >= 0) & (need <= cap) & (cached <= held * PAGE) & (held <= cap)
    want = torch.where(valid, new, 0)
    room = valid & ((want == 0) | (torch.cumsum(want, 0) <= max_rows))
    take = torch.where(room, torch.clamp(need - held, min=0), 0)
    ends = torch.cumsum(take, 0)
    given = room & ((take == 0) | (ends <= len(s["free"])))
    s["state"].copy_(torch.where(given, 0, torch.where(room, 1, torch.where(valid, 2, 3))))
    take, new = torch.where(given, take, 0), torch.where(given, new, 0)
    first = torch.cumsum(take, 0) - take
    s["taken"].copy_(take.sum())
    s["num_pages"][slots] = (held + take).int()
    block = torch.arange(cap, device="cuda")
    fresh = (block >= held[:, None]) & (block < (held + take)[:, None])
    page = s["free"][torch.where(fresh, first[:, None] + block - held[:, None], 0)] if len(s["free"]) else block.int()
    s["tables"][slots] = torch.where(fresh, page, s["tables"][slots])
    row0 = torch.cumsum(new, 0)
    s["row0"][0] = 0
    s["row0"][1:] = row0
    row = torch.arange(max_rows, device="cuda")
    r = torch.searchsorted(row0, row, right=True)
    live, r = r < len(new), torch.clamp(r, max=len(new) - 1)
    t = row - (row0 - new)[r]
    slot = torch.where(live, cached[r] + t, 0)
    s["row_req"].copy_(torch.where(live, r, -1))
    s["slot_map"].copy_(torch.where(live, s["tables"][slots[r], slot // PAGE].long() * PAGE + slot % PAGE, -1))
    s["positions"].copy_(torch.where(live, s["pos"][r] + t, 0))


def _frequencies(case):
    """Inverse frequencies in 64 bits and the amplitude of cosine and sine."""
    rd, f, length = int(case["part"] * case["d"]), case["factor"], case["original"]
    i = torch.arange(0, rd, 2, dtype=torch.float64, device="cuda") / rd
    inv = case["theta"] ** -i
    if case["scaling"] == "linear":
        return inv / f, 1.0
    if case["scaling"] == "bands":  # long waves are stretched, short ones stay, between 1 and 4 turns they blend
        turns = length * inv / (2.0 * math.pi)
        keep = torch.clamp((turns - 1.0) / 3.0, 0.0, 1.0)
        return inv * (keep + (1.0 - keep) / f), 1.0
    if case["scaling"] == "ramp":  # pairs that turn more than 32 times stay, those under one turn are stretched
        def pair(turns):
            return rd * math.log(length / (turns * 2.0 * math.pi)) / (2.0 * math.log(case["theta"]))
        low, high = max(0, math.floor(pair(32.0))), min(rd - 1, math.ceil(pair(1.0)))
        j = torch.arange(rd // 2, dtype=torch.float64, device="cuda")
        stretch = torch.clamp((j - low) / max(high - low, 0.001), 0.0, 1.0)
        return inv * (1.0 - stretch + stretch / f), 0.1 * math.log(f) + 1.0
    return inv, 1.0


def _turned(x, cos, sin, case):
    rd, x = 2 * cos.shape[-1], x.to(cos.dtype)
    head, rest = x[..., :rd], x[..., rd:]
    if case["layout"] == "half":
        a, b = head[..., :rd // 2], head[..., rd // 2:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, rest], -1)
    a, b = head[..., 0::2], head[..., 1::2]
    return torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), rest], -1)


def _rotary(s):
    c, n = s["case"], s["rows"]
    inv, amplitude = _frequencies(c)
    ang = s["positions"][:n].double()[:, None, None] * inv  # far positions
    cos, sin = (torch.cos(ang) * amplitude).float(), (torch.sin(ang) * amplitude).float()
    page, slot = s["slot_map"][:n] // PAGE, s["slot_map"][:n] % PAGE
    s["q_rot"][:n] = _turned(s["q"][:n], cos, sin, c).to(s["q_rot"].dtype)
    s["k"][0].transpose(1, 2)[page, slot] = _turned(s["k_new"][:n], cos, sin, c).to(s["k"].dtype)
    s["v"][0].transpose(1, 2)[page, slot] = s["v_new"][:n]


def _exponent(top):
    """The least integer e >= -100 with top <= 127 * 2^e."""
    m, e = torch.frexp(top)
    e = torch.where(m > 127.0 / 128.0, e - 6, e - 7)
    return torch.where(top > 0.0, torch.clamp(e, -100, 100), torch.full_like(e, -100))


def _power(e):
    """2^e of whole numbers in [-100, 100]."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _held_bounds(lo, hi):
    """Bounds of keys [..., d] in 8 bits, and their scale."""
    e = _exponent(torch.maximum(lo.abs(), hi.abs()).amax(-1))
    held = torch.stack([torch.floor(lo * _power(-e)[..., None]), torch.ceil(hi * _power(-e)[..., None])], -2)
    return held.clamp(-127, 127).to(torch.int8), _power(e)


def _bounds(s):
    c, B = s["case"], s["case"]["block"]
    total = s["num_cached"] + s["num_new"]
    first = torch.div(s["num_cached"], B, rounding_mode="floor")
    count = torch.where(s["num_new"] > 0, (total - 1) // B - first + 1, 0).long()
    blocks = sum((a + b - 1) // B - a // B + 1 for a, b in zip(s["cached"], s["new"]) if b)
    r = torch.repeat_interleave(torch.arange(len(count), device="cuda"), count, output_size=blocks)
    block = first[r] + torch.arange(len(r), device="cuda") - (torch.cumsum(count, 0) - count)[r]
    page, at = s["tables"][s["slots"][r].long(), block * B // PAGE].long(), block % (PAGE // B)
    k = s["k"][0].unflatten(2, (PAGE // B, B)).transpose(1, 2)[page, at].float()  # [blocks, hkv, B, d]
    past = (block[:, None] * B + torch.arange(B, device="cuda") >= total[r][:, None])[:, None, :, None]
    lo, hi = k.masked_fill(past, math.inf).amin(2), k.masked_fill(past, -math.inf).amax(2)
    held, scale = _held_bounds(lo, hi)
    s["bounds"][0].transpose(1, 2)[page, at] = held
    s["scales"][0].transpose(1, 2)[page, at] = scale


def _select(s):
    c, B, K, hkv, d = s["case"], s["case"]["block"], s["case"]["top"], s["case"]["hkv"], s["case"]["d"]
    if s["rows"] == 0:
        return
    r, t = _packed(s)
    own_block = (s["num_cached"][r] + t) // B  # of every row
    n, m, nb = len(s["new"]), max(s["new"]), int(max(a + b for a, b in zip(s["cached"], s["new"])) - 1) // B + 1
    q = s["q"][:s["rows"]].float().unflatten(1, (hkv, -1))  # [rows, hkv, G, d]
    e = _exponent(q.abs().amax((2, 3)))
    q = torch.round(q * _power(-e)[:, :, None, None])
    reach = torch.zeros(n, m, hkv, 2, d, device="cuda")  # of the low and of the high bounds
    reach[r, t] = torch.stack([q.clamp(max=0.0).sum(2), q.clamp(min=0.0).sum(2)], 2)
    pages = torch.clamp(s["tables"][s["slots"].long()], min=0).long()  # [n, cap]
    held = s["bounds"][0][pages].transpose(1, 2).flatten(2, 3)[:, :, :nb].flatten(3).float()  # [n, hkv, nb, 2 d]
    scale = s["scales"][0][pages].transpose(1, 2).flatten(2, 3)[:, :, :nb]
    # whole numbers under 2^24: the products are exact in any order
    score = reach.flatten(3).transpose(1, 2) @ held.transpose(-1, -2) * scale[:, :, None]  # [n, hkv, m, nb]
    score = score.transpose(1, 2)[r, t]  # [rows, hkv, nb]
    block, last = torch.arange(nb, device="cuda"), own_block[:, None, None]
    score = score.masked_fill((block < c["sink"]) | (block > last - c["recent"]), math.inf).masked_fill(block > last, -math.inf)
    order = torch.sort(score, dim=-1, descending=True, stable=True).indices  # equal scores: the lower block first
    some = torch.minimum(last + 1, torch.full_like(last, K))
    kept = torch.zeros_like(score, dtype=torch.bool).scatter_(-1, order, (block < some).expand_as(order))
    row, head, b = kept.nonzero(as_tuple=True)
    place = (torch.cumsum(kept, -1) - 1)[row, head, b]
    s["blocks"][:s["rows"]] = -1
    s["blocks"][row, head, place] = b.int()


def _attend(s):
    c, B, K, hkv, d = s["case"], s["case"]["block"], s["case"]["top"], s["case"]["hkv"], s["case"]["d"]
    if s["rows"] == 0:
        return
    r, t = _packed(s)
    last = s["num_cached"][r] + t
    k, v = (x[0].unflatten(2, (PAGE // B, B)) for x in (s["k"], s["v"]))  # [pages, hkv, blocks, B, d]
    head = torch.arange(hkv, device="cuda")[:, None]
    for a in range(0, s["rows"], max(1, (1 << 28) // (hkv * K * B * d))):
        b = min(s["rows"], a + max(1, (1 << 28) // (hkv * K * B * d)))
        block = s["blocks"][a:b].long()  # [rows, hkv, K]
        page = s["tables"][s["slots"][r[a:b]].long()[:, None, None], block.clamp(min=0) * B // PAGE].long()
        keys = k[page, head, block % (PAGE // B)].flatten(2, 3).float()  # [rows, hkv, K B, d]
        z = s["q"][a:b].float().unflatten(1, (hkv, -1)) @ keys.transpose(-1, -2) / math.sqrt(d)
        token = block[..., None] * B + torch.arange(B, device="cuda")
        z = z.masked_fill(((block < 0)[..., None] | (token > last[a:b, None, None, None])).flatten(2)[:, :, None], -math.inf)
        e = torch.exp(z - z.amax(-1, keepdim=True))
        vals = v[page, head, block % (PAGE // B)].flatten(2, 3).float()
        s["out"][a:b] = (e / e.sum(-1, keepdim=True) @ vals).flatten(1, 2).to(s["out"].dtype)


# ---- what a pass cannot do without -------------------------------------------

def work(case):
    cached, new = _lengths(case)
    hq, hkv, d, op = (case[k] for k in ("hq", "hkv", "d", "op"))
    e = 4 if case["kv"] == "f32" else 2
    rows, n = sum(new), len(new)
    if op == "tables":
        pages = sum(_pages(a + b) for a, b in zip(cached, new))
        return {"bytes": 36 * n + 4 * pages + 20 * (rows + case["pad"]), "flops": 4 * rows}
    if op == "rotary":
        return {"bytes": rows * ((2 * hq + 4 * hkv) * d * e + 16), "flops": 3 * rows * (hq + hkv) * int(case["part"] * d)}
    B = case["block"]
    if op == "bounds":
        tokens = sum(a + b - a // B * B for a, b in zip(cached, new) if b)
        blocks = sum((a + b - 1) // B - a // B + 1 for a, b in zip(cached, new) if b)
        return {"bytes": hkv * (tokens * d * e + blocks * (2 * d + 4)), "flops": 2 * tokens * hkv * d}
    seen = sum((a + t) // B + 1 for a, b in zip(cached, new) for t in range(b))  # (row, block) pairs
    if op == "select":
        blocks = sum((a + b - 1) // B + 1 for a, b in zip(cached, new) if b)
        return {"bytes": hkv * blocks * (2 * d + 4) + rows * (hq * d * e + 4 * hkv * case["top"]), "flops": 4 * seen * hkv * d}
    # a row's tokens; of a request's keys and values no more than there are
    taken = [[min(a + t + 1, case["top"] * B) for t in range(b)] for a, b in zip(cached, new)]
    read = sum(min(a + b, sum(x)) for a, b, x in zip(cached, new, taken))
    return {"bytes": read * hkv * 2 * d * e + rows * (2 * hq * d * e + 4 * hkv * case["top"]),
            "flops": 4 * sum(map(sum, taken)) * hq * d}


# ---- the definition in 64 bits -------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op, hkv, d = case["op"], case["hkv"], case["d"]
    G = case["hq"] // hkv
    slots, tables = s["slots"].cpu().numpy(), s["tables"].cpu().numpy()
    cached, new = s["cached"], s["new"]
    if op == "tables":
        out = {k: s[k].cpu().numpy().copy() for k in ("tables", "num_pages", "row0", "row_req", "slot_map", "positions", "state", "taken")}
        held, free, pos = s["held"].cpu().numpy(), s["free"].cpu().numpy(), s["pos"].cpu().numpy()
        out["row_req"][:], out["slot_map"][:], out["positions"][:] = -1, -1, 0
        at = taken = 0
        for r, sl in enumerate(slots):
            while out["num_pages"][sl] * PAGE < cached[r] + new[r]:  # (the pool and the rows are large enough)
                out["tables"][sl, out["num_pages"][sl]] = free[taken]
                out["num_pages"][sl] += 1
                taken += 1
            out["state"][r], out["row0"][r] = 0, at
            for t in range(new[r]):
                page, slot = divmod(cached[r] + t, PAGE)
                out["row_req"][at], out["positions"][at] = r, pos[r] + t
                out["slot_map"][at] = int(out["tables"][sl, page]) * PAGE + slot
                at += 1
        out["row0"][len(new)], out["taken"][0] = at, taken
        return {k: torch.as_tensor(v) for k, v in out.items()}
    if op == "rotary":
        rd, inv, amplitude = int(case["part"] * d), *_exact_frequencies(case)
        n = s["rows"]
        # a pair is a complex number, the rotation a product with one
        ang = torch.as_tensor(s["positions"][:n].cpu().numpy()[:, None] * inv, device="cuda")
        turn = torch.polar(torch.full_like(ang, amplitude), ang)[:, None]
        first = np.arange(rd // 2) if case["layout"] == "half" else np.arange(0, rd, 2)
        second = torch.as_tensor(first + (rd // 2 if case["layout"] == "half" else 1), device="cuda")
        first = torch.as_tensor(first, device="cuda")

        def turned(x):
            x = x.double().clone()
            z = torch.complex(x[..., first], x[..., second]) * turn
            x[..., first], x[..., second] = z.real, z.imag
            return x

        q, k, v = s["q_rot"].double(), s["k"].double(), s["v"].double()
        q[:n] = turned(s["q"][:n])
        page, slot = s["slot_map"][:n] // PAGE, s["slot_map"][:n] % PAGE
        k[0, page, :, slot] = turned(s["k_new"][:n])
        v[0, page, :, slot] = s["v_new"][:n].double()
        return {"q_rot": q, "k": k, "v": v}
    B = case["block"]
    per = PAGE // B
    if op == "bounds":
        values, scales = s["bounds"].double() * s["scales"].double()[..., None, None], s["scales"].double()
        todo, parts = [], []
        for r, sl in enumerate(slots):
            for b in range(cached[r] // B, (cached[r] + new[r] - 1) // B + 1 if new[r] else 0):
                todo.append((tables[sl, b // per], b % per))
                k = s["k"][0, todo[-1][0], :, b % per * B:min(b % per * B + B, cached[r] + new[r] - b // per * PAGE)]
                parts.append(torch.stack([k.min(1).values, k.max(1).values], 1))
        if todo:
            ends = torch.stack(parts).double().cpu().numpy()  # [blocks, hkv, 2, d]
            top = np.abs(ends).max((2, 3))
            unit = 2.0 ** np.maximum(np.ceil(np.log2(np.maximum(top, 2.0 ** -300) / 127.0)), -100.0)
            unit = np.where(127.0 * unit < top, 2.0 * unit, np.where((127.0 * unit / 2.0 >= top) & (unit > 2.0 ** -100), unit / 2.0, unit))
            got = np.stack([np.floor(ends[:, :, 0] / unit[..., None]), np.ceil(ends[:, :, 1] / unit[..., None])], 2) * unit[..., None, None]
            page, at = (torch.as_tensor([x[i] for x in todo], device="cuda").long() for i in (0, 1))
            values[0, page, :, at] = torch.as_tensor(got, device="cuda")
            scales[0, page, :, at] = torch.as_tensor(unit, device="cuda")
        return {"bounds": values, "scales": scales}
    at = 0
    if op == "select":
        out = s["blocks"].cpu()
        for r, sl in enumerate(slots):
            nb = (cached[r] + new[r] - 1) // B + 1 if new[r] else 0
            b = np.arange(nb)
            value = (s["bounds"].double() * s["scales"].double()[..., None, None])[0, tables[sl, b // per], :, b % per]  # [nb, hkv, 2, d]
            q = s["q"][at:at + new[r]].double().reshape(new[r], hkv, G, d).cpu().numpy()
            top = np.abs(q).max((2, 3))
            unit = 2.0 ** np.ceil(np.log2(np.maximum(top, 2.0 ** -90) / 127.0))
            q = torch.as_tensor(np.rint(q / unit[:, :, None, None]), device="cuda")
            score = torch.zeros(new[r], hkv, nb, dtype=torch.float64, device="cuda")
            for g in range(G):  # the most that each head's query reaches between the bounds
                score += torch.einsum("mhd,bhd->mhb", q[:, :, g].clamp(min=0), value[:, :, 1])
                score += torch.einsum("mhd,bhd->mhb", q[:, :, g].clamp(max=0), value[:, :, 0])
            score = score.cpu().numpy()
            for t in range(new[r]):
                last = (cached[r] + t) // B
                rest = np.arange(case["sink"], max(case["sink"], last + 1 - case["recent"]))
                always = np.setdiff1d(np.arange(last + 1), rest)
                for h in range(hkv):
                    more = rest[np.argsort(-score[t, h, rest], kind="stable")[:case["top"] - len(always)]]
                    kept = np.sort(np.concatenate([always, more]))
                    out[at + t, h] = -1
                    out[at + t, h, :len(kept)] = torch.as_tensor(kept.astype(np.int32))
            at += new[r]
        return {"blocks": out}
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    chosen = s["blocks"].cpu().numpy()
    for r, sl in enumerate(slots):
        T = cached[r] + new[r]
        table = torch.as_tensor(tables[sl, :_pages(T)], device="cuda").long()
        for h in range(hkv):
            keys, vals = (x[0, table, h].reshape(-1, d)[:T].double() for x in (s["k"], s["v"]))
            if new[r] * 8 * B * case["top"] < T * new[r]:  # few of the blocks: row by row
                groups = [(t, t + 1) for t in range(new[r])]
            else:
                groups = [(t, min(t + 512, new[r])) for t in range(0, new[r], 512)]
            for t0, t1 in groups:
                seen = np.zeros((t1 - t0, _pages(T) * per), dtype=bool)
                for t in range(t0, t1):
                    x = chosen[at + t, h]
                    seen[t - t0, x[x >= 0]] = True
                some = np.flatnonzero(np.repeat(seen.any(0), B)[:T])
                some = torch.as_tensor(some, device="cuda")
                see = torch.as_tensor(seen, device="cuda").repeat_interleave(B, 1)[:, some]
                see &= some <= cached[r] + torch.arange(t0, t1, device="cuda")[:, None]
                for g in range(h * G, h * G + G):
                    z = s["q"][at + t0:at + t1, g].double() @ keys[some].T / math.sqrt(d)
                    p = torch.softmax(z.masked_fill(~see, -math.inf), -1)
                    out[at + t0:at + t1, g] = p @ vals[some]
        at += new[r]
    return {"out": out}


def _exact_frequencies(case):
    rd, f, length = int(case["part"] * case["d"]), case["factor"], case["original"]
    out = []
    for j in range(rd // 2):
        inv = case["theta"] ** (-2.0 * j / rd)
        wave = 2.0 * math.pi / inv
        if case["scaling"] == "linear":
            inv /= f
        elif case["scaling"] == "bands":
            if wave > length:
                inv /= f
            elif wave > length / 4.0:
                keep = (length / wave - 1.0) / 3.0
                inv = keep * inv + (1.0 - keep) * inv / f
        elif case["scaling"] == "ramp":
            # the pair, as a real number, that turns so often over the original length
            low, high = (rd * math.log(length / (2.0 * math.pi * turns)) / (2.0 * math.log(case["theta"])) for turns in (32.0, 1.0))
            low, high = max(math.floor(low), 0), min(math.ceil(high), rd - 1)
            x = min(1.0, max(0.0, (j - low) / ((high - low) or 0.001)))
            inv = x * inv / f + (1.0 - x) * inv
        out.append(inv)
    return np.array(out), 0.1 * math.log(f) + 1.0 if case["scaling"] == "ramp" else 1.0
