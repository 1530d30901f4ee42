"""What is measured of the operators around eviction by accumulated attention weight.

Four operators over the paged K/V cache, each with its plain form in torch:

  append  gp_append_tokens: RoPE of the new tokens' queries and keys, the rotated
          keys and the values written into the pages, their weights cleared
  decode  gp_decode_attention_weighted: attention of one new token a request, its
          weights added to the cache's accumulated weights
  chunk   gp_chunk_attention: causal attention of several new tokens a request,
          their weights added to the accumulated weights
  evict   gp_evict_weighted: the recent window and the tokens of most accumulated
          weight kept per (layer, KV head), K, V and weights compacted in order

A case: op, model shape (layers, hq, hkv, d, kv: type of cache and queries),
n requests whose lengths are drawn between two ends by `mix` (the same for every
seed), and the pages of all requests shuffled over the pool.
"""

import math
import random

import numpy as np
import torch

own = False

PAGE = 256
RECENT = 16
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    llama = dict(layers=1, hq=32, hkv=8, d=128, kv="bf16", theta=5.0e5)
    whole = dict(layers=32, hq=32, hkv=8, d=128, kv="bf16", theta=5.0e5)
    tiny = dict(layers=1, hq=4, hkv=2, d=64, kv="f32", theta=1.0e4)
    g2 = dict(layers=1, hq=16, hkv=8, d=64, kv="bf16", theta=1.0e4)
    return [
        # one decode step's tokens of 64 requests, one layer: the call every step makes
        dict(name="append_step", op="append", n=64, cached=900, spread=3000, new=1, new_spread=0, mix=1, **llama),
        # prompts of four requests on their way into the cache
        dict(name="append_prompt", op="append", n=4, cached=0, spread=700, new=3001, new_spread=1700, mix=2, **llama),
        # a single request of 32 pages: the latency of a decode step
        dict(name="decode_one", op="decode", n=1, cached=8192, spread=0, new=0, new_spread=0, mix=3, **llama),
        # 64 requests of 4 to 128 pages, lengths that end inside a page
        dict(name="decode_batch", op="decode", n=64, cached=1024, spread=31744, new=0, new_spread=0, mix=4, **llama),
        # a cache kept in 32 bits, small heads
        dict(name="decode_f32", op="decode", n=6, cached=900, spread=3000, new=0, new_spread=0, mix=5, **tiny),
        # a few drafted tokens a request over long caches
        dict(name="chunk_draft", op="chunk", n=16, cached=1500, spread=7000, new=5, new_spread=3, mix=6, **llama),
        # one long prompt, the second part of it
        dict(name="chunk_prompt", op="chunk", n=1, cached=4099, spread=0, new=6007, new_spread=0, mix=7, **llama),
        # ragged prompts, 64 wide heads in groups of two
        dict(name="chunk_ragged", op="chunk", n=5, cached=0, spread=900, new=300, new_spread=1500, mix=8, **g2),
        # a prompt over a cache kept in 32 bits
        dict(name="chunk_f32", op="chunk", n=2, cached=100, spread=300, new=400, new_spread=300, mix=9, **tiny),
        # one request of 32 pages, every layer, back to half of its length
        dict(name="evict_one", op="evict", n=1, cached=8192, spread=0, new=0, new_spread=0, keep=0.5, mix=10, **whole),
        # a batch of requests back to a budget that ends inside a page
        dict(name="evict_batch", op="evict", n=10, cached=2000, spread=9000, new=0, new_spread=0, keep=0.37, mix=11, **whole),
        # few short requests of two layers, a cache kept in 32 bits
        dict(name="evict_small", op="evict", n=3, cached=700, spread=900, new=0, new_spread=0, keep=0.7, mix=12,
             **dict(tiny, layers=2)),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "decode", "chunk", "evict"])
    d, group, kv = rng.choice([64, 128]), rng.choice([2, 4]), rng.choice(["bf16", "bf16", "bf16", "f32"])
    hkv = rng.choice([1, 2, 4, 8])
    c = dict(op=op, layers=1, hq=group * hkv, hkv=hkv, d=d, kv=kv, theta=rng.choice([1.0e4, 5.0e5, 1.0e6]), new=0,
             new_spread=0, mix=rng.randrange(1 << 20))
    if op == "append":
        c.update(n=_log(rng, 1, 64), cached=rng.randrange(0, 500), spread=_log(rng, 1, 8000))
        c.update(new=_log(rng, 1, 2000), new_spread=_log(rng, 1, 500))
    elif op == "decode":
        n = _log(rng, 1, 64)
        c.update(n=n, cached=rng.randrange(1, 600), spread=_log(rng, 50, 32000))
    elif op == "chunk":
        small = kv == "f32"
        n = _log(rng, 1, 4 if small else 12)
        c.update(n=n, cached=rng.randrange(0, 500), spread=_log(rng, 20, (1500 if small else 16000) // n + 20))
        c.update(new=_log(rng, 1, (400 if small else 4000) // n + 1), new_spread=_log(rng, 1, 200))
    else:
        n = _log(rng, 1, 8)
        c.update(n=n, layers=rng.choice([2, 8, 16, 32]), cached=rng.randrange(100, 600), spread=_log(rng, 100, 9000))
        c["keep"] = round(rng.uniform(0.05, 0.95), 3)
    return c


def _lengths(case):
    """Per request: tokens in the cache before the call, and new ones."""
    rng = random.Random(case["mix"])
    cached = [case["cached"] + rng.randrange(case["spread"] + 1) for _ in range(case["n"])]
    return cached, [case["new"] + rng.randrange(case["new_spread"] + 1) for _ in range(case["n"])]


def _budget(case, cached):
    return [max(1, int(t * case["keep"])) for t in cached]


def prepare(case, seed):
    cached, new = _lengths(case)
    n, L, hq, hkv, d = (case[k] for k in ("n", "layers", "hq", "hkv", "d"))
    dt = TYPES[case["kv"]]
    total = [a + b for a, b in zip(cached, new)]
    pages = [-(-t // PAGE) for t in total]
    cap = max(pages)
    pool = sum(pages)
    order = np.random.default_rng(seed).permutation(pool).astype(np.int32)
    tables = np.zeros((n, cap), dtype=np.int32)  # a block table a request, as the scheduler holds it
    at = 0
    for r, p in enumerate(pages):
        tables[r, :p] = order[at:at + p]
        at += p
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=gen)

    # keys are stored rotated; two in a hundred point the way that half of the
    # heads' queries look, in the dimensions that RoPE hardly turns
    slow = torch.zeros(d, device="cuda")
    slow[d // 2 - d // 16:d // 2] = 1.0
    slow[d - d // 16:] = 1.0
    look = slow * normal(L, 1, hkv, 1, d).sign() * math.sqrt(8.0)
    shape = (L, pool, hkv, PAGE, d)
    k = torch.empty(shape, dtype=dt, device="cuda")
    v = torch.empty(shape, dtype=dt, device="cuda")
    for layer in range(L):
        planted = (torch.rand(pool, hkv, PAGE, 1, device="cuda", generator=gen) < 0.02).float()
        k[layer] = (normal(*shape[1:]) + 1.2 * planted * look[layer]).to(dt)
        v[layer] = normal(*shape[1:]).to(dt)
    # weights gathered so far: a few tokens hold most, one in ten was never looked at
    w = torch.exp(1.5 * normal(L, n, hkv, cap * PAGE) - 2.0)
    w = w * (torch.rand(L, n, hkv, 1, device="cuda", generator=gen) * 0.5 + 0.75)
    w = w * (torch.rand(w.shape, device="cuda", generator=gen) > 0.1)
    s = dict(case=case, cached=cached, new=new, pages=pages, tables=tables, k=k, v=v, w=w,
             pos=[t + 5000 * (r % 3) for r, t in enumerate(cached)])  # positions count evicted tokens too
    rows = sum(new) if case["op"] in ("append", "chunk") else n
    q = normal(rows, hkv, hq // hkv, d)
    q[:, ::2] += 0.8 * look[0, :, ::2]
    s["q"] = q.reshape(rows, hq, d).to(dt)
    if case["op"] == "append":
        s["k_new"], s["v_new"] = normal(rows, hkv, d).to(dt), normal(rows, hkv, d).to(dt)
        s["q_rot"] = torch.empty_like(s["q"])
    if case["op"] == "chunk":
        s["out"] = torch.empty_like(s["q"])
    if case["op"] == "decode":
        s["out"] = torch.empty(n, hq, d, device="cuda")
    if case["op"] == "evict":
        s["keep"] = _budget(case, cached)
        s["w0"] = w.clone()
    if own:
        _engine(s)
    return s


def _engine(s):
    """The engine over the caches and its requests, as a serving process keeps them."""
    import paged_kv_cache_step_gb300 as gp
    c, dt = s["case"], gp.GP_DTYPE_F32 if s["case"]["kv"] == "f32" else gp.GP_DTYPE_BF16
    cfg = gp.gp_config_default(num_layers=c["layers"], num_q_heads=c["hq"], num_kv_heads=c["hkv"], head_dim=c["d"],
                               kv_dtype=dt, q_dtype=dt, max_slots=c["n"], num_pages=s["k"].shape[1],
                               max_pages_per_req=s["tables"].shape[1], recent_window=RECENT, rope_theta=c["theta"])
    ctx = gp.gp_create(cfg, s["k"], s["v"], torch.cuda.current_stream())
    for _ in range(cfg.num_pages):
        gp.gp_page_alloc(ctx)
    reqs = []
    for r, p in enumerate(s["pages"]):
        reqs.append(gp.Request(gp.gp_slot_acquire(ctx), s["tables"][r, :p], s["pos"][r], cfg.max_pages_per_req))

    class Handle:
        def __del__(self, destroy=gp.gp_destroy, ctx=ctx):
            destroy(ctx)

    s.update(gp=gp, ctx=ctx, reqs=reqs, handle=Handle())


def run(s):
    op = s["case"]["op"]
    if own:
        gp, ctx, reqs = s["gp"], s["ctx"], s["reqs"]
        if op == "append":
            gp.gp_append_tokens(ctx, 0, reqs, s["cached"], s["new"], s["q"], s["k_new"], s["v_new"], s["q_rot"], s["w"])
        elif op == "decode":
            gp.gp_decode_attention_weighted(ctx, 0, reqs, s["cached"], s["q"], None, s["out"], s["w"])
        elif op == "chunk":
            gp.gp_chunk_attention(ctx, 0, reqs, s["cached"], s["new"], s["q"], s["out"], s["w"])
        else:
            # the weights start anew, so that every pass moves the rows of a first
            # one; both forms pay for this copy (under 1 % of the rows' bytes)
            s["w"].copy_(s["w0"])
            gp.gp_evict_weighted(ctx, reqs, s["cached"], s["keep"], s["w"])
    else:
        {"append": _append, "decode": _decode, "chunk": _chunk, "evict": _evict}[op](s)
    if op == "append":
        return {"q_rot": s["q_rot"], "k": s["k"], "v": s["v"], "w": s["w"]}
    if op == "evict":
        return {"k": s["k"], "v": s["v"], "w": s["w"]}
    return {"out": s["out"], "w": s["w"]}


# ---- plain forms ------------------------------------------------------------

def _dev(x, dtype=torch.int64):
    return torch.as_tensor(np.asarray(x), device="cuda").to(dtype)


def _angles(pos, case):
    """cos, sin [rows, 1, d/2] in 32 bits of angles in 64: far positions."""
    inv = case["theta"] ** (-torch.arange(0, case["d"], 2, dtype=torch.float64, device="cuda") / case["d"])
    ang = pos.double()[:, None, None] * inv
    return torch.cos(ang).float(), torch.sin(ang).float()


def _rotate(x, cos, sin):
    a, b = x.float().chunk(2, dim=-1)
    return torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)


def _packed(s):
    """Request and index within it of every packed row of new tokens."""
    new = _dev(s["new"])
    r = torch.repeat_interleave(torch.arange(len(s["new"]), device="cuda"), new, output_size=sum(s["new"]))
    first = torch.cumsum(new, 0) - new
    return r, torch.arange(sum(s["new"]), device="cuda") - first[r]


def _append(s):
    c = s["case"]
    r, t = _packed(s)
    slot = _dev(s["cached"])[r] + t
    cos, sin = _angles(_dev(s["pos"])[r] + t, c)
    page = _dev(s["tables"])[r, slot // PAGE]
    s["q_rot"].copy_(_rotate(s["q"], cos, sin))
    s["k"][0].transpose(1, 2)[page, slot % PAGE] = _rotate(s["k_new"], cos, sin).to(s["k"].dtype)
    s["v"][0].transpose(1, 2)[page, slot % PAGE] = s["v_new"]
    s["w"][0].transpose(1, 2)[r, slot] = 0.0


def _gathered(s, cache, length):
    """[n, hkv, tokens, d] in 32 bits, zero past each request's length."""
    c, top = s["case"], max(length)
    x = cache[0][_dev(s["tables"])]  # [n, pages, hkv, PAGE, d]
    x = x.transpose(1, 2).reshape(c["n"], c["hkv"], -1, c["d"])[:, :, :top].float()
    return x.masked_fill_(torch.arange(top, device="cuda")[None, None, :, None] >= _dev(length)[:, None, None, None], 0.0)


def _decode(s):
    c, T = s["case"], max(s["cached"])
    cos, sin = _angles(_dev(s["pos"]), c)
    q = _rotate(s["q"], cos, sin).reshape(c["n"], c["hkv"], -1, c["d"])
    z = q @ _gathered(s, s["k"], s["cached"]).transpose(-1, -2) / math.sqrt(c["d"])
    z.masked_fill_(torch.arange(T, device="cuda") >= _dev(s["cached"])[:, None, None, None], -math.inf)
    e = torch.exp(z - z.amax(-1, keepdim=True))
    a = e / e.sum(-1, keepdim=True)
    s["out"].copy_((a @ _gathered(s, s["v"], s["cached"])).reshape(s["out"].shape))
    s["w"][0, :, :, :T] += a.sum(2)


def _chunk(s):
    c, G, m = s["case"], s["case"]["hq"] // s["case"]["hkv"], max(s["new"])
    total = [a + b for a, b in zip(s["cached"], s["new"])]
    T = max(total)
    r, t = _packed(s)
    q = torch.zeros(c["n"], m, c["hq"], c["d"], device="cuda")
    q[r, t] = s["q"].float()
    q = q.reshape(c["n"], m, c["hkv"], G, c["d"]).permute(0, 2, 3, 1, 4).reshape(c["n"], c["hkv"], G * m, c["d"])
    z = q @ _gathered(s, s["k"], total).transpose(-1, -2)
    z = z.div_(math.sqrt(c["d"])).view(c["n"], c["hkv"], G, m, T)
    step, key = torch.arange(m, device="cuda"), torch.arange(T, device="cuda")
    seen = key <= _dev(s["cached"])[:, None, None] + step[:, None]  # [n, m, T]
    z.masked_fill_(~seen[:, None, None], -math.inf)
    a = z.sub_(z.amax(-1, keepdim=True)).exp_()
    a = a.div_(a.sum(-1, keepdim=True))
    a.masked_fill_((step >= _dev(s["new"])[:, None])[:, None, None, :, None], 0.0)  # past a request's last token
    o = a.view(c["n"], c["hkv"], G * m, T) @ _gathered(s, s["v"], total)
    o = o.view(c["n"], c["hkv"], G, m, c["d"]).permute(0, 3, 1, 2, 4).reshape(c["n"], m, c["hq"], c["d"])
    s["out"].copy_(o[r, t])
    s["w"][0, :, :, :T] += a.sum((2, 3))


def _evict(s):
    c = s["case"]
    s["w"].copy_(s["w0"])
    T = max(s["cached"])
    slot = torch.arange(T, device="cuda")
    have, keep = _dev(s["cached"])[:, None, None], _dev(s["keep"])[:, None, None]  # [n, 1, 1]
    w = s["w"][:, :, :, :T].clone()  # [L, n, hkv, T]
    w.masked_fill_(slot >= have - torch.clamp(keep, max=RECENT), math.inf)  # the recent window
    w.masked_fill_(slot >= have, -math.inf)  # past the request
    order = torch.sort(w, dim=-1, descending=True, stable=True).indices  # equal weights: the lower slot first
    kept = torch.zeros_like(w, dtype=torch.bool).scatter_(-1, order, (slot < keep).expand_as(order))
    layer, r, h, src = kept.nonzero(as_tuple=True)
    dst = (torch.cumsum(kept, -1) - 1)[layer, r, h, src]
    table = _dev(s["tables"])

    def row(x):
        return ((layer * s["k"].shape[1] + table[r, x // PAGE]) * c["hkv"] + h) * PAGE + x % PAGE

    a, b = row(src), row(dst)
    for cache in (s["k"], s["v"]):
        flat = cache.view(-1, c["d"])
        flat[b] = flat[a]
    s["w"][layer, r, h, dst] = s["w"][layer, r, h, src]


# ---- what a pass cannot do without -------------------------------------------

def work(case):
    cached, new = _lengths(case)
    L, hq, hkv, d = (case[k] for k in ("layers", "hq", "hkv", "d"))
    e = 4 if case["kv"] == "f32" else 2
    N, T = sum(new), sum(cached)
    if case["op"] == "append":
        return {"bytes": N * ((2 * hq + 4 * hkv) * d * e + 4 * hkv), "flops": 3 * N * (hq + hkv) * d}
    if case["op"] == "decode":
        return {"bytes": T * hkv * (2 * d * e + 8) + case["n"] * hq * d * (e + 4), "flops": 4 * T * hq * d}
    if case["op"] == "chunk":
        seen = sum(b * a + b * (b + 1) // 2 for a, b in zip(cached, new))  # (query, key) pairs of a head
        return {"bytes": (T + N) * hkv * (2 * d * e + 8) + 2 * N * hq * d * e, "flops": 4 * seen * hq * d}
    rows = sum(k for k in _budget(case, cached))
    return {"bytes": L * hkv * (4 * T + 2 * rows * (2 * d * e + 4)), "flops": L * hkv * T}


# ---- the definition in 64 bits -------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op, d, G = case["op"], case["d"], case["hq"] // case["hkv"]
    inv = np.power(case["theta"], -np.arange(0, d, 2) / d)
    at = 0
    if op == "evict":
        for r, (T, keep) in enumerate(zip(s["cached"], s["keep"])):
            recent = min(RECENT, keep)
            for layer in range(case["layers"]):
                w = s["w"][layer, r, :, :T]
                rank = w[:, :T - recent].double().neg().argsort(dim=-1, stable=True)[:, :keep - recent]
                tail = torch.arange(T - recent, T, device="cuda").expand(case["hkv"], recent)
                index = torch.cat([rank, tail], 1).sort(-1).values  # [hkv, keep]
                table = torch.as_tensor(s["tables"][r], device="cuda").long()
                h = torch.arange(case["hkv"], device="cuda")[:, None]
                to = torch.arange(keep, device="cuda").expand_as(index)
                for x in (s["k"][layer], s["v"][layer]):
                    x[table[to // PAGE], h, to % PAGE] = x[table[index // PAGE], h, index % PAGE].clone()
                w[:, :keep] = w.gather(1, index)
        return {"k": s["k"], "v": s["v"], "w": s["w"]}
    out, w = (torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda"), s["w"].double())
    if op == "append":
        k, v = s["k"].double(), s["v"].double()
    for r, (c, m) in enumerate(zip(s["cached"], s["new"])):
        m = 1 if op == "decode" else m
        ang = torch.as_tensor((s["pos"][r] + np.arange(m))[:, None, None] * inv, device="cuda")
        cos, sin = ang.cos(), ang.sin()

        def turn(x):
            x = x.double()
            lo, hi = x[..., :d // 2], x[..., d // 2:]
            return torch.cat([lo * cos - hi * sin, lo * sin + hi * cos], -1)

        table = torch.as_tensor(s["tables"][r], device="cuda").long()
        q = s["q"][at:at + m]
        if op == "append":
            slots = torch.arange(c, c + m, device="cuda")
            out[at:at + m] = turn(q)
            k[0, table[slots // PAGE], :, slots % PAGE] = turn(s["k_new"][at:at + m])
            v[0, table[slots // PAGE], :, slots % PAGE] = s["v_new"][at:at + m].double()
            w[0, r, :, c:c + m] = 0.0
        else:
            T = c if op == "decode" else c + m
            q = turn(q) if op == "decode" else q.double()
            for h in range(case["hkv"]):
                keys = s["k"][0, table, h].reshape(-1, d)[:T].double()
                vals = s["v"][0, table, h].reshape(-1, d)[:T].double()
                for g in range(h * G, h * G + G):
                    z = q[:, g] @ keys.T / math.sqrt(d)
                    if op == "chunk":
                        z = z + torch.full_like(z, -math.inf).triu(c + 1)
                    p = torch.softmax(z, -1)
                    out[at:at + m, g] = p @ vals
                    w[0, r, h, :T] += p.sum(0)
        at += m
    return {"q_rot": out, "k": k, "v": v, "w": w} if op == "append" else {"out": out, "w": w}
