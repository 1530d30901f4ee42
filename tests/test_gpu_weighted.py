"""Accumulated attention weights, through the C ABI, against plain formulas in
64 bits: gp_append_tokens, gp_decode_attention_weighted, gp_chunk_attention and
gp_evict_weighted, each at the lengths, masks and types where it can go wrong,
and a run of them together.

Tolerances (worst cases of the arithmetic, set before the first run):
  * a rounding to type t: |x| eps(t) / 2 (bf16 2^-8, fp32 2^-24);
  * RoPE: the angle is reduced in fp64 and rounded to fp32 (|angle| <= pi:
    pi 2^-24 < 1.9e-7), sincosf adds at most 2 ulp (1.2e-7), two products and a
    sum 2^-23 each: |error| <= 6e-7 (|a| + |b|) for the pair (a, b);
  * a logit: d products summed in fp32, in any order, each partial sum off by
    at most 2^-23 (a truncating accumulator) of sum |q_i k_i| <= |q| |k|, and
    the rotated query off by 6e-7 of its pair: dz = ((d + 16) 2^-23 + 1.2e-6)
    |q| |k| / sqrt(d);
  * a weight e^(z - m) / l: relative error 2 dz + (T + 64) 2^-23, T weights in
    the sum;
  * an output sum a v: that twice, of sum a |v|; where the weights are rounded
    to bf16 for the tensor core, 2^-8 of sum a |v| more; then its own rounding;
  * an accumulated weight: its terms' errors, plus one fp32 rounding of the
    sum per term or fewer, (terms + 2) 2^-23 of it.
Moved and cleared rows, kept sets and everything not written are exact.
"""

import math

import numpy as np
import pytest
import torch

import paged_kv_cache_step_gb300 as gp

pytestmark = pytest.mark.gpu

PAGE = 256
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
GPD = {"bf16": gp.GP_DTYPE_BF16, "f32": gp.GP_DTYPE_F32}
EPS = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


class Engine:
    """A small engine over random caches: n requests of the given pages, the
    pages shuffled, NaN in every cache slot and weight (a call may use only
    what the caller put there)."""

    def __init__(self, pages, L=2, hq=8, hkv=2, d=128, kv="bf16", q="bf16", theta=5.0e5, spare=0, seed=0, stream=None,
                 recent=16, kernel=None, cap=None):
        self.L, self.hq, self.hkv, self.d, self.G, self.kv, self.qt, self.theta = L, hq, hkv, d, hq // hkv, kv, q, theta
        self.recent = recent
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        self.pool = sum(pages) + spare
        self.cap = cap or max(pages)
        shape = (L, self.pool, hkv, PAGE, d)
        self.k = torch.full(shape, math.nan, dtype=DT[kv], device="cuda")
        self.v = torch.full(shape, math.nan, dtype=DT[kv], device="cuda")
        self.w = torch.full((L, len(pages), hkv, self.cap * PAGE), math.nan, device="cuda")
        cfg = gp.gp_config_default(num_layers=L, num_q_heads=hq, num_kv_heads=hkv, head_dim=d, kv_dtype=GPD[kv],
                                   q_dtype=GPD[q], max_slots=len(pages), num_pages=self.pool, rope_theta=theta,
                                   max_pages_per_req=self.cap, recent_window=recent)
        self.stream = stream
        self.ctx = gp.gp_create(cfg, self.k, self.v, stream or torch.cuda.current_stream())
        if kernel is not None:
            gp.gp_set_scan_kernel(self.ctx, kernel)
        order = np.random.default_rng(seed).permutation(self.pool)
        for _ in range(self.pool):
            gp.gp_page_alloc(self.ctx)
        at, self.reqs = 0, []
        for p in pages:
            self.reqs.append(gp.Request(gp.gp_slot_acquire(self.ctx), order[at:at + p], 0, self.cap))
            at += p
        for pg in order[at:]:
            gp.gp_page_unref(self.ctx, int(pg))

    def close(self):
        torch.cuda.synchronize()
        gp.gp_destroy(self.ctx)

    def randn(self, *shape):
        return torch.randn(*shape, device="cuda", generator=self.gen)

    def fill(self, tokens, weights=True):
        """Random rows (and weights) for the first tokens[r] slots of each request."""
        for r, T in enumerate(tokens):
            pages, slots = self.at(r, torch.arange(T, device="cuda"))
            for cache in (self.k, self.v):
                cache[:, pages, :, slots] = self.randn(T, self.L, self.hkv, self.d).to(cache.dtype)
            if weights:
                self.w[:, r, :, :T] = torch.exp(self.randn(self.L, self.hkv, T))

    def at(self, r, slots):
        """Pages and in-page slots of logical slots, as index tensors."""
        table = torch.as_tensor(self.reqs[r].table.astype(np.int64), device="cuda")
        return table[slots // PAGE], slots % PAGE

    def rows(self, cache, r, layer, h, T):
        pages, slots = self.at(r, torch.arange(T, device="cuda"))
        return cache[layer, pages, h, slots].double()

    def rope(self, x, pos):
        """x [rows, heads, d], pos [rows]; in 64 bits."""
        inv = self.theta ** (-torch.arange(0, self.d, 2, dtype=torch.float64, device="cuda") / self.d)
        ang = pos.double()[:, None, None] * inv
        a, b = x.double().chunk(2, -1)
        return torch.cat([a * ang.cos() - b * ang.sin(), b * ang.cos() + a * ang.sin()], -1)


def rope_tol(x, ref, eps):
    a, b = x.double().abs().chunk(2, -1)
    return eps * ref.abs() + 6.1e-7 * torch.cat([a + b, a + b], -1)


def bits(t):
    return t.view(torch.int16 if t.element_size() == 2 else torch.int32)


def softmax_reference(q, keys, vals, first):
    """q [m, G, d] (rotated, 64 bits); token t sees `first` + t + 1 slots:
    outputs [m, G, d], weights summed [T], and their bounds (see above)."""
    m, G, d = q.shape
    T = keys.shape[0]
    z = torch.einsum("mgd,td->gmt", q, keys) / math.sqrt(d)
    see = torch.arange(T, device="cuda") <= first + torch.arange(m, device="cuda")[:, None]
    z = z.masked_fill(~see, -math.inf)
    a = torch.softmax(z, -1)
    dz = ((d + 16) * 2.0 ** -23 + 1.2e-6) * q.norm(dim=-1).max() * keys.norm(dim=-1).max() / math.sqrt(d)
    rel = 2 * dz + (T + 64) * 2.0 ** -23
    out = torch.einsum("gmt,td->mgd", a, vals)
    mag = torch.einsum("gmt,td->mgd", a, vals.abs())
    return out, mag, a.sum((0, 1)), rel.item()


# ---- gp_append_tokens --------------------------------------------------------

APPEND = [("bf16", "bf16", 128, 8, 2), ("bf16", "bf16", 64, 4, 2), ("f32", "f32", 64, 4, 1), ("bf16", "f32", 128, 6, 3),
          ("f32", "bf16", 128, 4, 2)]


@pytest.mark.parametrize("kv,q,d,hq,hkv", APPEND)
@pytest.mark.parametrize("in_place", [False, True])
def test_append_tokens(kv, q, d, hq, hkv, in_place):
    cached, new = [0, 255, 256, 7, 100, 511, 0], [1, 2, 256, 0, 700, 1, 513]
    e = Engine([-(-(a + b) // PAGE) + 1 for a, b in zip(cached, new)], hq=hq, hkv=hkv, d=d, kv=kv, q=q, seed=d + hq)
    try:
        for r, pos in enumerate([0, 255, 1_000_003, 7, 123_456, 2 ** 31 + 11, 65_535]):
            e.reqs[r].pos = pos
        layer, n = 1, sum(new)
        qx = e.randn(n, hq, d).to(DT[q])
        kx, vx = (3.0 * e.randn(n, hkv, d)).to(DT[kv]), e.randn(n, hkv, d).to(DT[kv])
        vx[0, 0, :2] = torch.tensor([math.inf, math.nan])  # values are copied, whatever they are
        want_k, want_v, want_w = e.k.clone(), e.v.clone(), e.w.clone()
        r = torch.as_tensor(np.repeat(np.arange(len(new)), new), device="cuda")
        t = torch.cat([torch.arange(x) for x in new]).cuda()
        pos = torch.tensor([x.pos for x in e.reqs], device="cuda")[r] + t
        kr, qr = e.rope(kx, pos), e.rope(qx, pos)
        src = qx.clone()
        rot = src if in_place else torch.full_like(qx, math.nan)
        gp.gp_append_tokens(e.ctx, layer, e.reqs, cached, new, src, kx, vx, rot, e.w)
        gp.gp_synchronize(e.ctx)
        assert torch.all((rot.double() - qr).abs() <= rope_tol(qx, qr, EPS[q]))
        at = 0
        for i, (c, m) in enumerate(zip(cached, new)):
            pages, slots = e.at(i, torch.arange(c, c + m, device="cuda"))
            got = e.k[layer, pages, :, slots].double()
            assert torch.all((got - kr[at:at + m]).abs() <= rope_tol(kx[at:at + m], kr[at:at + m], EPS[kv]))
            want_k[layer, pages, :, slots] = e.k[layer, pages, :, slots]
            want_v[layer, pages, :, slots] = vx[at:at + m]
            want_w[layer, i, :, c:c + m] = 0.0
            at += m
        # the values, the cleared weights, and nothing else
        assert torch.equal(bits(e.v), bits(want_v)) and torch.equal(bits(e.w), bits(want_w))
        assert torch.equal(bits(e.k), bits(want_k))
    finally:
        e.close()


def test_append_without_queries_or_weights():
    e = Engine([2], L=1)
    try:
        k, v = e.randn(300, 2, 128).bfloat16(), e.randn(300, 2, 128).bfloat16()
        gp.gp_append_tokens(e.ctx, 0, e.reqs, [0], [300], None, k, v, None)
        gp.gp_synchronize(e.ctx)
        ref = e.rope(k, torch.arange(300, device="cuda"))
        for h in range(2):
            assert torch.all((e.rows(e.k, 0, 0, h, 300) - ref[:, h]).abs() <= rope_tol(k, ref, EPS["bf16"])[:, h])
            assert torch.equal(e.rows(e.v, 0, 0, h, 300), v[:, h].double())
        assert torch.isnan(e.w).all()
    finally:
        e.close()


@pytest.mark.parametrize("pages,new", [([1] * 66, [1] * 66), ([131, 1], [33_100, 200]), ([2] * 64, [300] * 64),
                                       ([2] * 65, [256] * 65)])
def test_append_tables_beyond_the_launch_parameters(pages, new):
    """At and over the 64 requests and 128 pages whose tables travel as launch parameters."""
    e = Engine(pages, L=1, hq=2, hkv=1, d=64, seed=16)
    try:
        cached = [200 if m == 1 else 0 for m in new]
        for r, req in enumerate(e.reqs):
            req.pos = 1000 * r
        n = sum(new)
        q, k, v = e.randn(n, 2, 64).bfloat16(), e.randn(n, 1, 64).bfloat16(), e.randn(n, 1, 64).bfloat16()
        rot = torch.empty_like(q)
        gp.gp_append_tokens(e.ctx, 0, e.reqs, cached, new, q, k, v, rot, e.w)
        gp.gp_synchronize(e.ctx)
        pos = torch.cat([1000 * r + torch.arange(m) for r, m in enumerate(new)]).cuda()
        kr, qr = e.rope(k, pos), e.rope(q, pos)
        assert torch.all((rot.double() - qr).abs() <= rope_tol(q, qr, EPS["bf16"]))
        tol, at = rope_tol(k, kr, EPS["bf16"]), 0
        for r, (c, m) in enumerate(zip(cached, new)):
            assert torch.all((e.rows(e.k, r, 0, 0, c + m)[c:] - kr[at:at + m, 0]).abs() <= tol[at:at + m, 0])
            assert torch.equal(e.rows(e.v, r, 0, 0, c + m)[c:], v[at:at + m, 0].double())
            assert not e.w[0, r, 0, c:c + m].any() and torch.isnan(e.w[0, r, 0, c + m:]).all()
            at += m
    finally:
        e.close()


# ---- gp_decode_attention_weighted ---------------------------------------------

SHAPES = {"bf16_g4_d128": dict(hq=8, hkv=2), "bf16_g2_d128": dict(hq=4, hkv=2), "bf16_g2_d64": dict(hq=4, hkv=2, d=64),
          "bf16_g4_d64": dict(hq=4, hkv=1, d=64), "f32_g4_d128": dict(hq=8, hkv=2, kv="f32", q="f32"),
          "f32_g2_d64": dict(hq=6, hkv=3, d=64, kv="f32", q="f32"), "bf16_q32_g2_d128": dict(hq=4, hkv=2, q="f32")}


def kernels(shape, decode):
    """AUTO, and the other kernel where AUTO is the tensor core."""
    s = SHAPES[shape]
    tc = s.get("kv", "bf16") == "bf16" and (s.get("d", 128) == 128 if decode else s.get("q", "bf16") == "bf16")
    return [gp.GP_SCAN_TENSOR_CORE, gp.GP_SCAN_CUDA_CORE] if tc else [gp.GP_SCAN_AUTO]


@pytest.mark.parametrize("shape,kernel", [(s, k) for s in SHAPES for k in kernels(s, True)])
@pytest.mark.parametrize("summaries", [False, True])
def test_decode_attention_weighted(shape, kernel, summaries):
    tokens = [0, 1, 255, 256, 257, 640, 1024, 9 * PAGE - 130]
    e = Engine([max(1, -(-t // PAGE)) for t in tokens], kernel=kernel, seed=3, **SHAPES[shape])
    try:
        e.fill(tokens)
        w0, layer, n = e.w.double(), 1, len(tokens)
        for r, req in enumerate(e.reqs):
            req.pos = tokens[r] + 1000 * r
        q = e.randn(n, e.hq, e.d).to(DT[e.qt])
        first = torch.ones(n, dtype=torch.uint8, device="cuda") if summaries else None
        out = torch.full((n, e.hq, e.d), math.nan, device="cuda")
        untouched = e.w.clone()
        gp.gp_decode_attention_weighted(e.ctx, layer, e.reqs, tokens, q, first, out, e.w)
        gp.gp_synchronize(e.ctx)
        qr = e.rope(q, torch.tensor([x.pos for x in e.reqs], device="cuda"))
        for r, T in enumerate(tokens):
            s = gp.gp_read_summaries(e.ctx, e.reqs[r].slot, e.L, e.hq, e.d)
            assert np.array_equal(s[layer], np.broadcast_to(q[r].double().cpu().numpy(), s[layer].shape)) or not summaries
            assert summaries or not s.any()
            for h in range(e.hkv):
                heads = slice(h * e.G, h * e.G + e.G)
                if T == 0:
                    assert torch.all(out[r, heads] == 0.0)
                    continue
                ref, mag, w, rel = softmax_reference(qr[r:r + 1, heads], e.rows(e.k, r, layer, h, T),
                                                     e.rows(e.v, r, layer, h, T), T)
                assert torch.all((out[r, heads].double() - ref[0]).abs() <= 2 * rel * mag[0]), (shape, r, h)
                want = w0[layer, r, h, :T] + w
                err = (e.w[layer, r, h, :T].double() - want).abs()
                assert torch.all(err <= rel * w + (e.G + 2) * 2.0 ** -23 * want), (shape, r, h, err.max())
                untouched[layer, r, h, :T] = e.w[layer, r, h, :T]
        assert torch.equal(bits(e.w), bits(untouched))
        # a second step adds to the first's; the same calls give the same bits
        again, twin = e.w.clone(), e.w.clone()
        o1, o2 = torch.empty_like(out), torch.empty_like(out)
        for w_, o_ in ((again, o1), (twin, o2)):
            gp.gp_decode_attention_weighted(e.ctx, layer, e.reqs, tokens, q, None, o_, w_)
        gp.gp_synchronize(e.ctx)
        assert torch.equal(bits(again), bits(twin)) and torch.equal(o1, o2)
        # and the outputs are gp_decode_attention's
        zero = torch.zeros(n, dtype=torch.uint8, device="cuda")
        gp.gp_decode_attention(e.ctx, layer, e.reqs, tokens, q, zero, o2)
        gp.gp_synchronize(e.ctx)
        assert torch.equal(o1, o2)
    finally:
        e.close()


def test_decode_weighted_many_pairs():
    """More pairs than SMs and pairs in several pieces: weights of one row sum to G."""
    rng = np.random.default_rng(5)
    pages = [int(x) for x in rng.integers(1, 4, size=90)] + [70]
    tokens = [int(rng.integers(1, p * PAGE + 1)) for p in pages]
    e = Engine(pages, L=1, seed=6)
    try:
        e.fill(tokens, weights=False)
        for r, T in enumerate(tokens):
            e.w[0, r, :, :T] = 0.0
        q = e.randn(len(pages), 8, 128).bfloat16()
        out = torch.empty(len(pages), 8, 128, device="cuda")
        gp.gp_decode_attention_weighted(e.ctx, 0, e.reqs, tokens, q, None, out, e.w)
        gp.gp_synchronize(e.ctx)
        qr = e.rope(q, torch.zeros(len(pages), device="cuda"))
        for r, T in enumerate(tokens):
            for h in range(2):
                _, _, w, rel = softmax_reference(qr[r:r + 1, 4 * h:4 * h + 4], e.rows(e.k, r, 0, h, T),
                                                 e.rows(e.v, r, 0, h, T), T)
                err = (e.w[0, r, h, :T].double() - w).abs()
                assert torch.all(err <= (rel + 6 * 2.0 ** -23) * w), (r, h)
    finally:
        e.close()


# ---- gp_chunk_attention --------------------------------------------------------

CHUNKS = {
    "short": ([0, 0, 1, 127, 128, 1000, 255, 40], [1, 2, 1, 5, 17, 0, 3, 33]),
    "tiles": ([0, 0, 64, 128, 200], [128, 129, 127, 256, 65]),
    "long": ([0, 513], [700, 391]),
    "one_over_long": ([7777], [3]),
}


def check_chunk(e, layer, cached, new, q, out, w_before, w_after, tc):
    at, untouched = 0, w_before.clone()
    for r, (c, m) in enumerate(zip(cached, new)):
        if m == 0:
            continue
        T = c + m
        for h in range(e.hkv):
            heads = slice(h * e.G, h * e.G + e.G)
            ref, mag, w, rel = softmax_reference(q[at:at + m, heads].double(), e.rows(e.k, r, layer, h, T),
                                                 e.rows(e.v, r, layer, h, T), c)
            tol = (2 * rel + (2.0 ** -8 if tc else 0.0)) * mag
            tol = tol + EPS[e.qt] * (ref.abs() + tol)
            err = (out[at:at + m, heads].double() - ref).abs()
            assert torch.all(err <= tol), (r, h, (err / tol).max())
            if w_after is not None:
                want = w_before[layer, r, h, :T].double() + w
                err = (w_after[layer, r, h, :T].double() - want).abs()
                assert torch.all(err <= rel * w + (m * e.G + 2) * 2.0 ** -23 * want), (r, h, err.max())
                untouched[layer, r, h, :T] = w_after[layer, r, h, :T]
        at += m
    if w_after is not None:
        assert torch.equal(bits(w_after), bits(untouched))


@pytest.mark.parametrize("shape,kernel", [(s, k) for s in SHAPES for k in kernels(s, False)])
@pytest.mark.parametrize("chunk", sorted(CHUNKS))
def test_chunk_attention(shape, kernel, chunk):
    cached, new = CHUNKS[chunk]
    e = Engine([-(-max(1, a + b) // PAGE) for a, b in zip(cached, new)], kernel=kernel, seed=11, **SHAPES[shape])
    tc = kernel == gp.GP_SCAN_TENSOR_CORE
    try:
        e.fill([a + b for a, b in zip(cached, new)])
        n, layer = sum(new), 1
        # a buffer longer than the rows: what lies behind the last sequence stays
        q = torch.full((n + 5, e.hq, e.d), math.nan, device="cuda", dtype=DT[e.qt])
        q[:n] = e.randn(n, e.hq, e.d).to(q.dtype)
        out = torch.full_like(q, 7.0)
        w = e.w.clone()
        gp.gp_chunk_attention(e.ctx, layer, e.reqs, cached, new, q, out, w)
        gp.gp_synchronize(e.ctx)
        assert torch.all(out[n:] == 7.0)
        check_chunk(e, layer, cached, new, q, out, e.w, w, tc)
        # without weights: the same outputs; twice: the same bits
        o2, w2 = torch.full_like(q, 7.0), e.w.clone()
        gp.gp_chunk_attention(e.ctx, layer, e.reqs, cached, new, q, o2, None)
        gp.gp_synchronize(e.ctx)
        assert torch.equal(bits(o2), bits(out))
        gp.gp_chunk_attention(e.ctx, layer, e.reqs, cached, new, q, o2, w2)
        gp.gp_synchronize(e.ctx)
        assert torch.equal(bits(o2), bits(out)) and torch.equal(bits(w), bits(w2))
    finally:
        e.close()


@pytest.mark.parametrize("kernel", [gp.GP_SCAN_AUTO, gp.GP_SCAN_CUDA_CORE])
def test_chunk_attention_concentrated(kernel):
    """Logits up to hundreds, the maximum late in the cache, then early: the
    running maximum moves far in both directions."""
    cached, new = [900, 0], [200, 300]
    e = Engine([5, 2], L=1, kernel=kernel, seed=13)
    try:
        e.fill([1100, 300])
        pages, slots = e.at(0, torch.arange(0, 1100, device="cuda"))
        ramp = torch.linspace(0.2, 6.0, 1100, device="cuda")[:, None, None]
        e.k[0, pages, :, slots] = (ramp * e.k[0, pages, :, slots].float()).to(e.k.dtype)
        pages, slots = e.at(1, torch.arange(0, 300, device="cuda"))
        e.k[0, pages, :, slots] = (torch.linspace(8.0, 0.1, 300, device="cuda")[:, None, None]
                                   * e.k[0, pages, :, slots].float()).to(e.k.dtype)
        q = (4.0 * e.randn(500, 8, 128)).bfloat16()
        out, w = torch.empty_like(q), e.w.clone()
        gp.gp_chunk_attention(e.ctx, 0, e.reqs, cached, new, q, out, w)
        gp.gp_synchronize(e.ctx)
        check_chunk(e, 0, cached, new, q, out, e.w, w, kernel != gp.GP_SCAN_CUDA_CORE)
    finally:
        e.close()


@pytest.mark.parametrize("shape", ["bf16_g2_d64", "bf16_g4_d128"])
def test_chunk_attention_long_beside_short(shape):
    """One drafted token chunk over a cache long enough that single query tiles
    get a launch of their own, beside prompts of pairs and of odd tiles; rows
    of the weights longer than any request."""
    cached, new = [33000, 0, 130, 0], [5, 300, 2, 1]
    d = SHAPES[shape].get("d", 128)
    e = Engine([130, 2, 1, 1], L=1, hq=16 if d == 64 else 32, hkv=8, d=d, seed=14, cap=140)
    try:
        e.fill([33005, 300, 132, 1])
        q = e.randn(sum(new), e.hq, e.d).bfloat16()
        out, w = torch.full_like(q, math.nan), e.w.clone()
        gp.gp_chunk_attention(e.ctx, 0, e.reqs, cached, new, q, out, w)
        gp.gp_synchronize(e.ctx)
        check_chunk(e, 0, cached, new, q, out, e.w, w, True)
    finally:
        e.close()


def test_the_longest_request():
    """256 pages, 65 536 tokens: appended to, attended to by a chunk and a step,
    evicted by one and by half (over the length that the selection stages)."""
    T = 65536
    e = Engine([256], L=1, hq=2, hkv=1, d=64, seed=15)
    try:
        e.fill([T - 40])
        e.reqs[0].pos = 1_000_000
        qx, kx, vx = (e.randn(40, h, 64).bfloat16() for h in (2, 1, 1))
        rot = torch.empty_like(qx)
        gp.gp_append_tokens(e.ctx, 0, e.reqs, [T - 40], [40], qx, kx, vx, rot, e.w)
        out, w = torch.empty_like(rot), e.w.clone()
        gp.gp_chunk_attention(e.ctx, 0, e.reqs, [T - 40], [40], rot, out, w)
        gp.gp_synchronize(e.ctx)
        check_chunk(e, 0, [T - 40], [40], rot, out, e.w, w, True)
        e.w.copy_(w)
        one, w1 = torch.empty(1, 2, 64, device="cuda"), e.w.clone()
        gp.gp_decode_attention_weighted(e.ctx, 0, e.reqs, [T], qx[:1].contiguous(), None, one, w1)
        gp.gp_synchronize(e.ctx)
        qr = e.rope(qx[:1], torch.tensor([1_000_000], device="cuda"))
        ref, mag, ws, rel = softmax_reference(qr, e.rows(e.k, 0, 0, 0, T), e.rows(e.v, 0, 0, 0, T), T)
        assert torch.all((one[0].double() - ref[0]).abs() <= 2 * rel * mag[0])
        want = e.w[0, 0, 0].double() + ws
        assert torch.all((w1[0, 0, 0].double() - want).abs() <= rel * ws + 4 * 2.0 ** -23 * want)
        for tokens, keep in ((T, T - 1), (T - 1, 30001)):
            k0, v0, w0, t0 = e.k.clone(), e.v.clone(), e.w.clone(), [e.reqs[0].pages]
            gp.gp_evict_weighted(e.ctx, e.reqs, [tokens], [keep], e.w)
            gp.gp_synchronize(e.ctx)
            check_evict(e, [tokens], [keep], k0, v0, w0, t0)
    finally:
        e.close()


@pytest.mark.parametrize("kernel", [gp.GP_SCAN_AUTO, gp.GP_SCAN_CUDA_CORE])
def test_requests_on_shared_pages_gather_their_own_weights(kernel):
    """Two requests with the same first two pages: chunks and decode steps of both
    in one call, each with weights of its own."""
    cached, new = [512, 700], [9, 150]
    e = Engine([3, 4], L=1, seed=17, kernel=kernel)
    try:
        for j in range(2):
            gp.gp_page_ref(e.ctx, int(e.reqs[0].table[j]))
            gp.gp_page_unref(e.ctx, int(e.reqs[1].table[j]))
            e.reqs[1].table[j] = e.reqs[0].table[j]
        e.fill([521, 850])
        q = e.randn(159, e.hq, e.d).bfloat16()
        out, w = torch.full_like(q, math.nan), e.w.clone()
        gp.gp_chunk_attention(e.ctx, 0, e.reqs, cached, new, q, out, w)
        gp.gp_synchronize(e.ctx)
        check_chunk(e, 0, cached, new, q, out, e.w, w, kernel == gp.GP_SCAN_AUTO)
        one, w1 = torch.empty(2, e.hq, e.d, device="cuda"), w.clone()
        gp.gp_decode_attention_weighted(e.ctx, 0, e.reqs, [521, 850], q[:2].contiguous(), None, one, w1)
        gp.gp_synchronize(e.ctx)
        qr = e.rope(q[:2], torch.zeros(2, device="cuda"))
        for r, T in enumerate([521, 850]):
            for h in range(e.hkv):
                heads = slice(h * e.G, h * e.G + e.G)
                ref, mag, ws, rel = softmax_reference(qr[r:r + 1, heads], e.rows(e.k, r, 0, h, T), e.rows(e.v, r, 0, h, T), T)
                assert torch.all((one[r, heads].double() - ref[0]).abs() <= 2 * rel * mag[0])
                want = w[0, r, h, :T].double() + ws
                assert torch.all((w1[0, r, h, :T].double() - want).abs() <= rel * ws + (e.G + 2) * 2.0 ** -23 * want)
    finally:
        e.close()


# ---- gp_evict_weighted ---------------------------------------------------------

def order_key(w):
    """The order that eviction goes by: NaN above every number, -0 equal to 0."""
    return np.where(np.isnan(w), np.inf, np.where(w == np.inf, np.finfo(np.float32).max, w)).astype(np.float64)


def kept_slots(w, T, keep, recent):
    recent = min(recent, keep)
    key = order_key(w[:T - recent])
    top = np.argsort(-key, kind="stable")[:keep - recent]
    return np.sort(np.concatenate([top, np.arange(T - recent, T)]))


def check_evict(e, tokens, keep, k0, v0, w0, tables0):
    """Everything after an eviction against the definition, bit for bit."""
    want_w = w0.clone()
    for r, (T, kp) in enumerate(zip(tokens, keep)):
        if T <= kp:
            assert e.reqs[r].pages == tables0[r]
            continue
        mask = gp.unpack_mask(gp.gp_debug_keep_mask(e.ctx, r, e.L * e.hkv, e.reqs[r].num_pages),
                              e.reqs[r].num_pages * PAGE)
        old = torch.as_tensor(np.asarray(tables0[r], dtype=np.int64), device="cuda")
        for layer in range(e.L):
            for h in range(e.hkv):
                idx = kept_slots(w0[layer, r, h].cpu().numpy(), T, kp, e.recent)
                assert np.array_equal(np.nonzero(mask[layer * e.hkv + h])[0], idx), (r, layer, h)
                i = torch.as_tensor(idx, device="cuda")
                pages, slots = e.at(r, torch.arange(kp, device="cuda"))
                for now, was in ((e.k, k0), (e.v, v0)):
                    assert torch.equal(bits(now[layer, pages, h, slots]), bits(was[layer, old[i // PAGE], h, i % PAGE])), \
                        (r, layer, h)
                want_w[layer, r, h, :kp] = w0[layer, r, h, i]
    assert torch.equal(bits(e.w), bits(want_w))


EVICT_SHAPES = {"bf16_d128": dict(hq=8, hkv=2), "bf16_d64": dict(hq=4, hkv=2, d=64), "f32_d128": dict(hq=4, hkv=1, kv="f32", q="f32"),
                "f32_d64": dict(hq=6, hkv=3, d=64, kv="f32", q="f32")}


@pytest.mark.parametrize("shape", sorted(EVICT_SHAPES))
@pytest.mark.parametrize("recent", [0, 16, 255])
def test_evict_weighted(shape, recent):
    tokens = [0, 1, 2, 33, 256, 300, 700, 1111, 2048, 5000, 640]
    keep = [1, 1, 1, 20, 255, 64, 513, 5, 2047, 1300, 640]
    e = Engine([max(1, -(-t // PAGE)) for t in tokens], seed=21, recent=recent, **EVICT_SHAPES[shape])
    try:
        e.fill(tokens)
        k0, v0, w0, t0 = e.k.clone(), e.v.clone(), e.w.clone(), [x.pages for x in e.reqs]
        moved = gp.gp_stats(e.ctx)["moved_rows"]
        gp.gp_evict_weighted(e.ctx, e.reqs, tokens, keep, e.w)
        gp.gp_synchronize(e.ctx)
        check_evict(e, tokens, keep, k0, v0, w0, t0)
        assert gp.gp_stats(e.ctx)["moved_rows"] > moved
    finally:
        e.close()


@pytest.mark.parametrize("ties", ["few values", "all equal", "zeros", "special", "ascending", "descending"])
def test_evict_order_of_equal_and_special_weights(ties):
    tokens, keep = [3000, 777, 513], [1234, 76, 512]
    e = Engine([12, 4, 3], L=1, seed=22)
    try:
        e.fill(tokens)
        for r, T in enumerate(tokens):
            w = e.w[0, r, :, :T]
            if ties == "few values":
                w.copy_(torch.floor(4 * w.clamp(max=2.0)) / 4)
            elif ties == "all equal":
                w.fill_(0.37)
            elif ties == "zeros":
                w.copy_(torch.where(w > 1.5, w, torch.where(w > 0.7, 0.0, -0.0)))
            elif ties == "special":
                w[:, ::7], w[:, 1::11], w[:, 2::13] = math.inf, math.nan, -math.inf
                w[:, 3::17], w[:, 4::19] = -math.nan, 1.0e-45  # either NaN, a subnormal
            else:
                w.copy_(torch.arange(T, device="cuda").float() * (1 if ties == "ascending" else -1))
        k0, v0, w0, t0 = e.k.clone(), e.v.clone(), e.w.clone(), [x.pages for x in e.reqs]
        gp.gp_evict_weighted(e.ctx, e.reqs, tokens, keep, e.w)
        gp.gp_synchronize(e.ctx)
        check_evict(e, tokens, keep, k0, v0, w0, t0)
    finally:
        e.close()


@pytest.mark.parametrize("side", [False, True])
def test_evict_copies_shared_pages(side):
    """Three requests share a prefix page, one of them too short to evict: the
    evicting ones take fresh pages, the prefix stays as it was."""
    tokens, keep = [900, 1000, 400], [300, 700, 400]
    e = Engine([4, 4, 2], spare=4, seed=23, L=1)
    try:
        prefix = e.reqs[0].pages[0]
        for req in e.reqs[1:]:
            own = int(req.table[0])
            req.table[0] = prefix
            gp.gp_page_ref(e.ctx, prefix)
            gp.gp_page_unref(e.ctx, own)
        e.fill(tokens)
        k0, v0, w0, t0 = e.k.clone(), e.v.clone(), e.w.clone(), [x.pages for x in e.reqs]
        stream = torch.cuda.Stream()
        if side:
            gp.gp_set_compaction_stream(e.ctx, stream)
        free = gp.gp_free_page_count(e.ctx)
        torch.cuda.synchronize()
        gp.gp_evict_weighted(e.ctx, e.reqs, tokens, keep, e.w)
        if side:  # a decode step of the request that shares the pages waits for it on the device
            out = torch.empty(1, 8, 128, device="cuda")
            q = e.randn(1, 8, 128).bfloat16()
            gp.gp_decode_attention_weighted(e.ctx, 0, e.reqs[2:], [400], q, None, out, e.w.clone())
            gp.gp_wait_compaction(e.ctx)
        gp.gp_synchronize(e.ctx)
        assert gp.gp_free_page_count(e.ctx) == free - 2 and gp.gp_page_refcount(e.ctx, prefix) == 1
        assert e.reqs[2].pages == t0[2] and e.reqs[0].pages[0] != prefix and e.reqs[1].pages[0] != prefix
        assert e.reqs[0].pages[1:] == t0[0][1:] and gp.gp_stats(e.ctx)["cow_pages"] == 2
        assert torch.equal(bits(e.k[0, prefix]), bits(k0[0, prefix])) and torch.equal(bits(e.v[0, prefix]), bits(v0[0, prefix]))
        check_evict(e, tokens, keep, k0, v0, w0, t0)
    finally:
        gp.gp_set_compaction_stream(e.ctx, None)
        e.close()


def test_a_slot_taken_again_while_its_eviction_is_pending():
    """A request is finished while its eviction waits on the side stream; its slot
    goes to another, on a page that the eviction does not touch.  The new one's
    append clears the slot's weights after the eviction has moved them."""
    e = Engine([4], spare=1, seed=26, L=1)
    side = torch.cuda.Stream()
    try:
        e.fill([901])
        k = e.randn(200, 2, 128).bfloat16()
        gp.gp_set_compaction_stream(e.ctx, side)
        # the kernels' first launches load them, which may wait for the device
        gp.gp_append_tokens(e.ctx, 0, e.reqs, [901], [1], None, k[:1], k[:1], None, None)
        gp.gp_evict_weighted(e.ctx, e.reqs, [901], [900], e.w)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(100_000_000)  # the eviction starts well after the append has been issued
        gp.gp_evict_weighted(e.ctx, e.reqs, [900], [300], e.w)
        old = e.reqs[0]
        gp.gp_slot_release(e.ctx, old.slot)
        slot, page = gp.gp_slot_acquire(e.ctx), gp.gp_page_alloc(e.ctx)
        assert slot == old.slot and page not in old.pages
        new = gp.Request(slot, np.array([page]), 0, 4)
        gp.gp_append_tokens(e.ctx, 0, [new], [0], [200], None, k, k, None, e.w)
        gp.gp_wait_compaction(e.ctx)
        gp.gp_synchronize(e.ctx)
        torch.cuda.synchronize()
        assert not e.w[0, slot, :, :200].any() and bool((e.w[0, slot, :, 200:300] > 0).all())
    finally:
        gp.gp_set_compaction_stream(e.ctx, None)
        e.close()


def test_evict_without_pages_or_launch_changes_nothing():
    tokens, keep = [900, 1000], [300, 700]
    e = Engine([4, 4], spare=2, seed=24, L=1)
    try:
        for req, other in ((e.reqs[0], e.reqs[1]),):
            for j in range(2):  # two shared pages: four fresh ones to copy them
                own = int(other.table[j])
                other.table[j] = req.table[j]
                gp.gp_page_ref(e.ctx, int(req.table[j]))
                gp.gp_page_unref(e.ctx, own)
        spare = [gp.gp_page_alloc(e.ctx) for _ in range(gp.gp_free_page_count(e.ctx) - 1)]
        e.fill(tokens)
        k0, v0, w0, t0 = e.k.clone(), e.v.clone(), e.w.clone(), [x.pages for x in e.reqs]

        def same():
            gp.gp_synchronize(e.ctx)
            return (torch.equal(bits(e.k), bits(k0)) and torch.equal(bits(e.v), bits(v0)) and torch.equal(bits(e.w), bits(w0))
                    and [x.pages for x in e.reqs] == t0 and [gp.gp_page_refcount(e.ctx, p) for p in t0[0][:2]] == [2, 2])

        with pytest.raises(gp.GrowPageError) as err:
            gp.gp_evict_weighted(e.ctx, e.reqs, tokens, keep, e.w)
        assert err.value.status == gp.GP_ERR_NO_PAGES and same() and gp.gp_free_page_count(e.ctx) == 1
        for p in spare:
            gp.gp_page_unref(e.ctx, p)
        free = gp.gp_free_page_count(e.ctx)
        for kernel in (gp.GP_KERNEL_EVICT_SELECT, gp.GP_KERNEL_EVICT):
            gp.gp_debug_fail_next_launch(e.ctx, kernel)
            with pytest.raises(gp.GrowPageError) as err:
                gp.gp_evict_weighted(e.ctx, e.reqs, tokens, keep, e.w)
            assert err.value.status == gp.GP_ERR_CUDA and same() and gp.gp_free_page_count(e.ctx) == free
        gp.gp_evict_weighted(e.ctx, e.reqs, tokens, keep, e.w)
        gp.gp_synchronize(e.ctx)
        check_evict(e, tokens, keep, k0, v0, w0, t0)
    finally:
        e.close()


def test_evict_wait_that_gives_up_is_reported():
    e = Engine([16], seed=25)
    try:
        e.fill([4096])
        gp.gp_debug_set_wait_limit(e.ctx, gp.GP_KERNEL_EVICT, 0)
        gp.gp_evict_weighted(e.ctx, e.reqs, [4096], [2000], e.w)
        with pytest.raises(gp.GrowPageError) as err:
            gp.gp_synchronize(e.ctx)
        assert err.value.status == gp.GP_ERR_TIMEOUT
        gp.gp_debug_set_wait_limit(e.ctx, gp.GP_KERNEL_EVICT, -1)
        e.fill([4096])
        k0, v0, w0, t0 = e.k.clone(), e.v.clone(), e.w.clone(), [x.pages for x in e.reqs]
        gp.gp_evict_weighted(e.ctx, e.reqs, [4096], [2000], e.w)
        gp.gp_synchronize(e.ctx)
        check_evict(e, [4096], [2000], k0, v0, w0, t0)
    finally:
        e.close()


# ---- together, and what is refused with a device --------------------------------

@pytest.mark.parametrize("shape", ["bf16_g4_d128", "bf16_g2_d64", "f32_g2_d64"])
def test_a_request_from_prompt_to_eviction(shape):
    """Two requests: prompts in two chunks, decode steps, an eviction, decode
    steps after it.  Outputs and weights of every call against 64 bits on the
    cache as it then is; the weights' sum is the number of (query, head) pairs."""
    e = Engine([3, 4], L=1, seed=31, **SHAPES[shape])
    tc = shape != "f32_g2_d64"
    try:
        lengths, pos = [0, 0], [0, 0]

        def append(new):
            n = sum(new)
            q, k, v = (e.randn(n, x, e.d).to(DT[e.kv]) for x in (e.hq, e.hkv, e.hkv))
            rot = torch.empty_like(q)
            for r, req in enumerate(e.reqs):
                req.pos = pos[r]
            gp.gp_append_tokens(e.ctx, 0, e.reqs, lengths, new, q, k, v, rot, e.w)
            return q, rot

        for new in ([300, 1], [117, 513]):
            _, rot = append(new)
            before, out = e.w.clone(), torch.empty_like(rot)
            gp.gp_chunk_attention(e.ctx, 0, e.reqs, lengths, new, rot, out, e.w)
            gp.gp_synchronize(e.ctx)
            check_chunk(e, 0, lengths, new, rot, out, before, e.w, tc)
            for r in range(2):
                lengths[r] += new[r]
                pos[r] += new[r]
        for step in range(6):
            if step == 3:
                k0, v0, w0, t0 = e.k.clone(), e.v.clone(), e.w.clone(), [x.pages for x in e.reqs]
                keep = [200, lengths[1] + 9]
                gp.gp_evict_weighted(e.ctx, e.reqs, lengths, keep, e.w)
                gp.gp_synchronize(e.ctx)
                check_evict(e, lengths, keep, k0, v0, w0, t0)
                lengths[0] = 200
            q, _ = append([1, 1])
            for r, req in enumerate(e.reqs):
                req.pos = pos[r]
                lengths[r] += 1
                pos[r] += 1
            before, out = e.w.clone(), torch.empty(2, e.hq, e.d, device="cuda")
            gp.gp_decode_attention_weighted(e.ctx, 0, e.reqs, lengths, q, None, out, e.w)
            gp.gp_synchronize(e.ctx)
            qr = e.rope(q, torch.tensor([x.pos for x in e.reqs], device="cuda"))
            for r, T in enumerate(lengths):
                for h in range(e.hkv):
                    heads = slice(h * e.G, h * e.G + e.G)
                    ref, mag, w, rel = softmax_reference(qr[r:r + 1, heads], e.rows(e.k, r, 0, h, T),
                                                         e.rows(e.v, r, 0, h, T), T)
                    assert torch.all((out[r, heads].double() - ref[0]).abs() <= 2 * rel * mag[0])
                    want = before[0, r, h, :T].double() + w
                    assert torch.all((e.w[0, r, h, :T].double() - want).abs() <= rel * w + (e.G + 2) * 2.0 ** -23 * want)
            if step == 2:  # nothing evicted yet: every query's weights are still there
                for r in range(2):
                    total = e.w[0, r, :, :lengths[r]].double().sum(-1)
                    assert torch.allclose(total, torch.full_like(total, float(lengths[r] * e.G)), rtol=1e-5)
    finally:
        e.close()


def test_appended_tokens_make_a_demand_result_stale():
    e = Engine([2], seed=41)
    try:
        e.fill([512])
        q = e.randn(2, 1, 8, 128).bfloat16()
        first, slots = torch.ones(1, dtype=torch.uint8, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
        k = e.randn(1, 2, 128).bfloat16()

        def demand():
            gp.gp_update_summaries(e.ctx, 1, slots, q, first)
            gp.gp_boundary_demand(e.ctx, e.reqs, q)

        demand()
        gp.gp_append_tokens(e.ctx, 0, e.reqs, [511], [1], None, k, k, None)
        with pytest.raises(gp.GrowPageError) as err:
            gp.gp_compress_hold(e.ctx, e.reqs)
        assert err.value.status == gp.GP_ERR_STATE
        demand()
        gp.gp_compress_hold(e.ctx, e.reqs)
        gp.gp_synchronize(e.ctx)
    finally:
        e.close()


def test_strided_buffers_are_refused():
    e = Engine([2], L=1, seed=44)
    try:
        e.fill([300])
        q = e.randn(8, 2, 128).bfloat16().transpose(0, 1)  # [2][8][128], not packed
        kv, out = e.randn(2, 2, 128).bfloat16(), torch.zeros(2, 8, 128, device="cuda", dtype=torch.bfloat16)
        k0, w0 = e.k.clone(), e.w.clone()
        for call in (lambda: gp.gp_append_tokens(e.ctx, 0, e.reqs, [300], [2], q, kv, kv, out, e.w),
                     lambda: gp.gp_append_tokens(e.ctx, 0, e.reqs, [300], [2], None, kv, kv.transpose(0, 1), None, e.w),
                     lambda: gp.gp_chunk_attention(e.ctx, 0, e.reqs, [298], [2], q, out, e.w),
                     lambda: gp.gp_chunk_attention(e.ctx, 0, e.reqs, [298], [2], out, q, e.w),
                     lambda: gp.gp_decode_attention_weighted(e.ctx, 0, e.reqs, [300], q[:1], None, out.float()[:1], e.w),
                     lambda: gp.gp_evict_weighted(e.ctx, e.reqs, [300], [100], e.w.transpose(2, 3))):
            with pytest.raises(gp.GrowPageError) as err:
                call()
            assert err.value.status == gp.GP_ERR_INVALID
        gp.gp_synchronize(e.ctx)
        assert torch.equal(bits(e.k), bits(k0)) and torch.equal(bits(e.w), bits(w0)) and not out.any()
    finally:
        e.close()


def test_refused_while_the_stream_is_captured():
    stream = torch.cuda.Stream()
    e = Engine([2], L=1, seed=42, stream=stream)
    try:
        e.fill([300])
        q = e.randn(1, 8, 128).bfloat16()
        k, out, fout = e.randn(1, 2, 128).bfloat16(), torch.empty_like(q), torch.empty(1, 8, 128, device="cuda")
        torch.cuda.synchronize()
        calls = [lambda: gp.gp_append_tokens(e.ctx, 0, e.reqs, [300], [1], q, k, k, out, e.w),
                 lambda: gp.gp_chunk_attention(e.ctx, 0, e.reqs, [299], [1], q, out, e.w),
                 lambda: gp.gp_decode_attention_weighted(e.ctx, 0, e.reqs, [300], q, None, fout, e.w),
                 lambda: gp.gp_evict_weighted(e.ctx, e.reqs, [300], [100], e.w)]
        graph = torch.cuda.CUDAGraph()
        statuses = []
        with torch.cuda.graph(graph, stream=stream):
            fout.zero_()
            for call in calls:
                try:
                    call()
                except gp.GrowPageError as err:
                    statuses.append(err.status)
        assert statuses == [gp.GP_ERR_UNSUPPORTED] * 4
        graph.replay()
        torch.cuda.synchronize()
        for call in calls:  # and the context works on
            call()
        gp.gp_synchronize(e.ctx)
    finally:
        e.close()


def test_eviction_refused_while_the_side_stream_is_captured():
    side = torch.cuda.Stream()
    e = Engine([2], L=1, seed=43)
    try:
        e.fill([300])
        gp.gp_set_compaction_stream(e.ctx, side)
        x, w0 = torch.ones(8, device="cuda"), e.w.clone()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side, capture_error_mode="relaxed"):
            x.mul_(2)
            with pytest.raises(gp.GrowPageError) as err:
                gp.gp_evict_weighted(e.ctx, e.reqs, [300], [100], e.w)
        assert err.value.status == gp.GP_ERR_UNSUPPORTED
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(bits(e.w), bits(w0)) and x[0] == 2
        gp.gp_evict_weighted(e.ctx, e.reqs, [300], [100], e.w)  # and the context works on
        gp.gp_wait_compaction(e.ctx)
        gp.gp_synchronize(e.ctx)
    finally:
        gp.gp_set_compaction_stream(e.ctx, None)
        e.close()


def test_two_engines_on_two_streams():
    """Two contexts issue interleaved calls on streams of their own; each gives
    what it gives alone."""
    cached, new = [200, 700], [150, 33]

    def build(stream):
        e = Engine([3, 4], L=1, seed=51, stream=stream)
        e.fill([350, 733])
        return e, e.randn(183, 8, 128).bfloat16(), torch.empty(183, 8, 128, device="cuda", dtype=torch.bfloat16)

    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    engines = [build(s) for s in streams] + [build(torch.cuda.current_stream())]
    torch.cuda.synchronize()
    try:
        for _ in range(12):  # more calls than staging slots
            for e, q, out in engines[:2]:
                gp.gp_chunk_attention(e.ctx, 0, e.reqs, cached, new, q, out, e.w)
        e, q, out = engines[2]
        for _ in range(12):
            gp.gp_chunk_attention(e.ctx, 0, e.reqs, cached, new, q, out, e.w)
        for e, _, _ in engines:
            gp.gp_evict_weighted(e.ctx, e.reqs, [350, 733], [100, 256], e.w)
        for e, _, _ in engines:
            gp.gp_synchronize(e.ctx)
        for e, _, out in engines[:2]:
            assert torch.equal(bits(out), bits(engines[2][2])) and torch.equal(bits(e.w), bits(engines[2][0].w))
            for r, kp in enumerate([100, 256]):
                for h in range(2):
                    assert torch.equal(e.rows(e.k, r, 0, h, kp), engines[2][0].rows(engines[2][0].k, r, 0, h, kp))
    finally:
        for e, _, _ in engines:
            e.close()
