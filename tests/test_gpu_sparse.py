"""The calls over a step's device arrays, through the C ABI, against plain formulas
in whole numbers and 64 bits: gp_build_tables, gp_append_mapped, gp_block_bounds,
gp_select_blocks and gp_sparse_attention, each at the lengths, lists and types
where it can go wrong, and a run of them together, eager and captured.

Tables, bounds, scales, selected blocks, copied values and everything not written
are exact.  Tolerances of the rest (worst cases of the arithmetic, set before the
first run):
  * a rounding to type t: |x| eps(t) / 2 (bf16 2^-8, fp32 2^-24);
  * rotary forms: the angle is reduced in fp64 and rounded to fp32 (|angle| <= pi:
    pi 2^-24 < 1.9e-7), sincosf adds at most 2 ulp (1.2e-7), the amplitude one
    rounding (2^-24 of up to 1.4), two products and a sum 2^-23 each:
    |error| <= 8e-7 amplitude (|a| + |b|) for the pair (a, b);
  * a logit: d products summed in fp32, in any order, each partial sum off by at
    most 2^-23 (a truncating accumulator) of sum |q_i k_i| <= |q| |k|, scaling and
    subtraction of the maximum 2^-23 of it each: dz = (d + 16) 2^-23 |q| |k| / sqrt(d);
  * a weight e^(z - m) / l: relative error 2 dz + (T + 64) 2^-23, T weights in the sum;
  * an output sum a v: that twice, of sum a |v|; the two bf16 parts of a weight on the
    tensor cores leave 2^-15 of sum a |v| more; then its own rounding.
"""

import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import paged_kv_cache_step_gb300 as gp

pytestmark = pytest.mark.gpu

PAGE = 256
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
GPD = {"bf16": gp.GP_DTYPE_BF16, "f32": gp.GP_DTYPE_F32}
EPS = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
CUDA = dict(device="cuda")


def i32(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32), **CUDA)


def i64(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int64), **CUDA)


class Engine:
    """An engine over caches full of NaN, n requests in shuffled slots and pages, and
    the arrays of a step of `new` tokens behind `cached` ones (built here, or by the
    call when build is False)."""

    def __init__(self, cached, new, L=2, layer=1, hq=8, hkv=2, d=128, kv="bf16", q="bf16", pad=0, seed=0, cap=None, pos=None,
                 spare=0, kernel=None, stream=None, pool=None):
        self.L, self.layer, self.hq, self.hkv, self.d, self.kv, self.qt = L, layer, hq, hkv, d, kv, q
        self.cached, self.new, n = list(cached), list(new), len(cached)
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        rng = np.random.default_rng(seed)
        pages = [-(-(a + b) // PAGE) for a, b in zip(cached, new)]
        self.cap = cap or max(1, max(pages, default=1))
        self.pool = pool or max(1, sum(pages) + spare)
        shape = (L, self.pool, hkv, PAGE, d)
        if pool:
            self.k, self.v = torch.empty(shape, dtype=DT[kv], **CUDA), torch.empty(shape, dtype=DT[kv], **CUDA)
        else:
            self.k, self.v = (torch.full(shape, math.nan, dtype=DT[kv], **CUDA) for _ in range(2))
        self.M = n + 3
        cfg = gp.gp_config_default(num_layers=L, num_q_heads=hq, num_kv_heads=hkv, head_dim=d, kv_dtype=GPD[kv], q_dtype=GPD[q],
                                   max_slots=self.M, num_pages=self.pool, max_pages_per_req=self.cap)
        self.ctx = gp.gp_create(cfg, self.k, self.v, stream or torch.cuda.current_stream())
        if kernel is not None:
            gp.gp_set_scan_kernel(self.ctx, kernel)
        order = rng.permutation(self.pool) if not pool else np.arange(self.pool)[::-1]
        self.slots = rng.permutation(self.M)[:n]
        tables = np.full((self.M, self.cap), -7, dtype=np.int32)
        rows, at, self.row0 = sum(new), 0, np.concatenate([[0], np.cumsum(new)]).astype(int)
        pos = cached if pos is None else pos
        row_req, slot_map, positions = np.full(rows + pad, -1), np.full(rows + pad, -1), np.zeros(rows + pad, dtype=np.int64)
        for r, s in enumerate(self.slots):
            tables[s, :pages[r]] = order[at:at + pages[r]]
            at += pages[r]
            t, x = cached[r] + np.arange(new[r]), slice(self.row0[r], self.row0[r + 1])
            row_req[x], positions[x] = r, pos[r] + np.arange(new[r])
            slot_map[x] = tables[s, t // PAGE] * PAGE + t % PAGE
        self.tables_host, self.positions_host, self.rows, self.max_rows = tables, positions, rows, rows + pad
        self.arrays = dict(slots=i32(self.slots), num_cached=i32(cached), num_new=i32(new), pos=i64(pos), tables=i32(tables),
                           row0=i32(self.row0), row_req=i32(row_req), slot_map=i64(slot_map), positions=i64(positions))
        self.step = gp.Step(self.ctx, **self.arrays)

    def close(self):
        torch.cuda.synchronize()
        gp.gp_destroy(self.ctx)

    def randn(self, *shape):
        return torch.randn(*shape, device="cuda", generator=self.gen)

    def at(self, r, T, T0=0):
        """Pages and places of the logical slots [T0, T) of request r."""
        t = np.arange(T0, T)
        return i64(self.tables_host[self.slots[r], t // PAGE]), i64(t % PAGE)

    def fill(self):
        """Random rows in every slot up to the requests' last tokens."""
        for r in range(len(self.new)):
            pages, places = self.at(r, self.cached[r] + self.new[r])
            for cache in (self.k, self.v):
                cache[self.layer, pages, :, places] = self.randn(len(pages), self.hkv, self.d).to(cache.dtype)

    def rows_of(self, cache, r, T):
        pages, places = self.at(r, T)
        return cache[self.layer, pages, :, places].double()  # [T, hkv, d]


def bits(t):
    return t.contiguous().view(torch.int16 if t.element_size() == 2 else torch.int32)


# ---- gp_build_tables -------------------------------------------------------------


def tables_reference(slots, cached, new, pos, tables, held, free, taken, max_rows, cap):
    """The call's definition, request by request."""
    n, out = len(slots), dict(tables=tables.copy(), num_pages=held.copy(), row0=[0], state=[])
    row_req, slot_map, positions = [], [], []
    wanted_rows = wanted_pages = 0
    room = len(free) - taken if 0 <= taken <= len(free) else 0
    for r, s in enumerate(slots):
        c, m = int(cached[r]), int(new[r])
        valid = 0 <= s < len(held) and list(slots).count(s) == 1 and c >= 0 and m >= 0 and c + m <= cap * PAGE
        valid = valid and -(-c // PAGE) <= held[s] <= cap
        state = gp.GP_STEP_GIVEN if valid else gp.GP_STEP_INVALID
        take = 0
        if valid:
            wanted_rows += m
            if m and wanted_rows > max_rows:
                state = gp.GP_STEP_NO_ROWS
            else:
                take = max(0, -(-(c + m) // PAGE) - int(held[s]))
                wanted_pages += take
                if take and wanted_pages > room:
                    state = gp.GP_STEP_NO_PAGES
        if state == gp.GP_STEP_GIVEN:
            for j in range(take):
                out["tables"][s, held[s] + j] = free[taken]
                taken += 1
            out["num_pages"][s] += take
            for t in range(m):
                page = out["tables"][s, (c + t) // PAGE]
                row_req.append(r)
                slot_map.append(int(page) * PAGE + (c + t) % PAGE)
                positions.append(int(pos[r]) + t)
        out["state"].append(state)
        out["row0"].append(len(row_req))
    pad = max_rows - len(row_req)
    out.update(row_req=row_req + [-1] * pad, slot_map=slot_map + [-1] * pad, positions=positions + [0] * pad, taken=[taken])
    return {k: np.asarray(v) for k, v in out.items()}


class Tables:
    """Inputs of gp_build_tables, held and free pages drawn, and both answers."""

    def __init__(self, cached, new, max_rows, free, taken=0, M=None, cap=8, slots=None, held=None, pos=None, seed=0, alias=False,
                 num_pages=4000):
        rng = np.random.default_rng(seed)
        n, M = len(cached), M or len(cached) + 3
        slots = rng.permutation(M)[:n] if slots is None else np.asarray(slots)
        order = rng.permutation(num_pages)
        if held is None:
            held = np.zeros(M, dtype=np.int64)
            for r, s in enumerate(slots):
                held[s] = -(-cached[r] // PAGE) + (r % 3 == 0 and cached[r] + new[r] + PAGE <= cap * PAGE)
        tables, at = np.full((M, cap), -7), 0
        for s in range(M):
            k = min(max(int(held[s]), 0), cap)
            tables[s, :k] = order[at:at + k]
            at += k
        free_pages = order[at:at + free]
        pos = cached if pos is None else pos
        cfg = gp.gp_config_default(num_layers=1, num_q_heads=2, num_kv_heads=1, head_dim=64, max_slots=M, num_pages=num_pages,
                                   max_pages_per_req=cap)
        k = torch.zeros(16, dtype=torch.bfloat16, **CUDA)  # (the call touches no cache)
        self.ctx = gp.gp_create(cfg, k, k, torch.cuda.current_stream())
        self.want = tables_reference(slots, cached, new, pos, tables, np.asarray(held), free_pages, taken, max_rows, cap)
        full = lambda size, t: torch.full((size,), -9, dtype=t, **CUDA)
        self.a = dict(slots=i32(slots), num_cached=i32(cached), num_new=i32(new), pos=i64(pos), tables=i32(tables),
                      row0=full(n + 1, torch.int32), row_req=full(max_rows, torch.int32), slot_map=full(max_rows, torch.int64),
                      positions=full(max_rows, torch.int64))
        self.held, self.free, self.taken = i32(held), i32(free_pages), i32([taken])
        self.num_pages = self.held if alias else self.held.clone()
        self.state = full(n, torch.int32)
        step = gp.Step(self.ctx, **self.a)
        gp.gp_build_tables(self.ctx, step, self.held, self.num_pages, self.free, self.taken, self.taken, self.state)

    def check(self):
        try:
            gp.gp_synchronize(self.ctx)
            got = dict(self.a, num_pages=self.num_pages, state=self.state, taken=self.taken)
            for name, want in self.want.items():
                assert np.array_equal(got[name].cpu().numpy().astype(np.int64), want.astype(np.int64)), name
        finally:
            gp.gp_destroy(self.ctx)


@pytest.mark.parametrize("alias", [False, True])
@pytest.mark.parametrize("n", [1, 5, 64, 257, 1030])
def test_tables(n, alias):
    rng = np.random.default_rng(n)
    cached, new = rng.integers(0, 900, n), rng.integers(0, 3 if n > 100 else 500, n)
    Tables(cached, new, int(new.sum()) + n % 7, 3 * n + 5, taken=3 if n > 1 else 0, seed=n, alias=alias, num_pages=20000).check()


def test_tables_of_prompts():
    """Rows enough for the larger launch, page ends and starts among them."""
    Tables([0, 0, 255, 256, 257, 0], [2048, 1, 1, 1, 600, 0], 2651 + 40, 60, seed=1).check()
    Tables([0] * 40, [1000] * 40, 40_000, 160, seed=2).check()


@pytest.mark.parametrize("free", [0, 1, 4, 5, 6])
def test_tables_when_pages_run_out(free):
    """Requests take in order; those after one that is refused still get rows that need no page."""
    Tables([0, 100, 256, 0, 300, 512], [300, 3, 1, 700, 5, 1], 1200, free, seed=3).check()
    Tables([0, 100, 256, 0, 300, 512], [300, 3, 1, 700, 5, 1], 1200, free + 2, taken=2, seed=3).check()


@pytest.mark.parametrize("rows", [0, 3, 4, 303, 304, 1003, 1004, 1010])
def test_tables_when_rows_run_out(rows):
    Tables([100, 0, 256, 0, 7], [3, 300, 1, 700, 0], rows, 50, seed=4).check()


def test_tables_of_invalid_requests():
    """Negative or too many tokens, slots out of range or twice, cached tokens without a
    page, more pages than a table: no rows, no pages, the others unharmed."""
    big = 2 ** 31 - 1
    Tables([0, -1, 5, 5, 2000, big, 0, 3, 300, 1], [4, 3, -2, 3, 49, 1, big, 2, 1, 1], 40, 50,
           slots=[0, 1, 2, 99, 4, 5, 6, 7, 8, -3], M=12, held=[0, 1, 1, 0, 7, 8, 0, 99, 1, 0, 0, 0], seed=5).check()
    Tables([5, 5, 5, 5], [1, 1, 1, 1], 9, 5, slots=[2, 1, 2, 0], M=4, held=[1, 1, 1, 1], seed=6).check()
    Tables([0, 10], [3, 3], 9, 5, taken=-1, seed=7).check()
    Tables([0, 10], [3, 3], 9, 5, taken=6, seed=7).check()


def test_tables_of_nothing():
    Tables([], [], 5, 3, M=4, held=[0] * 4).check()
    Tables([5], [0], 0, 0, seed=8).check()
    Tables([5, 0], [0, 0], 3, 2, seed=9).check()


def test_tables_with_far_positions():
    Tables([100, 3], [5, 300], 310, 5, pos=[2 ** 40, 123_456_789_012], seed=10).check()


def test_a_repeated_call_takes_nothing():
    t = Tables([0, 200], [300, 100], 400, 9, seed=11, alias=True)
    step = gp.Step(t.ctx, **t.a)
    gp.gp_build_tables(t.ctx, step, t.held, t.num_pages, t.free, t.taken, t.taken, t.state)
    t.check()


def test_a_page_outside_the_pool_is_reported():
    """In the free list or an old table: the row is left out, the next call that synchronises tells."""
    for where in ("free", "table"):
        t = Tables([0, 300], [3, 4], 10, 5, slots=[1, 0], M=4, held=[2, 0, 0, 0], seed=12)
        gp.gp_synchronize(t.ctx)
        if where == "free":
            t.free[0] = 4000
        else:
            t.a["tables"][t.a["slots"][1].long(), 1] = -3
        gp.gp_build_tables(t.ctx, gp.Step(t.ctx, **t.a), t.held, t.num_pages, t.free, None, t.taken, t.state)
        with pytest.raises(gp.GrowPageError) as e:
            gp.gp_synchronize(t.ctx)
        assert e.value.status == gp.GP_ERR_INVALID
        rows = slice(0, 3) if where == "free" else slice(3, 7)
        assert (t.a["slot_map"][rows] == -1).all() and (t.a["slot_map"][:7] != -1).sum() == (4 if where == "free" else 3)
        gp.gp_synchronize(t.ctx)
        gp.gp_destroy(t.ctx)


# ---- gp_append_mapped --------------------------------------------------------------


def frequencies(rd, layout, scaling, theta, factor, original, low, high):
    """Pair by pair, from the header's words."""
    out = []
    for i in range(rd // 2):
        f = theta ** (-2 * i / rd)
        part = 0.0
        if scaling == gp.GP_ROPE_LINEAR:
            part = 1.0
        elif scaling == gp.GP_ROPE_BANDS:
            turns = original * f / (2 * math.pi)
            part = 1.0 if turns <= low else 0.0 if turns >= high else 1.0 - (turns - low) / (high - low)
        elif scaling == gp.GP_ROPE_RAMP:
            pair = lambda t: rd * math.log(original / (2 * math.pi * t)) / (2 * math.log(theta))
            a, b = max(0, math.floor(pair(high))), min(rd - 1, math.ceil(pair(low)))
            part = min(1.0, max(0.0, (i - a) / max(b - a, 0.001)))
        out.append((1 - part) * f + part * f / factor if part else f)
    return np.array(out)


def rotated(x, pos, inv, interleaved, amplitude):
    """x [rows, heads, d] in 64 bits, and the tolerance of its rotated part."""
    x, rd = x.double(), 2 * len(inv)
    ang = torch.as_tensor(np.asarray(pos, dtype=np.float64)[:, None] * inv, **CUDA)[:, None]
    cos, sin = amplitude * ang.cos(), amplitude * ang.sin()
    first = torch.arange(0, rd, 2, **CUDA) if interleaved else torch.arange(rd // 2, **CUDA)
    second = first + (1 if interleaved else rd // 2)
    out, tol = x.clone(), torch.zeros_like(x)
    a, b = x[..., first], x[..., second]
    out[..., first], out[..., second] = a * cos - b * sin, b * cos + a * sin
    tol[..., first] = tol[..., second] = 8e-7 * amplitude * (a.abs() + b.abs())
    return out, tol


FORMS = [dict(), dict(layout=gp.GP_ROPE_INTERLEAVED), dict(rotary_dim=16), dict(layout=gp.GP_ROPE_INTERLEAVED, rotary_dim=48),
         dict(rotary_dim=0), dict(scaling=gp.GP_ROPE_LINEAR, factor=4.0, layout=gp.GP_ROPE_INTERLEAVED),
         dict(scaling=gp.GP_ROPE_BANDS, factor=8.0, theta=5e5),
         dict(scaling=gp.GP_ROPE_BANDS, factor=2.0, low_turns=2.0, high_turns=9.0, original_length=4096, rotary_dim=32),
         dict(scaling=gp.GP_ROPE_RAMP, factor=32.0, theta=1e6), dict(scaling=gp.GP_ROPE_RAMP, factor=4.0, amplitude=1.0, rotary_dim=32),
         dict(scaling=gp.GP_ROPE_RAMP, factor=4.0, original_length=1, layout=gp.GP_ROPE_INTERLEAVED), dict(amplitude=0.5, theta=100.0),
         dict(factor=0.0, original_length=0, low_turns=math.nan)]


def check_append(e, form, packed="columns"):
    rope = gp.gp_rope_default(**dict(dict(rotary_dim=e.d), **form))
    high = rope.high_turns or (32.0 if rope.scaling == gp.GP_ROPE_RAMP else 4.0)
    inv = frequencies(rope.rotary_dim, rope.layout, rope.scaling, rope.theta, rope.factor, rope.original_length, rope.low_turns, high)
    amplitude = rope.amplitude or (0.1 * math.log(rope.factor) + 1.0 if rope.scaling == gp.GP_ROPE_RAMP else 1.0)
    rows, n = e.max_rows, e.rows
    if packed == "columns" and e.kv == e.qt:  # of one projection
        both = e.randn(rows, (e.hq + 2 * e.hkv) * e.d + 16).to(DT[e.kv])
        q, k, v = (both[:, a * e.d:b * e.d].unflatten(1, (b - a, e.d)) for a, b in
                   ((0, e.hq), (e.hq, e.hq + e.hkv), (e.hq + e.hkv, e.hq + 2 * e.hkv)))
    else:
        q, k, v = e.randn(rows, e.hq, e.d).to(DT[e.qt]), e.randn(rows, e.hkv, e.d).to(DT[e.kv]), e.randn(rows, e.hkv, e.d).to(DT[e.kv])
    v[:1, 0, :2] = torch.tensor([math.inf, math.nan])  # values are copied, whatever they are
    want_k, want_v = e.k.clone(), e.v.clone()
    src = q.contiguous().clone() if packed == "in place" else q
    rot = src if packed == "in place" else torch.full((rows, e.hq, e.d), 7.0, dtype=DT[e.qt], **CUDA)
    qr, qtol = rotated(q[:n], e.positions_host[:n], inv, rope.layout == gp.GP_ROPE_INTERLEAVED, amplitude)
    kr, ktol = rotated(k[:n], e.positions_host[:n], inv, rope.layout == gp.GP_ROPE_INTERLEAVED, amplitude)
    behind = rot[n:].clone()
    gp.gp_append_mapped(e.ctx, e.layer, e.step, rope, src, k, v, rot)
    gp.gp_synchronize(e.ctx)
    rd = rope.rotary_dim
    assert torch.all((rot[:n].double() - qr).abs() <= qtol + EPS[e.qt] * qr.abs())
    assert torch.equal(bits(rot[:n, :, rd:]), bits(q[:n, :, rd:])) and torch.equal(bits(rot[n:]), bits(behind))
    at = e.arrays["slot_map"][:n]
    got = e.k[e.layer, at // PAGE, :, at % PAGE]
    assert torch.all((got.double() - kr).abs() <= ktol + EPS[e.kv] * kr.abs())
    assert torch.equal(bits(got[..., rd:]), bits(k[:n, :, rd:]))
    want_k[e.layer, at // PAGE, :, at % PAGE] = got
    want_v[e.layer, at // PAGE, :, at % PAGE] = v[:n]
    assert torch.equal(bits(e.k), bits(want_k)) and torch.equal(bits(e.v), bits(want_v))  # and nothing else


@pytest.mark.parametrize("form", FORMS)
def test_append_mapped_forms(form):
    for d in (64, 128):
        e = Engine([0, 255, 7, 300], [1, 2, 0, 270], d=d, pad=3, pos=[0, 65_535, 1, 1_000_003], seed=d)
        try:
            check_append(e, form)
        finally:
            e.close()


@pytest.mark.parametrize("kv,q,d,hq,hkv", [("f32", "f32", 64, 4, 1), ("f32", "f32", 128, 8, 2), ("bf16", "f32", 128, 6, 3),
                                            ("f32", "bf16", 128, 4, 2), ("bf16", "bf16", 128, 32, 8)])
@pytest.mark.parametrize("packed", ["columns", "packed", "in place"])
def test_append_mapped_types(kv, q, d, hq, hkv, packed):
    for form in (dict(), dict(layout=gp.GP_ROPE_INTERLEAVED, rotary_dim=32)):
        e = Engine([3, 500], [17, 30], d=d, kv=kv, q=q, hq=hq, hkv=hkv, pos=[2 ** 31 + 11, 9], seed=hq)
        try:
            check_append(e, form, packed)
        finally:
            e.close()


def test_append_mapped_is_append_tokens():
    """The half layout without scaling gives the bits of gp_append_tokens."""
    e = Engine([0, 255, 300], [5, 2, 270], L=1, layer=0, pos=[10, 70_000, 3], seed=1)
    try:
        k, v, q = e.randn(277, 2, 128).bfloat16(), e.randn(277, 2, 128).bfloat16(), e.randn(277, 8, 128).bfloat16()
        rots = [torch.empty_like(q), torch.empty_like(q)]
        gp.gp_append_mapped(e.ctx, 0, e.step, gp.gp_rope_default(rotary_dim=128), q, k, v, rots[0])
        gp.gp_synchronize(e.ctx)
        first = e.k.clone(), e.v.clone()
        for _ in range(e.pool):
            gp.gp_page_alloc(e.ctx)
        reqs = [None] * e.M
        for s in range(e.M):
            slot, r = gp.gp_slot_acquire(e.ctx), list(e.slots).index(s) if s in e.slots else -1
            if r >= 0:
                pages = -(-(e.cached[r] + e.new[r]) // PAGE)
                reqs[r] = gp.Request(slot, e.tables_host[slot, :pages], [10, 70_000, 3][r], e.cap)
        gp.gp_append_tokens(e.ctx, 0, reqs[:3], e.cached, e.new, q, k, v, rots[1])
        gp.gp_synchronize(e.ctx)
        assert torch.equal(bits(rots[0]), bits(rots[1]))
        assert torch.equal(bits(e.k), bits(first[0])) and torch.equal(bits(e.v), bits(first[1]))
    finally:
        e.close()


def test_append_mapped_without_queries():
    e = Engine([0], [300], L=1, layer=0)
    try:
        k, v = e.randn(300, 2, 128).bfloat16(), e.randn(300, 2, 128).bfloat16()
        gp.gp_append_mapped(e.ctx, 0, e.step, gp.gp_rope_default(), None, k, v, None)
        gp.gp_synchronize(e.ctx)
        assert torch.equal(e.rows_of(e.k, 0, 300), k.double()) and torch.equal(e.rows_of(e.v, 0, 300), v.double())
    finally:
        e.close()


# ---- gp_block_bounds ----------------------------------------------------------------


def bounds_reference(k):
    """[tokens, hkv, d] -> whole numbers [hkv, 2, d] and scales [hkv]."""
    k = k.double().cpu().numpy()
    with np.errstate(invalid="ignore"):
        lo, hi = np.fmin.reduce(k, 0), np.fmax.reduce(k, 0)  # NaN left out
    lo, hi = np.where(np.isnan(lo), 0.0, lo), np.where(np.isnan(hi), 0.0, hi)
    scales = np.empty(k.shape[1])
    for h in range(k.shape[1]):
        top = max(np.abs(lo[h]).max(), np.abs(hi[h]).max())
        e = -100
        while e < 100 and 127.0 * 2.0 ** e < top:
            e += 1
        scales[h] = 2.0 ** e
    held = np.stack([np.floor(lo / scales[:, None]), np.ceil(hi / scales[:, None])], 1)
    return np.clip(held, -127, 127), scales


def bounds_arrays(e, block, fill=99):
    shape = (e.L, e.pool, e.hkv, PAGE // block)
    return torch.full((*shape, 2, e.d), fill, dtype=torch.int8, **CUDA), torch.full(shape, -3.0, **CUDA)


def check_bounds(e, block, bounds, scales):
    want_b, want_s = torch.full_like(bounds, 99), torch.full_like(scales, -3.0)
    per = PAGE // block
    for r in range(len(e.new)):
        T = e.cached[r] + e.new[r]
        rows = e.rows_of(e.k, r, T)
        for b in range(e.cached[r] // block, (T - 1) // block + 1 if e.new[r] else 0):
            held, scale = bounds_reference(rows[b * block:min(T, b * block + block)])
            page = int(e.tables_host[e.slots[r], b // per])
            want_b[e.layer, page, :, b % per] = torch.as_tensor(held.astype(np.int8), **CUDA)
            want_s[e.layer, page, :, b % per] = torch.as_tensor(scale, **CUDA).float()
    assert torch.equal(scales, want_s)
    assert torch.equal(bounds, want_b)


@pytest.mark.parametrize("kv,d,hkv", [("bf16", 128, 2), ("bf16", 64, 8), ("f32", 128, 3), ("f32", 64, 1)])
@pytest.mark.parametrize("block", [16, 32, 64, 128, 256])
def test_block_bounds(block, kv, d, hkv):
    e = Engine([0, 255, 256, 7, 100, 511, 31], [1, 2, 256, 0, 700, 1, 2], d=d, hkv=hkv, hq=2 * hkv, kv=kv, pad=2, seed=block + d)
    try:
        e.fill()
        bounds, scales = bounds_arrays(e, block)
        gp.gp_block_bounds(e.ctx, e.layer, e.step, block, bounds, scales)
        gp.gp_synchronize(e.ctx)
        check_bounds(e, block, bounds, scales)
    finally:
        e.close()


def test_block_bounds_of_extreme_keys():
    """Zeros, subnormals, infinities, NaN, exact multiples and the ends of a scale."""
    e = Engine([0], [16 * 9], d=64, hkv=2, hq=4, kv="f32", L=1, layer=0, seed=3)
    try:
        e.fill()
        rows = torch.zeros(16 * 9, 2, 64, **CUDA)
        rows[16:32] = e.randn(16, 2, 64) * 1e-42                        # subnormal
        rows[32:48, :, 3] = math.inf
        rows[33, :, 4] = -math.inf
        rows[48:64] = e.randn(16, 2, 64)
        rows[50] = math.nan
        rows[48:64, 1, 7] = math.nan                                    # nothing left in a dimension
        rows[64:80] = 127.0 * 2.0 ** 5
        rows[80:96] = torch.nextafter(torch.tensor(127.0 * 2.0 ** 5), torch.tensor(1e9))
        rows[96:112] = -torch.arange(16, **CUDA)[:, None, None].float() / 4
        rows[112:128] = 3.0e38
        rows[128:144] = e.randn(16, 2, 64) * 2.0 ** -99
        pages, places = e.at(0, 144)
        e.k[0, pages, :, places] = rows
        bounds, scales = bounds_arrays(e, 16)
        gp.gp_block_bounds(e.ctx, 0, e.step, 16, bounds, scales)
        gp.gp_synchronize(e.ctx)
        check_bounds(e, 16, bounds, scales)
    finally:
        e.close()


# ---- gp_select_blocks -----------------------------------------------------------------


def select_reference(e, q, bounds, scales, block, top, sink, recent):
    """[rows, hkv, top] in whole numbers (scores as 64 bit floats, which hold them)."""
    per, G = PAGE // block, e.hq // e.hkv
    out = np.full((e.rows, e.hkv, top), -1)
    for r in range(len(e.new)):
        for t in range(e.new[r]):
            row, own = e.row0[r] + t, (e.cached[r] + t) // block
            b = np.arange(own + 1)
            table = e.tables_host[e.slots[r]]
            for h in range(e.hkv):
                x = q[row, h * G:h * G + G].double().cpu().numpy()
                x = np.where(np.isnan(x), 0.0, x)
                u, most = -100, np.abs(x).max()
                while u < 100 and 127.0 * 2.0 ** u < most:
                    u += 1
                x = np.clip(np.rint(x / 2.0 ** u), -127, 127)
                held = bounds[e.layer, table[b // per], h, b % per].astype(np.float64)  # [own + 1, 2, d]
                score = np.maximum(x[:, None] * held[None, :, 0], x[:, None] * held[None, :, 1]).sum((0, 2))
                score *= scales[e.layer, table[b // per], h, b % per]
                kept = b if own + 1 <= top else None
                if kept is None:
                    rest = b[sink:own + 1 - recent]
                    best = rest[np.argsort(-score[rest], kind="stable")[:top - sink - recent]]
                    kept = np.sort(np.concatenate([b[:sink], best, b[own + 1 - recent:]]))
                out[row, h, :len(kept)] = kept
    return out


def check_select(e, block, top, sink, recent, extreme=False, seed=0):
    rng = np.random.default_rng(seed)
    shape = (e.L, e.pool, e.hkv, PAGE // block)
    if extreme:  # the largest sums, and ties of all kinds
        bounds = np.sort(rng.choice([-127, 127], (*shape, 2, e.d)), -2)
        scales = 2.0 ** rng.integers(-1, 1, shape)
        bounds[rng.random(shape) < 0.3] = 0
        q = torch.as_tensor(rng.choice([-127.0, 127.0, 126.0], (e.max_rows, e.hq, e.d), p=[0.5, 0.45, 0.05]), **CUDA).to(DT[e.qt])
    else:
        bounds = np.sort(rng.integers(-127, 128, (*shape, 2, e.d)), -2)
        scales = 2.0 ** rng.integers(-6, 3, shape)
        q = (e.randn(e.max_rows, e.hq, e.d) * torch.exp(e.randn(e.max_rows, e.hq, 1))).to(DT[e.qt])
        if e.max_rows > 1:
            q[0, 0, 3], q[1] = math.nan, 0.0
    blocks = torch.full((e.max_rows, e.hkv, top), -5, dtype=torch.int32, **CUDA)
    gp.gp_select_blocks(e.ctx, e.layer, e.step, block, top, sink, recent, q, torch.as_tensor(bounds.astype(np.int8), **CUDA),
                        torch.as_tensor(scales.astype(np.float32), **CUDA), blocks)
    gp.gp_synchronize(e.ctx)
    want = select_reference(e, q, bounds, scales, block, top, sink, recent)
    assert np.array_equal(blocks[:e.rows].cpu().numpy(), want)
    assert (blocks[e.rows:] == -5).all()


@pytest.mark.parametrize("hq,hkv,d,q", [(8, 2, 128, "bf16"), (4, 2, 64, "bf16"), (4, 2, 64, "f32"), (4, 1, 128, "f32"),
                                        (32, 8, 128, "bf16")])
@pytest.mark.parametrize("block,top,sink,recent", [(64, 9, 1, 2), (16, 40, 0, 1), (32, 8, 4, 4), (128, 3, 0, 3), (256, 2, 1, 1),
                                                   (16, 1, 0, 1), (64, 100, 2, 2)])
def test_select_blocks(block, top, sink, recent, hq, hkv, d, q):
    e = Engine([0, 255, 256, 7, 1000, 2511, 31], [1, 2, 30, 0, 9, 1, 2], hq=hq, hkv=hkv, d=d, q=q, pad=2, seed=top + d)
    try:
        check_select(e, block, top, sink, recent, seed=top)
        check_select(e, block, top, sink, recent, extreme=True, seed=top)
    finally:
        e.close()


def test_select_blocks_of_the_longest_request():
    """256 pages in blocks of 16: 4096 to choose from, and one that is nearly empty."""
    e = Engine([65_531, 0], [5, 2], L=1, layer=0, hq=4, hkv=1, d=64, seed=2)
    try:
        for top in (3, 130, 4000, 5000):
            check_select(e, 16, top, 1, 2, seed=top)
        check_select(e, 16, 130, 1, 2, extreme=True)
    finally:
        e.close()


# ---- gp_sparse_attention ------------------------------------------------------------------


def attention_reference(e, q, lists):
    """Outputs [rows, hq, d] in 64 bits and their bounds; lists[row][h]: blocks, with e.block."""
    G = e.hq // e.hkv
    out = torch.zeros(e.rows, e.hq, e.d, dtype=torch.float64, **CUDA)
    tol = torch.zeros_like(out)
    for r in range(len(e.new)):
        T = e.cached[r] + e.new[r]
        keys, vals = e.rows_of(e.k, r, T), e.rows_of(e.v, r, T)
        for t in range(e.new[r]):
            row = e.row0[r] + t
            for h in range(e.hkv):
                chosen = np.asarray(lists[row][h], dtype=int)
                tok = (chosen[:, None] * e.block + np.arange(e.block)).ravel()
                tok = i64(tok[tok <= e.cached[r] + t])
                if len(tok) == 0:
                    continue
                x = q[row, h * G:h * G + G].double()
                k, v = keys[tok, h], vals[tok, h]
                a = torch.softmax(x @ k.T / math.sqrt(e.d), -1)
                dz = (e.d + 16) * 2.0 ** -23 * x.norm(dim=-1) * k.norm(dim=-1).max() / math.sqrt(e.d)
                rel = 2 * dz + (len(tok) + 64) * 2.0 ** -23
                out[row, h * G:h * G + G] = a @ v
                tol[row, h * G:h * G + G] = (2 * rel[:, None] + (2.0 ** -15 if e.kv == e.qt == "bf16" else 0.0)) * (a @ v.abs())
    return out, tol + EPS[e.qt] * out.abs()


def random_lists(e, top, seed=0):
    """Ascending lists of up to `top` blocks, the row's own usually among them; some empty."""
    rng = np.random.default_rng(seed)
    lists = []
    for r in range(len(e.new)):
        for t in range(e.new[r]):
            own = (e.cached[r] + t) // e.block
            row = []
            for _ in range(e.hkv):
                k = 0 if rng.random() < 0.05 else rng.integers(1, min(top, own + 1) + 1)
                x = np.sort(rng.permutation(own + 1)[:k])
                if k and rng.random() < 0.8:
                    x[-1] = own
                row.append(x)
            lists.append(row)
    return lists


def check_attention(e, block, top, lists=None, seed=0, scale=1.0):
    e.block = block
    lists = random_lists(e, top, seed) if lists is None else lists
    blocks = np.full((e.max_rows, e.hkv, top), -1)
    for row, x in enumerate(lists):
        for h in range(e.hkv):
            blocks[row, h, :len(x[h])] = x[h]
    q = (scale * e.randn(e.max_rows, e.hq, e.d)).to(DT[e.qt])
    out = torch.full((e.max_rows, e.hq, e.d), 7.0, dtype=DT[e.qt], **CUDA)
    gp.gp_sparse_attention(e.ctx, e.layer, e.step, block, top, q, i32(blocks), out)
    gp.gp_synchronize(e.ctx)
    want, tol = attention_reference(e, q, lists)
    worst = ((out[:e.rows].double() - want).abs() - tol).max().item() if e.rows else 0.0
    assert worst <= 0.0, worst
    assert (out[e.rows:] == 7.0).all()
    return q, i32(blocks), out


SHAPES = {"bf16_g4_d128": dict(hq=8, hkv=2), "bf16_g2_d64": dict(hq=6, hkv=3, d=64), "bf16_g4_d64": dict(hq=4, hkv=1, d=64),
          "bf16_g2_d128": dict(hq=4, hkv=2), "f32_g4_d128": dict(hq=8, hkv=2, kv="f32", q="f32"), "f32_g2_d64": dict(hq=4, hkv=2, d=64, kv="f32", q="f32"),
          "bf16_q32": dict(hq=4, hkv=2, q="f32"), "f32_q16": dict(hq=4, hkv=1, d=64, kv="f32")}


def kernels(shape):
    s = SHAPES[shape]
    both = s.get("kv", "bf16") == s.get("q", "bf16") == "bf16"
    return [gp.GP_SCAN_TENSOR_CORE, gp.GP_SCAN_CUDA_CORE] if both else [gp.GP_SCAN_AUTO]


@pytest.mark.parametrize("block,top", [(16, 40), (32, 5), (64, 9), (128, 4), (256, 3), (16, 1)])
@pytest.mark.parametrize("shape", SHAPES)
def test_sparse_attention(shape, block, top):
    for kernel in kernels(shape):
        e = Engine([0, 255, 256, 7, 1000, 2511, 31], [1, 2, 30, 0, 9, 1, 2], pad=2, seed=top + block, kernel=kernel, **SHAPES[shape])
        try:
            e.fill()
            check_attention(e, block, top, seed=block)
        finally:
            e.close()


@pytest.mark.parametrize("shape", ["bf16_g4_d128", "bf16_g4_d64", "f32_g2_d64", "bf16_g2_d64"])
@pytest.mark.parametrize("new", [1, 3, 70, 400])
def test_sparse_attention_of_chunks(shape, new):
    """One request and two, from one token to several tiles; dense lists among them."""
    for kernel in kernels(shape):
        for cached in ([0], [517, 40]):
            e = Engine(cached, [new] * len(cached), seed=new, kernel=kernel, **SHAPES[shape])
            try:
                e.fill()
                check_attention(e, 64, 6, seed=new)
                own = [(c + t) // 16 for c in cached for t in range(new)]
                check_attention(e, 16, 64, lists=[[np.arange(o + 1)] * e.hkv for o in own])
            finally:
                e.close()


@pytest.mark.parametrize("block,top", [(16, 70), (32, 33), (64, 8), (128, 5), (256, 2)])
@pytest.mark.parametrize("shape", ["bf16_g4_d128", "bf16_g2_d128", "bf16_g4_d64", "bf16_g2_d64"])
def test_sparse_attention_of_few_rows(shape, block, top):
    """One row a request, and as many as a small piece takes: the kernel of decode steps."""
    for new in ([1] * 9, [4, 1, 3, 2, 4, 0, 1, 4, 4] if "g4" in shape else [8, 1, 7, 2, 8, 0, 5, 8, 8]):
        e = Engine([0, 255, 256, 7, 1000, 2511, 31, 1023, 4090], new, pad=0, seed=block + len(shape), **SHAPES[shape])
        try:
            e.fill()
            check_attention(e, block, top, seed=block)
        finally:
            e.close()


@pytest.mark.parametrize("block,top", [(16, 70), (32, 33), (64, 8), (128, 5), (256, 2)])
@pytest.mark.parametrize("shape", ["bf16_g4_d128", "bf16_g2_d128", "bf16_g4_d64", "bf16_g2_d64"])
def test_sparse_attention_of_many_rows(shape, block, top):
    """Whole pieces of 128 / G rows, one row more and one less, beside requests of a row or
    none, with rows behind the last one."""
    n = 32 if "g4" in shape else 64
    e = Engine([0, 700, 255, 3000, 7, 100], [n, n + 1, 1, n - 1, 0, 2 * n], pad=5, seed=block + len(shape), **SHAPES[shape])
    try:
        e.fill()
        check_attention(e, block, top, seed=block)
    finally:
        e.close()


@pytest.mark.parametrize("new", [1, 4, 60])
def test_rows_without_blocks(new):
    """Empty lists only, in every kernel: zeros, whatever the caches hold."""
    for kernel in (gp.GP_SCAN_TENSOR_CORE, gp.GP_SCAN_CUDA_CORE):
        e = Engine([300, 0], [new, new], seed=new, kernel=kernel)
        try:
            q = e.randn(2 * new, 8, 128).bfloat16()
            out = torch.full_like(q, math.nan)
            gp.gp_sparse_attention(e.ctx, e.layer, e.step, 64, 3, q, torch.full((2 * new, 2, 3), -1, dtype=torch.int32, **CUDA), out)
            gp.gp_synchronize(e.ctx)
            assert not out.any()
        finally:
            e.close()


@pytest.mark.parametrize("new", [4, 70])
def test_queries_of_other_rows_do_not_matter(new):
    """NaN in the queries of one request, and behind the last row, stays there."""
    e = Engine([500, 300], [new, new], pad=40, seed=3)
    e.block = 32
    try:
        e.fill()
        lists = random_lists(e, 5, 1)
        blocks = np.full((e.max_rows, 2, 5), -1)
        for row, x in enumerate(lists):
            for h in range(2):
                blocks[row, h, :len(x[h])] = x[h]
        q = e.randn(e.max_rows, 8, 128).bfloat16()
        want, tol = attention_reference(e, q, lists)
        q[new:] = math.nan
        out = torch.zeros_like(q)
        gp.gp_sparse_attention(e.ctx, e.layer, e.step, 32, 5, q, i32(blocks), out)
        gp.gp_synchronize(e.ctx)
        assert torch.all((out[:new].double() - want[:new]).abs() <= tol[:new])
        assert not out[2 * new:].any()
    finally:
        e.close()


@pytest.mark.parametrize("seed", range(12))
def test_sparse_attention_at_random(seed):
    rng = np.random.default_rng(seed)
    for _ in range(3):
        n = int(rng.integers(1, 9))
        shape = list(SHAPES)[rng.integers(len(SHAPES))]
        cached = (rng.random(n) ** 3 * 5000).astype(int)
        new = (rng.random(n) ** 3 * rng.choice([3, 12, 150])).astype(int)
        new[rng.integers(n)] += 1
        block = int(rng.choice([16, 32, 64, 128, 256]))
        e = Engine(cached.tolist(), new.tolist(), pad=int(rng.integers(0, 9)), seed=seed, **SHAPES[shape])
        try:
            e.fill()
            check_attention(e, block, int(rng.integers(1, 1 + 2048 // block)), seed=seed)
        finally:
            e.close()


@pytest.mark.parametrize("shape", ["bf16_g4_d128", "f32_g4_d128"])
def test_lists_end_where_they_stop_ascending(shape):
    """At an entry that is negative, not above the one before it, or past the row's own block."""
    for kernel in kernels(shape):
        e = Engine([900], [6], seed=5, kernel=kernel, **SHAPES[shape])
        e.block = 64
        try:
            e.fill()
            raw = [[0, 3, 3, 5, 6], [0, 3, 2, 9, 14], [-1, 0, 1, 2, 3], [4, 14, 15, 16, 2], [14, 2 ** 30, 1, 2, 3], [2, 7, -9, 9, 10]]
            used = [[0, 3], [0, 3], [], [4, 14], [14], [2, 7]]
            blocks = i32([[x] * e.hkv for x in raw])
            q = e.randn(6, e.hq, e.d).to(DT[e.qt])
            out = torch.full_like(q, math.nan)
            gp.gp_sparse_attention(e.ctx, e.layer, e.step, 64, 5, q, blocks, out)
            gp.gp_synchronize(e.ctx)
            want, tol = attention_reference(e, q, [[np.array(x, dtype=int)] * e.hkv for x in used])
            assert torch.all((out.double() - want).abs() <= tol) and not out[2].any()
        finally:
            e.close()


@pytest.mark.parametrize("shape", ["bf16_g4_d128", "f32_g2_d64"])
def test_large_logits(shape):
    """Logits of a few hundred: one key takes all, whichever split or tile holds it."""
    for kernel in kernels(shape):
        e = Engine([3000, 100], [2, 40], seed=6, kernel=kernel, **SHAPES[shape])
        try:
            e.fill()
            check_attention(e, 64, 40, seed=1, scale=30.0)
        finally:
            e.close()


def test_long_and_many():
    """Every split, a single long request, and more rows than places on the GPU."""
    for cached, new, top in (([60_000], [1], 64), ([30_000, 9], [4, 4], 128), ([700] * 300, [1] * 300, 8)):
        e = Engine(cached, new, L=1, layer=0, hq=8, hkv=2, seed=top)
        try:
            e.fill()
            check_attention(e, 64, top, seed=top)
        finally:
            e.close()


@pytest.mark.parametrize("n", [63, 64, 65, 97, 300])
def test_many_requests(n):
    """At and over the 64 requests that a warp looks at together."""
    rng = np.random.default_rng(n)
    e = Engine(rng.integers(0, 500, n).tolist(), rng.integers(0, 6, n).tolist(), L=1, layer=0, hq=4, hkv=2, d=64, pad=3, seed=n)
    try:
        e.fill()
        bounds, scales = bounds_arrays(e, 32)
        gp.gp_block_bounds(e.ctx, 0, e.step, 32, bounds, scales)
        gp.gp_synchronize(e.ctx)
        check_bounds(e, 32, bounds, scales)
        check_select(e, 32, 6, 1, 2, seed=n)
        check_attention(e, 32, 6, seed=n)
    finally:
        e.close()


def test_cache_offsets_beyond_32_bits():
    """Pages at the far end of caches of 4.6e9 elements."""
    e = Engine([700, 300], [20, 1], L=1, layer=0, hq=16, hkv=8, pool=17_600, seed=7)
    try:
        e.fill()
        q, blocks, out = check_attention(e, 64, 6)
        gp.gp_set_scan_kernel(e.ctx, gp.GP_SCAN_CUDA_CORE)
        check_attention(e, 64, 6)
        bounds, scales = bounds_arrays(e, 64)
        gp.gp_block_bounds(e.ctx, 0, e.step, 64, bounds, scales)
        gp.gp_synchronize(e.ctx)
        rows = e.rows_of(e.k, 0, 720)
        held, scale = bounds_reference(rows[704:720])
        page = int(e.tables_host[e.slots[0], 2])
        assert np.array_equal(bounds[0, page, :, 3].cpu().numpy(), held) and np.array_equal(scales[0, page, :, 3].cpu().numpy(), scale)
        k = e.randn(21, 8, 128).bfloat16()
        gp.gp_append_mapped(e.ctx, 0, e.step, gp.gp_rope_default(), None, k, k, None)
        gp.gp_synchronize(e.ctx)
        assert torch.equal(e.rows_of(e.k, 0, 720)[700:], k[:20].double()) and torch.equal(e.rows_of(e.v, 1, 301)[300:], k[20:].double())
    finally:
        e.close()


def test_bad_device_data_is_reported_and_left_out():
    """Requests, slots, lengths and pages outside the engine's sizes: those rows stay as
    they were, the others are right, and the next call that synchronises tells."""
    def run(spoil, dead):
        e = Engine([300, 300, 300], [2, 2, 2], L=1, layer=0, seed=8)
        e.block = 64
        try:
            e.fill()
            q = e.randn(6, 8, 128).bfloat16()
            lists = [[np.array([0, 2, 4])] * 2] * 6
            blocks = i32([[[0, 2, 4]] * 2] * 6)
            want, tol = attention_reference(e, q, lists)
            spoil(e)
            out = torch.full_like(q, 7.0)
            gp.gp_sparse_attention(e.ctx, 0, e.step, 64, 3, q, blocks, out)
            with pytest.raises(gp.GrowPageError) as err:
                gp.gp_synchronize(e.ctx)
            assert err.value.status == gp.GP_ERR_INVALID
            live = [i for i in range(6) if i not in dead]
            assert torch.all((out[live].double() - want[live]).abs() <= tol[live])
            gp.gp_block_bounds(e.ctx, 0, e.step, 64, *bounds_arrays(e, 64))
            gp.gp_select_blocks(e.ctx, 0, e.step, 64, 3, 0, 1, q, *bounds_arrays(e, 64), blocks)
            try:
                gp.gp_synchronize(e.ctx)
            except gp.GrowPageError as again:
                assert again.status == gp.GP_ERR_INVALID
            return out
        finally:
            e.close()

    def put(name, at, value):
        return lambda e: e.arrays[name].__setitem__(at, value)

    assert (run(put("slots", 1, -1), [2, 3])[2:4] == 7.0).all()
    assert (run(put("slots", 1, 6), [2, 3])[2:4] == 7.0).all()
    assert (run(put("num_cached", 0, -400), [0, 1])[:2] == 7.0).all()
    assert (run(put("num_cached", 0, 2 ** 31 - 1), [0, 1])[:2] == 7.0).all()

    def page(e):
        e.arrays["tables"][int(e.slots[2]), 0] = e.pool
    run(page, [4, 5])


@pytest.mark.parametrize("new", [2, 50])
def test_a_bad_page_is_left_out(new):
    """Blocks on a page outside the pool count for nothing, in each kernel; the rest does."""
    for kernel in (gp.GP_SCAN_TENSOR_CORE, gp.GP_SCAN_CUDA_CORE):
        e = Engine([700], [new], L=1, layer=0, seed=8, kernel=kernel)
        e.block = 64
        try:
            e.fill()
            q = e.randn(new, 8, 128).bfloat16()
            blocks = i32([[[0, 2, 5, 6, 9]] * 2] * new)
            want, tol = attention_reference(e, q, [[np.array([0, 2, 9])] * 2] * new)
            for bad in (-1, e.pool, 2 ** 31 - 1, -2 ** 31):
                e.arrays["tables"][int(e.slots[0]), 1] = bad  # blocks 4 to 7
                out = torch.full_like(q, 7.0)
                gp.gp_sparse_attention(e.ctx, 0, e.step, 64, 5, q, blocks, out)
                with pytest.raises(gp.GrowPageError) as err:
                    gp.gp_synchronize(e.ctx)
                assert err.value.status == gp.GP_ERR_INVALID
                assert torch.all((out.double() - want).abs() <= tol)
        finally:
            e.close()


# ---- together ------------------------------------------------------------------------------


class Serving:
    """A decode loop over the calls: buffers of a serving process, two layers."""

    def __init__(self, prompts, block=32, top=6, stream=None, seed=0):
        self.L, self.hq, self.hkv, self.d, self.block, self.top = 2, 8, 2, 128, block, top
        self.n, self.pool, self.cap, self.rows = len(prompts), 64, 16, 1500
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        shape = (self.L, self.pool, self.hkv, PAGE, self.d)
        self.k, self.v = (torch.full(shape, math.nan, dtype=torch.bfloat16, **CUDA) for _ in range(2))
        self.M = self.n + 2
        cfg = gp.gp_config_default(num_layers=self.L, num_q_heads=self.hq, num_kv_heads=self.hkv, head_dim=self.d, max_slots=self.M,
                                   num_pages=self.pool, max_pages_per_req=self.cap)
        self.ctx = gp.gp_create(cfg, self.k, self.v, stream or torch.cuda.current_stream())
        self.free = i32([gp.gp_page_alloc(self.ctx) for _ in range(self.pool)][::-1])
        self.slots = [gp.gp_slot_acquire(self.ctx) for _ in prompts]
        z32 = lambda *s: torch.zeros(*s, dtype=torch.int32, **CUDA)
        self.cached, self.new = z32(self.n), i32(prompts)
        self.pos = torch.zeros(self.n, dtype=torch.int64, **CUDA)
        self.held, self.taken, self.state = z32(self.M), z32(1), z32(self.n)
        self.tables = torch.full((self.M, self.cap), -1, dtype=torch.int32, **CUDA)
        self.bounds = torch.zeros(self.L, self.pool, self.hkv, PAGE // block, 2, self.d, dtype=torch.int8, **CUDA)
        self.scales = torch.zeros(self.L, self.pool, self.hkv, PAGE // block, **CUDA)
        self.rope = gp.gp_rope_default(rotary_dim=64, layout=gp.GP_ROPE_INTERLEAVED, scaling=gp.GP_ROPE_RAMP, factor=4.0)
        self.history = [[[] for _ in prompts] for _ in range(2 * self.L)]  # what was appended: keys, values

    def buffers(self, rows):
        z = lambda *s, t=torch.bfloat16: torch.zeros(*s, dtype=t, **CUDA)
        b = dict(qkv=z(self.L, rows, (self.hq + 2 * self.hkv) * self.d), rot=z(self.L, rows, self.hq, self.d), rows=rows,
                 out=z(self.L, rows, self.hq, self.d), blocks=z(self.L, rows, self.hkv, self.top, t=torch.int32))
        b["step"] = gp.Step(self.ctx, slots=i32(self.slots), num_cached=self.cached, num_new=self.new, pos=self.pos, tables=self.tables,
                            row0=z(self.n + 1, t=torch.int32), row_req=z(rows, t=torch.int32), slot_map=z(rows, t=torch.int64),
                            positions=z(rows, t=torch.int64))
        return b

    def pass_(self, b):
        """The calls of a step, as they would be captured."""
        a, c, k = b["step"], self.hq * self.d, (self.hq + self.hkv) * self.d
        gp.gp_build_tables(self.ctx, a, self.held, self.held, self.free, self.taken, self.taken, self.state)
        for layer in range(self.L):
            x, rot = b["qkv"][layer], b["rot"][layer]
            q, key, val = (x[:, i:j].unflatten(1, (-1, self.d)) for i, j in ((0, c), (c, k), (k, x.shape[1])))
            gp.gp_append_mapped(self.ctx, layer, a, self.rope, q, key, val, rot)
            gp.gp_block_bounds(self.ctx, layer, a, self.block, self.bounds, self.scales)
            gp.gp_select_blocks(self.ctx, layer, a, self.block, self.top, 1, 2, rot, self.bounds, self.scales, b["blocks"][layer])
            gp.gp_sparse_attention(self.ctx, layer, a, self.block, self.top, rot, b["blocks"][layer], b["out"][layer])

    def after(self):
        """The lengths move on, on the GPU."""
        self.cached += self.new
        self.pos += self.new


def check_serving(s, b, new, cached):
    """The step's outputs from what was appended so far, in 64 bits, and its bounds and
    blocks from the caches."""
    e = Engine.__new__(Engine)
    e.L, e.hq, e.hkv, e.d, e.kv, e.qt, e.block, e.pool = s.L, s.hq, s.hkv, s.d, "bf16", "bf16", s.block, s.pool
    e.cached, e.new, e.slots, e.k, e.v = list(cached), list(new), s.slots, s.k, s.v
    e.row0, e.rows, e.tables_host = np.concatenate([[0], np.cumsum(new)]).astype(int), sum(new), s.tables.cpu().numpy()
    assert np.array_equal(s.held.cpu().numpy()[s.slots], [-(-(a + m) // PAGE) for a, m in zip(cached, new)])
    for layer in range(s.L):
        e.layer = layer
        x = b["qkv"][layer, :e.rows].unflatten(1, (-1, s.d))
        pos = np.concatenate([c + np.arange(m) for c, m in zip(cached, new)])
        inv = frequencies(64, gp.GP_ROPE_INTERLEAVED, gp.GP_ROPE_RAMP, 1e4, 4.0, 8192, 1.0, 32.0)
        want, tol = rotated(x[:, s.hq:s.hq + s.hkv], pos, inv, True, 0.1 * math.log(4.0) + 1.0)
        for r in range(s.n):
            at = slice(e.row0[r], e.row0[r + 1])
            keys, vals = e.rows_of(s.k, r, cached[r] + new[r]), e.rows_of(s.v, r, cached[r] + new[r])
            assert torch.all((keys[cached[r]:] - want[at]).abs() <= tol[at] + 2.0 ** -8 * want[at].abs())
            assert torch.equal(vals[cached[r]:], x[at, s.hq + s.hkv:].double())
            held = s.history[2 * layer][r]
            assert not len(held) or torch.equal(keys[:cached[r]], held) and torch.equal(vals[:cached[r]], s.history[2 * layer + 1][r])
            s.history[2 * layer][r], s.history[2 * layer + 1][r] = keys, vals
            for blk in range((cached[r] + new[r] - 1) // s.block + 1):
                got = bounds_reference(keys[blk * s.block:(blk + 1) * s.block])
                page, sub = e.tables_host[s.slots[r], blk * s.block // PAGE], blk % (PAGE // s.block)
                assert np.array_equal(s.bounds[layer, page, :, sub].cpu().numpy(), got[0])
                assert np.array_equal(s.scales[layer, page, :, sub].cpu().numpy(), got[1])
        rot = b["rot"][layer]
        blocks = select_reference(e, rot, s.bounds.cpu().numpy(), s.scales.cpu().numpy(), s.block, s.top, 1, 2)
        assert np.array_equal(b["blocks"][layer, :e.rows].cpu().numpy(), blocks)
        out, bound = attention_reference(e, rot, [[h[h >= 0] for h in row] for row in blocks])
        assert torch.all((b["out"][layer, :e.rows].double() - out).abs() <= bound)


def run_serving(graph):
    prompts = [300, 1, 513, 40]
    stream = torch.cuda.Stream()
    s = Serving(prompts, stream=stream)
    with torch.cuda.stream(stream):
        big, small = s.buffers(sum(prompts) + 5), s.buffers(12)
        torch.cuda.synchronize()
        cached = [0] * 4
        plan = None
        outs = []
        for step in range(5):
            new = prompts if step == 0 else [[1, 1, 1, 1], [3, 0, 2, 1], [1, 3, 1, 1], [3, 3, 3, 3]][step - 1]
            b = big if step == 0 else small
            b["qkv"].copy_(torch.randn(b["qkv"].shape, device="cuda", generator=s.gen))
            s.new.copy_(i32(new))
            if not graph or step < 2:  # the second step is eager in both: its kernels are loaded when the third is captured
                s.pass_(b)
            elif plan is None:
                stream.synchronize()
                plan = torch.cuda.CUDAGraph()
                with torch.cuda.graph(plan, stream=stream):
                    s.pass_(b)
                    s.after()
                plan.replay()
            else:
                plan.replay()
            gp.gp_synchronize(s.ctx)
            assert (s.state == gp.GP_STEP_GIVEN).all()
            check_serving(s, b, new, cached)
            outs.append(b["out"].clone())
            cached = [a + m for a, m in zip(cached, new)]
            if not graph or step < 2:
                s.after()
            torch.cuda.synchronize()
            assert s.cached.tolist() == cached
        del plan
        torch.cuda.synchronize()
        gp.gp_destroy(s.ctx)
    return outs


def test_a_run_of_steps_eager_and_replayed():
    """Prompts, decode steps and drafted tokens of two layers, the lengths moved on by
    the GPU alone; a graph of the same calls gives the same bits."""
    eager, replayed = run_serving(False), run_serving(True)
    for a, b in zip(eager, replayed):
        assert torch.equal(bits(a), bits(b))


def test_a_captured_prompt():
    """Prompts in a graph: the larger kernels and their tensor maps, replayed over other contents."""
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        e = Engine([300, 0], [400, 90], L=1, layer=0, seed=11, stream=stream)
        e.block = 32
        e.fill()
        q = e.randn(490, 8, 128).bfloat16()
        blocks = torch.full((490, 2, 6), -1, dtype=torch.int32, **CUDA)
        bounds, scales = bounds_arrays(e, 32)
        out = torch.zeros_like(q)

        def calls():
            gp.gp_block_bounds(e.ctx, 0, e.step, 32, bounds, scales)
            gp.gp_select_blocks(e.ctx, 0, e.step, 32, 6, 0, 1, q, bounds, scales, blocks)
            gp.gp_sparse_attention(e.ctx, 0, e.step, 32, 6, q, blocks, out)

        e.cached, e.new = [0, 0], [700, 90]  # the bounds of every block
        calls()
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            calls()
        for _ in range(2):
            q.copy_(e.randn(490, 8, 128))
            e.fill()
            graph.replay()
            gp.gp_synchronize(e.ctx)
            e.cached, e.new = [300, 0], [400, 90]
            lists = [[h[h >= 0] for h in row] for row in blocks.cpu().numpy()]
            want, tol = attention_reference(e, q, lists)
            assert torch.all((out.double() - want).abs() <= tol)
            first = out.clone()
            calls()
            gp.gp_synchronize(e.ctx)
            assert torch.equal(bits(first), bits(out))
        del graph
        e.close()


FIRST_CAPTURE = """
import math, sys
sys.path[:0] = [%r, %r]
import torch
import test_gpu_sparse as t
stream = torch.cuda.Stream()
with torch.cuda.stream(stream):
    s = t.Serving([300, 1], stream=stream)
    b = s.buffers(310)
    s.new.copy_(t.i32([300, 1]))
    b["qkv"].copy_(torch.randn(b["qkv"].shape, device="cuda", generator=s.gen))
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        s.pass_(b)
    graph.replay()
    t.gp.gp_synchronize(s.ctx)
    t.check_serving(s, b, [300, 1], [0, 0])
    del graph
print("captured first")
"""


def test_the_first_calls_of_a_process_are_captured():
    """Nothing has to run before a capture: kernels and settings are made during it."""
    here = os.path.dirname(os.path.abspath(__file__))
    got = subprocess.run([sys.executable, "-c", FIRST_CAPTURE % (os.path.dirname(here), here)], capture_output=True, text=True, timeout=200)
    assert got.returncode == 0 and "captured first" in got.stdout, got.stdout + got.stderr


def test_two_engines_at_once():
    """Two contexts on two streams, the same calls at the same time: nothing shared."""
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    engines, outs = [], []
    for i, st in enumerate(streams):
        with torch.cuda.stream(st):
            e = Engine([2000, 30], [300, 1], L=1, layer=0, seed=20 + i, stream=st)
            e.fill()
            e.block = 64
            lists = random_lists(e, 8, i)
            blocks = np.full((301, 2, 8), -1)
            for row, x in enumerate(lists):
                for h in range(2):
                    blocks[row, h, :len(x[h])] = x[h]
            q = e.randn(301, 8, 128).bfloat16()
            engines.append((e, q, i32(blocks), lists))
    torch.cuda.synchronize()
    for i, st in enumerate(streams):
        with torch.cuda.stream(st):
            outs.append([torch.zeros_like(engines[i][1]) for _ in range(10)])
    torch.cuda.synchronize()
    for k in range(10):
        for i in range(2):
            e, q, blocks, _ = engines[i]
            gp.gp_sparse_attention(e.ctx, 0, e.step, 64, 8, q, blocks, outs[i][k])
    for i in range(2):
        e, q, blocks, lists = engines[i]
        gp.gp_synchronize(e.ctx)
        want, tol = attention_reference(e, q, lists)
        for out in outs[i]:
            assert torch.all((out.double() - want).abs() <= tol) and torch.equal(bits(out), bits(outs[i][0]))
        e.close()


def test_bounds_after_an_eviction():
    """An eviction moves keys; a step over all tokens left forms their bounds anew."""
    e = Engine([0], [700], L=1, layer=0, seed=9, cap=3)
    try:
        e.fill()
        for _ in range(e.pool):
            gp.gp_page_alloc(e.ctx)
        slots = [gp.gp_slot_acquire(e.ctx) for _ in range(e.M)]
        assert slots[e.slots[0]] == e.slots[0]
        req = gp.Request(int(e.slots[0]), e.tables_host[e.slots[0], :3], 700, 3)
        w = torch.rand(1, e.M, 2, 3 * PAGE, device="cuda", generator=e.gen)
        gp.gp_evict_weighted(e.ctx, [req], [700], [333], w)
        e.new = [333]
        for name, x in (("num_new", [333]), ("row0", [0, 333])):
            e.arrays[name].copy_(i32(x))
        bounds, scales = bounds_arrays(e, 64)
        gp.gp_block_bounds(e.ctx, 0, e.step, 64, bounds, scales)
        gp.gp_synchronize(e.ctx)
        check_bounds(e, 64, bounds, scales)
    finally:
        e.close()


def test_capture_and_side_stream():
    """A captured call while a compaction is pending is refused; eager ones wait for it."""
    stream, side = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(stream):
        e = Engine([0], [700], L=1, layer=0, seed=10, cap=3, stream=stream)
        e.fill()
        for _ in range(e.pool):
            gp.gp_page_alloc(e.ctx)
        [gp.gp_slot_acquire(e.ctx) for _ in range(e.M)]
        req = gp.Request(int(e.slots[0]), e.tables_host[e.slots[0], :3], 700, 3)
        w = torch.rand(1, e.M, 2, 3 * PAGE, device="cuda", generator=e.gen)
        gp.gp_set_compaction_stream(e.ctx, side)
        e.block = 64
        q, out = e.randn(700, 8, 128).bfloat16(), torch.zeros(700, 8, 128, dtype=torch.bfloat16, **CUDA)
        blocks = torch.zeros(700, 2, 1, dtype=torch.int32, **CUDA)
        gp.gp_sparse_attention(e.ctx, 0, e.step, 64, 1, q, blocks, out)
        stream.synchronize()
        gp.gp_evict_weighted(e.ctx, [req], [700], [333], w)
        graph = torch.cuda.CUDAGraph()
        with pytest.raises(gp.GrowPageError) as err:
            with torch.cuda.graph(graph, stream=stream):
                gp.gp_sparse_attention(e.ctx, 0, e.step, 64, 1, q, blocks, out)
        assert err.value.status == gp.GP_ERR_STATE
        e.new = [333]
        for name, x in (("num_new", [333]), ("row0", [0, 333])):
            e.arrays[name].copy_(i32(x))
        bounds, scales = bounds_arrays(e, 64)
        gp.gp_block_bounds(e.ctx, 0, e.step, 64, bounds, scales)  # waits for the eviction
        gp.gp_synchronize(e.ctx)
        check_bounds(e, 64, bounds, scales)
        e.close()


def test_calls_wait_for_a_long_eviction():
    """Calls whose launches overlap those before them still wait for the side stream: an
    eviction of many pages and layers, at once followed by bounds and attention."""
    stream, side = torch.cuda.Stream(), torch.cuda.Stream()
    T, keep, L = 60 * PAGE, 40 * PAGE, 24
    with torch.cuda.stream(stream):
        e = Engine([T - 1], [1], L=L, layer=L - 1, hq=16, hkv=8, seed=30, cap=60, stream=stream)
        for layer in range(L):
            e.layer = layer
            e.fill()
        e.block = 64
        for _ in range(e.pool):
            gp.gp_page_alloc(e.ctx)
        [gp.gp_slot_acquire(e.ctx) for _ in range(e.M)]
        req = gp.Request(int(e.slots[0]), e.tables_host[e.slots[0], :60], T, 60)
        w = torch.rand(L, e.M, 8, 60 * PAGE, device="cuda", generator=e.gen)
        q, out = e.randn(1, 16, 128).bfloat16(), torch.zeros(1, 16, 128, dtype=torch.bfloat16, **CUDA)
        blocks = i32(np.tile(np.arange(0, 640, 5), (1, 8, 1)))
        gp.gp_set_compaction_stream(e.ctx, side)
        bounds, scales = bounds_arrays(e, 64)
        lengths = i32([keep - 1])
        stream.synchronize()
        for _ in range(3):  # kernels ahead of the wait, for the launches behind it to overlap
            gp.gp_sparse_attention(e.ctx, e.layer, e.step, 64, 128, q, blocks, out)
        gp.gp_evict_weighted(e.ctx, [req], [T], [keep], w)
        e.arrays["num_cached"].copy_(lengths)
        gp.gp_block_bounds(e.ctx, e.layer, e.step, 64, bounds, scales)
        gp.gp_sparse_attention(e.ctx, e.layer, e.step, 64, 128, q, blocks, out)
        gp.gp_synchronize(e.ctx)
        e.cached = [keep - 1]
        check_bounds(e, 64, bounds, scales)
        want, tol = attention_reference(e, q, [[np.arange(0, 640, 5)] * 8])
        assert torch.all((out.double() - want).abs() <= tol)
        e.close()


@pytest.mark.parametrize("kernel", [gp.GP_SCAN_TENSOR_CORE, gp.GP_SCAN_CUDA_CORE])
def test_calls_behind_chunk_attention(kernel):
    """Attention whose queries are what chunk attention has just written, and appends to the
    pages that it has just read, with and without its other kernels in between."""
    e = Engine([3000], [300], L=1, layer=0, seed=32, cap=13, kernel=kernel)
    try:
        e.fill()
        for _ in range(e.pool):
            gp.gp_page_alloc(e.ctx)
        [gp.gp_slot_acquire(e.ctx) for _ in range(e.M)]
        req = gp.Request(int(e.slots[0]), e.tables_host[e.slots[0], :13], 3300, 13)
        q = e.randn(300, 8, 128).bfloat16()
        blocks = i32(np.tile(np.arange(0, 46, 3), (300, 2, 1)))
        k, v = e.randn(300, 2, 128).bfloat16(), e.randn(300, 2, 128).bfloat16()
        k0, v0 = e.k.clone(), e.v.clone()
        rope = gp.gp_rope_default()
        for weights in (None, torch.zeros(1, e.M, 2, 13 * PAGE, **CUDA)):
            results = []
            for sync in (True, False, False):
                e.k.copy_(k0)
                e.v.copy_(v0)
                mid, out = torch.zeros_like(q), torch.zeros_like(q)
                torch.cuda.synchronize()
                gp.gp_chunk_attention(e.ctx, 0, [req], [3000], [300], q, mid, weights)
                if sync:
                    torch.cuda.synchronize()
                gp.gp_sparse_attention(e.ctx, 0, e.step, 64, 16, mid, blocks, out)
                gp.gp_append_mapped(e.ctx, 0, e.step, rope, None, k, v, None)
                gp.gp_synchronize(e.ctx)
                results.append((mid, out, e.k.clone(), e.v.clone()))
            for other in results[1:]:
                assert all(torch.equal(bits(a), bits(b)) for a, b in zip(results[0], other))
            assert results[0][1].abs().sum() > 0
    finally:
        e.close()


def test_captured_behind_copies_and_other_streams():
    """In a graph, calls behind a copy, and behind another stream's work that an event joins."""
    stream, other = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(stream):
        e = Engine([300], [50], L=1, layer=0, seed=31, stream=stream)
        e.fill()
        e.block = 32
        lists = random_lists(e, 5, 3)
        blocks = np.full((50, 2, 5), -1)
        for row, x in enumerate(lists):
            for h in range(2):
                blocks[row, h, :len(x[h])] = x[h]
        blocks = i32(blocks)
        src, q, half = e.randn(50, 8, 128).bfloat16(), torch.zeros(50, 8, 128, dtype=torch.bfloat16, **CUDA), e.randn(50, 8, 128).bfloat16()
        out, out2 = torch.zeros_like(q), torch.zeros_like(q)
        gp.gp_sparse_attention(e.ctx, 0, e.step, 32, 5, q, blocks, out)
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            q.copy_(src)
            gp.gp_sparse_attention(e.ctx, 0, e.step, 32, 5, q, blocks, out)
            other.wait_stream(stream)
            with torch.cuda.stream(other):
                for _ in range(20):
                    half.mul_(0.5)
                    half.mul_(2.0)
                half.add_(1.0)
            stream.wait_stream(other)
            gp.gp_sparse_attention(e.ctx, 0, e.step, 32, 5, half, blocks, out2)
        base = half.clone()
        graph.replay()
        gp.gp_synchronize(e.ctx)
        want, tol = attention_reference(e, src, lists)
        assert torch.all((out.double() - want).abs() <= tol)
        assert torch.equal(half, base + 1.0)
        want, tol = attention_reference(e, half, lists)
        assert torch.all((out2.double() - want).abs() <= tol)
        del graph
        e.close()


def test_kernel_times_are_counted():
    e = Engine([100], [3], L=1, layer=0)
    try:
        e.fill()
        gp.gp_set_timing(e.ctx, True)
        check_attention(e, 16, 3)
        ms, launches = gp.gp_kernel_time(e.ctx, gp.GP_KERNEL_SPARSE)
        assert ms > 0.0 and launches >= 1
        gp.gp_debug_fail_next_launch(e.ctx, gp.GP_KERNEL_BOUNDS)
        with pytest.raises(gp.GrowPageError) as err:
            gp.gp_block_bounds(e.ctx, 0, e.step, 64, *bounds_arrays(e, 64))
        assert err.value.status == gp.GP_ERR_CUDA
    finally:
        e.close()
