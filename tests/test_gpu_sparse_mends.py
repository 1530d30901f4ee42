"""What earlier tests of the calls over a step's device arrays do not show: not-a-number
queries, one rule for the rows that are left out, and waits that run out, in every
kernel.  The engine, the formulas in 64 bits and the tolerances are test_gpu_sparse.py's."""

import math

import numpy as np
import pytest
import torch

import paged_kv_cache_step_gb300 as gp
from test_gpu_sparse import (CUDA, DT, PAGE, SHAPES, Engine, Tables, attention_reference, bits, bounds_arrays, bounds_reference,
                             i32, kernels, random_lists, select_reference)

pytestmark = pytest.mark.gpu

ROWS = [1, 3, 70]  # a request: a decode step, drafted tokens, several pieces of 128 / G rows


def packed(e, lists, top):
    blocks = np.full((e.max_rows, e.hkv, top), -1)
    for row, x in enumerate(lists):
        for h in range(e.hkv):
            blocks[row, h, :len(x[h])] = x[h]
    return i32(blocks)


@pytest.mark.parametrize("new", ROWS)
@pytest.mark.parametrize("shape", ["bf16_g4_d128", "bf16_g2_d64", "f32_g4_d128", "f32_g2_d64", "bf16_q32"])
def test_a_query_that_is_not_a_number_gives_none(shape, new):
    """NaN in one head's query: that row and head come out NaN in every kernel, as the softmax
    of NaN does; an infinite logit too; the others are right and an empty list gives 0."""
    for kernel in kernels(shape):
        for cached in ([900] * 3, [6000]):  # (one request: clusters)
            e = Engine(cached, [new] * len(cached), seed=new, kernel=kernel, **SHAPES[shape])
            e.block = 64
            try:
                e.fill()
                lists = [[np.arange(5)] * e.hkv for _ in range(e.rows)]
                if e.rows > 1:
                    lists[-1] = [np.arange(0)] * e.hkv
                blocks = packed(e, lists, 40)
                q = e.randn(e.rows, e.hq, e.d).to(DT[e.qt])
                q[0, 0, 3] = math.nan
                want, tol = attention_reference(e, q, lists)
                out = torch.full_like(q, 7.0)
                gp.gp_sparse_attention(e.ctx, e.layer, e.step, 64, 40, q, blocks, out)
                gp.gp_synchronize(e.ctx)
                assert out[0, 0].isnan().all()
                flat, right, bound = (x.reshape(-1, e.d)[1:] for x in (out.double(), want, tol))
                assert torch.all((flat - right).abs() <= bound)
                assert e.rows == 1 or not out[-1].any()
                pages, places = e.at(0, 1)
                e.k[e.layer, pages, 0, places, 5] = 2.0
                q[0, 0] = 1.0
                q[0, 0, 5] = math.inf
                gp.gp_sparse_attention(e.ctx, e.layer, e.step, 64, 40, q, blocks, out)
                gp.gp_synchronize(e.ctx)
                assert out[0, 0].isnan().all()
            finally:
                e.close()


def told(e, reported):
    """The next call that synchronises reports bad device data, or nothing."""
    if reported:
        with pytest.raises(gp.GrowPageError) as err:
            gp.gp_synchronize(e.ctx)
        assert err.value.status == gp.GP_ERR_INVALID
    gp.gp_synchronize(e.ctx)


def check_rows(e, dead, reported, spoil):
    """Bounds, selected blocks and attention of a spoiled step: rows of `dead` are left
    out, every other is right, and each call is reported by itself."""
    block, per, layer = 64, PAGE // 64, e.layer
    e.block = block
    live = [i for i in range(e.rows) if i not in dead]
    rest = [i for i in range(e.max_rows) if i not in live]
    lists = random_lists(e, 6, 1)
    q, blocks = e.randn(e.max_rows, e.hq, e.d).to(DT[e.qt]), np.full((e.max_rows, e.hkv, 6), -1)
    blocks[e.rows:] = np.arange(6)
    for row, x in enumerate(lists):
        for h in range(e.hkv):
            blocks[row, h, :len(x[h])] = x[h]
    rng = np.random.default_rng(2)
    shape = (e.L, e.pool, e.hkv, per)
    held = np.sort(rng.integers(-127, 128, (*shape, 2, e.d)), -2)
    scales = 2.0 ** rng.integers(-6, 3, shape)
    want, tol = attention_reference(e, q, lists)
    chosen = select_reference(e, q, held, scales, block, 5, 1, 2)
    want_b, want_s = bounds_arrays(e, block)
    for r in range(len(e.new)):
        mine = [t for t in range(e.new[r]) if e.row0[r] + t in live]
        rows = e.rows_of(e.k, r, e.cached[r] + e.new[r])
        for b in {(e.cached[r] + t) // block for t in mine}:
            x = bounds_reference(rows[b * block:(b + 1) * block])
            page = int(e.tables_host[e.slots[r], b // per])
            want_b[layer, page, :, b % per] = torch.as_tensor(x[0].astype(np.int8), **CUDA)
            want_s[layer, page, :, b % per] = torch.as_tensor(x[1], **CUDA).float()
    spoil(e)
    got_b, got_s = bounds_arrays(e, block)
    gp.gp_block_bounds(e.ctx, layer, e.step, block, got_b, got_s)
    told(e, reported)
    assert torch.equal(got_b, want_b) and torch.equal(got_s, want_s)
    got = torch.full((e.max_rows, e.hkv, 5), -5, dtype=torch.int32, **CUDA)
    gp.gp_select_blocks(e.ctx, layer, e.step, block, 5, 1, 2, q, torch.as_tensor(held.astype(np.int8), **CUDA),
                        torch.as_tensor(scales.astype(np.float32), **CUDA), got)
    told(e, reported)
    assert np.array_equal(got[live].cpu().numpy(), chosen[live]) and (got[rest] == -5).all()
    out = torch.full((e.max_rows, e.hq, e.d), 7.0, dtype=DT[e.qt], **CUDA)
    gp.gp_sparse_attention(e.ctx, layer, e.step, block, 6, q, i32(blocks), out)
    told(e, reported)
    assert torch.all((out[live].double() - want[live]).abs() <= tol[live]) and (out[rest] == 7.0).all()


def put(name, at, value):
    return lambda e: e.arrays[name].__setitem__(at, value)


# three requests of `new` rows each, the second of which, or its second row, is spoiled:
# what is spoiled, how, which rows are left out, whether that is reported
SPOILED = [("row_req", "row", -1, "row", False), ("row_req", "row", 3, "row", True), ("row_req", "row", -2, "row", True),
           ("row_req", "row", 2 ** 31 - 1, "row", True), ("row_req", "row", 0, "row", True), ("row_req", "row", 2, "row", True),
           ("slots", 1, -1, "request", True), ("slots", 1, 6, "request", True), ("num_cached", 1, -400, "request", True),
           ("num_cached", 1, 2 ** 31 - 1, "request", True), ("row0", 3, 2 ** 31 - 1, "last", True)]


@pytest.mark.parametrize("new", [2, 50])
@pytest.mark.parametrize("shape", ["bf16_g4_d128", "bf16_g2_d64", "f32_g2_d64"])
@pytest.mark.parametrize("name,at,value,dead,reported", SPOILED)
def test_rows_that_are_left_out(name, at, value, dead, reported, shape, new):
    """The same rows in the bounds, the selection and each attention kernel."""
    for kernel in kernels(shape):
        e = Engine([700, 300, 40], [new] * 3, pad=2, seed=new, kernel=kernel, **SHAPES[shape])
        try:
            e.fill()
            rows = {"row": [new + 1], "request": range(new, 2 * new), "last": range(2 * new, 3 * new)}[dead]
            check_rows(e, rows, reported, put(name, new + 1 if at == "row" else at, value))
        finally:
            e.close()


@pytest.mark.parametrize("fit,past", [(1, 1), (1, 2), (3, 1), (40, 30), (64, 1), (63, 65), (129, 3)])
@pytest.mark.parametrize("shape", ["bf16_g4_d128", "bf16_g2_d64", "f32_g2_d64"])
def test_rows_past_the_end_of_the_table(shape, fit, past):
    """A request whose first `fit` rows have a place in its table and whose last `past` have
    none: those alone are left out, and reported."""
    def spoil(e):
        e.arrays["row0"][2] = 5 + fit + past
        e.arrays["row_req"][5 + fit:5 + fit + past] = 1

    for kernel in kernels(shape):
        e = Engine([300, 4 * PAGE - fit], [5, fit], pad=past + 2, cap=4, seed=fit, kernel=kernel, **SHAPES[shape])
        try:
            e.fill()
            check_rows(e, (), True, spoil)
        finally:
            e.close()


@pytest.mark.parametrize("new", [1, 40])
def test_rows_behind_the_last_are_not_looked_at(new):
    """Whatever row_req holds there, in every kernel."""
    for kernel in (gp.GP_SCAN_TENSOR_CORE, gp.GP_SCAN_CUDA_CORE):
        for value in (0, 1, 2, -5):
            e = Engine([300, 70], [new, new], pad=20, seed=4, kernel=kernel)
            try:
                e.fill()
                check_rows(e, (), False, put("row_req", slice(2 * new, None), value))
            finally:
                e.close()


# One request or many: with and without clusters; a row each, or pieces of 128 / G rows.
# Every share is longer than the ring of buffers.
@pytest.mark.parametrize("cached,new,top", [([60_000], [1], 400), ([9000] * 80, [1] * 80, 40), ([12_000], [40], 150), ([4000] * 40, [70] * 40, 20)])
@pytest.mark.parametrize("shape", ["bf16_g4_d128", "bf16_g2_d64"])
def test_waits_that_give_up_are_reported(shape, cached, new, top):
    """Without patience every CTA stops with copies and products in flight; with a little
    some may.  A row and head is right or as it was, and the next call is right."""
    s = SHAPES[shape]
    e = Engine(cached, new, L=1, layer=0, seed=top, **dict(s, hq=4 * s["hq"] // s["hkv"], hkv=4) if len(new) > 1 else s)
    e.block = 64
    try:
        e.fill()
        rng = np.random.default_rng(top)
        lists = [[np.sort(rng.permutation((e.cached[r] + t) // 64 + 1)[:top]) for _ in range(e.hkv)]
                 for r in range(len(new)) for t in range(new[r])]
        blocks = packed(e, lists, top)
        q = e.randn(e.rows, e.hq, e.d).bfloat16()
        want, tol = attention_reference(e, q, lists)
        gave_up = 0
        for limit in (0, 1, 300, 3000, 30_000, 0, -1):
            gp.gp_debug_set_wait_limit(e.ctx, gp.GP_KERNEL_SPARSE, limit)
            out = torch.full_like(q, 7.0)
            gp.gp_sparse_attention(e.ctx, 0, e.step, 64, top, q, blocks, out)
            try:
                gp.gp_synchronize(e.ctx)
                assert limit != 0
            except gp.GrowPageError as err:
                assert err.status == gp.GP_ERR_TIMEOUT and limit >= 0
            right = ((out.double() - want).abs() <= tol).all(-1)
            left = (out == 7.0).all(-1)
            assert torch.all(right | left)
            assert limit >= 0 or right.all()
            gave_up += int(left.any())
        assert gave_up >= 2
    finally:
        e.close()


@pytest.mark.parametrize("n", [4, 300])
def test_pages_of_a_slot_that_is_listed_twice(n):
    """num_pages_dev, a buffer of its own, gets the pages of every listed slot, of refused ones too."""
    slots = np.arange(n)
    slots[[1, n - 1]] = 0, 2  # slots 0 and 2 twice
    held = np.arange(n + 3) % 3 + 1
    t = Tables([5] * n, [1] * n, 2 * n, 5, slots=slots, M=n + 3, held=held, seed=n)
    gp.gp_synchronize(t.ctx)
    t.num_pages = torch.full_like(t.held, -9)
    t.taken.zero_()
    gp.gp_build_tables(t.ctx, gp.Step(t.ctx, **t.a), t.held, t.num_pages, t.free, None, t.taken, t.state)
    t.want["num_pages"] = np.where(np.isin(np.arange(n + 3), slots), held, -9)
    assert (t.want["state"][[0, 1, 2, n - 1]] == gp.GP_STEP_INVALID).all()
    t.check()


@pytest.mark.parametrize("new,rows,free,states", [
    ([3, 300, 1, 0], 4, 9, [0, 2, 2, 0]),    # 303 rows asked for before the third: it has none, though one is left
    ([3, 300, 1, 0], 304, 9, [0, 0, 0, 0]),
    ([300, 3, 1], 304, 1, [1, 1, 1]),        # two pages missing, one left: no later request takes it
    ([300, 3, 1], 303, 9, [0, 0, 2]),
    ([300, 200, 1], 400, 1, [1, 2, 2])])     # rows of a request refused for its pages count
def test_rows_and_pages_are_given_in_order(new, rows, free, states):
    t = Tables([0] * len(new), new, rows, free, held=[0] * (len(new) + 3), seed=1)
    gp.gp_synchronize(t.ctx)
    assert t.state.tolist() == states
    t.check()


def test_pages_go_back_to_the_pool():
    """What the table on the device names comes back through the host: a request's entries, one
    gp_page_unref each."""
    e = Engine([0, 0], [700, 20], L=1, layer=0, cap=4, spare=3)
    try:
        pages = [gp.gp_page_alloc(e.ctx) for _ in range(e.pool)]
        held, taken, state = (torch.zeros(k, dtype=torch.int32, **CUDA) for k in (e.M, 1, 2))
        gp.gp_build_tables(e.ctx, e.step, held, held, i32(pages), taken, taken, state)
        gp.gp_synchronize(e.ctx)
        assert gp.gp_free_page_count(e.ctx) == 0
        tables, counts = e.arrays["tables"].cpu().numpy(), held.cpu().numpy()
        for s in e.slots:
            for page in tables[s, :counts[s]]:
                gp.gp_page_unref(e.ctx, int(page))
        assert gp.gp_free_page_count(e.ctx) == 4 and taken.tolist() == [4]
        for page in pages[4:]:
            gp.gp_page_unref(e.ctx, page)
        assert gp.gp_free_page_count(e.ctx) == e.pool
    finally:
        e.close()


def test_two_graphs_of_one_engine_at_once():
    """Graphs share the caller's buffers alone: two of one engine, of a decode step and of a
    prompt, replayed on two streams at the same time, give what each gives by itself."""
    stream, other = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(stream):
        e = Engine([2000, 900, 30], [300, 1, 1], L=1, layer=0, seed=40, stream=stream)
        e.fill()
        small = gp.Step(e.ctx, **dict(e.arrays, row0=i32([0, 0, 1, 2]), row_req=i32([1, 2]), slot_map=e.arrays["slot_map"][300:].clone(),
                                      positions=e.arrays["positions"][300:].clone()))
        runs = []
        for step, rows in ((e.step, 302), (small, 2)):
            q, out = e.randn(rows, 8, 128).bfloat16(), torch.zeros(rows, 8, 128, dtype=torch.bfloat16, **CUDA)
            blocks = torch.full((rows, 2, 9), -1, dtype=torch.int32, **CUDA)
            runs.append((step, q, blocks, out, *bounds_arrays(e, 32)))
        whole = gp.Step(e.ctx, **dict(e.arrays, num_cached=i32([0, 0, 0]), row0=i32([0, 2300, 3201, 3232]),
                                      row_req=i32(np.repeat([0, 1, 2], [2300, 901, 31])),
                                      slot_map=torch.zeros(3232, dtype=torch.int64, **CUDA), positions=torch.zeros(3232, dtype=torch.int64, **CUDA)))
        for x in runs:
            gp.gp_block_bounds(e.ctx, 0, whole, 32, x[4], x[5])

        def calls(step, q, blocks, out, bounds, scales):
            for _ in range(8):
                gp.gp_block_bounds(e.ctx, 0, step, 32, bounds, scales)
                gp.gp_select_blocks(e.ctx, 0, step, 32, 9, 1, 2, q, bounds, scales, blocks)
                gp.gp_sparse_attention(e.ctx, 0, step, 32, 9, q, blocks, out)

        graphs, alone = [], []
        for x in runs:
            calls(*x)
            stream.synchronize()
            alone.append([t.clone() for t in x[2:]])
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1], stream=stream):
                calls(*x)
        for x, want in zip(runs, alone):
            lists = [[h[h >= 0] for h in row] for row in x[2].cpu().numpy()]
            e.block, first = 32, 302 - len(lists)
            ref, tol = attention_reference(e, torch.cat([torch.zeros(first, 8, 128, **CUDA).bfloat16(), x[1]]), [[[], []]] * first + lists)
            assert torch.all((want[1].double() - ref[first:]).abs() <= tol[first:])
    for _ in range(20):
        for x in runs:
            x[2].fill_(-3)
            x[3].zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            graphs[0].replay()
        with torch.cuda.stream(other):
            for _ in range(6):
                graphs[1].replay()
        torch.cuda.synchronize()
        for x, want in zip(runs, alone):
            assert all(torch.equal(bits(a) if a.is_floating_point() else a, bits(b) if b.is_floating_point() else b)
                       for a, b in zip(x[2:], want))
    gp.gp_synchronize(e.ctx)
    del graphs
    e.close()


@pytest.mark.parametrize("new", [[1] * 9, [1, 300, 1, 0, 5]])
@pytest.mark.parametrize("shape", ["bf16_g4_d128", "bf16_g2_d64", "f32_g2_d64"])
def test_room_for_many_more_rows(shape, new):
    """Buffers of 3000 rows for a step of few: the same rows right, the others as they were."""
    for kernel in kernels(shape):
        e = Engine([900, 40, 3000, 255, 256, 7, 0, 513, 64][:len(new)], new, pad=3000, seed=len(new), kernel=kernel, **SHAPES[shape])
        try:
            e.fill()
            check_rows(e, (), False, lambda e: None)
        finally:
            e.close()
