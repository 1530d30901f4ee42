"""What the calls over a step's device arrays refuse, on a host-only context: every
bad argument is GP_ERR_INVALID (GP_ERR_UNSUPPORTED for a step too large) before
anything else is looked at, good ones reach the device check (GP_ERR_STATE without a
device).  And the defaults, layouts and names of the interface."""

import os
import subprocess
import tempfile

import pytest

import paged_kv_cache_step_gb300 as gp
from paged_kv_cache_step_gb300 import binding

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
AT = [(i + 1) << 24 for i in range(24)]  # stand for device addresses, 16 MiB apart; never followed
NAMES = ("slots", "num_cached", "num_new", "pos", "tables", "row0", "row_req", "slot_map", "positions")


@pytest.fixture
def ctx():
    c = gp.gp_create(gp.gp_config_default(num_layers=2, num_q_heads=8, num_kv_heads=2, head_dim=128, max_slots=6, num_pages=16,
                                          max_pages_per_req=4))
    yield c
    gp.gp_destroy(c)


def step(ctx, n=3, max_rows=20, **other):
    return gp.Step(ctx, n=n, max_rows=max_rows, **dict(zip(NAMES, AT), **other))


def tables(ctx, s=None, held=AT[9], pages=AT[10], free=AT[11], taken_in=AT[12], taken=AT[12], state=AT[13], num_free=7):
    gp.gp_build_tables(ctx, s or step(ctx), held, pages, free, taken_in, taken, state, num_free=num_free)


def append(ctx, s=None, layer=0, rope=None, q=AT[9], k=AT[10], v=AT[11], rot=AT[12]):
    gp.gp_append_mapped(ctx, layer, s or step(ctx), rope or gp.gp_rope_default(rotary_dim=128), q, k, v, rot)


def bounds(ctx, s=None, layer=0, block=64, b=AT[9], scales=AT[10]):
    gp.gp_block_bounds(ctx, layer, s or step(ctx), block, b, scales)


def select(ctx, s=None, layer=0, block=64, top=8, sink=1, recent=2, q=AT[9], b=AT[10], scales=AT[11], out=AT[12]):
    gp.gp_select_blocks(ctx, layer, s or step(ctx), block, top, sink, recent, q, b, scales, out)


def attend(ctx, s=None, layer=0, block=64, top=8, q=AT[9], blocks=AT[10], out=AT[11]):
    gp.gp_sparse_attention(ctx, layer, s or step(ctx), block, top, q, blocks, out)


CALLS = [tables, append, bounds, select, attend]


def status(call, *a, **kw):
    with pytest.raises(gp.GrowPageError) as e:
        call(*a, **kw)
    return e.value.status


@pytest.mark.parametrize("call", CALLS)
def test_good_arguments_reach_the_device_check(ctx, call):
    assert status(call, ctx) == gp.GP_ERR_STATE
    assert status(call, ctx, step(ctx, n=0)) == gp.GP_ERR_STATE
    assert status(call, ctx, step(ctx, max_rows=0, row_req=None, slot_map=None, positions=None)) == gp.GP_ERR_STATE
    none = dict.fromkeys(("slots", "num_cached", "num_new", "pos"))
    assert status(call, ctx, step(ctx, n=0, **none)) == gp.GP_ERR_STATE
    assert status(call, ctx, step(ctx, n=6)) == gp.GP_ERR_STATE
    assert gp.gp_free_page_count(ctx) == 16


@pytest.mark.parametrize("call", CALLS)
def test_bad_steps(ctx, call):
    for bad in (dict(n=-1), dict(n=7), dict(max_rows=-1), *({name: None} for name in NAMES), *({name: AT[0] + 2} for name in NAMES),
                dict(pos=AT[3] + 4), dict(slot_map=AT[7] + 4), dict(positions=AT[8] + 4)):
        assert status(call, ctx, step(ctx, **bad)) == gp.GP_ERR_INVALID, bad
    assert status(call, ctx, step(ctx, max_rows=1 << 27)) == gp.GP_ERR_UNSUPPORTED
    lib = gp.load()
    assert lib.gp_build_tables(ctx, None, AT[9], AT[10], AT[11], 7, None, AT[12], AT[13]) == gp.GP_ERR_INVALID
    assert lib.gp_sparse_attention(ctx, 0, None, 64, 8, AT[9], AT[10], AT[11]) == gp.GP_ERR_INVALID
    assert lib.gp_sparse_attention(None, 0, step(ctx)._raw, 64, 8, AT[9], AT[10], AT[11]) == gp.GP_ERR_INVALID


def test_a_step_of_many_requests_is_refused():
    c = gp.gp_create(gp.gp_config_default(num_layers=1, num_q_heads=2, num_kv_heads=1, head_dim=64, max_slots=300_000, num_pages=4,
                                          max_pages_per_req=4))
    try:
        assert status(bounds, c, step(c, n=4096)) == gp.GP_ERR_STATE
        assert status(bounds, c, step(c, n=4097)) == gp.GP_ERR_INVALID
        assert status(tables, c, step(c, n=4)) == gp.GP_ERR_UNSUPPORTED
    finally:
        gp.gp_destroy(c)


def test_bad_tables(ctx):
    for bad in (dict(held=None), dict(pages=None), dict(taken=None), dict(state=None), dict(num_free=-1), dict(free=None),
                dict(held=AT[9] + 1), dict(pages=AT[10] + 2), dict(free=AT[11] + 3), dict(taken_in=AT[12] + 2), dict(state=AT[13] + 1)):
        assert status(tables, ctx, **bad) == gp.GP_ERR_INVALID, bad
    for good in (dict(taken_in=None), dict(free=None, num_free=0), dict(pages=AT[9]), dict(taken_in=AT[14])):
        assert status(tables, ctx, **good) == gp.GP_ERR_STATE, good


def test_tables_that_overlap(ctx):
    for bad in (dict(pages=AT[9] + 4), dict(taken=AT[9]), dict(state=AT[1]), dict(state=AT[11] + 24), dict(pages=AT[11]), dict(taken=AT[13])):
        assert status(tables, ctx, **bad) == gp.GP_ERR_INVALID, bad
    for bad in (dict(row0=AT[0] + 8), dict(row_req=AT[7] + 80), dict(tables=AT[9]), dict(positions=AT[7] + 8), dict(tables=AT[5] - 92)):
        assert status(tables, ctx, step(ctx, **bad)) == gp.GP_ERR_INVALID, bad
    assert status(tables, ctx, step(ctx, tables=AT[5] - 96)) == gp.GP_ERR_STATE  # 6 x 4 entries, right before row0
    assert status(tables, ctx, state=AT[11] + 28) == gp.GP_ERR_STATE             # right behind the free list


def test_bad_appends(ctx):
    for bad in (dict(layer=-1), dict(layer=2), dict(k=None), dict(v=None), dict(q=None), dict(rot=None), dict(q=AT[9] + 8), dict(k=AT[10] + 8),
                dict(v=AT[11] + 4), dict(rot=AT[12] + 2), dict(rot=AT[10]), dict(rot=AT[11] + 16), dict(rot=AT[9] + 16)):
        assert status(append, ctx, **bad) == gp.GP_ERR_INVALID, bad
    for good in (dict(q=None, rot=None), dict(rot=AT[9]), dict(layer=1), dict(rot=AT[10] - 20 * 8 * 128 * 2)):
        assert status(append, ctx, **good) == gp.GP_ERR_STATE, good


def test_bad_strides(ctx):
    lib, s, rope = gp.load(), step(ctx)._raw, gp.gp_rope_default(rotary_dim=64)

    def call(q=1024, k=256, v=256, rot=AT[12]):
        return lib.gp_append_mapped(ctx, 0, s, rope, AT[9], q, AT[10], k, AT[11], v, rot)

    assert call() == gp.GP_ERR_STATE and call(1536, 1536, 264) == gp.GP_ERR_STATE
    for bad in (dict(q=1016), dict(k=248), dict(v=0), dict(q=-1024), dict(q=1028), dict(k=260), dict(v=2 ** 62), dict(q=1032, rot=AT[9])):
        assert call(**bad) == gp.GP_ERR_INVALID, bad


def test_bad_rotary_forms(ctx):
    for bad in (dict(layout=2), dict(layout=-1), dict(rotary_dim=144), dict(rotary_dim=-16), dict(rotary_dim=24), dict(scaling=4), dict(scaling=-1),
                dict(theta=1.0), dict(theta=-3.0), dict(theta=float("nan")), dict(theta=float("inf")), dict(amplitude=float("inf")),
                dict(scaling=gp.GP_ROPE_LINEAR, factor=0.5), dict(scaling=gp.GP_ROPE_LINEAR, factor=float("nan")),
                dict(scaling=gp.GP_ROPE_BANDS, original_length=0), dict(scaling=gp.GP_ROPE_BANDS, low_turns=0.0),
                dict(scaling=gp.GP_ROPE_BANDS, low_turns=4.0), dict(scaling=gp.GP_ROPE_RAMP, low_turns=32.0),
                dict(scaling=gp.GP_ROPE_RAMP, high_turns=0.5), dict(scaling=gp.GP_ROPE_RAMP, high_turns=float("inf"))):
        assert status(append, ctx, rope=gp.gp_rope_default(**dict(dict(rotary_dim=128), **bad))) == gp.GP_ERR_INVALID, bad
    for good in (dict(rotary_dim=0), dict(factor=0.1), dict(scaling=gp.GP_ROPE_BANDS, low_turns=2.0), dict(scaling=gp.GP_ROPE_RAMP, low_turns=4.0)):
        assert status(append, ctx, rope=gp.gp_rope_default(**good)) == gp.GP_ERR_STATE, good
    assert gp.load().gp_append_mapped(ctx, 0, step(ctx)._raw, None, AT[9], 1024, AT[10], 256, AT[11], 256, AT[12]) == gp.GP_ERR_INVALID
    with pytest.raises(TypeError):
        gp.gp_rope_default(rotary=3)


def test_bad_bounds_and_lists(ctx):
    for block in (0, 8, 48, 512, -16):
        for call in (bounds, select, attend):
            assert status(call, ctx, block=block) == gp.GP_ERR_INVALID
    for call in (bounds, select, attend):
        assert status(call, ctx, layer=2) == gp.GP_ERR_INVALID and status(call, ctx, layer=-1) == gp.GP_ERR_INVALID
        for block in (16, 32, 128, 256):
            assert status(call, ctx, block=block) == gp.GP_ERR_STATE
    for bad in (dict(b=None), dict(scales=None), dict(b=AT[9] + 8), dict(scales=AT[10] + 2)):
        assert status(bounds, ctx, **bad) == gp.GP_ERR_INVALID, bad
    for bad in (dict(top=0, sink=0, recent=0), dict(top=2), dict(recent=0), dict(sink=-1), dict(top=65_537), dict(sink=2 ** 31 - 1, recent=2 ** 31 - 1),
                dict(q=None), dict(b=None), dict(scales=None), dict(out=None), dict(q=AT[9] + 4), dict(b=AT[10] + 4), dict(scales=AT[11] + 1),
                dict(out=AT[12] + 2)):
        assert status(select, ctx, **bad) == gp.GP_ERR_INVALID, bad
    assert status(select, ctx, top=3) == gp.GP_ERR_STATE and status(select, ctx, top=65_536) == gp.GP_ERR_STATE
    for bad in (dict(top=0), dict(top=-1), dict(top=65_537), dict(q=None), dict(blocks=None), dict(out=None), dict(q=AT[9] + 8), dict(out=AT[11] + 8),
                dict(blocks=AT[10] + 2), dict(out=AT[9]), dict(out=AT[9] + 16), dict(out=AT[10]), dict(out=AT[10] + 20 * 2 * 8 * 4 - 16)):
        assert status(attend, ctx, **bad) == gp.GP_ERR_INVALID, bad
    assert status(attend, ctx, out=AT[10] + 20 * 2 * 8 * 4) == gp.GP_ERR_STATE


def test_buffers_that_are_no_device_tensors(ctx):
    torch = pytest.importorskip("torch")
    x = torch.zeros(64, dtype=torch.int32)
    with pytest.raises(gp.GrowPageError):
        step(ctx, slots=x)
    with pytest.raises(gp.GrowPageError):
        append(ctx, k=torch.zeros(20, 2, 128, dtype=torch.bfloat16))
    with pytest.raises(gp.GrowPageError):
        attend(ctx, blocks=x)


def test_rope_default_and_layouts():
    r = gp.gp_rope_default()
    assert (r.layout, r.rotary_dim, r.scaling, r.original_length) == (gp.GP_ROPE_HALF, 0, gp.GP_ROPE_NONE, 8192)
    assert (r.theta, r.factor, r.low_turns, r.high_turns, r.amplitude) == (1e4, 1.0, 1.0, 0.0, 0.0)
    src = r"""
#include <stdio.h>
#include <stddef.h>
#include "growpage.h"
int main(void) {
  printf("%zu %zu %zu %zu %zu %zu %zu %d %d %d\n", sizeof(gp_step), offsetof(gp_step, slots), offsetof(gp_step, tables),
         offsetof(gp_step, positions), sizeof(gp_rope), offsetof(gp_rope, theta), offsetof(gp_rope, amplitude), GP_KERNEL_SPARSE,
         GP_STEP_INVALID, GP_ROPE_RAMP);
  return 0;
}
"""
    with tempfile.TemporaryDirectory() as d:
        c, exe = os.path.join(d, "t.c"), os.path.join(d, "t")
        open(c, "w").write(src)
        subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), c, "-o", exe], check=True)
        got = [int(x) for x in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]
    rope = binding.GpRope
    assert got == [binding._STEP_PACK.size, 8, 8 + 4 * 8, 8 + 8 * 8, binding.C.sizeof(rope), rope.theta.offset, rope.amplitude.offset,
                   gp.GP_KERNEL_SPARSE, gp.GP_STEP_INVALID, gp.GP_ROPE_RAMP]
