"""The host side of the accumulated-weight calls over a runtime without a device
(fake_runtime.cpp): what a failing call leaves behind, what is allocated when, and
what an inspection call reads."""

import os
import shutil
import subprocess
import types

import numpy as np
import pytest

import paged_kv_cache_step_gb300 as gp
from paged_kv_cache_step_gb300 import _build_lib, binding

HERE = os.path.dirname(os.path.abspath(__file__))
DEV = 1 << 20  # stands for a device address; no kernel runs


@pytest.fixture(scope="module")
def fake_library(tmp_path_factory):
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_build_lib._nvcc()))), "include")
    if not os.path.exists(os.path.join(cuda, "cuda_runtime.h")) or not shutil.which("g++"):
        pytest.skip("no CUDA headers or no compiler")
    _build_lib.build()
    lib = str(tmp_path_factory.mktemp("fake") / "libfake.so")
    objs = [os.path.join(_build_lib.BUILD, f + ".o") for f in ("growpage", "weighted")]
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-Wl,-Bsymbolic", "-Wl,--no-undefined", "-I", _build_lib.INCLUDE,
                    "-I", _build_lib.CSRC, "-I", cuda, os.path.join(HERE, "fake_runtime.cpp"), *objs, "-o", lib], check=True)
    return lib


@pytest.fixture
def fake(fake_library, monkeypatch):
    """An engine of two layers over it, and its controls."""
    monkeypatch.setattr(_build_lib, "LIB", fake_library)
    monkeypatch.setattr(binding, "_LIB", None)
    lib = gp.load(build_if_missing=False)
    lib.fake_reset()
    cfg = gp.gp_config_default(num_layers=2, num_q_heads=4, num_kv_heads=2, head_dim=64, max_slots=4, num_pages=40,
                               max_pages_per_req=12)
    ctx = gp.gp_create(cfg, DEV, DEV, None)
    reqs = [gp.Request(gp.gp_slot_acquire(ctx), [gp.gp_page_alloc(ctx) for _ in range(p)], 0, 12) for p in (2, 12)]
    yield types.SimpleNamespace(ctx=ctx, reqs=reqs, calls=lambda name: lib.fake_calls(name.encode()),
                                fail=lambda name, after=1: lib.fake_fail(name.encode(), after))
    gp.gp_destroy(ctx)


def _masks(ctx, index, num_pages):
    return gp.unpack_mask(gp.gp_debug_keep_mask(ctx, index, 4, num_pages), num_pages * 256)


def test_keep_masks_of_a_budget_that_evicts_nothing(fake):
    """A budget over the tokens leaves a request as it is, however large it is."""
    gp.gp_evict_weighted(fake.ctx, fake.reqs, [500, 3000], [2 ** 31 - 1, 700], DEV)
    mask = _masks(fake.ctx, 0, 2)
    assert mask[:, :500].all() and not mask[:, 500:].any()
    mask = _masks(fake.ctx, 1, 12)
    assert mask[:, :700].all() and not mask[:, 700:].any()


def test_an_eviction_that_fails_half_way_leaves_no_record(fake):
    """The scratch with the last eviction's lists is given back for a larger one,
    and then the call fails: the lists are not read any more."""
    small, large = fake.reqs
    gp.gp_evict_weighted(fake.ctx, [small], [500], [300], DEV)
    assert _masks(fake.ctx, 0, 2)[:, :300].all()
    fake.fail("cudaEventSynchronize")  # the descriptors' place
    with pytest.raises(gp.GrowPageError) as err:
        gp.gp_evict_weighted(fake.ctx, [large], [3000], [2500], DEV)
    assert err.value.status == gp.GP_ERR_CUDA
    out = np.zeros(4 * 2 * 8 + 8192, dtype=np.uint32)  # room behind the masks, for what should not be written
    st = gp.load().gp_debug_keep_mask(fake.ctx, 0, out.ctypes.data)
    assert st == gp.GP_ERR_INVALID and not out.any()


def test_lists_that_hold_no_slots_are_not_made_into_masks(fake):
    """Lists that the selection has not written (its launch went lost): an error, and
    nothing behind the masks."""
    small = fake.reqs[0]
    gp.load().fake_skip_select(1)
    gp.gp_evict_weighted(fake.ctx, [small], [500], [300], DEV)
    out = np.zeros(4 * 2 * 8 + 8192, dtype=np.uint32)
    st = gp.load().gp_debug_keep_mask(fake.ctx, 0, out.ctypes.data)
    assert st == gp.GP_ERR_STATE and not out[4 * 2 * 8:].any()


def _alloc_count(fake):
    return [fake.calls(x) for x in ("cudaMalloc", "cudaHostAlloc", "cudaFree", "cudaFreeHost", "cudaEventCreate")]


@pytest.mark.parametrize("which", ["decode", "weighted decode", "chunk", "evict"])
def test_only_the_first_call_of_a_size_allocates(fake, which):
    """Descriptors go through eight slots in turn; they are made together, so the
    second call is as quick as any later one."""
    def call():
        if which == "decode":
            gp.gp_decode_attention(fake.ctx, 0, fake.reqs, [500, 3000], DEV, DEV, DEV)
        elif which == "weighted decode":
            gp.gp_decode_attention_weighted(fake.ctx, 0, fake.reqs, [500, 3000], DEV, None, DEV, DEV)
        elif which == "chunk":
            gp.gp_chunk_attention(fake.ctx, 0, fake.reqs, [400, 2000], [100, 50], DEV, DEV << 4, DEV)
        else:
            gp.gp_evict_weighted(fake.ctx, fake.reqs, [500, 3000], [300, 2900], DEV)

    call()
    first = _alloc_count(fake)
    for _ in range(20):
        call()
    assert _alloc_count(fake) == first


def test_descriptors_of_many_sizes(fake):
    """Calls that need more and more room: a slot that grows frees nothing that a copy
    still reads, and all slots have the new size."""
    grown = 0
    for n in (1, 400, 2500, 400, 2500, 1):
        before, waits = _alloc_count(fake), fake.calls("cudaEventSynchronize")
        for _ in range(9):
            gp.gp_chunk_attention(fake.ctx, 0, fake.reqs[1:], [0], [n], DEV, DEV << 4, None)
        after = _alloc_count(fake)
        if after[1] > before[1]:
            grown += 1
            assert after[1] == before[1] + 1 and fake.calls("cudaEventSynchronize") == waits + 8 + 9
    assert grown >= 1


@pytest.mark.parametrize("name", ["cudaHostAlloc", "cudaMalloc", "cudaEventCreate", "cudaEventSynchronize"])
def test_a_call_after_one_that_found_no_memory(fake, name):
    for after in (1, 2, 3):
        fake.fail(name, after)
        for _ in range(3):
            try:
                gp.gp_chunk_attention(fake.ctx, 0, fake.reqs, [400, 2000], [100, 50], DEV, DEV << 4, None)
            except gp.GrowPageError as err:
                assert err.status == gp.GP_ERR_CUDA
    for _ in range(20):
        gp.gp_chunk_attention(fake.ctx, 0, fake.reqs, [400, 2000], [100, 50], DEV, DEV << 4, None)


def _pool(fake):
    return ([(r.slot, r.num_pages, r.pages) for r in fake.reqs], gp.gp_free_page_count(fake.ctx),
            [gp.gp_page_refcount(fake.ctx, p) for p in range(40)])


@pytest.mark.parametrize("which", ["append", "decode", "weighted decode", "chunk", "evict", "evict on a side stream"])
def test_host_memory_that_runs_out_is_an_error(fake, which):
    """Every allocation of a call fails once: the call says so and changes nothing, no
    exception leaves the library, and the next call is as ever."""
    gp.gp_page_ref(fake.ctx, fake.reqs[0].pages[0])  # copied by an eviction
    if which == "evict on a side stream":
        gp.gp_set_compaction_stream(fake.ctx, 48)

    def call():
        if which == "append":
            gp.gp_append_tokens(fake.ctx, 0, fake.reqs, [500, 2000], [12, 900], DEV, DEV, DEV, DEV, DEV)
        elif which == "decode":
            gp.gp_decode_attention(fake.ctx, 0, fake.reqs, [500, 3000], DEV, DEV, DEV)
        elif which == "weighted decode":
            gp.gp_decode_attention_weighted(fake.ctx, 0, fake.reqs, [500, 3000], DEV, None, DEV, DEV)
        elif which == "chunk":
            gp.gp_chunk_attention(fake.ctx, 0, fake.reqs, [400, 2000], [100, 50], DEV, DEV << 4, DEV)
        else:
            gp.gp_evict_weighted(fake.ctx, fake.reqs, [500, 3000], [300, 2900], DEV)

    before, failed = _pool(fake), 0
    for k in range(1, 2000):
        gp.load().fake_fail_new(k)
        try:
            call()
            gp.load().fake_fail_new(-1)
            break
        except gp.GrowPageError as err:
            gp.load().fake_fail_new(-1)
            assert err.status == gp.GP_ERR_CUDA and "host memory" in str(err), (k, err)
            failed += 1
            assert _pool(fake) == before, k
    assert 0 < failed < 1999
    if "evict" in which:
        assert gp.gp_free_page_count(fake.ctx) == before[1] - 1
        gp.gp_set_compaction_stream(fake.ctx, None)
