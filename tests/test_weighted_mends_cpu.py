"""Faults of the accumulated-weight calls that need no device to show: what the
sources must not do, and what the calls and the binding refuse."""

import os
import re

import numpy as np
import pytest

import paged_kv_cache_step_gb300 as gp
from test_weighted_cpu import _append, _chunk, _decode, _evict, _state, _status, eng  # noqa: F401 (a fixture)

CSRC = os.path.join(os.path.dirname(gp.__file__), "csrc")


def _source(name):
    with open(os.path.join(CSRC, name)) as f:
        return f.read()


def _sources(suffix=(".cu", ".cuh", ".cpp", ".h")):
    return [f for f in sorted(os.listdir(CSRC)) if f.endswith(suffix)]


def _arguments(text, call):
    """The argument of every `call(...)` in the text, comments left out."""
    text = re.sub(r"//[^\n]*", "", text)
    for m in re.finditer(re.escape(call) + r"\(", text):
        depth, i = 1, m.end()
        while depth:
            depth += {"(": 1, ")": -1}.get(text[i], 0)
            i += 1
        yield " ".join(text[m.end():i - 1].split())


@pytest.mark.parametrize("name", ["k_chunk.cu", "k_chunk_tc.cu", "k_weights.cu", "k_evict.cu", "k_append.cu"])
def test_the_read_only_path_is_for_descriptors(name):
    """These kernels are on the device before the one ahead of them has ended: what
    that one writes (partials, log-sums, weights) is not read-only for their whole
    life.  Items, requests and block tables are uploaded before the first of them."""
    descriptor = re.compile(r"reinterpret_cast<const int4\*>\(p\)( \+ 1)?|s( \+ \d)?|a\.bt \+ rq\.bt_off \+ .*")
    for arg in _arguments(_source(name), "__ldg"):
        assert descriptor.fullmatch(arg), arg


@pytest.mark.parametrize("name", _sources((".cu", ".cuh")))
def test_no_kernel_attribute_hangs_on_a_flag_of_the_process(name):
    """A kernel's shared memory limit is set per device: a flag that the first launch
    sets leaves it unset on every other device."""
    assert not re.search(r"static\s+bool", _source(name))


def test_evict_a_page_with_fewer_references_than_requests(eng):  # noqa: F811
    """Three requests that evict from one page of two references: each would drop one."""
    ctx, reqs = eng
    page = int(reqs[0].table[0])
    for req in reqs[1:]:
        gp.gp_page_unref(ctx, int(req.table[0]))
        req.table[0] = page
    gp.gp_page_ref(ctx, page)
    before = _state(ctx, reqs)
    assert _status(_evict, ctx, reqs, (512, 512, 512), (10, 10, 10)) == gp.GP_ERR_INVALID
    assert _status(_evict, ctx, reqs, (512, 512, 512), (10, 10, 512)) == gp.GP_ERR_STATE  # two of them evict
    assert _state(ctx, reqs) == before
    gp.gp_page_ref(ctx, page)
    assert _status(_evict, ctx, reqs, (512, 512, 512), (10, 10, 10)) == gp.GP_ERR_STATE


class Buffer:
    """A tensor on a device, as far as the binding looks at it."""
    is_cuda = True

    def __init__(self, count, dtype, device=0, address=1 << 20):
        self.count, self.dtype, self.device, self.address = count, dtype, device, address

    def is_contiguous(self):
        return True

    def numel(self):
        return self.count

    def get_device(self):
        return self.device

    def data_ptr(self):
        return self.address


def test_buffers_of_the_wrong_type_or_size(eng):  # noqa: F811
    """Every buffer of every call, one at a time: too few elements, another type."""
    torch = pytest.importorskip("torch")
    bf, f32, u8 = torch.bfloat16, torch.float32, torch.uint8
    ctx, reqs = eng  # 2 layers, 8 and 2 heads of 128, 6 slots, 4 pages a request, bf16
    weights = Buffer(2 * 6 * 2 * 4 * 256, f32)
    rows = 257
    far = 1 << 30
    calls = [
        (_append, dict(q=Buffer(rows * 1024, bf), k=Buffer(rows * 256, bf), v=Buffer(rows * 256, bf),
                       rot=Buffer(rows * 1024, bf, address=far), w=weights)),
        (_chunk, dict(q=Buffer(rows * 1024, bf), out=Buffer(rows * 1024, bf, address=far), w=weights)),
        (_decode, dict(q=Buffer(3 * 1024, bf), first=Buffer(3, u8), out=Buffer(3 * 1024, f32), w=weights)),
        (_evict, dict(w=weights)),
    ]
    for call, kw in calls:
        assert _status(call, ctx, reqs, **kw) == gp.GP_ERR_STATE  # up to the device check
        for name, b in kw.items():
            for bad in (Buffer(b.count - 1, b.dtype, address=b.address), Buffer(b.count, torch.float16, address=b.address),
                        Buffer(b.count, f32 if b.dtype is bf else bf, address=b.address)):
                assert _status(call, ctx, reqs, **dict(kw, **{name: bad})) == gp.GP_ERR_INVALID, (call, name)
            more = Buffer(b.count + 1, b.dtype, address=b.address)  # rows behind the last are left alone; weights have one shape
            assert _status(call, ctx, reqs, **dict(kw, **{name: more})) == (
                gp.GP_ERR_INVALID if name == "w" else gp.GP_ERR_STATE), (call, name)
    ctx.buffers.device = 1
    assert _status(_evict, ctx, reqs, w=weights) == gp.GP_ERR_INVALID
    ctx.buffers.device = 0
    assert _status(_evict, ctx, reqs, w=weights) == gp.GP_ERR_STATE
    assert _status(_decode, ctx, reqs, **dict(calls[2][1], first=Buffer(3, torch.bool))) == gp.GP_ERR_STATE
    bare = type(ctx)(ctx.value)  # the context's address alone: its shape is not known
    assert _status(_evict, bare, reqs, w=Buffer(1, bf)) == gp.GP_ERR_STATE


def test_counts_that_32_bits_do_not_hold(eng):  # noqa: F811
    """A count of 64 bits is not cut to its lower half, nor a fraction to a whole number."""
    ctx, reqs = eng
    far = 2 ** 32 + 1  # the lower half is 1
    for bad in ([1, 1, far], (1, 1, far), np.array([1, 1, far]), np.array([1, 1, -far]), [1, 1, 1.5], np.array([1, 1, 1.5])):
        assert _status(_append, ctx, reqs, (0, 0, 0), bad) == gp.GP_ERR_INVALID
        assert _status(_append, ctx, reqs, bad, (0, 0, 0)) == gp.GP_ERR_INVALID
        assert _status(_decode, ctx, reqs, bad) == gp.GP_ERR_INVALID
        assert _status(_evict, ctx, reqs, (2, 2, 2), bad) == gp.GP_ERR_INVALID
    for good in ([1, 1, 1], np.array([1, 1, 1]), np.array([1, 1, 1], dtype=np.uint8), np.array([1, 9, 1, 9, 1, 9], dtype=np.int32)[::2]):
        assert _status(_append, ctx, reqs, (0, 0, 0), good) == gp.GP_ERR_STATE
        assert _status(_evict, ctx, reqs, (2, 2, 2), good) == gp.GP_ERR_STATE


def test_the_demand_scan_sets_its_shared_memory_limit_on_every_device():
    body = _source("k_demand_tc.cu").split("size_t prepare_t()")[1].split("\n}\n")[0]
    assert "allow_shared<" in body and not re.search(r"if \(\w+\) return", body)
