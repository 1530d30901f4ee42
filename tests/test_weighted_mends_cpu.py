"""Faults of the accumulated-weight calls that need no device to show: what the
sources must not do, and what the calls and the binding refuse."""

import os
import re

import pytest

import paged_kv_cache_step_gb300 as gp
from test_weighted_cpu import _evict, _state, _status, eng  # noqa: F401 (a fixture)

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
