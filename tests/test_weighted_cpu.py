"""What the accumulated-weight calls refuse, on a host-only context: every bad
argument is GP_ERR_INVALID before anything else is looked at, good ones reach
the device check (GP_ERR_STATE without a device), and neither changes the
pool, the tables or the slots."""

import numpy as np
import pytest

import paged_kv_cache_step_gb300 as gp

PAGE = 256
DEV = 1 << 20  # stands for a device address, 16-byte aligned; never followed


@pytest.fixture
def eng():
    cfg = gp.gp_config_default(num_layers=2, num_q_heads=8, num_kv_heads=2, head_dim=128, max_slots=6, num_pages=16,
                               max_pages_per_req=4)
    ctx = gp.gp_create(cfg)
    reqs = []
    for _ in range(3):
        pages = [gp.gp_page_alloc(ctx) for _ in range(2)]
        reqs.append(gp.Request(gp.gp_slot_acquire(ctx), pages, 100, 4))
    yield ctx, reqs
    gp.gp_destroy(ctx)


def _append(ctx, reqs, cached=(0, 5, 256), new=(1, 0, 256), layer=0, q=DEV, k=DEV, v=DEV, rot=DEV, w=DEV):
    gp.gp_append_tokens(ctx, layer, reqs, cached, new, q, k, v, rot, w)


def _chunk(ctx, reqs, cached=(0, 5, 256), new=(1, 0, 256), layer=0, q=DEV, out=DEV << 4, w=DEV):
    gp.gp_chunk_attention(ctx, layer, reqs, cached, new, q, out, w)


def _decode(ctx, reqs, tokens=(0, 5, 512), layer=0, q=DEV, first=None, out=DEV, w=DEV):
    gp.gp_decode_attention_weighted(ctx, layer, reqs, tokens, q, first, out, w)


def _evict(ctx, reqs, tokens=(0, 5, 512), keep=(1, 7, 300), w=DEV):
    gp.gp_evict_weighted(ctx, reqs, tokens, keep, w)


def _status(call, *a, **kw):
    with pytest.raises(gp.GrowPageError) as e:
        call(*a, **kw)
    return e.value.status


def _state(ctx, reqs):
    return ([(r.slot, r.num_pages, r.pages) for r in reqs], gp.gp_free_page_count(ctx),
            [gp.gp_page_refcount(ctx, p) for p in range(16)])


@pytest.mark.parametrize("call", [_append, _chunk, _decode, _evict])
def test_good_arguments_reach_the_device_check(eng, call):
    ctx, reqs = eng
    before = _state(ctx, reqs)
    assert _status(call, ctx, reqs) == gp.GP_ERR_STATE
    assert _status(call, ctx, [], *[[]] * 2 if call is not _decode else [[]]) == gp.GP_ERR_STATE
    assert _state(ctx, reqs) == before


@pytest.mark.parametrize("call", [_append, _chunk, _decode, _evict])
def test_bad_requests(eng, call):
    ctx, reqs = eng
    before = _state(ctx, reqs)
    other = gp.Request(5, reqs[0].pages, 0, 4)
    for bad in (gp.Request(5, [0, 1], 0, 4),                    # slot not bound
                gp.Request(-1, [0, 1], 0, 4), gp.Request(6, [0, 1], 0, 4),
                gp.Request(reqs[0].slot, [], 0, 4),             # no pages
                gp.Request(reqs[0].slot, [0, 99], 0, 4),        # page out of range
                gp.Request(reqs[0].slot, [0, -1], 0, 4),
                gp.Request(reqs[0].slot, [0, 15], 0, 4),        # page not allocated
                gp.Request(reqs[0].slot, [0, 0], 0, 4),         # page twice
                gp.Request(reqs[0].slot, [0, 1], -1, 4),        # negative position
                other):
        assert _status(call, ctx, [bad] + reqs[1:]) == gp.GP_ERR_INVALID
    twice = gp.Request(reqs[0].slot, reqs[1].pages, 0, 4)
    assert _status(call, ctx, [reqs[0], twice, reqs[2]]) == gp.GP_ERR_INVALID  # slot twice
    assert _state(ctx, reqs) == before


@pytest.mark.parametrize("call", [_append, _chunk])
def test_new_tokens_outside_the_pages(eng, call):
    ctx, reqs = eng
    for cached, new in (((-1, 0, 0), (1, 1, 1)), ((0, 0, 0), (1, -1, 1)), ((0, 0, 512), (1, 1, 1)),
                        ((0, 0, 1), (1, 1, 512)), ((2 ** 31 - 1, 0, 0), (1, 1, 1)), ((0, 0, 0), (2 ** 31 - 1, 1, 1))):
        assert _status(call, ctx, reqs, cached, new) == gp.GP_ERR_INVALID
    assert _status(call, ctx, reqs, (0, 0), (1, 1)) == gp.GP_ERR_INVALID  # a count for every request
    for layer in (-1, 2):
        assert _status(call, ctx, reqs, layer=layer) == gp.GP_ERR_INVALID


def test_append_pointers_and_shared_pages(eng):
    ctx, reqs = eng
    for kw in (dict(k=None), dict(v=None), dict(q=None), dict(rot=None), dict(q=DEV + 2), dict(k=DEV + 8),
               dict(v=DEV + 4), dict(rot=DEV + 8), dict(rot=DEV + 16), dict(q=DEV + 16), dict(w=DEV + 2)):
        assert _status(_append, ctx, reqs, **kw) == gp.GP_ERR_INVALID
    assert _status(_append, ctx, reqs, q=None, rot=None) == gp.GP_ERR_STATE
    assert _status(_append, ctx, reqs, w=None) == gp.GP_ERR_STATE
    # a page that two requests hold is not written; beside the written ones it may be shared
    gp.gp_page_ref(ctx, reqs[0].pages[1])
    assert _status(_append, ctx, reqs, (200, 0, 0), (100, 0, 0)) == gp.GP_ERR_INVALID
    assert _status(_append, ctx, reqs, (200, 0, 0), (56, 0, 0)) == gp.GP_ERR_STATE
    # a page with one reference in two tables is written by one request at most
    twin = gp.Request(reqs[1].slot, [reqs[0].pages[0], reqs[1].pages[1]], 0, 4)
    assert _status(_append, ctx, [reqs[0], twin], (0, 0), (1, 1)) == gp.GP_ERR_INVALID
    assert _status(_append, ctx, [reqs[0], twin], (0, 256), (1, 1)) == gp.GP_ERR_STATE


def test_attention_pointers_and_lengths(eng):
    ctx, reqs = eng
    bytes_ = 257 * 8 * 128 * 2  # rows x heads x d, bf16
    far = DEV + 2 * bytes_
    for kw in (dict(q=None), dict(out=None), dict(q=DEV + 8), dict(out=far + 4), dict(out=DEV), dict(w=DEV + 2),
               dict(out=DEV + bytes_ - 16), dict(q=DEV + bytes_ - 16, out=DEV)):
        assert _status(_chunk, ctx, reqs, **dict(dict(out=far), **kw)) == gp.GP_ERR_INVALID
    assert _status(_chunk, ctx, reqs, out=DEV + bytes_) == gp.GP_ERR_STATE
    assert _status(_chunk, ctx, reqs, w=None) == gp.GP_ERR_STATE
    for kw in (dict(q=None), dict(out=None), dict(w=None), dict(w=DEV + 1), dict(tokens=(0, -1, 0)), dict(tokens=(0, 513, 0)),
               dict(layer=2), dict(layer=-1)):
        assert _status(_decode, ctx, reqs, **kw) == gp.GP_ERR_INVALID


def test_evict_lengths(eng):
    ctx, reqs = eng
    for kw in (dict(w=None), dict(w=DEV + 2), dict(tokens=(0, -1, 0)), dict(tokens=(0, 0, 513)), dict(keep=(0, 1, 1)),
               dict(keep=(-5, 1, 1))):
        assert _status(_evict, ctx, reqs, **kw) == gp.GP_ERR_INVALID
    assert _status(_evict, ctx, reqs, (1, 2), (1, 2)) == gp.GP_ERR_INVALID


def test_evict_a_page_of_two_requests(eng):
    ctx, reqs = eng
    own, page = int(reqs[1].table[1]), int(reqs[0].table[0])
    reqs[1].table[1] = page  # without a reference of its own
    assert _status(_evict, ctx, reqs, (512, 512, 0), (10, 10, 1)) == gp.GP_ERR_INVALID
    assert _status(_evict, ctx, reqs, (512, 512, 0), (10, 512, 1)) == gp.GP_ERR_STATE  # one of them evicts
    gp.gp_page_ref(ctx, page)
    gp.gp_page_unref(ctx, own)
    assert _status(_evict, ctx, reqs, (512, 512, 0), (10, 10, 1)) == gp.GP_ERR_STATE  # shared: both copy it


def test_buffers_on_the_host(eng):
    torch = pytest.importorskip("torch")
    ctx, reqs = eng
    for host in (torch.zeros(4, 4), torch.zeros(4, 4).t(), np.zeros((4, 4), dtype=np.float32)):
        for name in ("q", "k", "v", "rot", "w"):
            assert _status(_append, ctx, reqs, **{name: host}) == gp.GP_ERR_INVALID
        for name in ("q", "out", "w"):
            assert _status(_chunk, ctx, reqs, **{name: host}) == gp.GP_ERR_INVALID
            assert _status(_decode, ctx, reqs, **{name: host}) == gp.GP_ERR_INVALID
        assert _status(_decode, ctx, reqs, first=host) == gp.GP_ERR_INVALID
        assert _status(_evict, ctx, reqs, w=host) == gp.GP_ERR_INVALID


def test_null_context():
    lib = gp.load()
    n = np.zeros(1, dtype=np.int32)
    assert lib.gp_append_tokens(None, 0, 0, None, n.ctypes.data, n.ctypes.data, None, None, None, None, None) == 1
    assert lib.gp_chunk_attention(None, 0, 0, None, n.ctypes.data, n.ctypes.data, None, None, None) == 1
    assert lib.gp_decode_attention_weighted(None, 0, 0, None, n.ctypes.data, None, None, None, None) == 1
    assert lib.gp_evict_weighted(None, 0, None, n.ctypes.data, n.ctypes.data, None) == 1
