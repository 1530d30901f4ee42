"""The accumulated-weight calls where they once went wrong: precision of the
softmax weights, evictions at the same time, records kept from call to call,
lengths and sizes at their ends.  The engine, the formulas in 64 bits and the
arithmetic behind the tolerances are test_gpu_weighted.py's."""

import math
import threading

import pytest
import torch

import paged_kv_cache_step_gb300 as gp
from test_gpu_weighted import EPS, Engine, bits, check_chunk, kept_slots, softmax_reference

pytestmark = pytest.mark.gpu


# One pair of query tiles, one tile whose keys two groups share, a long cache cut
# into parts and joined.
@pytest.mark.parametrize("cached,new", [([300, 0], [130, 260]), ([100, 640], [5, 33]), ([6000], [3])])
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (4, 2, 128), (4, 1, 64), (4, 2, 64)])
def test_chunk_weights_keep_their_bits_for_the_values(cached, new, hq, hkv, d):
    """Values of either sign that nearly cancel: an output's error shows what the
    softmax weights were rounded to.  They are held to 2^-15 (two bf16 parts, the
    first cut off, 2^-7, the second rounded, 2^-8), beside the logits' error and
    the sum's; a single bf16 part is off by up to 2^-8."""
    e = Engine([-(-(a + b) // 256) for a, b in zip(cached, new)], L=1, hq=hq, hkv=hkv, d=d, seed=61)
    try:
        e.fill([a + b for a, b in zip(cached, new)])
        for r, (a, b) in enumerate(zip(cached, new)):
            pages, slots = e.at(r, torch.arange(a + b, device="cuda"))
            sign = (1 - 2 * (torch.arange(a + b, device="cuda") % 2))[:, None, None]
            e.v[0, pages, :, slots] = (sign * (1 + torch.arange(d, device="cuda") / d)).to(e.v.dtype).expand(-1, hkv, -1)
        q = (e.randn(sum(new), hq, d) / 32).bfloat16()  # logits of about 1/32
        out = torch.full_like(q, math.nan)
        gp.gp_chunk_attention(e.ctx, 0, e.reqs, cached, new, q, out, None)
        gp.gp_synchronize(e.ctx)
        at, worst = 0, 0.0
        for r, (c, m) in enumerate(zip(cached, new)):
            for h in range(hkv):
                heads = slice(h * e.G, h * e.G + e.G)
                ref, mag, _, rel = softmax_reference(q[at:at + m, heads].double(), e.rows(e.k, r, 0, h, c + m),
                                                     e.rows(e.v, r, 0, h, c + m), c)
                tol = (2 * rel + 2.0 ** -15) * mag
                tol = tol + EPS["bf16"] * (ref.abs() + tol)
                worst = max(worst, ((out[at:at + m, heads].double() - ref).abs() / tol).max().item())
            at += m
        assert worst <= 1.0, worst
    finally:
        e.close()


def test_evictions_of_two_threads():
    """Two contexts, a host thread each, evict requests of very different lengths at
    the same time: the limit of shared memory of the selection is one for both."""
    lengths, errors = [30000, 300], []
    engines = [Engine([-(-T // 256)], L=1, hq=2, hkv=1, d=64, seed=62, stream=torch.cuda.Stream()) for T in lengths]
    together = threading.Barrier(2)

    def work(e, T):
        try:
            together.wait()
            for _ in range(600):
                gp.gp_evict_weighted(e.ctx, e.reqs, [T], [T - 1], e.w)
            gp.gp_synchronize(e.ctx)
        except gp.GrowPageError as err:
            errors.append(str(err))

    try:
        for e, T in zip(engines, lengths):
            e.fill([T])
        torch.cuda.synchronize()
        threads = [threading.Thread(target=work, args=x) for x in zip(engines, lengths)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        assert not errors
    finally:
        for e in engines:
            e.close()


def test_descriptors_that_grow_while_calls_are_in_flight():
    """Calls of few and of many requests in turn, the first ones still waiting on the
    device when the descriptors' memory grows: the same bits as one call at a time."""
    n, results = 70, []
    for held in (False, True):
        e = Engine([1] * n, L=1, hq=2, hkv=1, d=64, seed=63, cap=256)
        try:
            e.fill([200] * n)
            q = e.randn(n, 2, 64).bfloat16()
            outs = []
            torch.cuda.synchronize()
            if held:
                torch.cuda._sleep(50_000_000)
            for i, m in enumerate([2, 3, 1, n, 5, n, 2, n - 1, 4, 1, n, 3]):
                outs.append(torch.zeros(n, 2, 64, dtype=torch.bfloat16, device="cuda"))
                gp.gp_chunk_attention(e.ctx, 0, e.reqs[:m], [199 - i] * m, [1] * m, q, outs[-1], e.w)
                if not held:
                    gp.gp_synchronize(e.ctx)
            gp.gp_synchronize(e.ctx)
            results.append((torch.stack(outs), e.w.clone()))
        finally:
            e.close()
    for a, b in zip(*results):
        assert torch.equal(bits(a), bits(b))


@pytest.mark.parametrize("hq,hkv,d", [(16, 4, 128), (8, 4, 64)])
@pytest.mark.parametrize("kernel", [gp.GP_KERNEL_CHUNK, gp.GP_KERNEL_WEIGHTS])
def test_chunk_waits_that_give_up_are_reported(kernel, hq, hkv, d):
    """Pairs of query tiles, single ones and joins, more tiles a CTA than its buffers
    hold.  Without patience every CTA stops with copies and products in flight; with
    a little some may.  The next call is right."""
    cached, new = [20000, 0, 52000], [900, 300, 3]
    e = Engine([82, 2, 204], L=1, hq=hq, hkv=hkv, d=d, seed=64)
    try:
        e.fill([a + b for a, b in zip(cached, new)])
        q = e.randn(sum(new), hq, d).bfloat16()
        out = torch.empty_like(q)
        for limit in (0, 1, 300, 3000, 30000, 0):
            gp.gp_debug_set_wait_limit(e.ctx, kernel, limit)
            gp.gp_chunk_attention(e.ctx, 0, e.reqs, cached, new, q, out, e.w.clone())
            try:
                gp.gp_synchronize(e.ctx)
                assert limit > 0
            except gp.GrowPageError as err:
                assert err.status == gp.GP_ERR_TIMEOUT
        gp.gp_debug_set_wait_limit(e.ctx, kernel, -1)
        w = e.w.clone()
        gp.gp_chunk_attention(e.ctx, 0, e.reqs, cached, new, q, out, w)
        gp.gp_synchronize(e.ctx)
        check_chunk(e, 0, cached, new, q, out, e.w, w, True)
    finally:
        e.close()


def test_only_accepted_drafted_tokens_are_counted():
    """Drafted tokens attend without weights; the accepted ones' are added by a second
    call over them, and the next append takes the rejected ones' slots."""
    cached, drafted, accepted = [700, 255, 40], [5, 6, 3], [2, 6, 0]
    e = Engine([3, 2, 1], L=1, seed=65)
    try:
        e.fill(cached)
        x = [e.randn(sum(drafted), h, 128).bfloat16() for h in (8, 2, 2)]
        for r, req in enumerate(e.reqs):
            req.pos = cached[r]
        rot = torch.empty_like(x[0])
        gp.gp_append_tokens(e.ctx, 0, e.reqs, cached, drafted, *x, rot, e.w)
        before, out = e.w.clone(), torch.empty_like(rot)
        gp.gp_chunk_attention(e.ctx, 0, e.reqs, cached, drafted, rot, out, None)
        gp.gp_synchronize(e.ctx)
        assert torch.equal(bits(e.w), bits(before))
        taken = torch.cat([torch.arange(sum(drafted[:r]), sum(drafted[:r]) + a) for r, a in enumerate(accepted)]).cuda()
        q, again = rot[taken].contiguous(), torch.empty_like(rot[taken])
        gp.gp_chunk_attention(e.ctx, 0, e.reqs, cached, accepted, q, again, e.w)
        gp.gp_synchronize(e.ctx)
        check_chunk(e, 0, cached, accepted, q, again, before, e.w, True)
        now = [c + a for c, a in zip(cached, accepted)]
        gp.gp_append_tokens(e.ctx, 0, e.reqs, now, [1] * 3, None, x[1][:3], x[2][:3], None, e.w)
        gp.gp_synchronize(e.ctx)
        for r, t in enumerate(now):
            assert not e.w[0, r, :, t].any() and torch.equal(e.rows(e.v, r, 0, 1, t + 1)[t], x[2][r, 1].double())
    finally:
        e.close()


@pytest.mark.parametrize("side", [False, True])
def test_emptied_pages_go_to_another_request(side):
    """After an eviction its emptied pages are given back and taken by a request that
    appends to them at once, while the eviction may not have read them yet."""
    e = Engine([8, 1], seed=66, spare=1, cap=8)
    stream = torch.cuda.Stream()
    try:
        T, keep = 2000, 300
        old, new = e.reqs
        prefix = old.pages[7]  # a shared page past the budget: replaced, and the fresh one given back
        e.fill([T + 1, 0])
        # the kernels' first launches load them, which may wait for the device
        gp.gp_evict_weighted(e.ctx, [old], [T + 1], [T], e.w)
        gp.gp_append_tokens(e.ctx, 0, [new], [0], [1], None, e.randn(1, 2, 128).bfloat16(), e.randn(1, 2, 128).bfloat16(), None, None)
        gp.gp_synchronize(e.ctx)
        gp.gp_page_ref(e.ctx, prefix)
        k0, v0, w0, t0 = e.k.clone(), e.v.clone(), e.w.clone(), [x.pages for x in e.reqs]
        rows = [e.randn(1000, 2, 128).bfloat16() for _ in range(2)]
        if side:
            gp.gp_set_compaction_stream(e.ctx, stream)
        torch.cuda.synchronize()
        if side:
            with torch.cuda.stream(stream):
                torch.cuda._sleep(50_000_000)
        gp.gp_evict_weighted(e.ctx, [old], [T], [keep], e.w)
        assert prefix not in old.pages and gp.gp_page_refcount(e.ctx, prefix) == 1
        for page in old.pages[2:]:
            gp.gp_page_unref(e.ctx, page)
        old.num_pages = 2
        taken = [gp.gp_page_alloc(e.ctx) for _ in range(3)]
        assert len(set(taken) & set(t0[0])) >= 2  # pages that the eviction reads
        new.table[1:4] = taken
        new.num_pages = 4
        for layer in range(2):
            gp.gp_append_tokens(e.ctx, layer, [new], [0], [1000], None, *rows, None, e.w)
        gp.gp_wait_compaction(e.ctx)
        gp.gp_synchronize(e.ctx)
        torch.cuda.synchronize()
        for layer in range(2):
            for h in range(2):
                assert torch.equal(e.rows(e.v, 1, layer, h, 1000), rows[1][:, h].double())
                idx = torch.as_tensor(kept_slots(w0[layer, 0, h].cpu().numpy(), T, keep, e.recent), device="cuda")
                src = torch.as_tensor(t0[0], device="cuda")[idx // 256]
                for cache, was in ((e.k, k0), (e.v, v0)):
                    assert torch.equal(e.rows(cache, 0, layer, h, keep), was[layer, src, h, idx % 256].double())
                assert torch.equal(e.w[layer, 0, h, :keep], w0[layer, 0, h, idx])
    finally:
        gp.gp_set_compaction_stream(e.ctx, None)
        e.close()


def test_decode_attention_is_refused_while_the_stream_is_captured():
    """A replay would read its tables from memory that later calls have written."""
    stream = torch.cuda.Stream()
    e = Engine([2], L=1, seed=67, stream=stream)
    try:
        e.fill([300])
        q, out = e.randn(1, 8, 128).bfloat16(), torch.zeros(1, 8, 128, device="cuda")
        first, x = torch.ones(1, dtype=torch.uint8, device="cuda"), torch.ones(8, device="cuda")
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            x.mul_(2)
            with pytest.raises(gp.GrowPageError) as err:
                gp.gp_decode_attention(e.ctx, 0, e.reqs, [300], q, first, out)
        assert err.value.status == gp.GP_ERR_UNSUPPORTED
        graph.replay()
        torch.cuda.synchronize()
        assert x[0] == 2 and not out.any()
        for _ in range(10):  # and the context works on, whichever slot a call takes
            gp.gp_decode_attention(e.ctx, 0, e.reqs, [300], q, first, out)
        gp.gp_synchronize(e.ctx)
        assert out.any()
    finally:
        e.close()
