"""What earlier tests of the calls over a step's device arrays do not show: not-a-number
queries, in every kernel."""

import math

import numpy as np
import pytest
import torch

import paged_kv_cache_step_gb300 as gp
from test_gpu_sparse import DT, SHAPES, Engine, attention_reference, i32, kernels

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
