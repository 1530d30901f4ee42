"""What the calls over a step's device arrays take and refuse on the host, beside
test_sparse_cpu.py."""

import pytest

import paged_kv_cache_step_gb300 as gp


def test_waits_of_sparse_attention_have_a_limit():
    ctx = gp.gp_create(gp.gp_config_default(num_layers=1, num_q_heads=8, num_kv_heads=2, head_dim=128, max_slots=2, num_pages=4,
                                            max_pages_per_req=4))
    try:
        for limit in (0, 300, -1):
            gp.gp_debug_set_wait_limit(ctx, gp.GP_KERNEL_SPARSE, limit)
        for other in (gp.GP_KERNEL_TABLES, gp.GP_KERNEL_MAPPED, gp.GP_KERNEL_BOUNDS, gp.GP_KERNEL_BLOCK_SELECT):
            with pytest.raises(gp.GrowPageError) as err:
                gp.gp_debug_set_wait_limit(ctx, other, 0)
            assert err.value.status == gp.GP_ERR_UNSUPPORTED
    finally:
        gp.gp_destroy(ctx)
