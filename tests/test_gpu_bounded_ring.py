"""A ring of copies that never arrive: one wait runs out, not one for every tile."""
import time

import pytest

pytestmark = pytest.mark.gpu


def test_the_first_wait_that_runs_out_is_the_last():
    import torch
    from sparse_kv_offload_gb300 import build
    build.build()
    from sparse_kv_offload_gb300 import dd
    with dd.Context(dd.Shape(1, 1, 1, 128, 64, 16, 1, 1), max_misses=0) as ctx:
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        ctx.selftest_bounded_wait(2)
        assert ctx.status() == dd.DD_ERR_TIMEOUT
        took = time.perf_counter() - t0
        assert 2.0 < took < 12.0                       # 64 tiles: one wait of 2 s and one for the copies behind it
        assert ctx.status() == 0                       # read and cleared
        for kind in (-1, 3):
            with pytest.raises(dd.DDError):
                ctx.selftest_bounded_wait(kind)
