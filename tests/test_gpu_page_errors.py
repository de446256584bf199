"""Errors that one (request, KV head) of a call reports: what it leaves out, and that all others are done."""
import numpy as np
import pytest

import test_gpu_evict as te

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dd():
    import torch
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from sparse_kv_offload_gb300 import build
    build.build()
    from sparse_kv_offload_gb300 import dd as mod
    return mod


@pytest.mark.parametrize("C", [2048, 8193])
@pytest.mark.parametrize("what", ["short", "twice", "outside", "length"])
def test_eviction_of_the_other_units(dd, what, C):
    """Several times as many units as fit the GPU at once; the first of them are short of slots or not in order."""
    import torch
    B, H, cs, S, keep, first, last = 80, 8, 16, 16, 8, 0, 16
    x = te.make(31, B, H, C, cs, S, keep)
    if what == "short":
        # no chunk of the first request may leave
        x["kv"][0], x["n"][0] = C * cs // 2, 40
        x["slot"][0] = -1
        for h in range(H):
            x["slot"][0, h, C // 2 - S:C // 2] = h * S + np.arange(S)
    elif what == "length":
        x["kv"][0], x["n"][0] = C * cs, 1
    else:
        x["slot"][0] = -1
        for h in range(H):
            x["slot"][0, h, 5], x["slot"][0, h, 6] = h * S, h * S if what == "twice" else h * S + S
    before = te.buffers(x, S)
    y = dict(x, kv=x["kv"].copy(), slot=x["slot"].copy())  # of the requests that are in order
    if what != "short":
        y["kv"][0], y["slot"][0] = 0, -1
    want, short = te.want_of(y, first, last, before)
    if what != "short":
        # the first request stays as it was
        for n in te.OUT:
            want[n][0] = before[n][0]
        want["resident_out"][0] = x["slot"][0]
        want["evicted_cnt"][0] = want["union_cnt"][0] = 0
    inputs = [torch.from_numpy(x[n]).cuda() for n in ("w", "kv", "slot", "n")]
    with dd.Context(dd.Shape(B, H, H, 128, C * cs, cs, S, 1), 0, B * H * S) as ctx:
        def call():
            t = {n: torch.from_numpy(v).cuda() for n, v in before.items()}
            ctx.evict_chunks(*inputs[:3], t["resident_out"], keep, S, first=first, last=last, new_len=inputs[3], step=77,
                             **{n: t[n] for n in te.OUT[1:]})
            return t

        def equal(t, r):
            for n in te.OUT:
                assert np.array_equal(t[n].cpu().numpy(), r[n]), n
        for _ in range(3):
            got = call()
            idle = call()                                  # the error of the call before is pending
            equal(got, want)
            equal(idle, before)
            status = ctx.status()
            # (where both are reported the first one stands)
            assert status in ((dd.DD_ERR_CAPACITY,) if what == "short" else
                              (dd.DD_ERR_DEVICE_CHECK, dd.DD_ERR_CAPACITY) if short else (dd.DD_ERR_DEVICE_CHECK,))
        assert ctx.status() == 0
