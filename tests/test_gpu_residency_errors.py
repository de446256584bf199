"""The residency update where one unit reports an error: every other unit is done, or left as it was, as a whole."""
import numpy as np
import pytest

import dd_testlib as tl
import oracle

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


def test_a_bad_slot_in_one_of_many_units(dd):
    """Several times as many units as fit the GPU at once; the first one's union names a slot of another."""
    B, H, C, cs, S, cap, umax = 300, 8, 12, 16, 5, 3, 6
    units = B * H
    rng = np.random.default_rng(8)
    rs = np.full((units, C), -1, np.int32)
    sc = np.full((units, S), -1, np.int32)
    lu = np.full((units, S), -1, np.int32)
    idx, slot = (np.zeros((units, umax), np.int32) for _ in range(2))
    cnt = np.full(units, umax, np.int32)
    m = 0
    for u in range(units):
        held = rng.choice(C, 4, replace=False)
        sc[u, :4], lu[u, :4] = held, rng.integers(0, 9, 4)
        rs[u, held] = u * S + np.arange(4)
        idx[u] = np.sort(rng.choice(C, umax, replace=False))
        for i, c in enumerate(idx[u]):
            if rs[u, c] >= 0:
                slot[u, i] = rs[u, c]
            else:
                slot[u, i], m = -1 - m, m + 1
    Kst, Vst = (rng.integers(0, 1 << 15, (m, cs, 128)).astype(np.uint16) for _ in range(2))
    pools = [np.zeros((units * S, cs, 128), np.uint16) for _ in range(2)]
    shape = lambda a: a.reshape(B, H, -1)
    want = oracle.update_residency(9, cap, shape(idx), shape(slot), cnt.reshape(B, H), Kst, Vst, shape(rs), shape(sc), shape(lu), *pools)
    bad = slot.copy()
    bad[0, 0] = units * S - 1
    d = {k: tl.to_i32(v) for k, v in dict(idx=idx, slot=bad, cnt=cnt, m=np.array([m])).items()}
    k, v = tl.to_bf16(Kst), tl.to_bf16(Vst)
    before = dict(resident_slot=rs, slot_chunk=sc, last_used=lu, admitted=np.full(units, -7, np.int32))
    with dd.Context(dd.Shape(B, H, H, 128, C * cs, cs, umax, 1), max_misses=m, hot_slots=units * S) as ctx:
        for _ in range(5):
            t = {n: tl.to_i32(a) for n, a in before.items()}
            Kh, Vh = (tl.to_bf16(p) for p in pools)
            ctx.update_residency(9, cap, S, k, v, t["resident_slot"], t["slot_chunk"], t["last_used"], Kh, Vh, admitted=t["admitted"],
                                 union_idx=d["idx"], union_slot=d["slot"], union_cnt=d["cnt"], miss_count=d["m"])
            assert ctx.status() == dd.DD_ERR_DEVICE_CHECK
            got = {n: a.cpu().numpy().reshape(before[n].shape) for n, a in t.items()}
            done = got["admitted"] != -7
            assert done[0] and (done | (got["admitted"] == -7)).all()
            for n in before:
                ref = np.asarray(want[n]).reshape(before[n].shape)
                assert np.array_equal(got[n][1:][done[1:]], ref[1:][done[1:]]), n
                assert np.array_equal(got[n][~done], before[n][~done]), n
            for a, n in ((Kh, "Khot"), (Vh, "Vhot")):
                a = tl.from_bf16(a).reshape(units, -1)
                assert np.array_equal(a[1:][done[1:]], np.asarray(want[n]).reshape(units, -1)[1:][done[1:]])
                assert not a[~done].any()
