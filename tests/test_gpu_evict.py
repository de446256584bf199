"""Eviction by gathered weight against the oracle: every output equal."""
import numpy as np
import pytest

import oracle

pytestmark = pytest.mark.gpu

OUT = ("resident_out", "slot_chunk", "last_used", "evicted", "evicted_cnt", "union_idx", "union_slot", "union_cnt")


@pytest.fixture(scope="module")
def dd():
    import torch
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from sparse_kv_offload_gb300 import build
    build.build()
    from sparse_kv_offload_gb300 import dd as mod
    return mod


def make(seed, B, H, C, cs, S, keep, ties=0.3, new=True, full=0.7):
    rng = np.random.default_rng(seed)
    L = C * cs
    n = rng.integers(0, min(L, 3 * cs) + 1, B) if new else np.zeros(B, int)
    kv = np.array([rng.integers(0, L - n[b] + 1) for b in range(B)])
    slot = np.full((B, H, C), -1, np.int32)
    for b in range(B):
        for h in range(H):
            have = -(-kv[b] // cs)
            r = min(have, S, int(round(full * S)) if rng.random() < 0.8 else S)
            c = rng.choice(have, r, replace=False) if r else []
            slot[b, h, c] = (b * H + h) * S + rng.permutation(S)[:r]
    w = rng.exponential(1.0, (B, H, C)).astype(np.float32)
    w[rng.random(w.shape) < ties] = 0.0
    w[rng.random(w.shape) < 0.05] = -0.0
    return dict(B=B, H=H, C=C, cs=cs, S=S, keep=keep, kv=kv.astype(np.int32), n=n.astype(np.int32), slot=slot, w=w)


def want_of(x, first, last, before):
    B, H, C, cs, S = x["B"], x["H"], x["C"], x["cs"], x["S"]
    r = {k: v.copy() for k, v in before.items()}
    short = False
    for b in range(B):
        n0, n1 = -(-int(x["kv"][b]) // cs), -(-int(x["kv"][b] + x["n"][b]) // cs)
        for h in range(H):
            base = (b * H + h) * S
            now, gone, out = oracle.evict_unit(x["w"][b, h], x["slot"][b, h], base, S, n0, n1, x["keep"], first, last)
            short |= out
            stay = np.flatnonzero(now >= 0)
            r["resident_out"][b, h] = now
            r["slot_chunk"][b, h] = -1
            r["slot_chunk"][b, h, now[stay] - base] = stay
            fresh = [c for c in stay if x["slot"][b, h, c] < 0]
            r["last_used"][b, h, r["slot_chunk"][b, h] < 0] = -1
            r["last_used"][b, h, now[fresh] - base] = 77
            r["evicted"][b, h, :len(gone)] = gone
            r["evicted_cnt"][b, h] = len(gone)
            r["union_idx"][b, h, :len(stay)] = stay
            r["union_slot"][b, h, :len(stay)] = now[stay]
            r["union_cnt"][b, h] = len(stay)
    return r, short


def buffers(x, umax):
    B, H, C, S = x["B"], x["H"], x["C"], x["S"]
    rng = np.random.default_rng(5)
    shapes = dict(resident_out=(B, H, C), slot_chunk=(B, H, S), last_used=(B, H, S), evicted=(B, H, S), evicted_cnt=(B, H),
                  union_idx=(B, H, umax), union_slot=(B, H, umax), union_cnt=(B, H))
    return {k: rng.integers(1000, 2000, s).astype(np.int32) for k, s in shapes.items()}


def run(dd, x, first, last, before, k=None, in_place=False, optional=True):
    import torch
    B, H, C, S = x["B"], x["H"], x["C"], x["S"]
    t = {n: torch.from_numpy(v).cuda() for n, v in before.items()}
    with dd.Context(dd.Shape(B, H, H, 128, C * x["cs"], x["cs"], k or min(C, max(S, 1)), 1), 0, B * H * S) as ctx:
        slot = torch.from_numpy(x["slot"]).cuda()
        if in_place:
            t["resident_out"] = slot
        rest = {n: t[n] for n in OUT[1:]} if optional else {}
        ctx.evict_chunks(torch.from_numpy(x["w"]).cuda(), torch.from_numpy(x["kv"]).cuda(), slot, t["resident_out"],
                         x["keep"], S, first=first, last=last, new_len=torch.from_numpy(x["n"]).cuda(), step=77, **rest)
        status = ctx.status()
    return {n: v.cpu().numpy() for n, v in t.items()}, status


# B, H, C, cs, S, keep, first, last
SHAPES = {
    "one_chunk": (1, 1, 1, 16, 1, 1, 0, 0),
    "keep_nothing": (2, 2, 9, 16, 7, 0, 0, 0),
    "small": (2, 3, 40, 32, 20, 12, 1, 2),
    "protected_more_than_kept": (2, 2, 50, 16, 30, 4, 6, 8),
    "odd_sizes": (3, 2, 333, 16, 77, 50, 2, 5),
    "all_fits": (2, 2, 100, 64, 100, 100, 0, 0),
    "pool_as_large_as_the_cache": (1, 2, 1000, 16, 1000, 100, 4, 16),
    "largest": (1, 2, 16384, 16, 16384, 2000, 4, 64),
    "many_units": (40, 8, 130, 16, 64, 40, 1, 1),
}


@pytest.mark.parametrize("name", list(SHAPES))
@pytest.mark.parametrize("in_place", [False, True])
def test_evict(dd, name, in_place):
    B, H, C, cs, S, keep, first, last = SHAPES[name]
    x = make(3, B, H, C, cs, S, keep)
    umax = min(C, S)
    before = buffers(x, umax)
    got, status = run(dd, x, first, last, before, in_place=in_place)
    want, short = want_of(x, first, last, before)
    for n in OUT:
        assert np.array_equal(got[n], want[n]), n
    assert status == (dd.DD_ERR_CAPACITY if short else 0)
