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


def test_only_the_map(dd):
    """No optional output: the map alone."""
    x = make(9, 2, 2, 60, 16, 40, 20)
    before = buffers(x, 40)
    got, status = run(dd, x, 1, 2, before, optional=False)
    want, _ = want_of(x, 1, 2, before)
    assert status == 0 and np.array_equal(got["resident_out"], want["resident_out"])
    for n in OUT[1:]:
        assert np.array_equal(got[n], before[n]), n


@pytest.mark.parametrize("kind", ["equal", "nan", "inf", "negative", "tiny", "near"])
def test_weights_of_all_kinds(dd, kind):
    """Ties by chunk, NaN below every number, signs, subnormals, neighbours in the last bit."""
    x = make(11, 2, 2, 500, 16, 300, 100, ties=0.0)
    rng = np.random.default_rng(2)
    w = x["w"]
    if kind == "equal":
        w[:] = 1.5
    elif kind == "nan":
        w[rng.random(w.shape) < 0.4] = np.nan
        w[rng.random(w.shape) < 0.1] = -np.nan
    elif kind == "inf":
        w[rng.random(w.shape) < 0.4] = np.inf
        w[rng.random(w.shape) < 0.4] = -np.inf
    elif kind == "negative":
        w[:] = rng.standard_normal(w.shape).astype(np.float32)
        w[rng.random(w.shape) < 0.3] = -0.0
        w[rng.random(w.shape) < 0.3] = 0.0
    elif kind == "tiny":
        w[:] = (rng.integers(0, 40, w.shape) * 1.4e-45).astype(np.float32)
    else:
        w[:] = (np.float32(1.0).view(np.uint32) + rng.integers(0, 3, w.shape).astype(np.uint32)).view(np.float32)
    before = buffers(x, 300)
    got, status = run(dd, x, 3, 5, before)
    want, _ = want_of(x, 3, 5, before)
    for n in OUT:
        assert np.array_equal(got[n], want[n]), n
    assert status == 0


def test_lengths_from_nothing_to_all(dd):
    """Empty caches, full ones, chunks that are resident ahead of their rows, protected ranges that cover all."""
    x = make(12, 6, 1, 32, 16, 32, 8, ties=0.0)
    x["kv"][:] = [0, 1, 16, 17, 511, 512]
    x["n"][:] = [0, 15, 0, 495, 1, 0]
    x["slot"][:] = -1
    for b in range(6):
        x["slot"][b, 0, :20] = b * 32 + np.arange(20)        # (for the short ones: behind their rows)
    for first, last in ((0, 0), (32, 0), (0, 40), (5, 5)):
        before = buffers(x, 32)
        got, status = run(dd, x, first, last, before)
        want, short = want_of(x, first, last, before)
        for n in OUT:
            assert np.array_equal(got[n], want[n]), (n, first, last)
        assert status == (dd.DD_ERR_CAPACITY if short else 0)


def test_device_checks(dd):
    """A slot outside the unit's range, of two chunks, a length out of range: the unit stays as it was."""
    for what in ("outside", "other_unit", "twice", "kv", "kv_negative", "new"):
        x = make(13, 3, 2, 50, 16, 30, 10)
        before = buffers(x, 30)
        want, _ = want_of(x, 1, 1, before)                # of the units that are as they should be
        s = x["slot"][1, 1]
        here = np.flatnonzero(s >= 0)
        if what == "outside":
            s[here[0]] = 3 * 2 * 30
        elif what == "other_unit":
            s[here[0]] = 5
        elif what == "twice":
            s[here[0]] = s[here[1]]
        elif what == "kv":
            x["kv"][1], x["n"][1] = 801, 0
        elif what == "kv_negative":
            x["kv"][1] = -1
        else:
            x["kv"][1], x["n"][1] = 700, 101
        got, status = run(dd, x, 1, 1, before)
        assert status == dd.DD_ERR_DEVICE_CHECK
        for b in (0, 2):                                   # (or as they were: a CTA that finds the error pending does nothing)
            for h in range(2):
                assert np.array_equal(got["resident_out"][b, h], want["resident_out"][b, h]) or \
                    np.array_equal(got["resident_out"][b, h], before["resident_out"][b, h])
        assert np.array_equal(got["resident_out"][1, 1], x["slot"][1, 1]) or \
            np.array_equal(got["resident_out"][1, 1], before["resident_out"][1, 1])
        for n in ("slot_chunk", "last_used", "evicted", "union_idx", "union_slot"):
            assert np.array_equal(got[n][1, 1], before[n][1, 1]), n


# more chunks than a CTA's registers hold
MANY = {
    "a_few_more": (3, 2, 8193, 16, 3000, 2500, 4, 64, 0.3),
    "whole_pool_leaves": (2, 2, 9000, 16, 1000, 0, 0, 0, 0.3),
    "nothing_leaves": (2, 2, 12289, 16, 4096, 4096, 0, 0, 0.3),
    "ties": (4, 2, 10000, 16, 5000, 2000, 3, 7, 0.9),
    "odd_pool": (3, 1, 16383, 16, 77, 50, 2, 5, 0.0),
    "protected": (2, 2, 9001, 16, 2222, 5, 4000, 4000, 0.1),
    "many_units": (24, 8, 8200, 16, 512, 300, 1, 1, 0.3),
    "pool_larger_than_half_of_shared_memory": (2, 2, 16384, 16, 9001, 3001, 0, 1, 0.5),
}


@pytest.mark.parametrize("name", list(MANY))
@pytest.mark.parametrize("in_place", [False, True])
def test_evict_many_chunks(dd, name, in_place):
    B, H, C, cs, S, keep, first, last, ties = MANY[name]
    x = make(17, B, H, C, cs, S, keep, ties=ties)
    x["kv"][0], x["n"][0] = C * cs - 40, 40               # (new chunks at the very end, where the pool is not full)
    before = buffers(x, min(C, S))
    got, status = run(dd, x, first, last, before, in_place=in_place)
    want, short = want_of(x, first, last, before)
    for n in OUT:
        assert np.array_equal(got[n], want[n]), n
    assert status == (dd.DD_ERR_CAPACITY if short else 0)
    got, status = run(dd, x, first, last, before, in_place=in_place, optional=False)
    assert np.array_equal(got["resident_out"], want["resident_out"])
    for n in OUT[1:]:
        assert np.array_equal(got[n], before[n]), n


@pytest.mark.parametrize("kind", ["equal", "nan", "inf", "near", "tiny"])
def test_many_chunks_weights_of_all_kinds(dd, kind):
    x = make(18, 2, 2, 8800, 16, 2000, 700, ties=0.0)
    rng = np.random.default_rng(2)
    w = x["w"]
    if kind == "equal":
        w[:] = 1.5
    elif kind == "nan":
        w[rng.random(w.shape) < 0.6] = np.nan
        w[rng.random(w.shape) < 0.2] = -np.nan
    elif kind == "inf":
        w[rng.random(w.shape) < 0.5] = np.inf
        w[rng.random(w.shape) < 0.5] = -np.inf
    elif kind == "near":
        w[:] = (np.float32(1.0).view(np.uint32) + rng.integers(0, 3, w.shape).astype(np.uint32)).view(np.float32)
    else:
        w[:] = (rng.integers(0, 40, w.shape) * 1.4e-45).astype(np.float32)
    before = buffers(x, 2000)
    got, status = run(dd, x, 3, 5, before)
    want, _ = want_of(x, 3, 5, before)
    for n in OUT:
        assert np.array_equal(got[n], want[n]), n
    assert status == 0


@pytest.mark.parametrize("what", ["outside", "negative_side", "twice", "more_than_slots", "kv"])
def test_many_chunks_device_checks(dd, what):
    x = make(19, 2, 2, 9000, 16, 300, 100)
    before = buffers(x, 300)
    s = x["slot"][1, 1]
    here = np.flatnonzero(s >= 0)
    base = 3 * 300
    if what == "outside":
        s[8999] = base + 300
    elif what == "negative_side":
        s[here[0]] = base - 1
    elif what == "twice":
        s[here[0]] = s[here[1]]
    elif what == "more_than_slots":
        s[:] = base + np.arange(9000) % 300
    else:
        x["kv"][1], x["n"][1] = 9000 * 16, 1
    got, status = run(dd, x, 1, 1, before)
    assert status == dd.DD_ERR_DEVICE_CHECK
    assert np.array_equal(got["resident_out"][1, 1], s) or np.array_equal(got["resident_out"][1, 1], before["resident_out"][1, 1])
    assert got["evicted_cnt"][1, 1] in (0, before["evicted_cnt"][1, 1]) and got["union_cnt"][1, 1] in (0, before["union_cnt"][1, 1])
    for n in ("slot_chunk", "last_used", "evicted", "union_idx", "union_slot"):
        assert np.array_equal(got[n][1, 1], before[n][1, 1]), n


@pytest.mark.parametrize("C,S", [(40, 100), (100, 16384), (9000, 16384)])
def test_more_slots_than_chunks(dd, C, S):
    """Pools larger than the cache: no list (it has Umax places), the rest as ever."""
    import torch
    x = make(21, 2, 1, C, 16, S, C // 2, ties=0.2, full=0.9)
    before = buffers(x, 1)
    want, short = want_of(x, 1, 2, buffers(x, C))
    t = {n: torch.from_numpy(v).cuda() for n, v in before.items()}
    with dd.Context(dd.Shape(2, 1, 1, 128, C * 16, 16, C, 1), 0, 2 * S) as ctx:
        args = (torch.from_numpy(x["w"]).cuda(), torch.from_numpy(x["kv"]).cuda(), torch.from_numpy(x["slot"]).cuda(), t["resident_out"],
                x["keep"], S)
        rest = {n: t[n] for n in OUT[1:5]}
        ctx.evict_chunks(*args, first=1, last=2, new_len=torch.from_numpy(x["n"]).cuda(), step=77, **rest)
        assert ctx.status() == 0 and not short
        with pytest.raises(dd.DDError):                   # lists of Umax = C places
            lists = [torch.zeros(2 * C, dtype=torch.int32, device="cuda") for _ in range(2)]
            ctx.evict_chunks(*args, union_idx=lists[0], union_slot=lists[1], union_cnt=t["union_cnt"])
    for n in OUT[:5]:
        got = t[n].cpu().numpy()
        if n == "evicted":                                # (entries behind the counts keep what they held)
            for b in range(2):
                k = want["evicted_cnt"][b, 0]
                assert np.array_equal(got[b, 0, :k], want[n][b, 0, :k]) and np.array_equal(got[b, 0, k:], before[n][b, 0, k:])
        else:
            assert np.array_equal(got, want[n]), n
