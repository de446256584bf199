"""Attention over 4-bit pages where its inputs are at their limits."""
import numpy as np
import pytest

import oracle
from sparse_kv_offload_gb300 import synth

import dd_testlib as tl
from test_gpu_attn4 import make_case, run, want_of

pytestmark = pytest.mark.gpu

D = 128


@pytest.fixture(scope="module")
def dd():
    import torch
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from sparse_kv_offload_gb300 import build
    build.build()
    from sparse_kv_offload_gb300 import dd as mod
    return mod


def unit_scale():
    """A softmax scale whose fp32 product with log2(e) is 1: scores are whole numbers of log2 units."""
    s = np.float32(np.log(2.0))
    for c in (np.nextafter(s, np.float32(0)), s, np.nextafter(s, np.float32(1))):
        if c * np.float32(1.4426950408889634) == np.float32(1.0):
            return float(c)
    raise AssertionError


@pytest.mark.parametrize("G", [3, 4, 8, 11, 16, 24, 64])
def test_scores_whose_floats_are_far_apart(dd, G):
    """From 2^25 on the next float is 4, 8, 16, ... away: a later row's score above the softmax's reference by every
    such step, for query vectors of both signs, the same for all of a unit."""
    import torch
    B, cs, C = 320, 64, 16                             # several tiles of a unit follow one another on every warp
    pairs = [(sign * m * 2.0 ** e, up * 2.0 ** (e - 23)) for e in range(24, 30) for m in (1.25, 1.5) for sign in (1, -1)
             for up in (1, 2, 3, 4, 5, 6)]
    pairs += [(2.0 ** e, up * 2.0 ** (e - 23)) for e in range(25, 29) for up in (1, 2, 3, 4)]
    pairs = [(a, d) for a, d in pairs if d <= 40.0]
    rng = np.random.default_rng(G)
    # slot 0: rows with score q0, slot 1: rows with score q0 + q1; both with any values
    K = np.zeros((2, cs, D), np.uint8)
    K[:, :, 0] = 2                                     # code of 1.0, the scales are 1.0
    K[1, :, 1] = 2
    K = oracle.kv4_pack(K, np.full((2, cs, 8), 0x38, np.uint8))
    V = oracle.kv4_pack(rng.integers(0, 16, (2, cs, D)).astype(np.uint8), np.full((2, cs, 8), 0x38, np.uint8))
    q = np.zeros((B, 1, G, D), np.float32)
    which = np.repeat(np.arange(B)[:, None] % len(pairs), G, 1)
    assert len(pairs) <= B
    q[:, 0, :, :2] = np.array(pairs)[which]
    scale = unit_scale()
    slot = np.repeat([0, 1], C // 2)[None].repeat(B, 0)
    out = torch.full((B, 1, G, D), float("nan"), device="cuda")
    with dd.Context(dd.Shape(B, G, 1, D, C * cs, cs, C, 1), max_misses=0, hot_slots=2) as ctx:
        ctx.sparse_attn_decode_kv4(tl.to_bf16(synth.f32_to_bf16(q)), torch.from_numpy(K).cuda(), torch.from_numpy(V).cuda(),
                                   None, None, tl.to_i32(slot), tl.to_i32(np.full(B, C)), out, softmax_scale=scale)
        assert ctx.status() == 0
    v = oracle.kv4_values(V, np.zeros(2)).mean(1)      # every row of a slot has the same weight
    up = np.array([d for _, d in pairs])
    w = np.exp(-up * scale)[:, None]
    want = ((w * v[0] + v[1]) / (1.0 + w))[which]
    # the scores are exact, so what is left is 2^-18 of the largest value for weights, sums and joins; the scale's own
    # last bit moves a weight below 2^-1 by 40 * 2^-24 of itself at most
    assert (np.abs(out.cpu().numpy()[:, 0] - want) <= 2.0 ** -18 * 6.0).all()


@pytest.mark.parametrize("G", [1, 2, 4, 6, 8, 16, 32], ids=lambda g: f"nq{2 * g}")
@pytest.mark.parametrize("cs", [16, 64])
def test_pages_that_no_query_sees_need_no_slot(dd, G, cs):
    """Entries behind kv_len, and entries that no query selected, may hold any slot, wherever they lie in a tile."""
    rng = np.random.default_rng(G * cs)
    for seed in range(4):
        x = make_case(300 + seed, 3, 2, G, 2, cs, 40, 14, empty=0.1)
        L = 40 * cs
        x["length"] = np.array([[0, 5, L // 3], [1, L // 2 + 7, L], [cs, 3 * cs + 1, L - 1], [17, 200, 333]][seed])
        seen = x["idx"] * cs < x["length"][:, None, None]
        unseen = ~seen | (rng.random(seen.shape) < 0.2)
        x["qmask"] = np.where(seen & unseen, 0, x["qmask"]).astype(np.uint8)
        inside = np.arange(x["U"]) < x["cnt"][..., None]
        bad = rng.choice([x["n_hot"], -1 - x["n_st"], 2 ** 31 - 1, -2 ** 31], seen.shape)
        assert (inside & unseen).any()
        for tails in (False, True):
            want, tol = want_of(x, tails)
            y = {**x, "slot": np.where(unseen, bad, x["slot"]).astype(np.int32)}
            got, st = run(dd, y, tails)
            assert st == 0
            assert (np.abs(got - want) <= tol).all()
        # and one that a query does see is reported
        y["slot"] = x["slot"].copy()
        at = np.argwhere(inside & ~unseen & (x["qmask"] != 0))
        if len(at):
            y["slot"][tuple(at[-1])] = x["n_hot"]
            assert run(dd, y)[1] == dd.DD_ERR_DEVICE_CHECK


@pytest.mark.parametrize("G", [4, 12, 30], ids=["nq4", "nq12", "nq30"])
def test_an_error_of_the_call_itself_leaves_no_mixture(dd, G):
    """A bad page in one short unit, while other streams' work holds a part of the SMs, so that some CTAs of the long units
    start after the error has been reported: every unit's output is its own result, or as it was.  (An earlier call
    with other queries has left its sums in the workspace.)"""
    import torch
    B, C, cs, n = 130, 400, 16, 64
    rng = np.random.default_rng(400 + G)
    codes, s8 = oracle.quantise_rows(rng.standard_normal((2 * n, cs, D)), np.zeros((2 * n, cs)))
    p = list(torch.from_numpy(oracle.kv4_pack(codes, s8)).cuda().split(n))
    q, other = (tl.to_bf16(synth.f32_to_bf16(rng.standard_normal((B, 1, G, D)).astype(np.float32))) for _ in range(2))
    slot, cnt = tl.to_i32(rng.integers(0, n, (B, 1, C))), tl.to_i32(np.where(np.arange(B) < 100, 2, C))
    bad = slot.clone()
    bad[0, 0, 1] = n
    busy = torch.zeros(512, 1 << 15, device="cuda")
    sides = [torch.cuda.Stream() for _ in range(4)]
    with dd.Context(dd.Shape(B, G, 1, D, C * cs, cs, C, 1), max_misses=0, hot_slots=n) as ctx:
        want, junk = (torch.zeros(B, 1, G, D, device="cuda") for _ in range(2))
        ctx.sparse_attn_decode_kv4(q, *p, None, None, slot, cnt, want)
        assert ctx.status() == 0
        for i in range(40):
            ctx.sparse_attn_decode_kv4(other, *p, None, None, slot, cnt, junk)
            assert ctx.status() == 0
            out = torch.full((B, 1, G, D), 7.0, device="cuda")
            torch.cuda.synchronize()
            for s in sides[:1 + i % 4]:
                with torch.cuda.stream(s):
                    torch.cumsum(busy, 1)
            ctx.sparse_attn_decode_kv4(q, *p, None, None, bad, cnt, out)
            assert ctx.status() == dd.DD_ERR_DEVICE_CHECK
            same = (out == want).flatten(1).all(1) | (out == 7.0).flatten(1).all(1)
            assert same[1:].all()
        out = torch.zeros(B, 1, G, D, device="cuda")
        ctx.sparse_attn_decode_kv4(q, *p, None, None, slot, cnt, out)
        assert ctx.status() == 0 and torch.equal(out, want)


@pytest.mark.parametrize("G", [2, 6, 12, 24], ids=lambda g: f"nq{g}")
def test_infinite_queries(dd, G):
    """A query vector with an infinite value beside finite ones of any size: NaN where a row's score is +inf or NaN,
    no weight where it is -inf, whatever the finite values are."""
    x = make_case(500, 2, 2, G, 1, 16, 30, 12, p_hot=1.0, empty=0.0, ragged=False)
    codes, s8 = oracle.kv4_unpack(x["Khot"])
    s8 = s8 | 0x08                                                 # no zero scale
    codes[..., 5] = np.where(codes[..., 5] & 7, codes[..., 5] & 7, 3)      # above zero: the score has q's sign
    x["Khot"] = oracle.kv4_pack(codes, s8)
    want, tol = want_of(x, False)
    q = x["q"].copy()
    big = synth.f32_to_bf16(np.array([1.0, 6e4, 7e4, 1e10, 3e38], np.float32))
    for i, size in enumerate(big):
        y = q.copy()
        y[:, 0, 0::2, 5] = 0xFF80                                  # every other head: -inf
        y[:, 0, 0::2, 9] = size
        y[:, 0, 0::2, 77] = size | 0x8000
        y[0, 0, 0, 5] = 0x7F80                                     # one with +inf
        got, st = run(dd, {**x, "q": y}, False)
        assert st == 0
        assert np.isnan(got[0, 0, 0]).all()
        assert not got[0, 0, 2::2].any() and not got[1, 0, 0::2].any()
        assert (np.abs(got - want) <= tol)[:, :, 1::2].all()


@pytest.mark.parametrize("G", [4, 6, 12, 24], ids=lambda g: f"nq{g}")
def test_a_factor_beyond_fp32_keeps_zero_scores(dd, G):
    """Queries and a head's exponent so large that their factor alone passes fp32: rows of zeros still score zero."""
    x = make_case(600, 2, 2, G, 1, 16, 30, 12, p_hot=1.0, empty=0.0, ragged=False, qscale=2.0 ** 90)
    x["ke"] = np.full(2, 64)
    x["Khot"] = np.zeros_like(x["Khot"])
    want, tol = want_of(x, False)                                  # the mean of V
    got, st = run(dd, x, False)
    assert st == 0 and (np.abs(got - want) <= tol).all()
