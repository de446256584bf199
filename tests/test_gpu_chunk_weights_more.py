"""Chunk weights where keys are infinite, where a list goes on behind the tokens, and where there are none."""
import numpy as np
import pytest

import oracle
import page_list_lib as pl

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


# (heads of a KV head, tokens): query rows that fill no block of 32 columns, one and a part, several tiles
ROWS = [(1, 1), (4, 1), (16, 1), (5, 7), (3, 90), (7, 20), (8, 40), (64, 1)]


@pytest.mark.parametrize("G,T", ROWS)
@pytest.mark.parametrize("cs", [16, 64])
def test_a_key_of_minus_infinity_has_no_weight(dd, G, T, cs):
    """One key of a chunk that all rows see whole has scores of -inf: its chunk keeps the other keys' weights."""
    C = 8 + -(-T // cs)
    x = pl.make_case(91, 1, 2, G, T, cs, C, 1.0, ragged=False, start=[C * cs - T])
    i, row = 3, 5
    at = (int(x["slot"][0, 0, i]), row, 7)
    x["q64"][..., 7] = np.abs(x["q64"][..., 7]) + 1.0      # (all that bf16 holds: below)
    x["q"], x["q64"] = pl.bf16(x["q64"])
    t = pl.tensors(x)
    t["Khot"][at] = -float("inf")
    y = dict(x, Khot64=x["Khot64"].copy())
    y["Khot64"][at] = -1e30                                # a weight of exactly 0, in numbers
    lse = pl.want_extend(y)[1].astype(np.float32)
    w0 = np.random.default_rng(5).random((1, 2, C)).astype(np.float32)
    got, status = pl.run_weights(dd, x, lse, w0, 0, 0.5, t=t)
    assert status == 0 and np.isfinite(got).all()
    for g in range(2):
        K, _, pos = pl.unit_rows(y, 0, g)
        hs = slice(g * G, (g + 1) * G)
        new = oracle.chunk_weights(x["q64"][0, :, hs], int(x["start"][0]), lse[0, :, hs], K, pos, cs, 128 ** -0.5)
        # as elsewhere, the scores' errors from the keys that are numbers
        Kn = pl.unit_rows(x, 0, g)[0]
        dx = max(pl.score_error(q, Kn, 128 ** -0.5, z) for q, z in zip(x["q64"][0, :, hs].reshape(-1, 128), lse[0, :, hs].reshape(-1)))
        want = 0.5 * w0[0, g] + new
        assert (np.abs(got[0, g] - want) <= (dx + 2.0 ** -21 + 256 * 2.0 ** -24) * new + 2.0 ** -23 * want).all()


def both(dd, x, t, lse, w0):
    """Attention, then weights with decay 0.5: (out, lse, weights)."""
    ctx = pl.context(dd, x)
    out, z, status = pl.run_extend(dd, x, ctx=ctx, t=t)
    assert status == 0
    w, status = pl.run_weights(dd, x, lse, w0, 0, 0.5, ctx=ctx, t=t)
    assert status == 0
    ctx.close()
    return out, z, w


@pytest.mark.parametrize("G,T", [(4, 1), (8, 5), (8, 40), (2, 150)])
@pytest.mark.parametrize("cs", [16, 64])
def test_chunks_that_no_token_sees_are_not_looked_at(dd, G, T, cs):
    """Behind the last token: slots of no pool, staging slots that are not filled, and one that is."""
    C = 30
    x = pl.make_case(93, 2, 2, G, T, cs, C, 1.0, ragged=False, start=[3 * cs + 5, 20 * cs - T])
    lse = pl.lse_of(x)
    w0 = np.random.default_rng(6).random((2, 2, C)).astype(np.float32)
    t = pl.tensors(x)
    out, z, w = both(dd, x, t, lse, w0)
    y = {k: (v.copy() if isinstance(v, np.ndarray) else v) for k, v in x.items()}
    for b in range(2):
        for g in range(2):
            n = x["cnt"][b, g]
            first = x["idx"][b, g, n - 1] + 1               # (lists end with the last token's chunk)
            more = min(6, C - n, C - first)
            y["idx"][b, g, n:n + more] = first + np.arange(more)
            y["slot"][b, g, n:n + more] = [x["n_hot"], -1, -99, 2 ** 31 - 1, -2 ** 31, 0][:more]
            y["cnt"][b, g] = n + more
    u = dict(t, **{k: v for k, v in pl.tensors(y).items() if k in ("idx", "slot", "cnt")})
    o2, z2, w2 = both(dd, y, u, lse, w0)
    assert np.array_equal(out, o2, equal_nan=True) and np.array_equal(z, z2, equal_nan=True)
    want, tol = pl.want_weights(x, lse, 0, 0.5, w0)
    for b in range(2):
        for g in range(2):
            n = x["cnt"][b, g]
            at = x["idx"][b, g, :n]
            assert (np.abs(w2 - want)[b, g, at] <= tol[b, g, at]).all()
            behind = list(y["idx"][b, g, n:y["cnt"][b, g]])
            assert len(behind) >= 4
            assert np.array_equal(w2[b, g, behind], w0[b, g, behind] * np.float32(0.5))
            rest = sorted(set(range(C)) - set(at) - set(behind))
            assert np.array_equal(w2[b, g, rest], w0[b, g, rest].astype(np.float64))


def test_a_request_without_tokens_looks_at_no_slot(dd):
    """Its chunks decay, whatever the list's slots are; the others are as ever."""
    x = pl.make_case(94, 3, 2, 4, 9, 16, 25, 1.0, lens=[9, 0, 3])
    lse = pl.lse_of(x)
    w0 = np.random.default_rng(7).random((3, 2, 25)).astype(np.float32)
    want, tol = pl.want_weights(x, lse, 0, 0.25, w0)
    y = dict(x, slot=x["slot"].copy(), idx=x["idx"].copy())
    y["slot"][1] = [[x["n_hot"] + 5] * 25, [-77] * 25]
    got, status = pl.run_weights(dd, y, lse, w0, 0, 0.25)
    assert status == 0
    for b in range(3):
        for g in range(2):
            at = x["idx"][b, g, :x["cnt"][b, g]]
            assert (np.abs(got - want)[b, g, at] <= tol[b, g, at]).all()
            if b == 1:
                assert len(at) and np.array_equal(got[b, g, at], w0[b, g, at] * np.float32(0.25))


@pytest.mark.parametrize("decay", [0.0, 0.5, 1.0])
def test_no_tokens_at_all(dd, decay):
    """T = 0: the listed chunks decay, as with new_len 0, and nothing else changes."""
    import torch
    x = pl.make_case(95, 2, 2, 4, 5, 16, 12, 0.7, lens=[5, 2], start=[100, 40])
    t = pl.tensors(x)
    w0 = np.random.default_rng(8).random((2, 2, 12)).astype(np.float32)
    w0[0, 0, x["idx"][0, 0, 0]] = np.inf
    want = w0.copy()
    for b in range(2):
        for g in range(2):
            at = x["idx"][b, g, :x["cnt"][b, g]]
            want[b, g, at] = w0[b, g, at] * np.float32(decay) if decay else 0.0
    with pl.context(dd, x) as ctx:
        for q, lens in ((t["q"][:, :0], None), (t["q"][:, :0], torch.zeros_like(t["lens"])), (t["q"], torch.zeros_like(t["lens"]))):
            w = torch.from_numpy(w0).cuda()
            z = torch.empty(2, q.shape[1], 8, device="cuda")
            ctx.chunk_weights(q, t["start"], z, t["Khot"], t["idx"], t["slot"], t["cnt"], w, new_len=lens, decay=decay)
            assert ctx.status() == 0
            assert np.array_equal(w.cpu().numpy(), want)
        # a position is still one of the cache
        w = torch.from_numpy(w0).cuda()
        ctx.chunk_weights(t["q"][:, :0], t["start"] - 1000, z, t["Khot"], t["idx"], t["slot"], t["cnt"], w, decay=decay)
        assert ctx.status() == dd.DD_ERR_DEVICE_CHECK
        out = t["q"][:, :0].clone()
        ctx.extend_attn(t["q"][:, :0], t["start"], t["Khot"], t["Vhot"], t["idx"], t["slot"], t["cnt"], out)
        assert ctx.status() == 0
