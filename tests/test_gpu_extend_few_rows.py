"""Attention of new tokens with up to 32 query rows a KV head: weights keep more than bf16's bits."""
import numpy as np
import pytest

import page_list_lib as pl

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


# requests, KV heads, heads of each, tokens, rows of a chunk, chunks: one part and joined ones, up to 32 rows
ROWS = [(1, 1, 1, 1, 16, 3), (2, 2, 4, 1, 16, 40), (1, 2, 32, 1, 64, 20), (3, 2, 8, 4, 32, 25), (1, 1, 5, 6, 16, 300), (2, 8, 16, 2, 16, 9)]


@pytest.mark.parametrize("B,H,G,T,cs,C", ROWS)
def test_outputs_have_more_than_bf16_weights(dd, B, H, G, T, cs, C):
    x = pl.make_case(101, B, H, G, T, cs, C, 0.9, False, 0.2)
    x["Vhot"], x["Vhot64"] = pl.bf16(x["Vhot64"] + 3.0 * np.sign(x["Vhot64"]))      # sums that cancel
    out, lse, status = pl.run_extend(dd, x)
    assert status == 0
    want, z, _, _ = pl.want_extend(x)
    scale = D ** -0.5
    worst = 0.0
    for b in range(B):
        for g in range(H):
            K, V, pos = pl.unit_rows(x, b, g)
            for t in range(T):
                see = pos <= x["start"][b] + t
                for h in range(g * G, g * G + G):
                    q = x["q64"][b, t, h]
                    w = np.exp(K[see] @ q * scale - z[b, t, h])
                    # a weight: its score's error twice (also in the sum), 2^-20 for the exponential and fp32 sums, and
                    # 2^-15 + 2^-20 for its two parts (the upper 16 bits leave less than 2^-7, bf16 of that is off by 2^-8 of
                    # it; 2^-20 that is added); fp32 sums of products, 2^-24 an addition, below 2^-15 for these lengths; the
                    # output's own rounding, 2^-8 of it
                    av = w @ np.abs(V[see])
                    dx = pl.score_error(q, K[see], scale, z[b, t, h])
                    tol = (2 * dx + 2.0 ** -20 + 2.0 ** -15 + 2.0 ** -20 + 2.0 ** -15) * av + 2.0 ** -8 * np.abs(want[b, t, h])
                    off = np.abs(out[b, t, h] - want[b, t, h])
                    worst = max(worst, (off / tol).max())
    assert worst <= 1.0, worst


@pytest.mark.parametrize("G,T", [(4, 1), (8, 4), (1, 3)])
def test_an_infinity_in_a_tile_that_all_rows_see(dd, G, T):
    """Early in the cache: its column is that infinity in every row that gives it weight, also beside NaN and the other one."""
    C = 60
    x = pl.make_case(102, 1, 2, G, T, 16, C, 1.0, ragged=False, start=[C * 16 - T])
    t = pl.tensors(x)
    base = pl.run_extend(dd, x, t=t)
    u = dict(t, Vhot=t["Vhot"].clone())
    slot = x["slot"][0, 0]
    inf = float("inf")
    for col, (i, row, val) in ((3, (2, 1, inf)), (70, (40, 15, -inf)), (127, (0, 0, float("nan")))):
        u["Vhot"][int(slot[i]), row, col] = val
    u["Vhot"][int(slot[5]), 3, 9], u["Vhot"][int(slot[33]), 3, 9] = inf, -inf
    got = pl.run_extend(dd, x, t=u)
    assert got[2] == 0 and np.array_equal(got[1], base[1])
    rows = got[0][0, :, :G]
    assert (rows[..., 3] == inf).all() and (rows[..., 70] == -inf).all()
    assert np.isnan(rows[..., 127]).all() and np.isnan(rows[..., 9]).all()
    rest = [c for c in range(D) if c not in (3, 70, 127, 9)]
    assert np.array_equal(rows[..., rest], base[0][0, :, :G][..., rest])
    assert np.array_equal(got[0][0, :, G:], base[0][0, :, G:])
