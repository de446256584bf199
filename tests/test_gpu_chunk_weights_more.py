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
