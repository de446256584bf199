"""Chunk weights against the 64-bit oracle."""
import numpy as np
import pytest

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


# B, Hkv, G, T, cs, C, kept, ragged, staged, window, decay
SHAPES = {
    "one_token_one_chunk": (1, 1, 1, 1, 16, 1, 1.0, False, 0.0, 0, 1.0),
    "one_token": (2, 2, 4, 1, 16, 75, 1.0, False, 0.0, 0, 0.5),
    "one_token_staged": (2, 2, 8, 1, 64, 30, 0.5, False, 0.4, 0, 0.9),
    "five_tokens_gaps": (3, 2, 8, 5, 16, 64, 0.5, False, 0.0, 0, 0.0),
    "ragged_window": (3, 2, 5, 40, 32, 20, 0.6, True, 0.2, 7, 0.5),
    "window_longer_than_tokens": (2, 1, 4, 40, 16, 20, 1.0, True, 0.0, 39, 1.0),
    "many_rows": (1, 2, 8, 200, 16, 40, 0.7, True, 0.1, 0, 1.0),
    "many_rows_few_keys": (1, 1, 7, 300, 64, 5, 1.0, False, 0.0, 0, 0.25),
    "group_of_64": (1, 1, 64, 9, 32, 25, 1.0, True, 0.0, 0, 1.0),
}


@pytest.mark.parametrize("name", list(SHAPES))
def test_chunk_weights(dd, name):
    B, H, G, T, cs, C, kept, ragged, staged, window, decay = SHAPES[name]
    x = pl.make_case(11, B, H, G, T, cs, C, kept, ragged, staged)
    lse = pl.lse_of(x)
    w0 = np.random.default_rng(3).random((B, H, C)).astype(np.float32)
    if decay == 0.0:
        w0[0, 0, :3] = [np.nan, np.inf, -np.inf]       # nothing is taken over
    got, status = pl.run_weights(dd, x, lse, w0, window, decay)
    assert status == 0
    want, tol = pl.want_weights(x, lse, window, decay, w0)
    same = np.isnan(want) | np.isinf(want)             # chunks outside the list keep theirs
    listed = np.zeros(want.shape, bool)
    for b in range(B):
        for g in range(H):
            listed[b, g, x["idx"][b, g, :x["cnt"][b, g]]] = True
    assert np.array_equal(got[~listed], w0[~listed].astype(np.float64), equal_nan=True)
    assert not same[listed].any()
    assert (np.abs(got - want)[listed] <= tol[listed]).all(), float((np.abs(got - want) / tol)[listed].max())
