"""Attention of new tokens over a paged cache against the 64-bit oracle."""
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


# B, Hkv, G, T, cs, C, kept, ragged, staged
SHAPES = {
    "one_token_one_chunk": (1, 1, 1, 1, 16, 1, 1.0, False, 0.0),
    "one_token": (1, 2, 4, 1, 16, 40, 1.0, False, 0.0),
    "one_token_long": (2, 2, 8, 1, 64, 70, 1.0, False, 0.0),
    "five_tokens_gaps": (3, 2, 8, 5, 16, 64, 0.5, False, 0.0),
    "rows_fill_a_tile": (1, 2, 8, 16, 32, 33, 1.0, False, 0.0),
    "one_more_than_a_tile": (1, 2, 8, 17, 32, 33, 1.0, False, 0.0),
    "two_tiles": (2, 1, 4, 64, 16, 30, 1.0, True, 0.0),
    "odd_group_ragged_staged": (3, 3, 5, 77, 32, 20, 0.6, True, 0.3),
    "group_of_seven": (2, 2, 7, 60, 64, 9, 0.7, True, 0.2),
    "group_of_64": (1, 1, 64, 9, 16, 25, 1.0, True, 0.0),
    "no_sharing_of_heads": (2, 3, 1, 200, 16, 40, 0.8, True, 0.1),
    "whole_prompt": (2, 2, 4, 300, 16, 19, 1.0, False, 0.0),
    "prompt_of_several_pairs": (1, 1, 8, 130, 64, 10, 1.0, False, 0.0),
}


@pytest.mark.parametrize("name", list(SHAPES))
def test_extend(dd, name):
    B, H, G, T, cs, C, kept, ragged, staged = SHAPES[name]
    x = pl.make_case(7, B, H, G, T, cs, C, kept, ragged, staged)
    got = pl.run_extend(dd, x)
    assert got[2] == 0
    pl.check_extend(got, pl.want_extend(x))
