"""The chunk that the next tokens are written to: kept by default, and had again after a call that ran out of slots."""
import numpy as np
import pytest

import oracle
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


def state(H, C, S):
    import torch
    i32 = torch.int32
    return (torch.full((1, H, C), -1, dtype=i32, device="cuda"), torch.zeros(1, dtype=i32, device="cuda"),
            torch.zeros(1, dtype=i32, device="cuda"),
            dict(union_idx=torch.zeros(1, H, S, dtype=i32, device="cuda"), union_slot=torch.zeros(1, H, S, dtype=i32, device="cuda"),
                 union_cnt=torch.zeros(1, H, dtype=i32, device="cuda")))


@pytest.mark.parametrize("C", [24, 8200])
def test_by_default_a_token_always_sees_itself(dd, C):
    """Tokens one to nine at a time under a budget of three chunks, the newest chunks the lightest."""
    import torch
    H, G, cs, S, keep = 2, 4, 16, 6, 3
    rng = np.random.default_rng(6)
    slots, length, new, lists = state(H, C, S)
    weight = torch.arange(C, 0, -1, dtype=torch.float32, device="cuda").expand(1, H, C).contiguous()
    K, V = (torch.zeros(H * S, cs, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    cache = np.zeros((2, H, C * cs, D))
    with dd.Context(dd.Shape(1, H * G, H, D, C * cs, cs, S, 1), 0, H * S) as ctx:
        n0 = 0
        for n in (9, 1, 1, 5, 9, 7, 1, 9, 9, 9, 1, 1, 9, 3, 9, 9, 8, 1):
            rows = {k: pl.bf16(rng.standard_normal((1, n, h, D))) for k, h in (("q", H * G), ("k", H), ("v", H))}
            q, k, v = (torch.from_numpy(rows[i][0].view(np.int16)).view(torch.bfloat16).cuda() for i in "qkv")
            length.fill_(n0), new.fill_(n)
            ctx.evict_chunks(weight, length, slots, slots, keep, S, new_len=new, **lists)
            ctx.append_kv(k, v, length, Khot=K, Vhot=V, resident_slot=slots)
            out, lse = torch.zeros_like(q), torch.zeros(1, n, H * G, device="cuda")
            ctx.extend_attn(q, length, K, V, *lists.values(), out, lse=lse)
            assert ctx.status() == 0
            here = slots.cpu().numpy()[0]
            for h in range(H):
                assert (here[h, n0 // cs:(n0 + n - 1) // cs + 1] >= 0).all(), (n0, n)
                cache[0, h, n0:n0 + n], cache[1, h, n0:n0 + n] = rows["k"][1][0, :, h], rows["v"][1][0, :, h]
                stay = np.flatnonzero(here[h] >= 0)
                pos = (stay[:, None] * cs + np.arange(cs)).reshape(-1)
                hs = slice(h * G, h * G + G)
                o, z = oracle.extend_attention(rows["q"][1][0, :, hs], n0, cache[0, h, pos], cache[1, h, pos], pos, D ** -0.5)
                # bf16 weights and output: 2^-8 of the values that are averaged, at most 6 of them, and 2^-8 of the output
                assert np.abs(out[0, :, hs].double().cpu().numpy() - o).max() <= 2.0 ** -8 * 6 + 2.0 ** -8 * np.abs(o).max()
                assert np.abs(lse[0, :, hs].cpu().numpy() - z).max() <= 128 * 2.0 ** -23 * 20 + 2.0 ** -18
            n0 += n
        assert n0 > (keep + 1) * cs                         # the budget was felt


@pytest.mark.parametrize("C", [24, 8200])
def test_new_chunks_without_a_slot_are_new_again(dd, C):
    """Short of slots, then the same call with less to keep, before anything is appended."""
    import torch
    H, cs, S = 2, 16, 6
    slots, length, new, lists = state(H, C, S)
    for h in range(H):
        slots[0, h, :5] = torch.arange(5, dtype=torch.int32) + h * S
    weight = torch.ones(1, H, C, device="cuda")
    length.fill_(5 * cs - 3), new.fill_(3 + 2 * cs + 1)     # the rest of chunk 4, chunks 5, 6, 7
    with dd.Context(dd.Shape(1, H, H, D, C * cs, cs, S, 1), 0, H * S) as ctx:
        ctx.evict_chunks(weight, length, slots, slots, S, S, first=5, new_len=new, **lists)
        assert ctx.status() == dd.DD_ERR_CAPACITY
        assert [np.flatnonzero(s >= 0).tolist() for s in slots.cpu().numpy()[0]] == [[0, 1, 2, 3, 4, 5]] * H
        ctx.evict_chunks(weight, length, slots, slots, S, S, new_len=new, **lists)
        assert ctx.status() == 0
        for h in range(H):
            here = slots.cpu().numpy()[0, h]
            assert np.flatnonzero(here >= 0).tolist() == [2, 3, 4, 5, 6, 7]
            assert sorted(here[here >= 0]) == list(range(h * S, h * S + S))
            assert lists["union_idx"].cpu().numpy()[0, h].tolist() == [2, 3, 4, 5, 6, 7]
