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


def all_close(got, want, tol, x):
    for b in range(x["B"]):
        for g in range(x["Hkv"]):
            at = x["idx"][b, g, :x["cnt"][b, g]]
            off = np.abs(got[b, g, at] - want[b, g, at])
            assert (off <= tol[b, g, at]).all(), (b, g, float((off / tol[b, g, at]).max()))


def test_long_lists_and_many_rows(dd):
    """Several pairs of tiles a CTA, query rows cut into ranges, and both, against the sum of single tokens' calls."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(3)
    for B, H, G, T, cs, C in ((4, 8, 4, 1, 16, 900), (1, 1, 8, 400, 16, 40), (2, 4, 8, 100, 32, 300)):
        L = C * cs
        K = torch.randn(B * H * C, cs, 128, generator=g, device="cuda").to(torch.bfloat16)
        V = torch.randn(B * H * C, cs, 128, generator=g, device="cuda").to(torch.bfloat16)
        slot = torch.randperm(B * H * C, generator=g, device="cuda").to(torch.int32).view(B, H, C)
        idx = torch.arange(C, dtype=torch.int32, device="cuda").expand(B, H, C).contiguous()
        cnt = torch.full((B, H), C, dtype=torch.int32, device="cuda")
        q = torch.randn(B, T, H * G, 128, generator=g, device="cuda").to(torch.bfloat16)
        start = torch.randint(0, L - T + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
        start[0] = L - T
        with dd.Context(dd.Shape(B, H * G, H, 128, L, cs, C, 1), 0, B * H * C) as ctx:
            out, z = torch.empty_like(q), torch.empty(B, T, H * G, device="cuda")
            ctx.extend_attn(q, start, K, V, idx, slot, cnt, out, lse=z)
            w = torch.zeros(B, H, C, device="cuda")
            ctx.chunk_weights(q, start, z, K, idx, slot, cnt, w)
            again = torch.zeros_like(w)
            ctx.chunk_weights(q, start, z, K, idx, slot, cnt, again)
            assert torch.equal(w, again)
            # every row's weights add up to one
            want = torch.full((B, H), float(T * G), device="cuda")
            assert ((w.sum(-1) - want).abs() <= want * (L * 2.0 ** -24 + 1e-5)).all()
            one = torch.zeros_like(w)
            for t in range(0, T):
                ctx.chunk_weights(q[:, t:t + 1], start + t, z[:, t:t + 1].contiguous(), K, idx, slot, cnt, one)
            assert ctx.status() == 0
            # sums of T * G * cs positive numbers either way: 2^-24 an addition, and the scores' errors twice
            tol = one * (T * 2.0 ** -24 + 4e-5)
            assert ((w - one).abs() <= tol + 1e-30).all()


def test_rows_without_keys_and_padding(dd):
    """Log-sum-exps of -inf add nothing; those of padding (NaN here) are not looked at; no tokens: decay alone."""
    x = pl.make_case(13, 3, 2, 4, 9, 16, 12, 1.0, lens=[9, 4, 0])
    lse = pl.lse_of(x)
    w0 = np.random.default_rng(4).random((3, 2, 12)).astype(np.float32)
    lse[0, 3] = -np.inf
    got, status = pl.run_weights(dd, x, lse, w0, decay=0.5)
    assert status == 0
    want, tol = pl.want_weights(x, lse, 0, 0.5, w0)
    all_close(got, want, tol, x)
    # a list that goes on behind the tokens: those chunks decay
    y = pl.make_case(14, 1, 1, 4, 3, 16, 12, 1.0, start=[40], lens=[3])
    y["idx"][0, 0], y["cnt"][0, 0], y["slot"][0, 0] = np.arange(12), 12, 0
    z = pl.lse_of(y)
    got, status = pl.run_weights(dd, y, z, w0[:1, :1], decay=0.25)
    assert status == 0
    want, tol = pl.want_weights(y, z, 0, 0.25, w0[:1, :1])
    all_close(got, want, tol, y)
    assert np.array_equal(got[0, 0, 3:], w0[0, 0, 3:].astype(np.float64) * 0.25)


@pytest.mark.parametrize("G,T", [(4, 2), (8, 60)])
def test_nan(dd, G, T):
    """Keys that no token sees do not matter; a key or log-sum-exp that is NaN does, where it is seen."""
    x = pl.make_case(15, 1, 2, G, T, 16, 20, 1.0, ragged=False, start=[200 - T])
    lse = pl.lse_of(x)
    t = pl.tensors(x)
    w0 = np.zeros((1, 2, 20), np.float32)
    base, _ = pl.run_weights(dd, x, lse, w0, t=t)
    last = 199
    i = list(x["idx"][0, 0, :x["cnt"][0, 0]]).index(last // 16)
    u = dict(t, Khot=t["Khot"].clone())
    u["Khot"][int(x["slot"][0, 0, i]), last % 16 + 1:] = float("nan")
    got, _ = pl.run_weights(dd, x, lse, w0, t=u)
    assert np.array_equal(got, base)
    u["Khot"][int(x["slot"][0, 0, 2]), 3, 3] = float("nan")
    got, _ = pl.run_weights(dd, x, lse, w0, t=u)
    want = base.copy()
    want[0, 0, x["idx"][0, 0, 2]] = np.nan
    assert np.array_equal(got, want, equal_nan=True)
    z = lse.copy()
    z[0, 0, 0] = np.nan                                   # a row of head 0: every chunk that it sees
    got, _ = pl.run_weights(dd, x, z, w0, t=t)
    seen = x["idx"][0, 0, :x["cnt"][0, 0]] * 16 <= x["start"][0]
    assert np.isnan(got[0, 0, x["idx"][0, 0, :x["cnt"][0, 0]][seen]]).all() and np.array_equal(got[0, 1], base[0, 1])


def test_strides_streams_and_graphs(dd):
    import torch
    x = pl.make_case(16, 2, 2, 8, 50, 32, 14, 0.7, start=[20, 300])
    lse = pl.lse_of(x)
    w0 = np.random.default_rng(5).random((2, 2, 14)).astype(np.float32)
    want, tol = pl.want_weights(x, lse, 20, 0.5, w0)
    t = pl.tensors(x)
    wide = torch.full((2, 50, 20, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, :, 1:17] = t["q"]
    z = torch.from_numpy(lse).cuda()
    w = torch.from_numpy(w0).cuda()
    side = torch.cuda.Stream()
    with pl.context(dd, x) as ctx:
        def call(stream=None):
            ctx.chunk_weights(wide[:, :, 1:17], t["start"], z, t["Khot"], t["idx"], t["slot"], t["cnt"], w, new_len=t["lens"],
                              window=20, decay=0.5, stream=stream)
        side.wait_stream(torch.cuda.current_stream())
        call(side)
        torch.cuda.synchronize()
        all_close(w.double().cpu().numpy(), want, tol, x)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        w.copy_(torch.from_numpy(w0))
        g.replay()
        assert ctx.status() == 0
        all_close(w.double().cpu().numpy(), want, tol, x)
        # and another window and length through the same graph's tensors
        t["lens"].copy_(torch.tensor([3, 50], dtype=torch.int32))
        x["lens"] = np.array([3, 50], np.int32)
        z.copy_(torch.from_numpy(pl.lse_of(x)))
        w.copy_(torch.from_numpy(w0))
        g.replay()
        assert ctx.status() == 0
        want, tol = pl.want_weights(x, z.cpu().numpy(), 20, 0.5, w0)
        all_close(w.double().cpu().numpy(), want, tol, x)


def test_device_checks(dd):
    x = pl.make_case(17, 3, 2, 4, 6, 16, 20, 1.0, ragged=False, staged=0.3)
    lse = pl.lse_of(x)
    w0 = np.ones((3, 2, 20), np.float32)
    want, tol = pl.want_weights(x, lse, 0, 1.0, w0)
    for key, at, val in (("slot", (1, 0, 0), x["n_hot"]), ("slot", (1, 0, 0), -1 - x["n_st"]), ("idx", (1, 0, 0), -1),
                         ("idx", (1, 0, 0), 20), ("cnt", (1, 0), 21), ("start", 1, -2), ("lens", 1, 7)):
        y = {k: (v.copy() if isinstance(v, np.ndarray) else v) for k, v in x.items()}
        y[key][at] = val
        got, status = pl.run_weights(dd, y, lse, w0)
        assert status == dd.DD_ERR_DEVICE_CHECK
        for b, g in ((0, 0), (0, 1), (2, 0), (2, 1)):
            ids = x["idx"][b, g, :x["cnt"][b, g]]
            off = np.abs(got[b, g, ids] - want[b, g, ids])
            assert ((off <= tol[b, g, ids]) | (got[b, g, ids] == 1.0)).all()


@pytest.mark.parametrize("B,H,G,T,C", [(140, 8, 2, 1, 9), (131, 8, 64, 3, 3)])
def test_many_requests_and_heads(dd, B, H, G, T, C):
    x = pl.make_case(24, B, H, G, T, 16, C, 0.8, True, 0.1)
    lse = pl.lse_of(x)
    w0 = np.random.default_rng(3).random((B, H, C)).astype(np.float32)
    got, status = pl.run_weights(dd, x, lse, w0, 0, 0.75)
    want, tol = pl.want_weights(x, lse, 0, 0.75, w0)
    assert status == 0
    all_close(got, want, tol, x)
