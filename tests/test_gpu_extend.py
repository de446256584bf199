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


def test_results_do_not_depend_on_the_order_of_work(dd):
    """The same call twice, and beside padding rows of any contents: the same bits."""
    import torch
    x = pl.make_case(19, 6, 2, 4, 3, 16, 60, 0.8)
    t = pl.tensors(x)
    first = pl.run_extend(dd, x, t=t)
    again = pl.run_extend(dd, x, t=t)
    rows = torch.arange(x["T"])[None] >= torch.from_numpy(x["lens"])[:, None]
    t["q"][rows.cuda()] = float("nan")
    other = pl.run_extend(dd, x, t=t)
    for r in (again, other):
        assert np.array_equal(first[0], r[0], equal_nan=True) and np.array_equal(first[1], r[1], equal_nan=True)


def test_strided_rows(dd):
    """Queries out of a fused projection, outputs into one, and both with heads in front of tokens."""
    import torch
    x = pl.make_case(23, 2, 2, 4, 37, 16, 20, 0.7)
    B, T, H = 2, 37, 8
    want = pl.want_extend(x)
    for make in (lambda: torch.full((B, T, H + 4, 128), float("nan"), dtype=torch.bfloat16, device="cuda")[:, :, 2:H + 2],
                 lambda: torch.full((B, H, T, 128), float("nan"), dtype=torch.bfloat16, device="cuda").transpose(1, 2),
                 lambda: torch.full((T, B, H, 136), float("nan"), dtype=torch.bfloat16, device="cuda")[..., 8:].transpose(0, 1)):
        t = pl.tensors(x)
        q, out = make(), make()
        q.copy_(t["q"])
        z = torch.full((B, T, H), float("nan"), device="cuda")
        with pl.context(dd, x) as ctx:
            ctx.extend_attn(q, t["start"], t["Khot"], t["Vhot"], t["idx"], t["slot"], t["cnt"], out, new_len=t["lens"], lse=z)
            assert ctx.status() == 0
        pl.check_extend((out.double().cpu().numpy(), z.double().cpu().numpy()), want)
        if out._base is not None and out._base.shape[-1] == 136:
            assert torch.isnan(out._base[..., :8].float()).all()


def test_lists_that_are_empty_or_hold_nothing_visible(dd):
    """No chunk at all, or only chunks behind the tokens: zeros and -inf."""
    x = pl.make_case(29, 3, 2, 8, 40, 16, 30, 1.0, ragged=False)
    x["cnt"][0, 0] = 0                                   # no list
    x["cnt"][1, 1], x["idx"][1, 1, 0] = 1, 29            # one chunk, behind all tokens of request 1
    x["start"][1] = 100
    n = x["cnt"][2, 0]                                   # request 2, head 0: its own chunks alone
    keep = x["idx"][2, 0, :n] >= x["start"][2] // 16
    m = int(keep.sum())
    x["idx"][2, 0, :m], x["slot"][2, 0, :m] = x["idx"][2, 0, :n][keep], x["slot"][2, 0, :n][keep]
    x["cnt"][2, 0] = m
    got = pl.run_extend(dd, x)
    assert got[2] == 0
    pl.check_extend(got, pl.want_extend(x))
    assert (got[0][0, :, :8] == 0).all() and np.isneginf(got[1][0, :, :8]).all()
    assert (got[0][1, :, 8:] == 0).all() and np.isneginf(got[1][1, :, 8:]).all()


@pytest.mark.parametrize("G,T", [(8, 40), (4, 3)])
def test_what_a_token_does_not_see_does_not_reach_it(dd, G, T):
    """NaN and infinities behind each token: rows not written yet, later tokens' rows, slots that no list names."""
    import torch
    x = pl.make_case(31, 2, 2, G, T, 16, 24, 1.0, ragged=False, start=[100, 333 - T])
    t = pl.tensors(x)
    want = pl.want_extend(x)
    for name, bad in (("Khot", float("nan")), ("Vhot", float("nan")), ("Vhot", float("inf")), ("Vhot", -float("inf"))):
        u = dict(t)
        u[name] = t[name].clone()
        for b in range(2):
            for g in range(2):
                last = int(x["start"][b]) + T - 1            # what lies behind the last token in its chunk
                c = last // 16
                i = list(x["idx"][b, g, :x["cnt"][b, g]]).index(c)
                u[name][int(x["slot"][b, g, i]), last % 16 + 1:] = bad
        pl.check_extend(pl.run_extend(dd, x, t=u), want)


@pytest.mark.parametrize("G,T", [(8, 40), (4, 3), (1, 200)])
def test_infinities_and_nan_reach_who_sees_them(dd, G, T):
    """A value of V at a new token's position: later tokens have it in its column, earlier ones do not."""
    x = pl.make_case(37, 1, 2, G, T, 32, 16, 1.0, ragged=False, start=[300 - T])
    t = pl.tensors(x)
    base = pl.run_extend(dd, x, t=t)
    H = 2 * G
    at = T // 2
    pos = int(x["start"][0]) + at
    i = list(x["idx"][0, 0, :x["cnt"][0, 0]]).index(pos // 32)
    slot, row = int(x["slot"][0, 0, i]), pos % 32
    for col, val in ((5, float("nan")), (77, float("inf")), (127, -float("inf"))):
        u = dict(t)
        u["Vhot"] = t["Vhot"].clone()
        u["Vhot"][slot, row, col] = val
        got = pl.run_extend(dd, x, t=u)
        hit = np.zeros((1, T, H, D), bool)
        hit[0, at:, :G, col] = True
        assert np.array_equal(got[0][~hit], base[0][~hit])
        assert np.array_equal(got[0][hit], np.full(hit.sum(), val), equal_nan=True)
        assert np.array_equal(got[1], base[1])
    # both infinities in one column: NaN once both are seen
    u = dict(t)
    u["Vhot"] = t["Vhot"].clone()
    u["Vhot"][slot, row, 9] = float("inf")
    if row + 1 < 32 and at + 1 < T:
        u["Vhot"][slot, row + 1, 9] = -float("inf")
        got = pl.run_extend(dd, x, t=u)[0]
        assert (got[0, at, :G, 9] == np.inf).all() and np.isnan(got[0, at + 1:, :G, 9]).all()
    # a key that is NaN makes rows that see it NaN, and their log-sum-exp
    u = dict(t)
    u["Khot"] = t["Khot"].clone()
    u["Khot"][slot, row, 3] = float("nan")
    got = pl.run_extend(dd, x, t=u)
    assert np.isnan(got[0][0, at:, :G]).all() and np.isnan(got[1][0, at:, :G]).all()
    assert np.array_equal(got[0][0, :at], base[0][0, :at]) and np.array_equal(got[0][0, :, G:], base[0][0, :, G:])


@pytest.mark.parametrize("G,T", [(8, 40), (4, 2)])
def test_scores_of_any_size(dd, G, T):
    """Scores far beyond what fp32 resolves to 1: a softmax of one row, the largest."""
    import torch
    for scale in (64.0, 2.0 ** 20, 2.0 ** 32, 2.0 ** 60):
        x = pl.make_case(41, 1, 1, G, T, 16, 30, 1.0, ragged=False)
        got = pl.run_extend(dd, x, scale=scale)
        assert got[2] == 0 and np.isfinite(got[0]).all() and np.isfinite(got[1]).all()
        K, V, pos = pl.unit_rows(x, 0, 0)
        for t in range(T):
            for h in range(G):
                s = np.where(pos <= x["start"][0] + t, K @ x["q64"][0, t, h], -np.inf)
                top = np.sort(s)[::-1]
                # (the fp32 sums of 128 products, 128 steps of 2^-24 of at most 2^7, tell these two rows apart)
                if (top[0] - top[1]) * scale > 100 and top[0] - top[1] > 2.0 ** -8:
                    i = int(s.argmax())
                    assert np.array_equal(got[0][0, t, h], V[i])
                    assert abs(got[1][0, t, h] - s[i] * scale) <= 2.0 ** -8 * scale + 2.0 ** -22 * abs(s[i] * scale)


def test_a_score_of_minus_infinity_has_no_weight(dd):
    x = pl.make_case(43, 1, 1, 4, 2, 16, 20, 1.0, ragged=False)
    t = pl.tensors(x)
    i = 3
    t["Khot"][int(x["slot"][0, 0, i]), 5, 7] = -float("inf")
    t["q"][..., 7] = 1.0
    got = pl.run_extend(dd, x, t=t)
    y = dict(x)
    y["q64"] = x["q64"].copy()
    y["q64"][..., 7] = 1.0
    y["Khot64"] = x["Khot64"].copy()
    y["Khot64"][x["slot"][0, 0, i], 5, 7] = -1e30         # (the oracle's bound wants numbers)
    o, z, tol, ltol = pl.want_extend(y)
    K, V, pos = pl.unit_rows(x, 0, 0)
    ltol[:] = 1e-4 + 0 * ltol                             # the bound of rows without that key: |q||K| 128 * 2^-23 / sqrt(128) < 1e-4
    tol[:] = 2.0 ** -7 * np.abs(V).max()
    pl.check_extend(got, (o, z, tol, ltol))


def test_captured_and_replayed_on_other_contents(dd):
    """A graph of two calls of different lengths, replayed with new inputs in the same tensors, on a side stream."""
    import torch
    xs = [pl.make_case(s, 2, 2, 4, T, 16, 40, 0.8, start=[5, 200]) for s, T in ((47, 60), (48, 2))]
    big = max(x["n_hot"] for x in xs)
    for x in xs:                                          # one pool size for both
        pad = ((0, big - x["n_hot"]), (0, 0), (0, 0))
        for n in ("Khot", "Vhot"):
            x[n], x[n + "64"] = np.pad(x[n], pad), np.pad(x[n + "64"], pad)
        x["n_hot"] = big
    ts = [pl.tensors(x) for x in xs]
    outs = [torch.full_like(t["q"], float("nan")) for t in ts]
    lses = [torch.full(t["q"].shape[:3], float("nan"), device="cuda") for t in ts]
    side = torch.cuda.Stream()
    with pl.context(dd, xs[0]) as ctx:
        def calls(stream=None):
            for t, o, z in zip(ts, outs, lses):
                ctx.extend_attn(t["q"], t["start"], t["Khot"], t["Vhot"], t["idx"], t["slot"], t["cnt"], o, new_len=t["lens"],
                                lse=z, stream=stream)
        side.wait_stream(torch.cuda.current_stream())
        calls(side)                                       # eager, on a stream that is not the current one
        torch.cuda.synchronize()
        for x, o, z in zip(xs, outs, lses):
            pl.check_extend((o.double().cpu().numpy(), z.double().cpu().numpy()), pl.want_extend(x))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            calls()
        for o in outs:
            o.fill_(float("nan"))
        new = [pl.make_case(s, 2, 2, 4, x["T"], 16, 40, 0.8, start=[77, 130]) for s, x in ((57, xs[0]), (58, xs[1]))]
        for x, y, t in zip(xs, new, ts):
            n = min(big, y["n_hot"])
            y["slot"] = np.minimum(y["slot"], big - 1)
            pad = ((0, max(0, big - y["n_hot"])), (0, 0), (0, 0))
            for k in ("Khot", "Vhot"):
                y[k], y[k + "64"] = np.pad(y[k][:big], pad), np.pad(y[k + "64"][:big], pad)
            for k, v in pl.tensors(y).items():
                if k in ("q", "idx", "slot", "cnt", "lens", "start", "Khot", "Vhot"):
                    t[k].copy_(v)
        for z in lses:
            z.fill_(float("nan"))
        for _ in range(3):
            g.replay()
        assert ctx.status() == 0
        for y, o, z in zip(new, outs, lses):
            pl.check_extend((o.double().cpu().numpy(), z.double().cpu().numpy()), pl.want_extend(y))


def test_pools_beyond_4_gib(dd):
    """A slot whose rows lie behind byte 2^32 of the pool."""
    import torch
    slots, cs = (1 << 32) // (64 * 256) + 3, 64
    x = pl.make_case(53, 1, 1, 4, 5, cs, 3, 1.0, ragged=False)
    t = pl.tensors(x)
    pools = {}
    for n in ("Khot", "Vhot"):
        p = torch.empty(slots, cs, 128, dtype=torch.bfloat16, device="cuda")
        p[-t[n].shape[0]:] = t[n]
        p[:t[n].shape[0]] = 7.0                           # where 32 bits of the address would lead
        pools[n] = p
    off = slots - x["n_hot"]
    with dd.Context(dd.Shape(1, 4, 1, 128, 3 * cs, cs, 3, 1), 0, slots) as ctx:
        out = torch.full_like(t["q"], float("nan"))
        z = torch.full(out.shape[:3], float("nan"), device="cuda")
        ctx.extend_attn(t["q"], t["start"], pools["Khot"], pools["Vhot"], t["idx"], t["slot"] + off, t["cnt"], out, lse=z)
        assert ctx.status() == 0
    pl.check_extend((out.double().cpu().numpy(), z.double().cpu().numpy()), pl.want_extend(x))


def test_whole_rounds_and_cut_rest(dd):
    """More pairs of row tiles than SMs, so that some are taken whole and the rest is cut, against single-token calls."""
    import torch
    B, H, G, T, cs, C = 3, 8, 8, 260, 16, 400
    g = torch.Generator(device="cuda").manual_seed(5)
    L = C * cs
    K, V = (torch.randn(B * H * C, cs, 128, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    slot = torch.randperm(B * H * C, generator=g, device="cuda").to(torch.int32).view(B, H, C)
    idx = torch.arange(C, dtype=torch.int32, device="cuda").expand(B, H, C).contiguous()
    cnt = torch.full((B, H), C, dtype=torch.int32, device="cuda")
    q = torch.randn(B, T, H * G, 128, generator=g, device="cuda").to(torch.bfloat16)
    start = torch.tensor([L - T, 3000, 0], dtype=torch.int32, device="cuda")
    with dd.Context(dd.Shape(B, H * G, H, 128, L, cs, C, 1), 0, B * H * C) as ctx:
        out, z = torch.empty_like(q), torch.empty(B, T, H * G, device="cuda")
        ctx.extend_attn(q, start, K, V, idx, slot, cnt, out, lse=z)
        assert ctx.status() == 0
        for t in (0, 1, 31, 32, 100, 255, 259):
            o1, z1 = torch.empty_like(q[:, :1]), torch.empty(B, 1, H * G, device="cuda")
            ctx.extend_attn(q[:, t:t + 1], start + t, K, V, idx, slot, cnt, o1, lse=z1)
            assert ctx.status() == 0
            # each is within its bound of the exact value: outputs some 2^-8 of |V| <= 6 from weights and 2^-8 of themselves
            assert (out[:, t].float() - o1[:, 0].float()).abs().max().item() <= 2 * (2.0 ** -8 * 6 * 0.2 + 2.0 ** -8)
            assert (z[:, t] - z1[:, 0]).abs().max().item() <= 1e-4


def test_device_checks(dd):
    """Bad lists, positions and lengths: reported, left out, everything else as it should be."""
    x = pl.make_case(59, 4, 2, 4, 6, 16, 20, 1.0, ragged=False, staged=0.3)
    want = pl.want_extend(x)

    def check(change, rows_ok):
        y = {k: (v.copy() if isinstance(v, np.ndarray) else v) for k, v in x.items()}
        change(y)
        out, lse, status = pl.run_extend(dd, y)
        assert status == dd.DD_ERR_DEVICE_CHECK
        for b, g in rows_ok:
            hs = slice(g * 4, g * 4 + 4)
            sel = lambda a: a[b:b + 1, :, hs]
            if not np.isnan(out[b, :, hs]).any():         # (or as it was)
                pl.check_extend((sel(out), sel(lse)), tuple(sel(a) for a in want))
    rest = [(b, g) for b in range(4) for g in range(2) if (b, g) != (1, 0)]
    check(lambda y: y["slot"].__setitem__((1, 0, 0), y["n_hot"]), rest)
    check(lambda y: y["slot"].__setitem__((1, 0, 0), -1 - y["n_st"]), rest)
    check(lambda y: y["idx"].__setitem__((1, 0, 0), -3), rest)
    check(lambda y: y["cnt"].__setitem__((1, 0), 21), rest)
    check(lambda y: y["cnt"].__setitem__((1, 0), -1), rest)
    rest = [(b, g) for b in (0, 2, 3) for g in range(2)]
    check(lambda y: y["start"].__setitem__(1, -1), rest)
    check(lambda y: y["start"].__setitem__(1, 20 * 16 - 5), rest)
    check(lambda y: y["lens"].__setitem__(1, 7), rest)
    check(lambda y: y["lens"].__setitem__(1, -1), rest)


def test_pending_error_stops_the_call_and_the_next_one_works(dd):
    import torch
    x = pl.make_case(61, 2, 2, 8, 50, 16, 30, 1.0, ragged=False)
    t = pl.tensors(x)
    with pl.context(dd, x) as ctx:
        bad = dict(t, cnt=torch.full_like(t["cnt"], 99))
        z = torch.zeros(2, 50, 16, device="cuda")
        out = torch.zeros_like(t["q"])
        for u in (bad, t):                                # the second call finds the error pending
            ctx.extend_attn(u["q"], u["start"], u["Khot"], u["Vhot"], u["idx"], u["slot"], u["cnt"], out, new_len=u["lens"], lse=z)
        assert ctx.status() == dd.DD_ERR_DEVICE_CHECK
        got = pl.run_extend(dd, x, ctx=ctx, t=t)
        assert got[2] == 0
        pl.check_extend(got, pl.want_extend(x))


@pytest.mark.parametrize("B,H,G,T,C", [(140, 8, 2, 1, 9), (5, 7, 4, 2, 40), (131, 8, 64, 3, 3)])
def test_many_requests_and_heads(dd, B, H, G, T, C):
    """More (request, KV head)s than a warp's lanes, and than their sums' places: slices and pairs of tiles."""
    x = pl.make_case(23, B, H, G, T, 16, C, 0.8, True, 0.1)
    got = pl.run_extend(dd, x)
    assert got[2] == 0
    pl.check_extend(got, pl.want_extend(x))
