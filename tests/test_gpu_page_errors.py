"""Errors that one (request, KV head) of a call reports: what it leaves out, and that all others are done."""
import numpy as np
import pytest

import page_list_lib as pl
import test_gpu_evict as te

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


@pytest.mark.parametrize("C", [2048, 8193])
@pytest.mark.parametrize("what", ["short", "twice", "outside", "length"])
def test_eviction_of_the_other_units(dd, what, C):
    """Several times as many units as fit the GPU at once; the first of them are short of slots or not in order."""
    import torch
    B, H, cs, S, keep, first, last = 80, 8, 16, 16, 8, 0, 16
    x = te.make(31, B, H, C, cs, S, keep)
    if what == "short":
        # no chunk of the first request may leave
        x["kv"][0], x["n"][0] = C * cs // 2, 40
        x["slot"][0] = -1
        for h in range(H):
            x["slot"][0, h, C // 2 - S:C // 2] = h * S + np.arange(S)
    elif what == "length":
        x["kv"][0], x["n"][0] = C * cs, 1
    else:
        x["slot"][0] = -1
        for h in range(H):
            x["slot"][0, h, 5], x["slot"][0, h, 6] = h * S, h * S if what == "twice" else h * S + S
    before = te.buffers(x, S)
    y = dict(x, kv=x["kv"].copy(), slot=x["slot"].copy())  # of the requests that are in order
    if what != "short":
        y["kv"][0], y["slot"][0] = 0, -1
    want, short = te.want_of(y, first, last, before)
    if what != "short":
        # the first request stays as it was
        for n in te.OUT:
            want[n][0] = before[n][0]
        want["resident_out"][0] = x["slot"][0]
        want["evicted_cnt"][0] = want["union_cnt"][0] = 0
    inputs = [torch.from_numpy(x[n]).cuda() for n in ("w", "kv", "slot", "n")]
    with dd.Context(dd.Shape(B, H, H, 128, C * cs, cs, S, 1), 0, B * H * S) as ctx:
        def call():
            t = {n: torch.from_numpy(v).cuda() for n, v in before.items()}
            ctx.evict_chunks(*inputs[:3], t["resident_out"], keep, S, first=first, last=last, new_len=inputs[3], step=77,
                             **{n: t[n] for n in te.OUT[1:]})
            return t

        def equal(t, r):
            for n in te.OUT:
                assert np.array_equal(t[n].cpu().numpy(), r[n]), n
        for _ in range(3):
            got = call()
            idle = call()                                  # the error of the call before is pending
            equal(got, want)
            equal(idle, before)
            status = ctx.status()
            # (where both are reported the first one stands)
            assert status in ((dd.DD_ERR_CAPACITY,) if what == "short" else
                              (dd.DD_ERR_DEVICE_CHECK, dd.DD_ERR_CAPACITY) if short else (dd.DD_ERR_DEVICE_CHECK,))
        assert ctx.status() == 0


def without_entry(x, b, g, i):
    """The case without entry i of a list."""
    y = {k: (v.copy() if isinstance(v, np.ndarray) else v) for k, v in x.items()}
    n = y["cnt"][b, g]
    for k in ("idx", "slot"):
        y[k][b, g, i:n - 1] = x[k][b, g, i + 1:n]
    y["cnt"][b, g] -= 1
    return y


# requests, KV heads, heads of each, tokens, chunks: slices of one row tile, pairs of row tiles, many of them
MANY = [(40, 8, 2, 1, 12), (6, 4, 8, 40, 20), (3, 2, 8, 130, 30)]


@pytest.mark.parametrize("B,H,G,T,C", MANY)
def test_attention_and_weights_of_the_other_units(dd, B, H, G, T, C):
    """A slot, a count and a length out of range in the first request: whoever starts later does its work all the same."""
    x = pl.make_case(81, B, H, G, T, 16, C, 1.0, ragged=False, staged=0.2)
    want = pl.want_extend(x)
    lse = want[1].astype(np.float32)
    w0 = np.random.default_rng(3).random((B, H, C)).astype(np.float32)
    w_want = pl.want_weights(x, lse, 0, 0.5, w0)
    ctx = pl.context(dd, x)
    clean = pl.run_extend(dd, x, ctx=ctx)
    w_clean, status = pl.run_weights(dd, x, lse, w0, 0, 0.5, ctx=ctx)
    assert clean[2] == status == 0
    y = {k: (v.copy() if isinstance(v, np.ndarray) else v) for k, v in x.items()}
    y["slot"][0, 0, 0] = y["n_hot"]
    less = without_entry(x, 0, 0, 0)
    less_want = pl.want_extend(less)
    less_w = pl.want_weights(less, lse, 0, 0.5, w0)
    for _ in range(10):
        # (a list's length shares out the work, and that it keeps: the same bits)
        got = pl.run_extend(dd, y, ctx=ctx)
        w, status = pl.run_weights(dd, y, lse, w0, 0, 0.5, ctx=ctx)
        assert got[2] == status == dd.DD_ERR_DEVICE_CHECK
        hs = np.ones((B, H * G), bool)
        hs[0, :G] = False
        for a, b in zip(got, clean[:2]):
            assert np.array_equal(a.swapaxes(1, 2)[hs], b.swapaxes(1, 2)[hs], equal_nan=True)
        pl.check_extend(got, less_want)
        units = np.ones((B, H), bool)
        units[0, 0] = False
        assert np.array_equal(w[units], w_clean[units])
        at = less["idx"][0, 0, :less["cnt"][0, 0]]
        assert (np.abs(w - less_w[0])[0, 0, at] <= less_w[1][0, 0, at]).all()
        out = x["idx"][0, 0, 0]
        assert w[0, 0, out] == w0[0, 0, out]               # as it was
    for key, at, val in (("cnt", (0, 0), C + 1), ("lens", 0, T + 1), ("start", 0, -1)):
        z = {k: (v.copy() if isinstance(v, np.ndarray) else v) for k, v in x.items()}
        z[key][at] = val
        rest = [(b, g) for b in range(B) for g in range(H) if (b, g) != (0, 0) and (b or key == "cnt")]
        for _ in range(10):
            out, z_lse, status = pl.run_extend(dd, z, ctx=ctx)
            assert status == dd.DD_ERR_DEVICE_CHECK
            w, status = pl.run_weights(dd, z, lse, w0, 0, 0.5, ctx=ctx)
            assert status == dd.DD_ERR_DEVICE_CHECK
            sel = lambda a: np.stack([a[b][:, g * G:(g + 1) * G] for b, g in rest])
            pl.check_extend((sel(out), sel(z_lse)), tuple(sel(a) for a in want))
            for b, g in rest:
                at = x["idx"][b, g, :x["cnt"][b, g]]
                assert (np.abs(w - w_want[0])[b, g, at] <= w_want[1][b, g, at]).all()
            if key == "cnt":
                # a list that is left out: rows without keys, weights as they were
                assert (out[0, :, :G] == 0).all() and np.isneginf(z_lse[0, :, :G]).all()
                assert np.array_equal(w[0, 0], w0[0, 0])
            else:
                assert np.isnan(out[0]).all() and np.isnan(z_lse[0]).all()
                for g in range(H):
                    at = x["idx"][0, g, :x["cnt"][0, g]]
                    assert np.array_equal(w[0, g, at], w0[0, g, at] * np.float32(0.5))
    # the context goes on
    got = pl.run_extend(dd, x, ctx=ctx)
    assert got[2] == 0 and all(np.array_equal(a, b, equal_nan=True) for a, b in zip(got[:2], clean[:2]))
    ctx.close()
