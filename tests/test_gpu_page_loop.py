"""Prompts and decode steps under a budget of chunks, as a serving loop runs them: room made by weight, rows appended,
attention, weights -- against the 64-bit oracle, eager and captured; and the calls' refusals."""
import ctypes

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


class Loop:
    """The device side: a pool of S slots a unit, kept to `keep` chunks."""

    def __init__(self, dd, B, H, G, C, cs, S, keep, T):
        import torch
        i32 = torch.int32
        self.dd, self.args = dd, (B, H, G, C, cs, S, keep)
        self.ctx = dd.Context(dd.Shape(B, H * G, H, D, C * cs, cs, S, 1), 0, B * H * S)
        self.K, self.V = (torch.full((B * H * S, cs, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.map = torch.full((B, H, C), -1, dtype=i32, device="cuda")
        self.idx, self.slot = (torch.zeros(B, H, S, dtype=i32, device="cuda") for _ in range(2))
        self.cnt = torch.zeros(B, H, dtype=i32, device="cuda")
        self.w = torch.zeros(B, H, C, device="cuda")
        self.length = torch.zeros(B, dtype=i32, device="cuda")
        self.new = torch.zeros(B, dtype=i32, device="cuda")
        self.q = torch.zeros(B, T, H * G, D, dtype=torch.bfloat16, device="cuda")
        self.k, self.v = (torch.zeros(B, T, H, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.out, self.lse = torch.zeros_like(self.q), torch.zeros(B, T, H * G, device="cuda")
        self.gone, self.gone_cnt = torch.zeros(B, H, S, dtype=i32, device="cuda"), torch.zeros(B, H, dtype=i32, device="cuda")

    def step(self):
        B, H, G, C, cs, S, keep = self.args
        c = self.ctx
        c.evict_chunks(self.w, self.length, self.map, self.map, keep, S, first=1, last=2, new_len=self.new,
                       evicted=self.gone, evicted_cnt=self.gone_cnt, union_idx=self.idx, union_slot=self.slot, union_cnt=self.cnt)
        c.append_kv(self.k, self.v, self.length, new_len=self.new, Khot=self.K, Vhot=self.V, resident_slot=self.map)
        c.extend_attn(self.q, self.length, self.K, self.V, self.idx, self.slot, self.cnt, self.out, new_len=self.new, lse=self.lse)
        c.chunk_weights(self.q, self.length, self.lse, self.K, self.idx, self.slot, self.cnt, self.w, new_len=self.new,
                        window=16, decay=0.9)
        self.length += self.new


@pytest.mark.parametrize("captured", [False, True])
def test_loop(dd, captured):
    import torch
    B, H, G, C, cs, T = 2, 2, 4, 64, 16, 40
    S, keep = 12, 8                                       # of the 13 chunks that the steps below fill
    rng = np.random.default_rng(71)
    loop = Loop(dd, B, H, G, C, cs, S, keep, T)
    cache = np.zeros((2, B, H, C * cs, D))                # keys and values of all positions
    maps = np.full((B, H, C), -1, np.int64)
    length = np.zeros(B, int)
    graph = None
    if captured:
        side = torch.cuda.Stream()                        # warm up on lengths of zero, which change nothing
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            loop.step()
        torch.cuda.current_stream().wait_stream(side)
        loop.w.zero_()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            loop.step()
    w_dev = np.zeros((B, H, C), np.float32)
    seen = 0
    for step, news in enumerate([(40, 33), (40, 40), (40, 7), (40, 40), (1, 1), (1, 0), (5, 2), (40, 40), (1, 1), (40, 40)]):
        n = np.array(news)
        rows = {}
        for name, heads in (("q", H * G), ("k", H), ("v", H)):
            bits, vals = pl.bf16(rng.standard_normal((B, T, heads, D)))
            rows[name] = vals
            getattr(loop, name).copy_(torch.from_numpy(bits.view(np.int16)).view(torch.bfloat16))
        loop.new.copy_(torch.from_numpy(n.astype(np.int32)))
        graph.replay() if graph else loop.step()
        assert loop.ctx.status() == 0
        out, lse = loop.out.double().cpu().numpy(), loop.lse.double().cpu().numpy()
        idx, slot, cnt = (t.cpu().numpy() for t in (loop.idx, loop.slot, loop.cnt))
        w_new = loop.w.cpu().numpy()
        for b in range(B):
            n0, n1 = -(-length[b] // cs), -(-(length[b] + n[b]) // cs)
            for h in range(H):
                # the map, from the weights that the device had
                u = b * H + h
                now, gone, short = oracle.evict_unit(w_dev[b, h], maps[b, h], u * S, S, n0, n1, keep, 1, 2)
                assert not short
                maps[b, h] = now
                stay = np.flatnonzero(now >= 0)
                assert np.array_equal(idx[b, h, :cnt[b, h]], stay) and np.array_equal(slot[b, h, :cnt[b, h]], now[stay])
                assert np.array_equal(loop.gone[b, h, :len(gone)].cpu().numpy(), gone) and int(loop.gone_cnt[b, h]) == len(gone)
                seen += len(gone)
                for j, name in enumerate(("k", "v")):
                    cache[j, b, h, length[b]:length[b] + n[b]] = rows[name][b, :n[b], h]
                pos = (stay[:, None] * cs + np.arange(cs)).reshape(-1)
                K, V = cache[0, b, h, pos], cache[1, b, h, pos]
                hs = slice(h * G, h * G + G)
                o, z = oracle.extend_attention(rows["q"][b, :n[b], hs], int(length[b]), K, V, pos, D ** -0.5)
                # bf16 weights and output: 2^-8 of the values that are averaged, at most 6 of them, and 2^-8 of the output
                assert np.abs(out[b, :n[b], hs] - o).max(initial=0.0) <= 2.0 ** -8 * 6 + 2.0 ** -8 * np.abs(o).max(initial=0.0)
                # scores' errors: 128 steps of 2^-23 of |q||K| / sqrt(128) <= 20
                assert np.abs(lse[b, :n[b], hs] - z).max(initial=0.0) <= 128 * 2.0 ** -23 * 20 + 2.0 ** -18
                first = max(0, n[b] - 16)
                got = oracle.chunk_weights(rows["q"][b, :n[b], hs], int(length[b]), lse[b, :n[b], hs], K, pos, cs, D ** -0.5, first)
                want = w_dev[b, h].astype(np.float64)
                want[stay] = 0.9 * want[stay] + got
                assert (np.abs(w_new[b, h] - want) <= 1e-3 * want + 1e-30).all()
        w_dev = w_new
        length += n
        assert np.array_equal(loop.length.cpu().numpy(), length)
    assert seen > 20                                      # the budget was felt
    loop.ctx.close()


def test_refusals(dd):
    """Every rule that the host checks, at the C ABI and in the binding."""
    import torch
    x = pl.make_case(73, 2, 2, 4, 3, 16, 20, 1.0, ragged=False, staged=0.3)
    t = pl.tensors(x)
    B, T, H = 2, 3, 8
    out, z = torch.empty_like(t["q"]), torch.empty(B, T, H, device="cuda")
    w = torch.zeros(B, 2, 20, device="cuda")
    pages = (t["Khot"], t["Vhot"], t["idx"], t["slot"], t["cnt"])
    with pl.context(dd, x) as ctx:
        st = dict(Kst=t["Kst"], Vst=t["Vst"])

        def extend(q=t["q"], start=t["start"], pages=pages, out=out, **kw):
            ctx.extend_attn(q, start, *pages, out, **{**st, **kw})

        def weights(q=t["q"], lse=z, weight=w, Khot=t["Khot"], **kw):
            ctx.chunk_weights(q, t["start"], lse, Khot, t["idx"], t["slot"], t["cnt"], weight, **{"Kst": t["Kst"], **kw})

        extend(), weights()
        assert ctx.status() == 0
        for bad in (dict(q=t["q"].float()), dict(q=t["q"][..., :64]), dict(q=t["q"][:1]), dict(q=t["q"].cpu()), dict(q=None),
                    dict(out=out.float()), dict(out=out[:, :2]), dict(out=out[:, :, :1].expand_as(out)), dict(start=None),
                    dict(start=t["start"].long()), dict(start=t["start"][:1]), dict(lse=z.double()), dict(lse=z[:1]),
                    dict(new_len=t["lens"].float()), dict(workspace=torch.empty(16, dtype=torch.uint8, device="cuda")),
                    dict(pages=(t["Khot"][:1], *pages[1:])), dict(pages=(t["Khot"], t["Vhot"], None, *pages[3:])),
                    dict(pages=(t["Khot"], t["Vhot"], t["idx"][:1], *pages[3:]))):
            with pytest.raises((TypeError, ValueError, AttributeError)):
                extend(**bad)
        for bad in (dict(Kst=None), dict(pages=(None, *pages[1:])), dict(pages=(t["Khot"], None, *pages[2:])), dict(Vst=None)):
            with pytest.raises(dd.DDError) as e:
                extend(**bad)
            assert e.value.status == dd.DD_ERR_INVALID_ARG
        # an address off by one element of eight
        with pytest.raises(dd.DDError):
            extend(q=torch.empty(B * T * H * D + 8, dtype=torch.bfloat16, device="cuda")[4:-4].view(B, T, H, D))
        for bad in (dict(lse=None), dict(weight=None), dict(lse=z.half()), dict(weight=w[:1])):
            with pytest.raises((TypeError, ValueError)):
                weights(**bad)
        for bad in (dict(window=-1), dict(decay=-0.1), dict(decay=1.5), dict(decay=float("nan")), dict(Kst=None), dict(Khot=None)):
            with pytest.raises(dd.DDError) as e:
                weights(**bad)
            assert e.value.status == dd.DD_ERR_INVALID_ARG
        assert ctx.extend_attn_workspace(-1) == -1
        lib = dd._lib
        assert lib.dd_extend_attn(None, b"\0" * 184, None) == dd.DD_ERR_INVALID_ARG
        assert lib.dd_extend_attn(ctx._h, None, None) == dd.DD_ERR_INVALID_ARG
        assert lib.dd_chunk_weights(None, b"\0" * 168, None) == dd.DD_ERR_INVALID_ARG
        assert lib.dd_evict_chunks(None, b"\0" * 120, None) == dd.DD_ERR_INVALID_ARG
        # no tokens: nothing to do
        extend(q=t["q"][:, :0], out=out[:, :0])
        weights(q=t["q"][:, :0])
        assert ctx.status() == 0
    i32 = torch.int32
    m = torch.full((2, 2, 20), -1, dtype=i32, device="cuda")
    lens = torch.zeros(2, dtype=i32, device="cuda")
    with dd.Context(dd.Shape(2, 2, 2, D, 320, 16, 8, 1), 0, 2 * 2 * 10) as ctx:
        def evict(keep=5, S=10, weight=w, kv=lens, a=m, b=m, **kw):
            ctx.evict_chunks(weight, kv, a, b, keep, S, **kw)
        evict()
        assert ctx.status() == 0
        lists = {n: torch.zeros(2, 2, 10, dtype=i32, device="cuda") for n in ("union_idx", "union_slot")}
        cnt = torch.zeros(2, 2, dtype=i32, device="cuda")
        for bad in (dict(S=9), dict(S=0), dict(keep=-1), dict(keep=11), dict(first=-1), dict(last=-1),
                    dict(**lists), dict(**lists, union_cnt=cnt),              # S beyond the list's length of 8
                    dict(evicted=torch.zeros(2, 2, 10, dtype=i32, device="cuda"))):
            with pytest.raises(dd.DDError) as e:
                evict(**bad)
            assert e.value.status == dd.DD_ERR_INVALID_ARG
        for bad in (dict(weight=w.double()), dict(weight=None), dict(kv=lens.long()), dict(a=m[:1]), dict(b=m.cpu()), dict(kv=None)):
            with pytest.raises((TypeError, ValueError, AttributeError)):
                evict(**bad)


def test_empty_batch(dd):
    import torch
    with dd.Context(dd.Shape(0, 8, 2, D, 320, 16, 20, 1), 0, 0) as ctx:
        e = torch.empty(0, 4, 8, D, dtype=torch.bfloat16, device="cuda")
        i = torch.empty(0, dtype=torch.int32, device="cuda")
        f = torch.empty(0, device="cuda")
        k = torch.empty(0, 16, D, dtype=torch.bfloat16, device="cuda")
        ctx.extend_attn(e, i, k, k, i, i, i, e.clone())
        ctx.chunk_weights(e, i, f, k, i, i, i, f)
        ctx.evict_chunks(f, i, i, i, 3, 5)
        assert ctx.status() == 0


def test_broadcast_queries(dd):
    """A stride of zero over requests: the same queries for all."""
    import torch
    x = pl.make_case(75, 3, 2, 4, 5, 16, 20, 1.0, ragged=False)
    t = pl.tensors(x)
    t["q"] = t["q"][:1].expand(3, -1, -1, -1)
    x["q64"] = np.broadcast_to(x["q64"][:1], x["q64"].shape)
    out, z = torch.full(t["q"].shape, float("nan"), dtype=torch.bfloat16, device="cuda"), torch.full((3, 5, 8), float("nan"), device="cuda")
    with pl.context(dd, x) as ctx:
        ctx.extend_attn(t["q"], t["start"], t["Khot"], t["Vhot"], t["idx"], t["slot"], t["cnt"], out, lse=z)
        assert ctx.status() == 0
    pl.check_extend((out.double().cpu().numpy(), z.double().cpu().numpy()), pl.want_extend(x))


def test_two_contexts_at_once(dd):
    """Calls of two contexts on two streams do not share counters or workspaces."""
    import torch
    xs = [pl.make_case(s, 2, 2, 8, T, 16, 60, 0.9) for s, T in ((76, 90), (77, 2))]
    ts = [pl.tensors(x) for x in xs]
    wants = [pl.want_extend(x) for x in xs]
    ctxs = [pl.context(dd, x) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    outs = [[torch.full_like(t["q"], float("nan")) for _ in range(8)] for t in ts]
    lses = [[torch.full(t["q"].shape[:3], float("nan"), device="cuda") for _ in range(8)] for t in ts]
    torch.cuda.synchronize()
    for i in range(8):
        for c, t, st, o, z in zip(ctxs, ts, streams, outs, lses):
            c.extend_attn(t["q"], t["start"], t["Khot"], t["Vhot"], t["idx"], t["slot"], t["cnt"], o[i], new_len=t["lens"],
                          lse=z[i], stream=st)
    for c, want, o, z in zip(ctxs, wants, outs, lses):
        assert c.status() == 0
        for i in range(8):
            pl.check_extend((o[i].double().cpu().numpy(), z[i].double().cpu().numpy()), want)
        c.close()
