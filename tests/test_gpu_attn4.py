"""Attention over 4-bit pages against the 64-bit oracle, and the cache operators run
together as a decode loop uses them."""
import numpy as np
import pytest

import oracle
from sparse_kv_offload_gb300 import synth

import dd_testlib as tl

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


def pages(rng, n, cs, scale=1.0):
    codes, s = oracle.quantise_rows(rng.standard_normal((n, cs, D)) * scale, np.zeros((n, cs)))
    return oracle.kv4_pack(codes, s)


def make_case(seed, B, Hkv, G, n_q, cs, C, k, p_hot=0.5, empty=0.15, ragged=True, qscale=1.0):
    rng = np.random.default_rng(seed)
    U = min(C, n_q * k)
    x = dict(B=B, Hkv=Hkv, G=G, n_q=n_q, cs=cs, C=C, k=k, U=U)
    idx = np.zeros((B, Hkv, U), np.int32)
    slot = np.zeros((B, Hkv, U), np.int32)
    qmask = np.zeros((B, Hkv, U), np.uint8)
    cnt = np.zeros((B, Hkv), np.int32)
    n_hot = n_st = 0
    for b in range(B):
        for g in range(Hkv):
            picks = [set() if rng.random() < empty else set(rng.choice(C, k, replace=False).tolist()) for _ in range(n_q)]
            if rng.random() < empty:
                picks = [set()] * n_q
            for i, c in enumerate(sorted(set().union(*picks))):
                idx[b, g, i] = c
                qmask[b, g, i] = sum(1 << j for j in range(n_q) if c in picks[j])
                if rng.random() < p_hot:
                    slot[b, g, i], n_hot = n_hot, n_hot + 1
                else:
                    slot[b, g, i], n_st = -1 - n_st, n_st + 1
                cnt[b, g] += 1
    ph = rng.permutation(n_hot + 2)[:max(1, n_hot)]
    slot = np.where(slot >= 0, ph[np.clip(slot, 0, len(ph) - 1)], slot).astype(np.int32)
    x.update(idx=idx, slot=slot, qmask=qmask, cnt=cnt, n_hot=n_hot + 2, n_st=n_st,
             Khot=pages(rng, n_hot + 2, cs), Vhot=pages(rng, n_hot + 2, cs),
             Kst=pages(rng, max(1, n_st), cs), Vst=pages(rng, max(1, n_st), cs),
             ke=rng.integers(-2, 3, Hkv), ve=rng.integers(-3, 4, Hkv),
             q=synth.f32_to_bf16((rng.standard_normal((B, n_q, Hkv * G, D)) * qscale).astype(np.float32)),
             Kt=synth.f32_to_bf16(rng.standard_normal((B, n_q, Hkv, D)).astype(np.float32)),
             Vt=synth.f32_to_bf16(rng.standard_normal((B, n_q, Hkv, D)).astype(np.float32)))
    L = C * cs
    x["length"] = rng.integers(0, L + 1, B) if ragged else np.full(B, L)
    return x


def want_of(x, tails, scale=D ** -0.5, mask=True, length=True):
    """(outputs, bound on each query vector's error) in 64 bits."""
    B, n_q, H, G, cs = x["B"], x["n_q"], x["Hkv"], x["G"], x["cs"]
    out = np.zeros((B, n_q, H * G, D))
    tol = np.zeros((B, n_q, H * G, 1))
    q = oracle.bf16_decode(x["q"])
    vals = {n: oracle.kv4_values(x[n], np.zeros(len(x[n]))) for n in ("Khot", "Vhot", "Kst", "Vst")}
    for b in range(B):
        for g in range(H):
            n = x["cnt"][b, g]
            K, V, pos = [], [], []
            for i in range(n):
                s = x["slot"][b, g, i]
                K.append(vals["Khot"][s] if s >= 0 else vals["Kst"][-1 - s])
                V.append(vals["Vhot"][s] if s >= 0 else vals["Vst"][-1 - s])
                pos.append(x["idx"][b, g, i] * cs + np.arange(cs))
            K = np.array(K).reshape(-1, D) * 2.0 ** x["ke"][g]
            V = np.array(V).reshape(-1, D) * 2.0 ** x["ve"][g]
            pos = np.array(pos).reshape(-1)
            for j in range(n_q):
                keep = pos < x["length"][b] if length else np.ones(len(pos), bool)
                if mask:
                    keep &= np.repeat((x["qmask"][b, g, :n] >> j) & 1, cs) == 1
                Kj, Vj = K[keep], V[keep]
                if tails:
                    Kj = np.concatenate([Kj, oracle.bf16_decode(x["Kt"][b, :j + 1, g])])
                    Vj = np.concatenate([Vj, oracle.bf16_decode(x["Vt"][b, :j + 1, g])])
                for h in range(g * G, (g + 1) * G):
                    out[b, j, h] = oracle.attention_rows(q[b, j, h], Kj, Vj, scale)
                    if len(Kj):
                        # scores: 128 exact products summed in fp32 (2^-23 each, truncation allowed for) move every
                        # weight by twice that; 2^-18 for the exponential (2^-21), its weight's 22 bits, the scaled
                        # score's last bit at |x| <= 32 and the joins, of the largest value either way
                        dx = 128 * 2.0 ** -23 * (np.abs(Kj) @ np.abs(q[b, j, h])).max() * scale
                        tol[b, j, h] = (2 * dx + 2.0 ** -18) * np.abs(Vj).max()
    return out, tol


def run(dd, x, tails=False, mask=True, length=True, scale=0.0, ctx=None, hot=True):
    import torch
    B, n_q, H, G = x["B"], x["n_q"], x["Hkv"], x["G"]
    out = torch.full((B, n_q, H * G, D), float("nan"), device="cuda")
    made = ctx is None
    if made:
        ctx = dd.Context(dd.Shape(B, H * G, H, D, x["C"] * x["cs"], x["cs"], x["k"], n_q), max_misses=x["n_st"],
                         hot_slots=x["n_hot"])
    kw = dict(K_tail=tl.to_bf16(x["Kt"]), V_tail=tl.to_bf16(x["Vt"])) if tails else {}
    if mask:
        kw["union_qmask"] = torch.from_numpy(x["qmask"].reshape(-1)).cuda()
    if length:
        kw.update(kv_len=tl.to_i32(x["length"]), union_idx=tl.to_i32(x["idx"]))
    p = [torch.from_numpy(x[n]).cuda() for n in ("Khot", "Vhot", "Kst", "Vst")]
    ctx.sparse_attn_decode_kv4(tl.to_bf16(x["q"]), *p, tl.to_i32(x["slot"]), tl.to_i32(x["cnt"]), out,
                               miss_count=tl.to_i32([x["n_st"]]), k_exp=tl.to_i32(x["ke"]), v_exp=tl.to_i32(x["ve"]),
                               softmax_scale=scale, **kw)
    st = ctx.status()
    if made:
        ctx.close()
    return out.cpu().numpy().astype(np.float64), st


# (B, Hkv, G, n_q, cs, C, k): from one row's chunk to unions over every CTA, query vectors on both sides of
# each tile of 8 and of 16, up to 64
SHAPES = [
    (1, 1, 1, 1, 16, 1, 1), (1, 2, 4, 1, 16, 40, 16), (2, 2, 4, 2, 16, 64, 24), (2, 1, 1, 7, 32, 33, 9),
    (1, 3, 3, 3, 64, 21, 7), (2, 2, 8, 2, 32, 300, 60), (1, 1, 17, 1, 16, 50, 20), (1, 2, 8, 5, 16, 90, 30),
    (1, 1, 8, 8, 16, 40, 10), (1, 2, 7, 7, 64, 8, 3), (3, 2, 12, 2, 32, 25, 11), (1, 1, 4, 1, 64, 1200, 1200),
    (7, 3, 5, 1, 16, 30, 30), (1, 1, 33, 1, 32, 9, 4), (1, 1, 64, 1, 16, 64, 64),
]


@pytest.mark.parametrize("tails", [False, True], ids=["no_tail", "tail"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_attention_matches_oracle(dd, shape, tails):
    x = make_case(hash(shape) % 1000, *shape)
    want, tol = want_of(x, tails)
    got, st = run(dd, x, tails)
    assert st == 0
    assert (np.abs(got - want) <= tol).all(), np.abs(got - want).max()
    assert np.linalg.norm(got - want) <= 2e-5 * np.linalg.norm(want) + 1e-30


@pytest.mark.parametrize("mask,length", [(False, True), (True, False), (False, False)])
@pytest.mark.parametrize("shape", [(2, 2, 4, 2, 16, 40, 12), (1, 2, 8, 4, 32, 20, 6)], ids=str)
def test_optional_masks(dd, shape, mask, length):
    x = make_case(5, *shape)
    want, tol = want_of(x, True, mask=mask, length=length, scale=0.03)
    got, st = run(dd, x, True, mask=mask, length=length, scale=0.03)
    assert st == 0 and (np.abs(got - want) <= tol).all()


def test_large_scores(dd):
    """Scores hundreds of units apart, and queries of very different sizes side by side: one row's weight is 1."""
    x = make_case(21, 1, 2, 8, 2, 16, 60, 20, qscale=30.0, ragged=False)
    f = np.array([1e-30, 1e-3, 1.0, 4.0, 1e-38, 0.0, 2.0, 0.5] * 2, np.float32)
    q = oracle.bf16_decode(x["q"]).astype(np.float32) * f[None, None, :, None]
    x["q"] = synth.f32_to_bf16(q)
    want, tol = want_of(x, False)
    got, st = run(dd, x, False)
    assert st == 0 and (np.abs(got - want) <= np.minimum(tol, 4.0 * 2.0 ** 3)).all()
    small = np.abs(want).max(-1) > 0
    assert small.all() or x["cnt"].min() == 0


@pytest.mark.parametrize("G", [2, 4, 16], ids=["nq4", "nq8", "nq32"])
def test_rows_behind_the_end_may_hold_anything(dd, G):
    """NaN scales and random codes behind kv_len, in chunks that end inside and in chunks wholly behind."""
    x = make_case(31, 3, 2, G, 2, 32, 12, 8, empty=0.0)
    x["length"] = np.array([0, 5, 200])
    want, tol = want_of(x, False)
    rng = np.random.default_rng(1)
    for n in ("Khot", "Vhot", "Kst", "Vst"):
        junk = rng.integers(0, 256, x[n].shape, dtype=np.uint8)
        junk.reshape(len(junk), -1, 1152)[..., 1024:] |= 0x7F
        x["old_" + n] = x[n]
        x[n] = junk
    for b in range(3):                                             # put back what lies before the end
        for g in range(2):
            for i in range(x["cnt"][b, g]):
                rows = int(np.clip(x["length"][b] - x["idx"][b, g, i] * 32, 0, 32))
                s = x["slot"][b, g, i]
                for kv in "KV":
                    n, at = (kv + "hot", s) if s >= 0 else (kv + "st", -1 - s)
                    for t in range(rows):
                        blk, r = t // 16 * 1152, t % 16
                        for o, w in ((blk + r * 64, 64), (blk + 1024 + r * 8, 8)):
                            x[n][at, o:o + w] = x["old_" + n][at, o:o + w]
    got, st = run(dd, x, False)
    assert st == 0 and (np.abs(got - want) <= tol).all()
    assert not got[0].any()                                       # no row at all: zeros


@pytest.mark.parametrize("G", [1, 2, 4, 8], ids=["nq3", "nq6", "nq12", "nq24"])
def test_nan_stays_with_the_queries_that_see_it(dd, G):
    """A NaN scale in a chunk: the queries that picked the chunk get NaN (in the columns of a V group, everywhere for
    K), the others their own result."""
    for which in ("V", "K"):
        x = make_case(41, 1, 1, G, 3, 16, 30, 10, p_hot=1.0, empty=0.0, ragged=False)
        want, tol = want_of(x, True)
        i = int(np.flatnonzero((x["qmask"][0, 0, :x["cnt"][0, 0]] & 7) < 7)[0])
        x[which + "hot"].reshape(len(x[which + "hot"]), -1, 1152)[x["slot"][0, 0, i], 0, 1024 + 3 * 8 + 2] = 0x7F
        got, st = run(dd, x, True)
        assert st == 0
        for j in range(3):
            hit = (x["qmask"][0, 0, i] >> j) & 1
            bad = np.zeros(D, bool)
            if hit:
                bad[32:48 if which == "V" else D] = True
                bad[:] |= which == "K"
            assert np.isnan(got[0, j][:, bad]).all()
            assert (np.abs(got - want)[0, j][:, ~bad] <= tol[0, j]).all()


@pytest.mark.parametrize("G", [1, 4, 8], ids=["nq3", "nq12", "nq24"])
def test_scores_that_underflow_keep_the_mask(dd, G):
    """Queries and keys so small that every score is zero in fp32: equal weights for the rows that are seen, none for
    the others."""
    x = make_case(61, 2, 2, G, 3, 16, 40, 12, qscale=2.0 ** -126)
    x["ke"] = np.full(2, -64)
    want, tol = want_of(x, False)
    got, st = run(dd, x, False)
    assert st == 0 and (np.abs(got - want) <= tol).all()


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("G", [2, 12, 24])
def test_infinite_scores_of_the_new_rows(dd, G, sign):
    """A new row whose key is infinite: NaN for the query vectors whose score is +inf, no weight where it is -inf."""
    for empty in (0.0, 1.0):
        x = make_case(62, 2, 2, G, 1, 16, 40, 12, empty=empty, ragged=False)
        x["Kt"] = x["Kt"].copy()
        x["Kt"][..., 0] = synth.f32_to_bf16(np.full(1, sign * np.inf, np.float32))[0]
        want, tol = want_of(x, False)
        got, st = run(dd, x, True)
        assert st == 0
        up = oracle.bf16_decode(x["q"])[..., 0] * sign >= 0        # 0 * inf: NaN too
        assert 0 < up.sum() < up.size
        if empty:
            assert np.isnan(got).all()                             # nothing else: -inf - -inf
        else:
            assert np.isnan(got[up]).all() and (np.abs(got - want) <= tol)[~up].all()


def test_bad_pages_are_reported(dd):
    x = make_case(51, 1, 2, 4, 1, 16, 30, 10, empty=0.0, ragged=False)
    for name, value in (("slot", x["n_hot"]), ("slot", -1 - x["n_st"]), ("slot", -2 ** 31), ("cnt", x["U"] + 1), ("cnt", -1),
                        ("ke", 65), ("ve", -65)):
        y = {**x, name: x[name].copy()}
        y[name].reshape(-1)[1] = value
        _, st = run(dd, y)
        assert st == dd.DD_ERR_DEVICE_CHECK
        # and the same context goes on afterwards
    with dd.Context(dd.Shape(1, 8, 2, D, 480, 16, 10, 1), max_misses=x["n_st"], hot_slots=x["n_hot"]) as ctx:
        y = {**x, "slot": np.full_like(x["slot"], 10 ** 6)}
        assert run(dd, y, ctx=ctx)[1] == dd.DD_ERR_DEVICE_CHECK
        want, tol = want_of(x, False)
        for _ in range(2):
            got, st = run(dd, x, ctx=ctx)
            assert st == 0 and (np.abs(got - want) <= tol).all()


def test_refusals(dd):
    import torch
    x = make_case(61, 1, 2, 4, 1, 16, 30, 10)
    with dd.Context(dd.Shape(1, 8, 2, D, 480, 16, 10, 1), max_misses=x["n_st"], hot_slots=x["n_hot"]) as ctx:
        q, out = tl.to_bf16(x["q"]), torch.zeros(1, 1, 8, D, device="cuda")
        p = [torch.from_numpy(x[n]).cuda() for n in ("Khot", "Vhot", "Kst", "Vst")]
        slot, cnt, idx = tl.to_i32(x["slot"]), tl.to_i32(x["cnt"]), tl.to_i32(x["idx"])
        n = tl.to_i32([5])
        good = [q, *p, slot, cnt, out]
        for i, v in ((0, None), (0, q.float()), (1, None), (2, p[0][:1]), (3, None), (4, p[1].float()), (5, None), (6, None),
                     (7, None), (7, out.bfloat16()), (7, out.cpu()), (0, q[..., ::2])):
            with pytest.raises((ValueError, TypeError, dd.DDError)):
                ctx.sparse_attn_decode_kv4(*good[:i], v, *good[i + 1:])
        tail = tl.to_bf16(x["Kt"])
        for kw in (dict(kv_len=n), dict(K_tail=tail), dict(V_tail=tail), dict(k_exp=n), dict(union_qmask=slot),
                   dict(kv_len=n.long(), union_idx=idx)):
            with pytest.raises((ValueError, TypeError, dd.DDError)):
                ctx.sparse_attn_decode_kv4(*good, **kw)
        assert ctx.launch_count() == 0
    with dd.Context(dd.Shape(0, 8, 2, D, 480, 16, 10, 1), max_misses=0) as ctx:
        ctx.sparse_attn_decode_kv4(q, None, None, None, None, slot, cnt, out)
        assert ctx.launch_count() == 0 and ctx.status() == 0


@pytest.mark.parametrize("n_heads", [4, 16, 64], ids=["nq4", "nq16", "nq64"])
def test_same_result_every_time_and_in_graphs(dd, n_heads):
    """Repeated, captured (two graphs of one context, replayed in turn) and run on another stream: the same bits."""
    import torch
    x = make_case(71, 2, 2, n_heads // 2, 2, 16, 400, 150, ragged=True)
    Hq = n_heads
    p = [torch.from_numpy(x[n]).cuda() for n in ("Khot", "Vhot", "Kst", "Vst")]
    q, slot, cnt = tl.to_bf16(x["q"]), tl.to_i32(x["slot"]), tl.to_i32(x["cnt"])
    kw = dict(union_qmask=torch.from_numpy(x["qmask"].reshape(-1)).cuda(), kv_len=tl.to_i32(x["length"]),
              union_idx=tl.to_i32(x["idx"]), K_tail=tl.to_bf16(x["Kt"]), V_tail=tl.to_bf16(x["Vt"]))
    with dd.Context(dd.Shape(2, Hq, 2, D, 6400, 16, 150, 2), max_misses=x["n_st"], hot_slots=x["n_hot"]) as ctx:
        outs = [torch.zeros(2, 2, Hq, D, device="cuda") for _ in range(4)]
        ctx.sparse_attn_decode_kv4(q, *p, slot, cnt, outs[0], **kw)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            ctx.sparse_attn_decode_kv4(q, *p, slot, cnt, outs[1], **kw)
        torch.cuda.current_stream().wait_stream(side)
        graphs = []
        for o in outs[2:]:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                ctx.sparse_attn_decode_kv4(q, *p, slot, cnt, o, **kw)
            graphs.append(g)
        for _ in range(3):
            for g in graphs:
                g.replay()
        assert ctx.status() == 0
        for o in outs[1:]:
            assert torch.equal(o, outs[0])
        assert outs[0].any()


def test_offsets_past_32_bits(dd):
    """Pages whose byte offsets pass 2^32: the pool's last slots."""
    import torch
    cs, n = 64, (1 << 32) // (64 * 72) + 8
    x = make_case(81, 1, 1, 4, 1, cs, 4, 4, p_hot=1.0, empty=0.0, ragged=False)
    pool = [torch.zeros(n, cs * 72, dtype=torch.uint8, device="cuda") for _ in range(2)]
    k = x["cnt"][0, 0]
    at = n - 1 - np.arange(k)
    for t, name in zip(pool, ("Khot", "Vhot")):
        t[torch.from_numpy(at).cuda()] = torch.from_numpy(x[name][x["slot"][0, 0, :k]]).cuda()
    out = torch.zeros(1, 1, 4, D, device="cuda")
    slot = x["slot"].copy()
    slot[0, 0, :k] = at
    with dd.Context(dd.Shape(1, 4, 1, D, 4 * cs, cs, 4, 1), max_misses=0, hot_slots=n) as ctx:
        ctx.sparse_attn_decode_kv4(tl.to_bf16(x["q"]), *pool, None, None, tl.to_i32(slot), tl.to_i32(x["cnt"]), out,
                                   k_exp=tl.to_i32(x["ke"]), v_exp=tl.to_i32(x["ve"]))
        assert ctx.status() == 0
    want, tol = want_of(x, False, mask=False)
    assert (np.abs(out.cpu().numpy() - want) <= tol).all()


# more units than a CTA has threads, and more units per CTA than it lists at a time
@pytest.mark.parametrize("B,Hkv,G", [(80, 8, 3), (96, 6, 20), (1280, 8, 4), (512, 8, 20), (512, 8, 12)])
def test_many_small_units(dd, B, Hkv, G):
    import torch
    cs, units, n = 16, B * Hkv, 64
    rng = np.random.default_rng(B)
    K, V = pages(rng, n, cs), pages(rng, n, cs)
    cnt = rng.integers(0, 3, units)
    slot = rng.integers(0, n, (units, 2))
    length = rng.integers(0, 2 * cs + 1, B)
    g = torch.Generator(device="cuda")
    g.manual_seed(B)
    q = torch.randn(B, 1, Hkv * G, D, generator=g, device="cuda").to(torch.bfloat16)
    out = torch.full((B, 1, Hkv * G, D), float("nan"), device="cuda")
    with dd.Context(dd.Shape(B, Hkv * G, Hkv, D, 2 * cs, cs, 2, 1), max_misses=0, hot_slots=n) as ctx:
        idx = tl.to_i32(np.tile([0, 1], (units, 1)))
        for _ in range(2):
            ctx.sparse_attn_decode_kv4(q, torch.from_numpy(K).cuda(), torch.from_numpy(V).cuda(), None, None, tl.to_i32(slot),
                                       tl.to_i32(cnt), out, union_idx=idx, kv_len=tl.to_i32(length))
            assert ctx.status() == 0
    dev64 = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()       # noqa: E731
    Kv, Vv = (dev64(oracle.kv4_values(p, np.zeros(n)))[dev64(slot)].flatten(1, 2) for p in (K, V))      # [units, 32, D]
    pos = torch.arange(2 * cs, device="cuda")
    seen = (pos < dev64(cnt)[:, None] * cs) & (pos < dev64(np.repeat(length, Hkv))[:, None])
    qd = q.double().view(units, G, D)
    x = (qd @ Kv.transpose(1, 2) * D ** -0.5).masked_fill(~seen[:, None], -np.inf)
    w = torch.nan_to_num(torch.softmax(x, -1), nan=0.0)
    want = w @ Vv
    # scores off by 128 * 2^-23 of the sum of magnitudes, twice in a weight, and 2^-18 for the rest (as above)
    dx = 128 * 2.0 ** -23 * (qd.abs() @ Kv.abs().transpose(1, 2)).amax(-1, keepdim=True) * D ** -0.5
    assert ((out.double().view(units, G, D) - want).abs() <= (2 * dx + 2.0 ** -18) * Vv.abs().max()).all()


@pytest.mark.parametrize("G", [4, 12, 30])
def test_pending_errors_stop_the_work_and_nothing_else(dd, G):
    """While the status word is set the call leaves its output alone, also where CTAs share units; then all is as before."""
    import torch
    x = make_case(91, 2, 2, G, 1, 16, 500, 400, p_hot=1.0, empty=0.0, ragged=False)
    p = [torch.from_numpy(x[n]).cuda() for n in ("Khot", "Vhot")]
    kw = dict(k_exp=tl.to_i32(x["ke"]), v_exp=tl.to_i32(x["ve"]))
    q, slot, cnt = tl.to_bf16(x["q"]), tl.to_i32(x["slot"]), tl.to_i32(x["cnt"])
    want, tol = want_of(x, False, mask=False)
    with dd.Context(dd.Shape(2, 2 * G, 2, D, 8000, 16, 400, 1), max_misses=0, hot_slots=x["n_hot"]) as ctx:
        for _ in range(2):
            bad = slot.clone()
            bad[0, 0, 3] = x["n_hot"]
            trash = torch.zeros(2, 1, 2 * G, D, device="cuda")
            ctx.sparse_attn_decode_kv4(q, *p, None, None, bad, cnt, trash, **kw)
            out = torch.full((2, 1, 2 * G, D), 7.0, device="cuda")
            ctx.sparse_attn_decode_kv4(q, *p, None, None, slot, cnt, out, **kw)
            assert ctx.status() == dd.DD_ERR_DEVICE_CHECK and (out == 7.0).all()
            ctx.sparse_attn_decode_kv4(q, *p, None, None, slot, cnt, out, **kw)
            assert ctx.status() == 0
            assert (np.abs(out.cpu().numpy() - want) <= tol).all()


def test_two_contexts_at_once(dd):
    """Calls of two contexts on two streams, overlapping: each context has its own workspace."""
    import torch
    cases = [make_case(95, 2, 2, 4, 1, 16, 300, 250), make_case(96, 2, 2, 20, 1, 16, 300, 250)]
    wants = [want_of(x, False) for x in cases]
    ctxs, args, outs, streams = [], [], [], []
    for x in cases:
        G = x["G"]
        ctxs.append(dd.Context(dd.Shape(2, 2 * G, 2, D, 4800, 16, 250, 1), max_misses=x["n_st"], hot_slots=x["n_hot"]))
        args.append(([tl.to_bf16(x["q"])] + [torch.from_numpy(x[n]).cuda() for n in ("Khot", "Vhot", "Kst", "Vst")]
                     + [tl.to_i32(x["slot"]), tl.to_i32(x["cnt"])],
                     dict(union_qmask=torch.from_numpy(x["qmask"].reshape(-1)).cuda(), kv_len=tl.to_i32(x["length"]),
                          union_idx=tl.to_i32(x["idx"]), miss_count=tl.to_i32([x["n_st"]]), k_exp=tl.to_i32(x["ke"]),
                          v_exp=tl.to_i32(x["ve"]))))
        outs.append(torch.zeros(2, 1, 2 * G, D, device="cuda"))
        streams.append(torch.cuda.Stream())
    torch.cuda.synchronize()
    for _ in range(20):
        for c, (a, kw), o, s in zip(ctxs, args, outs, streams):
            c.sparse_attn_decode_kv4(*a, o, stream=s, **kw)
    for c, o, (want, tol) in zip(ctxs, outs, wants):
        assert c.status() == 0
        assert (np.abs(o.cpu().numpy() - want) <= tol).all()
        c.close()


@pytest.mark.parametrize("cs,host", [(16, True), (64, False)])
def test_decode_loop(dd, cs, host):
    """As a decode loop uses them: the prompt's rows appended in 4 bits, landmarks from the expanded chunks, then steps of
    two queries (rotated) that score, select, resolve, gather the missing 4-bit chunks, attend with their own rows as
    tails, and append what was accepted."""
    import torch
    B, Hkv, G, n_q, C, k = 2, 2, 4, 2, 24, 6
    Hq, L = Hkv * G, C * cs
    rng = np.random.default_rng(cs)
    shape = dd.Shape(B, Hq, Hkv, D, L, cs, k, n_q)
    total = B * Hkv * C
    freq = oracle.rope_frequencies(D, 1e4)
    rope = dd.rope_table(D)
    bits = lambda *s: synth.f32_to_bf16(rng.standard_normal(s).astype(np.float32))   # noqa: E731
    with dd.Context(shape, max_misses=total, hot_slots=total) as ctx:
        home = [torch.zeros(total, cs * 72, dtype=torch.uint8) for _ in range(2)]
        home = [h.pin_memory() if host else h.cuda() for h in home]
        pool = [torch.zeros(total, cs * 72, dtype=torch.uint8, device="cuda") for _ in range(2)]
        res = np.where(np.arange(total) % 3 == 0, rng.permutation(total), -1).astype(np.int32)
        resd = tl.to_i32(res)
        cache = dict(kv_format=dd.KV_4BIT, rope=rope, Kh=home[0], Vh=home[1], Khot=pool[0], Vhot=pool[1], resident_slot=resd)
        T = L - 3 * cs + 5
        lens = np.array([T, T - cs - 3], np.int32)
        ctx.append_kv(tl.to_bf16(bits(B, T, Hkv, D)), tl.to_bf16(bits(B, T, Hkv, D)), tl.to_i32([0] * B),
                      new_len=tl.to_i32(lens), **cache)
        wide = [torch.zeros(total, cs, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        st = [torch.zeros(total, cs * 72, dtype=torch.uint8, device="cuda") for _ in range(2)]
        i32 = dict(dtype=torch.int32, device="cuda")
        U = shape.umax
        sel, attn = (torch.zeros(B * n_q * Hkv * k, **i32) for _ in range(2))
        u_idx, u_slot = (torch.zeros(B * Hkv * U, **i32) for _ in range(2))
        u_qm = torch.zeros(B * Hkv * U, dtype=torch.uint8, device="cuda")
        u_cnt, misses, n_miss = torch.zeros(B * Hkv, **i32), torch.zeros(total, **i32), torch.zeros(1, **i32)
        lm = torch.zeros(total * D, dtype=torch.bfloat16, device="cuda")
        scores = torch.zeros(B * n_q * Hkv * C, device="cuda")
        for step in range(3):
            every = torch.arange(total, **i32)
            ctx.gather_kv4(home[0], home[1], every, torch.tensor([total], **i32), wide[0], wide[1], expand=True)
            ctx.build_landmarks(wide[0], lm)
            q, kt, vt = bits(B, n_q, Hq, D), bits(B, n_q, Hkv, D), bits(B, n_q, Hkv, D)
            qd, ktd = torch.zeros(B, n_q, Hq, D, dtype=torch.bfloat16, device="cuda"), tl.to_bf16(kt)
            lend = tl.to_i32(lens)
            ctx.rope(rope, tl.to_bf16(q), qd, lend)
            turned = torch.zeros_like(ktd)
            ctx.rope(rope, ktd, turned, lend)
            ctx.score_landmarks(qd, lm, scores)
            ctx.select_topk(scores, sel)
            ctx.resolve_union(sel, resd, u_idx, u_slot, u_qm, u_cnt, misses, n_miss, attn)
            ctx.gather_kv4(home[0], home[1], misses, n_miss, st[0], st[1])
            out = torch.full((B, n_q, Hq, D), float("nan"), device="cuda")
            ctx.sparse_attn_decode_kv4(qd, pool[0], pool[1], st[0], st[1], u_slot, u_cnt, out, union_qmask=u_qm,
                                       union_idx=u_idx, kv_len=lend, miss_count=n_miss, K_tail=turned,
                                       V_tail=tl.to_bf16(vt))
            assert ctx.status() == 0
            # from the home cache's values and the library's own selection
            Kv, Vv = (oracle.kv4_values(h.cpu().numpy(), np.zeros(total)).reshape(B, Hkv, L, D) for h in home)
            s = sel.cpu().numpy().reshape(B, n_q, Hkv, k)
            qr = oracle.bf16_decode(tl.from_bf16(qd))
            kr, vr = oracle.bf16_decode(tl.from_bf16(turned)), oracle.bf16_decode(vt)
            exact = oracle.rope_rotate(oracle.bf16_decode(q), lens[:, None] + np.arange(n_q), freq, True)
            assert np.abs(qr - exact).max() <= 2.0 ** -8 * np.abs(exact).max()
            got = out.cpu().numpy()
            for b in range(B):
                for j in range(n_q):
                    for h in range(Hq):
                        g = h // G
                        at = (s[b, j, g][:, None] * cs + np.arange(cs)).reshape(-1)
                        at = at[at < lens[b]]
                        Kj = np.concatenate([Kv[b, g, at], kr[b, :j + 1, g]])
                        Vj = np.concatenate([Vv[b, g, at], vr[b, :j + 1, g]])
                        want = oracle.attention_rows(qr[b, j, h], Kj, Vj, D ** -0.5)
                        dx = 128 * 2.0 ** -23 * (np.abs(Kj) @ np.abs(qr[b, j, h])).max() * D ** -0.5
                        assert np.abs(got[b, j, h] - want).max() <= (2 * dx + 2.0 ** -18) * np.abs(Vj).max()
            accepted = np.array([n_q, 1], np.int32)
            before = [h.cpu().clone() for h in home]
            ctx.append_kv(ktd, tl.to_bf16(vt), lend, new_len=tl.to_i32(accepted), **cache)
            assert ctx.status() == 0
            for w in range(2):                                     # resident copies and home agree, and only new rows changed
                h = home[w].cpu()
                assert (h != before[w]).any(-1).sum() <= Hkv * 2 * B
                on = torch.from_numpy(np.flatnonzero(res >= 0))
                assert torch.equal(pool[w].cpu()[torch.from_numpy(res[res >= 0]).long()], h[on])
            lens = lens + accepted
