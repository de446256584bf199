"""Cases of the operators over lists of cached chunks, their 64-bit results and the error
that each output may have.  Used by the GPU tests; the CPU tests check it against closed forms."""
import numpy as np

import oracle
from sparse_kv_offload_gb300 import synth

D = 128


def bf16(x):
    """fp64 -> bf16 bits and their values."""
    bits = synth.f32_to_bf16(np.asarray(x, np.float32))
    return bits, oracle.bf16_decode(bits)


def make_case(seed, B, Hkv, G, T, cs, C, kept=1.0, ragged=True, staged=0.0, start=None, lens=None, qscale=1.0):
    """Requests of up to T new tokens behind others, a share `kept` of the earlier chunks in the cache."""
    rng = np.random.default_rng(seed)
    L = C * cs
    lens = rng.integers(0 if ragged else T, T + 1, B) if lens is None else np.array(lens)
    start = rng.integers(0, L - T + 1, B) if start is None else np.array(start)
    idx = np.zeros((B, Hkv, C), np.int32)
    cnt = np.zeros((B, Hkv), np.int32)
    slot = np.zeros((B, Hkv, C), np.int32)
    n_hot = n_st = 0
    for b in range(B):
        old, end = start[b] // cs, -(-(start[b] + lens[b]) // cs)
        for g in range(Hkv):
            here = [c for c in range(C) if (c < old and rng.random() < kept) or old <= c < end]
            cnt[b, g] = len(here)
            idx[b, g, :len(here)] = here
            for i in range(len(here)):
                if rng.random() < staged:
                    slot[b, g, i], n_st = -1 - n_st, n_st + 1
                else:
                    slot[b, g, i], n_hot = n_hot, n_hot + 1
    hot = n_hot + 2
    ph = rng.permutation(hot).astype(np.int32)
    slot = np.where(slot >= 0, ph[np.clip(slot, 0, hot - 1)], slot).astype(np.int32)
    x = dict(B=B, Hkv=Hkv, G=G, T=T, cs=cs, C=C, lens=lens.astype(np.int32), start=start.astype(np.int32), idx=idx,
             cnt=cnt, slot=slot, n_hot=hot, n_st=max(1, n_st), has_st=n_st > 0)
    x["q"], x["q64"] = bf16(rng.standard_normal((B, T, Hkv * G, D)) * qscale)
    for name, n in (("Khot", hot), ("Vhot", hot), ("Kst", max(1, n_st)), ("Vst", max(1, n_st))):
        x[name], x[name + "64"] = bf16(rng.standard_normal((n, cs, D)))
    return x


def unit_rows(x, b, g):
    n = x["cnt"][b, g]
    i, s = x["idx"][b, g, :n], x["slot"][b, g, :n]
    K, pos = oracle.list_rows(x["Khot64"], x["Kst64"], i, s, x["cs"])
    V, _ = oracle.list_rows(x["Vhot64"], x["Vst64"], i, s, x["cs"])
    return K, V, pos


def score_error(q, K, scale, lse=0.0):
    """Bound on the absolute error of a score q.K*scale in natural units: 128 exact products added in fp32, 2^-23 of
    the sum of their magnitudes a step (truncation allowed for), one rounding of the factor, of the
    scaled score and of the reference each, 2^-24 of their magnitude."""
    mag = (np.abs(K) @ np.abs(q)).max() * scale if len(K) else 0.0
    return 128 * 2.0 ** -23 * mag + 4 * 2.0 ** -24 * (mag + abs(lse))


def want_extend(x, scale=D ** -0.5):
    """(out, lse, bound on |out - exact|, bound on |lse - exact|); nothing (NaN) where a row is padding."""
    B, T, H, G = x["B"], x["T"], x["Hkv"], x["G"]
    out = np.full((B, T, H * G, D), np.nan)
    lse = np.full((B, T, H * G), np.nan)
    tol, ltol = np.zeros(out.shape), np.zeros(lse.shape)
    for b in range(B):
        n = x["lens"][b]
        for g in range(H):
            K, V, pos = unit_rows(x, b, g)
            hs = slice(g * G, (g + 1) * G)
            o, z = oracle.extend_attention(x["q64"][b, :n, hs], int(x["start"][b]), K, V, pos, scale)
            out[b, :n, hs], lse[b, :n, hs] = o, z
            for t in range(n):
                see = pos <= x["start"][b] + t
                for h in range(G):
                    if not see.any():
                        continue
                    q = x["q64"][b, t, g * G + h]
                    with np.errstate(invalid="ignore"):
                        w = np.exp(K[see] @ q * scale - z[t, h])
                        dx = score_error(q, K[see], scale, z[t, h])
                        # a weight: its score's error, 2^-20 for the exponential (2^-22) and fp32 sums, then bf16's
                        # half step, 2^-8 of it; the sum's own rounding, 2^-8 of the output
                        av = w @ np.abs(V[see])
                        tol[b, t, g * G + h] = (2 * dx + 2.0 ** -20 + 2.0 ** -8) * av + 2.0 ** -8 * np.abs(o[t, h])
                    ltol[b, t, g * G + h] = dx + 2.0 ** -20 + 2.0 ** -22 * abs(z[t, h])
    return out, lse, tol, ltol


def tensors(x, dev="cuda"):
    import torch

    def bf(a):
        return torch.from_numpy(np.ascontiguousarray(a).view(np.int16)).view(torch.bfloat16).to(dev)

    i = {k: torch.from_numpy(np.ascontiguousarray(x[k])).to(dev) for k in ("idx", "slot", "cnt", "lens", "start")}
    i.update({k: bf(x[k]) for k in ("q", "Khot", "Vhot", "Kst", "Vst")})
    return i


def context(dd, x, k=None):
    H, C, cs = x["Hkv"], x["C"], x["cs"]
    return dd.Context(dd.Shape(x["B"], H * x["G"], H, D, C * cs, cs, k or C, 1), max_misses=x["n_st"] if x["has_st"] else 0,
                      hot_slots=x["n_hot"])


def run_extend(dd, x, ctx=None, t=None, scale=0.0, lse=True, **kw):
    """(out fp64, lse fp64, raw out bits): buffers start as NaN."""
    import torch
    made = ctx is None
    ctx = ctx or context(dd, x)
    t = t or tensors(x)
    B, T, H = x["B"], x["T"], x["Hkv"] * x["G"]
    out = torch.full((B, T, H, D), float("nan"), device="cuda", dtype=torch.bfloat16)
    z = torch.full((B, T, H), float("nan"), device="cuda") if lse else None
    st = dict(Kst=t["Kst"], Vst=t["Vst"]) if x["has_st"] else {}
    ctx.extend_attn(t["q"], t["start"], t["Khot"], t["Vhot"], t["idx"], t["slot"], t["cnt"], out, new_len=t["lens"],
                    lse=z, softmax_scale=scale, **st, **kw)
    status = ctx.status()
    if made:
        ctx.close()
    return out.double().cpu().numpy(), (z.double().cpu().numpy() if lse else None), status


def check_extend(got, want):
    """Every row that is a token within its bound, padding untouched (NaN), empty rows exactly 0 and -inf."""
    out, lse = got[:2]
    w_out, w_lse, tol, ltol = want
    pad = np.isnan(w_lse)
    assert np.isnan(out[pad]).all()
    off = np.abs(out - w_out)[~pad]
    assert (off <= tol[~pad]).all(), float((off / np.maximum(tol[~pad], 1e-300)).max())
    if lse is not None:
        assert np.isnan(lse[pad]).all()
        empty = np.isneginf(w_lse)
        assert (np.isneginf(lse) == empty).all()
        some = ~pad & ~empty
        off = np.abs(lse - w_lse)[some]
        assert (off <= ltol[some]).all(), float((off / ltol[some]).max())


def want_weights(x, lse, window=0, decay=1.0, w0=None, scale=D ** -0.5):
    """(weights [B, Hkv, C], bound on their error) from the log-sum-exps given (fp32 values)."""
    B, H, G, C = x["B"], x["Hkv"], x["G"], x["C"]
    w = np.array(w0, np.float64)
    tol = np.zeros(w.shape)
    for b in range(B):
        n = x["lens"][b]
        first = max(0, n - window) if window else 0
        for g in range(H):
            K, _, pos = unit_rows(x, b, g)
            hs = slice(g * G, (g + 1) * G)
            got = oracle.chunk_weights(x["q64"][b, :n, hs], int(x["start"][b]), lse[b, :n, hs], K, pos, x["cs"], scale, first)
            at = x["idx"][b, g, :x["cnt"][b, g]]
            old = decay * w[b, g, at] if decay else 0.0
            w[b, g, at] = old + got
            # every weight: its score's error and 2^-21 of the exponential; sums of positive numbers in fp32, a few
            # dozen additions one after another at most in these cases and a tree of the rest: 2^-24 each
            dx = max([score_error(q, K, scale, z) for t in range(first, n) for q, z in
                      zip(x["q64"][b, t, hs], lse[b, t, hs]) if np.isfinite(z)], default=0.0)
            tol[b, g, at] = (dx + 2.0 ** -21 + 256 * 2.0 ** -24) * got + 2.0 ** -23 * np.abs(w[b, g, at])
    return w, tol


def run_weights(dd, x, lse, w0, window=0, decay=1.0, ctx=None, t=None, scale=0.0, **kw):
    """(weights fp64, status)."""
    import torch
    made = ctx is None
    ctx = ctx or context(dd, x)
    t = t or tensors(x)
    w = torch.from_numpy(np.asarray(w0, np.float32)).cuda()
    z = torch.from_numpy(np.asarray(lse, np.float32)).cuda()
    st = dict(Kst=t["Kst"]) if x["has_st"] else {}
    ctx.chunk_weights(t["q"], t["start"], z, t["Khot"], t["idx"], t["slot"], t["cnt"], w, new_len=t["lens"], window=window,
                      decay=decay, softmax_scale=scale, **st, **kw)
    status = ctx.status()
    if made:
        ctx.close()
    return w.double().cpu().numpy(), status


def lse_of(x, scale=D ** -0.5):
    """The rows' exact log-sum-exps as fp32; NaN for padding, which nothing may look at."""
    return want_extend(x, scale)[1].astype(np.float32)
