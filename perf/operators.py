"""Operators on the KV cache: rotary positions, appending to the paged cache, and
attention over a cache held in 4 bits, as cases to be timed and compared.

``own = False``: ``run`` computes in elementary torch operations.  ``own = True``:
``run`` makes the library's calls.

A 4-bit row of 128 values is 64 bytes of e2m1 codes (byte i: value 2i in the low
nibble, 2i+1 in the high one) and 8 e4m3 scales, one per 16 values.  Rows are
stored in blocks of 16: 16 x 64 bytes of codes, then 16 x 8 of scales (1152
bytes); a chunk of cs rows is cs/16 such blocks.  A value is code * scale * 2^e, e
the head's exponent.
"""
import functools
import math

import torch

own = False

D = 128
ROW4 = 72                      # bytes of a 4-bit row
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ----------------------------------------------------------------------- cases
def _rope(name, B, T, H, rot, layout, scaling, far, strided=False):
    return dict(name=name, op="rope", B=B, T=T, H=H, rot=rot, layout=layout, scaling=scaling, far=far, strided=strided)


def _append(name, bits, B, T, Hkv, cs, L, rot, layout, scaling, ragged):
    return dict(name=name, op="append", bits=bits, B=B, T=T, Hkv=Hkv, cs=cs, L=L, rot=rot, layout=layout,
                scaling=scaling, ragged=ragged)


def _attn(name, B, Hq, Hkv, n_q, cs, C, k, tails, ragged, staged=0.0):
    return dict(name=name, op="attn4", B=B, Hq=Hq, Hkv=Hkv, n_q=n_q, cs=cs, C=C, k=k, tails=tails, ragged=ragged,
                staged=staged)


def listed():
    return [
        # the two queries of a decode step of the Llama-3-8B layer (16 requests): latency
        _rope("rope step", 16, 2, 32, 128, "half", "parts", 32768),
        # queries of four prompts of 4K, half of the head rotated, a slice of a fused projection
        _rope("rope prefill", 4, 4096, 64, 64, "interleaved", "none", 524288, strided=True),
        # accepted tokens of a speculative step (1 to 5 a request) into resident pages
        _append("append step", 16, 32, 5, 8, 16, 8192, 128, "half", "none", True),
        # ragged prompts of up to 8K tokens into pages
        _append("append prefill", 16, 4, 8192, 8, 32, 8192, 128, "half", "parts", True),
        # one token a request into the 4-bit home cache
        _append("append 4-bit step", 4, 16, 1, 8, 16, 4096, 128, "half", "linear", False),
        # long prompts into the 4-bit home cache
        _append("append 4-bit prefill", 4, 2, 32768, 8, 64, 32768, 96, "half", "none", True),
        # one short request: latency
        _attn("attn 4-bit single", 1, 32, 8, 1, 16, 256, 16, False, False),
        # the Llama-3-8B layer's sparse step, its own rows as tails
        _attn("attn 4-bit 2 queries", 16, 32, 8, 2, 16, 2048, 64, True, False),
        # the 32B-class layer with five queries (40 query vectors a KV head)
        _attn("attn 4-bit 5 queries", 32, 64, 8, 5, 16, 2048, 128, True, False),
        # odd head ratio and lengths, half of the chunks in staging
        _attn("attn 4-bit odd", 3, 35, 7, 3, 32, 333, 77, True, True, staged=0.5),
        # every page of long contexts, one token a request
        _attn("attn 4-bit whole cache", 8, 32, 8, 1, 64, 2048, 2048, False, True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "append4", "attn4", "attn4"])
    layout = rng.choice(["half", "interleaved"])
    scaling = rng.choice(["none", "linear", "ntk", "parts"])
    rot = rng.choice([32, 64, 96, 128])
    if op == "rope":
        H = rng.randint(1, 64)
        rows = _log(rng, 8, 16384)
        B = rng.randint(1, min(32, rows))
        c = _rope("", B, max(1, rows // B), H, rot, layout, scaling, _log(rng, 128, 1 << 20), rng.random() < 0.5)
    elif op in ("append", "append4"):
        B, Hkv, cs = rng.randint(1, 32), rng.randint(1, 16), rng.choice([16, 32, 64])
        T = _log(rng, 1, 2 * 32768 // B * 8 // max(8, Hkv))
        L = -(-(T + rng.randint(0, 2000)) // cs) * cs
        c = _append("", 4 if op == "append4" else 16, B, T, Hkv, cs, L, rot, layout, scaling, rng.random() < 0.7)
    else:
        n_q = rng.randint(1, 8)
        G = rng.randint(1, min(16, 64 // n_q))
        cs, Hkv, B = rng.choice([16, 32, 64]), rng.randint(1, 12), rng.randint(1, 32)
        C = _log(rng, 4, 4096)
        k = min(C, _log(rng, 1, 2048))
        while B * Hkv * min(C, n_q * k) * cs * n_q * G > 1 << 26:
            k = max(1, k // 2)
            C = max(k, C // 2)
            B = max(1, B - 1)
        c = _attn("", B, Hkv * G, Hkv, n_q, cs, C, k, rng.random() < 0.5, rng.random() < 0.7,
                  rng.choice([0.0, 0.0, 0.3]))
    del c["name"]
    return c


# ----------------------------------------------------- frequencies (host, 64 bits)
BASE = 500000.0
SCALING = {"none": dict(factor=1.0), "linear": dict(factor=4.0), "ntk": dict(factor=4.0),
           "parts": dict(factor=8.0, orig_len=8192.0, beta_fast=32.0, beta_slow=1.0)}


def _frequencies(rot, scaling):
    """(radians per position of each pair, factor on cos and sin)."""
    p = SCALING[scaling]
    base = BASE * p["factor"] ** (rot / (rot - 2.0)) if scaling == "ntk" else BASE
    f = base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    if scaling == "linear":
        return f / p["factor"], 1.0
    if scaling != "parts":
        return f, 1.0
    # pairs that turn more than beta_fast times within orig_len keep their frequency, those that turn
    # less than beta_slow times have it divided, with a ramp over the pairs' numbers between the two
    at = [rot * math.log(p["orig_len"] / (b * 2.0 * math.pi)) / (2.0 * math.log(BASE)) for b in (p["beta_fast"], p["beta_slow"])]
    lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
    ramp = ((torch.arange(rot // 2, dtype=torch.float64) - lo) / max(hi - lo, 1e-3)).clamp(0.0, 1.0)
    return f / p["factor"] * ramp + f * (1.0 - ramp), 0.1 * math.log(p["factor"]) + 1.0


# ----------------------------------------------------------------- 4-bit pages
def _blocks(pages):
    """Views of [n, cs*72] pages: codes [n, cs/16, 16, 64], scale bytes [n, cs/16, 16, 8]."""
    b = pages.view(pages.shape[0], -1, 16 * ROW4)
    return b[:, :, :1024].unflatten(2, (16, 64)), b[:, :, 1024:].unflatten(2, (16, 8))


def _decode(codes, scales, exps, to=torch.float32):
    """codes uint8 [..., 64], scale bytes [..., 8], exps broadcast against [...]: values [..., 128]."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=to, device=codes.device)
    v = torch.stack((table[(codes & 15).long()], table[(codes >> 4).long()]), -1).flatten(-2)
    s = scales.contiguous().view(torch.float8_e4m3fn).to(to) * torch.exp2(exps.to(to)).unsqueeze(-1)
    return (v.unflatten(-1, (8, 16)) * s.unsqueeze(-1)).flatten(-2)


def _encode(x, exps):
    """x float [..., 128] (bf16 values): codes [..., 64] and scale bytes [..., 8]."""
    g = (x.float() * torch.exp2(-exps.float()).unsqueeze(-1)).unflatten(-1, (8, 16))
    s8 = (g.abs().amax(-1) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = s8.float().unsqueeze(-1)
    a = torch.where(s > 0, g.abs() / s, torch.zeros((), device=x.device))
    n = (a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)
    n = (n + 8 * (g < 0).to(torch.uint8)).flatten(-2)
    return n[..., 0::2] | (n[..., 1::2] << 4), s8.view(torch.uint8)


def _bf16(x):
    """Doubles rounded once to bf16: an inexact float keeps its last bit set, so no tie appears on the way."""
    y = x.float()
    bits = y.view(torch.int32)
    off = y.double() - x
    bits = torch.where((off != 0) & ((off > 0) == (y > 0)), bits - 1, bits)
    return torch.where(off != 0, bits | 1, bits).view(torch.float32).to(torch.bfloat16)


def _make_pages(x, exps):
    """Pages [n, cs*72] of values x [n, cs, 128], exps [n, cs]."""
    pages = torch.empty(x.shape[0], x.shape[1] * ROW4, dtype=torch.uint8, device=x.device)
    codes, scales = _encode(x, exps)
    b, s = _blocks(pages)
    b.copy_(codes.unflatten(1, (-1, 16)))
    s.copy_(scales.unflatten(1, (-1, 16)))
    return pages


# --------------------------------------------------------------------- prepare
def _heads(n, g):
    """Channel gains of n heads: a few channels are far larger than the rest, as in keys."""
    return torch.exp(0.7 * torch.randn(n, D, generator=g, device="cuda"))


@functools.lru_cache(maxsize=None)
def _context(B, Hq, Hkv, L, cs, k, n_q, max_misses, hot_slots):
    """A program makes one context per shape and keeps it."""
    from sparse_kv_offload_gb300 import dd
    return dd.Context(dd.Shape(B, Hq, Hkv, D, L, cs, k, n_q), max_misses=max_misses, hot_slots=hot_slots)


@functools.lru_cache(maxsize=None)
def _table(rot, layout, scaling):
    from sparse_kv_offload_gb300 import dd
    kind = {"none": dd.ROPE_PLAIN, "linear": dd.ROPE_LINEAR, "ntk": dd.ROPE_NTK, "parts": dd.ROPE_BY_PARTS}[scaling]
    return dd.rope_table(rot, base=BASE, layout={"half": dd.ROPE_HALF, "interleaved": dd.ROPE_INTERLEAVED}[layout],
                         scaling=kind, **SCALING[scaling])


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"rope": _prepare_rope, "append": _prepare_append, "attn4": _prepare_attn}[case["op"]](case, g)
    s["case"] = case
    return s


def _prepare_rope(c, g):
    B, T, H = c["B"], c["T"], c["H"]
    wide = H + 16 if c["strided"] else H      # the queries lie in front of keys and values
    x = torch.randn(B, T, wide, D, generator=g, device="cuda").to(torch.bfloat16)[:, :, :H]
    pos = torch.randint(0, max(1, c["far"] - T), (B,), generator=g, device="cuda", dtype=torch.int32)
    f, m = _frequencies(c["rot"], c["scaling"])
    s = dict(x=x, start=pos, freq=f.cuda(), gain=m, out=torch.empty(B, T, H, D, dtype=torch.bfloat16, device="cuda"))
    if own:
        L = -(-max(c["far"], 64) // 64) * 64
        s.update(ctx=_context(B, H, H, L, 64, 1, 1, 0, 0), rope=_table(c["rot"], c["layout"], c["scaling"]))
    return s


def _prepare_append(c, g):
    B, T, H, cs, L = c["B"], c["T"], c["Hkv"], c["cs"], c["L"]
    C = L // cs
    gain = _heads(H, g)
    k = (torch.randn(B, T, H, D, generator=g, device="cuda") * gain).to(torch.bfloat16)
    v = (torch.randn(B, T, H, D, generator=g, device="cuda") * 0.2).to(torch.bfloat16)
    if c["ragged"]:
        n = torch.randint(min(T, T // 2 + 1), T + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
        start = (torch.rand(B, generator=g, device="cuda") * (L - n + 1)).to(torch.int32).minimum(L - n)
    else:
        n = torch.full((B,), T, dtype=torch.int32, device="cuda")
        start = torch.randint(0, L - T + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    f, m = _frequencies(c["rot"], c["scaling"])
    s = dict(k=k, v=v, n=n, start=start, freq=f.cuda(), gain=m)
    if c["bits"] == 16:
        # a pool of pages, the chunks of all requests in any order
        s["slot"] = torch.randperm(B * H * C, generator=g, device="cuda").to(torch.int32).view(B, H, C)
        s["K"] = torch.randn(B * H * C, cs, D, generator=g, device="cuda", dtype=torch.bfloat16)
        s["V"] = torch.randn(B * H * C, cs, D, generator=g, device="cuda", dtype=torch.bfloat16)
        hot, misses = B * H * C, 0
    else:
        # the home cache, a page for every chunk, holding earlier rows
        s["ke"] = torch.randint(-1, 3, (H,), generator=g, device="cuda", dtype=torch.int32)
        s["ve"] = torch.randint(-4, -1, (H,), generator=g, device="cuda", dtype=torch.int32)
        old = torch.randn(B * H * C, cs, D, generator=g, device="cuda")
        zero = torch.zeros(1, 1, device="cuda").expand(B * H * C, cs)
        s["K"], s["V"] = _make_pages(old, zero), _make_pages(old.flip(0), zero)
        # the chunks that the new rows touch, as the gather's list
        first, last = start.long() // cs, (start + n - 1).long() // cs
        at = torch.arange(C, device="cuda")
        hit = (at >= first[:, None]) & (at <= last[:, None])
        s["touched"] = hit[:, None].expand(B, H, C).reshape(-1).nonzero()[:, 0].to(torch.int32)
        s["count"] = torch.tensor([s["touched"].numel()], dtype=torch.int32, device="cuda")
        hot, misses = 0, B * H * min(C, (T + cs - 2) // cs + 1)
        s["Kx"] = torch.zeros(misses, cs, D, dtype=torch.bfloat16, device="cuda")
        s["Vx"] = torch.zeros(misses, cs, D, dtype=torch.bfloat16, device="cuda")
    if own:
        s.update(ctx=_context(B, H, H, L, cs, 1, 1, misses, hot), rope=_table(c["rot"], c["layout"], c["scaling"]))
    return s


def _prepare_attn(c, g):
    B, Hq, H, n_q, cs, C, k = c["B"], c["Hq"], c["Hkv"], c["n_q"], c["cs"], c["C"], c["k"]
    G, U = Hq // H, min(C, n_q * k)
    dev = "cuda"
    # selections of a step: the queries largely agree on their chunks
    if k < C:
        score = torch.randn(B, H, 1, C, generator=g, device=dev) + 0.5 * torch.randn(B, H, n_q, C, generator=g, device=dev)
        sel = torch.zeros(B, H, n_q, C, dtype=torch.bool, device=dev).scatter_(-1, score.topk(k, -1).indices, True)
    else:
        sel = torch.ones(B, H, n_q, C, dtype=torch.bool, device=dev)
    if c["ragged"] and k < C:   # a query of a unit here and there has an empty selection
        sel &= torch.rand(B, H, n_q, 1, generator=g, device=dev) > 0.1
    bit = (1 << torch.arange(n_q, device=dev)).view(1, 1, n_q, 1)
    mask = (sel * bit).sum(2)
    cnt = (mask > 0).sum(-1)
    idx = torch.sort((mask == 0).to(torch.uint8), dim=-1, stable=True).indices[..., :U]
    used = torch.arange(U, device=dev) < cnt[..., None]
    idx = torch.where(used, idx, 0)
    qmask = torch.where(used, mask.gather(-1, idx), 0)
    # pages: most resident in the pool in any order, a share in staging
    n = B * H * U
    staged = torch.rand(B, H, U, generator=g, device=dev) < c["staged"]
    slot = torch.randperm(n, generator=g, device=dev).view(B, H, U)
    slot = torch.where(staged, -1 - slot, slot)
    gain = _heads(1, g)[0]
    ke = torch.randint(-1, 2, (H,), generator=g, device=dev, dtype=torch.int32)
    ve = torch.randint(-4, -1, (H,), generator=g, device=dev, dtype=torch.int32)
    zero = torch.zeros(1, 1, device=dev)

    def pool(scale, rows):
        return _make_pages(torch.randn(rows, cs, D, generator=g, device=dev) * scale, zero.expand(rows, cs))

    length = torch.full((B,), C * cs, dtype=torch.int32, device=dev)
    if c["ragged"]:
        length = (length * (0.4 + 0.6 * torch.rand(B, generator=g, device=dev))).to(torch.int32).clamp(min=1)
    s = dict(q=torch.randn(B, n_q, Hq, D, generator=g, device=dev).to(torch.bfloat16), K=pool(0.7 * gain, n), V=pool(1.0, n),
             idx=idx.to(torch.int32), slot=slot.to(torch.int32), qmask=qmask.to(torch.uint8), cnt=cnt.to(torch.int32),
             length=length, ke=ke, ve=ve, out=torch.empty(B, n_q, Hq, D, device=dev))
    if c["staged"] > 0:
        s.update(Kst=pool(0.7 * gain, n), Vst=pool(1.0, n), misses=torch.tensor([n], dtype=torch.int32, device=dev))
    if c["tails"]:
        s.update(Kt=(torch.randn(B, n_q, H, D, generator=g, device=dev) * gain).to(torch.bfloat16),
                 Vt=(torch.randn(B, n_q, H, D, generator=g, device=dev) * 0.2).to(torch.bfloat16))
    if own:
        s["ctx"] = _context(B, Hq, H, C * cs, cs, k, n_q, n if c["staged"] > 0 else 0, n)
    return s


# -------------------------------------------------------------------------- run
def run(s):
    op = s["case"]["op"]
    if own:
        return {"rope": _own_rope, "append": _own_append, "attn4": _own_attn}[op](s)
    return {"rope": _plain_rope, "append": _plain_append, "attn4": _plain_attn}[op](s)


def _own_rope(s):
    s["ctx"].rope(s["rope"], s["x"], s["out"], s["start"])
    return s["out"]


def _own_append(s):
    ctx = s["ctx"]
    if s["case"]["bits"] == 16:
        ctx.append_kv(s["k"], s["v"], s["start"], new_len=s["n"], rope=s["rope"], Khot=s["K"], Vhot=s["V"],
                      resident_slot=s["slot"])
        return s["K"], s["V"]
    from sparse_kv_offload_gb300 import dd
    ctx.append_kv(s["k"], s["v"], s["start"], new_len=s["n"], rope=s["rope"], Kh=s["K"], Vh=s["V"],
                  kv_format=dd.KV_4BIT, k_exp=s["ke"], v_exp=s["ve"])
    ctx.gather_kv4(s["K"], s["V"], s["touched"], s["count"], s["Kx"], s["Vx"], expand=True, k_exp=s["ke"], v_exp=s["ve"])
    return s["Kx"], s["Vx"]


def _own_attn(s):
    s["ctx"].sparse_attn_decode_kv4(
        s["q"], s["K"], s["V"], s.get("Kst"), s.get("Vst"), s["slot"], s["cnt"], s["out"], union_qmask=s["qmask"],
        union_idx=s["idx"], kv_len=s["length"], miss_count=s.get("misses"), k_exp=s["ke"], v_exp=s["ve"],
        K_tail=s.get("Kt"), V_tail=s.get("Vt"))
    return s["out"]


def _rotated(x, start, freq, gain, layout):
    """x bf16 [B, T, H, 128]: the first 2 * len(freq) values of each row rotated, rounded once."""
    T, n = x.shape[1], freq.numel()
    turn = (start.double()[:, None] + torch.arange(T, device=x.device))[:, :, None, None] * freq
    cos, sin = torch.cos(turn) * gain, torch.sin(turn) * gain
    y = x[..., :2 * n].double()
    a, b = (y[..., :n], y[..., n:]) if layout == "half" else (y[..., 0::2], y[..., 1::2])
    a, b = a * cos - b * sin, b * cos + a * sin
    y = torch.cat((a, b), -1) if layout == "half" else torch.stack((a, b), -1).flatten(-2)
    return torch.cat((_bf16(y), x[..., 2 * n:]), -1)


def _plain_rope(s):
    return _rotated(s["x"], s["start"], s["freq"], s["gain"], s["case"]["layout"])


def _plain_append(s):
    c = s["case"]
    B, T, H, cs, C = c["B"], c["T"], c["Hkv"], c["cs"], c["L"] // c["cs"]
    k = _rotated(s["k"], s["start"], s["freq"], s["gain"], c["layout"])
    t = torch.arange(T, device="cuda")
    b, t = (t < s["n"][:, None]).nonzero(as_tuple=True)         # the rows that are there
    pos = s["start"][b].long() + t
    h = torch.arange(H, device="cuda")
    page = (b[:, None] * H + h) * C + (pos // cs)[:, None]       # [rows, H]
    row = (pos % cs)[:, None].expand_as(page)
    if c["bits"] == 16:
        page = s["slot"].view(-1)[page].long()
        s["K"][page, row] = k[b, t]
        s["V"][page, row] = s["v"][b, t]
        return s["K"], s["V"]
    out = []
    for cache, x, exps, to in (("K", k, s["ke"], "Kx"), ("V", s["v"], s["ve"], "Vx")):
        codes, scales = _encode(x[b, t], exps.expand(b.numel(), H))
        at_codes, at_scales = _blocks(s[cache])
        at_codes[page, row // 16, row % 16] = codes
        at_scales[page, row // 16, row % 16] = scales
        touched = s["touched"].long()
        at_codes, at_scales = _blocks(s[cache][touched])
        e = exps[touched // C % H].view(-1, 1, 1)
        s[to][:touched.numel()] = _decode(at_codes, at_scales, e.expand(at_codes.shape[:3])).flatten(1, 2).to(torch.bfloat16)
        out.append(s[to])
    return tuple(out)


def _plain_attn(s):
    c = s["case"]
    B, H, n_q, cs = c["B"], c["Hkv"], c["n_q"], c["cs"]
    U, G = s["slot"].shape[-1], c["Hq"] // c["Hkv"]
    slot = s["slot"].long()

    def rows(hot, staged, exps):
        pages = hot[slot.clamp(min=0).view(-1)]
        if staged is not None:
            pages = torch.where((slot < 0).view(-1, 1), staged[(-1 - slot).clamp(min=0).view(-1)], pages)
        codes, scales = _blocks(pages)
        e = exps.view(1, H, 1).expand(B, H, U).reshape(-1, 1, 1).expand(codes.shape[:3])
        return _decode(codes, scales, e).view(B, H, U * cs, D)

    pos = s["idx"].long()[..., None] * cs + torch.arange(cs, device="cuda")
    there = (torch.arange(U, device="cuda") < s["cnt"][..., None])[..., None] & (pos < s["length"].view(B, 1, 1, 1))
    seen = (s["qmask"].long()[:, :, None] >> torch.arange(n_q, device="cuda").view(1, 1, n_q, 1)) & 1 == 1
    seen = (seen[..., None] & there[:, :, None]).view(B, H, n_q, 1, U * cs)
    q = s["q"].float().view(B, n_q, H, G, D).transpose(1, 2)                   # [B, H, n_q, G, D]
    K, V = rows(s["K"], s.get("Kst"), s["ke"]), rows(s["V"], s.get("Vst"), s["ve"])
    x = (q.reshape(B, H, n_q * G, D) @ K.transpose(-1, -2)).view(B, H, n_q, G, -1)
    x = torch.where(seen, x / math.sqrt(D), torch.tensor(-math.inf, device="cuda"))
    if "Kt" in s:
        kt = s["Kt"].float().permute(0, 2, 3, 1)                               # [B, H, D, n_q]
        xt = (q.reshape(B, H, n_q * G, D) @ kt).view(B, H, n_q, G, n_q) / math.sqrt(D)
        late = torch.ones(n_q, n_q, dtype=torch.bool, device="cuda").triu(1)
        x = torch.cat((x, xt.masked_fill(late[:, None], -math.inf)), -1)
        V = torch.cat((V, s["Vt"].float().transpose(1, 2)), 2)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    o = (p.reshape(B, H, n_q * G, -1) @ V).view(B, H, n_q, G, D)
    o = torch.where(total > 0, o / total, torch.zeros((), device="cuda"))
    return o.transpose(1, 2).reshape(B, n_q, c["Hq"], D)


# ------------------------------------------------------------------------- work
def work(case):
    c = case
    if c["op"] == "rope":
        n = c["B"] * c["T"] * c["H"]
        return {"bytes": 4.0 * n * D, "flops": 3.0 * n * c["rot"]}
    if c["op"] == "append":
        n = c["B"] * c["T"] * c["Hkv"] * (0.75 if c["ragged"] and c["T"] > 1 else 1.0)
        if c["bits"] == 16:
            return {"bytes": n * 1024.0, "flops": 3.0 * n * c["rot"]}
        # the rows in and their codes out, then the touched chunks' codes in and their values out
        touched = c["B"] * c["Hkv"] * c["cs"] * max(1, -(-c["T"] // c["cs"]))
        touched = max(touched * (0.75 if c["ragged"] and c["T"] > c["cs"] else 1.0), n)
        return {"bytes": n * (512.0 + 144.0) + touched * (144.0 + 512.0), "flops": 6.0 * n * D}
    share = 1.0 if c["k"] == c["C"] else min(1.0, c["k"] / c["C"] * (1.0 + 0.3 * (c["n_q"] - 1)))
    rows = c["B"] * c["Hkv"] * min(c["C"] * share, c["n_q"] * c["k"]) * c["cs"]
    rows *= 0.7 if c["ragged"] else 1.0
    NQ = c["n_q"] * c["Hq"] // c["Hkv"]
    return {"bytes": rows * 2.0 * ROW4 + 6.0 * c["B"] * c["n_q"] * c["Hq"] * D, "flops": 4.0 * rows * NQ * D}


# ------------------------------------------------------------------------ exact
def exact(case, seed):
    """From the definitions, in 64 bits, request by request and head by head."""
    s = prepare(case, seed)
    return {"rope": _exact_rope, "append": _exact_append, "attn4": _exact_attn}[case["op"]](case, s)


def _exact_turn(x, start, s, layout):
    """x double [T, H, 128] of one request: rotation as multiplication of complex numbers."""
    n = s["freq"].numel()
    at = torch.arange(start, start + x.shape[0], dtype=torch.float64, device=x.device)
    unit = torch.polar(torch.full((1,), s["gain"], dtype=torch.float64, device=x.device), torch.outer(at, s["freq"]))
    i = torch.arange(n, device=x.device)
    re, im = (i, i + n) if layout == "half" else (2 * i, 2 * i + 1)
    z = torch.complex(x[..., re], x[..., im]) * unit[:, None]
    y = x.clone()
    y[..., re], y[..., im] = z.real, z.imag
    return y


def _exact_rope(c, s):
    starts = s["start"].tolist()
    return torch.stack([_exact_turn(s["x"][b].double(), starts[b], s, c["layout"]) for b in range(c["B"])])


def _exact_append(c, s):
    H, cs, C = c["Hkv"], c["cs"], c["L"] // c["cs"]
    four = c["bits"] == 4
    if four:
        def values(pages, e):
            codes, scales = _blocks(pages)
            heads = (torch.arange(pages.shape[0], device="cuda") // C % H)
            return _decode(codes, scales, e[heads].view(-1, 1, 1).expand(codes.shape[:3]), torch.float64).flatten(1, 2)
        K, V = values(s["K"], s["ke"]), values(s["V"], s["ve"])
    else:
        K, V = s["K"].double(), s["V"].double()
    K, V = K.view(-1, cs, D), V.view(-1, cs, D)
    starts, ns = s["start"].tolist(), s["n"].tolist()
    for b in range(c["B"]):
        pos = torch.arange(starts[b], starts[b] + ns[b], device="cuda")
        k = _exact_turn(s["k"][b, :ns[b]].double(), starts[b], s, c["layout"])
        v = s["v"][b, :ns[b]].double()
        if four:
            k, v = _exact_quant(_bf16(k).double(), s["ke"]), _exact_quant(v, s["ve"])
        for h in range(H):
            page = (b * H + h) * C + pos // cs
            page = page if four else s["slot"].view(-1)[page].long()
            K[page, pos % cs], V[page, pos % cs] = k[:, h], v[:, h]
    if not four:
        return K, V
    t, out = s["touched"].long(), []
    for src, like in ((K, s["Kx"]), (V, s["Vx"])):
        y = torch.zeros(like.shape, dtype=torch.float64, device="cuda")
        y[:t.numel()] = src[t]
        out.append(y)
    return tuple(out)


def _exact_quant(x, exps):
    """Nearest representable values: the scales among e4m3's numbers, the values among e2m1's, ties to even."""
    one = torch.exp2(exps.double()).view(1, -1, 1, 1)
    g = x.view(*x.shape[:-1], 8, 16) / one

    def nearest(v, table):
        hi = torch.searchsorted(table, v.contiguous()).clamp(max=table.numel() - 1)
        lo = (hi - 1).clamp(min=0)
        up, down = table[hi] - v, v - table[lo]
        return table[torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)]

    e4m3 = torch.arange(127, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn).double()
    s = nearest((g.abs().amax(-1, keepdim=True) / 6.0).clamp(max=448.0), e4m3)
    a = nearest((g.abs() / torch.where(s > 0, s, 1.0)).clamp(max=6.0), torch.tensor(E2M1, dtype=torch.float64, device="cuda"))
    return (torch.where(s > 0, a, 0.0) * g.sign() * s * one).view(x.shape)


def _exact_attn(c, s):
    B, H, n_q, cs, G = c["B"], c["Hkv"], c["n_q"], c["cs"], c["Hq"] // c["Hkv"]
    out = torch.zeros(B, n_q, c["Hq"], D, dtype=torch.float64, device="cuda")
    cnts, lens = s["cnt"].tolist(), s["length"].tolist()
    for b in range(B):
        for h in range(H):
            n = cnts[b][h]
            slot, idx, mask = (s[w][b, h, :n].long() for w in ("slot", "idx", "qmask"))
            parts = []
            for hot, st, e in (("K", "Kst", "ke"), ("V", "Vst", "ve")):
                pages = s[hot][slot.clamp(min=0)]
                if st in s:
                    pages = torch.where((slot < 0)[:, None], s[st][(-1 - slot).clamp(min=0)], pages)
                codes, scales = _blocks(pages)
                parts.append(_decode(codes, scales, s[e][h].expand(codes.shape[:3]), torch.float64).reshape(-1, D))
            at = (idx[:, None] * cs + torch.arange(cs, device="cuda")).view(-1)
            for j in range(n_q):
                keep = (at < lens[b]) & ((mask >> j) & 1 == 1).repeat_interleave(cs)
                Kj, Vj = parts[0][keep], parts[1][keep]
                if "Kt" in s:
                    Kj = torch.cat((Kj, s["Kt"][b, :j + 1, h].double()))
                    Vj = torch.cat((Vj, s["Vt"][b, :j + 1, h].double()))
                if Kj.shape[0]:
                    q = s["q"][b, j, h * G:(h + 1) * G].double()
                    w = torch.softmax(q @ Kj.T * D ** -0.5, -1)
                    out[b, j, h * G:(h + 1) * G] = w @ Vj
    return out
