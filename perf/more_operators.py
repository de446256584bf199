"""Operators around a paged KV cache that grows and is kept to a budget: attention of new
tokens over the cache's pages, the attention weight that each chunk has gathered, and
eviction by that weight, as cases to be timed and compared.

``own = False``: ``run`` computes in elementary torch operations.  ``own = True``:
``run`` makes the library's calls.

Pages are bf16 [slots, cs, 128].  A list per (request, KV head) names the chunks that
are in the cache, ascending, and the slot of each one (>= 0 in the pool, -(m+1) in
staging slot m); row r of chunk c holds position c*cs + r, and a token sees the
positions up to its own.
"""
import functools
import math

import numpy as np
import torch

own = False

D = 128
NEG = -math.inf


# ----------------------------------------------------------------------- cases
def _extend(name, B, Hq, Hkv, T, L, cs, kept=1.0, ragged=False, staged=0.0, strided=False):
    return dict(name=name, op="extend", B=B, Hq=Hq, Hkv=Hkv, T=T, L=L, cs=cs, kept=kept, ragged=ragged, staged=staged,
                strided=strided)


def _weights(name, B, Hq, Hkv, T, L, cs, window=0, decay=1.0, kept=1.0, ragged=False, staged=0.0, strided=False):
    return dict(name=name, op="weights", B=B, Hq=Hq, Hkv=Hkv, T=T, L=L, cs=cs, window=window, decay=decay, kept=kept,
                ragged=ragged, staged=staged, strided=strided)


def _evict(name, B, Hkv, C, cs, keep, first, last, new, ragged):
    return dict(name=name, op="evict", B=B, Hkv=Hkv, C=C, cs=cs, keep=keep, first=first, last=last, new=new,
                ragged=ragged)


def listed():
    return [
        # one token of one request with 4K context: latency
        _extend("extend single", 1, 32, 8, 1, 4096, 16),
        # a decode step over whole caches of the Llama-3-8B layer, contexts of up to 32K
        _extend("extend decode", 16, 32, 8, 1, 32768, 16, ragged=True),
        # five tokens to verify a request, 32B-class layer, caches kept to a sixteenth of 32K
        _extend("extend verify", 32, 64, 8, 5, 32768, 16, kept=0.0625),
        # odd head ratio, lengths and strides, a part of the chunks in staging, others evicted
        _extend("extend odd", 3, 35, 7, 77, 10656, 32, kept=0.6, ragged=True, staged=0.3, strided=True),
        # the first 2K tokens of four prompts, 32B-class layer
        _extend("extend prompt", 4, 64, 8, 2048, 2048, 16),
        # 2K tokens of a long prompt behind 62K others
        _extend("extend long prompt", 1, 64, 8, 2048, 65536, 64),
        # the weights of a decode step's token over whole caches, forgotten slowly
        _weights("weights decode", 16, 32, 8, 1, 32768, 16, decay=0.98, ragged=True),
        # a prompt's last 32 tokens observe the whole prompt, ragged lengths
        _weights("weights window", 8, 64, 8, 64, 32768, 16, window=32, decay=0.0, ragged=True),
        # all 2K tokens of a prompt's part
        _weights("weights prompt", 2, 64, 8, 2048, 16384, 32),
        # one request's pool with 4K context: latency
        _evict("evict single", 1, 8, 256, 16, 64, 1, 4, 16, False),
        # a step of 32 requests with pools of 256 chunks
        _evict("evict step", 32, 8, 2048, 16, 240, 2, 8, 64, True),
        # contexts of up to 256K brought down to a quarter after their prompts
        _evict("evict prompts", 64, 8, 16384, 16, 4096, 4, 64, 2048, True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["extend", "extend", "weights", "evict"])
    cs, Hkv, B = rng.choice([16, 32, 64]), rng.randint(1, 12), _log(rng, 1, 64)
    if op == "evict":
        C = _log(rng, 4, 16384)
        while B * Hkv * C > 1 << 23:
            B = max(1, B // 2)
        keep = max(1, min(C, _log(rng, 1, C)))
        last = rng.randint(0, max(1, keep // 2))
        c = _evict("", B, Hkv, C, cs, keep, rng.randint(0, 4), last, rng.randint(0, max(1, keep // 4) * cs),
                   rng.random() < 0.7)
        del c["name"]
        return c
    G = rng.randint(1, 16)
    T = _log(rng, 1, 4096)
    L = -(-(T + _log(rng, 1, 131072)) // cs) * cs
    L = min(L, 16384 * cs)
    while B * Hkv * L > 1 << 22 or B * T * L * Hkv * G > 1 << 33:
        if B > 1:
            B //= 2
        elif L > 4 * T + 64:
            L = max(-(-T // cs) * cs, L // 2 // cs * cs)
        else:
            T = max(1, T // 2)
            L = max(cs, -(-T // cs) * cs, L // 2 // cs * cs)
    T = min(T, L)
    kept = rng.choice([1.0, 1.0, 0.5, 0.1])
    rest = dict(kept=kept, ragged=rng.random() < 0.7, staged=rng.choice([0.0, 0.0, 0.3]), strided=rng.random() < 0.5)
    if op == "extend":
        c = _extend("", B, Hkv * G, Hkv, T, L, cs, **rest)
    else:
        c = _weights("", B, Hkv * G, Hkv, T, L, cs, window=rng.choice([0, rng.randint(1, T)]),
                     decay=rng.choice([0.0, 0.9, 1.0]), **rest)
    del c["name"]
    return c


# --------------------------------------------------------------------- prepare
@functools.lru_cache(maxsize=None)
def _context(B, Hq, Hkv, L, cs, k, max_misses, hot_slots):
    """A program makes one context per shape and keeps it."""
    from sparse_kv_offload_gb300 import dd
    return dd.Context(dd.Shape(B, Hq, Hkv, D, L, cs, k, 1), max_misses=max_misses, hot_slots=hot_slots)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = _prepare_evict(case, g) if case["op"] == "evict" else _prepare_rows(case, g)
    s["case"] = case
    return s


def _rows_in(c, g, heads):
    """bf16 rows [B, T, heads, 128], of a wider projection where the case says so."""
    x = torch.randn(c["B"], c["T"], heads + (c["Hkv"] if c["strided"] else 0), D, generator=g, device="cuda")
    return x.to(torch.bfloat16)[:, :, :heads]


def _prepare_rows(c, g):
    B, Hq, H, T, L, cs = c["B"], c["Hq"], c["Hkv"], c["T"], c["L"], c["cs"]
    C, dev = L // cs, "cuda"
    if c["ragged"]:
        n = torch.randint(T - T // 2, T + 1, (B,), generator=g, device=dev)
        start = ((0.4 + 0.6 * torch.rand(B, generator=g, device=dev, dtype=torch.float64)) * (L - n)).long()
    else:
        n = torch.full((B,), T, device=dev)
        start = L - n
    # in the cache: a share of the chunks that lie before the new tokens, and all that the new ones are in
    at = torch.arange(C, device=dev)
    old = start // cs
    keep = torch.ceil(old * c["kept"]).long().view(B, 1, 1)
    order = torch.rand(B, H, C, generator=g, device=dev) + 2.0 * (at >= old.view(B, 1, 1))
    rank = order.argsort(-1).argsort(-1)
    here = (rank < keep) | ((at >= old.view(B, 1, 1)) & (at <= ((start + n - 1) // cs).view(B, 1, 1)))
    cnt = here.sum(-1)
    idx = torch.sort((~here).to(torch.uint8), dim=-1, stable=True).indices
    used = at < cnt[..., None]
    per_unit = min(C, math.ceil(C * c["kept"]) + (T + cs - 2) // cs + 1)
    slots = B * H * per_unit
    slot = torch.zeros(B, H, C, dtype=torch.long, device=dev)
    slot[used] = torch.randperm(slots, generator=g, device=dev)[:int(cnt.sum())]
    staged = torch.rand(B, H, C, generator=g, device=dev) < c["staged"]
    slot = torch.where(staged, -1 - slot, slot)
    gain = torch.exp(0.7 * torch.randn(D, generator=g, device=dev))       # a few channels of keys are far larger

    def pool(scale):
        x = torch.empty(slots, cs, D, dtype=torch.bfloat16, device=dev)
        for part in x.split(max(1, (1 << 27) // (cs * D))):
            part.copy_(torch.randn(part.shape, generator=g, device=dev) * scale)
        return x

    s = dict(q=_rows_in(c, g, Hq), n=n.to(torch.int32), start=start.to(torch.int32),
             idx=torch.where(used, idx, 0).to(torch.int32), slot=torch.where(used, slot, 0).to(torch.int32),
             cnt=cnt.to(torch.int32), K=pool(gain))
    if c["staged"] > 0:
        s.update(Kst=pool(gain), misses=torch.tensor([slots], dtype=torch.int32, device=dev))
    if c["op"] == "extend":
        s.update(V=pool(1.0), out=torch.zeros(B, T, Hq, D, dtype=torch.bfloat16, device=dev),
                 lse=torch.zeros(B, T, Hq, device=dev))
        if c["staged"] > 0:
            s["Vst"] = pool(1.0)
    else:
        # the rows' log-sum-exps, as the attention before has left them
        s["lse"] = _lse(c, s)
        s["w0"] = torch.rand(B, H, C, generator=g, device=dev) * 4.0
        s["w"] = torch.empty_like(s["w0"])
    if own:
        s["ctx"] = _context(B, Hq, H, L, cs, C, slots if c["staged"] > 0 else 0, slots)
    return s


def _prepare_evict(c, g):
    B, H, C, cs, keep, dev = c["B"], c["Hkv"], c["C"], c["cs"], c["keep"], "cuda"
    more = -(-c["new"] // cs) + 1
    S = min(C, keep + more)
    if c["ragged"]:
        n = torch.randint(0, c["new"] + 1, (B,), generator=g, device=dev)
        length = ((0.3 + 0.7 * torch.rand(B, generator=g, device=dev, dtype=torch.float64)) * (C * cs - n).clamp(min=0)).long()
    else:
        n = torch.full((B,), min(c["new"], C * cs), device=dev)
        length = C * cs - n
    chunks = (length + cs - 1) // cs
    # the chunks in the pool: as many as fit beside the ones to come, any of those that have rows
    room = (S - (length + n + cs - 1) // cs + chunks).clamp(max=S).view(B, 1, 1)
    at = torch.arange(C, device=dev)
    order = torch.rand(B, H, C, generator=g, device=dev) + 2.0 * (at >= chunks.view(B, 1, 1))
    here = (order.argsort(-1).argsort(-1) < room) & (at < chunks.view(B, 1, 1))
    place = torch.rand(B, H, S, generator=g, device=dev).argsort(-1)
    which = (here.cumsum(-1) - 1).clamp(min=0, max=S - 1)
    unit = torch.arange(B * H, device=dev).view(B, H, 1)
    slot = torch.where(here, unit * S + place.gather(-1, which), -1)
    # gathered weights: most of it on few chunks, and many that nothing has looked at
    w = torch.exp(2.0 * torch.randn(B, H, C, generator=g, device=dev))
    w = torch.where(torch.rand(B, H, C, generator=g, device=dev) < 0.2, 0.0, w)
    i32 = torch.int32
    s = dict(w=w, length=length.to(i32), n=n.to(i32), slot=slot.to(i32), S=S,
             slot_out=torch.zeros(B, H, C, dtype=i32, device=dev), owner=torch.zeros(B, H, S, dtype=i32, device=dev),
             gone=torch.zeros(B, H, S, dtype=i32, device=dev), gone_cnt=torch.zeros(B, H, dtype=i32, device=dev),
             idx=torch.zeros(B, H, S, dtype=i32, device=dev), list_slot=torch.zeros(B, H, S, dtype=i32, device=dev),
             cnt=torch.zeros(B, H, dtype=i32, device=dev))
    if own:
        s["ctx"] = _context(B, H, H, C * cs, cs, S, 0, B * H * S)
    return s


# -------------------------------------------------------------------------- run
def run(s):
    op = s["case"]["op"]
    if own:
        return {"extend": _own_extend, "weights": _own_weights, "evict": _own_evict}[op](s)
    return {"extend": _plain_extend, "weights": _plain_weights, "evict": _plain_evict}[op](s)


def _own_extend(s):
    s["ctx"].extend_attn(s["q"], s["start"], s["K"], s["V"], s["idx"], s["slot"], s["cnt"], s["out"], new_len=s["n"],
                         lse=s["lse"], Kst=s.get("Kst"), Vst=s.get("Vst"), miss_count=s.get("misses"))
    return s["out"], s["lse"]


def _own_weights(s):
    s["w"].copy_(s["w0"])
    s["ctx"].chunk_weights(s["q"], s["start"], s["lse"], s["K"], s["idx"], s["slot"], s["cnt"], s["w"], new_len=s["n"],
                           window=s["case"]["window"], decay=s["case"]["decay"], Kst=s.get("Kst"),
                           miss_count=s.get("misses"))
    return s["w"]


def _own_evict(s):
    c = s["case"]
    s["ctx"].evict_chunks(s["w"], s["length"], s["slot"], s["slot_out"], c["keep"], s["S"], first=c["first"],
                          last=c["last"], new_len=s["n"], slot_chunk=s["owner"], evicted=s["gone"],
                          evicted_cnt=s["gone_cnt"], union_idx=s["idx"], union_slot=s["list_slot"], union_cnt=s["cnt"])
    return s["slot_out"], s["owner"], s["gone"], s["gone_cnt"], s["idx"], s["list_slot"], s["cnt"]


def _gather(c, s, b, pool, staged, width):
    """fp32 rows [H, width*cs, 128] of request b's listed chunks."""
    slot = s["slot"][b, :, :width].long()
    rows = s[pool][slot.clamp(min=0)]
    if staged in s:
        rows = torch.where((slot < 0)[..., None, None], s[staged][(-1 - slot).clamp(min=0)], rows)
    return rows.float().flatten(1, 2)


def _blocks(c, s):
    """For every request and every block of its tokens that keeps the score matrix small:
    (request, first token, end, list width, queries fp32 [H, G*tokens, 128], visible [H, tokens, keys])."""
    H, cs, G = c["Hkv"], c["cs"], c["Hq"] // c["Hkv"]
    widths, ns, starts = s["cnt"].amax(-1).tolist(), s["n"].tolist(), s["start"].tolist()
    for b in range(c["B"]):
        width, n = widths[b], ns[b]
        pos = (s["idx"][b, :, :width].long()[..., None] * cs + torch.arange(cs, device="cuda")).flatten(1)
        there = (torch.arange(width, device="cuda") < s["cnt"][b, :, None]).repeat_interleave(cs, -1)
        step = max(1, (1 << 28) // max(1, H * G * width * cs))
        for t0 in range(0, n, step):
            t1 = min(n, t0 + step)
            at = torch.arange(starts[b] + t0, starts[b] + t1, device="cuda")
            seen = there[:, None] & (pos[:, None] <= at[:, None])
            q = s["q"][b, t0:t1].float().view(t1 - t0, H, G, D).permute(1, 2, 0, 3).flatten(1, 2)
            yield b, t0, t1, width, q, seen


def _scores(c, q, K, seen):
    """Scaled scores [H, G, tokens, keys], -inf where not visible."""
    H, G = c["Hkv"], c["Hq"] // c["Hkv"]
    x = (q @ K.transpose(-1, -2)).view(H, G, seen.shape[1], -1) / math.sqrt(D)
    return torch.where(seen[:, None], x, NEG)


def _plain_extend(s, values=True):
    c = s["case"]
    H, G = c["Hkv"], c["Hq"] // c["Hkv"]
    last = None
    for b, t0, t1, width, q, seen in _blocks(c, s):
        if b != last:
            K = _gather(c, s, b, "K", "Kst", width)
            V = _gather(c, s, b, "V", "Vst", width) if values else None
            last = b
        x = _scores(c, q, K, seen)
        top = x.amax(-1, keepdim=True)
        top = torch.where(top == NEG, 0.0, top)
        p = torch.exp(x - top)
        total = p.sum(-1, keepdim=True)
        lse = (top + torch.log(total))[..., 0]                                       # [H, G, tokens]
        s["lse"][b, t0:t1] = lse.permute(2, 0, 1).flatten(1)
        if values:
            o = (p.flatten(1, 2) @ V).view(H, G, t1 - t0, D)
            o = torch.where(total > 0, o / total, 0.0)
            s["out"][b, t0:t1] = o.permute(2, 0, 1, 3).flatten(1, 2).to(torch.bfloat16)
    return (s["out"], s["lse"]) if values else s["lse"]


def _lse(c, s):
    t = dict(s, case=c, lse=torch.zeros(c["B"], c["T"], c["Hq"], device="cuda"))
    return _plain_extend(t, values=False)


def _plain_weights(s):
    c = s["case"]
    H, G, cs = c["Hkv"], c["Hq"] // c["Hkv"], c["cs"]
    ns = s["n"].tolist()
    w = s["w"].copy_(s["w0"])
    last = None
    total = torch.zeros(c["B"], H, c["L"] // cs, dtype=torch.float64, device="cuda")
    for b, t0, t1, width, q, seen in _blocks(c, s):
        if b != last:
            K = _gather(c, s, b, "K", "Kst", width)
            last = b
        x = _scores(c, q, K, seen)
        lse = s["lse"][b, t0:t1].view(t1 - t0, H, G).permute(1, 2, 0)
        p = torch.where(lse[..., None] == NEG, 0.0, torch.exp(x - lse[..., None]))
        if c["window"]:
            inside = torch.arange(t0, t1, device="cuda") >= ns[b] - c["window"]
            p = torch.where(inside[:, None], p, 0.0)
        total[b, :, :width] += p.reshape(H, -1, width, cs).sum(-1).sum(1, dtype=torch.float64)
    used = torch.arange(w.shape[-1], device="cuda") < s["cnt"][..., None]
    b, h, i = used.nonzero(as_tuple=True)
    at = s["idx"][b, h, i].long()
    w[b, h, at] = (w[b, h, at].double() * c["decay"] + total[b, h, i]).float()
    return w


def _plain_evict(s):
    c = s["case"]
    B, H, C, cs, S = c["B"], c["Hkv"], c["C"], c["cs"], s["S"]
    at = torch.arange(C, device="cuda")
    n0 = ((s["length"].long() + cs - 1) // cs).view(B, 1, 1)
    n1 = ((s["length"].long() + s["n"] + cs - 1) // cs).view(B, 1, 1)
    slot = s["slot"].long()
    here = slot >= 0
    fresh = ~here & (at >= n0) & (at < n1)
    may = here & (at >= c["first"]) & (at < n0 - c["last"])
    leave = (here.sum(-1) + fresh.sum(-1) - c["keep"]).clamp(min=0).minimum(may.sum(-1))
    order = torch.sort(torch.where(may, s["w"], math.inf), dim=-1, stable=True).indices
    rank = torch.empty_like(order).scatter_(-1, order, at.expand(B, H, C))
    gone = may & (rank < leave[..., None])
    stay = here & ~gone
    # free slots of the unit, ascending, to the new chunks, ascending
    unit = torch.arange(B * H, device="cuda").view(B, H, 1) * S
    taken = torch.zeros(B, H, S + 1, dtype=torch.bool, device="cuda")
    taken.scatter_(-1, torch.where(stay, slot - unit, S), True)
    free = torch.sort(taken[..., :S].to(torch.uint8), dim=-1, stable=True).indices
    mine = (fresh.cumsum(-1) - 1).clamp(min=0, max=S - 1)
    out = torch.where(stay, slot, torch.where(fresh, unit + free.gather(-1, mine), -1))
    s["slot_out"].copy_(out)
    owner = torch.full((B, H, S + 1), -1, dtype=torch.long, device="cuda")
    owner.scatter_(-1, torch.where(out >= 0, out - unit, S), at.expand(B, H, C))
    s["owner"].copy_(owner[..., :S])
    for mask, cnt, to in ((gone, "gone_cnt", ((None, "gone"),)), (out >= 0, "cnt", ((None, "idx"), (out, "list_slot")))):
        s[cnt].copy_(mask.sum(-1))
        first = torch.sort((~mask).to(torch.uint8), dim=-1, stable=True).indices[..., :S]
        used = torch.arange(S, device="cuda") < s[cnt][..., None]
        for values, name in to:
            v = first if values is None else values.gather(-1, first)
            s[name].copy_(torch.where(used, v, 0))
    return s["slot_out"], s["owner"], s["gone"], s["gone_cnt"], s["idx"], s["list_slot"], s["cnt"]


# ------------------------------------------------------------------------- work
def work(case):
    c = case
    if c["op"] == "evict":
        n, per = c["B"] * c["Hkv"], min(c["C"], c["keep"] + -(-c["new"] // c["cs"]) + 1)
        return {"bytes": n * (12.0 * c["C"] + 16.0 * per), "flops": n * 4.0 * c["C"]}
    share = 0.75 if c["ragged"] and c["T"] > 1 else 1.0
    T = c["T"] * share
    before = max(0.0, c["L"] - c["T"]) * (0.7 if c["ragged"] else 1.0) * c["kept"]
    rows = c["B"] * c["Hkv"] * (before + T)
    if c["op"] == "weights" and c["window"]:
        T = min(T, c["window"])
    pairs = c["B"] * c["Hq"] * T * (before + 0.5 * (T + 1))
    if c["op"] == "extend":
        return {"bytes": rows * 512.0 + c["B"] * T * c["Hq"] * (4.0 * D + 4.0), "flops": 4.0 * D * pairs}
    return {"bytes": rows * 256.0 + c["B"] * T * c["Hq"] * (2.0 * D + 4.0) + rows / c["cs"] * 8.0,
            "flops": 2.0 * D * pairs}


# ------------------------------------------------------------------------ exact
def exact(case, seed):
    """From the definitions, in 64 bits, head by head."""
    s = prepare(case, seed)
    return {"extend": _exact_extend, "weights": _exact_weights, "evict": _exact_evict}[case["op"]](case, s)


def _exact_rows(c, s, pool, staged, b, h):
    n = int(s["cnt"][b, h])
    slots = s["slot"][b, h, :n].tolist()
    if not slots:
        return torch.zeros(0, D, dtype=torch.float64, device="cuda")
    rows = torch.empty(n, c["cs"], D, dtype=torch.float64, device="cuda")
    hot = torch.tensor([i for i, x in enumerate(slots) if x >= 0], dtype=torch.long, device="cuda")
    far = torch.tensor([i for i, x in enumerate(slots) if x < 0], dtype=torch.long, device="cuda")
    where = torch.tensor(slots, device="cuda")
    rows[hot] = s[pool][where[hot]].double()
    if far.numel():
        rows[far] = s[staged][-where[far] - 1].double()
    return rows.view(-1, D)


def _exact_softmax(c, s, b, h, K, lo, hi):
    """Tokens lo..hi of KV head h: scores [tokens, G, keys] in 64 bits, masked by position."""
    G = c["Hq"] // c["Hkv"]
    first = s["idx"][b, h, :int(s["cnt"][b, h])].long() * c["cs"]
    pos = torch.stack([first + r for r in range(c["cs"])], -1).view(-1)
    q = s["q"][b, lo:hi, h * G:(h + 1) * G].double()
    x = torch.einsum("tgd,kd->tgk", q, K) * D ** -0.5
    here = torch.arange(lo, hi, device="cuda") + int(s["start"][b])
    return x.masked_fill_((pos > here.view(-1, 1)).unsqueeze(1), NEG)


def _exact_extend(c, s):
    B, T, Hq, H = c["B"], c["T"], c["Hq"], c["Hkv"]
    G = Hq // H
    out = torch.zeros(B, T, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.zeros(B, T, Hq, dtype=torch.float64, device="cuda")
    for b in range(B):
        n = int(s["n"][b])
        for h in range(H):
            K, V = _exact_rows(c, s, "K", "Kst", b, h), _exact_rows(c, s, "V", "Vst", b, h)
            step = max(1, (1 << 27) // (G * max(1, K.shape[0])))
            for lo in range(0, n, step):
                hi = min(n, lo + step)
                x = _exact_softmax(c, s, b, h, K, lo, hi)
                z = torch.logsumexp(x, -1)
                lse[b, lo:hi, h * G:(h + 1) * G] = z
                p = torch.exp(x.sub_(torch.where(z == NEG, 0.0, z).unsqueeze(-1)))
                out[b, lo:hi, h * G:(h + 1) * G] = p @ V
    return out, lse


def _exact_weights(c, s):
    H, cs = c["Hkv"], c["cs"]
    G = c["Hq"] // H
    w = s["w0"].double()
    for b in range(c["B"]):
        n = int(s["n"][b])
        begin = max(0, n - c["window"]) if c["window"] else 0
        for h in range(H):
            m = int(s["cnt"][b, h])
            K = _exact_rows(c, s, "K", "Kst", b, h)
            got = torch.zeros(m, dtype=torch.float64, device="cuda")
            step = max(1, (1 << 27) // (G * max(1, K.shape[0])))
            for lo in range(begin, n, step):
                hi = min(n, lo + step)
                z = s["lse"][b, lo:hi, h * G:(h + 1) * G].double().unsqueeze(-1)
                p = torch.exp(_exact_softmax(c, s, b, h, K, lo, hi) - torch.where(z == NEG, math.inf, z))
                got += p.sum((0, 1)).view(m, cs).sum(-1)
            at = s["idx"][b, h, :m].long()
            w[b, h, at] = w[b, h, at] * c["decay"] + got
    return w


def _exact_evict(c, s):
    """Unit by unit on the host."""
    B, H, C, cs, S = c["B"], c["Hkv"], c["C"], c["cs"], s["S"]
    w, slot = s["w"].cpu().numpy(), s["slot"].cpu().numpy()
    length, new = s["length"].tolist(), s["n"].tolist()
    res = {k: s[k].cpu().numpy().copy() for k in ("slot_out", "owner", "gone", "gone_cnt", "idx", "list_slot", "cnt")}
    for b in range(B):
        n0, n1 = -(-length[b] // cs), -(-(length[b] + new[b]) // cs)
        for h in range(H):
            base = (b * H + h) * S
            now = slot[b, h].copy()
            held = np.flatnonzero(now >= 0)
            come = [x for x in range(n0, n1) if now[x] < 0]
            cand = held[(held >= c["first"]) & (held < n0 - c["last"])]
            e = min(max(0, len(held) + len(come) - c["keep"]), len(cand))
            out = np.sort(cand[np.lexsort((cand, w[b, h, cand]))[:e]])
            now[out] = -1
            free = np.setdiff1d(np.arange(S), now[now >= 0] - base)
            now[come] = base + free[:len(come)]
            stay = np.flatnonzero(now >= 0)
            res["slot_out"][b, h] = now
            res["owner"][b, h] = -1
            res["owner"][b, h, now[stay] - base] = stay
            res["gone"][b, h, :e], res["gone_cnt"][b, h] = out, e
            res["idx"][b, h, :len(stay)], res["list_slot"][b, h, :len(stay)] = stay, now[stay]
            res["cnt"][b, h] = len(stay)
    return tuple(torch.from_numpy(res[k]).cuda() for k in ("slot_out", "owner", "gone", "gone_cnt", "idx", "list_slot", "cnt"))
