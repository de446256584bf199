"""Rotary positions, appends to the paged cache (bf16 and 4 bits) and the gather of
4-bit chunks, against the 64-bit oracle."""
import numpy as np
import pytest

import oracle
from sparse_kv_offload_gb300 import synth

import dd_testlib as tl
from test_kv_cache_oracle import SCALINGS, code_of

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


def bf16(rng, shape, scale=1.0):
    return synth.f32_to_bf16((rng.standard_normal(shape) * scale).astype(np.float32))


def make_rope(dd, rot, half, scaling, base=5e5):
    rope = dd.rope_table(rot, base=base, layout=dd.ROPE_HALF if half else dd.ROPE_INTERLEAVED,
                         scaling=code_of(dd, scaling), **SCALINGS[scaling])
    gain = 0.1 * np.log(8.0) + 1.0 if scaling == "by_parts" else 1.0
    return rope, oracle.rope_frequencies(rot, base, scaling, **SCALINGS[scaling]), gain


def check_rotated(got_bits, x, pos, freq, half, gain):
    """Within half a bf16 step of the exact rotation, and 2^-32 of the pair's magnitude for the 64-bit angle
    at positions up to 2^20 (2^20 * 2^-53 of it, twice) and the kernel's own 2^-36."""
    want = oracle.rope_rotate(oracle.bf16_decode(x), pos, freq, half, gain)
    got = oracle.bf16_decode(got_bits)
    step = np.ldexp(1.0, np.frexp(want)[1] - 8)                 # one bf16 step at the exact value
    size = np.abs(oracle.bf16_decode(x)).max(-1, keepdims=True) * gain
    assert (np.abs(got - want) <= step / 2 + size * 2.0 ** -32).all()
    # and all but the values next to a tie are the nearest bf16 number itself
    assert (got != oracle.round_bf16(want)).mean() < 1e-4
    n = 2 * len(freq)
    assert np.array_equal(got_bits[..., n:], x[..., n:])


# (B, T, H, rot, half, scaling, largest position)
ROPE = [
    (1, 1, 1, 128, True, "plain", 1), (16, 2, 32, 128, True, "by_parts", 32768),
    (3, 5, 7, 64, False, "linear", 1000), (2, 33, 3, 32, True, "ntk", 1 << 20),
    (1, 300, 8, 96, False, "by_wavelength", 1 << 20), (2, 130, 5, 96, True, "plain", 524288),
    (1, 2, 64, 128, False, "plain", (1 << 31) - 3), (4, 1, 1, 64, True, "by_wavelength", 100),
]


@pytest.mark.parametrize("B,T,H,rot,half,scaling,far", ROPE)
def test_rope(dd, B, T, H, rot, half, scaling, far):
    import torch
    rng = np.random.default_rng(B * 1000 + T)
    x = bf16(rng, (B, T, H, D))
    start = rng.integers(max(0, far - 50), far, B)
    rope, freq, gain = make_rope(dd, rot, half, scaling)
    pos = start[:, None] + np.arange(T)
    with dd.Context(dd.Shape(B, H, H, D, 64, 16, 1, 1), max_misses=0) as ctx:
        xd = tl.to_bf16(x)
        out = torch.zeros_like(xd)
        ctx.rope(rope, xd, out, tl.to_i32(start))
        assert ctx.status() == 0
        got = tl.from_bf16(out)
        if far <= 1 << 20:
            check_rotated(got, x, pos, freq, half, gain)
        # in place, on strided rows with padding: the same bits, the padding and what lies between kept
        wide = torch.full((B, T, H + 3, D + 16), 7.0, dtype=torch.bfloat16, device="cuda")
        view = wide[:, :, 1:1 + H, 8:8 + D]
        view.copy_(xd)
        lens = rng.integers(0, T + 1, B)
        before = tl.from_bf16(wide)
        ctx.rope(rope, view, view, tl.to_i32(start), new_len=tl.to_i32(lens))
        assert ctx.status() == 0
        after = tl.from_bf16(wide)
        for b in range(B):
            before[b, :lens[b], 1:1 + H, 8:8 + D] = got[b, :lens[b]]
        assert np.array_equal(after, before)


def test_rope_of_special_values(dd):
    """Zeros, signed zeros, subnormals, the largest numbers, infinities and NaN, in pairs."""
    import torch
    vals = np.array([0.0, -0.0, 1e-40, 3.3e38, np.inf, -np.inf, np.nan, 1.0], np.float32)
    x = np.zeros((1, 64, 1, D), np.uint16)
    with np.errstate(all="ignore"):
        bits = (vals.view(np.uint32) >> 16).astype(np.uint16)
    x[0, :, 0, :64] = bits[np.arange(64) % 8][:, None]
    x[0, :, 0, 64:] = bits[np.arange(64) // 8][:, None]
    rope, freq, _ = make_rope(dd, 128, True, "plain")
    with dd.Context(dd.Shape(1, 1, 1, D, 64, 16, 1, 1), max_misses=0) as ctx:
        out = torch.zeros(1, 64, 1, D, dtype=torch.bfloat16, device="cuda")
        ctx.rope(rope, tl.to_bf16(x), out, tl.to_i32([1]))
        assert ctx.status() == 0
    with np.errstate(all="ignore"):
        want = oracle.rope_rotate(oracle.bf16_decode(x), 1 + np.arange(64)[None], freq, True)
    got = oracle.bf16_decode(tl.from_bf16(out))
    assert np.array_equal(np.isnan(got), np.isnan(want))
    top = np.isinf(want) | (np.abs(want) > 3.38e38)              # next to overflow: infinite or the largest number
    assert np.array_equal(np.sign(got[top]), np.sign(want[top])) and (np.abs(got[top]) > 3.3e38).all()
    fine = ~np.isnan(want) & ~top
    assert (np.abs(got[fine] - want[fine]) <= np.abs(want[fine]) * 2.0 ** -8 + 2.0 ** -133).all()


class Cache:
    """A cache on the host, its pages and its table: what an append has to leave."""

    def __init__(self, rng, B, H, C, cs, four, holes=0.3):
        self.B, self.H, self.C, self.cs, self.four = B, H, C, cs, four
        self.n = B * H * C
        row = 72 if four else 256
        self.home = rng.integers(0, 256, (2, self.n, cs * row), dtype=np.uint8)
        self.slots = self.n + 3
        self.pool = rng.integers(0, 256, (2, self.slots, cs * row), dtype=np.uint8)
        slot = rng.permutation(self.slots)[:self.n]
        self.slot = np.where(rng.random(self.n) < holes, -1, slot).astype(np.int32)

    def expect(self, rows, start, lens):
        """rows (k, v): bits [B, T, H, 128] as they go in: bf16 bits, or (codes, scales)."""
        for w, r in enumerate(rows):
            for b, t, pos in oracle.append_positions(start, lens):
                for h in range(self.H):
                    page = (b * self.H + h) * self.C + pos // self.cs
                    at = pos % self.cs
                    for dst in [self.home[w, page]] + ([self.pool[w, self.slot[page]]] if self.slot[page] >= 0 else []):
                        if self.four:
                            c, s = r[0][b, t, h], r[1][b, t, h]
                            blk = at // 16 * 1152
                            o = blk + at % 16 * 64
                            dst[o:o + 64] = c[0::2] | (c[1::2] << 4)
                            o = blk + 1024 + at % 16 * 8
                            dst[o:o + 8] = s
                        else:
                            dst[at * 256:(at + 1) * 256] = r[b, t, h].view(np.uint8)


def dev(a, four, pin=False):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a).copy())
    t = t if four else t.view(torch.bfloat16)
    return t.pin_memory() if pin else t.cuda()


# (B, T, H, cs, C, rot, half, home on the host)
APPEND = [
    (1, 1, 1, 16, 2, 128, True, False), (3, 5, 2, 16, 4, 128, True, True), (2, 37, 3, 32, 3, 64, False, False),
    (4, 2, 8, 64, 2, 96, True, True), (2, 130, 1, 16, 12, 32, True, False), (5, 3, 7, 32, 2, 0, True, True),
    (1, 64, 2, 64, 1, 128, False, False),
]


@pytest.mark.parametrize("four", [False, True], ids=["bf16", "4bit"])
@pytest.mark.parametrize("B,T,H,cs,C,rot,half,host", APPEND)
def test_append(dd, four, B, T, H, cs, C, rot, half, host):
    import torch
    rng = np.random.default_rng(T * 100 + B)
    L = C * cs
    k, v = bf16(rng, (B, T, H, D), 2.0), bf16(rng, (B, T, H, D), 0.1)
    lens = rng.integers(0, T + 1, B)
    lens[0] = T
    start = np.array([rng.integers(0, L - n + 1) for n in lens])
    rope, turned = None, k
    if rot:
        rope, freq, gain = make_rope(dd, rot, half, "by_parts")
    ke, ve = rng.integers(-3, 4, H), rng.integers(-64, 4, H)
    cache = Cache(rng, B, H, C, cs, four)
    with dd.Context(dd.Shape(B, H, H, D, L, cs, 1, 1), max_misses=0, hot_slots=cache.slots) as ctx:
        # rows of a fused projection: [B, T, (K heads, V heads), 128 + padding]
        both = torch.zeros(B, T, 2 * H + 1, D + 8, dtype=torch.bfloat16, device="cuda")
        kd, vd = both[:, :, :H, :D], both[:, :, H:2 * H, 8:]
        kd.copy_(tl.to_bf16(k))
        vd.copy_(tl.to_bf16(v))
        if rot:
            out = torch.zeros(B, T, H, D, dtype=torch.bfloat16, device="cuda")
            ctx.rope(rope, kd, out, tl.to_i32(start))
            turned = tl.from_bf16(out)
            check_rotated(turned, k, start[:, None] + np.arange(T), freq, half, gain)
        if four:
            rows = [oracle.quantise_rows(oracle.bf16_decode(x), e[None, None]) for x, e in ((turned, ke), (v, ve))]
            extra = dict(kv_format=dd.KV_4BIT, k_exp=tl.to_i32(ke), v_exp=tl.to_i32(ve))
        else:
            rows, extra = [turned, v], {}
        home = [dev(x, four, host) for x in cache.home]
        pool = [dev(x, four) for x in cache.pool]
        cache.expect(rows, start, lens)
        args = (kd, vd, tl.to_i32(start))
        kw = dict(new_len=tl.to_i32(lens), rope=rope, **extra)
        ctx.append_kv(*args, Kh=home[0], Vh=home[1], Khot=pool[0], Vhot=pool[1], resident_slot=tl.to_i32(cache.slot), **kw)
        assert ctx.status() == 0
        bytes_of = lambda t: t.cpu().view(torch.uint8).numpy().reshape(t.shape[0], -1)   # noqa: E731
        for w in range(2):
            assert np.array_equal(bytes_of(home[w]), cache.home[w])
            assert np.array_equal(bytes_of(pool[w]), cache.pool[w])
        # home alone and pool alone write the same rows
        only = [torch.zeros_like(x) for x in pool]
        ctx.append_kv(*args, Khot=only[0], Vhot=only[1], resident_slot=tl.to_i32(np.arange(cache.n)), **kw)
        flat = [torch.zeros_like(x, device="cuda") for x in home]
        ctx.append_kv(*args, Kh=flat[0], Vh=flat[1], **kw)
        assert ctx.status() == 0
        for w in range(2):
            assert torch.equal(only[w][:cache.n].view(torch.uint8), flat[w].view(torch.uint8))
            assert not only[w][cache.n:].view(torch.uint8).any()


# (H, rot, half): with 10,000 tokens a warp goes through several heads, with 200 through one
MANY = [(40, 128, True), (17, 64, False), (9, 96, True), (6, 32, False), (5, 96, False), (16, 64, True)]


@pytest.mark.parametrize("H,rot,half", MANY)
def test_many_tokens(dd, H, rot, half):
    """Prompts long enough for warps with many heads: the oracle's rotation on some rows, and on all of them, in place
    and in both formats of the cache, what calls of 200 tokens give."""
    import torch
    T, step, cs = 10000, 200, 16
    g = torch.Generator(device="cuda").manual_seed(H)
    k, v = (torch.randn(1, T, H, D, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    rope, freq, gain = make_rope(dd, rot, half, "by_parts")
    with dd.Context(dd.Shape(1, H, H, D, T, cs, 1, 1), max_misses=0, hot_slots=0) as ctx:
        whole, parts, same = torch.zeros_like(k), torch.zeros_like(k), k.clone()
        ctx.rope(rope, k, whole, tl.to_i32([77]))
        ctx.rope(rope, same, same, tl.to_i32([77]))
        for t in range(0, T, step):
            ctx.rope(rope, k[:, t:t + step], parts[:, t:t + step], tl.to_i32([77 + t]))
        assert ctx.status() == 0 and torch.equal(whole, parts) and torch.equal(whole, same)
        rows = torch.arange(0, T, 397, device="cuda")
        check_rotated(tl.from_bf16(whole[:, rows].contiguous()), tl.from_bf16(k[:, rows].contiguous()),
                      77 + rows.cpu().numpy()[None], freq, half, gain)
        for four in (False, True):
            shape = (H * T // cs, cs * 72) if four else (1, H, T, D)
            home = [torch.zeros(shape, dtype=torch.uint8 if four else torch.bfloat16, device="cuda") for _ in range(4)]
            kw = dict(rope=rope, kv_format=dd.KV_4BIT if four else dd.KV_BF16)
            n = T - 5                                              # an odd end
            ctx.append_kv(k[:, :n], v[:, :n], tl.to_i32([3]), Kh=home[0], Vh=home[1], **kw)
            for t in range(0, n, step):
                e = min(n, t + step)
                ctx.append_kv(k[:, t:e], v[:, t:e], tl.to_i32([3 + t]), Kh=home[2], Vh=home[3], **kw)
            assert ctx.status() == 0
            assert torch.equal(home[0], home[2]) and torch.equal(home[1], home[3]) and home[0].any() and home[1].any()


def test_quantiser_edges(dd):
    """Rows where the 4-bit rounding can go wrong: every tie of both formats, the smallest and the largest
    scales, zeros, subnormals, infinities and NaN."""
    import torch
    rng = np.random.default_rng(3)
    rows = []
    for e in range(-12, 12):
        for m in range(8):                                        # scales next to e4m3's ties, then values at e2m1's
            top = 6.0 * (1 + m / 8.0) * 2.0 ** e
            near = np.concatenate([np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]) * top / 6.0,
                                   rng.standard_normal(8) * top / 4.0])
            rows.append(np.concatenate([np.clip(near, -top, top), [top * (1 + (e % 3 - 1) / 16.0)]] * 8))
    rows = oracle.round_bf16(np.array(rows))
    special = np.zeros((8, D))
    special[0, 3] = np.inf
    special[1, 17] = -np.inf
    special[2, 40] = np.nan
    special[3] = 3.3e38
    special[4] = 1e-40
    special[5, 0::2] = -0.0
    special[6] = np.where(np.arange(D) % 16 == 0, 2689.0, 1e-3)
    x = synth.f32_to_bf16(np.nan_to_num(np.concatenate([rows, special]), nan=1.0, posinf=1.0, neginf=1.0).astype(np.float32))
    n = len(x)
    x[n - 8, 3], x[n - 7, 17], x[n - 6, 40] = 0x7F80, 0xFF80, 0x7FC0
    T = n
    L = -(-T // 16) * 16
    x = x.reshape(1, T, 1, D)
    with dd.Context(dd.Shape(1, 1, 1, D, L, 16, 1, 1), max_misses=L // 16) as ctx:
        for exp in (0, -7, 9):
            e = tl.to_i32([exp])
            K = torch.zeros(L // 16, 16 * 72, dtype=torch.uint8, device="cuda")
            V = torch.zeros_like(K)
            ctx.append_kv(tl.to_bf16(x), tl.to_bf16(x), tl.to_i32([0]), Kh=K, Vh=V, kv_format=dd.KV_4BIT, k_exp=e, v_exp=e)
            assert ctx.status() == 0
            assert torch.equal(K, V)
            vals = oracle.bf16_decode(x[0, :, 0])
            codes, s8 = oracle.quantise_rows(vals, np.full(T, exp))
            gc, gs = oracle.kv4_unpack(K.cpu().numpy())
            gc, gs = gc.reshape(-1, D)[:T], gs.reshape(-1, 8)[:T]
            assert np.array_equal(gs, s8)
            zero = np.repeat(s8 == 0, 16, -1) | np.repeat(s8 == 127, 16, -1)    # the sign of a zero, a NaN group's codes
            same = (gc == codes) | ((gc & 7 == 0) & (codes & 7 == 0)) | (zero & (np.repeat(s8, 16, -1) == 127))
            assert same.all()
            # and expanded
            Kx = torch.zeros(L // 16, 16, D, dtype=torch.bfloat16, device="cuda")
            Vx = torch.zeros_like(Kx)
            ctx.gather_kv4(K, V, tl.to_i32(np.arange(L // 16)), tl.to_i32([L // 16]), Kx, Vx, expand=True, k_exp=e, v_exp=e)
            assert ctx.status() == 0
            want = oracle.kv4_values(K.cpu().numpy(), np.full(L // 16, exp)).reshape(-1, D)
            assert np.array_equal(oracle.bf16_decode(tl.from_bf16(Kx)).reshape(-1, D), want, equal_nan=True)


@pytest.mark.parametrize("host", [False, True], ids=["device", "pinned"])
@pytest.mark.parametrize("cs,C,B,H,n", [(16, 5, 2, 3, 7), (32, 40, 1, 2, 33), (64, 3, 3, 1, 1), (16, 9, 1, 1, 0)])
def test_gather4(dd, cs, C, B, H, n, host):
    import torch
    rng = np.random.default_rng(cs + n)
    total = B * H * C
    page = rng.integers(0, 256, (2, total, cs * 72), dtype=np.uint8)
    page.reshape(2, total, -1, 1152)[..., 1024:] &= 0x7E       # finite scales
    lst = rng.permutation(total)[:n].astype(np.int32)
    ke, ve = rng.integers(-64, 65, H), rng.integers(-2, 3, H)
    cap = n + 2
    with dd.Context(dd.Shape(B, H, H, D, C * cs, cs, 1, 1), max_misses=cap) as ctx:
        home = [dev(x, True, host) for x in page]
        raw = [torch.full((cap, cs * 72), 5, dtype=torch.uint8, device="cuda") for _ in range(2)]
        ml = tl.to_i32(np.concatenate([lst, [10 ** 6, 10 ** 6]]))   # behind the count: not looked at
        ctx.gather_kv4(home[0], home[1], ml, tl.to_i32([n]), raw[0], raw[1])
        wide = [torch.full((cap, cs, D), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        ctx.gather_kv4(home[0], home[1], ml, tl.to_i32([n]), wide[0], wide[1], expand=True, k_exp=tl.to_i32(ke),
                       v_exp=tl.to_i32(ve))
        assert ctx.status() == 0
        for w, e in ((0, ke), (1, ve)):
            assert np.array_equal(raw[w].cpu().numpy()[:n], page[w][lst]) and (raw[w][n:] == 5).all()
            want = oracle.kv4_values(page[w][lst], e[lst // C % H])
            assert np.array_equal(oracle.bf16_decode(tl.from_bf16(wide[w]))[:n], want) and (wide[w][n:] == 5).all()


def test_gather4_of_many_chunks(dd):
    """More blocks than the grid has warps, and pages in any order."""
    test_gather4(dd, 64, 1000, 1, 3, 2900, False)


def test_device_checks(dd):
    """Positions, lengths, slots, chunks and exponents out of range: reported, their rows left out, the rest written."""
    import torch
    B, T, H, cs, C = 3, 4, 2, 16, 2
    L = C * cs
    rng = np.random.default_rng(9)
    k = tl.to_bf16(bf16(rng, (B, T, H, D)))
    with dd.Context(dd.Shape(B, H, H, D, L, cs, 1, 1), max_misses=4, hot_slots=4) as ctx:
        def appended(start, lens, **kw):
            K = torch.zeros(B, H, L, D, dtype=torch.bfloat16, device="cuda")
            V = torch.zeros_like(K)
            ctx.append_kv(k, k, tl.to_i32(start), new_len=tl.to_i32(lens), Kh=K, Vh=V, **kw)
            return K, ctx.status()
        good, st = appended([0, 5, 28], [4, 4, 4])
        assert st == 0
        for start, lens in (([0, -1, 28], [4, 4, 4]), ([0, 5, 28], [4, 5, 4]), ([0, 5, 28], [4, -1, 4])):
            K, st = appended(start, lens)
            assert st == dd.DD_ERR_DEVICE_CHECK
            assert torch.equal(K[0], good[0]) and torch.equal(K[2], good[2]) and not K[1].any()
        K, st = appended([0, 5, 30], [4, 4, 4])                   # the last two rows lie behind the end
        assert st == dd.DD_ERR_DEVICE_CHECK and torch.equal(K[:2], good[:2]) and torch.equal(K[2, :, 30:], good[2, :, 28:30])
        pool = torch.zeros(4, cs, D, dtype=torch.bfloat16, device="cuda")
        for bad in (4, -2):
            slot = torch.full((B * H * C,), -1, dtype=torch.int32, device="cuda")
            slot[0] = bad
            K, st = appended([0, 5, 28], [4, 4, 4], Khot=pool, Vhot=pool.clone(), resident_slot=slot)
            assert st == dd.DD_ERR_DEVICE_CHECK and torch.equal(K, good) and not pool.any()
        out = torch.zeros(B, T, H, D, dtype=torch.bfloat16, device="cuda")
        rope = dd.rope_table(128)
        ctx.rope(rope, k, out, tl.to_i32([0, -1, 5]))
        assert ctx.status() == dd.DD_ERR_DEVICE_CHECK and not out[1].any() and out[0].any()
        home = torch.zeros(B * H * C, cs * 72, dtype=torch.uint8, device="cuda")
        st4 = [torch.full((4, cs * 72), 1, dtype=torch.uint8, device="cuda") for _ in range(2)]
        for bad in (-1, B * H * C):
            ctx.gather_kv4(home, home, tl.to_i32([0, bad]), tl.to_i32([2]), *st4)
            assert ctx.status() == dd.DD_ERR_DEVICE_CHECK and not st4[0][0].any() and (st4[0][1] == 1).all()
        wide = [torch.ones(4, cs, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        ctx.gather_kv4(home, home, tl.to_i32([0]), tl.to_i32([1]), *wide, expand=True, k_exp=tl.to_i32([65, 0]))
        assert ctx.status() == dd.DD_ERR_DEVICE_CHECK


def test_refusals(dd):
    import torch
    B, T, H, cs, C = 2, 3, 2, 16, 2
    bf = dict(dtype=torch.bfloat16, device="cuda")
    k = torch.zeros(B, T, H, D, **bf)
    start = torch.zeros(B, dtype=torch.int32, device="cuda")
    home = torch.zeros(B, H, C * cs, D, **bf)
    home4 = torch.zeros(B * H * C, cs * 72, dtype=torch.uint8, device="cuda")
    rope = dd.rope_table(128)
    with dd.Context(dd.Shape(B, H, H, D, C * cs, cs, 1, 1), max_misses=2, hot_slots=2) as ctx:
        n0 = ctx.launch_count()
        wide = torch.zeros(B, T, H, D + 4, **bf)
        bad_rows = [k[:, :, :1], k[:1], k[..., ::2], k.float(), k.cpu(), wide[..., 4:], wide[..., :D],
                    torch.zeros(B, T, H, D + 1, **bf)[..., 1:], torch.zeros(B, T, H, 64, **bf), k.transpose(2, 3)]
        for x in bad_rows:
            with pytest.raises((ValueError, TypeError, dd.DDError)):
                ctx.append_kv(x, k, start, Kh=home, Vh=home)
            with pytest.raises((ValueError, TypeError, dd.DDError)):
                ctx.append_kv(k, x, start, Kh=home, Vh=home)
        off = torch.zeros(B * T * H * D + 8, **bf)[1:1 + B * T * H * D].view(B, T, H, D)      # not on 16 bytes
        tall = torch.zeros(B, T, 2 * H, D, **bf)       # the same first row, other strides
        for x, o in ((off, k), (k, off), (k, k[:, :, :1].expand(B, T, H, D)), (k[:1], k), (k[0], k),
                     (tall[:, :, :H], tall[:, :, ::2])):
            with pytest.raises((ValueError, dd.DDError)):
                ctx.rope(rope, x, o, start)
        for kw in (dict(), dict(Kh=home), dict(Kh=home, Vh=home, k_exp=start),
                   dict(Kh=home4, Vh=home4), dict(Kh=home, Vh=home, kv_format=dd.KV_4BIT),
                   dict(Kh=home, Vh=home, kv_format=2), dict(Khot=home, Vhot=home),
                   dict(Kh=home.cpu(), Vh=home.cpu()), dict(Kh=home[:1], Vh=home[:1]),
                   dict(Khot=home[:1, :1, :16], Vhot=home, resident_slot=start),
                   dict(Kh=home, Vh=home, new_len=start.long()), dict(Kh=home, Vh=home, new_len=start[:1])):
            with pytest.raises((ValueError, TypeError, dd.DDError)):
                ctx.append_kv(k, k, start, **kw)
        lst = torch.zeros(2, dtype=torch.int32, device="cuda")
        st4 = torch.zeros(2, cs * 72, dtype=torch.uint8, device="cuda")
        for a, kw in (((home, home4, lst, lst, st4, st4), {}), ((home4, home4, lst, lst, st4, None), {}),
                      ((home4, home4, lst, lst, st4, st4), dict(expand=True)),
                      ((home4, home4, lst, lst, st4, st4), dict(k_exp=lst)), ((home4, home4, lst, lst, st4[:1], st4), {})):
            with pytest.raises((ValueError, TypeError, dd.DDError)):
                ctx.gather_kv4(*a, **kw)
        assert ctx.launch_count() == n0
        # nothing to do
        ctx.append_kv(k[:, :0], k[:, :0], start, Kh=home, Vh=home)
        ctx.rope(rope, k[:, :0], k[:, :0], start)
        assert ctx.launch_count() == n0 and ctx.status() == 0
    with dd.Context(dd.Shape(0, H, H, D, C * cs, cs, 1, 1), max_misses=2) as ctx:
        ctx.append_kv(k[:0], k[:0], start, Kh=home[:0], Vh=home[:0])
        ctx.rope(rope, k[:0], k[:0], start)
        assert ctx.launch_count() == 0


def test_append_is_captured_and_replayed(dd):
    """A captured append reads its positions at replay: the caller's counter moves on in between."""
    import torch
    B, T, H, cs, C = 2, 2, 2, 16, 3
    rng = np.random.default_rng(11)
    k = tl.to_bf16(bf16(rng, (B, T, H, D)))
    rope = dd.rope_table(64)
    with dd.Context(dd.Shape(B, H, H, D, C * cs, cs, 1, 1), max_misses=0) as ctx:
        def pair():
            return [torch.zeros(B * H * C, cs * 72, dtype=torch.uint8, device="cuda") for _ in range(2)]
        start = torch.zeros(B, dtype=torch.int32, device="cuda")
        K, V = pair()
        side = torch.cuda.Stream()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            ctx.append_kv(k, k, start, rope=rope, Kh=K, Vh=V, kv_format=dd.KV_4BIT)
            start += T
        for _ in range(5):
            graph.replay()
        assert ctx.status() == 0
        K2, V2 = pair()
        for i in range(5):
            ctx.append_kv(k, k, tl.to_i32([i * T] * B), rope=rope, Kh=K2, Vh=V2, kv_format=dd.KV_4BIT)
        assert ctx.status() == 0
        assert torch.equal(K, K2) and torch.equal(V, V2) and K.any()


def test_home_memory_is_looked_up_on_every_call(dd):
    """The C calls refuse host memory that is no longer pinned, although they took the same address before."""
    import torch
    B, T, H, cs, C = 1, 2, 1, 16, 2
    k = torch.ones(B, T, H, D, dtype=torch.bfloat16, device="cuda")
    start = torch.zeros(B, dtype=torch.int32, device="cuda")
    lst, n = tl.to_i32([0]), tl.to_i32([1])
    home = [torch.zeros(1 << 16, dtype=torch.uint8) for _ in range(2)]
    at = [(t.data_ptr() + 4095) // 4096 * 4096 for t in home]      # a page of its own each
    st4 = [torch.zeros(1, cs * 72, dtype=torch.uint8, device="cuda") for _ in range(2)]
    strides = (T * H * D, H * D, D)
    with dd.Context(dd.Shape(B, H, H, D, C * cs, cs, 1, 1), max_misses=1) as ctx:
        args = dd._append_args.pack(k.data_ptr(), k.data_ptr(), *strides, *strides, T, dd.KV_4BIT, start.data_ptr(), 0, 0,
                                    *at, 0, 0, 0, 0, 0)

        def calls():
            a = dd._lib.dd_append_kv(ctx._h, args, None)
            g = dd._lib.dd_gather_kv4(ctx._h, *at, lst.data_ptr(), n.data_ptr(), st4[0].data_ptr(), st4[1].data_ptr(), 0,
                                      None, None, None)
            torch.cuda.synchronize()
            return a, g
        assert calls() == (dd.DD_ERR_INVALID_ARG,) * 2
        rt = torch.cuda.cudart()
        for p in at:
            assert int(rt.cudaHostRegister(p, 4096, 0)) == 0
        try:
            assert calls() == (dd.DD_OK,) * 2 and ctx.status() == 0 and st4[0].any()
        finally:
            for p in at:
                assert int(rt.cudaHostUnregister(p)) == 0
        assert calls() == (dd.DD_ERR_INVALID_ARG,) * 2
