"""CPU pins of the cache operators' oracle, and the host side of the library's:
the rotation table and the binding's refusals that need no GPU."""
import math

import numpy as np
import pytest

import oracle


@pytest.fixture(scope="module")
def dd():
    from sparse_kv_offload_gb300 import build
    build.build()
    from sparse_kv_offload_gb300 import dd as mod
    return mod


SCALINGS = {
    "plain": {}, "linear": dict(factor=4.0), "ntk": dict(factor=4.0),
    "by_parts": dict(factor=8.0, orig_len=8192.0, beta_fast=32.0, beta_slow=1.0),
    "by_wavelength": dict(factor=8.0, orig_len=8192.0, beta_fast=4.0, beta_slow=1.0),
}


def code_of(dd, scaling):
    return {"plain": dd.ROPE_PLAIN, "linear": dd.ROPE_LINEAR, "ntk": dd.ROPE_NTK, "by_parts": dd.ROPE_BY_PARTS,
            "by_wavelength": dd.ROPE_BY_WAVELENGTH}[scaling]


def test_rotation_is_a_rotation():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((5, 2, 128))
    f = oracle.rope_frequencies(128, 1e4)
    for half in (True, False):
        y = oracle.rope_rotate(x, np.arange(5), f, half)
        assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1))
        assert np.array_equal(y[0], x[0])                       # position 0
        # the angle between rotated rows depends on the distance alone
        k, q = oracle.rope_rotate(x[:1], [7], f, half), oracle.rope_rotate(x[1:2], [10], f, half)
        k2, q2 = oracle.rope_rotate(x[:1], [1007], f, half), oracle.rope_rotate(x[1:2], [1010], f, half)
        assert np.allclose((k * q).sum(-1), (k2 * q2).sum(-1))


def test_scalings_at_their_ends():
    f = oracle.rope_frequencies(128, 5e5)
    for s in ("by_parts", "by_wavelength"):
        g = oracle.rope_frequencies(128, 5e5, s, **SCALINGS[s])
        assert g[0] == f[0] and np.isclose(g[-1], f[-1] / 8.0)  # fast pairs stay, slow ones are divided
    assert np.isclose(oracle.rope_frequencies(128, 5e5, "ntk", factor=4.0)[-1], f[-1] / 4.0)


def test_quantiser_on_known_rows():
    x = np.zeros((1, 128))
    x[0, :16] = [6, -6, 5, 5.0625, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25, 0.2, -0.3, 0, 1, 2, 4]
    codes, s = oracle.quantise_rows(x, np.zeros(1))
    assert s[0, 0] == 0x38 and (s[0, 1:] == 0).all()            # 1.0
    assert codes[0, :16].tolist() == [7, 15, 6, 7, 6, 4, 4, 2, 2, 0, 0, 9, 0, 2, 4, 6]
    page = oracle.kv4_pack(np.repeat(codes[None], 16, 1), np.repeat(s[None], 16, 1))
    assert page.shape == (1, 16 * 72) and page[0, 0] == 0xF7
    v = oracle.kv4_values(page, np.array([1]))
    assert v[0, 3, :4].tolist() == [12.0, -12.0, 8.0, 12.0]


@pytest.mark.parametrize("rows", [1, 300])
def test_quantiser_is_nearest(rows):
    rng = np.random.default_rng(rows)
    x = oracle.round_bf16(rng.standard_normal((rows, 128)) * np.exp(rng.standard_normal((rows, 1))))
    codes, s = oracle.quantise_rows(x, np.zeros(rows))
    sc = oracle.e4m3_values()[s]
    assert (np.abs(x.reshape(rows, 8, 16)).max(-1) / sc <= 6.0 * 1.0625).all()     # e4m3: within 1/16
    v = (np.where(codes & 8, -1, 1) * oracle.E2M1[codes & 7]).reshape(rows, 8, 16) * sc[..., None]
    every = np.concatenate([oracle.E2M1, -oracle.E2M1])[:, None, None, None] * sc[None, ..., None]
    best = np.abs(every - x.reshape(rows, 8, 16)).min(0)
    assert np.array_equal(np.abs(v - x.reshape(rows, 8, 16)), best)


def test_attention_rows_against_uniform_scores():
    V = np.arange(6.0).reshape(3, 2)
    assert np.allclose(oracle.attention_rows(np.zeros(2), np.ones((3, 2)), V, 1.0), V.mean(0))
    assert not oracle.attention_rows(np.zeros(2), np.zeros((0, 2)), np.zeros((0, 2)), 1.0).any()


# ------------------------------------------------------------------ the library's table
@pytest.mark.parametrize("rot", [32, 64, 96, 128])
@pytest.mark.parametrize("scaling", sorted(SCALINGS))
def test_rope_table(dd, rot, scaling):
    t = dd.rope_host_table(rot, base=5e5, scaling=code_of(dd, scaling), **SCALINGS[scaling]).numpy().tobytes()
    freq = np.frombuffer(t, np.uint64, 64)
    want = oracle.rope_frequencies(rot, 5e5, scaling, **SCALINGS[scaling])
    got = freq[:rot // 2].astype(np.float64) * 2.0 ** -64 * 2.0 * math.pi
    assert np.allclose(got, want, rtol=1e-14, atol=2.0 ** -60) and not freq[rot // 2:].any()
    lut = np.frombuffer(t, np.float32, 2048, 512).astype(np.float64).reshape(512, 4)
    gain = 0.1 * math.log(8.0) + 1.0 if scaling == "by_parts" else 1.0
    a = 2.0 * math.pi * np.arange(512) / 512
    # hi + lo floats: 2^-48 of the gain, and the 64-bit libraries' own last bits
    assert np.abs(lut[:, 0] + lut[:, 2] - gain * np.cos(a)).max() < 2.0 ** -47
    assert np.abs(lut[:, 1] + lut[:, 3] - gain * np.sin(a)).max() < 2.0 ** -47


@pytest.mark.parametrize("bad", [
    dict(rot_dim=0), dict(rot_dim=48), dict(rot_dim=160), dict(base=1.0), dict(base=float("nan")),
    dict(base=float("inf")), dict(scaling=5), dict(scaling=-1), dict(scaling=1, factor=0.5),
    dict(scaling=2, factor=float("inf")), dict(scaling=3, factor=2.0, orig_len=0.0),
    dict(scaling=4, factor=2.0, orig_len=4096.0, beta_fast=1.0, beta_slow=1.0),
    dict(scaling=4, factor=2.0, orig_len=4096.0, beta_fast=1.0, beta_slow=-1.0), dict(gain=float("nan")),
])
def test_rope_table_refuses(dd, bad):
    with pytest.raises(dd.DDError):
        dd.rope_host_table(**{"rot_dim": 128, **bad})


def test_calls_without_a_context_are_refused(dd):
    lib = dd._lib
    assert lib.dd_rope_table(None, None) == dd.DD_ERR_INVALID_ARG
    assert lib.dd_rope_rows(*[None] * 6, 1, 1, None, None, None) == dd.DD_ERR_INVALID_ARG
    assert lib.dd_append_kv(None, None, None) == dd.DD_ERR_INVALID_ARG
    assert lib.dd_gather_kv4(*[None] * 7, 0, None, None, None) == dd.DD_ERR_INVALID_ARG
    assert lib.dd_sparse_attn_decode_kv4(*[None] * 16, 0.0, None, None) == dd.DD_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        dd.rope_table(128, layout=2)
    import torch
    with pytest.raises(ValueError):                               # host rows
        dd._rows(torch.zeros(1, 1, 1, 128, dtype=torch.bfloat16), (1, 1, 1, 128), "x")
