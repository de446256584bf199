"""The rotation table's frequencies against 50-digit arithmetic: the nearest 64-bit fractions of a turn."""
from decimal import ROUND_CEILING, ROUND_FLOOR, Decimal as Dec, getcontext

import numpy as np
import pytest

from test_kv_cache_oracle import SCALINGS, code_of

PI = Dec("3.1415926535897932384626433832795028841971693993751058209749445923078164062862089986280348253421170679")


@pytest.fixture(scope="module")
def dd():
    from sparse_kv_offload_gb300 import build
    build.build()
    from sparse_kv_offload_gb300 import dd as mod
    return mod


def exact_turns(rot, base, scaling, factor=1.0, orig_len=0.0, beta_fast=32.0, beta_slow=1.0):
    """Turns per position of each pair."""
    getcontext().prec = 50
    base, factor, orig_len, fast, slow = (Dec(float(v)) for v in (base, factor, orig_len, beta_fast, beta_slow))
    if scaling == "ntk":
        base = base * factor ** (Dec(rot) / (rot - 2))
    if scaling == "by_parts":
        lo, hi = (rot * (orig_len / (2 * PI * t)).ln() / (2 * base.ln()) for t in (fast, slow))
        lo = max(lo.to_integral_value(ROUND_FLOOR), Dec(0))
        hi = min(hi.to_integral_value(ROUND_CEILING), Dec(rot - 1))
    out = []
    for i in range(rot // 2):
        f = base ** (Dec(-2 * i) / rot)
        if scaling == "linear":
            f = f / factor
        elif scaling == "by_parts":
            r = min(max((i - lo) / max(hi - lo, Dec(0.001)), Dec(0)), Dec(1))
            f = f * (1 - r) + f / factor * r
        elif scaling == "by_wavelength":
            s = min(max((orig_len * f / (2 * PI) - slow) / (fast - slow), Dec(0)), Dec(1))
            f = f * s + f / factor * (1 - s)
        out.append(f / (2 * PI))
    return out


@pytest.mark.parametrize("base", [1.0 + 2.0 ** -40, 2.0, 1e4, 5e5, 1e7 / 3.0, 1e300])
@pytest.mark.parametrize("scaling", sorted(SCALINGS))
def test_frequencies_are_the_nearest_fractions_of_a_turn(dd, scaling, base):
    for rot in (32, 64, 96, 128):
        for factor in (None, 1.0, 3.7):
            kw = dict(SCALINGS[scaling])
            if factor and "factor" in kw:
                kw["factor"] = factor
            t = dd.rope_host_table(rot, base=base, scaling=code_of(dd, scaling), **kw).numpy().tobytes()
            freq = np.frombuffer(t, np.uint64, 64)
            for i, want in enumerate(exact_turns(rot, base, scaling, **kw)):
                # half a unit of 2^-64 turns, and what pairs of doubles add: some 2^-95 of 2^62 units
                assert abs(Dec(int(freq[i])) - want * 2 ** 64) <= Dec("0.5") + Dec(2) ** -30, (rot, i, factor)


def test_borders_of_the_ramps(dd):
    """Wavelength borders next to each other and contexts of any length: pairs stay or are divided, nothing overflows."""
    plain = np.frombuffer(dd.rope_host_table(128, base=5e5).numpy().tobytes(), np.uint64, 64)
    divided = np.frombuffer(dd.rope_host_table(128, base=5e5, scaling=dd.ROPE_LINEAR, factor=8.0).numpy().tobytes(),
                            np.uint64, 64)
    for orig_len, want in ((1e300, plain), (1e-300, divided)):
        for slow in (1.0, 1e-290, 1e290):
            if (orig_len > 1.0) == (slow > 1.0) and slow != 1.0:
                continue
            t = dd.rope_host_table(128, base=5e5, scaling=dd.ROPE_BY_WAVELENGTH, factor=8.0, orig_len=orig_len,
                                   beta_slow=slow, beta_fast=float(np.nextafter(slow, np.inf)))
            assert np.array_equal(np.frombuffer(t.numpy().tobytes(), np.uint64, 64), want)
    for orig_len, want in ((1e300, plain), (1e-300, divided)):
        t = dd.rope_host_table(128, base=5e5, scaling=dd.ROPE_BY_PARTS, factor=8.0, orig_len=orig_len, beta_slow=1.0,
                               beta_fast=32.0)
        got = np.frombuffer(t.numpy().tobytes(), np.uint64, 64)
        assert np.array_equal(got[1:], want[1:])       # (the ramp's first pair may lie on its border)
