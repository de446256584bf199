"""Rotation at the farthest positions, from the table's own 64-bit frequencies."""
import numpy as np
import pytest

import oracle
from sparse_kv_offload_gb300 import synth

import dd_testlib as tl
from test_kv_cache_oracle import SCALINGS, code_of

pytestmark = pytest.mark.gpu

D = 128


@pytest.mark.parametrize("start", [(1 << 20) + 3, (1 << 27) - 9, (1 << 31) - 40, (1 << 31) - 1])
@pytest.mark.parametrize("rot,half,scaling", [(128, True, "plain"), (96, False, "by_parts"), (32, True, "ntk"),
                                              (64, False, "by_wavelength")])
def test_far_positions(rot, half, scaling, start):
    import torch
    from sparse_kv_offload_gb300 import build
    build.build()
    from sparse_kv_offload_gb300 import dd
    T, H = 45, 3
    rng = np.random.default_rng(start % 1000)
    x = synth.f32_to_bf16(rng.standard_normal((1, T, H, D)).astype(np.float32))
    kw = dict(base=5e5, scaling=code_of(dd, scaling), **SCALINGS[scaling])
    freq = np.frombuffer(dd.rope_host_table(rot, **kw).numpy().tobytes(), np.uint64, 64)[:rot // 2]
    rope = dd.rope_table(rot, layout=dd.ROPE_HALF if half else dd.ROPE_INTERLEAVED, **kw)
    with dd.Context(dd.Shape(1, H, H, D, 64, 16, 1, 1), max_misses=0) as ctx:
        out = torch.zeros(1, T, H, D, dtype=torch.bfloat16, device="cuda")
        ctx.rope(rope, tl.to_bf16(x), out, tl.to_i32([start]))
        assert ctx.status() == 0
    # whole numbers modulo a turn, then 53 bits of what is left
    turn = np.array([[(start + t) * int(f) % 2 ** 64 / 2 ** 64 for f in freq] for t in range(T)]) * (2.0 * np.pi)
    gain = 0.1 * np.log(8.0) + 1.0 if scaling == "by_parts" else 1.0
    v = oracle.bf16_decode(x)[0]
    i = np.arange(rot // 2)
    a, b = (i, i + rot // 2) if half else (2 * i, 2 * i + 1)
    c, s = gain * np.cos(turn)[:, None], gain * np.sin(turn)[:, None]
    want = v.copy()
    want[..., a], want[..., b] = v[..., a] * c - v[..., b] * s, v[..., b] * c + v[..., a] * s
    got = oracle.bf16_decode(tl.from_bf16(out))[0]
    # half a bf16 step, and 2^-34 of the largest value: the kernel's 2^-36 of each of two, doubled for their sum
    step = np.ldexp(1.0, np.frexp(want)[1] - 8)
    assert (np.abs(got - want) <= step / 2 + np.abs(v).max() * gain * 2.0 ** -34).all()
