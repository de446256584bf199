"""Pins of the oracle's operators over lists of chunks (CPU): closed forms, torch's softmax attention in 64 bits,
brute force; and the host-side answers of the calls that need no GPU."""
import itertools
import os
import subprocess

import numpy as np
import pytest

import oracle

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
D = 128


def test_attention_over_a_whole_cache_is_causal_softmax_attention():
    import torch
    rng = np.random.default_rng(1)
    T, G, L = 9, 3, 32
    q, K, V = rng.standard_normal((T, G, D)), rng.standard_normal((L, D)), rng.standard_normal((L, D))
    out, lse = oracle.extend_attention(q, L - T, K, V, np.arange(L), D ** -0.5)
    mask = torch.arange(L) <= (L - T + torch.arange(T))[:, None]
    tq, tk, tv = torch.from_numpy(q).transpose(0, 1), torch.from_numpy(K).expand(G, L, D), torch.from_numpy(V).expand(G, L, D)
    want = torch.nn.functional.scaled_dot_product_attention(tq, tk, tv, attn_mask=mask).transpose(0, 1)
    assert np.abs(out - want.numpy()).max() < 1e-12
    x = torch.einsum("gtd,gkd->tgk", tq, tk) * D ** -0.5
    z = torch.logsumexp(x.masked_fill(~mask[:, None], -np.inf), -1)
    assert np.abs(lse - z.numpy()).max() < 1e-12


def test_gaps_and_rows_without_keys():
    rng = np.random.default_rng(2)
    q, K, V = rng.standard_normal((3, 2, D)), rng.standard_normal((32, D)), rng.standard_normal((32, D))
    pos = np.concatenate([np.arange(16), 48 + np.arange(16)])
    out, lse = oracle.extend_attention(q, 47, K, V, pos, 0.1)
    o0, z0 = oracle.extend_attention(q[:1], 47, K[:16], V[:16], pos[:16], 0.1)
    assert np.array_equal(out[0], o0[0]) and np.array_equal(lse[0], z0[0])
    o1, _ = oracle.extend_attention(q[1:2], 48, K[:17], V[:17], pos[:17], 0.1)
    assert np.allclose(out[1], o1[0], rtol=0, atol=1e-14)
    out, lse = oracle.extend_attention(q, 0, K, V, pos + 100, 0.1)
    assert (out == 0).all() and np.isneginf(lse).all()


def test_one_row_and_equal_rows():
    rng = np.random.default_rng(3)
    q, V = rng.standard_normal((1, 1, D)), rng.standard_normal((16, D))
    K = np.repeat(rng.standard_normal((1, D)), 16, 0)
    out, lse = oracle.extend_attention(q, 15, K, V, np.arange(16), 1.0)
    assert np.allclose(out[0, 0], V.mean(0)) and np.isclose(lse[0, 0], K[0] @ q[0, 0] + np.log(16))
    out, lse = oracle.extend_attention(q, 0, K, V, np.arange(16), 1.0)
    assert np.allclose(out[0, 0], V[0]) and np.isclose(lse[0, 0], K[0] @ q[0, 0])


def test_weights_of_a_row_add_up_to_one():
    rng = np.random.default_rng(4)
    q, K, V = rng.standard_normal((5, 2, D)), rng.standard_normal((64, D)), rng.standard_normal((64, D))
    pos = np.arange(64)
    _, lse = oracle.extend_attention(q, 40, K, V, pos, 0.3)
    w = oracle.chunk_weights(q, 40, lse, K, pos, 16, 0.3)
    assert np.isclose(w.sum(), 10.0) and (w[3:] == 0).all()
    assert np.allclose(w, oracle.chunk_weights(q[:2], 40, lse[:2], K, pos, 16, 0.3) +
                       oracle.chunk_weights(q, 40, lse, K, pos, 16, 0.3, first=2))
    lse[1] = -np.inf
    assert np.isclose(oracle.chunk_weights(q, 40, lse, K, pos, 16, 0.3).sum(), 8.0)


def test_eviction_against_brute_force():
    """Of all sets of E candidates the one with the least weight, then the lexicographically first."""
    rng = np.random.default_rng(5)
    for _ in range(200):
        C, S = 7, 6
        held = rng.choice(C, rng.integers(0, S + 1), replace=False)
        now = np.full(C, -1)
        now[held] = 60 + rng.permutation(S)[:len(held)]
        w = rng.integers(0, 3, C).astype(float)
        n0 = int(rng.integers(0, C + 1))
        n1 = int(rng.integers(n0, C + 1))
        keep, first, last = int(rng.integers(0, S + 1)), int(rng.integers(0, 3)), int(rng.integers(0, 3))
        got, gone, short = oracle.evict_unit(w, now, 60, S, n0, n1, keep, first, last)
        cand = [c for c in sorted(held) if first <= c < n0 - last]
        come = [c for c in range(n0, n1) if now[c] < 0]
        e = min(max(len(held) + len(come) - keep, 0), len(cand))
        # the set whose sorted (weight, chunk) pairs are least
        best = min((tuple(sorted((w[c], c) for c in s)) for s in itertools.combinations(cand, e)))
        assert gone == sorted(c for _, c in best)
        free = S - (len(held) - e)
        assert short == (len(come) > free)
        stay = [c for c in held if c not in gone]
        assert all(got[c] == now[c] for c in stay) and all(got[c] == -1 for c in gone if c not in come)
        given = come[:free]
        used = [got[c] for c in stay + given]
        assert len(set(used)) == len(used) and all(60 <= s < 66 for s in used)
        assert [got[c] for c in given] == sorted(set(range(60, 66)) - {now[c] for c in stay})[:len(given)]


def test_eviction_order_of_nan_and_zeros():
    w = np.array([0.0, -0.0, np.nan, -1.0, 2.0])
    now = np.arange(5)
    for e, want in ((1, [2]), (2, [2, 3]), (3, [0, 2, 3]), (4, [0, 1, 2, 3])):
        assert oracle.evict_unit(w, now, 0, 5, 5, 5, 5 - e, 0, 0)[1] == want


def test_argument_structs_have_the_header_s_layout(tmp_path):
    """Sizes and offsets that the C compiler gives the header's structs, against the binding's."""
    from sparse_kv_offload_gb300 import build
    build.build()
    from sparse_kv_offload_gb300 import dd
    src = tmp_path / "layout.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "dd.h"\nint main(void) {\n'
                   ' printf("%zu %zu %zu %zu %zu %zu\\n", sizeof(dd_extend_args), offsetof(dd_extend_args, workspace_bytes),\n'
                   '   sizeof(dd_weights_args), offsetof(dd_weights_args, decay), sizeof(dd_evict_args),\n'
                   '   offsetof(dd_evict_args, resident_slot));\n return 0;\n}\n')
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    import struct
    assert got == [dd._extend_args.size, 176, dd._weights_args.size, 140, dd._evict_args.size, struct.calcsize("@3P5i") + 4]


def test_host_answers_without_a_context():
    from sparse_kv_offload_gb300 import build
    build.build()
    from sparse_kv_offload_gb300 import dd
    lib = dd._lib
    for name, size in (("dd_extend_attn", 184), ("dd_chunk_weights", 168), ("dd_evict_chunks", 120)):
        assert getattr(lib, name)(None, b"\0" * size, None) == dd.DD_ERR_INVALID_ARG
    assert lib.dd_extend_attn_workspace(None, 5) == -1 and lib.dd_chunk_weights_workspace(None) == -1


@pytest.mark.parametrize("bad", ["dim", "type"])
def test_binding_refuses_without_a_context(bad):
    import torch
    from sparse_kv_offload_gb300 import build
    build.build()
    from sparse_kv_offload_gb300 import dd

    class Shaped(dd.Context):
        def __init__(self):
            self.shape, self.max_misses, self.hot_slots, self._h = dd.Shape(1, 4, 1, D, 64, 16, 4, 1), 0, 4, None
    c = Shaped()
    q = torch.zeros(1, 4, D) if bad == "dim" else torch.zeros(1, 2, 4, D)
    with pytest.raises((TypeError, ValueError)):
        c.extend_attn(q, None, None, None, None, None, None, q)
    with pytest.raises((TypeError, ValueError)):
        c.chunk_weights(q, None, None, None, None, None, None, None)
