"""More rows than a grid has CTAs for: refused, as a cut-off grid would leave rows out without a word."""
import pytest

pytestmark = pytest.mark.gpu


def test_too_many_rows_are_refused():
    import torch
    from sparse_kv_offload_gb300 import build
    build.build()
    from sparse_kv_offload_gb300 import dd
    B, L = 40, 16
    T = 2 ** 31 - 1                                    # 40 T / 16 CTAs are 2^30 modulo 2^32
    i32 = dict(dtype=torch.int32, device="cuda")
    row = torch.ones(1, 1, 1, 128, dtype=torch.bfloat16, device="cuda")
    start, one = torch.zeros(B, **i32), torch.ones(B, **i32)
    home = [torch.zeros(B, 1, L, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    rope = dd.rope_table(128)
    zero = dd._strides.pack(0, 0, 0)
    with dd.Context(dd.Shape(B, 1, 1, 128, L, 16, 1, 1), max_misses=0) as ctx:
        rows = row.expand(B, T, 1, 128)                # one row for all of them, of which new_len keeps one a request
        with pytest.raises(dd.DDError):
            ctx.append_kv(rows, rows, start, new_len=one, Kh=home[0], Vh=home[1])
        out = torch.zeros_like(row)
        assert dd._lib.dd_rope_rows(ctx._h, rope._addr, row.data_ptr(), zero, out.data_ptr(), zero, T, 1, start.data_ptr(),
                                    one.data_ptr(), None) == dd.DD_ERR_INVALID_ARG
        assert ctx.launch_count() == 0
        rows = row.expand(B, 300, 1, 128)
        ctx.append_kv(rows, rows, start, new_len=one, Kh=home[0], Vh=home[1])
        assert ctx.status() == 0 and home[0][:, :, 0].all() and not home[0][:, :, 1:].any()
