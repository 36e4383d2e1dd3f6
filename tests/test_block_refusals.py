"""Refusals of the recurrent block's operators that keep their arithmetic on sizes inside 32 bits (no GPU: each comes
before a device pointer is touched)."""
import ctypes

import pytest

import selective_scan_gb300 as ss

P = [0x10000 * (i + 1) for i in range(16)]  # aligned addresses that nothing may touch
INV = ss.ERR_INVALID_ARGUMENT
MOST = ss.MAX_BLOCK_SIZE


@pytest.mark.parametrize("size", [MOST + 8, (1 << 31) - 8, (1 << 31) - 1])
def test_sizes_that_a_tile_would_carry_past_32_bits(product_lib, size):
    lib = product_lib
    bf, f32, ws = ss.BF16, ss.F32, (P[12], 1 << 62)
    up = (size + 15) // 16 * 16 if size + 15 < 1 << 31 else MOST // 16 * 16 + 16  # of 16 bytes of 8-bit operands
    for rows, dim in ((size, 64), (1, size)):
        assert lib.mamba2_add_rmsnorm(*P[:6], rows, dim, 1e-5, bf, bf, ss.E4M3, None) == INV
        assert lib.mamba2_add_rmsnorm_backward(*P[:7], rows, dim, 1e-5, f32, f32, *ws, None) == INV
        assert lib.mamba2_add_rmsnorm_backward_workspace_bytes(rows, dim) == 0
        cu = (ctypes.c_int32 * 2)(0, rows)
        b = ss.Batch([0, rows], [0], [1])
        ld = (1 << 33,) * 5
        assert lib.mamba2_gated_recurrence(*P[:6], 1, rows, dim, *ld[:3], bf, b.ref(), *ws, None) == INV
        assert lib.mamba2_gated_recurrence_backward(*P[:10], rows, dim, *ld, bf, cu, 1, *ws, None) == INV
        if dim == size:
            assert lib.mamba2_gated_recurrence_workspace_bytes(cu, 1, dim, 0) == 0
            assert lib.mamba2_gated_recurrence_workspace_bytes(cu, 1, dim, 1) == 0
            assert lib.mamba2_gated_recurrence_step(*P[:5], 1, dim, *ld[:3], bf, b.ref(), None) == INV
            assert lib.mamba2_gated_recurrence_step_device(*P[:5], 1, dim, *ld[:3], bf, P[8], P[9], P[10], 1, P[11], None) == INV
    bf16 = [P[0], P[1], P[2], None, P[4], None, P[6], P[7]]
    for rows, k, n in ((size, 64, 32), (4, up, 32), (4, 64, size)):
        assert lib.mamba2_linear(*bf16, rows, k, n, 1 << 33, 1 << 33, 1 << 33, bf, bf, 0, None) == INV
        assert lib.mamba2_linear_backward(*P[:7], rows, k, n, 1 << 33, 2, *ws, None) == INV
        assert lib.mamba2_linear_backward_workspace_bytes(rows, k, n) == 0


def test_the_largest_size_is_the_headers(product_lib):
    from pathlib import Path
    import re
    text = (Path(ss.__file__).resolve().parent.parent / "include" / "block.h").read_text()
    assert int(re.search(r"#define MAMBA2_MAX_BLOCK_SIZE (0x[0-9a-f]+)", text).group(1), 16) == MOST
    assert product_lib.mamba2_add_rmsnorm_backward_workspace_bytes(MOST, 8) > 0
    assert product_lib.mamba2_linear_backward_workspace_bytes(1, MOST // 8 * 8, 8) > 0


def test_a_batch_of_fewer_boundaries_than_runs(product_lib):
    """The library reads one more boundary than there are slots."""
    with pytest.raises(ValueError):
        ss.Batch([0, 4], [0, 1], [1, 1])
    with pytest.raises(ValueError):
        ss.Batch([], [0], [1])
    assert ss.Batch([0, 4, 4], [0, 1], [1, 1]).rb.num_seqs == 2
    assert ss.Batch(None, [0, 1], [1, 1]).rb.num_seqs == 2 and ss.Batch([0], [], []).rb.num_seqs == 0
    assert ss.Batch([], [], []).rb.num_seqs == 0
