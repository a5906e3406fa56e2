"""Rows of codes that end where their array ends."""
import pytest

from test_gpu_i8 import gen, guarded, guards_ok, mpq  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cols", [1, 2, 3, 5, 127, 1023, 4095, 16385])
def test_dequantize_a_row_without_padding(mpq, cols):
    """One row of codes with nothing behind its last column, out to any alignment."""
    import torch
    codes = torch.randint(-128, 128, (1, cols), generator=gen(cols), device="cuda", dtype=torch.int8)
    q = mpq.i8_matrix(codes, torch.tensor([0.75], device="cuda"))
    for dt in (torch.float32, torch.bfloat16):
        for extra in (0, 1, 2, 3, 8):
            buf, out = guarded(1, cols, dt, extra)
            mpq.i8_dequantize(q, out=out)
            assert torch.equal(out, (codes.float() * 0.75).to(dt)) and guards_ok(buf, 1, cols)
