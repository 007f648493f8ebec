"""One row of more than 2^30 columns (2 GB of bfloat16), in every form of the
norm that has no scales of 128 columns: every column is written.

The row is made of +-1 and of one 3 at each end, so that the float32 sums are of
whole numbers: a thread adds 2^22 ones (exact below 2^24), 256 threads' sums are
2^30 in all, off by at most 8 half steps of 2^-24, and the square root halves
that.  y is then off by its own rounding, half a step of bfloat16, 2^-8 of the
value; an 8-bit value by half a step of e4m3, 2^-4."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import selective_state_space_m3_b200 as m3

WIDTH = (1 << 30) + 1


def test_every_column_of_a_wide_row_is_written():
    x = torch.ones(1, WIDTH, device="cuda", dtype=torch.bfloat16)
    x[0, 1::3] = -1
    x[0, 0] = x[0, -1] = 3
    y = torch.full_like(x, float("nan"))
    y8 = torch.zeros(1, WIDTH, device="cuda", dtype=torch.float8_e4m3fn)
    scale = torch.full((1, 1), float("nan"), device="cuda")
    m3.m3_rms_norm_fwd(x, 1e-5, y=y, y8=y8, scale=scale)
    rs = ((WIDTH + 16) / WIDTH + 1e-5) ** -0.5
    assert abs(float(scale) * 448 / (3 * rs) - 1) <= 2e-5
    step = 1 << 28
    for c in range(0, WIDTH, step):
        want = x[0, c:c + step].float() * rs
        for got, half in ((y[0, c:c + step].float(), 2.0 ** -8), (y8[0, c:c + step].float() * scale[0], 2.0 ** -4)):
            assert bool(((got - want).abs() <= (half + 2e-5) * want.abs()).all()), c
    del y8
    dx = torch.full_like(x, float("nan"))
    ws = torch.empty(m3.m3_rms_norm_bwd_workspace_size(1, WIDTH, m3.M3_BF16), dtype=torch.uint8, device="cuda")
    m3.m3_rms_norm_bwd(x, x, 1e-5, dx, ws, d_sum=x)
    # the gradient along the row itself is (1 - mean s^2 / (mean s^2 + eps)) rs x: 1e-5 of x, a difference of
    # float32 numbers near 1 (off by at most 1e-6); d_sum is what is left
    for c in range(0, WIDTH, step):
        want = x[0, c:c + step].float()
        assert bool(((dx[0, c:c + step].float() - want).abs() <= (2.0 ** -8 + 2e-5) * want.abs()).all()), c
