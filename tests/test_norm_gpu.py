"""The root-mean-square norm (m3_rms_norm_fwd, m3_rms_norm_bwd) on a B200
against the definition in 64 bits.

Tolerances.  float32 values: 2e-5 relative 2-norm (a sum of up to 40000 squares
or products in float32, added in at most 100 + log2 steps a thread, is off by
well under 335 half steps of 2^-24).  bfloat16 values: 2^-8, their one
rounding.  8-bit values: y8 * scale is off by half a step of e4m3, 2^-4 of the
value, or, below e4m3's smallest normal number 2^-6, by half its spacing there,
2^-10 of the scale; plus 2e-5 for y itself.
"""
import pytest
import torch

from tests._delta_ref import norm, norm_grads, rel

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import selective_state_space_m3_b200 as m3

F32, B16 = 2e-5, 2.0 ** -8
EPS = 1e-5
BF, FL = torch.bfloat16, torch.float32
SHAPES = [(1, 1), (3, 7), (5, 8), (2, 63), (300, 64), (257, 120), (1025, 128), (33, 136), (7, 1000), (300, 2048),
          (1, 2048), (3, 4104), (2, 32768), (2, 32776), (3, 40000)]


def _inputs(rows, width, dtype, seed=3):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, width, generator=gen).to(dtype)
    r = (2 * torch.randn(rows, width, generator=gen)).to(dtype)
    w = 1 + 0.2 * torch.randn(width, generator=gen)
    return x, r, w, torch.randn(rows, width, generator=gen).to(dtype)


def _close(got, want, dtype):
    assert rel(got, want) <= (B16 if dtype == BF else F32), rel(got, want)


@pytest.mark.parametrize("dtype", [BF, FL])
@pytest.mark.parametrize("rows,width", SHAPES)
def test_forward(rows, width, dtype):
    x, r, w, _ = _inputs(rows, width, dtype)
    s, y = norm(x, EPS, r, w)
    xc, rc, wc = x.cuda(), r.cuda(), w.cuda()
    sum_, out = torch.full_like(xc, float("nan")), torch.full_like(xc, float("nan"))
    m3.m3_rms_norm_fwd(xc, EPS, residual=rc, weight=wc, sum=sum_, y=out)
    _close(sum_, s, dtype)
    _close(out, y, dtype)
    m3.m3_rms_norm_fwd(xc, EPS, y=out)
    _close(out, norm(x, EPS)[1], dtype)
    m3.m3_rms_norm_fwd(xc, EPS, residual=rc, weight=wc, sum=xc, y=out)       # the sum over x
    assert torch.equal(xc, sum_)
    _close(out, y, dtype)


@pytest.mark.parametrize("block", [0, 128])
@pytest.mark.parametrize("dtype", [BF, FL])
@pytest.mark.parametrize("rows,width", SHAPES)
def test_eight_bits(rows, width, dtype, block):
    x, r, w, _ = _inputs(rows, width, dtype)
    _, y = norm(x, EPS, r, w)
    step = block or width
    nb = -(-width // step)
    y8 = torch.zeros(rows, width, device="cuda", dtype=torch.float8_e4m3fn)
    scale = torch.full((rows, nb), float("nan"), device="cuda")
    m3.m3_rms_norm_fwd(x.cuda(), EPS, residual=r.cuda(), weight=w.cuda(), y8=y8, scale=scale, scale_block=block)
    want = torch.stack([c.abs().amax(-1) / 448 for c in y.split(step, 1)], 1)
    assert rel(scale, want) <= F32
    wide = want.repeat_interleave(step, 1)[:, :width]
    got = y8.cpu().double() * scale.cpu().double().repeat_interleave(step, 1)[:, :width]
    bound = torch.maximum(y.abs() * 2.0 ** -4, wide * 2.0 ** -10) + F32 * y.abs().amax(-1, keepdim=True)
    assert bool(((got - y).abs() <= bound).all())


def test_rows_of_zeros_and_of_non_numbers():
    x = torch.ones(4, 256)
    x[1] = 0
    x[2, 5] = float("inf")
    x[3, 200] = float("nan")
    y8 = torch.empty(4, 256, device="cuda", dtype=torch.float8_e4m3fn)
    scale = torch.empty(4, 2, device="cuda")
    y = torch.empty(4, 256, device="cuda")
    m3.m3_rms_norm_fwd(x.cuda(), EPS, y=y, y8=y8, scale=scale, scale_block=128)
    y, q, scale = y.cpu(), y8.cpu().float(), scale.cpu()
    assert torch.allclose(y[0], torch.full((256,), (1 + EPS) ** -0.5))
    assert float(y[1].abs().sum()) == 0 and float(q[1].abs().sum()) == 0 and bool(torch.isfinite(scale[1]).all())
    # an infinite element makes the mean square infinite: its row is 0, and inf * 0 in its place
    assert bool(torch.isnan(y[2, 5])) and float(y[2, :5].abs().sum()) == 0
    assert bool(torch.isnan(y[3]).all()) and bool(torch.isnan(scale[3]).all())
    assert float(scale[0, 0]) > 0 and torch.equal(q[0], torch.full((256,), 448.0))


@pytest.mark.parametrize("dtype", [BF, FL])
@pytest.mark.parametrize("rows,width", SHAPES + [(5000, 128), (2000, 72)])
def test_gradient(rows, width, dtype):
    s, e, w, dy = _inputs(rows, width, dtype)
    sc, ec, wc, dc = s.cuda(), e.cuda(), w.cuda(), dy.cuda()
    io = m3.M3_BF16 if dtype == BF else m3.M3_F32
    ws = torch.empty(m3.m3_rms_norm_bwd_workspace_size(rows, width, io), dtype=torch.uint8, device="cuda")
    dx, dw = torch.full_like(sc, float("nan")), torch.full((width,), float("nan"), device="cuda")
    m3.m3_rms_norm_bwd(sc, dc, EPS, dx, ws, weight=wc, d_sum=ec, dweight=dw)
    wx, ww = norm_grads(s, dy, EPS, w, e)
    _close(dx, wx, dtype)
    assert rel(dw, ww) <= F32
    dw2 = torch.empty_like(dw)
    m3.m3_rms_norm_bwd(sc, dc, EPS, dc, ws, weight=wc, d_sum=ec, dweight=dw2)      # over dy
    assert torch.equal(dc, dx) and torch.equal(dw, dw2)
    m3.m3_rms_norm_bwd(sc, dy.cuda(), EPS, dx, ws)
    # one column: the norm of a row of one element hardly depends on it, and the
    # gradient is a difference of equal numbers; its error is that of its terms
    want = norm_grads(s, dy, EPS)[0]
    if width > 1:
        _close(dx, want, dtype)
    else:
        rs = (s.double().square() + EPS).rsqrt()
        assert bool(((dx.cpu().double() - want).abs() <= B16 * want.abs() + F32 * (rs * dy.double()).abs()).all())


def test_captured_and_replayed():
    x, r, w, dy = (t.cuda() for t in _inputs(200, 512, BF))
    s, y, dx, dw = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x), torch.empty_like(w)
    ws = torch.empty(m3.m3_rms_norm_bwd_workspace_size(200, 512, m3.M3_BF16), dtype=torch.uint8, device="cuda")

    def calls():
        m3.m3_rms_norm_fwd(x, EPS, residual=r, weight=w, sum=s, y=y)
        m3.m3_rms_norm_bwd(s, dy, EPS, dx, ws, weight=w, dweight=dw)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    x.copy_(_inputs(200, 512, BF, seed=4)[0])
    graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in (s, y, dx, dw)]
    calls()
    assert all(torch.equal(a, b) for a, b in zip(got, (s, y, dx, dw)))


def test_more_than_32_bits_of_elements():
    """2^31 + some elements of bfloat16 (4.3 GB a tensor): the last rows."""
    rows, width = (1 << 20) + 3, 2048
    x = torch.ones(rows, width, device="cuda", dtype=BF)
    x[-2:] = torch.randn(2, width, device="cuda").to(BF)
    y = torch.empty_like(x)
    m3.m3_rms_norm_fwd(x, EPS, y=y)
    assert rel(y[-2:], norm(x[-2:].cpu(), EPS)[1]) <= B16
    assert bool((y[:-2] == 1).all())
