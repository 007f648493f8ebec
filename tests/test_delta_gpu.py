"""The gated delta rule (m3_delta_fwd, m3_delta_step, m3_delta_bwd) on a B200
against the definition in 64 bits.

Tolerances, relative 2-norm.
  float32 values (states, and everything with float32 io): 2e-5.  A half step of
    float32 is 2^-24 = 6e-8; the longest sums here are the dot products of up
    to 256 terms, off by at most 256 half steps of their terms, plus the few
    operations of an update, and the recurrence contracts earlier errors:
    under 335 half steps = 2e-5.  The chunked path keeps every operand of the
    state's chain as sums of bfloat16 parts with at least 16 bits (an error of
    2^-17 = 7.6e-6 each), which stays inside too.
  bfloat16 y: 2^-8.  One rounding is off by up to 2^-8 of the value, 2^-8 /
    sqrt(3) in the 2-norm of many values; y has its own rounding and at most
    two operands of a product rounded to bfloat16, together 2^-8.
  bfloat16 gradients: 6e-3.  Their own rounding and at most six roundings of
    operands on the way, sqrt(7) 2^-8 / sqrt(3) = 6.0e-3.
Where a tensor has few values (a single token of a tiny head) one rounding is
off by up to 2^-8 = 3.9e-3 of the largest value, inside the same bounds.
"""
import numpy as np
import pytest
import torch

from tests._delta_ref import delta, delta_grads, delta_inputs, rel

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import selective_state_space_m3_b200 as m3

F32, Y16, D16 = 2e-5, 2.0 ** -8, 6e-3


def _dims(x, seqlen=None):
    b, t, h, p = x["v"].shape
    g, n = x["q"].shape[2:]
    return m3.Dims(b, t if seqlen is None else seqlen, h, g, p, n, 1, 64,
                   m3.M3_BF16 if x["v"].dtype == torch.bfloat16 else m3.M3_F32)


def _cuda(x):
    return {k: None if v is None else v.cuda() for k, v in x.items()}


def _fwd(x, scale, lengths=None, init=True, y=None, ws=None):
    d, c = _dims(x), _cuda(x)
    y = torch.full_like(c["v"], float("nan")) if y is None else y
    ws = torch.zeros(m3.m3_delta_workspace_size(d), dtype=torch.uint8, device="cuda") if ws is None else ws
    h = torch.full_like(c["h0"], float("nan"))
    m3.m3_delta_fwd(d, c["q"], c["k"], c["v"], c["g"], c["beta"], y, ws, scale=scale,
                    lengths=None if lengths is None else lengths.to(torch.int32).cuda(),
                    init_h=c["h0"] if init else None, final_h=h)
    assert m3.m3_device_status(ws) == m3.M3_OK
    return y, h


def _bwd(x, scale, lengths=None, init=True, d_final=True):
    d, c = _dims(x), _cuda(x)
    io = x["v"].dtype
    grads = {"d" + k: torch.full_like(c[k], float("nan")) for k in ("q", "k", "v")}
    for k in ("g", "beta"):
        grads["d" + k] = torch.full(x["beta"].shape, float("nan"), device="cuda", dtype=io)
    dh0 = torch.full_like(c["h0"], float("nan"))
    ws = torch.zeros(m3.m3_delta_bwd_workspace_size(d), dtype=torch.uint8, device="cuda")
    m3.m3_delta_bwd(d, c["q"], c["k"], c["v"], c["g"], c["beta"], c["dy"], grads, ws, scale=scale,
                    lengths=None if lengths is None else lengths.to(torch.int32).cuda(),
                    init_h=c["h0"] if init else None, d_final_h=c["dh"] if d_final else None, d_init_h=dh0)
    assert m3.m3_device_status(ws) == m3.M3_OK
    grads["dh0"] = dh0
    return grads


def _check_fwd(x, y, h, scale, lengths=None, init=True):
    wy, wh = delta(x["q"], x["k"], x["v"], x["g"], x["beta"], scale, x["h0"] if init else None, lengths)
    bf = x["v"].dtype == torch.bfloat16
    if lengths is not None:
        y = y.clone()
        for i, n in enumerate(lengths.clamp(0, y.shape[1]).tolist()):
            assert bool(torch.isnan(y[i, n:]).all()), "rows behind a sequence's end were written"
            y[i, n:] = 0
    ry, rh = rel(y, wy), rel(h, wh)
    print(f"y {ry:.2e} h {rh:.2e}")
    assert ry <= (Y16 if bf else F32) and rh <= F32


def _check_bwd(x, g, scale, lengths=None, init=True, d_final=True):
    want = delta_grads(x, scale, lengths, init=True, d_final=d_final) if init else \
        delta_grads({**x, "h0": torch.zeros_like(x["h0"])}, scale, lengths, init=True, d_final=d_final)
    bf = x["v"].dtype == torch.bfloat16
    got = {k: rel(g["d" + k], w) for k, w in want.items()}
    print(" ".join(f"d{k} {r:.2e}" for k, r in got.items()))
    for k, r in got.items():
        assert r <= (D16 if bf and k != "h0" else F32), (k, r)


BF, FL = torch.bfloat16, torch.float32
# batch, tokens, heads, groups, headdim, dstate
SHAPES = [
    (1, 1, 1, 1, 1, 2, FL), (2, 3, 2, 1, 5, 6, FL), (2, 17, 4, 2, 40, 48, FL), (1, 33, 2, 2, 16, 256, FL),
    (1, 16, 3, 3, 64, 128, FL), (1, 50, 2, 1, 17, 30, BF), (3, 1, 4, 1, 64, 128, BF), (1, 63, 2, 2, 64, 128, BF),
    (2, 64, 2, 1, 64, 128, BF), (1, 65, 4, 2, 64, 128, BF), (1, 193, 2, 1, 64, 128, BF), (1, 130, 2, 2, 128, 128, BF),
    (1, 129, 1, 1, 64, 64, BF),
]
IDS = ["b%d_t%d_h%d_g%d_p%d_n%d_%s" % (*s[:6], "bf16" if s[6] == BF else "f32") for s in SHAPES]


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
@pytest.mark.parametrize("init", [False, True])
def test_prefill(shape, init):
    x = delta_inputs(*shape, seed=11)
    y, h = _fwd(x, 0.125, init=init)
    _check_fwd(x, y, h, 0.125, init=init)


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
@pytest.mark.parametrize("carry", [False, True])
def test_gradient(shape, carry):
    x = delta_inputs(*shape, seed=12)
    _check_bwd(x, _bwd(x, 0.25, init=carry, d_final=carry), 0.25, init=carry, d_final=carry)


@pytest.mark.parametrize("path", ["", "token"])
@pytest.mark.parametrize("dtype", [BF, FL])
def test_padded_batch(dtype, path, monkeypatch):
    """Lengths 0, 1, in between, all, and out of range; what stands behind a
    sequence's end (NaN) reaches nothing."""
    monkeypatch.setenv("M3_DELTA_PATH", path)
    x = delta_inputs(7, 150, 2, 1, 64, 128, dtype, seed=13)
    lengths = torch.tensor([0, 1, 64, 65, 150, -3, 1000])
    for i, n in enumerate(lengths.clamp(0, 150).tolist()):
        for k in ("q", "k", "v", "dy"):
            x[k][i, n:] = float("nan")
        x["g"][i, n:] = float("inf")
        x["beta"][i, n:] = float("nan")
    clean = {k: torch.nan_to_num(v, nan=0.0, posinf=0.0) for k, v in x.items()}
    y, h = _fwd(x, 0.1, lengths)
    _check_fwd(clean, y, h, 0.1, lengths)
    g = _bwd(x, 0.1, lengths)
    _check_bwd(clean, g, 0.1, lengths)
    for i, n in enumerate(lengths.clamp(0, 150).tolist()):
        for k in ("dq", "dk", "dv", "dg", "dbeta"):
            assert float(g[k][i, n:].float().abs().sum()) == 0.0, k


@pytest.mark.parametrize("path", ["", "token"])
@pytest.mark.parametrize("dtype", [BF, FL])
def test_degenerate_values(dtype, path, monkeypatch):
    """No decay, a full reset (g = -inf), tokens that write nothing (beta = 0),
    zero keys, the same unit key many times with beta = 1, strong decay."""
    monkeypatch.setenv("M3_DELTA_PATH", path)
    x = delta_inputs(6, 140, 2, 2, 64, 128, dtype, seed=14)
    x["g"][0] = 0.0
    x["g"][1, ::37] = float("-inf")
    x["beta"][2, 5:90] = 0.0
    x["k"][3, 10:50] = 0.0
    x["k"][4] = x["k"][4, :1]
    x["beta"][4] = 1.0
    x["g"][5] = -30.0
    y, h = _fwd(x, 0.1)
    _check_fwd(x, y, h, 0.1)
    g = _bwd(x, 0.1)
    _check_bwd(x, g, 0.1)
    none = {**x, "g": None}
    zero = {**x, "g": torch.zeros_like(x["g"])}
    (y0, h0), (y1, h1) = _fwd(none, 0.1), _fwd(zero, 0.1)
    assert torch.equal(y0, y1) and torch.equal(h0, h1)
    g0, g1 = _bwd(none, 0.1), _bwd(zero, 0.1)
    assert all(torch.equal(g0[k], g1[k]) for k in ("dq", "dk", "dv", "dbeta", "dh0"))


STEPS = [(1, 8, 1, 64, 128, BF), (5, 4, 2, 64, 128, FL), (3, 2, 1, 128, 128, BF), (2, 2, 2, 16, 256, BF),
         (2, 3, 3, 256, 64, FL), (2, 2, 1, 40, 48, BF), (1, 1, 1, 1, 2, FL), (2, 2, 1, 256, 128, BF)]


@pytest.mark.parametrize("shape", STEPS, ids=["b%d_h%d_g%d_p%d_n%d_%s" % (*s[:5], str(s[5])[6:]) for s in STEPS])
def test_step(shape):
    b, h, g, p, n, dtype = shape
    x = delta_inputs(b, 1, h, g, p, n, dtype, seed=15)
    c, d = _cuda(x), _dims(x)
    wy, wh = delta(x["q"], x["k"], x["v"], x["g"], x["beta"], 0.3, x["h0"])
    y, out = torch.empty_like(c["v"]), torch.empty_like(c["h0"])
    m3.m3_delta_step(d, c["h0"], c["q"], c["k"], c["v"], c["g"], c["beta"], y, scale=0.3, h_out=out)
    assert torch.equal(c["h0"].cpu(), x["h0"])
    assert rel(y, wy) <= (Y16 if dtype == BF else F32) and rel(out, wh) <= F32
    y2 = torch.empty_like(y)
    m3.m3_delta_step(d, c["h0"], c["q"], c["k"], c["v"], c["g"], c["beta"], y2, scale=0.3)   # in place
    assert torch.equal(y, y2) and torch.equal(out, c["h0"])


@pytest.mark.parametrize("dtype", [BF, FL])
def test_prefill_resumed_and_followed_by_steps(dtype):
    """Prefill of 100 = prefill of 37, resumed for 60, then 3 single tokens."""
    x = delta_inputs(2, 100, 4, 2, 64, 128, dtype, seed=16)
    y, h = _fwd(x, 0.1)
    cut = lambda a, b: {k: (v[:, a:b].contiguous() if k in ("q", "k", "v", "g", "beta", "dy") else v) for k, v in x.items()}
    ya, ha = _fwd(cut(0, 37), 0.1)
    mid = {**cut(37, 97), "h0": ha.cpu()}
    yb, hb = _fwd(mid, 0.1)
    parts = [ya, yb]
    for t in range(97, 100):
        c = _cuda(cut(t, t + 1))
        yt = torch.empty_like(c["v"])
        m3.m3_delta_step(_dims(cut(t, t + 1)), hb, c["q"], c["k"], c["v"], c["g"], c["beta"], yt, scale=0.1)
        parts.append(yt)
    # two results, each within its bound of the exact one
    assert rel(torch.cat(parts, 1), y) <= 2 * (Y16 if dtype == BF else F32)
    assert rel(hb, h) <= 2 * F32
    _check_fwd(x, torch.cat(parts, 1), hb, 0.1)


def test_long_sequence_keeps_its_accuracy():
    x = delta_inputs(1, 3000, 1, 1, 64, 128, BF, seed=17)
    y, h = _fwd(x, 0.1)
    _check_fwd(x, y, h, 0.1)
    assert torch.equal(y, _fwd(x, 0.1)[0])


@pytest.mark.parametrize("dtype", [BF, FL])
def test_results_repeat_bit_by_bit(dtype):
    x = delta_inputs(2, 90, 8, 2, 64, 128, dtype, seed=18)
    a, b = _bwd(x, 0.1), _bwd(x, 0.1)
    assert all(torch.equal(a[k], b[k]) for k in a)


def test_gradient_against_differences():
    """Central differences of the library's own prefill, float32 io: a step of
    1e-2 leaves truncation of (1e-2)^2 and rounding of 2e-5 / 1e-2 relative."""
    x = delta_inputs(1, 20, 2, 1, 16, 16, FL, seed=19)
    g = _bwd(x, 0.5)

    def value(z):
        y, h = _fwd(z, 0.5)
        return float((y.cpu().double() * x["dy"].double()).sum() + (h.cpu().double() * x["dh"].double()).sum())

    gen = torch.Generator().manual_seed(1)
    for k in ("q", "k", "v", "g", "beta", "h0"):
        way = torch.randn(x[k].shape, generator=gen)
        way = way / way.norm()
        slope = (value({**x, k: x[k] + 1e-2 * way}) - value({**x, k: x[k] - 1e-2 * way})) / 2e-2
        want = float((g["d" + k].cpu().double() * way.double()).sum())
        size = float(g["d" + k].double().norm())
        assert abs(slope - want) <= 5e-3 * size, (k, slope, want, size)


@pytest.mark.parametrize("dtype", [BF, FL])
def test_captured_and_replayed(dtype):
    """Prefill, step and gradient in one CUDA graph, replayed on new inputs,
    beside an eager call on another stream with its own workspace."""
    x = delta_inputs(2, 70, 2, 1, 64, 128, dtype, seed=20)
    z = delta_inputs(2, 70, 2, 1, 64, 128, dtype, seed=21)
    c, d = _cuda(x), _dims(x)
    y, h = torch.empty_like(c["v"]), torch.empty_like(c["h0"])
    one = {k: c[k][:, 0].contiguous() for k in ("q", "k", "v", "g", "beta")}
    y1, h1 = torch.empty_like(one["v"]), torch.empty_like(c["h0"])
    grads = {"d" + k: torch.empty_like(c[k]) for k in ("q", "k", "v")}
    for k in ("g", "beta"):
        grads["d" + k] = torch.empty(x["beta"].shape, device="cuda", dtype=dtype)
    ws = torch.zeros(max(m3.m3_delta_workspace_size(d), m3.m3_delta_bwd_workspace_size(d)), dtype=torch.uint8, device="cuda")

    def calls():
        m3.m3_delta_fwd(d, c["q"], c["k"], c["v"], c["g"], c["beta"], y, ws, scale=0.1, init_h=c["h0"], final_h=h)
        m3.m3_delta_step(d, h, one["q"], one["k"], one["v"], one["g"], one["beta"], y1, scale=0.1, h_out=h1)
        m3.m3_delta_bwd(d, c["q"], c["k"], c["v"], c["g"], c["beta"], c["dy"], grads, ws, scale=0.1, init_h=c["h0"])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for k in ("q", "k", "v", "g", "beta", "h0", "dy"):
        c[k].copy_(z[k].cuda())
    graph.replay()
    with torch.cuda.stream(side):
        ye, he = _fwd(x, 0.1)
    torch.cuda.synchronize()
    wy, wh = _fwd(z, 0.1)
    assert torch.equal(y, wy) and torch.equal(h, wh)
    want = _bwd(z, 0.1, d_final=False)
    assert all(torch.equal(grads[k], want[k]) for k in grads)
    _check_fwd(x, ye, he, 0.1)


def test_state_past_32_bits():
    """A decode batch whose state has more than 2^31 elements (8.6 GB)."""
    b, h, p, n = 8200, 32, 64, 128
    gen = torch.Generator(device="cuda").manual_seed(3)
    io = dict(device="cuda", dtype=BF)
    hst = torch.zeros(b, h, n, p, device="cuda")
    hst[-2:].normal_(generator=gen)
    q = torch.randn(b, 1, n, generator=gen, **io) * 0.08
    k = torch.randn(b, 1, n, generator=gen, **io) * 0.08
    v = torch.randn(b, h, p, generator=gen, **io)
    g, beta = -torch.rand(b, h, generator=gen, device="cuda"), torch.rand(b, h, generator=gen, device="cuda")
    y = torch.empty_like(v)
    last = [t[-2:].cpu() for t in (q, k, v, g, beta, hst)]
    m3.m3_delta_step(m3.Dims(b, 1, h, 1, p, n, 1, 64, m3.M3_BF16), hst, q, k, v, g, beta, y)
    wy, wh = delta(last[0][:, None], last[1][:, None], last[2][:, None], last[3][:, None], last[4][:, None], 1.0, last[5])
    assert rel(y[-2:], wy[:, 0]) <= Y16 and rel(hst[-2:], wh) <= F32


def test_empty_calls_pass_the_state_through():
    x = delta_inputs(2, 4, 2, 1, 16, 16, FL, seed=22)
    c, d = _cuda(x), _dims(x, seqlen=0)
    e = lambda t: t[:, :0].contiguous()
    h = torch.empty_like(c["h0"])
    ws = torch.zeros(m3.m3_delta_workspace_size(d), dtype=torch.uint8, device="cuda")
    m3.m3_delta_fwd(d, e(c["q"]), e(c["k"]), e(c["v"]), e(c["g"]), e(c["beta"]), e(c["v"]), ws, init_h=c["h0"], final_h=h)
    assert torch.equal(h, c["h0"])
    m3.m3_delta_fwd(d, e(c["q"]), e(c["k"]), e(c["v"]), e(c["g"]), e(c["beta"]), e(c["v"]), ws, final_h=h)
    assert float(h.abs().sum()) == 0.0


def test_norm_projections_delta_rule_and_back():
    """A layer as it is used: residual norm, projections, key and query norms,
    the delta rule, and all their gradients, against differentiation in 64 bits
    of the same layer (float32 io: 2e-5 of each part, ten parts in a row)."""
    b, t, d, h, g, p, n = 2, 45, 64, 4, 2, 16, 32
    gen = torch.Generator().manual_seed(5)
    x, r = torch.randn(b, t, d, generator=gen), torch.randn(b, t, d, generator=gen)
    w = 1 + 0.1 * torch.randn(d, generator=gen)
    wq, wk, wv = (torch.randn(d, m, generator=gen) / d ** 0.5 for m in (g * n, g * n, h * p))
    wn = torch.full((n,), n ** -0.5)
    gate, beta = -torch.rand(b, t, h, generator=gen), torch.rand(b, t, h, generator=gen)
    dy = torch.randn(b, t, h, p, generator=gen)
    eps = 1e-5
    # 64 bits
    from tests._delta_ref import norm
    leaf = [v.double().requires_grad_() for v in (x, r, w, wq, wk, wv)]
    s_, z_ = norm(leaf[0], eps, leaf[1], leaf[2])
    q_ = norm((z_ @ leaf[3]).reshape(b, t, g, n), eps, weight=wn)[1]
    k_ = norm((z_ @ leaf[4]).reshape(b, t, g, n), eps, weight=wn)[1]
    y_, _ = delta(q_, k_, (z_ @ leaf[5]).reshape(b, t, h, p), gate, beta, 0.2)
    want = torch.autograd.grad((y_ * dy.double()).sum() + s_.sum(), leaf)
    # the library
    f = dict(device="cuda", dtype=FL)
    x, r, w, wq, wk, wv, wn, gate, beta, dy = (v.cuda() for v in (x, r, w, wq, wk, wv, wn, gate, beta, dy))
    s, z = torch.empty_like(x), torch.empty_like(x)
    m3.m3_rms_norm_fwd(x, eps, residual=r, weight=w, sum=s, y=z)
    zz = z.reshape(-1, d)
    qp, kp, v = (zz @ wq).reshape(b, t, g, n), (zz @ wk).reshape(b, t, g, n), (zz @ wv).reshape(b, t, h, p)
    q, k = torch.empty_like(qp), torch.empty_like(kp)
    m3.m3_rms_norm_fwd(qp, eps, weight=wn, y=q)
    m3.m3_rms_norm_fwd(kp, eps, weight=wn, y=k)
    dims = m3.Dims(b, t, h, g, p, n, 1, 64, m3.M3_F32)
    ws = torch.zeros(m3.m3_delta_bwd_workspace_size(dims), dtype=torch.uint8, device="cuda")
    y = torch.empty_like(v)
    m3.m3_delta_fwd(dims, q, k, v, gate, beta, y, ws, scale=0.2)
    assert rel(y, y_) <= 10 * F32
    gr = {"dq": torch.empty_like(q), "dk": torch.empty_like(k), "dv": torch.empty_like(v),
          "dg": torch.empty_like(gate), "dbeta": torch.empty_like(beta)}
    m3.m3_delta_bwd(dims, q, k, v, gate, beta, dy, gr, ws, scale=0.2)
    wsn = torch.zeros(max(m3.m3_rms_norm_bwd_workspace_size(b * t, d, m3.M3_F32),
                          m3.m3_rms_norm_bwd_workspace_size(b * t * g, n, m3.M3_F32)), dtype=torch.uint8, device="cuda")
    dqp, dkp = torch.empty_like(qp), torch.empty_like(kp)
    m3.m3_rms_norm_bwd(qp, gr["dq"], eps, dqp, wsn, weight=wn)
    m3.m3_rms_norm_bwd(kp, gr["dk"], eps, dkp, wsn, weight=wn)
    a, bb, cc = dqp.reshape(-1, g * n), dkp.reshape(-1, g * n), gr["dv"].reshape(-1, h * p)
    dz = (a @ wq.T + bb @ wk.T + cc @ wv.T).reshape(b, t, d)
    dx, dw = torch.empty_like(x), torch.empty(d, **f)
    m3.m3_rms_norm_bwd(s, dz, eps, dx, wsn, weight=w, d_sum=torch.ones_like(s), dweight=dw)
    got = (dx, dx, dw, zz.T @ a, zz.T @ bb, zz.T @ cc)
    for name, gv, wv_ in zip(("x", "r", "w", "wq", "wk", "wv"), got, want):
        assert rel(gv, wv_) <= 10 * F32, (name, rel(gv, wv_))
