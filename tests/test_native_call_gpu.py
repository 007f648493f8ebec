"""The binding's two ways to a call -- native argument handling, and the Python
code that takes what the native code hands back -- give the same results and
refuse the same arguments."""
import pytest
import torch

from tests._delta_ref import delta_inputs

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import selective_state_space_m3_b200 as m3


def _step(**over):
    x = {k: v.cuda() for k, v in delta_inputs(2, 1, 4, 2, 64, 128, torch.bfloat16, seed=41).items()}
    d = m3.Dims(2, 1, 4, 2, 64, 128, 1, 64, m3.M3_BF16)
    a = dict(h=x["h0"], q=x["q"], k=x["k"], v=x["v"], g=x["g"], beta=x["beta"], y=torch.zeros_like(x["v"]),
             h_out=torch.zeros_like(x["h0"]), scale=0.5)
    a.update(over)
    m3.m3_delta_step(d, **a)
    return a["y"], a["h_out"]


def test_a_given_stream_and_the_current_one_agree():
    native = _step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    plain = _step(stream=side)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        current = _step()
    torch.cuda.synchronize()
    for a, b, c in zip(native, plain, current):
        assert float(a.float().abs().sum()) > 0 and torch.equal(a, b) and torch.equal(a, c)


def test_the_native_code_takes_the_usual_call():
    x = torch.randn(4, 64, device="cuda")
    y = torch.empty_like(x)
    assert m3._native.rms_norm_fwd(x, 1e-5, None, None, None, y, None, None, 0) == m3.M3_OK
    assert m3._native.rms_norm_fwd(x, -1.0, None, None, None, y, None, None, 0) == m3.M3_ERR_INVALID_ARG
    with pytest.raises(m3.M3Error):
        m3.m3_rms_norm_fwd(x, -1.0, y=y)


@pytest.mark.parametrize("name", ["h", "q", "k", "v", "g", "beta", "y", "h_out"])
def test_wrong_tensors_are_refused(name):
    shape = {"h": (2, 4, 128, 64), "h_out": (2, 4, 128, 64), "q": (2, 2, 128), "k": (2, 2, 128), "v": (2, 4, 64),
             "y": (2, 4, 64), "g": (2, 4), "beta": (2, 4)}[name]
    io = torch.bfloat16 if name in ("q", "k", "v", "y") else torch.float32
    for bad, error, text in ((torch.zeros(*shape, dtype=torch.float64, device="cuda"), TypeError, name + " is"),
                             (torch.zeros(*shape, 2, dtype=io, device="cuda"), ValueError, "elements"),
                             (torch.zeros(*shape, 2, dtype=io, device="cuda")[..., 0], ValueError, "contiguous"),
                             (torch.zeros(*shape, dtype=io), ValueError, "device")):
        with pytest.raises(error, match=text):
            _step(**{name: bad})


def test_parameters_and_views_are_tensors_like_others():
    x = torch.randn(6, 64, device="cuda")
    w = torch.nn.Parameter(torch.rand(64, device="cuda"))
    y, z = torch.empty_like(x), torch.empty_like(x)
    m3.m3_rms_norm_fwd(x, 1e-5, weight=w, y=y)
    m3.m3_rms_norm_fwd(x[2:], 1e-5, weight=w.detach(), y=z[2:])
    torch.cuda.synchronize()
    assert torch.equal(y[2:], z[2:])
