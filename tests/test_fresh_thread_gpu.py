"""Calls from a host thread that has made no CUDA call of its own (all buffers
come from another thread): they give the results of the thread that has, bit by
bit."""
import threading

import pytest
import torch

import m3_synth
from tests._delta_ref import delta_inputs
from tests._util import dims_of
from tests.test_delta_gpu import _bwd, _cuda, _dims, _fwd
from tests.test_delta_streams_gpu import _outputs

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import selective_state_space_m3_b200 as m3


def _in_a_thread(work):
    errors = []

    def run():
        try:
            work()
        except Exception as e:  # noqa: BLE001 (shown by the test)
            errors.append(repr(e))

    t = threading.Thread(target=run)
    t.start()
    t.join()
    assert not errors, errors


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_delta_rule(dtype):
    x = delta_inputs(2, 70, 2, 1, 64, 128, dtype, seed=81)
    (wy, wh), want = _fwd(x, 0.1), _bwd(x, 0.1, d_final=False)
    c, d = _cuda(x), _dims(x)
    y, h, g, dh0 = torch.empty_like(c["v"]), torch.empty_like(c["h0"]), _outputs(x), torch.empty_like(c["h0"])
    ws = torch.zeros(max(m3.m3_delta_workspace_size(d), m3.m3_delta_bwd_workspace_size(d)), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    _in_a_thread(lambda: m3.m3_delta_fwd(d, c["q"], c["k"], c["v"], c["g"], c["beta"], y, ws, scale=0.1, init_h=c["h0"],
                                         final_h=h))
    _in_a_thread(lambda: m3.m3_delta_bwd(d, c["q"], c["k"], c["v"], c["g"], c["beta"], c["dy"], g, ws, scale=0.1,
                                         init_h=c["h0"], d_init_h=dh0))
    torch.cuda.synchronize()
    assert torch.equal(y, wy) and torch.equal(h, wh)
    assert all(torch.equal(dh0 if k == "dh0" else g[k], w) for k, w in want.items())
    s, n = torch.empty_like(y), torch.empty_like(y)
    _in_a_thread(lambda: m3.m3_rms_norm_fwd(y, 1e-5, y=n))
    m3.m3_rms_norm_fwd(y, 1e-5, y=s)
    assert torch.equal(n, s)


@pytest.mark.parametrize("kernel", ["", "persistent"])
@pytest.mark.parametrize("shape", [(2, 160, 2, 2, 64, 128, 4, 64, "bf16", 0.0, 5), (1, 64, 2, 1, 16, 16, 1, 32, "f32", 0.0, 6)])
def test_scan(shape, kernel, monkeypatch):
    monkeypatch.setenv("M3_TC_KERNEL", kernel)
    s = m3_synth.ScanShape(*shape)
    t, d = {k: v.cuda() for k, v in m3_synth.make_scan_inputs(s).items()}, dims_of(s)
    ws = torch.zeros(m3.m3_scan_workspace_size(d), dtype=torch.uint8, device="cuda")
    a, b = torch.empty_like(t["x"]), torch.empty_like(t["x"])
    args = (t["x"], t["B"], t["C"], t["dt"], t["A"], t["lam"], t["theta"])
    m3.m3_scan_fwd(d, *args, a, ws)
    torch.cuda.synchronize()
    _in_a_thread(lambda: m3.m3_scan_fwd(d, *args, b, ws))
    torch.cuda.synchronize()
    assert torch.equal(a, b)
