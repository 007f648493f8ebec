"""The gradient runs its two chains side by side on a second stream of the
calling thread where both fit the GPU.  Calls of several threads at once, calls
whose first one is captured, and calls on the default stream give the results
of a call alone, bit by bit."""
import threading

import pytest
import torch

from tests._delta_ref import delta_inputs
from tests.test_delta_gpu import _bwd, _check_bwd, _cuda, _dims

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import selective_state_space_m3_b200 as m3

# batch, tokens, heads, groups, headdim: both chains with 16, with 32, with 64 and 32 columns; one after the other
SHAPES = [(2, 200, 2, 1, 64), (4, 130, 8, 2, 64), (5, 130, 9, 9, 64), (6, 130, 9, 3, 64), (2, 70, 2, 2, 256)]


def _outputs(x):
    g = {"d" + k: torch.empty_like(x[k], device="cuda") for k in ("q", "k", "v")}
    for k in ("g", "beta"):
        g["d" + k] = torch.empty(x["beta"].shape, device="cuda", dtype=x["v"].dtype)
    return g


@pytest.mark.parametrize("shape", SHAPES, ids=["b%d_t%d_h%d_g%d_p%d" % s for s in SHAPES])
def test_gradient_of_every_choice(shape):
    b, t, h, g, p = shape
    x = delta_inputs(b, t, h, g, p, 128, torch.bfloat16, seed=51)
    lengths = torch.tensor([t - 13 * i for i in range(b)])
    _check_bwd(x, _bwd(x, 0.2, lengths), 0.2, lengths)


def test_threads_at_once_and_a_first_call_that_is_captured():
    x = [delta_inputs(2, 300, 4, 2, 64, 128, torch.bfloat16, seed=52 + i) for i in range(3)]
    want = [_bwd(z, 0.2, d_final=False) for z in x]
    got, errors = [None] * 3, []

    def work(i):
        try:
            c, d = _cuda(x[i]), _dims(x[i])
            g, dh0 = _outputs(x[i]), torch.empty_like(c["h0"])
            ws = torch.zeros(m3.m3_delta_bwd_workspace_size(d), dtype=torch.uint8, device="cuda")

            def call():
                m3.m3_delta_bwd(d, c["q"], c["k"], c["v"], c["g"], c["beta"], c["dy"], g, ws, scale=0.2,
                                init_h=c["h0"], d_init_h=dh0)
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    call()
                torch.cuda.current_stream().synchronize()
            assert m3.m3_device_status(ws) == m3.M3_OK
            got[i] = {**g, "dh0": dh0}
        except Exception as e:  # noqa: BLE001 (shown by the test)
            errors.append(repr(e))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(3)]
    torch.cuda.synchronize()
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for a, b in zip(got, want):
        assert all(torch.equal(a[k], b[k]) for k in b)

    def captured():
        try:
            c, d = _cuda(x[0]), _dims(x[0])
            g, dh0 = _outputs(x[0]), torch.empty_like(c["h0"])
            ws = torch.zeros(m3.m3_delta_bwd_workspace_size(d), dtype=torch.uint8, device="cuda")
            torch.cuda.synchronize()
            for _ in range(2):               # the second capture has the thread's second stream
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    m3.m3_delta_bwd(d, c["q"], c["k"], c["v"], c["g"], c["beta"], c["dy"], g, ws, scale=0.2,
                                    init_h=c["h0"], d_init_h=dh0)
                for z in (*g.values(), dh0):
                    z.fill_(float("nan"))
                graph.replay()
                graph.replay()
                torch.cuda.synchronize()
                for k, w in want[0].items():
                    assert torch.equal(dh0 if k == "dh0" else g[k], w), k
                m3.m3_delta_bwd(d, c["q"], c["k"], c["v"], c["g"], c["beta"], c["dy"], g, ws, scale=0.2, init_h=c["h0"])
                torch.cuda.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(repr(e))

    t = threading.Thread(target=captured)
    t.start()
    t.join()
    assert not errors, errors
