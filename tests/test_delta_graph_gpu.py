"""Captured gradients of the gated delta rule run their two chains side by side
as uncaptured ones do: in the graph, the kernel of the chunk matrices has two
kernels that depend on it, one a chain.  The results are those of a call alone,
bit by bit."""
import threading

import pytest
import torch

from tests._delta_ref import delta_inputs
from tests.test_delta_gpu import _bwd, _cuda, _dims
from tests.test_delta_streams_gpu import _outputs

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import selective_state_space_m3_b200 as m3

SHAPE = (2, 200, 4, 2, 64, 128, torch.bfloat16)


def _forks(graph):
    """Nodes of a captured graph on which more than one other node depends (not counting
    dependencies that follow from the others), and the number of nodes."""
    from cuda.bindings import runtime as rt
    g = rt.cudaGraph_t(init_value=graph.raw_cuda_graph())
    err, _, nodes = rt.cudaGraphGetNodes(g)
    assert int(err) == 0
    err, _, _, n = rt.cudaGraphGetEdges(g)[:4]
    assert int(err) == 0
    if not n:
        return 0, nodes
    out = rt.cudaGraphGetEdges(g, n)
    assert int(out[0]) == 0
    after = {}
    for u, v in zip(out[1], out[2]):
        after.setdefault(int(u), set()).add(int(v))

    def reached(u):
        seen, todo = set(), list(after.get(u, ()))
        while todo:
            v = todo.pop()
            if v not in seen:
                seen.add(v)
                todo.extend(after.get(v, ()))
        return seen

    return sum(len(vs - set().union(*(reached(v) for v in vs))) > 1 for vs in after.values()), nodes


def _state(seed):
    x = delta_inputs(*SHAPE, seed=seed)
    c, d = _cuda(x), _dims(x)
    return x, c, d, _outputs(x), torch.empty_like(c["h0"]), torch.zeros(m3.m3_delta_bwd_workspace_size(d), dtype=torch.uint8,
                                                                        device="cuda")


def _call(s):
    _, c, d, g, dh0, ws = s
    m3.m3_delta_bwd(d, c["q"], c["k"], c["v"], c["g"], c["beta"], c["dy"], g, ws, scale=0.2, init_h=c["h0"], d_init_h=dh0)


def _capture(states):
    for s in states:
        for z in (*s[3].values(), s[4]):
            z.fill_(float("nan"))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        for s in states:
            _call(s)
    forks = _forks(graph)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    for s in states:
        want = _bwd(s[0], 0.2, d_final=False)
        for k, w in want.items():
            assert torch.equal(s[4] if k == "dh0" else s[3][k], w), k
        assert m3.m3_device_status(s[5]) == m3.M3_OK
    return forks


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


def test_a_first_call_that_is_captured():
    """A thread, and a stream, that have never made the call before."""
    def work():
        with torch.cuda.stream(torch.cuda.Stream()):
            forks, nodes = _capture([_state(71)])
        assert forks == 1 and nodes == 5, (forks, nodes)
    _in_a_thread(work)


@pytest.mark.parametrize("calls", [1, 2, 3, 7])
def test_several_calls_in_a_capture(calls):
    """As the layers of a training step: every call has its fork."""
    forks, nodes = _capture([_state(73 + i) for i in range(calls)])
    assert forks == calls and nodes == 5 * calls, (forks, nodes)


def test_captures_after_one_another_and_one_that_was_broken_off():
    s = _state(72)
    for _ in range(2):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            _call(s)
        with pytest.raises(RuntimeError):
            with torch.cuda.graph(torch.cuda.CUDAGraph(), stream=stream):
                _call(s)
                stream.synchronize()                 # not allowed in a capture, which breaks it off
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            _call(s)
        torch.cuda.synchronize()
        assert _capture([s, s])[0] == 2


def test_threads_that_come_and_go():
    s = _state(72)
    want = _bwd(s[0], 0.2, d_final=False)
    for _ in range(30):
        _in_a_thread(lambda: (_call(s), torch.cuda.synchronize()))
    assert all(torch.equal(s[4] if k == "dh0" else s[3][k], w) for k, w in want.items())
