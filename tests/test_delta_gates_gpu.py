"""The gradient of the gates where they decay strongly: it has the factor e^g
and may be a millionth of its neighbours', yet keeps its relative accuracy, and
is zero where a gate resets the state.  Against 64 bits, every (batch, head) by
itself; tolerance of bfloat16 gradients as in test_delta_gpu.py (their own
rounding and at most six of operands; the terms of one gate's gradient all have
its factor, so that none of the errors is of another gate's size)."""
import pytest
import torch

from tests._delta_ref import delta_grads, delta_inputs, rel
from tests.test_delta_gpu import D16, _bwd, _check_bwd

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
PATHS = ["", "token"]
SHAPES = [(2, 200, 2, 1, 64), (1, 130, 2, 2, 128), (3, 65, 2, 1, 64)]
IDS = ["b%d_t%d_h%d_g%d_p%d" % s for s in SHAPES]


def _gates(x, lengths=None, init=True):
    got = _bwd(x, 0.1, lengths, init=init, d_final=init)["dg"].cpu()
    z = x if init else {**x, "h0": torch.zeros_like(x["h0"])}
    return got, delta_grads(z, 0.1, lengths, init=True, d_final=init)["g"]


def _each(got, want, where):
    for b in range(want.shape[0]):
        for h in range(want.shape[2]):
            w = where[b, :, h]
            r = rel(got[b, w, h], want[b, w, h])
            assert r <= D16, (b, h, r)


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
@pytest.mark.parametrize("mean", [-2.0, -8.0, -12.0, -16.0, -20.0, -30.0])
def test_strong_decay(mean, shape, path, monkeypatch):
    monkeypatch.setenv("M3_DELTA_PATH", path)
    x = delta_inputs(*shape, 128, BF, seed=61)
    x["g"] = x["g"] + mean
    got, want = _gates(x)
    _each(got, want, torch.ones_like(want, dtype=torch.bool))


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
@pytest.mark.parametrize("init", [False, True])
def test_strong_decay_among_weak(init, shape, path, monkeypatch):
    """Every fifth gate is -16, one -40: their gradients by themselves, the others by themselves."""
    monkeypatch.setenv("M3_DELTA_PATH", path)
    x = delta_inputs(*shape, 128, BF, seed=62)
    strong = torch.zeros_like(x["g"], dtype=torch.bool)
    strong[:, 3::5] = True
    x["g"][strong] = -16.0
    x["g"][:, 31] = -40.0
    got, want = _gates(x, init=init)
    last = torch.zeros_like(strong)
    last[:, 31] = True
    for where in (strong & ~last, last, ~strong & ~last):
        _each(got, want, where)
    if not init:
        assert float(got[:, 0].float().abs().sum()) == 0.0       # before the first token there is nothing to decay


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
@pytest.mark.parametrize("low", [float("-inf"), -2.0e4])
def test_resets_have_no_gradient(low, shape, path, monkeypatch):
    monkeypatch.setenv("M3_DELTA_PATH", path)
    x = delta_inputs(*shape, 128, BF, seed=63)
    reset = torch.zeros_like(x["g"], dtype=torch.bool)
    for t in (0, 1, 15, 16, 17, 32, 47, 48, 49, 63, 64):
        reset[:, t, t % 2] = True
    x["g"][reset] = low
    got, want = _gates(x)
    assert float(got[reset].float().abs().sum()) == 0.0 and float(want[reset].abs().sum()) == 0.0
    _each(got, want, ~reset)


def test_long_sequence_of_strong_decay():
    x = delta_inputs(1, 2500, 2, 1, 64, 128, BF, seed=64)
    x["g"] = 40.0 * x["g"]                                       # 0 to -20
    lengths = torch.tensor([2450])
    got, want = _gates(x, lengths)
    _each(got, want, torch.ones_like(want, dtype=torch.bool))
    for lo, hi in ((-20, -15), (-15, -10), (-10, -5), (-5, 0)):
        _each(got, want, (x["g"] > lo) & (x["g"] <= hi))
    assert float(got[:, 2450:].float().abs().sum()) == 0.0
    _check_bwd(x, _bwd(x, 0.1, lengths), 0.1, lengths)
