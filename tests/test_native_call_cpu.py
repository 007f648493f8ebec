"""The binding's native argument handling hands everything unusual back to the
Python code (None), which raises the error that names the argument.  Host
tensors only: nothing is launched."""
import pytest
import torch

import selective_state_space_m3_b200 as m3

D = m3.Dims(2, 3, 4, 2, 16, 16, 1, 64, m3.M3_F32)
T = torch.zeros(2, 3, 2, 16)

def test_unusual_arguments_are_handed_back():
    n = m3._native
    for d in (D, None, m3.Dims(1 << 40, 3, 4, 2, 16, 16), m3.Dims("a", 3, 4, 2, 16, 16)):
        for t in (T, None, 5, "x", T.bfloat16()):
            assert n.delta_step(d, t, t, t, t, t, t, t, 1.0, t) is None
            assert n.delta_fwd(d, t, t, t, t, t, 1.0, t, t, t, t, t) is None
            assert n.delta_bwd(d, *[t] * 5, 1.0, *[t] * 11) is None
    for t in (T, None, 5, torch.zeros(()), torch.zeros(3, 0), T.double()):
        assert n.rms_norm_fwd(t, 1e-5, t, t, t, t, t, t, 0) is None
        assert n.rms_norm_bwd(t, t, "eps", t, t, t, t, t) is None

def test_a_wrong_number_of_arguments_is_an_error():
    for f in ("delta_step", "delta_fwd", "delta_bwd", "rms_norm_fwd", "rms_norm_bwd"):
        with pytest.raises(TypeError):
            getattr(m3._native, f)(D, T)
