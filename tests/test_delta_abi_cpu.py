"""Refusals of the gated delta rule and the norm, before anything is launched
(no GPU): bad sizes, null and misaligned pointers, small workspaces, host
tensors, wrong types and sizes at the binding.  The addresses are never used."""
import ctypes

import pytest
import torch

import selective_state_space_m3_b200 as m3

LIB = m3.raw_lib()
GOOD, BAD = 0x10000, 0x10008


def dims(**kw):
    base = dict(batch=2, seqlen=64, nheads=4, ngroups=2, headdim=16, dstate=16, rank=1, chunk=64, io_dtype=m3.M3_BF16)
    base.update(kw)
    return m3.Dims(**base)


def fwd(d, ptr=GOOD, g=GOOD, lengths=None, init=None, y=GOOD, fin=None, ws=GOOD, size=1 << 40):
    return LIB.m3_delta_fwd(ctypes.byref(d.c()), ptr, ptr, ptr, g, ptr, 1.0, lengths, init, y, fin, ws, size, None)


def step(d, ptr=GOOD, h=GOOD, out=GOOD, y=GOOD):
    return LIB.m3_delta_step(ctypes.byref(d.c()), h, out, ptr, ptr, ptr, None, ptr, 1.0, y, None)


def bwd(d, ptr=GOOD, dy=GOOD, out=GOOD, dg=None, ws=GOOD, size=1 << 50):
    return LIB.m3_delta_bwd(ctypes.byref(d.c()), ptr, ptr, ptr, None, ptr, 1.0, None, None, dy, None, out, out, out, dg,
                            out, None, ws, size, None)


@pytest.mark.parametrize("bad,status", [
    (dict(dstate=15), 1), (dict(nheads=3), 1), (dict(batch=-1), 1), (dict(io_dtype=2), 1), (dict(headdim=0), 1),
    (dict(rank=2), 2), (dict(dstate=258), 2), (dict(batch=1 << 20, nheads=1 << 12), 2),
])
def test_sizes(bad, status):
    n = ctypes.c_size_t(0)
    d = dims(**bad)
    assert fwd(d) == status and step(d) == status and bwd(d) == status
    assert LIB.m3_delta_workspace_size(ctypes.byref(d.c()), ctypes.byref(n)) == status
    assert LIB.m3_delta_bwd_workspace_size(ctypes.byref(d.c()), ctypes.byref(n)) == status


def test_lengths_of_sequences():
    assert fwd(dims(seqlen=-1)) == m3.M3_ERR_INVALID_ARG
    assert step(dims(batch=0, seqlen=-1), ptr=None, h=None, out=None, y=None) == m3.M3_OK     # seqlen is ignored
    assert fwd(dims(batch=1 << 16, seqlen=1 << 16, ngroups=2)) == m3.M3_ERR_UNSUPPORTED


def test_pointers():
    d = dims()
    for p in (None, BAD):
        assert fwd(d, ptr=p) == m3.M3_ERR_INVALID_ARG and fwd(d, y=p) == m3.M3_ERR_INVALID_ARG
        assert step(d, ptr=p) == m3.M3_ERR_INVALID_ARG and step(d, h=p) == m3.M3_ERR_INVALID_ARG
        assert step(d, out=p) == m3.M3_ERR_INVALID_ARG and step(d, y=p) == m3.M3_ERR_INVALID_ARG
        assert bwd(d, ptr=p) == m3.M3_ERR_INVALID_ARG and bwd(d, dy=p) == m3.M3_ERR_INVALID_ARG
        assert bwd(d, out=p) == m3.M3_ERR_INVALID_ARG
    for kw in (dict(g=BAD), dict(lengths=BAD), dict(init=BAD), dict(fin=BAD)):
        assert fwd(d, **kw) == m3.M3_ERR_INVALID_ARG
    assert bwd(d, dg=BAD) == m3.M3_ERR_INVALID_ARG
    assert LIB.m3_delta_workspace_size(ctypes.byref(d.c()), None) == m3.M3_ERR_INVALID_ARG
    assert LIB.m3_delta_workspace_size(None, ctypes.byref(ctypes.c_size_t(0))) == m3.M3_ERR_INVALID_ARG


@pytest.mark.parametrize("over", [dict(), dict(dstate=128, headdim=64), dict(dstate=128, headdim=64, seqlen=1)])
def test_workspaces(over):
    d = dims(**over)
    n, nb = m3.m3_delta_workspace_size(d), m3.m3_delta_bwd_workspace_size(d)
    assert n >= 256 and nb >= 256
    assert fwd(d, size=n - 1) == m3.M3_ERR_WORKSPACE and fwd(d, ws=None) == m3.M3_ERR_WORKSPACE
    assert bwd(d, size=nb - 1) == m3.M3_ERR_WORKSPACE and bwd(d, ws=BAD) == m3.M3_ERR_WORKSPACE


def test_empty_calls():
    e = dims(batch=0)
    assert fwd(e, ptr=None, y=None, g=None) == m3.M3_OK and bwd(e, ptr=None, dy=None, out=None) == m3.M3_OK
    assert step(e, ptr=None, h=None, out=None, y=None) == m3.M3_OK
    assert fwd(dims(batch=0, seqlen=0), ptr=None, y=None, g=None) == m3.M3_OK
    assert norm(rows=0, x=None, y=None, y8=GOOD) == m3.M3_OK


def norm(rows=4, width=64, io=m3.M3_BF16, x=GOOD, r=None, w=None, eps=1e-5, s=None, y=GOOD, y8=None, scale=None, block=0):
    return LIB.m3_rms_norm_fwd(rows, width, io, x, r, w, eps, s, y, y8, scale, block, None)


def test_norm_refusals():
    inv, uns = m3.M3_ERR_INVALID_ARG, m3.M3_ERR_UNSUPPORTED
    assert norm(rows=-1) == inv and norm(width=0) == inv and norm(io=5) == inv and norm(rows=1 << 31) == uns
    assert norm(eps=-1.0) == inv and norm(eps=float("nan")) == inv
    assert norm(y=None) == inv                                # nothing to write
    assert norm(y8=GOOD) == inv and norm(y8=GOOD, scale=GOOD, block=64) == uns
    for kw in (dict(x=None), dict(x=BAD), dict(r=BAD), dict(w=BAD), dict(s=BAD), dict(y=BAD), dict(y8=BAD, scale=GOOD),
               dict(y8=GOOD, scale=BAD)):
        assert norm(**kw) == inv, kw


def test_norm_gradient_refusals():
    n = m3.m3_rms_norm_bwd_workspace_size(100, 64, m3.M3_F32)

    def call(rows=100, width=64, s=GOOD, w=None, eps=1e-5, dy=GOOD, ds=None, dx=GOOD, dw=None, ws=GOOD, size=n):
        return LIB.m3_rms_norm_bwd(rows, width, m3.M3_F32, s, w, eps, dy, ds, dx, dw, ws, size, None)

    for kw in (dict(rows=-1), dict(width=0), dict(s=None), dict(s=BAD), dict(w=BAD), dict(dy=None), dict(dx=BAD),
               dict(ds=BAD), dict(dw=BAD), dict(eps=-1.0)):
        assert call(**kw) == m3.M3_ERR_INVALID_ARG, kw
    assert call(size=n - 1) == m3.M3_ERR_WORKSPACE and call(ws=None) == m3.M3_ERR_WORKSPACE
    with pytest.raises(m3.M3Error):
        m3.m3_rms_norm_bwd_workspace_size(10, 0, m3.M3_F32)


def test_binding_refuses_host_tensors():
    d = dims(io_dtype=m3.M3_F32)
    f = torch.zeros
    q, v, g, h = f(2, 64, 2, 16), f(2, 64, 4, 16), f(2, 64, 4), f(2, 4, 16, 16)
    ws = f(1 << 10, dtype=torch.uint8)
    grads = dict(dq=q, dk=q, dv=v, dg=g, dbeta=g)
    for call in (lambda: m3.m3_delta_fwd(d, q, q, v, g, g, v, ws), lambda: m3.m3_delta_step(d, h, q, q, v, g, g, v),
                 lambda: m3.m3_delta_bwd(d, q, q, v, g, g, v, grads, ws), lambda: m3.m3_rms_norm_fwd(q, 1e-5, y=q),
                 lambda: m3.m3_rms_norm_bwd(q, q, 1e-5, q, ws)):
        with pytest.raises(ValueError, match="device tensors"):
            call()


class _OnDevice:
    """A host tensor that says it is on cuda:0 (nothing is launched)."""

    def __init__(self, t):
        self.t, self.is_cuda, self.dtype, self.device = t, True, t.dtype, torch.device("cuda", 0)

    def get_device(self):
        return 0

    def __getattr__(self, name):
        return getattr(self.t, name)


def test_binding_checks_types_and_sizes():
    t = torch.zeros(3, 4)
    with pytest.raises(TypeError, match="beta is"):
        m3._arg(_OnDevice(t), "beta", torch.bfloat16, 12, 0)
    with pytest.raises(ValueError, match="13 elements"):
        m3._arg(_OnDevice(t), "beta", torch.float32, 13, 0)
    with pytest.raises(ValueError, match="one device"):
        m3._arg(_OnDevice(t), "beta", torch.float32, 12, 1)
    with pytest.raises(ValueError, match="contiguous"):
        m3._arg(_OnDevice(t.T), "beta", torch.float32, 12, 0)
    assert m3._arg(None, "g", torch.float32, 12, 0) is None
