"""The native argument handling is an extension for one PyTorch and one Python;
the package imports and makes every call without it (no GPU: refusals)."""
import glob
import importlib.util
import os
import shutil
import subprocess
import sys

import pytest

import selective_state_space_m3_b200 as m3

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "selective_state_space_m3_b200")

CODE = """
import torch
import selective_state_space_m3_b200 as m3
assert m3.__file__.startswith({where!r}), m3.__file__
assert m3._native.delta_step(1, 2, 3) is None
d = m3.Dims(2, 64, 4, 2, 16, 16, 1, 64, m3.M3_F32)
assert m3.m3_delta_workspace_size(d) == 256 and m3.m3_scan_workspace_size(d) >= 256
q, v, g = torch.zeros(2, 64, 2, 16), torch.zeros(2, 64, 4, 16), torch.zeros(2, 64, 4)
for call in (lambda: m3.m3_delta_fwd(d, q, q, v, g, g, v, q), lambda: m3.m3_rms_norm_fwd(q, 1e-5, y=q),
             lambda: m3.m3_rms_norm_bwd(q, q, 1e-5, q, q), lambda: m3.m3_delta_step(d, v, q, q, v, g, g, v),
             lambda: m3.m3_delta_bwd(d, q, q, v, g, g, v, dict(dq=q, dk=q, dv=v, dg=g, dbeta=g), q)):
    try:
        call()
    except ValueError as e:
        assert "device tensors" in str(e)
    else:
        raise AssertionError("a host tensor was taken")
print("fine")
"""


@pytest.mark.parametrize("what", ["missing", "for another Python", "for another PyTorch", "broken"])
def test_import_without_the_extension(what, tmp_path):
    dst = tmp_path / "selective_state_space_m3_b200"
    dst.mkdir()
    for f in glob.glob(os.path.join(PKG, "*.py")) + [os.path.join(PKG, "libm3.so")]:
        shutil.copy(f, dst)
    name = m3.native_call_name()
    if what == "for another Python":
        (dst / name.replace("cpython-3", "cpython-9")).write_bytes(b"another Python's")
    elif what == "for another PyTorch":
        (dst / name.replace("torch-", "torch-0.")).write_bytes(b"another PyTorch's")
    elif what == "broken":
        (dst / name).write_bytes(b"no shared object")
    env = {k: v for k, v in os.environ.items() if k != "M3_DEBUG_BOUNDS"}
    r = subprocess.run([sys.executable, "-c", CODE.format(where=str(tmp_path))], cwd=tmp_path,
                       env={**env, "PYTHONPATH": str(tmp_path)}, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "fine", r.stderr[-2000:]


def test_the_built_extension_is_the_one_that_is_loaded():
    import torch
    spec = importlib.util.spec_from_file_location("m3_build", os.path.join(PKG, "build.py"))
    b = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(b)
    path = b.call_path(os.path.dirname(torch.__file__))
    assert os.path.basename(path) == m3.native_call_name() and os.path.exists(path)
    assert m3._native.__file__ == path
