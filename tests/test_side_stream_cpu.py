"""The gradient's second streams (csrc/side_stream.h) against a fake CUDA
runtime: one for a caller's stream, none left behind by host threads or by a
creation that failed, none of another context (no GPU; side_stream_fakes.cpp is
compiled with the host compiler)."""
import importlib.util
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_second_streams(tmp_path):
    spec = importlib.util.spec_from_file_location("m3_build", os.path.join(ROOT, "selective_state_space_m3_b200", "build.py"))
    b = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(b)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(b._nvcc())))
    exe = str(tmp_path / "fakes")
    r = subprocess.run([os.environ.get("CXX", "g++"), "-O1", "-std=c++17", "-pthread", "-isystem", os.path.join(cuda, "include"),
                        "-I", b.CSRC, os.path.join(ROOT, "tests", "side_stream_fakes.cpp"), "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr
