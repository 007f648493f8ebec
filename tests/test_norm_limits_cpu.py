"""The largest rows that the root-mean-square norm takes (no GPU): the kernels
walk a row's columns with 32-bit counters in steps of 256, so that widths above
2^31 - 256 are refused before anything is launched; the binding refuses widths
that no C int holds instead of cutting them off."""
import ctypes

import pytest
import torch

import selective_state_space_m3_b200 as m3

LIB = m3.raw_lib()
GOOD = 0x10000


@pytest.mark.parametrize("width", [0x7fffff01, 0x7fffff80, 0x7fffffff])
def test_widths_near_the_end_of_32_bits(width):
    n = ctypes.c_size_t(0)
    assert LIB.m3_rms_norm_bwd_workspace_size(1, width, m3.M3_F32, ctypes.byref(n)) == m3.M3_ERR_UNSUPPORTED
    assert LIB.m3_rms_norm_fwd(1, width, m3.M3_F32, GOOD, None, None, 1e-5, None, GOOD, None, None, 0, None) == m3.M3_ERR_UNSUPPORTED
    assert LIB.m3_rms_norm_bwd(1, width, m3.M3_F32, GOOD, None, 1e-5, GOOD, None, GOOD, None, GOOD, 1 << 50,
                               None) == m3.M3_ERR_UNSUPPORTED


def test_the_widest_row_has_a_workspace():
    assert m3.m3_rms_norm_bwd_workspace_size(1, 0x7fffff00, m3.M3_F32) >= 4 * 0x7fffff00


class _Wide:
    """A tensor without memory that says it is on cuda:0 (nothing is launched)."""

    def __init__(self, width, dtype=torch.float32):
        self.t, self.is_cuda, self.dtype = torch.empty(1, width, dtype=dtype, device="meta"), True, dtype

    def get_device(self):
        return 0

    def data_ptr(self):
        return GOOD

    def __getattr__(self, name):
        return getattr(self.t, name)


def test_the_binding_does_not_cut_a_width_off():
    x, ws = _Wide((1 << 32) + 64), _Wide(1 << 20, torch.uint8)
    for call in (lambda: m3.m3_rms_norm_bwd_workspace_size(1, (1 << 32) + 64, m3.M3_F32),
                 lambda: m3.m3_rms_norm_fwd(x, 1e-5, y=x), lambda: m3.m3_rms_norm_bwd(x, x, 1e-5, x, ws),
                 lambda: m3.m3_rms_norm_fwd(_Wide(64), 1e-5, y=_Wide(64), scale_block=(1 << 32) + 128)):
        with pytest.raises(m3.M3Error) as e:
            call()
        assert e.value.status == m3.M3_ERR_UNSUPPORTED
