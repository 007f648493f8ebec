"""The longest sequences that the gated delta rule takes (no GPU).  Its kernels
walk the tokens in blocks of 16 or 64 with 32-bit counters: behind the last
block of a sequence of more than 2^31 - 17 tokens the counter would be negative,
and the loop would go on in front of the buffers.  Such calls are refused before
anything is launched; only host-side queries and refusals are made here."""
import ctypes

import pytest

import selective_state_space_m3_b200 as m3

LIB = m3.raw_lib()


def _dims(seqlen):
    return m3.Dims(1, seqlen, 1, 1, 1, 2, 1, 64, m3.M3_F32)


@pytest.mark.parametrize("seqlen", [0x7fffff01, 0x7ffffff0, 0x7fffffff])
def test_sequences_near_the_end_of_32_bits(seqlen):
    d, n = _dims(seqlen).c(), ctypes.c_size_t(0)
    sizes = (LIB.m3_delta_workspace_size(ctypes.byref(d), ctypes.byref(n)),
             LIB.m3_delta_bwd_workspace_size(ctypes.byref(d), ctypes.byref(n)))
    assert sizes == (m3.M3_ERR_UNSUPPORTED, m3.M3_ERR_UNSUPPORTED)
    # the calls make the same check first (a workspace of no bytes is refused after it)
    assert LIB.m3_delta_fwd(ctypes.byref(d), *[0x10000] * 5, 1.0, None, None, 0x10000, None, None, 0,
                            None) == m3.M3_ERR_UNSUPPORTED
    assert LIB.m3_delta_bwd(ctypes.byref(d), *[0x10000] * 5, 1.0, None, None, 0x10000, None, *[0x10000] * 5, None, None, 0,
                            None) == m3.M3_ERR_UNSUPPORTED


def test_the_longest_sequence_has_a_workspace():
    d = _dims(0x7fffff00)
    assert m3.m3_delta_workspace_size(d) == 256
    assert m3.m3_delta_bwd_workspace_size(d) > 0x7fffff00
    # the last block's end, in each of the kernels' steps, is an int
    assert all(-(-d.seqlen // step) * step + step <= 0x7fffffff for step in (8, 16, 64))
