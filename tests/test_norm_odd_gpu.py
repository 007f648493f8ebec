"""The norm and its gradient on rows whose width is no multiple of 8, from one
column to more than registers hold, few rows and many; tolerances as in
test_norm_gpu.py, whose tests run on these sizes."""
import pytest
import torch

from tests import test_norm_gpu as base

pytestmark = pytest.mark.gpu

SIZES = [(300, 1), (1000, 31), (3000, 70), (7, 129), (257, 1025), (300, 2049), (255, 4097), (300, 4095), (9, 8191), (280, 8191),
         (6, 8193)]
IDS = ["%dx%d" % s for s in SIZES]


@pytest.mark.parametrize("dtype", [base.BF, base.FL])
@pytest.mark.parametrize("rows,width", SIZES, ids=IDS)
def test_forward_and_gradient(rows, width, dtype):
    base.test_forward(rows, width, dtype)
    base.test_gradient(rows, width, dtype)


@pytest.mark.parametrize("block", [0, 128])
@pytest.mark.parametrize("dtype", [base.BF, base.FL])
@pytest.mark.parametrize("rows,width", SIZES, ids=IDS)
def test_eight_bits(rows, width, dtype, block):
    base.test_eight_bits(rows, width, dtype, block)
