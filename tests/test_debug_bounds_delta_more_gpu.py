"""Further tests of the gated delta rule and the norm under the index-checked
library, as in test_delta_debug_bounds_gpu.py."""
import pytest

from tests import test_delta_debug_bounds_gpu as base

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("path", ["tests/test_delta_gates_gpu.py", "tests/test_delta_graph_gpu.py",
                                  "tests/test_fresh_thread_gpu.py", "tests/test_norm_wide_row_gpu.py"])
def test_under_the_checked_library(path):
    base.test_parity_under_the_checked_library(path)
