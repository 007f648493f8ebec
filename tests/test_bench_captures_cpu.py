"""bench.py reports a kernel's DRAM bytes while the sources that the capture was
taken of are the present ones (no GPU).  A capture of other sources is taken
again or taken out; sources that a kernel does not use stay out of its digest."""
import pytest

import bench


@pytest.mark.parametrize("kernel", sorted(bench.CAPTURES))
def test_captures_are_of_the_present_sources(kernel):
    work, segments, nbytes, digest = bench.CAPTURES[kernel]
    assert bench.source_digest(kernel) == digest
    assert bench.captured_traffic(kernel, work, segments)[0] == nbytes
