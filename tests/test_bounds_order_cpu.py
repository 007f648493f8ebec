"""m3_debug_bounds_report gives the first failure of the lowest-numbered source
file that has one: the readers of the files' records are asked in the order of
the files' numbers, each file's once (no GPU: read from the sources)."""
import glob
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "selective_state_space_m3_b200", "csrc")


def test_records_are_read_in_the_order_of_the_file_numbers():
    number = {}
    for path in glob.glob(os.path.join(CSRC, "*.cu")):
        text = open(path).read()
        n, tag = re.search(r"#define M3_BOUNDS_FILE (\d+)", text), re.search(r"^M3_BOUNDS_EXPORT\((\w+)\)", text, re.M)
        if n and tag:
            number[tag.group(1)] = int(n.group(1))
    assert sorted(number.values()) == list(range(1, len(number) + 1))
    api = open(os.path.join(CSRC, "m3_api.cu")).read()
    listed = re.findall(r"bounds_take_(\w+)", re.search(r"Take takes\[\] = \{(.*?)\};", api, re.S).group(1))
    assert [number[t] for t in listed] == sorted(number.values())
