"""The committed traffic records were taken on the kernels that are here."""
import hashlib
import json
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
RECORDS = json.load(open(os.path.join(ROOT, "profiles", "traffic.json")))


@pytest.mark.parametrize("kernel", sorted(RECORDS))
def test_records_are_of_the_current_sources(kernel):
    h = hashlib.sha256()
    for name in RECORDS[kernel]["sources"]:
        with open(os.path.join(ROOT, name), "rb") as f:
            h.update(f.read())
    assert h.hexdigest() == RECORDS[kernel]["sha256"]


def test_the_benchmark_reports_them():
    import bench
    assert bench.kernel_traffic("propose_kernel") == RECORDS["propose_kernel"]["bytes_per_launch"]
