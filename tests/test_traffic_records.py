"""The stored DRAM traffic records are of the kernels' present sources: bench.py leaves the
traffic out of its lines where they are not."""
import glob
import json
import os

import pytest

import bench
from conftest import ROOT

RECORDS = sorted(glob.glob(os.path.join(ROOT, "profiles", "*_traffic.json")))


@pytest.mark.parametrize("path", RECORDS, ids=os.path.basename)
def test_the_record_is_of_the_present_sources(path):
    kernel = next(k for k in bench.KERNEL_SOURCES if os.path.basename(path).startswith(k))
    record = json.load(open(path))
    assert record["kernel_source_sha"] == bench.kernel_source_sha(kernel)


def test_there_are_records():
    assert len(RECORDS) >= 4
