"""What the kernels' sources may not hold."""
import glob
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCES = sorted(f for ext in ("cu", "cuh", "h", "cpp") for d in ("combine_ep_get_dispatch_gb300/csrc", "include", "oracle")
                 for f in glob.glob(os.path.join(ROOT, d, "*." + ext)))


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_no_load_into_several_blocks_shared_memory(path):
    """Rows may lie in any memory that the device can read; a load that is delivered to several blocks at once
    is for this device's own memory alone, and nothing checks that a caller's rows are there."""
    with open(path) as f:
        assert "multi" + "cast" not in f.read().lower()


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_warps_wait_for_lanes_that_are_named(path):
    """The mask of the lanes that happen to run together names nobody that a wait is for."""
    with open(path) as f:
        assert "__activemask" not in f.read()
