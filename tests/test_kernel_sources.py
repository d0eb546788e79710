"""Host-side checks of the kernel sources (no GPU needed)."""
from __future__ import annotations

import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "combine_get_dispatch_04_gb300", "csrc")


def code(path):
    text = open(path).read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


def test_no_shuffle_mask_from_the_lanes_that_happen_to_run_together():
    """__activemask() does not say which lanes took a branch, so no mask comes from it."""
    for path in glob.glob(os.path.join(CSRC, "*.cu*")):
        assert "__activemask" not in code(path), path
