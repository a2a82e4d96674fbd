"""Edges of the output end of a model, host side."""
import glob
import os
import re

import sinkhorn_point_cloud_amd as sk

CSRC = os.path.join(os.path.dirname(os.path.abspath(sk.__file__)), "csrc")


def test_assembly_that_writes_m0_says_so():
    """The compiler may keep a value of its own there across a statement that does not name it."""
    seen = 0
    for path in glob.glob(os.path.join(CSRC, "*")):
        for text in re.findall(r"\basm\s+volatile\s*\((.*?)\);", open(path).read(), flags=re.S):
            if re.search(r"s_\w+ m0\b", text):
                seen += 1
                assert '"m0"' in text.rsplit(":", 1)[1], path
    assert seen
