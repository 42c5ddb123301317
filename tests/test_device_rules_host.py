"""Launch rules take the number of SMs from the device, not from the part they were measured on."""
import os
import re

from nvfp4_block_scaled_arc_b200 import _build


def test_no_sm_count_is_written_into_the_code():
    for path in _build.sources():
        with open(path) as f:
            code = re.sub(r"/\*.*?\*/|//[^\n]*", "", f.read(), flags=re.S)
        assert not re.search(r"\b148\b", code), os.path.basename(path)
