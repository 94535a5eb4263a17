"""No kernel of the built library has memory of its own beside registers and LDS: the
runtime would allocate it at a launch, and no call allocates."""
import os
import re
import subprocess

import pytest

from test_product_waits import OBJDUMP, code_objects

READELF = os.path.join(os.path.dirname(OBJDUMP), "llvm-readelf")


def test_private_segments(tmp_path):
    from combine_moe_layout_03_amd import build

    if not os.path.exists(build.LIB) or not os.path.exists(READELF):
        pytest.skip("no built library, or no reader for it")
    sizes = {}
    for i, obj in enumerate(code_objects(build.LIB)):
        path = tmp_path / f"{i}.o"
        path.write_bytes(obj)
        notes = subprocess.run([READELF, "--notes", str(path)], check=True, capture_output=True,
                               text=True).stdout
        for block in notes.split("\n  - ."):
            name = re.search(r"\.symbol:\s+(\S+)", block)
            size = re.search(r"\.private_segment_fixed_size:\s+(\d+)", block)
            if name and size:
                dynamic = re.search(r"\.uses_dynamic_stack:\s+true", block) is not None
                sizes[name.group(1)] = -1 if dynamic else int(size.group(1))
    assert len(sizes) > 100
    assert not {k: v for k, v in sizes.items() if v}
