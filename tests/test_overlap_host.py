"""What kernels that overlap their predecessors may not do (source check, no GPU needed)."""

import glob
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_no_read_only_loads():
    """Kernels start while the one before them still writes, also what they read once they have waited for its end.

    The read-only path (__ldg, ld.global.nc, and const __restrict__ pointers,
    which the compiler may read by it) is only defined for memory that nothing
    writes during the whole kernel.
    """
    found = []
    for path in sorted(glob.glob(os.path.join(ROOT, "trainable_block_sparse_infllm_gb300", "csrc", "*.cu*"))):
        with open(path) as f:
            for number, line in enumerate(f, 1):
                code = line.split("//")[0]
                if re.search(r"__ldg\b|ld\.global\.(\w+\.)*nc|const\b[^,;()]*__restrict__", code):
                    found.append(f"{os.path.basename(path)}:{number}: {line.strip()}")
    assert not found, "\n".join(found)
