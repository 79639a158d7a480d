"""Kernels that are scheduled while the kernel before them finishes (programmatic
dependent launch) read what that kernel wrote by ordinary loads only: the wait
makes it visible to those, and the non-coherent path is for data that nothing
writes during a kernel's life.  Held for all device code, since helpers are
shared between the kernels."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "io_aware_attention_flash_gb300", "csrc")


def test_no_non_coherent_loads():
    files = sorted(glob.glob(os.path.join(CSRC, "*.cu*")))
    assert files
    for f in files:
        code = re.sub(r"//[^\n]*", "", open(f).read())
        # (const __restrict__ pointers let the compiler choose such loads)
        assert not re.search(r"__ldg\s*\(|\.nc\b|__restrict__", code), os.path.basename(f)
