"""Kernels that start while the kernel before them still runs, by their sources."""

import glob
import os
import re

from strided_gemm_gb300 import build as sgbuild


def with_headers(name, seen):
    """The text of a source file and of the headers beside it that it includes."""
    if name in seen or not os.path.exists(os.path.join(sgbuild.CSRC, name)):
        return ""
    seen.add(name)
    with open(os.path.join(sgbuild.CSRC, name)) as f:
        text = f.read()
    return text + "".join(with_headers(h, seen) for h in re.findall(r'#include "([^"]+)"', text))


def test_no_read_only_load_in_a_kernel_that_starts_early():
    """What the kernel before writes may be read after the wait for it, by ordinary
    loads: the read-only path (__ldg, ld.global.nc, restricted pointers) is for data
    that stay as they are for the whole of a kernel, and is not ordered by the wait."""
    early = []
    for path in sorted(glob.glob(os.path.join(sgbuild.CSRC, "*.cu"))):
        text = with_headers(os.path.basename(path), set())
        if "griddepcontrol.wait" not in text:
            continue
        early.append(os.path.basename(path))
        code = re.sub(r"//[^\n]*", "", text)
        for word in ("__ldg", ".nc", "__restrict__"):
            assert word not in code, (early[-1], word)
    assert len(early) >= 6, early
