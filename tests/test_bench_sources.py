"""The sources by which the bench tells whether a stored counter reading is of today's kernel."""
import re

import bench

CSRC = bench.ROOT / "shape_adaptive_matrix_amd" / "csrc"


def test_a_kernels_sources_hold_the_kernel():
    for kernel, names in bench.SOURCES_OF_KERNEL.items():
        short = kernel.split("::")[-1]
        text = "".join((CSRC / n).read_text() for n in names)
        assert re.search(rf"__global__[^;{{]*\b{short}\(", text), kernel


def test_all_sources_hold_every_kernel():
    text = "".join((CSRC / n).read_text() for n in bench.KERNEL_SOURCES)
    for names in bench.KERNEL_OF.values():
        for kernel in names.split(" / "):
            short = kernel.split("::")[-1]
            assert re.search(rf"__global__[^;{{]*\b{short}\(", text), kernel
