"""Rules of the kernel sources that a run cannot show reliably (no GPU needed)."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "combine_moe_topk_gb300", "csrc")


def code_of(path):
    text = re.sub(r"/\*.*?\*/", "", open(path).read(), flags=re.S)
    return re.sub(r"//[^\n]*", "", text)


def test_no_constant_loads_where_a_launch_may_overlap_its_forerunner():
    """A kernel that waits at grid_dependency_wait() may have been started while the kernel before it still writes:
    a load declared constant for the kernel's whole life may be moved above that wait.  The headers' helpers are
    used by such kernels too."""
    looked = 0
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        code = code_of(path)
        if path.endswith(".cuh") or "grid_dependency_wait(" in code:
            looked += 1
            assert "__ldg(" not in code and "ld.global.nc" not in code, os.path.basename(path)
    assert looked >= 10


def test_every_overlapping_launch_waits():
    """launch_pdl and launch_chained are for kernels that call grid_dependency_wait()."""
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        code = code_of(path)
        if re.search(r"\blaunch_(pdl|chained)\(|ProgrammaticStreamSerialization;", code):
            kernels = re.findall(r"__global__[^;{]*?\b(\w+_kernel)\s*\(", code)
            bodies = re.split(r"__global__", code)[1:]
            for name, body in zip(kernels, bodies):
                chained = re.search(r"launch_(?:pdl|chained)\([^;]*\b%s\b" % name, code)
                assert not chained or "grid_dependency_wait(" in body, (os.path.basename(path), name)
