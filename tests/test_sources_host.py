"""What the CUDA sources must not contain, checked without a GPU."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..",
                    "gradient_reduce_optimizer_gb300", "csrc")


def code(path):
    """The source without its comments."""
    with open(path) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    return re.sub(r"//[^\n]*", "", text)


def test_kernels_that_start_early_read_nothing_through_the_read_only_path():
    """The read-only path wants memory that nobody writes for as long as the
    kernel runs.  A kernel that starts before the one ahead of it has ended
    (griddepcontrol.wait) cannot promise that of anything it reads."""
    early = [p for p in glob.glob(os.path.join(CSRC, "*.cu")) if "griddepcontrol.wait" in code(p)]
    assert len(early) >= 3
    for path in early:
        found = re.findall(r"__ldg\w*|ld\.global\.nc|__restrict__", code(path))
        assert not found, f"{os.path.basename(path)}: {found}"
