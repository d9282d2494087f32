"""Host check (no GPU): kernels that start before the preceding grid of their
stream ends read nothing through the read-only path, which is for data that no one
writes while the kernel runs."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "boolean_weight_matmul_b200", "csrc")


def _code(path):
    with open(path) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_no_read_only_loads_behind_an_early_launch():
    sources = {p: _code(p) for ext in ("*.cu", "*.cuh") for p in glob.glob(os.path.join(CSRC, ext))}
    early = {p: c for p, c in sources.items()
             if re.search(r"pdl_wait|grid_dependency_wait|griddepcontrol\.wait|scale_rows\.h", c)}
    assert len(early) >= 8
    for path, code in early.items():
        assert not re.search(r"__ldg\s*\(|ld\.global\.nc", code), os.path.basename(path)
