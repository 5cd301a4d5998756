"""What the CUDA sources of the paged-cache operators have to keep and no test
that runs them can show.  No GPU."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "sparse_moe_bit_gb300", "csrc")


def _code(name):
    src = open(os.path.join(CSRC, name)).read()
    return re.sub(r"/\*.*?\*/|//[^\n]*", "", src, flags=re.S)


def _body(src, head):
    """The braces' content of the first definition after `head`."""
    at = src.index("{", src.index(")", src.index(head)))
    depth = 0
    for i in range(at, len(src)):
        depth += {"{": 1, "}": -1}.get(src[i], 0)
        if depth == 0:
            return src[at:i]
    raise AssertionError("unbalanced braces")


def test_no_cta_of_a_dependent_grid_leaves_before_its_wait():
    """The join is set up while the grid before it runs.  If all of its CTAs left
    before the wait, what follows in the stream could start while that grid still
    writes to the workspace."""
    body = _body(_code("paged_rows.cu"), "paged_join_kernel(const AttnParams")
    wait = body.index("griddepcontrol.wait")
    assert not re.search(r"\breturn\b", body[:wait])
    # nothing of the grid before is read ahead of it either
    assert not re.search(r"part_o|part_ml|p\.before", body[:wait])
