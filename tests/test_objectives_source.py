"""What the objectives' kernels may not say (no GPU: read from their source)."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "convex_hull_pava_gb300", "csrc")


def kernels():
    """(name, parameters, body) of each kernel of the objectives."""
    for path in sorted(glob.glob(os.path.join(CSRC, "obj_*.cu"))):
        with open(path) as f:
            text = f.read()
        for m in re.finditer(r"__global__.*?\n(\w+)\(([^{;]*)\) \{\n(.*?)\n\}\n", text, re.S):
            yield m.group(1), m.group(2), m.group(3)


def test_no_read_only_loads_of_what_a_running_kernel_writes():
    """A kernel that waits for the one in front of it runs while that one writes.  const
    __restrict__ promises that nobody writes while the kernel runs: only a caller's own input that
    was there before both may be taken so (the labels)."""
    seen = [name for name, _, body in kernels() if "wait_for_previous()" in body]
    assert {"policy_rows_kernel", "score_backward_kernel", "balance_backward_kernel", "balance_finish_kernel",
            "preference_pairs_kernel"} <= set(seen)
    for name, parameters, body in kernels():
        if "wait_for_previous()" not in body:
            continue
        for p in parameters.split(","):
            if "__restrict__" in p:
                assert p.split()[-1] == "labels", (name, p.strip())
