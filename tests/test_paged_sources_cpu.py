"""What the sources of the many-request kernels have to keep to."""
import glob
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "cross_loop_sparse_b200", "csrc")


def code(path):
    """A source without its comments."""
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", open(path).read(), flags=re.S)


def test_kernels_that_start_early_read_through_coherent_loads():
    """A kernel that is launched before the one in front has ended may not take the read-only path: that asks for
    data that nothing writes while the kernel lives, and its loads are not ordered behind the wait."""
    early = [f for f in glob.glob(os.path.join(CSRC, "*.cu")) if "pg_launch_early(" in code(f)]
    assert len(early) == 4
    for f in early:
        for word in ("__ldg", "ld.global.nc", "__restrict__", "ldu"):
            assert word not in code(f), (os.path.basename(f), word)


def test_kernels_that_start_early_wait_before_global_memory():
    """Each of them waits for the end of the kernel in front, by all of its threads, outside of any branch."""
    for f in glob.glob(os.path.join(CSRC, "*.cu")):
        src = code(f)
        if "pg_launch_early(" not in src:
            continue
        kernels = re.split(r"__global__", src)[1:]
        for k in kernels:
            body = k[k.index("{"):]
            at = body.index("pg_wait_for_launch_before();")
            assert body[:at].count("{") - body[:at].count("}") == 1, f
            assert not re.search(r"\bg\.(kv|add|slot|table|cu|q|k|v|n_free)\b\s*[\[(]|\breturn\b", body[:at]), f
