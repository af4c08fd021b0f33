"""The binding of the many-request calls on the CPU: what it checks of its tensors before any launch, and which
marshalling it takes."""
import os
import shutil
import subprocess
import sys

import pytest
import torch

from cross_loop_sparse_b200 import build

F = pytest.importorskip("cross_loop_sparse_b200.flashloop")
PKG = os.path.dirname(os.path.abspath(build.__file__))


def test_tables_and_sums_come_in_rows():
    """Flat, or with rows of the length that the library steps by; another row length would be read and written askew."""
    i32 = torch.int32
    for shape in ((12,), (20,), (3, 4), (5, 4), (1, 3, 4), (3, 2, 2), (3, 4, 1)):
        t = torch.zeros(shape, dtype=i32)
        assert F._vec("f", "block_table", t, 12, i32, -1, 4) == t.data_ptr(), shape
    for shape in ((3, 5), (4, 3), (2, 6), (6, 2), (12, 1), (3, 3, 4, 3)):
        with pytest.raises(F.FlashLoopError) as e:
            F._vec("f", "block_table", torch.zeros(shape, dtype=i32), 12, i32, -1, 4)
        assert e.value.status == -1 and "rows of 4" in str(e.value), shape
    empty = torch.zeros(0, 7, dtype=i32)
    assert F._vec("f", "block_table", empty, 0, i32, -1, 4) == empty.data_ptr()
    for shape in ((2, 9), (18,), (9, 2)):  # plain vectors may have any shape
        assert F._vec("f", "kv_lens", torch.zeros(shape, dtype=i32), 12, i32, -1) is not None


def package(tmp_path, fast):
    """A copy of the package's Python files and library, with _fastcall.so made from what `fast` makes of its bytes (None: without)."""
    pkg = tmp_path / "cross_loop_sparse_b200"
    pkg.mkdir()
    for f in ("__init__.py", "flashloop.py", "build.py"):
        shutil.copy(os.path.join(PKG, f), pkg / f)
    os.symlink(os.path.join(PKG, "libflashloop.so"), pkg / "libflashloop.so")
    if fast is not None:
        with open(os.path.join(PKG, "_fastcall.so"), "rb") as f:
            (pkg / "_fastcall.so").write_bytes(fast(f.read()))


USE = """
import torch
from cross_loop_sparse_b200 import flashloop as F
p = F.PagedParams.make(1, 8, 8, 2, 2, 64)
assert F.flashloop_paged_attn_workspace_bytes(p) > 0 and F._lib.flashloop_status_string(0)
q, i = torch.zeros(8, 2, 64, dtype=torch.bfloat16), torch.zeros(8, dtype=torch.int32)
try:
    F.flashloop_prompt_attn(p, q, q, q, i, q, None, i)
except F.FlashLoopError as e:
    assert e.status == -1
print("fast" if F._fastcall is not F._NoFastcall else "plain")
"""


@pytest.mark.parametrize("case", ["missing", "other", "broken", "this"])
def test_package_imports_without_a_marshalling_for_this_torch(tmp_path, case):
    """The C++ marshalling belongs to one torch and interpreter; without one for these the package's calls go on."""
    target = build.fastcall_target().encode()
    other = target.replace(b"torch 2", b"torch 1")
    assert other != target
    fast = {"missing": None, "other": lambda b: b.replace(target, other), "broken": lambda b: b"not a library " + target + b"\0", "this": lambda b: b}[case]
    package(tmp_path, fast)
    out = subprocess.run([sys.executable, "-c", USE], cwd=tmp_path, capture_output=True, text=True, timeout=300)
    assert out.returncode == 0, out.stderr
    assert out.stdout.split() == ["fast" if case == "this" else "plain"]
    assert ("_fastcall.so" in out.stderr) == (case != "this")


def test_marshalling_is_built_again_for_another_torch(tmp_path, monkeypatch):
    """A newer file than the sources that was built for something else does not stand."""
    ran = []

    class Done:
        returncode = 0

    def run(cmd, **kw):
        ran.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "wb") as f:
            f.write(b"new " + build.fastcall_target().encode() + b"\0")
        return Done()

    fast = tmp_path / "_fastcall.so"
    fast.write_bytes(b"old torch 1.0\0")
    monkeypatch.setattr(build, "FAST", str(fast))
    monkeypatch.setattr(build.subprocess, "run", run)
    assert not build.fastcall_fits()
    build._build_fastcall(False)
    assert len(ran) == 1 and build.fastcall_fits() and any(build.fastcall_target() in a for a in ran[0])
    build._build_fastcall(False)
    assert len(ran) == 1


class Fake:
    """What the Python marshalling asks of a tensor, for sizes that need no memory."""
    dtype, device = torch.int32, "cuda:0"

    def __init__(self, *shape):
        self.shape = shape

    def get_device(self):
        return 0

    def numel(self):
        n = 1
        for d in self.shape:
            n *= d
        return n

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 4096


@pytest.mark.parametrize("entries,want", [(7, 7), (2 ** 31 - 1, 2 ** 31 - 1), (2 ** 31, 2 ** 31 - 1), (2 ** 32 + 1, 2 ** 31 - 1)])
def test_a_stack_of_any_size_keeps_its_capacity(monkeypatch, entries, want):
    """The library takes the capacity in 32 bits: a longer buffer must not wrap to a short or negative one."""
    seen = []
    monkeypatch.setattr(F, "_launch", lambda fn, dev, stream, *args: seen.append(args) or 0)
    p = F.PagedParams.make(2, 4, 2, 1, 1, 64, 16, 10, 3)
    F.flashloop_paged_plan(p, Fake(2), Fake(2), Fake(entries), Fake(1), Fake(2, 3), Fake(3), Fake(2), Fake(4), Fake(4), Fake(1), Fake(1))
    types = F._lib.flashloop_paged_plan.argtypes
    assert len(seen[0]) == len(types) - 1 and types[4](seen[0][4]).value == want
