"""The binding of the many-request calls on the CPU: what it checks of its tensors before any launch."""
import pytest
import torch

F = pytest.importorskip("cross_loop_sparse_b200.flashloop")


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
