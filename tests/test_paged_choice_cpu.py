"""The tests' own writing of the kernel choice agrees with the library's."""
import random

import pytest

from paged_choice import scratch, tiles

F = pytest.importorskip("cross_loop_sparse_b200.flashloop")


def test_choice_of_the_kernel_follows_the_bounds():
    rng = random.Random(3)
    taken = set()
    for _ in range(4000):
        Hk = rng.choice((1, 2, 3, 8, 16))
        most = int(2 ** rng.uniform(0, 13))
        p = F.PagedParams.make(batch=int(2 ** rng.uniform(0, 15.9)), max_tokens=most + int(2 ** rng.uniform(0, 16)), max_new=most, n_heads=Hk * rng.choice((1, 2, 4, 7, 16, 40)), n_kv_heads=Hk,
                               head_dim=rng.choice((64, 128)), page_size=rng.choice((16, 32, 64, 128, 256)), n_pages=100, max_blocks=int(2 ** rng.uniform(0, 11)))
        assert F.flashloop_paged_attn_workspace_bytes(p) == scratch(p), [getattr(p, n) for n, _ in p._fields_]
        taken.add((tiles(p, True), p.max_blocks * p.page_size > 512))
    assert len(taken) == 4
