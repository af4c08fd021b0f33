"""Calls of the many-request operators that the documentation allows or refuses: shapes, streams, captures,
requests beside refused ones."""
import pytest
import torch

from test_gpu_paged import BF, F, gen, ints, paged_inputs, randn, workspace

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("way", ["fast", "plain"])
def test_wider_tables_and_turned_sums_are_refused(way, monkeypatch):
    """A table with more columns than max_blocks and sums laid out [tokens, heads] have enough elements, in the wrong rows."""
    if way == "plain":
        monkeypatch.setattr(F, "_fastcall", type("Without", (), {n: staticmethod(lambda *a: None) for n in ("plan", "write", "attn", "prompt")}))
    total, new = [100, 40, 65], [2, 3, 1]
    p, q, kc, vc, table, cu = paged_inputs(total, new, 4, 2, 64, 16, BF, "thd", 0)
    o, err, ws, T, H = torch.full_like(q, 7.0), ints([0]), workspace(p), q.shape[0], 4
    kv, cus = ints(total), ints(cu)
    k = randn(gen(1), T, 2, 64, dtype=BF)
    wide = torch.cat([table, table[:, :1]], 1).contiguous()

    def paged(**a):
        F.flashloop_paged_attn(**{**dict(params=p, q=q, k_cache=kc, v_cache=vc, block_table=table, kv_lens=kv, cu=cus, o=o, lse=None, workspace=ws, err_word=err), **a})

    def prompt(lse):
        F.flashloop_prompt_attn(p, q, k, k, cus, o, lse, err)

    def plan(tab):
        F.flashloop_paged_plan(p, kv, ints([0, 0, 0]), ints([0]), ints([0]), tab, ints([0] * 4), ints([0] * 3), ints([0] * T), ints([0] * T), ints([0]), err)

    for call in (lambda: paged(block_table=wide), lambda: paged(lse=torch.zeros(T, H, device="cuda")), lambda: prompt(torch.zeros(T, H, device="cuda")), lambda: plan(wide)):
        with pytest.raises(F.FlashLoopError) as e:
            call()
        assert e.value.status == -1
    torch.cuda.synchronize()
    assert (o == 7).all() and err.item() == 0
    want = torch.full((H, T), 7.0, device="cuda")
    paged(lse=want)
    more = torch.cat([table, table[:2]]).contiguous()  # a table with rows for more requests
    for tab, lse in ((table.flatten(), torch.full((H * T,), 7.0, device="cuda")), (table[None], torch.full((H, T, 1), 7.0, device="cuda")), (more, torch.full((H + 1, T), 7.0, device="cuda"))):
        got = torch.full_like(o, 7.0)
        paged(block_table=tab, lse=lse, o=got)
        assert torch.equal(got, o) and torch.equal(lse.flatten()[:H * T], want.flatten())
    plan(table)
    prompt(want)
    assert err.item() == 0
