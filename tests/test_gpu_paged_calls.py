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


@pytest.mark.parametrize("n", [2, 300])  # few-row kernel, tile kernel
def test_capture_over_two_streams(n):
    """Early launches where a kernel follows one of its own stream and one of another: writes and attention of two
    pools side by side, each step on the other stream than the last, joined and forked in one graph."""
    B, H, Hk, dh, page, steps = 3, 8, 2, 64, 16, 6
    width = steps * n // page + 2

    def inputs(seed):
        p = F.PagedParams.make(batch=B, max_tokens=B * n, max_new=n, n_heads=H, n_kv_heads=Hk, head_dim=dh, page_size=page, n_pages=B * width, max_blocks=width)
        return dict(p=p, q0=randn(gen(seed), B * n, H, dh, dtype=BF), q=torch.empty(B * n, H, dh, dtype=BF, device="cuda"), o=torch.empty(B * n, H, dh, dtype=BF, device="cuda"),
                    kv=[ints([0] * B) for _ in range(2)], new=ints([n] * B), free=ints(list(range(B * width))), left=[ints([B * width]), ints([0])], start=ints([B * width]), none=ints([0] * B),
                    table=ints([[-1] * width] * B), cu=ints([0] * (B + 1)), slots=ints([0] * B * n), pos=ints([0] * B * n), err=ints([0]), ws=workspace(p),
                    kc=torch.zeros(B * width, page, Hk, dh, dtype=BF, device="cuda"), vc=torch.zeros(B * width, page, Hk, dh, dtype=BF, device="cuda"))

    def reset(c):
        c["q"].copy_(c["q0"])
        c["kv"][0].copy_(c["none"])
        c["left"][0].copy_(c["start"])

    def step(c, i):
        a, b = i % 2, (i + 1) % 2
        F.flashloop_paged_plan(c["p"], c["kv"][a], c["new"], c["free"], c["left"][a], c["table"], c["cu"], c["kv"][b], c["slots"], c["pos"], c["left"][b], c["err"])
        F.flashloop_paged_kv_write(c["p"], c["q"][:, :Hk], c["q"][:, Hk:2 * Hk], c["slots"], c["kc"], c["vc"], c["err"])
        F.flashloop_paged_attn(c["p"], c["q"], c["kc"], c["vc"], c["table"], c["kv"][b], c["cu"], c["o"], None, c["ws"], c["err"])
        F.flashloop_prompt_attn(c["p"], c["o"], c["o"][:, 2:4], c["o"][:, 4:6], c["cu"], c["q"], None, c["err"])

    pools = [inputs(1), inputs(2)]
    want = []
    for c in pools:
        reset(c)
        for i in range(steps):
            step(c, i)
            torch.cuda.synchronize()
        want.append([c[x].clone() for x in ("q", "o", "kc", "vc")])
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        for c in pools:
            reset(c)
        for i in range(steps):
            side.wait_stream(main)
            with torch.cuda.stream(side):
                step(pools[i % 2], i)
            step(pools[1 - i % 2], i)
            main.wait_stream(side)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        for c, w in zip(pools, want):
            assert all(torch.equal(c[x], y) for x, y in zip(("q", "o", "kc", "vc"), w)) and c["err"].item() == 0
        assert want[0][0].isfinite().all()


def test_plan_without_requests_or_rows():
    """No requests: every slot is padding and the stack stays; no rows: the lengths stay."""
    for B, T in ((0, 9), (3, 0), (0, 0)):
        p = F.PagedParams.make(batch=B, max_tokens=T, max_new=1, n_heads=1, n_kv_heads=1, head_dim=64, page_size=16, n_pages=6, max_blocks=2)
        kv, new, table = ints([5] * B), ints([0] * B), ints([[3, -1]] * B).view(B, 2)
        cu, kv_out, slots, pos, left, err = ints([9] * (B + 1)), ints([9] * B), ints([9] * T), ints([9] * T), ints([9]), ints([0])
        F.flashloop_paged_plan(p, kv, new, ints([4, 1]), ints([2]), table, cu, kv_out, slots, pos, left, err)
        assert cu.tolist() == [0] * (B + 1) and kv_out.tolist() == [5] * B and left.tolist() == [2] and err.item() == 0
        assert slots.tolist() == [-1] * T and pos.tolist() == [0] * T and table.tolist() == [[3, -1]] * B


@pytest.mark.parametrize("kind", ["none", "object", "handle"])
def test_every_way_to_name_a_stream(kind):
    """The current stream, a stream object and a raw handle: the call runs there."""
    p, q, kc, vc, table, cu = paged_inputs([300, 40], [2, 1], 4, 2, 64, 16, BF, "thd", 0)
    want, got, err, ws = torch.zeros_like(q), torch.zeros_like(q), ints([0]), workspace(p)
    F.flashloop_paged_attn(p, q, kc, vc, table, ints([300, 40]), ints(cu), want, None, ws, err)
    kv, cus = ints([300, 40]), ints(cu)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    if kind == "none":
        with torch.cuda.stream(s):
            F.flashloop_paged_attn(p, q, kc, vc, table, kv, cus, got, None, ws, err)
    else:
        F.flashloop_paged_attn(p, q, kc, vc, table, kv, cus, got, None, ws, err, stream=s if kind == "object" else s.cuda_stream)
    s.synchronize()
    assert torch.equal(got, want) and err.item() == 0
