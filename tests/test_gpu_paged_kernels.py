"""The many-request attention where a call's bounds decide on the kernel: each test says which one its calls take, so
that a change of the rule cannot move a test away from what it is about."""
import numpy as np
import pytest
import torch

from paged_choice import scratch, tiles
from paged_reference import attention, gather
from test_gpu_paged import BF, HF, F, check, gen, ints, paged_inputs, randn, starts, wide, workspace

pytestmark = pytest.mark.gpu


def takes(p, tile, paged=True):
    assert tiles(p, paged) == tile
    if paged:
        assert F.flashloop_paged_attn_workspace_bytes(p) == scratch(p)


def test_the_largest_batch_through_the_tile_kernel():
    """65535 requests, the cut line over 2048 chunks of 32 of them."""
    B, H, Hk, dh, page, width, most, T = 65535, 4, 1, 64, 16, 40, 90, 700000
    rng = np.random.default_rng(5)
    new = rng.integers(0, 2, B)
    new[rng.integers(0, B, 400)] = most
    new[[0, B - 1]] = most, 33
    total = np.minimum(np.maximum(new, rng.integers(0, 200, B)), page * width)
    cu = np.concatenate([[0], np.cumsum(new)])
    g, n_pages = gen(1), 5000
    table = torch.randint(0, n_pages, (B, width), generator=g, device="cuda", dtype=torch.int32)
    kc, vc = randn(g, n_pages, page, Hk, dh, dtype=BF), randn(g, n_pages, page, Hk, dh, dtype=BF)
    q = torch.zeros(T, H, dh, dtype=BF, device="cuda")
    q[:int(cu[-1])] = randn(g, int(cu[-1]), H, dh, dtype=BF)
    p = F.PagedParams.make(batch=B, max_tokens=T, max_new=most, n_heads=H, n_kv_heads=Hk, head_dim=dh, page_size=page, n_pages=n_pages, max_blocks=width)
    takes(p, True)
    o, lse, err = torch.full_like(q, 7.0), torch.full((H, T), 7.0, device="cuda"), ints([0])
    F.flashloop_paged_attn(p, q, kc, vc, table, ints(total.tolist()), ints(cu.tolist()), o, lse, workspace(p), err)
    assert err.item() == 0 and not (o[:int(cu[-1])] == 7.0).all(-1).any() and (o[int(cu[-1]):] == 7.0).all() and (lse[:, int(cu[-1]):] == 7.0).all()
    for b in [0, 1, 31, 32, 33, B - 33, B - 32, B - 2, B - 1] + rng.integers(0, B, 60).tolist() + np.argsort(new)[-20:].tolist():
        t, n, r = int(total[b]), int(new[b]), slice(int(cu[b]), int(cu[b + 1]))
        want, l, tol, lt = attention(q[r], gather(kc, table[b], t), gather(vc, table[b], t), t - n, dh ** -0.5)
        assert ((o[r].double() - want).abs() <= tol).all() and ((lse[:, r].double() - l).abs() <= lt).all(), b


@pytest.mark.parametrize("dt,dh", [(BF, 128), (HF, 64)])
def test_rows_of_o_on_16_bytes_out_of_the_tile_kernel(dt, dh):
    """o from the eighth element on: the write-back's narrow stores, whole items and parts of cut ones."""
    H, Hk, lens = 4, 2, [260, 40, 500]
    cu = starts(lens)
    T = cu[-1] + wide(H)
    g = gen(dh)
    q, k, v = randn(g, T, H, dh, dtype=dt), randn(g, T, Hk, dh, dtype=dt), randn(g, T, Hk, dh, dtype=dt)
    p = F.PagedParams.make(batch=3, max_tokens=T, max_new=500, n_heads=H, n_kv_heads=Hk, head_dim=dh, dtype=dt)
    takes(p, True, paged=False)
    refs = [attention(q[a:b], k[a:b], v[a:b], 0, dh ** -0.5) for a, b in zip(cu, cu[1:])]
    whole, err = torch.full((T, H, dh + 16), 7.0, dtype=dt, device="cuda"), ints([0])
    o = whole[:, :, 8:dh + 8]
    assert o.data_ptr() % 32 == 16
    F.flashloop_prompt_attn(p, q, k, v, ints(cu), o, None, err)
    check(o, None, cu, refs, False)
    assert (whole[:, :, :8] == 7).all() and (whole[:, :, dh + 8:] == 7).all()
    p, q, kc, vc, table, cu = paged_inputs([3000, 700, 90], [300, 40, 90], H, Hk, dh, 64, dt, "thd", wide(H))
    takes(p, True)
    whole = torch.full((q.shape[0], H, dh + 16), 7.0, dtype=dt, device="cuda")
    o, n = whole[:, :, 8:dh + 8], [300, 40, 90]
    F.flashloop_paged_attn(p, q, kc, vc, table, ints([3000, 700, 90]), ints(cu), o, None, workspace(p), err)
    check(o, None, cu, [attention(q[cu[b]:cu[b + 1]], gather(kc, table[b], t), gather(vc, table[b], t), t - n[b], dh ** -0.5) for b, t in enumerate((3000, 700, 90))], False)
    assert (whole[:, :, :8] == 7).all() and (whole[:, :, dh + 8:] == 7).all() and err.item() == 0


@pytest.mark.parametrize("layout", ["heads", "tokens", "pages"])
def test_strides_of_zero_on_calls_of_the_tile_kernels_size(layout):
    """Tensor copies take no stride of zero: the few-row kernel serves the call, without the scratch that it came with."""
    H, Hk, dh, page, T = 4, 2, 128, 64, 300 + wide(4)
    g, err = gen(3), ints([0])
    q = randn(g, T, H, dh, dtype=BF)
    if layout != "pages":
        n = 300
        k1, v1 = (randn(g, T, 1, dh, dtype=BF) if layout == "heads" else randn(g, 1, Hk, dh, dtype=BF) for _ in range(2))
        k, v = k1.expand(T, Hk, dh), v1.expand(T, Hk, dh)
        p = F.PagedParams.make(batch=1, max_tokens=T, max_new=n, n_heads=H, n_kv_heads=Hk, head_dim=dh)
        takes(p, True, paged=False)
        o = torch.full_like(q, 7.0)
        F.flashloop_prompt_attn(p, q, k, v, ints([0, n]), o, None, err)
        check(o, None, [0, n], [attention(q[:n], k[:n], v[:n], 0, dh ** -0.5)], False)
    total, new = [1000, 300], [130, 170]
    shape = {"heads": (20, page, 1, dh), "tokens": (20, 1, Hk, dh), "pages": (1, page, Hk, dh)}[layout]
    kc, vc = (randn(g, *shape, dtype=BF).expand(20, page, Hk, dh) for _ in range(2))
    p = F.PagedParams.make(batch=2, max_tokens=T, max_new=170, n_heads=H, n_kv_heads=Hk, head_dim=dh, page_size=page, n_pages=20, max_blocks=16)
    takes(p, True)
    table, cu = torch.randperm(20, generator=g, device="cuda").to(torch.int32)[None].repeat(2, 1)[:, :16].contiguous(), [0, 130, 300]
    o = torch.full_like(q, 7.0)
    F.flashloop_paged_attn(p, q, kc, vc, table, ints(total), ints(cu), o, None, workspace(p), err)
    check(o, None, cu, [attention(q[cu[b]:cu[b + 1]], gather(kc, table[b], t), gather(vc, table[b], t), t - new[b], dh ** -0.5) for b, t in enumerate(total)], False)
    assert err.item() == 0


@pytest.mark.parametrize("page", [64, 256])
def test_tensor_copies_from_beyond_32_bits(page):
    """Pages behind the first 2^31 elements of a pool, through the tile kernel."""
    Hk, dh, H = 4, 128, 8
    n_pages = (1 << 31) // (page * Hk * dh) + 900
    kc, vc = (torch.empty(n_pages, page, Hk, dh, dtype=BF, device="cuda") for _ in range(2))
    width = 768 // page
    table, total, new = ints([list(range(n_pages - width, n_pages)), list(range(width))]), [750, 700], [300, 50]
    g = gen(4)
    for c in (kc, vc):
        for b in range(2):
            c[table[b].long()] = randn(g, width, page, Hk, dh, dtype=BF)
    T = sum(new) + wide(H)
    p = F.PagedParams.make(batch=2, max_tokens=T, max_new=300, n_heads=H, n_kv_heads=Hk, head_dim=dh, page_size=page, n_pages=n_pages, max_blocks=width)
    takes(p, True)
    q, err, cu = randn(g, T, H, dh, dtype=BF), ints([0]), starts(new)
    o = torch.full_like(q, 7.0)
    F.flashloop_paged_attn(p, q, kc, vc, table, ints(total), ints(cu), o, None, workspace(p), err)
    check(o, None, cu, [attention(q[cu[b]:cu[b + 1]], gather(kc, table[b], t), gather(vc, table[b], t), t - new[b], dh ** -0.5) for b, t in enumerate(total)], False)
    assert err.item() == 0


@pytest.mark.parametrize("lens,H,Hk,dh,dt", [([1], 1, 1, 64, BF), ([1, 1, 1], 4, 2, 128, HF), ([0, 5, 0, 3, 0], 3, 1, 64, BF), ([7, 2, 32, 1], 16, 2, 128, BF)])
def test_single_rows_through_the_tile_kernel(lens, H, Hk, dh, dt):
    """Requests of a few rows in a call whose bounds allow many."""
    g, cu = gen(len(lens)), starts(lens)
    T = cu[-1] + wide(H)
    q, k, v = randn(g, T, H, dh, dtype=dt), randn(g, T, Hk, dh, dtype=dt), randn(g, T, Hk, dh, dtype=dt)
    p = F.PagedParams.make(batch=len(lens), max_tokens=T, max_new=200, n_heads=H, n_kv_heads=Hk, head_dim=dh, dtype=dt)
    takes(p, True, paged=False)
    o, lse, err = torch.full_like(q, 7.0), torch.full((H, T), 7.0, device="cuda"), ints([0])
    F.flashloop_prompt_attn(p, q, k, v, ints(cu), o, lse, err)
    check(o, lse, cu, [attention(q[a:b], k[a:b], v[a:b], 0, dh ** -0.5) for a, b in zip(cu, cu[1:])], True)
    assert err.item() == 0


WAYS = [("few whole", 20, 160, 0, False), ("few cut", 3, 3000, 0, False), ("tiles", 200, 1500, 1, True)]


@pytest.mark.parametrize("way,n,L,padded,tile", WAYS, ids=[w[0] for w in WAYS])
@pytest.mark.parametrize("bad", ["length", "negative", "start", "rows", "descending", "page"])
def test_requests_beside_a_refused_one_are_whole(way, n, L, padded, tile, bad):
    """A request whose lengths contradict the bounds is skipped, and those before and behind it are not; a bad page counts as zeros."""
    H, Hk, dh, page = 4, 2, 128, 16
    total, new = [L, L - 7, L - n, L // 2], [n, n, n, n - 1]
    p, q, kc, vc, table, cu = paged_inputs(total, new, H, Hk, dh, page, BF, "thd", 2 * n + padded * wide(H))
    takes(p, tile)
    lens, at, hit = list(total), list(cu), {1}
    if bad == "length":
        lens[1] = table.shape[1] * page + 1
    elif bad == "negative":
        lens[1] = -1
    elif bad == "start":  # the last request ends behind the rows
        at[4], hit = q.shape[0] + 1, {3}
    elif bad == "rows":  # more rows than max_new
        at = [0, n, 2 * n + 1, 3 * n + 1, 4 * n]
    elif bad == "descending":
        at, hit = [n + 1, n, 2 * n, 3 * n, 4 * n - 1], {0}
    else:
        table[1, 2], hit = p.n_pages, set()
    o, lse, err = torch.full_like(q, 7.0), torch.full((H, q.shape[0]), 7.0, device="cuda"), ints([0])
    F.flashloop_paged_attn(p, q, kc, vc, table, ints(lens), ints(at), o, lse, workspace(p), err)
    assert err.item() == 2
    written = torch.zeros(q.shape[0], dtype=torch.bool, device="cuda")
    for b in range(4):
        if b in hit:
            continue
        r, t = slice(at[b], at[b + 1]), total[b]
        tab = table[b].clone()
        if bad == "page" and b == 1:
            tab[2] = 0
        k, v = gather(kc, tab, t), gather(vc, tab, t)
        if bad == "page" and b == 1:
            k[2 * page:3 * page], v[2 * page:3 * page] = 0, 0
        want, l, tol, lt = attention(q[r], k, v, t - (at[b + 1] - at[b]), dh ** -0.5)
        assert ((o[r].double() - want).abs() <= tol).all() and ((lse[:, r].double() - l).abs() <= lt).all(), b
        written[r] = True
    assert (o[~written] == 7).all() and (lse[:, ~written] == 7).all()


@pytest.mark.parametrize("way,n,L,padded,tile", WAYS, ids=[w[0] for w in WAYS])
@pytest.mark.parametrize("odd", [False, True])
def test_results_over_the_queries(way, n, L, padded, tile, odd):
    """o may be q itself, also where values that are not finite make the few-row kernel take an item twice."""
    H, Hk, dh, page = 4, 2, 128, 16
    total, new = [L, L - 7, 40], [n, n, min(n, 20)]
    p, q, kc, vc, table, cu = paged_inputs(total, new, H, Hk, dh, page, BF, "thd", padded * wide(H))
    takes(p, tile)
    if odd:
        for b, t in enumerate(total):
            vc[table[b, (t - 1) // page].long(), (t - 1) % page, :, 5] = float("inf")
    want, err = torch.zeros_like(q), ints([0])
    F.flashloop_paged_attn(p, q, kc, vc, table, ints(total), ints(cu), want, None, workspace(p), err)
    got = q.clone()
    F.flashloop_paged_attn(p, got, kc, vc, table, ints(total), ints(cu), got, None, workspace(p), err)
    assert torch.equal(got[:cu[-1]], want[:cu[-1]]) and torch.equal(got[cu[-1]:], q[cu[-1]:]) and err.item() == 0
    assert want[:cu[-1]].isfinite().all() != odd
    if not padded:
        p = F.PagedParams.make(batch=3, max_tokens=cu[-1], max_new=n, n_heads=H, n_kv_heads=Hk, head_dim=dh)
        k, v = randn(gen(1), cu[-1], Hk, dh, dtype=BF), randn(gen(2), cu[-1], Hk, dh, dtype=BF)
        if odd:
            v[cu[1] - 1, :, 3] = float("nan")
        F.flashloop_prompt_attn(p, q, k, v, ints(cu), want, None, err)
        got = q.clone()
        F.flashloop_prompt_attn(p, got, k, v, ints(cu), got, None, err)
        assert torch.equal(torch.nan_to_num(got, 9.0), torch.nan_to_num(want, 9.0)) and want.isnan().any() == odd
