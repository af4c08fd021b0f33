"""The many-request attention where values are not finite: a row's result depends on the columns it sees alone."""
import math

import pytest
import torch

from paged_choice import scratch, tiles
from paged_reference import attention, gather
from test_gpu_paged import BF, HF, F, gen, ints, paged_inputs, randn, starts, wide, workspace

pytestmark = pytest.mark.gpu


def plant(v, seed, share=0.004):
    """Infinities of either sign and NaN among the values of [L, Hk, dh], at the ends and at random."""
    g = gen(seed)
    L = v.shape[0]
    at = torch.rand(v.shape, generator=g, device="cuda") < share
    at[0, :, 1], at[L - 1, :, 3], at[max(0, L - 2), :, 4], at[L // 2, :, 5] = True, True, True, True
    kind = torch.randint(0, 3, v.shape, generator=g, device="cuda")
    odd = torch.tensor([math.inf, -math.inf, math.nan], device="cuda")[kind].to(v.dtype)
    keep = torch.rand(v.shape[1:], generator=g, device="cuda") < 0.3  # channels without any
    keep[:, 1:6] = False
    return torch.where(at & ~keep, odd, v)


def expected(q, k, v, first, scale):
    """(o, tolerance, where o is +inf, -inf, nan) of rows that see j <= first + i."""
    o, _, tol, _ = attention(q, k, v, first, scale)
    n, G = q.shape[0], q.shape[1] // v.shape[1]
    lim = first + torch.arange(n, device=q.device)

    def seen(mask):  # [L, Hk, dh] -> [n, H, dh]: some column that the row sees
        c = torch.cat([torch.zeros_like(mask[:1]), mask.cumsum(0) > 0])
        return c[(lim + 1).clamp(0, mask.shape[0])].repeat_interleave(G, 1)
    if v.shape[0] == 0:
        z = torch.zeros(o.shape, dtype=torch.bool, device=q.device)
        return o, tol, z, z, z
    up, down, none = seen(v == math.inf), seen(v == -math.inf), seen(v.isnan())
    none = none | (up & down)
    return o, tol, up & ~none, down & ~none, none


def compare(got, want):
    o, tol, up, down, none = want
    assert torch.equal(got == math.inf, up) and torch.equal(got == -math.inf, down) and torch.equal(got.isnan(), none)
    fin = ~(up | down | none)
    off = torch.where(fin, (got.double() - o).abs() - tol, -1.0)
    assert not (off > 0).any(), off.max().item()
    return int((up | down | none).sum()), int(fin.sum())


def prompt_case(lens, H, Hk, dh, dt, extra, tile):
    g, cu = gen(sum(lens) + H), starts(lens)
    T = cu[-1] + extra
    q, k, v = randn(g, T, H, dh, dtype=dt), randn(g, T, Hk, dh, dtype=dt), randn(g, T, Hk, dh, dtype=dt)
    for b, (a, z) in enumerate(zip(cu, cu[1:])):
        if z > a and b % 3 != 2:
            v[a:z] = plant(v[a:z], b)
    if extra:
        v[cu[-1]:] = math.nan
    p = F.PagedParams.make(batch=len(lens), max_tokens=T, max_new=max(lens), n_heads=H, n_kv_heads=Hk, head_dim=dh, dtype=dt)
    assert tiles(p, False) == tile
    o, lse, err = torch.full_like(q, 7.0), torch.full((H, T), 7.0, device="cuda"), ints([0])
    F.flashloop_prompt_attn(p, q, k, v, ints(cu), o, lse, err)
    odd = fin = 0
    for a, z in zip(cu, cu[1:]):
        n, m = compare(o[a:z], expected(q[a:z], k[a:z], v[a:z], 0, dh ** -0.5))
        odd, fin = odd + n, fin + m
        _, l, _, tol = attention(q[a:z], k[a:z], torch.zeros_like(v[a:z]), 0, dh ** -0.5)
        assert ((lse[:, a:z].double() - l).abs() <= tol).all()
    assert odd > 0 and fin > 0 and err.item() == 0 and (o[cu[-1]:] == 7).all()


def paged_case(total, new, H, Hk, dh, page, dt, layout, extra, tile):
    p, q, kc, vc, table, cu = paged_inputs(total, new, H, Hk, dh, page, dt, layout, extra)
    assert (F.flashloop_paged_attn_workspace_bytes(p), tiles(p, True)) == (scratch(p), tile)
    for b, t in enumerate(total):
        if t and b % 3 != 2:
            j = torch.arange(t, device="cuda")
            vc[table[b].long()[j // page], j % page] = plant(gather(vc, table[b], t), b)
    o, err = torch.full_like(q, 7.0), ints([0])
    F.flashloop_paged_attn(p, q, kc, vc, table, ints(total), ints(cu), o, None, workspace(p), err)
    odd = fin = 0
    for b, t in enumerate(total):
        r = slice(cu[b], cu[b + 1])
        n, m = compare(o[r], expected(q[r], gather(kc, table[b], t), gather(vc, table[b], t), t - new[b], dh ** -0.5))
        odd, fin = odd + n, fin + m
    assert odd > 0 and fin > 0 and err.item() == 0 and (o[cu[-1]:] == 7).all()


FEW_PROMPTS = [
    ([5, 40, 3], 1, 1, 64, BF), ([9, 2, 14], 4, 4, 128, HF), ([16, 3, 70], 2, 1, 128, BF), ([100, 33, 80, 1], 4, 2, 64, HF), ([40] * 20, 8, 1, 128, BF), ([60] * 9, 8, 8, 64, HF), ([70, 150] * 4, 8, 2, 64, BF),
]


@pytest.mark.parametrize("lens,H,Hk,dh,dt", FEW_PROMPTS)
def test_prompt_rows_see_their_own_columns_values(lens, H, Hk, dh, dt):
    prompt_case(lens, H, Hk, dh, dt, 0, False)


FEW_PAGED = [  # whole requests up to 512 columns, cut lines beyond; 8, 16 and more packed rows
    ([60, 17, 200], [4, 2, 3], 2, 1, 64, 16, BF, "thd"), ([300, 40, 9], [8, 5, 3], 2, 1, 128, 32, HF, "htd"), ([400, 64, 30], [20, 30, 6], 4, 2, 128, 16, BF, "thd"),
    ([3000, 700, 70], [8, 3, 2], 1, 1, 128, 16, BF, "both"), ([2500, 64, 900], [4, 4, 4], 8, 2, 64, 64, HF, "thd"), ([5000, 333, 80], [4, 3, 4], 16, 2, 128, 256, BF, "thd"),
    ([700, 2, 5], [12, 6, 5], 3, 1, 64, 16, HF, "thd"),
]


@pytest.mark.parametrize("total,new,H,Hk,dh,page,dt,layout", FEW_PAGED)
def test_paged_rows_see_their_own_columns_values(total, new, H, Hk, dh, page, dt, layout):
    paged_case(total, new, H, Hk, dh, page, dt, layout, 0, False)


TILE_PROMPTS = [
    ([200, 1, 77, 640], 4, 2, 128, BF), ([1500], 2, 2, 64, HF), ([300, 129, 128, 1000], 8, 8, 128, HF), ([90, 257, 31], 16, 1, 64, BF), ([130, 70], 40, 2, 128, BF),
]


@pytest.mark.parametrize("lens,H,Hk,dh,dt", TILE_PROMPTS)
def test_prompt_tiles_see_their_own_columns_values(lens, H, Hk, dh, dt):
    prompt_case(lens, H, Hk, dh, dt, wide(H), True)


TILE_PAGED = [
    ([2000, 333, 900], [300, 40, 128], 4, 2, 128, 16, BF, "thd"), ([700, 130, 64], [700, 100, 64], 4, 4, 64, 128, HF, "htd"), ([9000, 50, 400], [513, 50, 1], 8, 1, 128, 256, BF, "both"),
    ([300, 700, 1000], [400, 37, 999], 6, 2, 128, 32, HF, "thd"),
]


@pytest.mark.parametrize("total,new,H,Hk,dh,page,dt,layout", TILE_PAGED)
def test_paged_tiles_see_their_own_columns_values(total, new, H, Hk, dh, page, dt, layout):
    paged_case(total, new, H, Hk, dh, page, dt, layout, wide(H), True)


def sink_tolerance(q, k, v, first, scale):
    """The bounds of `attention` for fp16 with the probabilities' absolute step at 2^-32 of the largest: rounded at
    2^-25 or better (half a step of its smallest numbers), with the largest at 2^7 or more."""
    o, _, tol, _ = attention(q, k, v, first, scale)
    each = v.double().abs().sum(0).repeat_interleave(q.shape[1] // v.shape[1], 0)[None]
    return o, tol - 2.0 ** -25 * each + 2.0 ** -32 * each


@pytest.mark.parametrize("gap", [6, 10, 14, 16, 18])  # nats between the first key's score and the others'
@pytest.mark.parametrize("new,H,extra", [(1, 4, False), (1, 16, False), (3, 8, False), (150, 8, True)])  # both roundings of few rows, 24 rows, tiles
def test_small_probabilities_of_fp16_count(gap, new, H, extra):
    """A first key that draws nearly all weight to a value of zero: the result is the many small probabilities'."""
    L, dh, page = 6000, 128, 64
    n_pages = -(-L // page)
    kc, vc = torch.zeros(n_pages, page, 1, dh, dtype=HF, device="cuda"), (4 + randn(gen(gap), n_pages, page, 1, dh)).to(HF)
    kc[0, 0, 0, 0], vc[0, 0] = gap, 0.0
    T = new + (wide(H) if extra else 0)
    q = torch.zeros(T, H, dh, dtype=HF, device="cuda")
    q[:, :, 0] = 1.0
    p = F.PagedParams.make(batch=1, max_tokens=T, max_new=new, n_heads=H, n_kv_heads=1, head_dim=dh, page_size=page, n_pages=n_pages, max_blocks=n_pages, dtype=HF, scale=1.0)
    assert tiles(p, True) == extra
    table, o, lse, err = ints([list(range(n_pages))]), torch.zeros_like(q), torch.zeros(H, T, device="cuda"), ints([0])
    F.flashloop_paged_attn(p, q, kc, vc, table, ints([L]), ints([0, new]), o, lse, workspace(p), err)
    k, v = gather(kc, table[0], L), gather(vc, table[0], L)
    want, tol = sink_tolerance(q[:new], k, v, L - new, 1.0)
    _, l, _, lt = attention(q[:new], k, v, L - new, 1.0)
    off = (o[:new].double() - want).abs()
    assert (off <= tol).all(), ((off / want.abs().clamp(min=1e-30)).median().item(), (off - tol).max().item())
    assert ((lse[:, :new].double() - l).abs() <= lt).all() and err.item() == 0


@pytest.mark.parametrize("n,H,Hk,dh,dt,extra", [(40, 4, 2, 128, BF, False), (150, 8, 1, 64, HF, False), (300, 4, 2, 128, HF, True), (520, 2, 2, 64, BF, True)])
@pytest.mark.parametrize("what", ["key", "query"])
def test_keys_and_queries_that_are_not_finite(n, H, Hk, dh, dt, extra, what):
    """A key reaches the rows that see its column, a query its own row and head, also within a tile."""
    g, T, at = gen(n), n + (wide(H) if extra else 0), n * 2 // 3
    q, k, v = randn(g, T, H, dh, dtype=dt), randn(g, T, Hk, dh, dtype=dt), randn(g, T, Hk, dh, dtype=dt)
    p = F.PagedParams.make(batch=1, max_tokens=T, max_new=n, n_heads=H, n_kv_heads=Hk, head_dim=dh, dtype=dt)
    assert tiles(p, False) == extra
    want, l, tol, lt = attention(q[:n], k[:n], v[:n], 0, dh ** -0.5)
    hit = torch.zeros(n, H, dtype=torch.bool, device="cuda")
    if what == "key":
        k[at, Hk - 1, 7] = math.nan
        hit[at:, H - H // Hk:] = True
    else:
        q[at, 1, 3], q[at + 5, 0, 9] = math.nan, math.inf
        hit[at, 1], hit[at + 5, 0] = True, True
    o, lse, err = torch.full_like(q, 7.0), torch.full((H, T), 7.0, device="cuda"), ints([0])
    F.flashloop_prompt_attn(p, q, k, v, ints([0, n]), o, lse, err)
    assert o[:n][hit].isnan().all() and not lse[:, :n].T[hit].isfinite().any()
    assert (((o[:n].double() - want).abs() - tol)[~hit] <= 0).all() and (((lse[:, :n].T.double() - l.T).abs() - lt.T)[~hit] <= 0).all()
    assert (o[n:] == 7).all() and err.item() == 0


@pytest.mark.parametrize("lens,H,Hk,dh,tile", [([6000, 900], 8, 8, 128, True), ([4000], 16, 1, 64, True), ([60] * 9, 8, 8, 128, False)])
def test_nothing_but_values_that_are_not_finite(lens, H, Hk, dh, tile):
    """Every value taken out and put back: no wait runs out, and every row is what it sees."""
    cu, g = starts(lens), gen(1)
    T = cu[-1]
    q, k = randn(g, T, H, dh, dtype=BF), randn(g, T, Hk, dh, dtype=BF)
    v = torch.full((T, Hk, dh), math.inf, dtype=BF, device="cuda")
    v[..., ::2], v[..., 1::4] = math.nan, -math.inf
    p = F.PagedParams.make(batch=len(lens), max_tokens=T, max_new=max(lens), n_heads=H, n_kv_heads=Hk, head_dim=dh)
    assert tiles(p, False) == tile
    o, err = torch.zeros_like(q), ints([0])
    F.flashloop_prompt_attn(p, q, k, v, ints(cu), o, None, err)
    assert o[..., ::2].isnan().all() and (o[..., 1::4] == -math.inf).all() and (o[..., 3::4] == math.inf).all() and err.item() == 0
