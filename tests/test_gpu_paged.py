"""The many-request operators on the GPU against plain 64-bit implementations:
block tables and slot maps, cache writes, attention over packed prompts and
over the paged cache."""
import math
import random

import numpy as np
import pytest
import torch

from paged_reference import attention, build_plan, gather

F = pytest.importorskip("cross_loop_sparse_b200.flashloop")
pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape, dtype=torch.float32, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


# ------------------------------------------------------------------------------- plan
PLANS = [
    ([0], [1], 16, 0), ([15], [1], 16, 3), ([16], [1], 16, 0), ([0, 0, 0], [0, 0, 0], 64, 5), ([7, 0, 31, 64], [0, 33, 1, 0], 32, 0),
    ([300], [2000], 128, 17), ([5] * 700, [3] * 700, 16, 1), (list(range(1300)), [i % 5 for i in range(1300)], 256, 40), ([0] * 40, [i * 37 % 900 for i in range(40)], 64, 0),
]


def plan_inputs(held, new, page, pad, seed=0, spare=4):
    rng = random.Random(seed)
    blocks = [-(-h // page) for h in held]
    opened = sum(-(-(h + n) // page) for h, n in zip(held, new)) - sum(blocks)
    ids = list(range(sum(blocks) + opened + spare))
    rng.shuffle(ids)
    width = max(-(-(h + n) // page) for h, n in zip(held, new)) + 2
    table, at = [], 0
    for k in blocks:
        table.append(ids[at:at + k] + [-7] * (width - k))
        at += k
    return table, ids[at:], len(ids), width, max(1, sum(new) + pad)


class Plan:
    """Buffers of one call of flashloop_paged_plan."""

    def __init__(self, held, new, table, stack, page, n_pages, width, T):
        B = len(held)
        self.p = F.PagedParams.make(batch=B, max_tokens=T, max_new=max(1, max(new, default=1)), n_heads=1, n_kv_heads=1, head_dim=64,
                                    page_size=page, n_pages=n_pages, max_blocks=width)
        self.kv, self.new, self.stack = ints(held), ints(new), ints(stack + [-9])
        self.n_free, self.table = ints([len(stack)]), ints(table)
        self.cu, self.kv_out, self.slots, self.pos = ints([-3] * (B + 1)), ints([-3] * B), ints([-3] * T), ints([-3] * T)
        self.n_out, self.err = ints([-3]), ints([0])

    def run(self, stream=None):
        F.flashloop_paged_plan(self.p, self.kv, self.new, self.stack, self.n_free, self.table, self.cu, self.kv_out, self.slots, self.pos,
                               self.n_out, self.err, stream)
        return self


@pytest.mark.parametrize("held,new,page,pad", PLANS)
def test_plan_matches_the_definition(held, new, page, pad):
    table, stack, n_pages, width, T = plan_inputs(held, new, page, pad)
    c = Plan(held, new, table, stack, page, n_pages, width, T)
    for _ in range(2):  # a second call on the same lengths gives the same
        c.run()
        cu, kv, tab, slots, pos, left = build_plan(held, new, table, stack, page)
        spare = T - len(slots)
        assert c.cu.tolist() == cu and c.kv_out.tolist() == kv and c.n_out.tolist() == [left]
        assert c.table.tolist() == tab
        assert c.slots.tolist() == slots + [-1] * spare and c.pos.tolist() == pos + [0] * spare
        assert c.err.item() == 0


@pytest.mark.parametrize("held,new,cut,code", [
    ([3, 20], [30, 9], "pages", 1), ([3, 20], [30, 9], "tokens", 1), ([3, 20], [30, 9], "blocks", 1), ([3, 20], [30, -1], "", 2), ([-4, 20], [30, 1], "", 2),
    ([2147483647, 0], [2147483647, 1], "", 1), ([3, 20], [30, 9], "count", 2),
])
def test_plan_appends_all_or_nothing(held, new, cut, code):
    page = 16
    table, stack, n_pages, width, T = plan_inputs([3, 20], [30, 9], page, 0, spare=0)
    stack = stack[1:] if cut == "pages" else stack
    T -= cut == "tokens"
    width = 2 if cut == "blocks" else width
    table = [r[:width] for r in table]
    c = Plan(held, new, table, stack, page, n_pages, width, T)
    if cut == "count":  # more free pages than the buffer holds
        c.stack = c.stack[:len(stack) - 1].contiguous()
    c.run()
    assert c.err.item() == code
    assert c.cu.tolist() == [0, 0, 0] and c.kv_out.tolist() == held and c.n_out.tolist() == [len(stack)]
    assert c.table.tolist() == table
    assert set(c.slots.tolist()) == {-1} and set(c.pos.tolist()) == {0}


def test_plan_reports_bad_pages():
    table, stack, n_pages, width, T = plan_inputs([3, 20], [30, 9], 16, 0, spare=0)
    want = build_plan([3, 20], [30, 9], table, stack, 16)[3]
    bad = stack[-1]
    c = Plan([3, 20], [30, 9], table, stack[:-1] + [n_pages], 16, n_pages, width, T).run()
    assert c.err.item() == 2
    assert c.slots.tolist() == [-1 if s // 16 == bad else s for s in want]


# ------------------------------------------------------------------------------- write
@pytest.mark.parametrize("T,H,dh,src,dt,page,layout", [
    (1, 1, 64, BF, BF, 16, "thd"), (7, 5, 128, HF, HF, 32, "htd"), (33, 4, 64, torch.float32, BF, 64, "fused"), (130, 3, 128, torch.float32, HF, 256, "thd"),
    (2001, 8, 128, BF, BF, 128, "fused"),
])
def test_write_puts_rows_into_their_slots(T, H, dh, src, dt, page, layout):
    g = gen(T)
    n_pages = -(-T // page) + 3
    if layout == "fused":
        qkv = randn(g, T, 3 * H, dh, dtype=src)
        k, v = qkv[:, H:2 * H], qkv[:, 2 * H:]
    else:
        k, v = randn(g, T, H, dh, dtype=src), randn(g, T, H, dh, dtype=src)
    if layout == "htd":  # pages with the heads outside
        kc, vc = (randn(g, n_pages, H, page, dh, dtype=dt).transpose(1, 2) for _ in range(2))
    else:
        both = randn(g, n_pages, 2, page, H, dh, dtype=dt)
        kc, vc = both[:, 0], both[:, 1]
    slots = torch.randperm(n_pages * page, generator=g, device="cuda")[:T].to(torch.int32)
    slots[::5] = -1
    want_k, want_v = kc.clone(), vc.clone()
    keep = (slots >= 0).nonzero().flatten()
    at = slots[keep].long()
    want_k[at // page, at % page] = k[keep].to(dt)
    want_v[at // page, at % page] = v[keep].to(dt)
    p = F.PagedParams.make(batch=1, max_tokens=T, max_new=T, n_heads=H, n_kv_heads=H, head_dim=dh, page_size=page, n_pages=n_pages, dtype=dt)
    err = ints([0])
    F.flashloop_paged_kv_write(p, k, v, slots, kc, vc, err)
    assert torch.equal(kc, want_k) and torch.equal(vc, want_v) and err.item() == 0


def test_write_rounds_to_nearest_even_and_reports_range():
    x = torch.tensor([1 + 2.0 ** -9, 1 + 3 * 2.0 ** -9, 65519.0, -65520.0, math.inf, -math.inf, math.nan, 2.0 ** -26] * 8, device="cuda")
    for dt, code in ((BF, 0), (HF, 4)):
        kc, vc = torch.zeros(1, 16, 1, 64, dtype=dt, device="cuda"), torch.zeros(1, 16, 1, 64, dtype=dt, device="cuda")
        p = F.PagedParams.make(batch=1, max_tokens=1, max_new=1, n_heads=1, n_kv_heads=1, head_dim=64, page_size=16, dtype=dt)
        err = ints([0])
        F.flashloop_paged_kv_write(p, x.view(1, 1, 64), torch.zeros(1, 1, 64, device="cuda"), ints([3]), kc, vc, err)
        assert torch.equal(torch.nan_to_num(kc[0, 3, 0], 7.0), torch.nan_to_num(x.to(dt), 7.0)) and err.item() == code
    err = ints([0])  # infinities alone are copied without a report
    F.flashloop_paged_kv_write(p, torch.full((1, 1, 64), math.inf, device="cuda"), torch.zeros(1, 1, 64, device="cuda"), ints([3]), kc, vc, err)
    assert err.item() == 0


def test_write_reports_slots_outside_the_pool():
    kc, vc = torch.zeros(2, 16, 1, 64, dtype=BF, device="cuda"), torch.zeros(2, 16, 1, 64, dtype=BF, device="cuda")
    p = F.PagedParams.make(batch=1, max_tokens=4, max_new=4, n_heads=1, n_kv_heads=1, head_dim=64, page_size=16, n_pages=2)
    k = torch.ones(4, 1, 64, dtype=BF, device="cuda")
    err = ints([0])
    F.flashloop_paged_kv_write(p, k, k, ints([32, -2, 31, 2147483647]), kc, vc, err)
    assert err.item() == 2 and kc.float().sum().item() == 64 and kc[1, 15].float().sum().item() == 64


# ------------------------------------------------------------------------------- attention
def check(got, got_lse, cu, refs, lse, untouched=7.0):
    for b, (o, l, ot, lt) in enumerate(refs):
        r = slice(cu[b], cu[b + 1])
        off = (got[r].double() - o).abs() - ot
        assert not (off > 0).any() and not got[r].isnan().any(), (b, off.max().item(), (off > 0).sum().item())
        if lse:
            empty = l == -math.inf
            d = got_lse[:, r].double()
            assert torch.equal(d == -math.inf, empty), b
            assert ((torch.where(empty, 0.0, d - l).abs() - lt) <= 0).all(), (b, (d - l).abs().max().item())
    assert (got[cu[-1]:] == untouched).all()
    if lse:
        assert (got_lse[:, cu[-1]:] == untouched).all()


def starts(n):
    return [0] + np.cumsum(n).tolist()


PROMPTS = [
    ([1], 1, 1, 64, BF, 0), ([1, 1, 1], 4, 2, 128, HF, 2), ([0, 5, 0, 3, 0], 3, 1, 64, BF, 1), ([127, 128, 129], 4, 4, 128, BF, 0), ([255, 256, 257, 1], 6, 2, 64, HF, 9),
    ([700, 33, 512], 7, 1, 128, BF, 0), ([1500], 16, 2, 128, HF, 3), ([2049], 2, 2, 64, BF, 0), ([3, 1000, 64, 640], 12, 4, 128, BF, 130), ([300] * 30, 4, 4, 64, HF, 0),
    ([40] * 200, 8, 1, 128, BF, 0), ([130, 70], 40, 1, 64, BF, 0),
]


def wide(H):
    """Rows to pad a call with so that its bounds send it to the tile kernel, which small ones do not reach."""
    return 60000 // H


@pytest.mark.parametrize("lens,H,Hk,dh,dt,pad", PROMPTS)
@pytest.mark.parametrize("fused,padded", [(False, False), (True, False), (False, True)])
def test_prompt_attention(lens, H, Hk, dh, dt, pad, fused, padded):
    g = gen(len(lens) * 1000 + H)
    pad += wide(H) if padded else 0
    cu = starts(lens)
    T = max(1, cu[-1] + pad)
    if fused:
        qkv = randn(g, T, H + 2 * Hk, dh, dtype=dt, std=1.3)
        q, k, v = qkv[:, :H], qkv[:, H:H + Hk], qkv[:, H + Hk:]
        o = torch.full((H, T, dh), 7.0, dtype=dt, device="cuda").transpose(0, 1)
    else:
        q, k, v = randn(g, T, H, dh, dtype=dt, std=1.5), randn(g, T, Hk, dh, dtype=dt), randn(g, T, Hk, dh, dtype=dt)
        o = torch.full((T, H, dh), 7.0, dtype=dt, device="cuda")
    if pad:
        k[cu[-1]:], v[cu[-1]:] = math.nan, math.inf
    lse = torch.full((H, T), 7.0, device="cuda")
    p = F.PagedParams.make(batch=len(lens), max_tokens=T, max_new=max(lens), n_heads=H, n_kv_heads=Hk, head_dim=dh, dtype=dt)
    err = ints([0])
    F.flashloop_prompt_attn(p, q, k, v, ints(cu), o, lse, err)
    refs = [attention(q[a:b], k[a:b], v[a:b], 0, dh ** -0.5) for a, b in zip(cu, cu[1:])]
    check(o, lse, cu, refs, True)
    assert err.item() == 0
    o2 = torch.full_like(o, 7.0)
    F.flashloop_prompt_attn(p, q, k, v, ints(cu), o2, None, err)
    assert torch.equal(o2, o)  # the same bits without the sums, and on a second call


@pytest.mark.parametrize("padded", [0, 1])
def test_prompt_neighbours_do_not_leak(padded):
    """Infinities and NaN in one request's rows stay in that request."""
    g, lens = gen(5), [200, 77, 300, 131]
    cu = starts(lens)
    T, H, Hk, dh = cu[-1] + padded * wide(4), 4, 2, 128
    q, k, v = randn(g, T, H, dh, dtype=BF), randn(g, T, Hk, dh, dtype=BF), randn(g, T, Hk, dh, dtype=BF)
    for x in (q, k, v):
        x[cu[1]:cu[2]] = math.nan
        x[cu[3] + 3] = math.inf
    p = F.PagedParams.make(batch=4, max_tokens=T, max_new=300, n_heads=H, n_kv_heads=Hk, head_dim=dh)
    o, lse, err = torch.empty(T, H, dh, dtype=BF, device="cuda"), torch.empty(H, T, device="cuda"), ints([0])
    F.flashloop_prompt_attn(p, q, k, v, ints(cu), o, lse, err)
    for b in (0, 2):
        r = slice(cu[b], cu[b + 1])
        want, l, ot, lt = attention(q[r], k[r], v[r], 0, dh ** -0.5)
        assert ((o[r].double() - want).abs() <= ot).all() and ((lse[:, r].double() - l).abs() <= lt).all()
    assert o[cu[1]:cu[2]].isnan().all()


PAGED = [  # cached lengths (new tokens included), new tokens, H, Hk, dh, page, type, layout, pad
    ([1], [1], 1, 1, 64, 16, BF, "thd", 0),
    ([256], [1], 4, 4, 64, 16, BF, "thd", 0),
    ([5, 0, 300, 16, 17], [1, 1, 1, 0, 1], 8, 2, 128, 16, HF, "thd", 1),
    ([4000, 63, 64, 65, 1], [1] * 5, 16, 16, 128, 64, BF, "htd", 2),
    ([9000], [1], 8, 1, 128, 32, BF, "both", 0),
    ([20000, 3], [1, 1], 2, 1, 64, 256, HF, "thd", 0),
    ([700, 41, 2000], [3, 4, 2], 7, 1, 128, 16, BF, "thd", 0),
    ([700, 41, 2000], [4, 4, 4], 8, 1, 64, 128, HF, "both", 3),
    ([130, 600], [130, 17], 4, 2, 128, 16, BF, "thd", 0),
    ([1000, 257, 128], [300, 257, 5], 12, 4, 128, 64, HF, "htd", 4),
    ([5000], [64], 8, 2, 64, 32, BF, "thd", 0),
    ([4100, 6000], [100, 333], 32, 8, 128, 64, BF, "both", 0),
    ([2000, 900, 3, 400, 1], [1, 500, 1, 37, 1], 16, 2, 128, 32, BF, "thd", 7),
    ([3, 2, 100, 9], [8, 2, 300, 40], 4, 1, 128, 16, BF, "thd", 0),       # fewer cached than new: rows that see nothing
    ([0, 0], [1, 200], 4, 2, 64, 16, HF, "thd", 0),
    ([513] * 70, [1] * 70, 4, 1, 128, 16, BF, "thd", 0),
    ([300] * 64, [9] * 64, 6, 2, 64, 64, HF, "thd", 0),
    ([900, 900], [1, 1], 40, 1, 128, 128, BF, "thd", 0),                   # more heads a group than a tile of the few-row kernel
]


def paged_inputs(total, new, H, Hk, dh, page, dt, layout, pad, seed=0):
    g = gen(seed + sum(total) + H)
    blocks = [-(-t // page) for t in total]
    n_pages, width = sum(blocks) + 2, max(1, max(blocks)) + 1
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(total), width), 2 ** 31 - 1, dtype=torch.int32, device="cuda")
    at = 0
    for b, k in enumerate(blocks):
        table[b, :k] = order[at:at + k]
        at += k
    if layout == "htd":
        kc, vc = (randn(g, n_pages, Hk, page, dh, dtype=dt).transpose(1, 2) for _ in range(2))
    elif layout == "both":
        both = randn(g, n_pages, 2, page, Hk, dh, dtype=dt)
        kc, vc = both[:, 0], both[:, 1]
    else:
        kc, vc = randn(g, n_pages, page, Hk, dh, dtype=dt), randn(g, n_pages, page, Hk, dh, dtype=dt)
    # bits of earlier owners behind every request's last token, and in the pages that nobody holds
    for b, t in enumerate(total):
        if t % page:
            kc[table[b, t // page].long(), t % page:], vc[table[b, t // page].long(), t % page:] = math.nan, math.inf
    kc[order[at:].long()], vc[order[at:].long()] = math.nan, math.nan
    cu = starts(new)
    T = max(1, cu[-1] + pad)
    q = randn(g, T, H, dh, dtype=dt, std=1.5)
    p = F.PagedParams.make(batch=len(total), max_tokens=T, max_new=max(1, max(new)), n_heads=H, n_kv_heads=Hk, head_dim=dh, page_size=page,
                           n_pages=n_pages, max_blocks=width, dtype=dt)
    return p, q, kc, vc, table, cu


def workspace(p):
    return torch.full((F.flashloop_paged_attn_workspace_bytes(p),), 0xA5, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("total,new,H,Hk,dh,page,dt,layout,pad", PAGED)
@pytest.mark.parametrize("padded", [False, True])
def test_paged_attention(total, new, H, Hk, dh, page, dt, layout, pad, padded):
    p, q, kc, vc, table, cu = paged_inputs(total, new, H, Hk, dh, page, dt, layout, pad + (wide(H) if padded else 0))
    if padded:
        p.max_new = max(p.max_new, 33)
    o, lse, err, ws = torch.full_like(q, 7.0), torch.full((H, q.shape[0]), 7.0, device="cuda"), ints([0]), workspace(p)
    F.flashloop_paged_attn(p, q, kc, vc, table, ints(total), ints(cu), o, lse, ws, err)
    refs = [attention(q[cu[b]:cu[b + 1]], gather(kc, table[b], t), gather(vc, table[b], t), t - new[b], dh ** -0.5) for b, t in enumerate(total)]
    check(o, lse, cu, refs, True)
    assert err.item() == 0
    o2 = torch.full_like(q, 7.0)
    F.flashloop_paged_attn(p, q, kc, vc, table, ints(total), ints(cu), o2, None, ws, err)
    assert torch.equal(o2, o)


def test_paged_attention_equals_prompt_attention():
    """A whole prompt as one chunk over an empty cache is the prompt's own attention."""
    p, q, kc, vc, table, cu = paged_inputs([700, 130], [700, 130], 8, 2, 128, 64, BF, "thd", 0)
    k = torch.cat([gather(kc, table[b], t) for b, t in enumerate((700, 130))])
    v = torch.cat([gather(vc, table[b], t) for b, t in enumerate((700, 130))])
    a, b, err = torch.empty_like(q), torch.empty_like(q), ints([0])
    F.flashloop_paged_attn(p, q, kc, vc, table, ints([700, 130]), ints(cu), a, None, workspace(p), err)
    F.flashloop_prompt_attn(p, q, k, v, ints(cu), b, None, err)
    r = attention(q[:700], k[:700], v[:700], 0, 128 ** -0.5)
    assert ((a[:700].double() - r[0]).abs() <= r[2]).all() and ((a.double() - b.double()).abs()[:700] <= 2 * r[2]).all()


@pytest.mark.parametrize("new,padded", [(1, 0), (200, 0), (200, 1)])
def test_paged_attention_reports_bad_pages_and_lengths(new, padded):
    total = [900, 700, 800]
    p, q, kc, vc, table, cu = paged_inputs(total, [new] * 3, 4, 2, 128, 16, BF, "thd", padded * wide(4))
    table[1, 3], table[2, 5] = p.n_pages, -1
    o, err, ws = torch.full_like(q, 7.0), ints([0]), workspace(p)
    F.flashloop_paged_attn(p, q, kc, vc, table, ints(total), ints(cu), o, None, ws, err)
    assert err.item() == 2
    r = attention(q[:new], gather(kc, table[0], 900), gather(vc, table[0], 900), 900 - new, 128 ** -0.5)
    assert ((o[:new].double() - r[0]).abs() <= r[2]).all()
    # the bad page's keys and values count as zero
    k, v = kc.clone(), vc.clone()
    tab = table.clone()
    tab[1, 3] = table[0, 0]
    kk, vv = gather(k, tab[1], 700), gather(v, tab[1], 700)
    kk[48:64], vv[48:64] = 0, 0
    r = attention(q[new:2 * new], kk, vv, 700 - new, 128 ** -0.5)
    assert ((o[new:2 * new].double() - r[0]).abs() <= r[2]).all()
    # a length beyond the table, starts that descend and a negative length skip their requests only
    table[1, 3], table[2, 5] = 0, 0
    for lens, c in (([900, table.shape[1] * 16 + 1, 800], cu), ([900, -1, 800], cu), ([900, 700, 800], [0, new, new - 1, 3 * new])):
        o, err = torch.full_like(q, 7.0), ints([0])
        F.flashloop_paged_attn(p, q, kc, vc, table, ints(lens), ints(c), o, None, ws, err)
        assert err.item() == 2 and (o[:new] != 7).any() and not (o[:new] == 7).all(2).any()
        assert c is not cu or (o[new:2 * new] == 7).all()


# ------------------------------------------------------------------------------- many shapes
def random_paged(seed):
    rng = random.Random(seed)
    Hk, G = rng.choice((1, 2, 3, 8)), rng.choice((1, 2, 3, 4, 5, 8, 16, 33))
    dh, page = rng.choice((64, 128)), rng.choice((16, 32, 64, 128, 256))
    B = rng.choice((1, 2, 5, 33, 70, 140))
    big = max(1, 6000 // (B * G * Hk))
    new = [rng.choice((0, 1, 1, 1, rng.randint(1, 4), rng.randint(1, 60 if B > 5 else 600))) for _ in range(B)]
    new = [min(n, big * 8) for n in new]
    total = [max(0, n + rng.choice((0, 0, rng.randint(0, 300), rng.randint(0, 3000 if B < 40 else 400), -rng.randint(0, 3)))) for n in new]
    return total, new, Hk * G, Hk, dh, page, rng.choice((BF, HF)), rng.choice(("thd", "htd", "both")), rng.choice((0, 3))


@pytest.mark.parametrize("seed", range(60))
def test_paged_attention_over_random_batches(seed):
    total, new, H, Hk, dh, page, dt, layout, pad = random_paged(seed)
    p, q, kc, vc, table, cu = paged_inputs(total, new, H, Hk, dh, page, dt, layout, pad + (wide(H) if seed % 2 else 0), seed)
    if seed % 2:
        p.max_new = max(p.max_new, 33)
    o, lse, err, ws = torch.full_like(q, 7.0), torch.full((H, q.shape[0]), 7.0, device="cuda"), ints([0]), workspace(p)
    F.flashloop_paged_attn(p, q, kc, vc, table, ints(total), ints(cu), o, lse, ws, err)
    refs = [attention(q[cu[b]:cu[b + 1]], gather(kc, table[b], t), gather(vc, table[b], t), t - new[b], dh ** -0.5) for b, t in enumerate(total)]
    check(o, lse, cu, refs, True)
    assert err.item() == 0


@pytest.mark.parametrize("seed", range(30))
def test_prompt_attention_over_random_batches(seed):
    rng = random.Random(1000 + seed)
    Hk, G, dh, dt = rng.choice((1, 2, 5)), rng.choice((1, 2, 3, 7, 8)), rng.choice((64, 128)), rng.choice((BF, HF))
    B = rng.choice((1, 3, 40, 130))
    lens = [rng.choice((0, 1, rng.randint(1, 100), rng.randint(1, 1500 if B < 4 else 300))) for _ in range(B)]
    g, cu, H = gen(seed), starts(lens), Hk * G
    T = max(1, cu[-1] + rng.choice((0, 9)) + (wide(H) if seed % 2 else 0))
    q, k, v = randn(g, T, H, dh, dtype=dt, std=2.0), randn(g, T, Hk, dh, dtype=dt), randn(g, T, Hk, dh, dtype=dt)
    o, lse, err = torch.full_like(q, 7.0), torch.full((H, T), 7.0, device="cuda"), ints([0])
    p = F.PagedParams.make(batch=B, max_tokens=T, max_new=max(1, max(lens)), n_heads=H, n_kv_heads=Hk, head_dim=dh, dtype=dt, scale=0.3)
    F.flashloop_prompt_attn(p, q, k, v, ints(cu), o, lse, err)
    check(o, lse, cu, [attention(q[a:b], k[a:b], v[a:b], 0, 0.3) for a, b in zip(cu, cu[1:])], True)
    assert err.item() == 0


def test_peaked_and_shifted_scores():
    """Scores hundreds apart, rising along the columns (the running reference is raised again and again), and far from zero."""
    g, n, dh = gen(9), 700, 128
    for rise in (1.0, -1.0):
        for T in (n, n + wide(2)):  # few-row and tile kernel
            q = torch.ones(T, 2, dh, device="cuda").to(BF)
            k = (torch.arange(T, device="cuda")[:, None, None] * rise * 0.05 + randn(g, T, 1, dh)).to(BF)
            v = randn(g, T, 1, dh, dtype=BF)
            p = F.PagedParams.make(batch=1, max_tokens=T, max_new=n, n_heads=2, n_kv_heads=1, head_dim=dh)
            o, lse, err = torch.full((T, 2, dh), 7.0, dtype=BF, device="cuda"), torch.full((2, T), 7.0, device="cuda"), ints([0])
            F.flashloop_prompt_attn(p, q, k, v, ints([0, n]), o, lse, err)
            check(o, lse, [0, n], [attention(q[:n], k[:n], v[:n], 0, dh ** -0.5)], True)


def test_equal_keys_average_the_values():
    n, dh = 300, 64
    q, k = torch.ones(n, 1, dh, dtype=HF, device="cuda"), torch.ones(n, 1, dh, dtype=HF, device="cuda")
    v = torch.full((n, 1, dh), 0.5, dtype=HF, device="cuda")
    p = F.PagedParams.make(batch=1, max_tokens=n, max_new=n, n_heads=1, n_kv_heads=1, head_dim=dh, dtype=HF)
    o, lse = torch.empty_like(q), torch.empty(1, n, device="cuda")
    F.flashloop_prompt_attn(p, q, k, v, ints([0, n]), o, lse, ints([0]))
    assert (o == 0.5).all()
    want = math.sqrt(dh) + torch.log(torch.arange(1, n + 1, device="cuda", dtype=torch.float64))
    assert ((lse[0].double() - want).abs() <= 2.0 ** -20 * want).all()


# ------------------------------------------------------------------------------- layouts, streams, graphs
def test_broadcast_keys_and_odd_alignment():
    """Key heads that are one head expanded, rows of o on 16 bytes only, queries transposed."""
    g, T, H, dh = gen(3), 260, 4, 128
    k1, v1 = randn(g, T, 1, dh, dtype=BF), randn(g, T, 1, dh, dtype=BF)
    k, v = k1.expand(T, 2, dh), v1.expand(T, 2, dh)
    q = randn(g, H, T, dh, dtype=BF).transpose(0, 1)
    wide = torch.full((T, H, dh + 8), 7.0, dtype=BF, device="cuda")
    o, err = wide[:, :, 8:], ints([0])
    p = F.PagedParams.make(batch=1, max_tokens=T, max_new=T, n_heads=H, n_kv_heads=2, head_dim=dh)
    F.flashloop_prompt_attn(p, q, k, v, ints([0, T]), o, None, err)
    ref = attention(q, k, v, 0, dh ** -0.5)
    assert ((o.double() - ref[0]).abs() <= ref[2]).all() and (wide[:, :, :8] == 7).all()
    o2 = torch.full((T, H, dh + 8), 7.0, dtype=BF, device="cuda")
    F.flashloop_prompt_attn(p, q, k.contiguous(), v.contiguous(), ints([0, T]), o2[:, :, 8:], None, err)
    assert ((o2[:, :, 8:].double() - ref[0]).abs() <= ref[2]).all() and (o2[:, :, :8] == 7).all()
    for new in (1, T):  # over a cache whose pages are one page expanded
        kc = k1[:64].view(1, 64, 1, dh).expand(4, 64, 2, dh)
        vc = v1[:64].view(1, 64, 1, dh).expand(4, 64, 2, dh)
        pp = F.PagedParams.make(batch=1, max_tokens=new, max_new=new, n_heads=H, n_kv_heads=2, head_dim=dh, page_size=64, n_pages=4, max_blocks=5)
        oo, table = torch.empty(new, H, dh, dtype=BF, device="cuda"), ints([[3, 1, 2, 0, 0]])
        F.flashloop_paged_attn(pp, q[:new], kc, vc, table, ints([T]), ints([0, new]), oo, None, workspace(pp), err)
        ref = attention(q[:new], gather(kc, table[0], T), gather(vc, table[0], T), T - new, dh ** -0.5)
        assert ((oo.double() - ref[0]).abs() <= ref[2]).all()
    assert err.item() == 0


def test_offsets_beyond_32_bits():
    """A pool of more than 2^31 elements a cache; the requests' pages lie at both ends."""
    page, Hk, dh, H = 64, 4, 128, 8
    n_pages = (1 << 31) // (page * Hk * dh) + 900
    kc = torch.empty(n_pages, page, Hk, dh, dtype=BF, device="cuda")
    vc = torch.empty(n_pages, page, Hk, dh, dtype=BF, device="cuda")
    table = ints([list(range(n_pages - 12, n_pages)), list(range(12))])
    g, total = gen(4), [750, 700]
    slots = torch.cat([table[b].long()[torch.arange(t, device="cuda") // page] * page + torch.arange(t, device="cuda") % page for b, t in enumerate(total)])
    k, v = randn(g, sum(total), Hk, dh, dtype=BF), randn(g, sum(total), Hk, dh, dtype=BF)
    err = ints([0])
    p = F.PagedParams.make(batch=2, max_tokens=sum(total), max_new=750, n_heads=H, n_kv_heads=Hk, head_dim=dh, page_size=page, n_pages=n_pages, max_blocks=12)
    F.flashloop_paged_kv_write(p, k, v, slots.to(torch.int32), kc, vc, err)
    assert torch.equal(gather(kc, table[0], 750), k[:750]) and torch.equal(gather(vc, table[1], 700), v[750:])
    for new in ([1, 1], [300, 50]):
        cu = starts(new)
        p = F.PagedParams.make(batch=2, max_tokens=cu[-1], max_new=max(new), n_heads=H, n_kv_heads=Hk, head_dim=dh, page_size=page, n_pages=n_pages, max_blocks=12)
        q = randn(g, cu[-1], H, dh, dtype=BF)
        o = torch.empty_like(q)
        F.flashloop_paged_attn(p, q, kc, vc, table, ints(total), ints(cu), o, None, workspace(p), err)
        for b, (a, z) in enumerate(((0, 750), (750, 1450))):
            ref = attention(q[cu[b]:cu[b + 1]], k[a:z], v[a:z], total[b] - new[b], dh ** -0.5)
            assert ((o[cu[b]:cu[b + 1]].double() - ref[0]).abs() <= ref[2]).all()
    assert err.item() == 0


def test_two_streams_at_once_and_a_shared_workspace_in_turn():
    a = paged_inputs([3000, 900, 70], [1, 200, 9], 8, 2, 128, 64, BF, "thd", wide(8), seed=1)
    b = paged_inputs([12000, 40, 5000], [1, 1, 1], 16, 2, 64, 16, HF, "thd", 0, seed=2)
    lens = (ints([3000, 900, 70]), ints([12000, 40, 5000]))
    ws = [workspace(a[0]), workspace(b[0])]
    both = torch.empty(max(w.numel() for w in ws), dtype=torch.uint8, device="cuda")
    err = ints([0])

    def run(x, kv, w, o):
        p, q, kc, vc, table, cu = x
        F.flashloop_paged_attn(p, q, kc, vc, table, kv, ints(cu) if not isinstance(cu, torch.Tensor) else cu, o, None, w, err)

    a, b = a[:5] + (ints(a[5]),), b[:5] + (ints(b[5]),)
    want = [torch.zeros_like(a[1]), torch.zeros_like(b[1])]
    run(a, lens[0], ws[0], want[0])
    run(b, lens[1], ws[1], want[1])
    torch.cuda.synchronize()
    got = [torch.zeros_like(a[1]), torch.zeros_like(b[1])]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):  # two calls at once, each with a workspace of its own
        for s, x, kv, w, o in zip(streams, (a, b), lens, ws, got):
            with torch.cuda.stream(s):
                run(x, kv, w, o)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # two captured graphs that share a workspace, replayed in turn
    graphs = []
    for x, kv, o in zip((a, b), lens, got):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run(x, kv, both, o)
        graphs.append(g)
    for o in got:
        o.zero_()
    both.fill_(0xFF)
    for i in range(6):
        graphs[i % 2].replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and err.item() == 0


class Served:
    """Requests served from one pool: plan, write, attention, as a captured step or eagerly."""

    def __init__(self, B, T, max_new, H, Hk, dh, page, n_pages, width, dt=BF):
        self.p = F.PagedParams.make(batch=B, max_tokens=T, max_new=max_new, n_heads=H, n_kv_heads=Hk, head_dim=dh, page_size=page, n_pages=n_pages,
                                    max_blocks=width, dtype=dt)
        self.kv, self.kv_out, self.new = ints([0] * B), ints([0] * B), ints([0] * B)
        self.free, self.n_free, self.n_out = ints(list(range(n_pages))), ints([n_pages]), ints([0])
        self.table, self.cu = torch.full((B, width), -1, dtype=torch.int32, device="cuda"), ints([0] * (B + 1))
        self.slots, self.pos, self.err = ints([0] * T), ints([0] * T), ints([0])
        self.kc, self.vc = (torch.full((n_pages, page, Hk, dh), math.nan, dtype=dt, device="cuda") for _ in range(2))
        self.q, self.k, self.v = (torch.zeros(T, h, dh, dtype=t, device="cuda") for h, t in ((H, dt), (Hk, torch.float32), (Hk, torch.float32)))
        self.o, self.ws = torch.zeros(T, H, dh, dtype=dt, device="cuda"), workspace(self.p)

    def step(self):
        F.flashloop_paged_plan(self.p, self.kv, self.new, self.free, self.n_free, self.table, self.cu, self.kv_out, self.slots, self.pos, self.n_out, self.err)
        F.flashloop_paged_kv_write(self.p, self.k, self.v, self.slots, self.kc, self.vc, self.err)
        F.flashloop_paged_attn(self.p, self.q, self.kc, self.vc, self.table, self.kv_out, self.cu, self.o, None, self.ws, self.err)
        self.kv.copy_(self.kv_out)
        self.n_free.copy_(self.n_out)


@pytest.mark.parametrize("captured,T", [(False, 320), (True, 320), (True, 7500)])  # the last one's bounds: tile kernel
def test_serving_steps_of_changing_lengths(captured, T):
    """Chunks, then single tokens, requests joining late: each step's rows attend to all that was written before."""
    H, Hk, dh, page = 8, 2, 64, 16
    s = Served(B=4, T=T, max_new=200, H=H, Hk=Hk, dh=dh, page=page, n_pages=96, width=32)
    g, hist = gen(11), [[[], []] for _ in range(4)]
    if captured:
        s.step()  # no new tokens
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            s.step()
    for new in ([100, 0, 33, 0], [100, 7, 1, 0], [1, 1, 1, 200], [1, 0, 1, 100], [1, 1, 1, 1], [1, 1, 1, 1], [0, 0, 0, 0], [16, 200, 16, 1]):
        n = sum(new)
        s.new.copy_(ints(new))
        s.q.copy_(randn(g, T, H, dh, dtype=BF))
        s.k.copy_(randn(g, T, Hk, dh))
        s.v.copy_(randn(g, T, Hk, dh))
        s.o.fill_(7.0)
        graph.replay() if captured else s.step()
        cu = starts(new)
        assert s.cu.tolist() == cu and s.err.item() == 0 and (s.o[n:] == 7).all()
        for b in range(4):
            r = slice(cu[b], cu[b + 1])
            hist[b][0].append(s.k[r].to(BF).clone())
            hist[b][1].append(s.v[r].to(BF).clone())
            k, v = torch.cat(hist[b][0]), torch.cat(hist[b][1])
            assert s.kv[b].item() == k.shape[0] and s.pos[r].tolist() == list(range(k.shape[0] - new[b], k.shape[0]))
            o, _, tol, _ = attention(s.q[r], k, v, k.shape[0] - new[b], dh ** -0.5)
            assert ((s.o[r].double() - o).abs() <= tol).all()
    held = {x for b in range(4) for x in s.table[b, :-(-s.kv[b].item() // page)].tolist()}
    assert len(held) == sum(-(-n // page) for n in s.kv.tolist()) and s.n_free.item() == 96 - len(held)
    assert not held & set(s.free[:s.n_free.item()].tolist())


def test_with_the_projections_of_the_sublayer():
    """Projection with RoPE at the planned positions, cache write, attention and output projection,
    for two requests in two chunks each and then a token each."""
    from workload import CONFIGS, make_weights
    from gpu_helpers import bf16_to_torch
    cfg = CONFIGS["tiny"]
    d, H, dh = cfg.d_model, cfg.n_heads, cfg.head_dim
    W = make_weights(cfg)
    wqkv, wo = bf16_to_torch(W["wqkv"]), bf16_to_torch(W["wo"])
    params = F.Params.from_config(cfg)
    rope = torch.zeros(256, dh // 2, 2, device="cuda")
    F.flashloop_rope_table(params, 256, rope)
    s = Served(B=2, T=256, max_new=120, H=H, Hk=H, dh=dh, page=32, n_pages=16, width=8)
    g = gen(21)
    x = [randn(g, n, d, dtype=BF) for n in (200, 90)]
    y, done = [[], []], [0, 0]
    for new in ([120, 50], [79, 39], [1, 1]):
        n = sum(new)
        rows = torch.zeros(256, d, dtype=BF, device="cuda")
        rows[:n] = torch.cat([x[b][done[b]:done[b] + new[b]] for b in range(2)])
        s.new.copy_(ints(new))
        F.flashloop_paged_plan(s.p, s.kv, s.new, s.free, s.n_free, s.table, s.cu, s.kv_out, s.slots, s.pos, s.n_out, s.err)
        cs = rope[s.pos.long()].contiguous()
        F.flashloop_qkv_gathered(params, rows, None, None, 256, wqkv, cs, s.q.view(256, d), s.k.view(256, d), s.v.view(256, d))
        F.flashloop_paged_kv_write(s.p, s.k, s.v, s.slots, s.kc, s.vc, s.err)
        F.flashloop_paged_attn(s.p, s.q, s.kc, s.vc, s.table, s.kv_out, s.cu, s.o, None, s.ws, s.err)
        out = torch.zeros(256, d, dtype=BF, device="cuda")
        F.flashloop_out_proj(params, s.o.view(256, d), None, None, 256, wo, out)
        for b, (a, z) in enumerate(((0, new[0]), (new[0], n))):
            y[b].append(out[a:z].clone())
            done[b] += new[b]
        s.kv.copy_(s.kv_out)
        s.n_free.copy_(s.n_out)
    assert s.err.item() == 0
    w = wqkv.double()
    ang = torch.arange(200, device="cuda", dtype=torch.float64)[:, None] * cfg.rope_theta ** (-torch.arange(dh // 2, device="cuda", dtype=torch.float64) * 2 / dh)
    cos, sin = torch.cos(ang)[:, None], torch.sin(ang)[:, None]
    for b, n in enumerate((200, 90)):
        q, k, v = (x[b].double() @ w.T).view(n, 3, H, dh).unbind(1)

        def turn(t):
            lo, hi = t[..., :dh // 2], t[..., dh // 2:]
            return torch.cat([lo * cos[:n] - hi * sin[:n], hi * cos[:n] + lo * sin[:n]], -1)
        q, k = turn(q), turn(k)
        a = torch.einsum("ihd,jhd->hij", q, k) / math.sqrt(dh)
        a = a.masked_fill(torch.ones(n, n, device="cuda", dtype=torch.bool).triu(1), -math.inf).softmax(-1)
        want = torch.einsum("hij,jhd->ihd", a, v).reshape(n, d) @ wo.double().T
        got = torch.cat(y[b]).double()
        # the sublayer's own bar: 1e-2 of a row's norm (q, K, V, P, O and Y are rounded to bf16)
        assert (((got - want).norm(dim=1) / want.norm(dim=1)) < 1e-2).all()


# ------------------------------------------------------------------------------- refusals on the device
def test_binding_refusals():
    g = gen(0)
    p = F.PagedParams.make(batch=1, max_tokens=8, max_new=8, n_heads=2, n_kv_heads=1, head_dim=64, page_size=16, n_pages=2, max_blocks=2)
    q, k = randn(g, 8, 2, 64, dtype=BF), randn(g, 8, 1, 64, dtype=BF)
    o, cu, err, ws = torch.full_like(q, 7.0), ints([0, 8]), ints([0]), workspace(p)
    kc = torch.zeros(2, 16, 1, 64, dtype=BF, device="cuda")
    table, kv = ints([[0, 1]]), ints([8])
    odd = torch.zeros(8 * 2 * 64 + 4, dtype=BF, device="cuda")[4:].view(8, 2, 64)
    prompt = lambda **a: F.flashloop_prompt_attn(**{**dict(params=p, q=q, k=k, v=k, cu=cu, o=o, lse=None, err_word=err), **a})  # noqa: E731
    paged = lambda **a: F.flashloop_paged_attn(**{**dict(params=p, q=q, k_cache=kc, v_cache=kc, block_table=table, kv_lens=kv, cu=cu, o=o, lse=None,  # noqa: E731
                                                          workspace=ws, err_word=err), **a})
    write = lambda **a: F.flashloop_paged_kv_write(**{**dict(params=p, k=k, v=k, slot_map=ints([0] * 8), k_cache=kc, v_cache=kc, err_word=err), **a})  # noqa: E731
    bad = [
        (prompt, dict(q=q.to(HF)), -1), (prompt, dict(q=q[:7]), -1), (prompt, dict(q=q.cpu()), -1), (prompt, dict(k=k.float()), -1), (prompt, dict(q=odd), -1),
        (prompt, dict(o=odd), -1), (prompt, dict(q=q.transpose(1, 2).contiguous().transpose(1, 2)), -1), (prompt, dict(cu=cu.long()), -1), (prompt, dict(cu=cu[:1]), -1),
        (prompt, dict(o=o[:1].expand(8, 2, 64)), -1), (prompt, dict(lse=torch.zeros(15, device="cuda")), -1), (prompt, dict(err_word=ints([0]).cpu()), -1),
        (paged, dict(block_table=table[:, :1]), -1), (paged, dict(workspace=ws[:8]), -1), (paged, dict(workspace=torch.empty(64, dtype=torch.uint8, device="cuda")[8:]), -1),
        (paged, dict(k_cache=kc[:1]), -1), (paged, dict(kv_lens=kv.cpu()), -1), (paged, dict(workspace=ws.cpu()), -1),
        (write, dict(k=k.to(HF), v=k.to(HF)), -2), (write, dict(v=k.float()), -1), (write, dict(k_cache=kc[:1].expand(2, 16, 1, 64)), -1),
        (write, dict(k=k.double(), v=k.double()), -2),
    ]
    for call, args, status in bad:
        with pytest.raises(F.FlashLoopError) as e:
            call(**args)
        assert e.value.status == status, args.keys()
    for field, value, status in (("head_dim", 96, -1), ("n_kv_heads", 3, -1), ("dtype", 2, -2), ("dtype", 7, -2)):
        bad = F.PagedParams.from_buffer_copy(p)
        setattr(bad, field, value)
        with pytest.raises(F.FlashLoopError) as e:
            prompt(params=bad)
        assert e.value.status == status
    assert (o == 7).all() and err.item() == 0


SMALL = [  # cached lengths, new tokens, H, Hk, dh, type: up to 16 packed rows a request and key head
    ([1, 77, 400], [1, 1, 1], 1, 1, 64, BF), ([3000, 5, 64], [1, 1, 1], 8, 1, 128, BF), ([5000, 9], [2, 1], 8, 2, 128, HF), ([2100, 65], [1, 1], 12, 1, 64, HF),
    ([4096, 300], [4, 3], 8, 2, 128, BF), ([450, 16], [2, 2], 7, 1, 64, BF), ([900] * 40, [1] * 40, 16, 1, 128, HF), ([700, 3000], [1, 16], 4, 4, 128, BF),
]


@pytest.mark.parametrize("total,new,H,Hk,dh,dt", SMALL)
def test_few_rows_keep_what_the_rounding_of_p_drops(total, new, H, Hk, dh, dt):
    p, q, kc, vc, table, cu = paged_inputs(total, new, H, Hk, dh, 16, dt, "thd", 0)
    o, err = torch.full_like(q, 7.0), ints([0])
    F.flashloop_paged_attn(p, q, kc, vc, table, ints(total), ints(cu), o, None, workspace(p), err)
    refs = [attention(q[cu[b]:cu[b + 1]], gather(kc, table[b], t), gather(vc, table[b], t), t - new[b], dh ** -0.5, 2) for b, t in enumerate(total)]
    check(o, None, cu, refs, False)


@pytest.mark.parametrize("G,dt", [(4, BF), (8, HF), (12, BF), (16, HF), (24, BF)])
@pytest.mark.parametrize("L", [40, 2000])
def test_infinite_values_stay_infinite(G, dt, L):
    """Seen by every row: an infinity of V is the result's, one of either sign none's."""
    p, q, kc, vc, table, cu = paged_inputs([L], [1], G, 1, 64, 16, dt, "thd", 0)
    vc[table[0, 1].long(), 3, 0, :2], vc[table[0, 0].long(), 9, 0, 1] = math.inf, -math.inf
    vc[table[0, 0].long(), 0, 0, 2] = math.nan
    o = torch.zeros_like(q)
    F.flashloop_paged_attn(p, q, kc, vc, table, ints([L]), ints(cu), o, None, workspace(p), ints([0]))
    assert (o[..., 0] == math.inf).all() and o[..., 1:3].isnan().all() and o[..., 3:].isfinite().all()


@pytest.mark.parametrize("mode", ["eager", "captured", "streams"])
@pytest.mark.parametrize("n", [2, 300])  # few-row kernel, tile kernel
def test_calls_back_to_back_see_each_other(mode, n):
    """Each call reads what the one before it wrote, and writes what the one before it read; nothing waits on the host.
    The same bits as with a wait after every call."""
    B, H, Hk, dh, page, steps = 3, 8, 2, 64, 16, 12
    width = steps * n // page + 2
    p = F.PagedParams.make(batch=B, max_tokens=B * n, max_new=n, n_heads=H, n_kv_heads=Hk, head_dim=dh, page_size=page, n_pages=B * width, max_blocks=width)
    q0 = randn(gen(3), B * n, H, dh, dtype=BF)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]

    def run(mode):
        q, o, ws, err = q0.clone(), torch.zeros_like(q0), workspace(p), ints([0])
        kv, new, free, left = [ints([0] * B), ints([0] * B)], ints([n] * B), ints(list(range(B * width))), [ints([B * width]), ints([0])]
        table, cu, slots, pos = torch.full((B, width), -1, dtype=torch.int32, device="cuda"), ints([0] * (B + 1)), ints([0] * B * n), ints([0] * B * n)
        kc, vc = (torch.full((B * width, page, Hk, dh), math.nan, dtype=BF, device="cuda") for _ in range(2))
        torch.cuda.synchronize()

        def calls():
            for i in range(steps):
                a, b = i % 2, (i + 1) % 2
                yield lambda: F.flashloop_paged_plan(p, kv[a], new, free, left[a], table, cu, kv[b], slots, pos, left[b], err)
                yield lambda: F.flashloop_paged_kv_write(p, q[:, :Hk], q[:, Hk:2 * Hk], slots, kc, vc, err)
                yield lambda: F.flashloop_paged_attn(p, q, kc, vc, table, kv[b], cu, o, None, ws, err)
                yield lambda: F.flashloop_prompt_attn(p, o, o[:, 2:4], q[:, 4:6], cu, q, None, err) if i % 3 == 2 else q.copy_(o)
                yield lambda: F.flashloop_prompt_attn(p, q, o[:, 2:4], o[:, 4:6], cu, q, None, err)

        if mode == "captured":
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                for call in calls():
                    call()
            graph.replay()
        else:
            for i, call in enumerate(calls()):
                if mode == "streams":
                    here, there = streams[i % 2], streams[(i + 1) % 2]
                    here.wait_stream(there)
                    with torch.cuda.stream(here):
                        call()
                else:
                    call()
                if mode == "waits":
                    torch.cuda.synchronize()
        torch.cuda.synchronize()
        assert err.item() == 0
        return q, o, kc[free.new_tensor(table[:, :steps * n // page].flatten().tolist()).long()]

    want = run("waits")
    assert want[0].isfinite().all() and want[0].abs().sum() > 0
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(run(mode), want))


@pytest.mark.parametrize("lens,H,Hk,dh,dt", [([100] * 4, 4, 4, 128, BF), ([17], 4, 4, 64, HF), ([33, 1, 80], 6, 2, 64, BF), ([300, 41], 4, 1, 128, HF), ([1024], 2, 2, 64, BF)])
def test_small_prompts_in_tiles_of_16_rows(lens, H, Hk, dh, dt):
    """At most a tile an SM: every tile of every request, whose probabilities keep what their rounding drops."""
    g, cu = gen(sum(lens)), starts(lens)
    q, k, v = randn(g, cu[-1], H, dh, dtype=dt, std=1.5), randn(g, cu[-1], Hk, dh, dtype=dt), randn(g, cu[-1], Hk, dh, dtype=dt)
    p = F.PagedParams.make(batch=len(lens), max_tokens=cu[-1], max_new=max(lens), n_heads=H, n_kv_heads=Hk, head_dim=dh, dtype=dt)
    assert cu[-1] * H // 16 + len(lens) * Hk // 2 <= 148
    o, lse, err = torch.full_like(q, 7.0), torch.full((H, cu[-1]), 7.0, device="cuda"), ints([0])
    F.flashloop_prompt_attn(p, q, k, v, ints(cu), o, lse, err)
    check(o, lse, cu, [attention(q[a:b], k[a:b], v[a:b], 0, dh ** -0.5, 2) for a, b in zip(cu, cu[1:])], True)
    assert err.item() == 0


def test_both_ways_into_the_library(monkeypatch):
    """The C++ marshalling takes plain calls, and gives what the Python one does; that refuses the same calls."""
    s = [Served(B=2, T=24, max_new=16, H=4, Hk=2, dh=64, page=16, n_pages=12, width=4) for _ in range(2)]
    g = gen(21)
    x = [randn(g, 24, h, 64) for h in (4, 2, 2)]
    for c in s:
        c.new.copy_(ints([16, 5]))
        for to, a in zip((c.q, c.k, c.v), x):
            to.copy_(a)

    def calls(c):
        o = torch.full_like(c.q, 7.0)
        yield "plan", (c.p, c.kv, c.new, c.free, c.n_free, c.table, c.cu, c.kv_out, c.slots, c.pos, c.n_out, c.err)
        yield "write", (c.p, c.k, c.v, c.slots, c.kc, c.vc, c.err)
        yield "attn", (c.p, c.q, c.kc, c.vc, c.table, c.kv_out, c.cu, c.o, None, c.ws, c.err)
        yield "prompt", (c.p, c.q, c.k.to(BF), c.v.to(BF), c.cu, o, None, c.err)
        c.o2 = o

    public = dict(plan=F.flashloop_paged_plan, write=F.flashloop_paged_kv_write, attn=F.flashloop_paged_attn, prompt=F.flashloop_prompt_attn)
    for name, args in calls(s[0]):
        assert getattr(F._fastcall, name)(*args, None) == 0
    here = torch.cuda.current_stream()
    for name, args in calls(s[1]):
        assert getattr(F._fastcall, name)(*args, here) is None  # a stream object: the Python path's
        assert getattr(F._fastcall, name)(*args[:-1], args[-1].cpu(), None) is None
        assert public[name](*args, stream=here) == 0
    for a, b in ((s[0].o, s[1].o), (s[0].o2, s[1].o2), (s[0].table, s[1].table), (s[0].slots, s[1].slots), (s[0].kv_out, s[1].kv_out), (s[0].n_out, s[1].n_out)):
        assert torch.equal(a, b)
    assert torch.equal(torch.nan_to_num(s[0].kc), torch.nan_to_num(s[1].kc)) and s[0].err.item() == s[1].err.item() == 0
    monkeypatch.setattr(F, "_fastcall", type("Without", (), {n: staticmethod(lambda *a: None) for n in public}))
    test_binding_refusals()


@pytest.mark.parametrize("width,most", [(2, 1), (40, 1), (40, 90)])  # few-row kernel whole and cut, tile kernel
def test_the_largest_batch(width, most):
    B, H, Hk, dh, page = 65535, 4, 1, 64, 16
    rng = np.random.default_rng(most * width)
    new = rng.integers(0, 2, B)
    if most > 1:
        new[rng.integers(0, B, 40)] = most
    total = new + rng.integers(0, page * 2 - 1 if width == 2 else 60, B) if most == 1 else np.maximum(new, rng.integers(0, 100, B))
    total = np.minimum(total, page * width)
    cu = np.concatenate([[0], np.cumsum(new)])
    T, n_pages = int(cu[-1]), 5000
    g = gen(width)
    table = torch.randint(0, n_pages, (B, width), generator=g, device="cuda", dtype=torch.int32)  # pages shared at random
    kc, vc, q = randn(g, n_pages, page, Hk, dh, dtype=BF), randn(g, n_pages, page, Hk, dh, dtype=BF), randn(g, T, H, dh, dtype=BF)
    p = F.PagedParams.make(batch=B, max_tokens=T, max_new=most, n_heads=H, n_kv_heads=Hk, head_dim=dh, page_size=page, n_pages=n_pages, max_blocks=width)
    o, err = torch.full_like(q, 7.0), ints([0])
    F.flashloop_paged_attn(p, q, kc, vc, table, ints(total.tolist()), ints(cu.tolist()), o, None, workspace(p), err)
    assert err.item() == 0 and not (o == 7.0).all(-1).any()
    for b in [0, 1, B - 2, B - 1] + rng.integers(0, B, 40).tolist() + np.argsort(new)[-10:].tolist():
        t, n, r = int(total[b]), int(new[b]), slice(int(cu[b]), int(cu[b + 1]))
        want, _, tol, _ = attention(q[r], gather(kc, table[b], t), gather(vc, table[b], t), t - n, dh ** -0.5)
        assert ((o[r].double() - want).abs() <= tol).all(), b
