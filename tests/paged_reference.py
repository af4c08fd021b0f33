"""Plain 64-bit implementations of the many-request operators, and how far the
kernels may be from them."""
import math

import torch


def build_plan(held, new, table, stack, page):
    """(cu, kv, table, slots, positions, pages left) by the definition, token by token."""
    table, stack = [list(r) for r in table], list(stack)
    cu, kv, slots, pos = [0], [], [], []
    for b, (h, n) in enumerate(zip(held, new)):
        for p in range(h, h + n):
            if p % page == 0:
                table[b][p // page] = stack.pop()
            slots.append(table[b][p // page] * page + p % page)
            pos.append(p)
        cu.append(cu[-1] + n)
        kv.append(h + n)
    return cu, kv, table, slots, pos, len(stack)


def attention(q, k, v, first, scale, p_parts=1):
    """q [n, H, dh], k and v [L, Hk, dh]; row i sees the columns j <= first + i.  Returns o, lse and
    the elementwise bounds of a kernel that takes scores and sums in float32 and rounds the
    probabilities (to a sum of p_parts numbers) and the output to q's type."""
    n, H, dh = q.shape
    L, G = k.shape[0], H // k.shape[1]
    u = torch.finfo(q.dtype).eps / 2
    o = torch.zeros(n, H, dh, dtype=torch.float64, device=q.device)
    lse = torch.full((H, n), -math.inf, dtype=torch.float64, device=q.device)
    o_tol, lse_tol = torch.zeros_like(o), torch.full_like(lse, 1e-30)
    if L == 0 or n == 0:
        return o, lse, o_tol, lse_tol
    seen = torch.arange(L, device=q.device)[None] <= first + torch.arange(n, device=q.device)[:, None]
    some = seen.any(1)
    for h in range(H):
        qh, kh, vh = q[:, h].double(), k[:, h // G].double(), v[:, h // G].double()
        s = (qh @ kh.T * scale).masked_fill(~seen, -math.inf)
        l = torch.logsumexp(s, 1)
        p = torch.exp(s - torch.where(some, l, 0.0)[:, None])
        vz = torch.nan_to_num(vh, 0.0, 0.0, 0.0)
        a = p @ vz.abs()  # what the probabilities' relative errors act on
        # a float32 dot product of dh exact products is off by dh 2^-24 of their absolute sum; the scaling
        # and the subtraction of the reference (both within |s|) add three roundings
        mag = (qh.abs() @ kh.abs().T * abs(scale)).masked_fill(~seen, 0.0).amax(1)
        ds = (dh + 4) * 2.0 ** -24 * mag
        # every p is also off by the exponential's own error (2^-21 covers ex2 and the polynomial), and the
        # sums of L terms by L 2^-24; numerator and denominator both
        rel = 2 * (ds + 2.0 ** -21 + (L + 16) * 2.0 ** -24)
        o[:, h] = p @ vz
        # half a step of p and of o; fp16 also has an absolute step of 2^-25 below 2^-14 (p and o)
        flat = 2.0 ** -25 if q.dtype == torch.float16 else 0.0
        # (of two parts the second is at most half a step, and off by half a step of its own)
        o_tol[:, h] = u * 1.01 * (u ** (p_parts - 1) * a + o[:, h].abs() + rel[:, None] * a) + rel[:, None] * a \
            + flat * (1 + vz.abs().sum(0))[None] + 1e-30
        lse[h] = l
        lse_tol[h] = ds + 2.0 ** -21 + (L + 16) * 2.0 ** -24 + 4 * 2.0 ** -24 * (mag + 20)
    o[~some], o_tol[~some] = 0.0, 0.0
    return o, lse, o_tol, lse_tol


def gather(cache, table_row, length):
    """The first `length` tokens of a request out of pages [n, page, Hk, dh]."""
    page = cache.shape[1]
    j = torch.arange(length, device=cache.device)
    return cache[table_row.long()[j // page], j % page]
