"""The paged-cache and packed-prompt operators: cases, plain forms and definitions in 64 bits.

Four operators that serve many requests at once from one pool of cache pages:

plan    block tables and slot maps of the tokens that the requests append
write   new keys and values into the cache pages of their slots
prompt  causal attention over whole prompts packed end to end, grouped heads
paged   attention of new tokens (one or a chunk a request) over the paged cache

With ``own`` false, ``run`` computes them from elementary torch operations in
32 bits; with ``own`` true it calls cross_loop_sparse_b200.flashloop.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of 64 requests in flight: a page is opened only by the few that fill one
        {"name": "plan_step", "op": "plan", "seqs": 64, "held": 8192, "new": 1, "page": 16, "pad": 0, "mix": 1},
        # admission of 512 requests of ragged lengths, long prompts among them, tables padded for a captured graph
        {"name": "plan_admit", "op": "plan", "seqs": 512, "held": 0, "new": 4096, "page": 64, "pad": 1000, "mix": 2},
        # the same decode step's new keys and values, cut out of a fused projection's rows
        {"name": "write_step", "op": "write", "tokens": 64, "kv_heads": 8, "dim": 128, "src": "bf16", "cache": "bf16", "page": 16, "fused": True, "pad": 3},
        # the prompt of 32768 tokens x 16 heads from the float32 keys and values of the gathered projection
        {"name": "write_prompt", "op": "write", "tokens": 32768, "kv_heads": 16, "dim": 128, "src": "fp32", "cache": "bf16", "page": 64, "fused": False, "pad": 0},
        # a batch of short questions, the tiny configuration's heads
        {"name": "prompt_short", "op": "prompt", "seqs": 24, "shortest": 1, "longest": 300, "heads": 4, "kv_heads": 4, "dim": 64, "type": "fp16", "lse": False, "pad": 5, "mix": 3},
        # ragged prompts with four query heads a key head
        {"name": "prompt_ragged", "op": "prompt", "seqs": 9, "shortest": 77, "longest": 6001, "heads": 32, "kv_heads": 8, "dim": 128, "type": "bf16", "lse": True, "pad": 0, "mix": 4},
        # the benchmark's prompt: 32768 tokens, 16 heads
        {"name": "prompt_32k", "op": "prompt", "seqs": 1, "shortest": 32768, "longest": 32768, "heads": 16, "kv_heads": 16, "dim": 128, "type": "bf16", "lse": False, "pad": 0, "mix": 5},
        # one user at the start of an answer: latency alone
        {"name": "decode_one", "op": "paged", "seqs": 1, "shortest": 256, "longest": 256, "new": 1, "chunks": 0, "chunk": 1, "heads": 4, "kv_heads": 4, "dim": 64, "page": 16, "type": "bf16", "lse": False, "mix": 6},
        # the benchmark's decode: 8 contexts of 32768 tokens, 16 heads
        {"name": "decode_8x32k", "op": "paged", "seqs": 8, "shortest": 32768, "longest": 32768, "new": 1, "chunks": 0, "chunk": 1, "heads": 16, "kv_heads": 16, "dim": 128, "page": 64, "type": "bf16", "lse": False, "mix": 7},
        # many users with contexts of every length, grouped heads, small pages
        {"name": "decode_ragged", "op": "paged", "seqs": 96, "shortest": 1, "longest": 16384, "new": 1, "chunks": 0, "chunk": 1, "heads": 32, "kv_heads": 8, "dim": 128, "page": 16, "type": "fp16", "lse": True, "mix": 8},
        # two long prompts taken in chunks of a thousand tokens
        {"name": "chunk_long", "op": "paged", "seqs": 2, "shortest": 9001, "longest": 24001, "new": 1000, "chunks": 0, "chunk": 1, "heads": 32, "kv_heads": 8, "dim": 128, "page": 64, "type": "bf16", "lse": True, "mix": 9},
        # a step that serves decoding users and prompts' chunks together, eight query heads a key head
        {"name": "mixed_step", "op": "paged", "seqs": 34, "shortest": 50, "longest": 12000, "new": 1, "chunks": 2, "chunk": 1500, "heads": 16, "kv_heads": 2, "dim": 128, "page": 32, "type": "bf16", "lse": False, "mix": 10},
    ]


def _log(rng, lo, hi):
    """An integer of [lo, hi], spread evenly over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(("plan", "write", "prompt", "paged", "prompt", "paged"))
    mix = rng.randrange(1 << 30)
    if op == "plan":
        step = rng.random() < 0.5
        return {"op": op, "seqs": _log(rng, 1, 512), "held": _log(rng, 1, 16384) if step else rng.choice((0, _log(rng, 1, 4096))),
                "new": _log(rng, 1, 4) if step else _log(rng, 5, 4096), "page": rng.choice((16, 32, 64, 128, 256)),
                "pad": rng.choice((0, _log(rng, 1, 2000))), "mix": mix}
    if op == "write":
        return {"op": op, "tokens": _log(rng, 1, 24000), "kv_heads": rng.choice((1, 2, 4, 5, 8, 16)), "dim": rng.choice((64, 128)),
                **rng.choice(({"src": "bf16", "cache": "bf16"}, {"src": "fp16", "cache": "fp16"}, {"src": "fp32", "cache": "bf16"}, {"src": "fp32", "cache": "fp16"})),
                "page": rng.choice((16, 32, 64, 128, 256)), "fused": rng.random() < 0.5, "pad": rng.choice((0, _log(rng, 1, 100)))}
    kv_heads, group = rng.choice((1, 2, 4, 8)), rng.choice((1, 2, 3, 4, 7, 8))
    heads = {"heads": kv_heads * group, "kv_heads": kv_heads, "dim": rng.choice((64, 128)), "type": rng.choice(("bf16", "fp16")), "lse": rng.random() < 0.5}
    if op == "prompt":
        seqs = _log(rng, 1, 32)
        longest = _log(rng, 1, min(16384, 48000 // seqs))
        return {"op": op, "seqs": seqs, "shortest": _log(rng, 1, longest), "longest": longest, **heads, "pad": rng.choice((0, _log(rng, 1, 200))), "mix": mix}
    page = rng.choice((16, 32, 64, 128, 256))
    kind = rng.choice(("decode", "chunk", "mixed"))
    seqs = _log(rng, 1, 96) if kind == "decode" else _log(rng, 1, 4) if kind == "chunk" else _log(rng, 2, 40)
    longest = _log(rng, 64, min(32768, 400000 // seqs))
    new = _log(rng, 1, 4) if kind == "decode" else _log(rng, 5, min(1200, longest)) if kind == "chunk" else 1
    chunks = rng.choice((1, 2)) if kind == "mixed" else 0
    chunk = _log(rng, 2, min(1500, longest)) if kind == "mixed" else 1
    return {"op": op, "seqs": seqs, "shortest": _log(rng, max(new, chunk), longest), "longest": longest, "new": new, "chunks": chunks, "chunk": chunk,
            **heads, "page": page, "mix": mix}


def _lengths(count, lo, hi, mix):
    """`count` lengths of [lo, hi], spread over their logarithm, the longest among them; the same for the same case."""
    rng = random.Random(mix)
    some = [_log(rng, lo, hi) for _ in range(count)]
    some[rng.randrange(count)] = hi
    return some


def _shape(case):
    """Host-known lengths of a case: what each request holds after the call, and what it appends in it."""
    if case["op"] == "plan":
        rng = random.Random(case["mix"])
        new = [rng.randrange(2) * case["new"] if case["new"] == 1 else _log(rng, 1, case["new"]) - rng.randrange(2) for _ in range(case["seqs"])]
        held = [_log(rng, 1, case["held"]) if case["held"] else 0 for _ in range(case["seqs"])]
        return [h + n for h, n in zip(held, new)], new
    total = _lengths(case["seqs"], case["shortest"], case["longest"], case["mix"])
    if case["op"] == "prompt":
        return total, total
    new = [case["new"]] * case["seqs"]
    for b in range(min(case["chunks"], case["seqs"])):
        new[b], total[b] = case["chunk"], max(case["chunk"], case["longest"] // (b + 1))
    return total, new


def _starts(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


# ---------------------------------------------------------------- inputs
def _pool(total, page, spare, gen):
    """A block table whose requests hold ceil(length / page) pages in no order, and the pages left over."""
    blocks = [-(-n // page) for n in total]
    pages = sum(blocks) + spare
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    width = max(1, max(blocks)) + 1
    first = torch.tensor(_starts(blocks), device="cuda")
    col = torch.arange(width, device="cuda")
    held = torch.tensor(blocks, device="cuda")
    table = torch.where(col < held[:, None], order[(first[:-1, None] + col).clamp(max=pages - 1)], -1).to(torch.int32)
    return table.contiguous(), order[sum(blocks):].contiguous(), pages, width


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, B = case["op"], case.get("seqs")

    def normal(*shape, dtype, std=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32 if dtype == torch.float32 else dtype) * std).contiguous()

    st = {"case": case}
    if op == "plan":
        total, new = _shape(case)
        held = [t - n for t, n in zip(total, new)]
        opened = sum(-(-t // case["page"]) - -(-h // case["page"]) for t, h in zip(total, held))
        table, free, pages, _ = _pool(held, case["page"], opened + 7, gen)
        width = max(-(-t // case["page"]) for t in total) + 2
        wide = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
        wide[:, :min(width, table.shape[1])] = table[:, :width]
        T = max(1, sum(new) + case["pad"])
        st.update(kv_lens=_ints(held), new_lens=_ints(new), table=wide, free=free, n_free=_ints([free.numel()]), tokens=T, pages=pages, max_blocks=width,
                  cu=_ints([0] * (B + 1)), kv_out=_ints([0] * B), slots=_ints([0] * T), pos=_ints([0] * T), n_free_out=_ints([0]), most=max(new))
    elif op == "write":
        T, H, dh, src = case["tokens"], case["kv_heads"], case["dim"], DTYPES[case["src"]]
        pages = -(-T // case["page"]) + 5
        slots = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
        slots = (slots[:, None] * case["page"] + _ints(list(range(case["page"])))).reshape(-1)[3:T + 3]
        st["slots"] = torch.cat([slots, _ints([-1] * case["pad"])]).contiguous()
        rows = T + case["pad"]
        if case["fused"]:  # rows of a fused projection: the queries, then the keys, then the values
            qkv = normal(rows, 3 * H, dh, dtype=src)
            st["k"], st["v"] = qkv[:, H:2 * H], qkv[:, 2 * H:]
        else:
            st["k"], st["v"] = normal(rows, H, dh, dtype=src), normal(rows, H, dh, dtype=src)
        st["k_cache"], st["v_cache"] = (normal(pages, case["page"], H, dh, dtype=DTYPES[case["cache"]]) for _ in range(2))
        st["pages"] = pages
    else:
        total, new = _shape(case)
        T, H, Hk, dh, dt = sum(new) + case.get("pad", 0), case["heads"], case["kv_heads"], case["dim"], DTYPES[case["type"]]
        st.update(total=total, new=new, cu_host=_starts(new), cu=_ints(_starts(new)), most=max(new))
        st["q"] = normal(T, H, dh, dtype=dt, std=1.5)
        st["out"] = torch.zeros(T, H, dh, dtype=dt, device="cuda")
        st["lse"] = torch.zeros(H, T, dtype=torch.float32, device="cuda") if case["lse"] else None
        if op == "prompt":
            st["k"], st["v"] = normal(T, Hk, dh, dtype=dt), normal(T, Hk, dh, dtype=dt)
        else:
            st["kv_lens"] = _ints(total)
            st["table"], _, pages, width = _pool(total, case["page"], 3, gen)
            st["k_cache"], st["v_cache"] = (normal(pages, case["page"], Hk, dh, dtype=dt) for _ in range(2))
            st.update(pages=pages, max_blocks=width)
    if own:
        _handles(case, st)
    return st


def _handles(case, st):
    """What a user's program builds once: the description of its shapes, and the workspace of their size."""
    from cross_loop_sparse_b200 import flashloop as F
    op, H = case["op"], case.get("kv_heads", 1)
    tokens = st["tokens"] if op == "plan" else st["k"].shape[0] if op == "write" else st["q"].shape[0]
    dtype = DTYPES[case.get("cache") or case.get("type") or "bf16"]
    st["params"] = F.PagedParams.make(batch=case.get("seqs", 1), max_tokens=tokens, max_new=st.get("most", 1), n_heads=case.get("heads", H), n_kv_heads=H,
                                      head_dim=case.get("dim", 128), page_size=case.get("page", 64), n_pages=st.get("pages", 1),
                                      max_blocks=st.get("max_blocks", 1), dtype=dtype)
    st["err"] = _ints([0])
    if op == "paged":
        st["workspace"] = torch.empty(max(16, F.flashloop_paged_attn_workspace_bytes(st["params"])), dtype=torch.uint8, device="cuda")


# ---------------------------------------------------------------- one pass
def run(st):
    op = st["case"]["op"]
    if own:
        return _run_own(op, st)
    return {"plan": _plan, "write": _write, "prompt": _prompt, "paged": _paged}[op](st)


def _run_own(op, st):
    from cross_loop_sparse_b200 import flashloop as F
    p, err = st["params"], st["err"]
    if op == "plan":
        F.flashloop_paged_plan(p, st["kv_lens"], st["new_lens"], st["free"], st["n_free"], st["table"], st["cu"], st["kv_out"], st["slots"], st["pos"],
                               st["n_free_out"], err)
        return st["cu"], st["kv_out"], st["table"], st["slots"], st["pos"], st["n_free_out"]
    if op == "write":
        F.flashloop_paged_kv_write(p, st["k"], st["v"], st["slots"], st["k_cache"], st["v_cache"], err)
        return st["k_cache"], st["v_cache"]
    if op == "prompt":
        F.flashloop_prompt_attn(p, st["q"], st["k"], st["v"], st["cu"], st["out"], st["lse"], err)
    else:
        F.flashloop_paged_attn(p, st["q"], st["k_cache"], st["v_cache"], st["table"], st["kv_lens"], st["cu"], st["out"], st["lse"], st["workspace"], err)
    return (st["out"], st["lse"]) if st["lse"] is not None else (st["out"],)


def _plan(st):
    """Request b appends new_b tokens at positions held_b.. of its cache; a page is taken from the stack's top for each that it opens."""
    page, T = st["case"]["page"], st["tokens"]
    held, new = st["kv_lens"].long(), st["new_lens"].long()
    total = held + new
    old, now = (held + page - 1) // page, (total + page - 1) // page
    cu = torch.cat([new.new_zeros(1), new.cumsum(0)])
    first = (now - old).cumsum(0) - (now - old)
    n_free = st["n_free"].long()
    col = torch.arange(st["max_blocks"], device="cuda")
    opened = (col >= old[:, None]) & (col < now[:, None])
    taken = (n_free - 1 - (first - old)[:, None] - col).clamp(0, st["free"].numel() - 1)
    table = torch.where(opened, st["free"][taken], st["table"])
    t = torch.arange(T, device="cuda")
    b = torch.bucketize(t, cu[1:], right=True).clamp(max=new.numel() - 1)
    pos = torch.where(t < cu[-1], held[b] + t - cu[b], 0)
    slot = torch.where(t < cu[-1], table[b, (pos // page).clamp(max=st["max_blocks"] - 1)].long() * page + pos % page, -1)
    return tuple(x.to(torch.int32) for x in (cu, total, table, slot, pos, n_free - (now - old).sum()))


def _write(st):
    n, H, dh = st["case"]["tokens"], st["case"]["kv_heads"], st["case"]["dim"]
    slot = st["slots"][:n].long()  # the padding behind them writes nothing
    st["k_cache"].view(-1, H, dh)[slot] = st["k"][:n].float().to(st["k_cache"].dtype)
    st["v_cache"].view(-1, H, dh)[slot] = st["v"][:n].float().to(st["v_cache"].dtype)
    return st["k_cache"], st["v_cache"]


def _softmax_rows(q, k, v, seen):
    """q [..., n, dh], k and v [..., L, dh] in 32 bits, `seen` where a row may look: (rows, log of their exponentials' sums). A row that sees nothing is zero."""
    s = (q @ k.transpose(-1, -2)) * (1.0 / math.sqrt(q.shape[-1]))
    s = s.masked_fill(~seen, -math.inf)
    m = s.amax(-1, keepdim=True)
    m0 = torch.where(m == -math.inf, 0.0, m)
    e = (s - m0).exp_()
    z = e.sum(-1, keepdim=True)
    return (e @ v) / torch.where(z == 0, 1.0, z), (m0 + z.log()).squeeze(-1)


def _outputs(st):
    out = torch.zeros_like(st["out"])
    return out, (torch.zeros_like(st["lse"]) if st["lse"] is not None else None)


def _prompt(st):
    """Blocks of packed rows against the packed columns from the first of their requests on, a row seeing its own request's up to itself."""
    H, Hk, cu = st["case"]["heads"], st["case"]["kv_heads"], st["cu_host"]
    out, lse = _outputs(st)
    T, g = cu[-1], H // Hk
    request = torch.bucketize(torch.arange(T, device="cuda"), st["cu"][1:].long(), right=True)
    step = max(64, min(2048, (1 << 30) // max(1, H * T)))
    first = 0
    for r0 in range(0, T, step):
        r1 = min(T, r0 + step)
        while cu[first + 1] <= r0:
            first += 1
        c0 = cu[first]
        row, col = torch.arange(r0, r1, device="cuda"), torch.arange(c0, r1, device="cuda")
        seen = (request[r0:r1, None] == request[None, c0:r1]) & (col <= row[:, None])
        q = st["q"][r0:r1].float().view(r1 - r0, Hk, g, -1).permute(1, 2, 0, 3).reshape(Hk, g * (r1 - r0), -1)
        o, l = _softmax_rows(q, st["k"][c0:r1].float().transpose(0, 1), st["v"][c0:r1].float().transpose(0, 1), seen.repeat(g, 1))
        out[r0:r1] = o.view(Hk, g, r1 - r0, -1).permute(2, 0, 1, 3).reshape(r1 - r0, H, -1).to(out.dtype)
        if lse is not None:
            lse[:, r0:r1] = l.view(H, r1 - r0)
    return (out, lse) if lse is not None else (out,)


def _gathered(cache, table, length):
    """The first `length` tokens of each of the table's requests, [b, Hk, length, dh] in 32 bits."""
    page = cache.shape[1]
    blocks = -(-length // page)
    x = cache[table[:, :blocks].long().clamp(min=0)].flatten(1, 2)[:, :length]
    return x.permute(0, 2, 1, 3).float()


def _paged(st):
    """Requests that append the same number of tokens go together, padded to the longest of them; long chunks go one at a time."""
    case = st["case"]
    H, Hk, total, new, cu = case["heads"], case["kv_heads"], st["total"], st["new"], st["cu_host"]
    out, lse = _outputs(st)
    g, lone = H // Hk, case["chunks"]
    groups = [[b] for b in range(len(new) if case["new"] > 4 else lone)]
    rest = list(range(len(groups), len(new)))
    groups += [rest] if rest else []
    for members in groups:
        b0, b1, n = members[0], members[-1] + 1, new[members[0]]
        B, L = b1 - b0, max(total[b0:b1])
        k, v = _gathered(st["k_cache"], st["table"][b0:b1], L), _gathered(st["v_cache"], st["table"][b0:b1], L)
        q = st["q"][cu[b0]:cu[b1]].float().view(B, n, Hk, g, -1).permute(0, 2, 3, 1, 4).reshape(B, Hk, g * n, -1)
        limit = st["kv_lens"][b0:b1, None] - n + torch.arange(n, device="cuda")
        seen = (torch.arange(L, device="cuda") <= limit[..., None]).repeat(1, g, 1)[:, None]
        o, l = _softmax_rows(q, k, v, seen)
        out[cu[b0]:cu[b1]] = o.view(B, Hk, g, n, -1).permute(0, 3, 1, 2, 4).reshape(B * n, H, -1).to(out.dtype)
        if lse is not None:
            lse[:, cu[b0]:cu[b1]] = l.view(B, Hk, g, n).permute(1, 2, 0, 3).reshape(H, B * n)
    return (out, lse) if lse is not None else (out,)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    op = case["op"]
    if op == "plan":
        total, new = _shape(case)
        page = case["page"]
        opened = sum(-(-t // page) - -(-(t - n) // page) for t, n in zip(total, new))
        # lengths in and out, starts, opened pages read and written, slots and positions of the tokens
        return {"bytes": 4 * (4 * case["seqs"] + 1 + 2 + 2 * opened + 2 * (sum(new) + case["pad"])), "flops": 0}
    if op == "write":
        src, dst = (4 if case["src"] == "fp32" else 2), 2
        return {"bytes": 2 * case["tokens"] * case["kv_heads"] * case["dim"] * (src + dst) + 4 * (case["tokens"] + case["pad"]), "flops": 0}
    total, new = _shape(case)
    H, Hk, dh = case["heads"], case["kv_heads"], case["dim"]
    pairs = sum(n * (t - n) + n * (n + 1) // 2 for t, n in zip(total, new))
    nbytes = 2 * 2 * sum(new) * H * dh + 2 * 2 * sum(total) * Hk * dh + (4 * H * sum(new) if case["lse"] else 0)
    if op == "paged":
        nbytes += 4 * sum(-(-t // case["page"]) for t in total)
    return {"bytes": nbytes, "flops": 4 * dh * H * pairs}


# ---------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "plan":
        return _exact_plan(case, st)
    if op == "write":
        k, v = st["k_cache"].double(), st["v_cache"].double()
        H, dh = case["kv_heads"], case["dim"]
        for cache, rows in ((k, st["k"]), (v, st["v"])):
            at = st["slots"][:case["tokens"]].long()
            cache.reshape(-1, H * dh).index_copy_(0, at, rows[:case["tokens"]].double().reshape(-1, H * dh))
        return k, v
    total, new = _shape(case)
    H, Hk, dh = case["heads"], case["kv_heads"], case["dim"]
    T = st["q"].shape[0]
    out = torch.zeros(T, H, dh, dtype=torch.float64, device="cuda")
    lse = torch.zeros(H, T, dtype=torch.float64, device="cuda")
    start = 0
    for b, (t, n) in enumerate(zip(total, new)):
        if op == "prompt":
            keys, values = st["k"][start:start + n].double(), st["v"][start:start + n].double()
        else:
            page = case["page"]
            at = torch.arange(t, device="cuda")
            slot = st["table"][b].long()[at // page] * page + at % page
            keys, values = (c.view(-1, Hk, dh)[slot].double() for c in (st["k_cache"], st["v_cache"]))
        for h in range(H):
            kh, vh = keys[:, h * Hk // H], values[:, h * Hk // H]
            for i0 in range(0, n, 4096):
                i1 = min(n, i0 + 4096)
                c = t - n + i1
                s = st["q"][start + i0:start + i1, h].double() @ kh[:c].T / math.sqrt(dh)
                last = t - n + torch.arange(i0, i1, device="cuda")
                s[torch.arange(c, device="cuda")[None] > last[:, None]] = -math.inf
                l = torch.logsumexp(s, 1)
                out[start + i0:start + i1, h] = s.sub_(l[:, None]).exp_() @ vh[:c]
                lse[h, start + i0:start + i1] = l
        start += n
    return (out, lse) if case["lse"] else (out,)


def _exact_plan(case, st):
    page, held, new = case["page"], st["kv_lens"].tolist(), st["new_lens"].tolist()
    table, stack = st["table"].tolist(), st["free"].tolist()
    cu, kv, slot, pos = [0], [], [], []
    for b, (h, n) in enumerate(zip(held, new)):
        for p in range(h, h + n):
            if p % page == 0:
                table[b][p // page] = stack.pop()
            slot.append(table[b][p // page] * page + p % page)
            pos.append(p)
        cu.append(cu[-1] + n)
        kv.append(h + n)
    spare = st["tokens"] - len(slot)
    return tuple(_ints(x) for x in (cu, kv, table, slot + [-1] * spare, pos + [0] * spare, [len(stack)]))
