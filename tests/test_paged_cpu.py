"""The many-request entry points on the CPU: struct layouts, sizing, refusals
before any device query, and models of how the kernels cut their work."""
import ctypes
import os
import random
import shutil
import subprocess
import tempfile

import pytest
import torch

try:
    from cross_loop_sparse_b200 import flashloop as F
except ImportError as exc:  # pragma: no cover - the library must be built first
    pytest.skip(f"libflashloop.so not built: {exc}", allow_module_level=True)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.skipif(shutil.which("gcc") is None, reason="gcc not available")
def test_struct_layout_matches_header():
    fields = [n for n, _ in F.PagedParams._fields_]
    src = '#include <stdio.h>\n#include <stddef.h>\n#include "flashloop.h"\nint main(void) {\n  printf("%zu %zu %zu", sizeof(flashloop_paged_params), sizeof(flashloop_rows), sizeof(flashloop_pages));\n'
    for s, c in (("paged_params", F.PagedParams), ("rows", F.RowsC), ("pages", F.PagesC)):
        for n, _ in c._fields_:
            src += f'  printf(" %zu", offsetof(flashloop_{s}, {n}));\n'
    src += "  return 0;\n}\n"
    with tempfile.TemporaryDirectory() as d:
        c, exe = os.path.join(d, "probe.c"), os.path.join(d, "probe")
        open(c, "w").write(src)
        subprocess.check_call(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), c, "-o", exe])
        got = [int(v) for v in subprocess.check_output([exe], text=True).split()]
    want = [ctypes.sizeof(c) for c in (F.PagedParams, F.RowsC, F.PagesC)]
    want += [getattr(c, n).offset for c in (F.PagedParams, F.RowsC, F.PagesC) for n, _ in c._fields_]
    assert got == want and fields[-1] == "scale"


def params(**over):
    p = F.PagedParams.make(batch=4, max_tokens=32, max_new=16, n_heads=8, n_kv_heads=2, head_dim=128, page_size=64, n_pages=100, max_blocks=30)
    for k, v in over.items():
        setattr(p, k, v)
    return p


SIZES = [dict(batch=-1), dict(max_tokens=-1), dict(max_new=0)]
PAGES = [dict(n_pages=0), dict(max_blocks=0)]
HEADS = [dict(n_kv_heads=0)]
QUERIES = [dict(n_heads=7), dict(n_heads=0), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("inf")), dict(scale=float("nan"))]
UNSUPPORTED_PAGES = [dict(page_size=8), dict(page_size=48), dict(page_size=512), dict(page_size=0), dict(n_pages=2 ** 26), dict(max_blocks=2 ** 25)]
UNSUPPORTED_HEADS = [dict(head_dim=96), dict(head_dim=256), dict(dtype=2), dict(dtype=-1), dict(n_kv_heads=70000)]


def test_bad_parameters_are_refused_before_any_device_query():
    a = ctypes.c_void_p(4096)
    rows, pages = F.RowsC(4096, 1024, 128), F.PagesC(4096, 65536, 1024, 128)
    R, P, B = ctypes.byref(rows), ctypes.byref(pages), ctypes.byref

    def plan(p):
        return F._lib.flashloop_paged_plan(B(p), a, a, a, 100, a, a, a, ctypes.c_void_p(8192), a, a, ctypes.c_void_p(12288), a, None)

    def write(p):
        return F._lib.flashloop_paged_kv_write(B(p), R, R, p.dtype, a, P, P, a, None)

    def prompt(p):
        return F._lib.flashloop_prompt_attn(B(p), R, R, R, a, R, a, a, None)

    def paged(p):
        return F._lib.flashloop_paged_attn(B(p), R, P, P, a, a, a, R, a, a, 1 << 40, a, None)

    for call, bad, unsupported in ((plan, SIZES + PAGES, UNSUPPORTED_PAGES + [dict(batch=70000)]), (write, SIZES + PAGES + HEADS, UNSUPPORTED_PAGES + UNSUPPORTED_HEADS),
                                   (prompt, SIZES + HEADS + QUERIES, UNSUPPORTED_HEADS + [dict(max_tokens=2 ** 29)]),
                                   (paged, SIZES + PAGES + HEADS + QUERIES, UNSUPPORTED_PAGES + UNSUPPORTED_HEADS + [dict(max_tokens=2 ** 29)])):
        for over in bad:
            assert call(params(**over)) == -1, (call.__name__, over)
        for over in unsupported:
            assert call(params(**over)) == -2, (call.__name__, over)
    for call in (F._lib.flashloop_paged_attn_workspace_bytes,):
        for over in SIZES + PAGES + HEADS + QUERIES + UNSUPPORTED_PAGES + UNSUPPORTED_HEADS:
            assert call(B(params(**over))) == 0


def test_bad_arguments_are_refused_before_any_device_query():
    p = params()
    a, B = ctypes.c_void_p(4096), ctypes.byref
    rows, pages = F.RowsC(4096, 1024, 128), F.PagesC(4096, 65536, 1024, 128)
    bad_rows = [F.RowsC(None, 1024, 128), F.RowsC(4104, 1024, 128), F.RowsC(4096, 1028, 128), F.RowsC(4096, 1024, 4), F.RowsC(4096, -1024, 128), F.RowsC(4096, 1 << 40, 128)]
    bad_pages = [F.PagesC(None, 65536, 1024, 128), F.PagesC(4098, 65536, 1024, 128), F.PagesC(4096, 65540, 1024, 128), F.PagesC(4096, 65536, 1, 128)]
    n = F.flashloop_paged_attn_workspace_bytes(p)
    assert n > 16

    def prompt(q=rows, k=rows, v=rows, cu=a, o=rows):
        return F._lib.flashloop_prompt_attn(B(p), B(q), B(k), B(v), cu, B(o), a, a, None)

    def paged(q=rows, kc=pages, vc=pages, table=a, kv=a, cu=a, o=rows, ws=a, size=n):
        return F._lib.flashloop_paged_attn(B(p), B(q), B(kc), B(vc), table, kv, cu, B(o), a, ws, size, a, None)

    def write(k=rows, v=rows, src=0, slots=a, kc=pages, vc=pages):
        return F._lib.flashloop_paged_kv_write(B(p), B(k), B(v), src, slots, B(kc), B(vc), a, None)

    for r in bad_rows:
        for arg in ("q", "k", "v", "o"):
            assert prompt(**{arg: r}) == -1, arg
        assert paged(q=r) == -1 and paged(o=r) == -1 and write(k=r) == -1 and write(v=r) == -1
    for c in bad_pages:
        assert paged(kc=c) == -1 and paged(vc=c) == -1 and write(kc=c) == -1 and write(vc=c) == -1
    assert prompt(cu=None) == -1 and write(slots=None) == -1
    for arg in ("table", "kv", "cu", "ws"):
        assert paged(**{arg: None}) == -1
    assert paged(size=n - 1) == -1 and paged(ws=ctypes.c_void_p(4104)) == -1
    assert write(src=1) == -2 and write(src=3) == -2
    # float32 rows: strides of 16 bytes are multiples of four elements
    assert write(k=F.RowsC(4096, 1026, 128), src=2) == -1
    # plan: a missing buffer, and new lengths that lie over the old
    args = [a, a, a, 100, a, a, a, ctypes.c_void_p(8192), a, a, ctypes.c_void_p(12288)]
    for i in range(11):
        some = list(args)
        some[i] = -1 if i == 3 else None
        assert F._lib.flashloop_paged_plan(B(p), *some, a, None) == -1, i
    for i, over in ((7, 4096), (7, 4096 + 12), (10, 4096)):
        some = list(args)
        some[i] = ctypes.c_void_p(over)
        assert F._lib.flashloop_paged_plan(B(p), *some, a, None) == -1, (i, over)


def test_nothing_to_do_is_no_error():
    """No requests or no rows: attention and writes launch nothing, with any buffers."""
    B = ctypes.byref
    rows, pages = F.RowsC(None, 0, 0), F.PagesC(4096, 65536, 1024, 128)
    for over in (dict(batch=0), dict(max_tokens=0)):
        p = params(**over)
        assert F._lib.flashloop_prompt_attn(B(p), B(rows), B(rows), B(rows), None, B(rows), None, None, None) == 0
        assert F._lib.flashloop_paged_attn(B(p), B(rows), B(pages), B(pages), None, None, None, B(rows), None, None, 0, None, None) == 0
    p = params(max_tokens=0)
    assert F._lib.flashloop_paged_kv_write(B(p), B(rows), B(rows), 0, None, B(pages), B(pages), None, None) == 0


def test_workspace_follows_the_shape_alone():
    small = F.flashloop_paged_attn_workspace_bytes(params(max_new=1, max_blocks=2))
    decode = F.flashloop_paged_attn_workspace_bytes(params(max_new=1, max_blocks=2000))
    chunk = F.flashloop_paged_attn_workspace_bytes(params(max_new=16, max_blocks=2000))
    assert small == 16 < decode < chunk < 64 << 20
    assert F.flashloop_paged_attn_workspace_bytes(params(max_new=16, max_blocks=2000, max_tokens=10000, batch=900)) == chunk


def test_binding_refuses_host_tensors_and_types():
    p = params()
    q = torch.zeros(32, 8, 128, dtype=torch.bfloat16)
    k = torch.zeros(32, 2, 128, dtype=torch.bfloat16)
    i = torch.zeros(32, dtype=torch.int32)
    with pytest.raises(F.FlashLoopError) as e:
        F.flashloop_prompt_attn(p, q, k, k, i, q, None, i)
    assert e.value.status == -1 and "CUDA" in str(e.value)
    with pytest.raises(F.FlashLoopError) as e:
        F.PagedParams.make(batch=1, max_tokens=1, max_new=1, n_heads=1, n_kv_heads=1, head_dim=64, dtype=torch.float32)
    assert e.value.status == -2


# ------------------------------------------------------------------------------- how the work is cut
def cut_line(items, per, start):
    """The cut of both kernels: items of `units` (the first `start` of them without work) laid end to end, block c
    takes units [c per, (c + 1) per).  Returns per item its parts [(block, slot, first unit, end)], and each block's record."""
    parts, records, at = [], {}, 0
    for n, units in enumerate(items):
        s0, u1 = at + start, at + units
        mine = []
        fc, lc = s0 // per, (u1 - 1) // per
        for c in range(at // per, lc + 1):
            x, end = max(at, c * per), min(u1, (c + 1) * per)
            if end <= s0:
                continue  # the next block has the work
            slot = c * 2 + (1 if fc == c and s0 != fc * per else 0)
            mine.append((c, slot, max(0, x - s0), end - s0))
            if lc > fc and fc == c:
                assert c not in records, "a block has part 0 of one cut item at most"
                records[c] = (n, lc - fc + 1, slot)
        parts.append(mine)
        at = u1
    return parts, records, at


@pytest.mark.parametrize("start", [0, 6])
def test_the_cut_covers_every_unit_once_and_slots_do_not_collide(start):
    rng = random.Random(start)
    for _ in range(400):
        blocks = rng.choice((148, 296))
        items = [start + rng.choice((1, rng.randint(1, 8), rng.randint(1, 600))) for _ in range(rng.choice((1, 3, 40, 900)))]
        per = max(4, -(-sum(items) // blocks))
        parts, records, total = cut_line(items, per, start)
        assert total == sum(items) and -(-total // per) <= blocks
        used = {}
        for n, mine in enumerate(parts):
            assert mine[0][2] == 0 and mine[-1][3] == items[n] - start
            assert all(a[3] == b[2] and b[0] == a[0] + 1 for a, b in zip(mine, mine[1:]))
            if len(mine) > 1:
                block, count, slot0 = mine[0][0], len(mine), mine[0][1]
                assert records[block] == (n, count, slot0)
                for k, (c, slot, _, _) in enumerate(mine):
                    assert slot == (slot0 if k == 0 else (slot0 & ~1) + 2 * k) and slot < 2 * blocks
                    assert slot not in used, "two parts in one slot"
                    used[slot] = n
        assert len(records) == sum(len(m) > 1 for m in parts)


def tiles_seen(n, L, G, end):
    f = L - n + (min(end, n * G) - 1) // G + 1
    return -(-f // 128) if f > 0 else 0


def first_pair(n, L, G, pairs, units):
    """The closed form the tile kernel deals its list with."""
    x = (units - 1) * 128 - (L - n)
    if units <= 1 or x <= 0:
        return 0
    if x > n - 1:
        return pairs
    return min(pairs - 1, (x * G + 256) // 256 - 1)


def test_dealt_list_holds_every_row_pair_once():
    rng = random.Random(7)
    for _ in range(300):
        G, Hk, grid = rng.choice((1, 2, 3, 7, 8, 40)), rng.choice((1, 2, 8)), rng.choice((1, 5, 148))
        reqs = [(n, rng.choice((n, n + rng.randint(0, 900), max(0, n - rng.randint(0, 50))))) for n in (rng.choice((0, 1, rng.randint(1, 2000))) for _ in range(rng.choice((1, 4, 40))))]
        most = max(n for n, _ in reqs)
        listed = []
        for cls in reversed(range(max(1, -(-max(1, most) // 128)).bit_length())):
            for b, (n, L) in enumerate(reqs):
                pairs = -(-n * G // 256)
                p0, p1 = first_pair(n, L, G, pairs, 1 << cls), first_pair(n, L, G, pairs, 2 << cls)
                units = [max(1, tiles_seen(n, L, G, (p + 1) * 256)) for p in range(pairs)]
                if L <= most:
                    assert [p for p in range(pairs) if (1 << cls) <= units[p] < (2 << cls)] == list(range(p0, p1))
                listed += [(b, p1 - 1 - i // Hk, i % Hk) for i in range((p1 - p0) * Hk)]
        if all(L <= most for _, L in reqs):  # prompts: a request's columns are its rows
            assert sorted(listed) == sorted((b, p, h) for b, (n, _) in enumerate(reqs) for p in range(-(-n * G // 256)) for h in range(Hk))
        dealt, r = [], 0
        while r * grid < len(listed):
            dealt += [r * grid + (grid - 1 - c if r & 1 else c) for c in range(grid)]
            r += 1
        assert sorted(i for i in dealt if i < len(listed)) == list(range(len(listed)))


def test_sizes_whose_sums_would_pass_32_bits_are_refused():
    """Row and column indexes are rounded up to tiles and advanced by strides in 32 bits, so the bounds end below 2^31."""
    a, B = ctypes.c_void_p(4096), ctypes.byref
    R, P = B(F.RowsC(4096, 1024, 128)), B(F.PagesC(4096, 65536, 1024, 128))

    def calls(p):
        yield F._lib.flashloop_paged_plan(B(p), a, a, a, 100, a, a, a, ctypes.c_void_p(8192), a, a, ctypes.c_void_p(12288), a, None)
        yield F._lib.flashloop_paged_kv_write(B(p), R, R, 0, a, P, P, a, None)
        yield F._lib.flashloop_prompt_attn(B(p), R, R, R, a, R, None, a, None)
        yield F._lib.flashloop_paged_attn(B(p), R, P, P, a, a, a, R, None, a, 1 << 62, a, None)

    for big in (2 ** 30 + 1, 2 ** 31 - 1):
        assert list(calls(params(max_tokens=big, n_heads=2, n_kv_heads=2))) == [-2] * 4, big
    for big in (2 ** 31 - 2 ** 16 + 1, 2 ** 31 - 1):
        assert list(calls(params(max_tokens=1, n_heads=big, n_kv_heads=1)))[2:] == [-2] * 2, big
    for page in (16, 64, 256):
        rcs = list(calls(params(page_size=page, n_pages=4, max_blocks=(2 ** 31 - 1) // page)))
        assert [rcs[0], rcs[1], rcs[3]] == [-2] * 3, page
    assert F.flashloop_paged_attn_workspace_bytes(params(max_blocks=(2 ** 31 - 2 ** 16) // 64)) > 0


def test_items_that_outlast_a_bounded_wait_go_to_the_kernel_without_waits():
    """The two kernels need scratch of different sizes: 148 x 2 slots of 256 rows, or 296 x 2 of 32."""
    tile, few = 2 * 148 * 256 * (128 * 4 + 8), 4 * 148 * 32 * (128 * 4 + 8)
    many = dict(max_tokens=4096, max_new=4096, n_pages=1000)
    at = F.flashloop_paged_attn_workspace_bytes(params(max_blocks=2 ** 24 // 64, **many))
    behind = F.flashloop_paged_attn_workspace_bytes(params(max_blocks=2 ** 24 // 64 + 1, **many))
    assert tile <= at < tile + 2 ** 15 and few <= behind < few + 2 ** 15


def test_strides_of_single_entries_do_not_matter():
    """torch may give a dimension of one any stride; the library asks for multiples of 16 bytes."""
    bf = torch.bfloat16
    t = torch.empty(4096, dtype=bf)
    for st, sh in ((1, 128), (1, 3), (256, 5), (0, 0)):
        shape = (1, 2 if sh == 128 else 1, 128)
        r = F._rows("f", "q", t.as_strided(shape, (st, sh, 1)), shape, bf, -1, written=True)
        assert r.stride_token % 8 == 0 and r.stride_head % 8 == 0 and r.stride_token > 0 and r.stride_head > 0
    p = F.PagedParams.make(1, 1, 1, 1, 1, 128, page_size=16, n_pages=1)
    c = F._pages("f", "k_cache", t.as_strided((1, 16, 1, 128), (3, 128, 5, 1)), p, bf, -1, written=True)
    assert (c.stride_page % 8, c.stride_token, c.stride_head % 8) == (0, 128, 0)
