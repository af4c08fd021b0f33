"""Model of how pg_tile_kernel (csrc/paged_tile.cu) looks over the V tiles that some row does not see whole: the
loads' warp does before it brings more, and the write-back reads what was found.  The other roles as in
test_paged_protocol_cpu; random schedules, planted mistakes."""
import random

import pytest

from test_protocol_models_cpu import Bar, Stuck, run_schedule, wait


def tile_cta(items, stages, rnd, plant=None):
    """items: (column tiles of tile A, of tile B, first of them that is looked over) of each work item."""
    B = {}
    for s in range(stages):
        B[("kv_full", s)], B[("kv_empty", s)] = Bar(1), Bar(2)
    for i in range(4):
        B[("s_full", i)], B[("p_full", i)] = Bar(1), Bar(1)
    for x in range(2):
        for n in ("acc_full", "inv_full", "n_free", "q_full", "q_empty", "item_full"):
            B[(n, x)] = Bar(1)
        B[("item_empty", x)] = Bar(6)  # loads, two issuers, queries, two row groups
    B["fin"], B["tail"] = Bar(2), Bar(1)
    loads, pipe, place, found, looked, held = [], [], [None, None], [set(), set()], set(), {}
    last = len(items)

    def schedule():
        for k in range(last + 1):
            yield from wait(B, ("item_empty", k & 1), (k >> 1) - 1)
            place[k & 1], found[k & 1] = k, set()
            B[("item_full", k & 1)].arrive()

    def item(k, release=True):
        yield from wait(B, ("item_full", k & 1), k >> 1)
        assert place[k & 1] == k
        if release:
            B[("item_empty", k & 1)].arrive()

    def tma():
        seq, tails, open_tile = 0, 0, None  # (slot, item, tile) that has not been looked over yet

        def look_over():
            nonlocal tails, open_tile
            yield from wait(B, "tail", tails)
            tails += 1
            slot, k, t = open_tile
            for _ in range(rnd.randint(0, 3)):
                assert held[slot] == (k, t, 1), "another tile in the slot"
                yield None
            assert place[k & 1] == k, "the item's place was given away"
            looked.add((k, t))
            found[k & 1].add(t)
            B[("kv_full", slot)].arrive()
            open_tile = None

        for k in range(last + 1):
            yield from item(k)
            if k == last:
                break
            for t in range(max(items[k][:2])):
                for kv in range(2):
                    slot = seq % stages
                    yield from wait(B, ("kv_empty", slot), seq // stages - 1)
                    held[slot] = (k, t, kv)
                    look = kv == 1 and t >= items[k][2]
                    if look:
                        open_tile = (slot, k, t)
                    loads.append("tail" if look else ("kv_full", slot))
                    seq += 1
                    if look and plant != "two_open":
                        yield from look_over()

    def issuer(x):
        seq = u = 0
        slot, phase = (lambda s: s % stages), (lambda s: s // stages)

        def skip(s):
            yield from wait(B, ("kv_full", slot(s)), phase(s))
            B[("kv_empty", slot(s))].arrive()

        for k in range(last + 1):
            yield from item(k)
            if k == last:
                break
            my, nt, base, first = items[k][x], max(items[k][:2]), seq, items[k][2]
            yield from wait(B, ("q_full", x), k)
            if my > 0:
                yield from wait(B, ("kv_full", slot(base)), phase(base))
                for hf in range(2):
                    pipe.extend([("mma", None), ("commit", ("s_full", 2 * x + hf))])
                if my == 1:
                    pipe.append(("commit", ("q_empty", x)))
                pipe.append(("commit", ("kv_empty", slot(base))))
                if k > 0:
                    yield from wait(B, ("n_free", x), k - 1)
            else:
                pipe.append(("commit", ("q_empty", x)))
                if nt > 0:
                    yield from skip(base)
            for t in range(my):
                vs, ks = base + 2 * t + 1, base + 2 * t + 2
                more = t + 1 < my
                yield from wait(B, ("kv_full", slot(vs)), phase(vs))
                if more:
                    yield from wait(B, ("kv_full", slot(ks)), phase(ks))
                for hf in range(2):
                    yield from wait(B, ("p_full", 2 * x + hf), u)
                    assert t < first or (k, t) in looked, "a product with values that were not looked over"
                    pipe.append(("mma", None))
                    if more:
                        pipe.extend([("mma", None), ("commit", ("s_full", 2 * x + hf))])
                    elif hf:
                        pipe.append(("commit", ("acc_full", x)))
                u += 1
                pipe.append(("commit", ("kv_empty", slot(vs))))
                if more:
                    pipe.append(("commit", ("kv_empty", slot(ks))))
                    if t + 2 == my:
                        pipe.append(("commit", ("q_empty", x)))
            for s in range(base + (2 * my if my > 0 else 1), base + 2 * nt):
                yield from skip(s)
            if my == 0:
                if k > 0:
                    yield from wait(B, ("n_free", x), k - 1)
                pipe.append(("commit", ("acc_full", x)))
            seq = base + 2 * nt
        pipe.append(("commit", "fin"))
        yield from wait(B, "fin", 0)

    def queries():
        def write_back(k):
            for x in range(2):
                yield from wait(B, ("acc_full", x), k)
                yield from wait(B, ("inv_full", x), k)
                my, first = items[k][x], items[k][2]
                assert place[k & 1] == k and found[k & 1] >= set(range(first, my)), "the numerators are read before all was found"
                yield None
                B[("n_free", x)].arrive()
                if plant == "early_release" and x == 0:
                    B[("item_empty", k & 1)].arrive()
            if plant != "early_release":
                B[("item_empty", k & 1)].arrive()

        for k in range(last + 1):
            yield from item(k, release=False)
            if k < last:
                for x in range(2):
                    if k > 0:
                        yield from wait(B, ("q_empty", x), k - 1)
                    B[("q_full", x)].arrive()
            if k > 0:
                yield from write_back(k - 1)

    def rows(x):
        u = 0
        for k in range(last + 1):
            yield from item(k, release=False)
            if k < last:
                for _ in range(items[k][x]):
                    for hf in range(2):
                        yield from wait(B, ("s_full", 2 * x + hf), u)
                        for _ in range(rnd.randint(0, 3)):
                            yield None
                        B[("p_full", 2 * x + hf)].arrive()
                    u += 1
                if k > 0:
                    yield from wait(B, ("n_free", x), k - 1)
                B[("inv_full", x)].arrive()
            B[("item_empty", k & 1)].arrive()

    run_schedule(B, [schedule(), tma(), issuer(0), issuer(1), queries(), rows(0), rows(1)], loads, pipe, rnd)
    assert looked == {(k, t) for k, (a, b, first) in enumerate(items) for t in range(first, max(a, b))}


def random_items(rnd):
    out = []
    for _ in range(rnd.randint(0, 8)):
        b = rnd.choice((0, 1, 2, 3, rnd.randint(0, 9)))
        a = rnd.choice((b, max(0, b - 1), max(0, b - 2), 0))
        out.append(((a, b) if rnd.random() < 0.7 else (b, 0)) + (rnd.choice((0, max(0, b - 2), max(0, b - 1), b, b + 3)),))
    return out


@pytest.mark.parametrize("stages", [5, 8])
def test_looking_over_keeps_phases_places_and_progress(stages):
    for seed in range(400):
        rnd = random.Random(seed)
        tile_cta(random_items(rnd), stages, rnd)


@pytest.mark.parametrize("plant", ["two_open", "early_release"])
def test_the_model_catches_planted_mistakes(plant):
    caught = 0
    for seed in range(60):
        rnd = random.Random(seed)
        try:
            tile_cta([(1, 9, 0), (3, 4, 0), (1, 3, 0), (2, 3, 0), (0, 1, 0), (4, 4, 0)], 5, rnd, plant=plant)
        except (AssertionError, Stuck):
            caught += 1
    assert caught > 0
