"""Model of pg_tile_kernel's mbarrier protocol (csrc/paged_tile.cu) under random
schedules: the work-item ring, the K / V slots that both tiles' issuers give
back, per-half score and P barriers with the next tile's scores issued behind
each P.V, the wait of a raised reference, the queries' places, and the
write-back by the query warps while the rows take the next item.  Barriers, polls and schedules as in the other kernels' models."""
import random

import pytest

from test_protocol_models_cpu import Bar, Stuck, run_schedule, wait


def tile_cta(items, stages, rnd, plant=None):
    """items: column tiles (of tile A, of tile B) of each work item."""
    B = {}
    for s in range(stages):
        B[("kv_full", s)], B[("kv_empty", s)] = Bar(1), Bar(1 if plant == "kv_empty_count" else 2)
    for i in range(4):
        B[("s_full", i)], B[("p_full", i)] = Bar(1), Bar(1)  # the four row warps of a tile move together
    for x in range(2):
        for n in ("pv0_done", "acc_full", "inv_full", "n_free", "q_full", "q_empty", "item_full"):
            B[(n, x)] = Bar(1)
        B[("item_empty", x)] = Bar(6)  # loads, two issuers, queries, two row groups
    B["fin"] = Bar(2)
    loads, pipe = [], []
    last = len(items)  # the invalid item that ends every role

    def schedule():
        for k in range(last + 1):
            yield from wait(B, ("item_empty", k & 1), (k >> 1) - 1)
            B[("item_full", k & 1)].arrive()

    def item(k, release=True):
        yield from wait(B, ("item_full", k & 1), k >> 1)
        if release:
            B[("item_empty", k & 1)].arrive()

    def tma():
        seq = 0
        for k in range(last + 1):
            yield from item(k)
            if k == last:
                return
            for _ in range(2 * max(items[k])):
                yield from wait(B, ("kv_empty", seq % stages), seq // stages - 1)
                loads.append(("kv_full", seq % stages))
                seq += 1

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
            my, nt, base = items[k][x], max(items[k]), seq
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
                    yield from wait(B, ("p_full", 2 * x + hf), u - (plant == "p_phase"))
                    pipe.append(("mma", None))
                    if more:
                        pipe.extend([("mma", None), ("commit", ("s_full", 2 * x + hf))])
                    else:
                        pipe.append(("commit", ("acc_full" if hf else "pv0_done", x)))
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

    held = [-1, -1]  # the item whose 1 / z lies in shared memory

    def queries():
        def write_back(k):
            for x in range(2):
                yield from wait(B, ("acc_full", x), k)
                yield from wait(B, ("inv_full", x), k)
                assert held[x] == k, "1 / z of another item"
                for _ in range(rnd.randint(0, 4)):
                    yield None
                B[("n_free", x)].arrive()
            B[("item_empty", k & 1)].arrive()

        for k in range(last + 1):
            yield from item(k, release=False)
            if k == last:
                if k > 0:
                    yield from write_back(k - 1)
                return
            if k > 0:
                yield from wait(B, ("q_empty", 0), k - 1)
            both = k == 0 or B[("q_empty", 1)].done > k - 1
            if not both:
                B[("q_full", 0)].arrive()
                yield from wait(B, ("q_empty", 1), k - 1)
            for _ in range(rnd.randint(0, 3)):
                yield None
            if both:
                B[("q_full", 0)].arrive()
            B[("q_full", 1)].arrive()
            if k > 0:
                yield from write_back(k - 1)

    def rows(x):
        u = full = 0
        for k in range(last + 1):
            yield from item(k, release=False)
            if k == last:
                B[("item_empty", k & 1)].arrive()
                return
            my = items[k][x]
            for t in range(my):
                for hf in range(2):
                    yield from wait(B, ("s_full", 2 * x + hf), u)
                    if (t > 0 or hf > 0) and rnd.random() < 0.3:  # the reference is raised
                        if hf == 0:
                            yield from wait(B, ("s_full", 2 * x + 1), u)
                        elif t + 1 < my:
                            yield from wait(B, ("s_full", 2 * x), u + 1)
                        else:
                            yield from wait(B, ("pv0_done", x), u if plant == "pv0_phase" else full)
                    for _ in range(rnd.randint(0, 3)):
                        yield None
                    B[("p_full", 2 * x + hf)].arrive()
                u += 1
            full += my > 0
            if k > 0 and plant != "inv_reuse":
                yield from wait(B, ("n_free", x), k - 1)
            held[x] = k
            B[("inv_full", x)].arrive()
            for _ in range(rnd.randint(0, 3)):
                yield None
            B[("item_empty", k & 1)].arrive()

    run_schedule(B, [schedule(), tma(), issuer(0), issuer(1), queries(), rows(0), rows(1)], loads, pipe, rnd)


def random_items(rnd):
    out = []
    for _ in range(rnd.randint(0, 8)):
        b = rnd.choice((0, 1, 2, 3, rnd.randint(0, 9)))
        a = rnd.choice((b, max(0, b - 1), max(0, b - 2), 0))
        out.append((a, b) if rnd.random() < 0.7 else (b, 0))  # without a tile B, too
    return out


@pytest.mark.parametrize("stages", [5, 8])
def test_tile_protocol_phases_and_progress(stages):
    for seed in range(150):
        rnd = random.Random(seed)
        tile_cta(random_items(rnd), stages, rnd)


@pytest.mark.parametrize("plant", ["kv_empty_count", "p_phase", "pv0_phase", "inv_reuse"])
def test_tile_protocol_model_catches_planted_mistakes(plant):
    caught = 0
    for seed in range(30):
        rnd = random.Random(seed)
        try:
            tile_cta([(3, 4), (1, 0), (2, 3), (0, 1), (4, 4)], 5, rnd, plant=plant)
        except (AssertionError, Stuck):
            caught += 1
    assert caught > 0
