"""A CPU model of the decode kernel's slot ring (csrc/attention.cu) with its two
halves a slot, under random interleavings. A loading warp per slot fills K (with
q and the row flags), then V, each once the half's "empty" barrier has released
it; each (half, consumer group) has its own "full" barrier; a group gives K back
after the scores and V after p.V, and reads the row flags, of which there are two
sets a slot, until the softmax. With `handed` (csrc/attention_few.cu) only the
loading warps find the items: a consumer takes the next one that is handed on with
K, until one says that there are no more. Checked: no deadlock, every half and flag set that
is read holds the reader's own item, nothing lands in what is being read. The
form with one flag set has to break."""
import math
import random

import pytest

from test_barrier_protocols import _Bar


def _run(slots, groups, items, seed, flag_sets=2, handed=False):
    rng = random.Random(seed)
    bars = lambda n: [_Bar(1) for _ in range(n)]
    full = {h: bars(slots * groups) for h in "KV"}
    empty = {h: bars(slots) for h in "KV"}
    data = {h: [None] * slots for h in "KV"}
    reading = {h: [None] * slots for h in "KV"}
    flags = [[None] * slots for _ in range(flag_sets)]
    pending = []
    bar_of = lambda h, k: full[h][(k % slots) * groups + k % groups]
    parity = lambda k: (k // math.lcm(slots, groups)) & 1
    flag_of = lambda k: flags[(k // slots) % flag_sets]

    def loader(lw):
        for k in range(lw, items, slots):
            for h in "KV":
                if k >= slots:
                    while not empty[h][k % slots].try_wait(((k // slots) - 1) & 1):
                        yield
                if h == "K":
                    flag_of(k)[k % slots] = k
                bar_of(h, k).arrive(tx=1)
                pending.append((h, k % slots, k, bar_of(h, k)))
                yield
        last = max((k for k in range(lw, items, slots)), default=None)
        if last is not None:                             # its copies land before the loader leaves
            while not bar_of("K", last).try_wait(parity(last)):
                yield
        if handed:                                       # no more items
            k = next(k for k in range(items, items + slots) if k % slots == lw)
            if k >= slots:
                while not empty["K"][k % slots].try_wait(((k // slots) - 1) & 1):
                    yield
            flag_of(k)[k % slots] = "none"
            bar_of("K", k).arrive()
        if last is not None:
            while not bar_of("V", last).try_wait(parity(last)):
                yield

    def consumer(g):
        for k in range(g, items + slots * groups if handed else items, groups):
            s = k % slots
            for h in "KV":
                while not bar_of(h, k).try_wait(parity(k)):
                    yield
                if handed and h == "K" and flag_of(k)[s] == "none":
                    assert k >= items
                    return
                if data[h][s] != k:
                    raise AssertionError(f"item {k}: {h} holds {data[h][s]}")
                reading[h][s] = k
                for _ in range(rng.randint(0, 4)):
                    yield
                reading[h][s] = None
                empty[h][s].arrive()
                if h == "K":                             # the softmax still reads the flags
                    for _ in range(rng.randint(0, 4)):
                        yield
                    if flag_of(k)[s] != k:
                        raise AssertionError(f"item {k}: flags of {flag_of(k)[s]}")

    progs = [loader(i) for i in range(slots)] + [consumer(g) for g in range(groups)]
    live = list(range(len(progs)))
    for _ in range(200000):
        if not live and not pending:
            return "ok"
        if pending and (not live or rng.random() < 0.3):
            h, s, k, bar = pending.pop(rng.randrange(len(pending)))
            if reading[h][s] is not None:
                raise AssertionError(f"{h} of item {k} lands while item {reading[h][s]} is read")
            data[h][s] = k
            bar.complete_tx(1)
            continue
        j = rng.choice(live)
        try:
            next(progs[j])
        except StopIteration:
            live.remove(j)
    return "stuck"


@pytest.mark.parametrize("slots,groups", [(3, 2), (1, 1)])
@pytest.mark.parametrize("items", [1, 2, 5, 7, 13, 40])
def test_ring_of_halves(slots, groups, items):
    for seed in range(150):
        assert _run(slots, groups, items, seed) == "ok", f"seed={seed}"


@pytest.mark.parametrize("items", [0, 1, 2, 3, 4, 5, 6, 7, 13, 40])
def test_items_handed_on(items):
    for slots in (3, 2):
        for seed in range(150):
            assert _run(slots, 2, items, seed, handed=True) == "ok", f"slots={slots} seed={seed}"


def test_the_model_catches_a_single_flag_set():
    broke = 0
    for seed in range(400):
        try:
            _run(3, 2, 24, seed, flag_sets=1)
        except AssertionError:
            broke += 1
    assert broke > 0
