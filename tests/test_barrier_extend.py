"""A CPU model of the windowed extend kernel's protocol (csrc/attention_extend.cu)
under random interleavings: a loading warp, consumer warps that each go at their own
pace (p.V of a chunk, then q.k of the next; one without rows only gives the buffers
back), two buffers of K and of V with "full" and "empty" barriers, row flags in four
sets. Checked: no deadlock, also where a copy never lands and the waits run out;
every buffer and flag set that is read holds the reader's chunk; nothing lands in
what is being read. The form with two flag sets has to break."""
import random

import pytest

from test_barrier_protocols import _Bar

STAGES, WARPS = 2, 4                     # buffers; consumer warps (the kernel has eight), the last one without rows


def _run(chunks, seed, flag_sets=4, lost=None):
    """lost: the chunk whose V never lands; waits then give up once the abort flag is set."""
    rng = random.Random(seed)
    full = {h: [_Bar(1) for _ in range(STAGES)] for h in "KV"}
    empty = {h: [_Bar(WARPS) for _ in range(STAGES)] for h in "KV"}
    data = {h: [None] * STAGES for h in "KV"}
    readers = {h: [0] * STAGES for h in "KV"}
    flags = [None] * flag_sets
    pending, abort = [], [False]

    def wait(bar, parity):
        tries = 0
        while not bar.try_wait(parity):
            tries += 1
            if abort[0] or (lost is not None and tries > 3000):
                abort[0] = True
                yield False
                return
            yield None
        yield True

    def until(gen):
        for r in gen:
            if r is not None:
                return r
            yield
        return True

    def loader():
        for c in range(chunks):
            s = c % STAGES
            for h in "KV":
                if c >= STAGES:
                    if not (yield from until(wait(empty[h][s], (c // STAGES - 1) & 1))):
                        return
                if h == "K":
                    flags[c % flag_sets] = c
                full[h][s].arrive(tx=1)
                if not (h == "V" and c == lost):
                    pending.append((h, s, c))
                yield

    def take(h, c, steps):
        s = c % STAGES
        ok = yield from until(wait(full[h][s], (c // STAGES) & 1))
        if ok and not abort[0] and data[h][s] != c:      # (after an abort the output counts for nothing)
            raise AssertionError(f"chunk {c}: {h} holds {data[h][s]}")
        readers[h][s] += 1
        for _ in range(rng.randint(0, steps)):
            yield
        readers[h][s] -= 1
        empty[h][s].arrive()

    def warp(i):
        if i == WARPS - 1:                                        # no rows
            for c in range(chunks):
                yield from take("K", c, 0)
                yield from take("V", c, 0)
            return
        yield from take("K", 0, 3)
        for c in range(chunks):
            for _ in range(rng.randint(0, 5)):                    # softmax, with the row flags
                yield
            if not abort[0] and flags[c % flag_sets] != c:
                raise AssertionError(f"chunk {c}: flags of {flags[c % flag_sets]}")
            yield from take("V", c, 3)
            if c + 1 < chunks:
                yield from take("K", c + 1, 3)

    progs = [loader()] + [warp(i) for i in range(WARPS)]
    live = list(range(len(progs)))
    for _ in range(400000):
        if not live and not pending:
            return "ok"
        if pending and (not live or rng.random() < 0.2):
            h, s, c = pending.pop(rng.randrange(len(pending)))
            if readers[h][s] and not abort[0]:
                raise AssertionError(f"{h} of chunk {c} lands in a buffer that is read")
            data[h][s] = c
            full[h][s].complete_tx(1)
            continue
        if not live:
            break
        j = rng.choice(live)
        try:
            next(progs[j])
        except StopIteration:
            live.remove(j)
    return "stuck"


@pytest.mark.parametrize("chunks", [1, 2, 3, 4, 7, 20])
def test_protocol(chunks):
    for seed in range(60):
        assert _run(chunks, seed) == "ok", f"seed={seed}"


@pytest.mark.parametrize("lost", [0, 1, 4, 6])
def test_a_copy_that_never_lands_ends_the_kernel(lost):
    for seed in range(3):
        assert _run(7, seed, lost=lost) == "ok", f"seed={seed}"


def test_the_model_catches_too_few_flag_sets():
    broke = 0
    for seed in range(200):
        try:
            _run(20, seed, flag_sets=2)
        except AssertionError:
            broke += 1
    assert broke > 0
