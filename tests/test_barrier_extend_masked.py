"""The CPU model of test_barrier_extend.py with the chunks that are masked for some token of the tile
(csrc/attention_extend.cu): their V lands on a barrier of the loading warp's own, counted by phases of its own; the warp
waits for it, zeroes and looks through rows, says whether p.V has to run token by token, and only then fills the
consumers' barrier. Checked under random interleavings and mixes of masked and other chunks: no deadlock, also where a
copy of either kind of chunk never lands; every buffer that is read holds the reader's chunk, looked through where it is
masked, with the flag of that chunk; nothing lands in, or is zeroed in, what is being read; no copy is on its way
when the kernel ends in good order. Three broken forms have to fail."""
import random

import pytest

from test_barrier_protocols import _Bar

STAGES, WARPS, FLAG_SETS = 2, 4, 4       # buffers; consumer warps (the kernel has eight), the last one without rows
LIMIT = 3000                             # tries of a wait, where a copy is lost


def _run(masked, seed, lost=None, broken=None):
    """masked: of each chunk. lost: (half, chunk) of a copy that never lands; waits then give up once the abort flag is
    set. broken: "parity" (the own barrier's phase taken from the chunk), "early" (the consumers' barrier filled before the
    look), "flag" (the flag written after it)."""
    chunks, rng = len(masked), random.Random(seed)
    full = {h: [_Bar(1) for _ in range(STAGES)] for h in "KV"}
    empty = {h: [_Bar(WARPS) for _ in range(STAGES)] for h in "KV"}
    land = _Bar(1)
    data = {h: [None] * STAGES for h in "KV"}              # (chunk, looked through or not masked)
    readers = {h: [0] * STAGES for h in "KV"}
    odd, flags, pending, abort = [None] * STAGES, [None] * FLAG_SETS, [], [False]

    def wait(bar, parity, limit=False):
        """limit: a wait that the abort flag does not end, but its own limit does."""
        tries = 0
        while not bar.try_wait(parity):
            tries += 1
            if (abort[0] and not limit) or (lost is not None and tries > LIMIT):
                abort[0] = True
                return False
            yield
        return True

    def issue(h, s, c, bar):
        bar.arrive(tx=1)
        if (h, c) != lost:
            pending.append((h, s, c, bar))

    def loader():
        lands, last = 0, {"K": -1, "V": -1}
        for c in range(chunks):
            s = c % STAGES
            if c >= STAGES and not (yield from wait(empty["K"][s], (c // STAGES - 1) & 1)):
                break
            flags[c % FLAG_SETS] = c
            issue("K", s, c, full["K"][s])
            last["K"] = c
            yield
            if c >= STAGES and not (yield from wait(empty["V"][s], (c // STAGES - 1) & 1)):
                break
            if not masked[c]:
                odd[s] = c
                yield
                issue("V", s, c, full["V"][s])
            else:
                issue("V", s, c, land)
                yield
                ok = yield from wait(land, (c if broken == "parity" else lands) & 1)
                lands += 1
                if not ok:
                    yield from wait(land, (lands - 1) & 1, limit=True)
                    break
                if broken == "early":
                    full["V"][s].arrive()
                for _ in range(rng.randint(1, 6)):         # zeroes and looks
                    if readers["V"][s] and not abort[0]:
                        raise AssertionError(f"V of chunk {c} is changed while it is read")
                    if data["V"][s] is None or data["V"][s][0] != c:
                        raise AssertionError(f"chunk {c}: looks through V of {data['V'][s]}")
                    yield
                data["V"][s] = (c, True)
                if broken != "flag":
                    odd[s] = c
                yield
                if broken != "early":
                    full["V"][s].arrive()
                if broken == "flag":
                    yield
                    odd[s] = c
            last["V"] = c
            yield
        for d in range(STAGES):                            # the last copies
            for h in "KV":
                if last[h] - d >= 0:
                    yield from wait(full[h][(last[h] - d) % STAGES], ((last[h] - d) // STAGES) & 1, limit=True)
        if lost is None and any(h in "KV" for h, _, _, _ in pending):
            raise AssertionError("a copy is on its way when the loading warp leaves")

    def take(h, c, steps):
        s = c % STAGES
        ok = yield from wait(full[h][s], (c // STAGES) & 1)
        if not ok:
            abort[0] = True
        if not abort[0]:
            if data[h][s] != (c, True):
                raise AssertionError(f"chunk {c}: {h} holds {data[h][s]}")
            if h == "V" and odd[s] != c:
                raise AssertionError(f"chunk {c}: flag of {odd[s]}")
        readers[h][s] += 1
        for _ in range(rng.randint(0, steps)):
            yield
            if not abort[0] and data[h][s] != (c, True):
                raise AssertionError(f"chunk {c}: {h} became {data[h][s]}")
        readers[h][s] -= 1
        empty[h][s].arrive()

    def warp(i):
        if i == WARPS - 1:                                 # no rows
            for c in range(chunks):
                yield from take("K", c, 0)
                yield from take("V", c, 0)
            return
        yield from take("K", 0, 3)
        for c in range(chunks):
            for _ in range(rng.randint(0, 5)):             # softmax, with the row flags
                yield
            if not abort[0] and flags[c % FLAG_SETS] != c:
                raise AssertionError(f"chunk {c}: flags of {flags[c % FLAG_SETS]}")
            yield from take("V", c, 9 if masked[c] else 3)  # (token by token: longer)
            if c + 1 < chunks:
                yield from take("K", c + 1, 3)

    progs = [loader()] + [warp(i) for i in range(WARPS)]
    live = list(range(len(progs)))
    for _ in range(400000):
        if not live and not pending:
            return "ok"
        if pending and (not live or rng.random() < 0.2):
            h, s, c, bar = pending.pop(rng.randrange(len(pending)))
            if readers[h][s] and not abort[0]:
                raise AssertionError(f"{h} of chunk {c} lands in a buffer that is read")
            data[h][s] = (c, h == "K" or not masked[c])
            bar.complete_tx(1)
            continue
        j = rng.choice(live)
        try:
            next(progs[j])
        except StopIteration:
            live.remove(j)
    return "stuck"


def mixes(n, seed):
    """As a window makes them (the ends masked), all, none, any."""
    r = random.Random(seed)
    return [[i == 0 or i >= n - 2 for i in range(n)], [True] * n, [False] * n, [r.random() < 0.5 for _ in range(n)]]


@pytest.mark.parametrize("chunks", [1, 2, 3, 4, 7, 20])
def test_protocol(chunks):
    for seed in range(30):
        for masked in mixes(chunks, seed):
            assert _run(masked, seed) == "ok", f"seed={seed} masked={masked}"


@pytest.mark.parametrize("lost", [("V", 0), ("V", 1), ("V", 4), ("V", 6), ("K", 0), ("K", 3), ("K", 6)])
def test_a_copy_that_never_lands_ends_the_kernel(lost):
    for seed in range(2):
        for masked in mixes(7, seed):
            assert _run(masked, seed, lost=lost) == "ok", f"seed={seed} masked={masked}"


@pytest.mark.parametrize("broken", ["parity", "early", "flag"])
def test_the_model_catches(broken):
    broke = 0
    for seed in range(60):
        for masked in mixes(9, seed):
            try:
                broke += _run(masked, seed, broken=broken) != "ok"
            except AssertionError:
                broke += 1
    assert broke > 0
