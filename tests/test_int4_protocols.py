"""CPU models of what the kernels of the 4-bit operators do when a bounded wait runs out: every copy in flight gets
another limit before its CTA leaves, a wait is made only for copies that were started, and all warps leave at the same
place. No GPU: such a wait cannot be made to run out on one without a fault. Each model is also run in the form that
breaks the rule, which pins it to a fault that it must catch."""
import random

import pytest

LIMIT = 1000                          # a bounded wait, in steps


# ------------------------------------------------- rows kernel of the linear

def _rows_cta(segments, stages, tiles, delay, waits):
    """One CTA of gemm_int4_rows_kernel: each segment walks `stages` blocks of each tile through its ring of two; the
    segments meet after a tile. delay(seg, k): steps that the segment's k-th copy takes. waits: "cta" (after a wait ran
    out, every segment waits for the stages between its place and its fill cursor) or "warp" (only the segment whose
    wait ran out does, for two stages). Returns the copies in flight when the CTA gave up, as (landing, end), and the
    step at which its last warp leaves; None where nothing ran out."""
    ring = 2
    seg = [dict(now=0, ft=0, fb=0, n=0, ring=[], ok=True, blk=0) for _ in range(segments)]

    def fill(i, s):
        if s["ft"] >= tiles:
            return
        s["ring"].append(s["now"] + delay(i, s["n"]))
        s["n"] += 1
        s["fb"] += 1
        if s["fb"] == stages:
            s["fb"], s["ft"] = 0, s["ft"] + 1

    for i, s in enumerate(seg):
        for _ in range(ring):
            fill(i, s)
    for tile in range(tiles):
        for i, s in enumerate(seg):
            s["blk"] = 0
            while s["blk"] < stages:
                if s["ring"][0] > s["now"] + LIMIT:
                    s["now"] += LIMIT
                    s["ok"] = False
                    break
                s["now"] = max(s["now"], s["ring"].pop(0)) + 1
                fill(i, s)
                s["blk"] += 1
        meet = max(s["now"] for s in seg)
        for s in seg:
            s["now"] = meet
        if all(s["ok"] for s in seg):
            continue
        flying = [x for s in seg for x in s["ring"] if x > meet]
        for s in seg:
            started = len(s["ring"])
            n = (s["ft"] - tile) * stages + s["fb"] - s["blk"]       # as the kernel counts them
            assert n == started
            if waits == "cta" or not s["ok"]:
                for x in s["ring"][:n]:
                    s["now"] = min(max(s["now"], x), s["now"] + LIMIT)
        return flying, meet, max(s["now"] for s in seg)
    return None


def _rows_faults(waits):
    """Runs in which a copy that lands within another limit of the give-up lands after the CTA has left."""
    faults = gave_up = 0
    for seed in range(600):
        r = random.Random(seed)
        segments, stages, tiles = r.randint(1, 8), r.randint(1, 6), r.randint(1, 5)
        slow = {(r.randrange(segments), r.randrange(stages * tiles)) for _ in range(r.randint(1, 4))}
        d = lambda i, k: r.randint(LIMIT + 1, 2 * LIMIT) if (i, k) in slow else r.randint(1, 50)
        out = _rows_cta(segments, stages, tiles, d, waits)
        if out is None:
            continue
        flying, meet, left = out
        gave_up += 1
        faults += any(left < x <= meet + LIMIT for x in flying)
    assert gave_up > 100
    return faults


def test_rows_kernel_leaves_no_copy_in_flight():
    assert _rows_faults("cta") == 0


def test_rows_model_catches_waits_of_the_failing_segment_only():
    assert _rows_faults("warp") > 0


# ------------------------------------------- a warp of the split attention

def _split_warp(items, delay, again):
    """One warp of attn_split_int4_kernel: its K and V buffers are filled one item ahead. delay(which, k): steps that the
    copy of item k takes. again: after a wait ran out, its own copy gets another limit too. Returns the copies in flight
    when the wait ran out, that step, and the step at which the warp leaves; None where nothing ran out."""
    now = 0
    copy = {"K": delay("K", 0), "V": delay("V", 0)}       # landing steps

    def wait(which):
        nonlocal now
        ok = copy[which] <= now + LIMIT
        now = max(now, min(copy[which], now + LIMIT))
        return ok

    for k in range(items):
        for which, other in (("K", "V"), ("V", "K")):
            if not wait(which):
                gave_up, flying = now, [copy[which]]
                if which == "K" or k + 1 < items:          # V of this item, or K of the next one
                    flying.append(copy[other])
                if again:
                    wait(which)
                if which == "K" or k + 1 < items:
                    wait(other)
                return flying, gave_up, now
            now += 5                                       # scores; softmax and values
            if k + 1 < items:
                copy[which] = now + delay(which, k + 1)
    return None


def _split_faults(again):
    faults = gave_up = 0
    for seed in range(600):
        r = random.Random(seed)
        items = r.randint(1, 12)
        slow = {(r.choice("KV"), r.randrange(items)) for _ in range(r.randint(1, 3))}
        out = _split_warp(items, lambda w, k: r.randint(LIMIT + 1, 2 * LIMIT) if (w, k) in slow else r.randint(1, 50), again)
        if out is None:
            continue
        flying, at, left = out
        gave_up += 1
        faults += any(left < x <= at + LIMIT for x in flying)
    assert gave_up > 100
    return faults


def test_split_warp_leaves_no_copy_in_flight():
    assert _split_faults(True) == 0


def test_split_model_catches_a_wait_for_the_other_copy_only():
    assert _split_faults(False) > 0


# --------------------------------------------------- the merge of the chunks

def _merge_loader(tiles, ring, lost, early=1):
    """The loading warp of attn_merge_int4_kernel over `tiles` tiles, of which `lost` never lands (None: all do).
    early: after the first tile, a wait's end is seen before that many copies of its turn are started. Returns (tiles
    waited for that were not started, tiles in flight that were not waited for at the exit)."""
    started, unstarted = set(), []

    def factors(t):                                        # waits for tile t
        if t not in started:
            unstarted.append(t)
        return t != lost and t in started

    started.update(range(min(tiles, ring)))
    ok = factors(0)
    for t in range(tiles):
        if not ok:                                         # seen behind the barrier, before the next copy is started
            waited = range(t, min(tiles, t + ring - (early if t > 0 else 0)))
            unstarted += [k for k in waited if k not in started]
            return unstarted, [k for k in started if k >= t and k not in waited]
        if t > 0 and t - 1 + ring < tiles:
            started.add(t - 1 + ring)
        if t + 1 < tiles:
            ok = factors(t + 1)
    return unstarted, []


def test_merge_waits_for_the_tiles_that_were_started():
    for ring in range(2, 9):
        for tiles in range(1, 30):
            for lost in [None, *range(tiles)]:
                assert _merge_loader(tiles, ring, lost) == ([], []), (ring, tiles, lost)


def test_merge_model_catches_a_wait_for_a_tile_that_was_not_started():
    assert _merge_loader(9, 4, 3, early=0) == ([6], [])


def test_merge_needs_two_tiles_of_room():
    """With one, the next tile's factors are wanted before its copy is started: the launch never takes it."""
    assert _merge_loader(1, 1, None) == ([], [])
    assert _merge_loader(2, 1, None)[0]


def _merge_exits(tiles, lost, flags, seed):
    """The iterations at which the merging warps leave, tile `lost` never landing: between the barriers t and t + 1 the
    loading warp sets flag (t + 1) % flags, at any moment, and each merging warp reads flag t % flags, at any moment."""
    r = random.Random(seed)
    failed = [False] * flags
    if lost == 0:
        failed[0] = True
    left = {}
    for t in range(tiles):
        events = [("set", None)] * (t + 1 == lost) + [("read", w) for w in range(4) if w not in left]
        r.shuffle(events)
        for kind, w in events:
            if kind == "set":
                failed[(t + 1) % flags] = True
            elif failed[t % flags]:
                left[w] = t
    return set(left.values())


@pytest.mark.parametrize("lost", [0, 1, 2, 5])
def test_merging_warps_leave_together(lost):
    for seed in range(200):
        assert _merge_exits(6, lost, 2, seed) == {lost}


def test_merge_model_catches_one_flag_for_two_tiles():
    assert any(len(_merge_exits(6, 2, 1, seed)) > 1 for seed in range(200))
