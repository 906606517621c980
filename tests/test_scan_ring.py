"""The ring of the gated linear recurrence's scan, modelled on the host: a loader whose copies land in any
order, groups of workers that take tiles in turn, carriers, and barriers that tell phases apart by
their parity alone.  A worker that passes its wait must find its own tile in the stage, landed."""
import os
import random
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "gated_delta_rule_75_b200", "csrc")


class Barrier:
    def __init__(self, count):
        self.count, self.left, self.phase = count, count, 0

    def arrive(self):
        self.left -= 1
        assert self.left >= 0
        if self.left == 0:
            self.left, self.phase = self.count, self.phase + 1

    def passed(self, parity):
        return (self.phase & 1) != parity


def simulate(NS, aggregators, finishers, tiles, taken_first, seed):
    """Runs the ring to its end under a random schedule.  Returns what went wrong, or None."""
    rng = random.Random(seed)
    stage = [dict(tile=None, landed=False, taken=Barrier(1), full=Barrier(2), agg=Barrier(1), carried=Barrier(1),
                  empty=Barrier(1)) for _ in range(NS)]
    wrong, in_flight = [], []

    def loader():
        ends, q = 0, 0
        while ends < NS - 1:
            s = stage[q % NS]
            while q >= NS and not s["empty"].passed((q // NS - 1) & 1):
                yield
            s["tile"], s["landed"] = (q if q < tiles else -1), q >= tiles
            s["taken"].arrive()
            if q < tiles:
                in_flight.append(s)
            else:
                s["full"].arrive()
                ends += 1
            s["full"].arrive()
            q += 1
            yield

    def tile_of(s, q):
        parity = (q // NS) & 1
        if taken_first:
            while not s["taken"].passed(parity):
                yield
        while not s["full"].passed(parity):
            yield
        if s["tile"] >= 0 and (s["tile"] != q or not s["landed"]):
            wrong.append((q, s["tile"], s["landed"]))
        return s["tile"] >= 0

    def aggregator(g):
        q = g
        while True:
            s = stage[q % NS]
            if not (yield from tile_of(s, q)):
                return
            s["agg"].arrive()
            q += aggregators
            yield

    def carrier(c):
        q = c
        while True:
            s = stage[q % NS]
            while not s["taken"].passed((q // NS) & 1):
                yield
            if s["tile"] < 0:
                return
            if s["tile"] != q:
                wrong.append(("carrier", q, s["tile"]))
            while not s["agg"].passed((q // NS) & 1):
                yield
            s["carried"].arrive()
            q += NS - 1
            yield

    def finisher(g):
        q = g
        while True:
            s = stage[q % NS]
            if not (yield from tile_of(s, q)):
                return
            while not s["carried"].passed((q // NS) & 1):
                yield
            s["empty"].arrive()
            q += finishers
            yield

    threads = [loader()] + [aggregator(g) for g in range(aggregators)] + [carrier(c) for c in range(NS - 1)] \
        + [finisher(g) for g in range(finishers)]
    slow = None
    for step in range(2000 * (tiles + NS)):
        if not threads or wrong:
            break
        t = rng.choice(threads)
        try:
            next(t)
        except StopIteration:
            threads.remove(t)
        # now and then one copy is much later than those asked for after it
        if slow is not None and slow not in in_flight:
            slow = None
        if in_flight and rng.random() < 0.5:
            s = rng.choice(in_flight)
            if slow is None and rng.random() < 0.2:
                slow = s
            if s is not slow or rng.random() < 0.005:
                in_flight.remove(s)
                s["landed"] = True
                s["full"].arrive()
    return wrong[0] if wrong else ("stuck", len(threads)) if threads else None


RINGS = [(8, 3, 2), (7, 3, 2), (6, 3, 2), (5, 3, 2), (6, 2, 2), (5, 2, 2), (4, 2, 2), (3, 2, 2)]     # stages, groups


def test_every_worker_finds_its_own_tile():
    for ring in RINGS:
        for seed in range(12):
            assert simulate(*ring, tiles=60, taken_first=True, seed=seed) is None, (ring, seed)


def test_the_wait_for_the_copies_alone_is_passed_early():
    """The model sees the fault: with eight stages and three groups a group may begin a wait two phases early."""
    found = [simulate(8, 3, 2, tiles=60, taken_first=False, seed=s) for s in range(60)]
    assert any(found)


def test_the_kernel_waits_as_the_model_does():
    with open(os.path.join(CSRC, "kda_glr.cu")) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    helper = re.search(r"bool await_tile\([^)]*\)\s*\{(.*?)\n\}", code, re.S).group(1)
    assert re.search(r"mbar_wait\(&s\.taken.*&&.*mbar_wait\(&s\.full", helper, re.S)
    for role in ("scan_aggregate", "scan_finish"):
        body = re.search(r"void %s\(.*?\n\}\n" % role, code, re.S).group(0)
        assert "await_tile(" in body and "s.full" not in body, role
    carry = re.search(r"void scan_carry\(.*?\n\}\n", code, re.S).group(0)
    assert carry.index("s.taken") < carry.index("s.agg") and "s.full" not in carry


def test_the_fold_reads_the_other_runs_in_order():
    """Lane 0 alone counts the runs that are there; a shuffle hands the count on but orders no memory, so the
    lanes that read the other runs meet at __syncwarp() first."""
    with open(os.path.join(CSRC, "kda_glr.cu")) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    fold = re.search(r"__shfl_sync\([^)]*before, 0\) == kRuns - 1\) \{(.*?)s\.A\[", code, re.S).group(1)
    assert fold.lstrip().startswith("__syncwarp();")
