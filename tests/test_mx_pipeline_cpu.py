"""Host model of the barrier protocol of the microscaled product's kernels.

Every role of every CTA is a generator that yields the waits of the kernel's
code; copies land and MMAs finish (in order) as events of their own, and a
scheduler picks among everything that can go on, at random, with random
weights, so that some roles lag far behind.  Barriers are waited for by
parity, as the hardware has it, and count bytes that may land before they are
expected.  Checked: every run ends with every role done; an MMA reads a stage
only while both CTAs' halves of its chunk are there, and no copy starts into a
stage that an MMA has yet to read; sums are read when all of a tile's MMAs are
done and none of the next has begun.
"""
import os
import random
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "expert_ffn_execution_b200", "csrc")


class Barrier:
    def __init__(self, count):
        self.count = self.left = count
        self.tx, self.phase = 0, 0

    def change(self, arrivals=0, tx=0):
        assert arrivals <= self.left, "an arrival too many"
        self.left -= arrivals
        self.tx += tx
        if self.left == 0 and self.tx == 0:
            self.left, self.phase = self.count, self.phase + 1

    def done(self, parity):  # the phase of that parity is complete
        return self.phase % 2 != parity


def run(rng, roles, events):
    """Runs the generators; `events` is the list of callables that may happen
    next, to which everything here appends."""
    weight = {i: rng.choice([1, 1, 4, 16]) for i in range(len(roles))}
    waits = {i: next(r, None) for i, r in enumerate(roles)}
    while any(w is not None for w in waits.values()) or events:
        ready = [i for i, w in waits.items() if w is not None and w[0].done(w[1])]
        pick = rng.choices(ready + [-1] * bool(events), [weight[i] for i in ready] + [8] * bool(events))[0] \
            if ready or events else None
        assert pick is not None, "deadlock"
        if pick == -1:
            events.pop(rng.randrange(len(events)))()
        else:
            waits[pick] = next(roles[pick], None)


class Pipe:
    """What a tensor core does for one thread: MMAs and commits, in order."""

    def __init__(self, events):
        self.queue, self.events, self.busy = [], events, False

    def put(self, *acts):
        self.queue += acts
        self.kick()

    def kick(self):
        if self.queue and not self.busy:
            self.busy = True
            self.events.append(self.step)

    def step(self):
        self.queue.pop(0)()
        self.busy = False
        self.kick()


def pair_kernel(rng, S, tiles, chunks, warps):
    """mx_gemm_kernel: two CTAs, copies of both counted on the even one's
    barriers, MMAs of both issued by it."""
    events = []
    full, tempty = [Barrier(1) for _ in range(S)], Barrier(2 * warps)
    empty = [[Barrier(1) for _ in range(S)] for _ in range(2)]
    tfull = [Barrier(1) for _ in range(2)]
    there = [[None] * S for _ in range(2)]  # the chunk a stage holds
    read, begun, done, seen = set(), [0], [0], [[0] * warps for _ in range(2)]
    pipe = Pipe(events)

    def producer(r):
        i = 0
        for _ in range(tiles):
            for _ in range(chunks):
                s = i % S
                yield empty[r][s], (i // S & 1) ^ 1
                if r == 0:
                    full[s].change(1, 2)
                assert i < S or i - S in read, "a copy into a stage that is still to be read"

                def land(s=s, i=i):
                    there[r][s] = i
                    full[s].change(0, -1)
                events.append(land)
                i += 1

    def issuer():
        i = 0
        for t in range(tiles):
            yield tempty, (t & 1) ^ 1
            for c in range(chunks):
                s = i % S
                yield full[s], i // S & 1

                def mma(s=s, i=i, t=t, c=c):
                    assert there[0][s] == there[1][s] == i, "an MMA of a chunk that is not there"
                    assert c or all(n == t for cta in seen for n in cta), "sums overwritten before they were read"
                    begun[0] = t + 1
                    read.add(i)
                pipe.put(mma, lambda s=s: [empty[r][s].change(1) for r in range(2)])
                i += 1
            pipe.put(lambda t=t: done.__setitem__(0, t + 1), lambda: [b.change(1) for b in tfull])

    def reader(r, w):
        for t in range(tiles):
            yield tfull[r], t & 1
            assert done[0] == t + 1 and begun[0] == t + 1, "sums read too early or too late"
            seen[r][w] = t + 1
            events.append(lambda: tempty.change(1))

    run(rng, [producer(0), producer(1), issuer()] + [reader(r, w) for r in range(2) for w in range(warps)], events)
    assert all(n == tiles for cta in seen for n in cta) and len(read) == tiles * chunks


def split_kernel(rng, S, chunks, splits, nt):
    """mx_linear_kernel: `splits` ranks, each its chunks, then each rank's sums
    of the tokens another joins in one copy to it."""
    events, roles = [], []
    per = -(-nt // splits)
    mine = [max(0, min(per, nt - r * per)) for r in range(splits)]
    assert sum(mine) == nt
    joined, started, got = [Barrier(1) for _ in range(splits)], Barrier(splits), [0] * splits

    def rank(r):
        n = chunks * (r + 1) // splits - chunks * r // splits
        assert n >= 1
        full, empty = [Barrier(1) for _ in range(S)], [Barrier(1) for _ in range(S)]
        tfull, pipe, there, read = Barrier(1), Pipe(events), [None] * S, set()
        joined[r].change(1, mine[r] * splits)
        events.append(lambda: started.change(1))

        def producer():
            for i in range(n):
                s = i % S
                yield empty[s], (i // S & 1) ^ 1
                assert i < S or i - S in read
                full[s].change(1, 1)

                def land(s=s, i=i):
                    there[s] = i
                    full[s].change(0, -1)
                events.append(land)

        def issuer():
            for i in range(n):
                s = i % S
                yield full[s], i // S & 1

                def mma(s=s, i=i):
                    assert there[s] == i
                    read.add(i)
                pipe.put(mma, lambda s=s: empty[s].change(1))
            pipe.put(lambda: tfull.change(1))

        def joiner():
            yield tfull, 0
            assert len(read) == n
            if splits == 1:
                return
            yield started, 0  # the cluster's barrier
            for to in range(splits):
                count = min(per, nt - to * per)
                if count > 0:
                    def land(to=to, count=count):
                        got[to] += count
                        joined[to].change(0, -count)
                    events.append(land)
            yield joined[r], 0
            assert got[r] == mine[r] * splits, "sums joined before they were there"

        return [producer(), issuer(), joiner()]

    for r in range(splits):
        roles += rank(r)
    run(rng, roles, events)


@pytest.mark.parametrize("S", [3, 4, 5, 6])
@pytest.mark.parametrize("tiles,chunks", [(1, 1), (3, 1), (2, 5), (4, 7), (2, 16)])
def test_pairs(S, tiles, chunks):
    for seed in range(60):
        pair_kernel(random.Random(seed), S, tiles, chunks, 2)


@pytest.mark.parametrize("splits", [1, 2, 4, 8])
@pytest.mark.parametrize("nt", [1, 3, 4, 16, 33, 64])
def test_splits(splits, nt):
    for seed in range(30):
        for chunks in (2 * splits, 2 * splits + 1, 5 * splits + 3):
            split_kernel(random.Random(seed), 3, chunks, splits, nt)


def test_the_model_finds_a_missing_wait():
    """A producer one stage too far ahead is flagged."""
    class Early(Barrier):
        def done(self, parity):
            return True
    real = globals()["Barrier"]
    try:
        globals()["Barrier"] = lambda n: Early(n) if n == 1 else real(n)
        with pytest.raises(AssertionError):
            for seed in range(60):
                pair_kernel(random.Random(seed), 3, 2, 5, 2)
    finally:
        globals()["Barrier"] = real


def test_the_model_is_of_the_kernels():
    """The counts and parities that the model has are the kernels'."""
    gemm = open(os.path.join(CSRC, "mx_gemm.cu")).read()
    for line in ("mbar_init(&full[s], 1);", "mbar_init(&empty[s], 1);", "mbar_init(tfull, 1);",
                 "mbar_init(tempty, 2 * kGEpi);", "mbar_wait_guarded(&empty[s], ph,",
                 "mbar_wait_guarded(&full[s], ph,", "uint32_t ph = 1;", "uint32_t ph = 0;",
                 "if (++s == C::S) s = 0, ph ^= 1u;", "mbar_wait_guarded(tempty, (it & 1) ^ 1",
                 "mbar_wait_guarded(tfull, it & 1", "mma_commit_pair(&empty[s]);", "mma_commit_pair(tfull);"):
        assert line in gemm, line
    linear = open(os.path.join(CSRC, "mx_linear.cu")).read()
    for line in ("mbar_init(&full[threadIdx.x], 1);", "uint32_t ph = 1;", "uint32_t ph = 0;", "if (++s == S) s = 0, ph ^= 1u;",
                 "per = (nt + splits - 1) >> lg_splits;", "mine = max(0, min(per, nt - first));",
                 "(uint32_t)(mine * splits * C::token)", "count = min(per, nt - to * per);"):
        assert line in linear, line
    assert re.search(r"chunks \* \(rank \+ 1\) >> lg_splits\) - c0", linear)
