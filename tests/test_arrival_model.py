"""The protocol by which the last of several workgroups of a launch is found (arrive and leave in
argreduce_logits_device.hpp), as a model on the CPU: every access to scratch is a step of its own, workgroups' steps are
interleaved at random, and between two launches with the same tag (replays of one captured call) scratch may change in
any way that a program's other kernels can change it."""
import random

import pytest

TAG, CONSTANT = 0x5EED, 7


class Launch:
    """One launch over `mem` (a list of words): an owner, slots and parts, in one level or in sets of `most` workgroups
    whose parts are joined by the last set's."""

    def __init__(self, mem, blocks, value, rng, most=None, counted=False):
        self.mem, self.blocks, self.value, self.rng, self.counted = mem, blocks, value, rng, counted
        self.most = most or blocks
        self.sets = -(-blocks // self.most)
        # where everything lies; `counted`: word 0 is a generation, part of the tag, and nothing is cleared
        self.owners = 1
        self.slots = self.owners + self.sets
        self.last = self.slots + blocks
        self.set_slots = self.last + 1
        self.parts = self.set_slots + self.sets
        self.set_parts = self.parts + blocks
        self.joined = []

    @staticmethod
    def words(blocks, most=None):
        sets = -(-blocks // (most or blocks))
        return 1 + sets + blocks + 1 + sets + blocks + sets

    def tag(self, generation):
        return (TAG, generation) if self.counted else TAG

    def arrive(self, owner, slots, mine, n, tag, store):
        """Generator: a step per access. Returns whether this workgroup is the last of n."""
        stores = [store]
        if mine == 0 and not self.counted:
            stores.append((owner, 0))
        self.rng.shuffle(stores)  # they are done before the slot is stored, in any order
        for at, value in stores:
            yield
            self.mem[at] = value
        yield
        self.mem[slots + mine] = tag
        there = True
        for i in self.rng.sample(range(n), n):
            yield
            there &= self.mem[slots + i] == tag
        if not there:
            return False
        yield
        taken = tag if self.counted else -TAG
        before, self.mem[owner] = self.mem[owner], taken
        return before != taken

    def workgroup(self, b):
        yield
        generation = self.mem[0]
        tag = self.tag(generation)
        s = b // self.most
        first = s * self.most
        n = min(self.most, self.blocks - first)
        if not (yield from self.arrive(self.owners + s, self.slots + first, b - first, n, tag,
                                       (self.parts + b, (self.value, b)))):
            return
        found = yield from self.read(self.parts + first, n)
        if self.sets > 1:
            if not (yield from self.arrive(self.last, self.set_slots, s, self.sets, tag,
                                           (self.set_parts + s, found))):
                return
            found = sum((yield from self.read(self.set_parts, self.sets)), [])
        self.joined.append(sorted(found, key=str))
        if self.counted:
            yield
            self.mem[0] = generation + 1
        else:
            yield from self.leave(self.slots, self.blocks)
            if self.sets > 1:
                yield from self.leave(self.set_slots, self.sets)

    def read(self, at, n):
        out = [None] * n
        for i in self.rng.sample(range(n), n):
            yield
            out[i] = self.mem[at + i]
        return out

    def leave(self, slots, n):
        for i in self.rng.sample(range(n), n):
            yield
            self.mem[slots + i] = 0

    def run(self):
        """Whether exactly one workgroup joined, and what it joined were this launch's parts."""
        running = [self.workgroup(b) for b in range(self.blocks)]
        self.rng.shuffle(running)
        pace = [self.rng.random() ** 4 + 1e-3 for _ in running]  # some far behind the others
        while running:
            i = self.rng.choices(range(len(running)), pace)[0]
            for _ in range(self.rng.randint(1, 9)):
                try:
                    next(running[i])
                except StopIteration:
                    del running[i], pace[i]
                    break
        return self.joined


def replays(blocks, most, kind, counted, seed, count):
    rng = random.Random(seed)
    size = Launch.words(blocks, most)
    mem = [rng.getrandbits(64) for _ in range(size)]
    cut = rng.randint(1, size)
    snapshot, wrong = None, {"stale": 0, "none": 0, "twice": 0}
    for value in range(count):
        want = sorted([(value, b) for b in range(blocks)], key=str)
        launch = Launch(mem, blocks, value, rng, most, counted)
        found = launch.run()
        wrong["none"] += not found
        wrong["twice"] += len(found) > 1
        wrong["stale"] += any(f != want for f in found)
        if kind == "word 0":
            mem[0] = CONSTANT
        elif kind == "a prefix":
            mem[:cut] = [CONSTANT] * cut
        elif kind == "a range":
            a = rng.randrange(size)
            b = rng.randint(a, size)
            mem[a:b] = [CONSTANT] * (b - a)
        elif kind == "garbage":
            mem[:] = [rng.getrandbits(64) for _ in range(size)]
        elif kind == "copies of its words":
            mem[:] = [rng.choice(mem) for _ in range(size)]
        elif kind == "as it was":
            snapshot = list(mem) if snapshot is None else snapshot
            mem[:] = snapshot
    return wrong


SHAPES = [(2, None), (5, None), (16, None), (40, None), (9, 4), (30, 8)]
KINDS = ["nothing", "word 0", "a prefix", "a range", "garbage", "copies of its words", "as it was"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("blocks,most", SHAPES)
def test_one_workgroup_joins_this_launchs_parts(blocks, most, kind):
    for seed in range(6):
        wrong = replays(blocks, most, kind, False, seed, 60 if blocks < 20 else 20)
        assert wrong == {"stale": 0, "none": 0, "twice": 0}, (seed, wrong)


def test_the_model_sees_a_tag_that_rests_on_scratch():
    """A generation in scratch as all that tells two replays apart: once something else has put it back, nobody joins,
    or a workgroup joins before the others have stored."""
    stale = none = 0
    for seed in range(40):
        wrong = replays(16, None, "word 0", True, seed, 20)
        none += wrong["none"]
        wrong = replays(16, None, "a prefix", True, seed, 20)
        stale += wrong["stale"]
    assert none > 100 and stale > 20
    assert replays(16, None, "nothing", True, 0, 50) == {"stale": 0, "none": 0, "twice": 0}
