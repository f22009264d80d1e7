"""The protocol of topk_paged_attention's ring of pieces, run step by step on the CPU with the arrivals of asynchronous
copies counted in any order: one copier, a warp that takes the keys' pieces, one that takes the values', and the softmax
between them. A parity wait passes if the phase before the current one has that parity, whichever phase that was."""
import itertools
import os
import random
import re

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_attention_row_gb300", "csrc", "paged_attention.cu")
BARRIERS = 6  # kMaxSlots


class Stale(AssertionError):
    pass


def run(slots, keys, values, tiles, scheme, seed):
    """scheme: "numbers" (barriers of keys' and values' pieces by their number) or "slots" (one barrier a slot, and the
    scores wait for the last tile's values where those fill the ring)."""
    rng = random.Random(seed)
    per = keys + values
    done = {}                 # barrier -> phases completed
    landed, counted = set(), []  # items copied, arrivals not yet counted
    freed = [0] * slots       # times each slot was given back
    scored, read, multiplied, probable = [0], [0], [0], [0]  # tiles

    def barrier(item):
        tile, u = divmod(item, per)
        if scheme == "slots":
            return ("slot", item % slots), item // slots
        if u < keys:
            n = tile * keys + u
            return ("key", n % BARRIERS), n // BARRIERS
        n = tile * values + u - keys
        return ("value", n % BARRIERS), n // BARRIERS

    def come(item):
        """A parity wait for the item's barrier; what passes has to have come."""
        b, phase = barrier(item)
        if done.get(b, 0) % 2 == phase % 2:
            return False
        if item not in landed:
            raise Stale(f"item {item} of {slots} slots, {keys} keys, {values} values")
        return True

    def copier():
        for item in range(tiles * per):
            while freed[item % slots] < item // slots:
                yield
            counted.append(item)
            yield

    def scores():
        for t in range(tiles):
            while read[0] < t - 1:  # two places for the scores
                yield
            if scheme == "slots" and t > 0 and slots <= values:
                while multiplied[0] < t:
                    yield
            for u in range(keys):
                while not come(t * per + u):
                    yield
                freed[(t * per + u) % slots] += 1
                yield
            scored[0] = t + 1

    def softmax():
        for t in range(tiles):
            while scored[0] <= t:
                yield
            read[0] = t + 1
            yield
            while multiplied[0] < t - 1:  # two places for the probabilities
                yield
            probable[0] = t + 1
            yield

    def products():
        for t in range(tiles):
            while probable[0] <= t:
                yield
            for u in range(values):
                while not come(t * per + keys + u):
                    yield
                freed[(t * per + keys + u) % slots] += 1
                yield
            multiplied[0] = t + 1

    agents = [copier(), scores(), softmax(), products()]
    idle = 0
    while agents:
        before = (tuple(freed), len(landed), scored[0], read[0], multiplied[0], probable[0], len(counted), len(agents))
        if counted and rng.random() < 0.3:
            item = counted.pop(rng.randrange(len(counted)))
            landed.add(item)
            b, _ = barrier(item)
            done[b] = done.get(b, 0) + 1
        else:
            agent = rng.choice(agents)
            for _ in range(rng.choice([1, 1, 5, 20])):
                try:
                    next(agent)
                except StopIteration:
                    agents.remove(agent)
                    break
        after = (tuple(freed), len(landed), scored[0], read[0], multiplied[0], probable[0], len(counted), len(agents))
        idle = idle + 1 if before == after else 0
        assert idle < 2000, "no one can go on"


SHAPES = [(s, k, v) for s, k, v in itertools.product(range(2, 7), range(1, 6), range(1, 5))]


def test_pieces_by_number_are_never_taken_early():
    for slots, keys, values in SHAPES:
        for seed in range(6):
            run(slots, keys, values, 9, "numbers", seed)


@pytest.mark.parametrize("slots, keys, values", [(3, 1, 1), (5, 1, 1), (3, 2, 2), (5, 2, 4)])
def test_the_model_sees_a_piece_taken_early(slots, keys, values):
    # one barrier a slot: a wait for keys may pass on the phase before the values that had the slot last
    with pytest.raises(Stale):
        for seed in range(3000):
            run(slots, keys, values, 9, "slots", seed)


def test_the_kernel_waits_by_number():
    text = re.sub(r"//[^\n]*", "", open(SOURCE).read())
    assert int(re.search(r"kMaxSlots = (\d+);", text).group(1)) == BARRIERS
    assert len(re.findall(r"mbar_wait_warp\(come \+ keys\.slot \* 8, keys\.phase, guard\);\s*keys\.step\(kMaxSlots\);", text)) == 2
    assert len(re.findall(r"mbar_wait_warp\(come \+ values\.slot \* 8, values\.phase, guard\);\s*values\.step\(kMaxSlots\);", text)) == 1
    assert len(re.findall(r"copies_arrive\(smem_addr\(come \+ number\.slot\)\);", text)) == 1
    assert not re.search(r"\bfull \+ at\.slot", text)
