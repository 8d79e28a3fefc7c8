"""The rings of stages of the layer for a few tokens, as a model on the host.

A producer fills slots in order, each once its last fill has been taken; copies land in any order.  Two groups of warps
take the fills in turn and wait for a barrier's parity.  With a barrier for each slot and group, every fill that a
barrier tells of is waited for.  With one barrier a slot, a ring of an odd number of slots gives the groups a slot's fills
in turn, and a group that waits for its next fill is let through while the other group's fill is still in flight."""
import random

import pytest


class Barrier:
    def __init__(self, count):
        self.count = self.left = count
        self.phase = self.bytes = 0

    def turn(self):
        if self.left == 0 and self.bytes == 0:
            self.left, self.phase = self.count, self.phase ^ 1

    def arrive(self):
        self.left -= 1
        assert self.left >= 0
        self.turn()

    def over(self, parity):
        return self.phase != parity


def run(seed, slots, groups, own, fills=40):
    """True if each fill was taken after it had landed."""
    rng = random.Random(seed)
    full = [[Barrier(1) for _ in range(slots)] for _ in range(groups if own else 1)]
    empty = [Barrier(1) for _ in range(slots)]
    landed, flying, issued, taken = set(), [], 0, list(range(groups))  # taken[g]: the next fill of group g

    def bar(n):
        return full[n % groups if own else 0][n % slots]

    def phase(n):  # as fill_phase() of the kernel
        return (n // slots >> 1 if own and groups == 2 and slots % 2 else n // slots) & 1

    while min(taken) < fills:
        step = rng.randrange(2 + groups)
        if step == 0 and issued < fills and empty[issued % slots].over((issued // slots & 1) ^ 1):
            bar(issued).bytes += 1
            bar(issued).arrive()
            flying.append(issued)
            issued += 1
        elif step == 1 and flying and rng.random() < 0.3:
            n = flying.pop(rng.randrange(len(flying)))
            landed.add(n)
            bar(n).bytes -= 1
            bar(n).turn()
        elif step >= 2 and taken[step - 2] < fills and bar(taken[step - 2]).over(phase(taken[step - 2])):
            n = taken[step - 2]
            if n not in landed:
                return False
            taken[step - 2] += groups
            empty[n % slots].arrive()
    return True


@pytest.mark.parametrize("groups", [1, 2])
@pytest.mark.parametrize("slots", range(2, 9))
def test_barriers_of_each_group(slots, groups):
    assert all(run(seed, slots, groups, own=True) for seed in range(200))


@pytest.mark.parametrize("slots", [3, 5])
def test_the_model_sees_barriers_that_groups_share(slots):
    assert not all(run(seed, slots, 2, own=False) for seed in range(200))
