"""The ring of the kernels that restore checkpoints on the way to the tensor core, as a model on the
CPU: five stages, two groups that take turns, loads that land in any order, barriers whose waits see
only the parity of a phase.  A group that waits for the load's barrier alone can take the phase of
two uses ago for its own while the other group's load has still to land; with the wait for the
stage's last use before it, it cannot."""
import os
import random
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
STAGES, GROUPS = 5, 2


def passed(phase, parity):
    """mbarrier.try_wait.parity: has the phase of this parity completed, the barrier being in
    `phase` (counted from 0)?"""
    return phase & 1 != parity


def run(steps, guarded, rng, stages=STAGES):
    """One interleaving of the producer, its loads, both groups and the matrix instructions; the
    number of steps restored before their load had landed."""
    full, free = [0] * stages, [0] * stages      # phases completed
    restored = [False] * steps
    flying, issued, consumed, early = [], 0, 0, 0
    at = list(range(GROUPS))                     # each group's next step
    while consumed < steps:
        moves = []
        if issued < steps and passed(free[issued % stages], (issued // stages & 1) ^ 1):
            moves.append("issue")
        moves += [("land", k) for k in flying]
        for g in range(GROUPS):
            st, r = at[g] % stages, at[g] // stages
            if at[g] < steps and passed(full[st], r & 1):
                if not guarded or r == 0 or passed(free[st], (r & 1) ^ 1):
                    moves.append(("restore", g))
        if consumed < steps and restored[consumed]:
            moves.append("consume")
        assert moves, "no move left"
        m = rng.choice(moves)
        if m == "issue":
            flying.append(issued)
            issued += 1
        elif m == "consume":
            free[consumed % stages] += 1
            consumed += 1
        elif m[0] == "land":
            flying.remove(m[1])
            full[m[1] % stages] += 1
        else:
            k = at[m[1]]
            if full[k % stages] != k // stages + 1:
                early += 1
                if not guarded:
                    return early                 # from here on anything may happen
            restored[k] = True
            at[m[1]] += GROUPS
    return early


def test_with_the_guard_no_step_is_restored_early():
    rng = random.Random(1)
    assert all(run(60, True, rng) == 0 for _ in range(2000))


def test_without_it_some_are():
    rng = random.Random(1)
    assert any(run(60, False, rng) for _ in range(2000))


def test_of_an_even_number_of_stages_each_group_has_its_own():
    rng = random.Random(1)
    assert all(run(60, False, rng, stages=4) == 0 for _ in range(2000))


@pytest.mark.parametrize("name", ["grouped.cu", "weight_grad.cu"])
def test_the_kernels_have_the_guard(name):
    code = open(os.path.join(ROOT, "gradient_reduction_gb300", "csrc", name)).read()
    assert re.search(r"round == 0 \|\| tc::mbar_wait\(free_\(st\), \(round & 1\) \^ 1\)\) &&\s+"
                     r"tc::mbar_wait\(full\(st\), round & 1\)", code)
