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


# --- the one look that the kernels take first ----------------------------------------------------

def run_looking(steps, order, rng, stages=STAGES):
    """As `run` with the guard, but a group looks at two barriers, one after the other while the rest
    goes on, and restores at once if both have passed; else it waits, for the stage's last use and then
    for its load.  `order`: "free, full" as the kernels look, or a mistake.  The number of early
    restores, at most one."""
    full, free = [0] * stages, [0] * stages
    restored = [False] * steps
    flying, issued, consumed = [], 0, 0
    at = list(range(GROUPS))
    state = ["first"] * GROUPS               # then "second", "wait free", "wait full"
    seen = [False] * GROUPS
    looks = order.split(", ")

    def look(what, k):
        st, r = k % stages, k // stages
        return passed(full[st], r & 1) if what == "full" else passed(free[st], (r & 1) ^ 1)

    while consumed < steps:
        moves = []
        if issued < steps and passed(free[issued % stages], (issued // stages & 1) ^ 1):
            moves.append("issue")
        moves += [("land", k) for k in flying]
        for g in range(GROUPS):
            k = at[g]
            if k >= steps:
                continue
            if state[g] in ("first", "second"):
                moves.append((state[g], g))
            elif state[g] == "wait free" and (k < stages or look("free", k)):
                moves.append(("wait free", g))
            elif state[g] == "wait full" and look("full", k):
                moves.append(("restore", g))
        if consumed < steps and restored[consumed]:
            moves.append("consume")
        assert moves, "no move left"
        m = rng.choice(moves)
        if m == "issue":
            flying.append(issued)
            issued += 1
            continue
        if m == "consume":
            free[consumed % stages] += 1
            consumed += 1
            continue
        if m[0] == "land":
            flying.remove(m[1])
            full[m[1] % stages] += 1
            continue
        what, g = m
        k = at[g]
        if what == "first":                  # a stage's first use has no use before: straight to the waits
            seen[g] = k >= stages and look(looks[0], k)
            state[g] = "second"
            continue
        if what == "wait free":
            state[g] = "wait full"
            continue
        if what == "second" and not (seen[g] and (len(looks) < 2 or look(looks[1], k))):
            state[g] = "wait free"
            continue
        if full[k % stages] != k // stages + 1:
            return 1
        restored[k] = True
        at[g] += GROUPS
        state[g] = "first"
    return 0


def test_a_look_at_both_barriers_is_as_good():
    rng = random.Random(2)
    assert all(run_looking(60, "free, full", rng) == 0 for _ in range(3000))


@pytest.mark.parametrize("order", ["full, free", "full"])
def test_a_look_in_the_other_order_or_at_one_is_not(order):
    rng = random.Random(2)
    assert any(run_looking(60, order, rng) for _ in range(3000))


def test_the_kernels_look_at_both_barriers_in_this_order():
    """The call, where it decides alone, the order in which the two are looked at, and the number of
    stages and groups that the model has."""
    csrc = os.path.join(ROOT, "gradient_reduction_gb300", "csrc")
    read = lambda name: re.sub(r"\s+", " ", open(os.path.join(csrc, name)).read())
    for name in ("grouped.cu", "weight_grad.cu"):
        code = read(name)
        assert code.count("tc::mbar_passed(") == 1
        assert ("bool landed = round > 0 && tc::mbar_passed(free_(st), (round & 1) ^ 1, full(st), round & 1); "
                "if (!__all_sync(0xFFFFFFFFu, landed)) landed = (round == 0 || "
                "tc::mbar_wait(free_(st), (round & 1) ^ 1)) && tc::mbar_wait(full(st), round & 1); "
                "if (!(ok = __all_sync(0xFFFFFFFFu, landed))) break;") in code, name
    device = read("tensor_core.cuh")
    look = device[device.index("bool mbar_passed(uint32_t first, uint32_t first_parity, uint32_t then, uint32_t then_parity)"):]
    look = look[:look.index("return done")]
    assert look.index("p, [%1], %2;") < look.index("q, [%3], %4;")
    assert '"r"(first), "r"(first_parity), "r"(then), "r"(then_parity)' in look
    stages = re.search(r"int stages\(int kind\) \{ return is_odd\(kind\) \? (\d+) : is_made\(kind\) \? (\d+) : \d+; \}",
                       read("grouped.cu"))
    assert int(stages[1]) % GROUPS == 0 and int(stages[2]) == STAGES
    assert f"constexpr int kStages = {STAGES};" in read("weight_grad.cu")
