"""The roles of a CTA of the prefill with modified scores hand items on through barriers that are waited for by parity: a
wait that is not looked at until the barrier has gone on by two phases waits for good. Which barrier and which parity the
roles use is read from the source, and every order in which they may take their steps is gone through."""
import os
import re

HERE = os.path.dirname(os.path.abspath(__file__))


def _source():
    with open(os.path.join(HERE, "..", "paged_kv_cache_kvh_gb300", "csrc", "prefill_mod.cu")) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def _uses(text, name):
    """(barrier, parity) of the wait for, and the barrier of the arrival at, the one named, as expressions of k."""
    waits = re.findall(r"wait_\w+\(bar\((%s[^,]*)\), ([^,]*), s_abort" % name, text)
    arrivals = re.findall(r"mbar_arrive\(bar\((%s[^;]*)\)\);" % name, text)
    return waits, arrivals


def _stuck(items, rows_wait, rows_arrive):
    """Orders of the steps of the loading warp, the softmax warps (as one) and the warp that computes rows again, over
    `items` items; True if one of them ends with a role that waits for good."""
    full, free, rows = 0, 2, 4                     # two barriers each, by item % 2

    def value(expression, k):
        return eval(expression, {"k": k, "kBarRows": rows})

    programs = [[], [], []]
    for k in range(items):
        if k >= 2:
            programs[0].append(("wait", free + (k & 1), ((k >> 1) - 1) & 1))
        programs[0].append(("arrive", full + (k & 1)))
        for role in (1, 2):
            programs[role].append(("wait", full + (k & 1), (k >> 1) & 1))
            if role == 1:
                programs[role].append(("arrive", value(rows_arrive, k)))
            else:
                programs[role].append(("wait", value(rows_wait[0], k), value(rows_wait[1], k) & 1))
            programs[role].append(("arrive", free + (k & 1)))
    counts = {full: 1, full + 1: 1, free: 2, free + 1: 2, rows: 1, rows + 1: 1}
    start = ((0, 0, 0), tuple(0 for _ in range(6)))   # steps done; arrivals at each barrier so far
    seen, stack = {start}, [start]
    while stack:
        at, arrivals = stack.pop()
        moved = False
        for role in range(3):
            if at[role] == len(programs[role]):
                continue
            step = programs[role][at[role]]
            then = list(arrivals)
            if step[0] == "wait":
                phase = arrivals[step[1]] // counts[step[1]]     # the phase that is under way
                if phase & 1 == step[2]:
                    continue
            else:
                then[step[1]] += 1
            moved = True
            state = (tuple(n + (r == role) for r, n in enumerate(at)), tuple(then))
            if state not in seen:
                seen.add(state)
                stack.append(state)
        if not moved and any(at[r] < len(programs[r]) for r in range(3)):
            return True
    return False


def test_no_order_of_the_roles_waits_for_good():
    waits, arrivals = _uses(_source(), "kBarRows")
    assert len(waits) == 1 and len(arrivals) == 1
    assert not _stuck(7, waits[0], arrivals[0])


def test_a_single_barrier_for_the_rows_would():
    assert _stuck(4, ("kBarRows", "k & 1"), "kBarRows")


def test_items_are_handed_on_as_modelled():
    text = _source()
    full, full_arrivals = _uses(text, "kBarItemFull")
    assert [w for w in full if w != ("kBarItemFull", "0")] == [("kBarItemFull + (k & 1)", "(k >> 1) & 1")] * 3
    assert full_arrivals == ["kBarItemFull + (k & 1)"] * 2
    free, free_arrivals = _uses(text, "kBarItemFree")
    assert free == [("kBarItemFree + (k & 1)", "((k >> 1) - 1) & 1")] * 2
    assert free_arrivals == ["kBarItemFree + (k & 1)"] * 3
