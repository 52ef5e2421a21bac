"""The order of waits and arrivals around a tile's values in attend_tc, played through on the CPU: a barrier has one bit
of phase, so that a wait that comes a whole phase late never ends."""
import os
import re

from gated_delta_net_gb300 import build

TILES = 7


def row_order():
    """What the threads of the rows do with a masked tile, in the order in which the source has it."""
    text = re.sub(r"//[^\n]*", "", open(os.path.join(build.CSRC, "attend_tc.cu")).read())
    rows = text[text.index("if (warp < S::kRowWarps) {"):text.index("} else if (warp == S::kRowWarps) {")]
    at = {rows.index("bar[S::READY"): "ready", rows.index("mbar_arrive(&bar[S::PROBS"): "probs"}
    assert rows.count("bar[S::READY") == rows.count("bar[S::PROBS") == 1
    return [at[i] for i in sorted(at)]


def programs(order, stages, buffers):
    """Each role's steps: (wait, barrier, phase) or (arrive, barrier).  With two buffers of scores they are a tile ahead."""
    rows, products, values = [], [], []
    scores = lambda c: [("arrive", ("SCORES", c % buffers))] if c < TILES else []  # noqa: E731
    if buffers == 2:
        products += scores(0)
    for c in range(TILES):
        ready, free, phase, probs = ("READY", c % stages), ("VEMPTY", c % stages), c // stages, ("PROBS", c % buffers)
        rows.append(("wait", ("SCORES", c % buffers), c // buffers))
        rows += [("wait", ready, phase) if step == "ready" else ("arrive", probs) for step in order]
        products += scores(c + buffers - 1) + [("wait", ready, phase), ("wait", probs, c // buffers), ("arrive", free)]
        values += ([("wait", free, phase - 1)] if phase else []) + [("arrive", ready)]
    return rows, products, values


def stuck(order, stages, buffers):
    """Whether some order of the roles' steps leaves one waiting for ever."""
    roles = programs(order, stages, buffers)
    seen, todo = set(), [(0, 0, 0)]
    while todo:
        at = todo.pop()
        if at in seen:
            continue
        seen.add(at)
        done = {}
        for role, n in zip(roles, at):
            for step in role[:n]:
                if step[0] == "arrive":
                    done[step[1]] = done.get(step[1], 0) + 1
        after = []
        for i, (role, n) in enumerate(zip(roles, at)):
            if n == len(role):
                continue
            step = role[n]
            # the phase that is under way has the other bit than the one waited for
            if step[0] == "arrive" or (done.get(step[1], 0) & 1) != (step[2] & 1):
                after.append(at[:i] + (n + 1,) + at[i + 1:])
        if not after and any(n < len(role) for role, n in zip(roles, at)):
            return True
        todo += after
    return False


def test_the_model_finds_a_phase_that_is_missed():
    for buffers in (1, 2):
        assert stuck(["probs", "ready"], 2, buffers) and not stuck(["ready", "probs"], 2, buffers)


def test_no_order_of_the_roles_leaves_one_waiting():
    for stages in (2, 5):
        for buffers in (1, 2):
            assert not stuck(row_order(), stages, buffers)
