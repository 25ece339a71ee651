"""The hand-over of S, P and O between the issuing thread, the tensor pipe and
the softmax warps of the cache attention for many rows, as an explicit-state
model on the CPU: every order in which the parties can move is walked through.

A barrier counts completed phases; a wait with parity p passes while the last
completed phase has that parity, which tells a phase from its neighbours and no
more.  So each wait must come where the phase that it means is the one under
way or the last one completed; the model finds the orders where it is not.  The
pipe works in order, but what it signals to different barriers may be seen in
any order.
"""
import pytest

WARPS = 2       # of a group (eight in the kernel, all alike)


class Handover:
    """Two softmax groups, unit n (S, then O += P V) of group n & 1 in S accumulator n % nb, signalled by barrier n % ns."""

    def __init__(self, units, nb, rule, idle=(), ns=None):
        self.units, self.nb, self.rule, self.idle = units, nb, rule, set(idle)
        self.ns = ns or (2 * nb if nb % 2 else nb)      # so that a barrier is one group's
        self.issue = []
        for n in range(min(nb, units)):
            self.issue.append(("qk", n))
        for n in range(units):
            self.issue.append(("pv", n))
            if n + nb < units:
                self.issue.append(("qk", n + nb))
        self.warps = [(w, x) for w in range(2) for x in range(WARPS)]
        self.programs = [self.program(w, (w, x) in self.idle) for w, x in self.warps]

    def program(self, w, idle):
        """Steps of a softmax warp: (wait, barrier, parity, phase meant), (rescale, phase meant), (arrive, barrier)."""
        steps = []
        for i, n in enumerate(range(w, self.units, 2)):
            b = n % self.nb
            steps.append(("wait", ("s", n % self.ns), n // self.ns & 1, n // self.ns))
            if self.rule == "two units back" and self.nb > 2 and i > 1:
                steps.append(("wait", ("pv", w), i & 1, i - 2))
            if idle:
                steps.append(("arrive", ("p", b)))
                continue
            if self.nb > 2 and i > 0:
                # the last P V: before O is rescaled and P is handed over (formerly: only where O is rescaled)
                steps.append(("wait" if self.rule == "every unit" else "may wait", ("pv", w), (i - 1) & 1, i - 1))
            steps.append(("rescale", i))
            steps.append(("arrive", ("p", b)))
        return steps

    def explore(self):
        """(orders that get stuck, waits that passed for another phase, rescales of an O in use)."""
        names = [("s", b) for b in range(self.ns)] + [("pv", w) for w in range(2)] + [("p", b) for b in range(self.nb)]
        at = {name: k for k, name in enumerate(names)}
        signals = self.ns + 2                   # barriers that the pipe signals
        made = [[0] * signals]                  # made[d]: phases of each that the first d steps of the pipe complete
        for kind, n in self.issue:
            row = list(made[-1])
            row[at["s", n % self.ns] if kind == "qk" else at["pv", n & 1]] += 1
            made.append(row)
        # state: phases seen, arrivals pending on p, steps issued, steps done by the pipe, the warps' places
        start = (tuple([0] * len(names)), tuple([0] * self.nb), 0, 0, tuple([0] * len(self.warps)))
        todo, seen = [start], {start}
        stuck = wrong = torn = 0

        def more(values, k):
            return values[:k] + (values[k] + 1,) + values[k + 1:]

        while todo:
            phases, pending, issued, done, place = todo.pop()
            out = []
            if issued < len(self.issue):
                kind, n = self.issue[issued]
                if kind == "qk" or phases[at["p", n % self.nb]] & 1 != (n // self.nb) & 1:
                    out.append((phases, pending, issued + 1, done, place))
            if done < issued:
                out.append((phases, pending, issued, done + 1, place))
            for k in range(signals):
                if phases[k] < made[done][k]:
                    out.append((more(phases, k), pending, issued, done, place))
            for k, (w, _) in enumerate(self.warps):
                if place[k] == len(self.programs[k]):
                    continue
                step, nxt = self.programs[k][place[k]], more(place, k)
                if step[0] == "rescale":
                    torn += made[done][at["pv", w]] < step[1]
                    out.append((phases, pending, issued, done, nxt))
                elif step[0] == "arrive":
                    b = step[1][1]
                    if pending[b] + 1 < WARPS:
                        out.append((phases, more(pending, b), issued, done, nxt))
                    else:
                        out.append((more(phases, at[step[1]]), pending[:b] + (0,) + pending[b + 1:], issued, done, nxt))
                else:
                    if phases[at[step[1]]] & 1 != step[2]:
                        wrong += phases[at[step[1]]] != step[3] + 1
                        out.append((phases, pending, issued, done, nxt))
                    if step[0] == "may wait":           # no rescale either
                        out.append((phases, pending, issued, done, more(nxt, k)))
            final = done == len(self.issue) and all(p == len(s) for p, s in zip(place, self.programs))
            stuck += not out and not final
            for s in out:
                if s not in seen:
                    seen.add(s)
                    todo.append(s)
        return stuck, wrong, torn


@pytest.mark.parametrize("idle", [(), ((1, 1),), ((1, 0), (1, 1))], ids=["all", "one idle", "a group idle"])
@pytest.mark.parametrize("nb", [2, 3])
@pytest.mark.parametrize("units", [1, 2, 5, 8, 12])
def test_every_order_ends(units, nb, idle):
    assert Handover(units, nb, "every unit", idle).explore() == (0, 0, 0)


def test_the_model_finds_waits_that_miss_their_phase():
    """Controls: a wait for the P V of two units ago gets stuck when the last one is done as well; without
    it, a wait that not every unit makes can pass for an earlier phase."""
    stuck, wrong, _ = Handover(6, 3, "two units back").explore()
    assert stuck > 0 and wrong == 0
    _, wrong, _ = Handover(6, 3, "only to rescale").explore()
    assert wrong > 0
    # one barrier for both groups' uses of an accumulator: a group waits for every other phase of it
    _, wrong, _ = Handover(5, 3, "every unit", ns=3).explore()
    assert wrong > 0
