"""The hand-over of k_attn_many's ring of key and value tiles, as a model on the
CPU: loader, MMA warp, gate warp and softmax as the lists of their barrier
operations, every order of their steps.  A wait knows a phase by its parity alone,
as mbarrier waits do, so a slot whose phase runs two ahead of a waiting warp stops
that warp for good."""
import pytest


class Model:
    """Operations: ("wait", barrier, phase waited for) and ("arrive", barrier)."""

    def __init__(self, stages, segments, hold_first_keys):
        self.need = {"s_full": 1, "p_ready": 2, "q_full": 1}   # p_ready: softmax and gate
        loader, mma, gate, softmax = [], [], [], []
        places = sum(2 * n for n in segments)

        def slot(kind, i):
            self.need.setdefault((kind, i % stages), 1)
            return kind, i % stages

        for i in range(places):
            if i >= stages:
                loader.append(("wait", slot("empty", i), i // stages - 1))
            loader.append(("arrive", slot("full", i)))
        it = done = scores = 0
        for n, tiles in enumerate(segments):
            mma += [("wait", slot("full", it), it // stages), ("wait", "q_full", n), ("arrive", "s_full")]
            back = ("arrive", slot("empty", it))   # the first keys' slot
            if not hold_first_keys:
                mma.append(back)
            gate.append(("wait", slot("full", it), it // stages))
            softmax.append(("arrive", "q_full"))
            it += 1
            for j in range(tiles):
                more = j + 1 < tiles
                gate.append(("wait", slot("full", it), it // stages))
                if more:
                    gate.append(("wait", slot("full", it + 1), (it + 1) // stages))
                gate += ([("wait", "p_ready", done - 1)] if done else []) + [("arrive", "p_ready")]
                softmax += [("wait", "s_full", scores), ("arrive", "p_ready")]
                mma += [("wait", "p_ready", done)] + ([("arrive", "s_full")] if more else [])
                if hold_first_keys and j == 0:
                    mma.append(back)
                mma.append(("arrive", slot("empty", it)))
                if more:
                    mma.append(("arrive", slot("empty", it + 1)))
                scores += 1
                done += 1
                it += 2 if more else 1
        self.roles = [loader, mma, gate, softmax]
        self.arrivals = []   # of each role, how often it has arrived on each barrier before its k-th step
        for ops in self.roles:
            seen, at = {}, [{}]
            for op in ops:
                if op[0] == "arrive":
                    seen = {**seen, op[1]: seen.get(op[1], 0) + 1}
                at.append(seen)
            self.arrivals.append(at)

    def phase(self, state, bar):
        return sum(self.arrivals[r][k].get(bar, 0) for r, k in enumerate(state)) // self.need[bar]

    def stuck(self):
        """States from which no role can step, and waits that let a wrong phase pass."""
        start = (0,) * len(self.roles)
        todo, seen, found = [start], {start}, []
        while todo:
            state = todo.pop()
            steps = 0
            for r, k in enumerate(state):
                if k == len(self.roles[r]):
                    continue
                op = self.roles[r][k]
                if op[0] == "wait":
                    phase = self.phase(state, op[1])
                    if phase % 2 == op[2] % 2:
                        continue
                    if phase != op[2] + 1:
                        found.append(("passed", state))
                steps += 1
                after = state[:r] + (k + 1,) + state[r + 1:]
                if after not in seen:
                    seen.add(after)
                    todo.append(after)
            if steps == 0 and any(k < len(ops) for k, ops in zip(state, self.roles)):
                found.append(("stopped", state))
        return found


SEGMENTS = [[1, 1, 1, 1], [3, 1, 2], [1, 5, 1], [4, 4]]


@pytest.mark.parametrize("segments", SEGMENTS, ids=str)
@pytest.mark.parametrize("stages", [3, 4, 5, 6])
def test_every_order_of_steps_ends(stages, segments):
    assert Model(stages, segments, True).stuck() == []


def test_first_keys_handed_back_before_the_gate_has_looked_stop():
    """The model tells: were the slot handed back on the MMA warp's own wait, it could be filled again
    before the gate sees it."""
    assert any(kind == "stopped" for kind, _ in Model(4, [1, 5, 1], False).stuck())
    assert any(kind == "stopped" for kind, _ in Model(6, [4, 4], False).stuck())
