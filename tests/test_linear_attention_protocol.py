"""A model of how the CTAs of the tensor-core linear attention prefill hand states to one
another, run under random interleavings (no GPU needed).

An item is (sequence, segment) of one head; item i belongs to CTA i mod G, which takes its
items in order. In a CTA the compute warps publish a segment's state (unless it is the
sequence's last), take the one that enters (unless it is the first) and, behind the last
segment, write the state that leaves, once the sequence's first item no longer needs the
entering one in its place. The courier waits for and sets the flags in global memory for
them. The scan turns published states into entering ones; each CTA has two slots for either
kind, used in turn.

Waits on a barrier go by the parity of its phase, as on the GPU: a waiter that comes when a
second phase is over misses its own. The model checks that this never happens, that every
state is read as it was meant, before its slot is written again, and that the run never
stops. It restates the protocol; it does not run the CUDA code.
"""
import random

import pytest

WARPS, RING = 3, 4


class Barrier:
    def __init__(self, count):
        self.count, self.left, self.phases = count, count, 0

    def arrive(self):
        self.left -= 1
        if self.left == 0:
            self.left, self.phases = self.count, self.phases + 1

    def over(self, phase):
        """What try_wait answers for `phase` (by its parity)."""
        done = (self.phases & 1) != (phase & 1)
        assert not done or self.phases == phase + 1, "a phase missed"
        return done


def run(lengths, G, rng, bad_rate=0.0, wait_for_out=True):
    """lengths: segments of each sequence. `wait_for_out`: whether the compute warps wait for kOutOk
    before they arrive at kGot. `bad_rate`: how many keep the entering state to the item's end."""
    items = [(n, j, J) for n, J in enumerate(lengths) for j in range(J)]
    first = {n: next(i for i, it in enumerate(items) if it[0] == n) for n in range(len(lengths))}
    flag = {(c, k, p): 0 for c in range(G) for k in ("ready", "scanned", "in") for p in (0, 1)}
    done = [0] * G
    pub_slot, in_slot = {}, {}               # (CTA, parity) -> the item whose state lies there
    state = {n: "in" for n in range(len(lengths))}   # in place: the entering or the leaving state
    log = []

    def wait(cond):
        while not cond():
            yield

    def cta(c):
        mine = list(range(c, len(items), G))
        bar = {k: Barrier(n) for k, n in (("free", 1), ("pub", WARPS), ("inready", 1), ("out", 1))}
        got = [Barrier(WARPS) for _ in range(RING)]
        full, empty = [Barrier(1) for _ in range(RING)], [Barrier(WARPS + 1) for _ in range(RING)]

        def load():
            for i in range(len(mine)):
                if i >= RING:
                    yield from wait(lambda: empty[i % RING].over(i // RING - 1))
                full[i % RING].arrive()
                yield

        def warp(w):
            phase = dict.fromkeys(bar, 0)

            def on(k):
                yield from wait(lambda: bar[k].over(phase[k]))
                phase[k] += 1

            for i, it in enumerate(mine):
                yield from wait(lambda: full[i % RING].over(i // RING))
                empty[i % RING].arrive()
                n, j, J = items[it]
                last, bad = j + 1 == J, random.Random(it * 31 + w).random() < bad_rate
                if not last:
                    yield from on("free")
                    yield
                    pub_slot[c, i & 1] = it
                    bar["pub"].arrive()
                if j > 0:
                    yield from on("inready")
                    assert in_slot[c, i & 1] == it
                else:
                    assert state[n] == "in"
                yield
                if not last and not bad:
                    got[i % RING].arrive()
                yield
                if last or bad:              # rows made again from the entering state
                    assert in_slot.get((c, i & 1)) == it if j > 0 else state[n] == "in"
                yield
                if last and J > 1 and wait_for_out:
                    yield from on("out")
                if last or bad:
                    got[i % RING].arrive()
                yield
                if last and J > 1 and not wait_for_out:
                    yield from on("out")
                if last and J > 1:
                    state[n] = "out"
                log.append((it, w))
                yield

        def courier():
            used, ins, pubs = [0, 0], [0, 0], 0
            for i, it in enumerate(mine):
                yield from wait(lambda: full[i % RING].over(i // RING))
                n, j, J = items[it]
                p, last = i & 1, j + 1 == J
                if not last:
                    yield from wait(lambda: flag[c, "scanned", p] >= used[p])
                    used[p] += 1
                    bar["free"].arrive()
                    yield from wait(lambda: bar["pub"].over(pubs))
                    pubs += 1
                    flag[c, "ready", p] = i + 1
                    yield
                if j > 0:
                    ins[p] += 1
                    yield from wait(lambda: flag[c, "in", p] >= ins[p])
                    bar["inready"].arrive()
                    yield
                if last and J > 1:
                    f = first[n]
                    yield from wait(lambda: done[f % G] >= f // G + 1)
                    bar["out"].arrive()
                    yield
                yield from wait(lambda: got[i % RING].over(i // RING))
                done[c] = i + 1
                yield
                empty[i % RING].arrive()
                yield

        return [load(), courier()] + [warp(w) for w in range(WARPS)]

    def scan():
        for n, J in enumerate(lengths):
            for j in range(J - 1):
                src, dst = first[n] + j, first[n] + j + 1
                (cs, rs), (cd, rd) = ((src % G, src // G), (dst % G, dst // G))
                yield from wait(lambda: flag[cs, "ready", rs & 1] >= rs + 1 and done[cd] >= rd - 1)
                assert pub_slot[cs, rs & 1] == src
                in_slot[cd, rd & 1] = dst
                yield
                flag[cs, "scanned", rs & 1] += 1
                flag[cd, "in", rd & 1] += 1
                yield

    agents = [a for c in range(G) for a in cta(c)] + [scan()]
    idle, turn, speed = 0, 0, {}
    while agents:
        before = (len(log), len(agents), tuple(done), tuple(flag.values()))
        if turn % 60 == 0:                   # some run far ahead of others for a while
            speed = {id(a): rng.choice((0.02, 0.3, 1.0)) for a in agents}
        turn += 1
        for a in rng.sample(agents, len(agents)):
            if rng.random() > speed[id(a)]:
                continue
            try:
                next(a)
            except StopIteration:
                agents.remove(a)
        idle = 0 if (len(log), len(agents), tuple(done), tuple(flag.values())) != before else idle + 1
        assert idle < 3000, "it stopped"
    assert sorted(log) == [(i, w) for i in range(len(items)) for w in range(WARPS)]


def problems(seed):
    rng = random.Random(seed)
    return [rng.choice((1, 1, 2, 2, 3, 5)) for _ in range(rng.randint(1, 14))], rng.randint(1, 4), rng


@pytest.mark.parametrize("bad_rate", [0.0, 0.3])
def test_every_state_is_handed_over(bad_rate):
    for seed in range(120):
        run(*problems(seed), bad_rate=bad_rate)


def test_the_model_sees_a_courier_that_is_a_phase_ahead():
    """kOutOk served before kGot needs compute warps that have seen the last one before they
    arrive at kGot."""
    missed = 0
    for seed in range(120):
        try:
            run(*problems(seed), wait_for_out=False)
        except AssertionError as e:
            missed += str(e).startswith(("a phase missed", "it stopped"))
    assert missed > 0
