"""The barriers of the paged chunk kernel (rkv_paged_attention.cu) as a model, without a GPU.

Every role of a thread block is an actor that may be held up anywhere and for any time; a wait looks
at the parity of its barrier whenever the actor is scheduled, as the hardware's does. A barrier that
completes two phases while some warp still waits for the first one leaves that warp waiting for good.
The model follows the kernel's waits and arrivals unit by unit: units of one or two query tiles, of
one to three key tiles, without keys, with and without stale V rows to clear at the end.
"""
import random

import pytest


class Bar:
    """An mbarrier: a phase completes when all arrivals and all copies announced with them are in."""

    def __init__(self, count):
        self.count, self.phase, self.left, self.copies = count, 0, count, 0

    def arrive(self, copies=0):
        self.copies += copies
        self.left -= 1
        assert self.left >= 0
        self._end()

    def landed(self):
        self.copies -= 1
        self._end()

    def _end(self):
        if self.left == 0 and self.copies == 0:
            self.phase += 1
            self.left = self.count


class Named:
    """A hardware barrier of `count` warps."""

    def __init__(self, count):
        self.count, self.here, self.turn = count, 0, 0

    def arrive(self):
        turn = self.turn
        self.here += 1
        if self.here == self.count:
            self.here, self.turn = 0, turn + 1
        return turn


def stalls(units, seed, fix_wait=True, tail_wait=True):
    """Whether some schedule step is reached from which nobody moves on. The two flags leave out one wait each."""
    rng = random.Random(seed)
    bars = {k: Bar(4 if k.startswith("p_full") else 1) for k in
            ("q", "q_empty", "k_full0", "k_full1", "k_empty0", "k_empty1", "v_full0", "v_full1", "v_empty0", "v_empty1",
             "s_full0", "s_full1", "p_full0", "p_full1", "o_done", "v_fix")}
    join, tail = Named(8), Named(8)
    pipe, copies = [], []  # commits of issued products, in order; copies on their way, in any order

    def wait(bar, use):
        while bars[bar].phase & 1 == use & 1:
            yield False

    def meet(named, turn):
        while named.turn == turn:
            yield False

    def producer():
        n = 0  # tiles issued
        for i, u in enumerate(units):
            if i:
                yield from wait("q_empty", i - 1)
            bars["q"].arrive(1)
            copies.append("q")
            for _ in range(u["tiles"]):
                yield True
                for x in "kv":
                    if n >= 2:
                        yield from wait(f"{x}_empty{n & 1}", (n - 2) >> 1)
                    bars[f"{x}_full{n & 1}"].arrive(int(u["keys"]))
                    if u["keys"]:
                        copies.append(f"{x}_full{n & 1}")
                n += 1
            if u["fix"]:
                yield from wait(f"v_full{(n - 1) & 1}", (n - 1) >> 1)
                if fix_wait and n >= 2:
                    yield from wait(f"v_empty{n & 1}", (n - 2) >> 1)
                bars["v_fix"].arrive()

    def issuer():
        g, fixes, used = 0, 0, [0, 0]
        for i, u in enumerate(units):
            n = u["tiles"]

            def wait_v(j):
                yield from wait(f"v_full{(g + j) & 1}", (g + j) >> 1)
                if j + 1 == n and u["fix"]:
                    yield True
                    yield from wait("v_fix", fixes)

            def value(t, j, use, frees):
                yield from wait(f"p_full{t}", used[t] + use)
                if frees:
                    pipe.append(f"v_empty{(g + j) & 1}")

            yield from wait("q", i)
            for j in range(n):
                yield from wait(f"k_full{(g + j) & 1}", (g + j) >> 1)
                last = ["q_empty"] if j + 1 == n else []
                if u["two"]:
                    pipe.append("s_full0")
                    yield True
                    if j:
                        yield from value(1, j - 1, j - 1, True)
                    pipe.extend(["s_full1", f"k_empty{(g + j) & 1}"] + last)
                    yield True
                    yield from wait_v(j)
                    yield from value(0, j, j, False)
                else:
                    pipe.extend([f"s_full{j & 1}", f"k_empty{(g + j) & 1}"] + last)
                    yield True
                    if j:
                        yield from wait_v(j - 1)
                        yield from value((j - 1) & 1, j - 1, (j - 1) >> 1, True)
            if u["two"]:
                yield from value(1, n - 1, n - 1, True)
            else:
                yield from wait_v(n - 1)
                yield from value((n - 1) & 1, n - 1, (n - 1) >> 1, True)
            pipe.append("o_done")
            for t in (0, 1):
                used[t] += n if u["two"] else (n + 1 - t) >> 1
            g += n
            fixes += u["fix"]

    def softmax(wg):
        taken = 0
        for i, u in enumerate(units):
            if tail_wait and not u["two"] and u["tiles"] == 1:
                turn = tail.arrive()
                if wg == 0:
                    yield from meet(tail, turn)
            for _ in range(u["tiles"] if u["two"] else (u["tiles"] + 1 - wg) >> 1):
                yield from wait(f"s_full{wg}", taken)
                yield True
                bars[f"p_full{wg}"].arrive()
                taken += 1
            yield from wait("o_done", i)
            yield True
            for _ in range(0 if u["two"] else 2):
                yield from meet(join, join.arrive())
                yield True

    def hardware(queue, act):
        while True:
            if queue:
                act()
            yield bool(queue)

    actors = {"producer": producer(), "issuer": issuer()}
    actors.update({f"softmax{wg}{w}": softmax(wg) for wg in (0, 1) for w in range(4)})
    actors["products"] = hardware(pipe, lambda: bars[pipe.pop(0)].arrive())
    actors["copies"] = hardware(copies, lambda: bars[copies.pop(rng.randrange(len(copies)))].landed())
    held, still = rng.choice(list(actors)), 0
    while len(actors) > 2:
        if rng.random() < 0.002:
            held = rng.choice(list(actors))  # this one runs a step in some three hundred
        name = held if held in actors and rng.random() < 0.003 else rng.choice([x for x in actors if x != held])
        try:
            still = 0 if next(actors[name]) else still + 1
        except StopIteration:
            del actors[name]
            still = 0
        if still > 4000:
            return True
    return False


def some_units(seed, n=24):
    rng = random.Random(seed)
    r = []
    for _ in range(n):
        tiles = rng.choice([1, 1, 1, 2, 3])
        keys = tiles > 1 or rng.random() < 0.8
        r.append(dict(two=rng.random() < 0.5, tiles=tiles, keys=keys, fix=keys and rng.random() < 0.7))
    return r


def test_no_warp_is_left_waiting():
    assert not any(stalls(some_units(seed), seed) for seed in range(60))


@pytest.mark.parametrize("flag", ["fix_wait", "tail_wait"])
def test_the_model_finds_a_missing_wait(flag):
    assert any(stalls(some_units(seed), seed, **{flag: False}) for seed in range(60))
