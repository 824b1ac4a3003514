"""The barriers of q8_attn_prefill as a small model, run on the CPU under random schedules.

An mbarrier tells a phase from the one before it only: a wait by parity passes early when the phase before the one it is
for is not complete, and never passes when two more have completed.  The model has the kernel's roles (loads, MMAs,
helpers, the softmax warps of both query tiles) as generators that name the phase they wait for; loads land in any order,
the tensor pipe completes in order, and some role may be slow or spend long between two items (a walk over requests
without rows).  Each wait must find its own phase.  ``shared`` is the form that the kernel must not take: landings of keys and
values on one barrier for each place of the ring, looked at by the helpers for both."""
import random

import pytest


class Missed(Exception):
    pass


class Bar:
    def __init__(self, arrivals, name):
        self.arrivals, self.left, self.done, self.name = arrivals, arrivals, 0, name

    def arrive(self):
        self.left -= 1
        assert self.left >= 0, f"too many arrivals at {self.name}"
        if self.left == 0:
            self.done += 1
            self.left = self.arrivals

    def passed(self, phase, who):
        ok = (self.done & 1) != (phase & 1)
        if ok and self.done != phase + 1:
            raise Missed(f"{who} passes {self.name} early")
        if not ok and self.done > phase:
            raise Missed(f"{who} missed its phase of {self.name}")
        return ok


def bars(n, arrivals, name):
    return [Bar(arrivals, f"{name}{i}") for i in range(n)]


def play(q8, dim, segments, rng, slow=None, shared=False):
    """segments: (key tiles, whether query tile B has rows, the longest pause before it)."""
    buffers = 3 if dim == 64 else 2
    places = (3 if dim == 128 else 6) if q8 else (5 if dim == 128 else 10)
    raw_places = 3 if dim == 128 else 4
    helpers, warps = (3, 2) if q8 else (2, 2)  # fewer than the kernel's: the same in kind
    full, ready, step = bars(10, 1, "full"), bars(10, helpers, "ready"), bars(16, 1, "step")
    raw_full, raw_empty = bars(4, 1, "raw_full"), bars(4, helpers, "raw_empty")
    q_raw, q_full, q_empty = Bar(1, "q_raw"), Bar(2 * warps if q8 else 1, "q_full"), Bar(1, "q_empty")
    s_full, p_ready = bars(3, 1, "s_full"), bars(3, warps, "p_ready")
    o_full, idle = bars(2, 1, "o_full"), Bar(warps, "idle")
    landing, pipe = [], []  # loads in flight, in any order; what the tensor pipe will arrive at, in order

    def by_place(c):
        return full[c % places], c // places

    def landed(c):  # of load c: the keys of tile c / 2, or its values
        if q8:
            return raw_full[c % raw_places], c // raw_places
        return by_place(c) if shared else (full[(c & 1) * 5 + (c >> 1) % 5], (c >> 1) // 5)

    def usable(c):
        if q8 or shared:
            return ready[c % places], c // places
        return ready[(c >> 1) % 5], (c >> 1) // 5

    def pause(longest):
        return range(rng.randint(0, longest))

    def load():
        c, steps, last = 0, 0, [0] * places
        for seg, (n, _, longest) in enumerate(segments):
            for _ in pause(longest):
                yield None
            if seg:
                yield q_empty, seg - 1
            landing.append(q_raw if q8 else q_full)
            for i in range(n):
                for kv in range(2):
                    around = raw_places if q8 else places
                    if c >= around:
                        yield (raw_empty[c % around], c // around - 1) if q8 else \
                            (step[last[c % around] % 16], last[c % around] // 16)
                    last[c % places] = steps + i + kv
                    landing.append(landed(c)[0])
                    c += 1
            steps += n + 1

    def helper():
        c, steps, last = 0, 0, [0] * places
        for n, _, longest in segments:
            for _ in pause(longest):
                yield None
            for i in range(n):
                for kv in range(2):
                    s = c % places
                    if q8:
                        if c >= places:
                            yield step[last[s] % 16], last[s] // 16
                        last[s] = steps + i + kv
                    if q8 or kv or shared:
                        yield landed(c)
                        yield None
                        if q8:
                            raw_empty[c % raw_places].arrive()
                        usable(c)[0].arrive()
                    c += 1
            steps += n + 1

    def mma():
        steps, key, value, job, weights = 0, 0, 0, 0, [0] * 3

        def keys():
            nonlocal key
            key += 1
            return usable(2 * key - 2) if q8 else landed(2 * key - 2)

        for seg, (n, two, longest) in enumerate(segments):
            for _ in pause(longest):
                yield None
            yield q_full, seg
            for m in range(min(buffers - 1, n)):
                yield keys()
                pipe.append(s_full[(job + 2 * m) % buffers])
                if m == 0 and two:
                    pipe.append(s_full[(job + 1) % buffers])
                if m + 1 == min(buffers - 1, n):
                    pipe.append(step[steps % 16])
                    if n == 1:
                        pipe.append(q_empty)
            steps += 1
            for i in range(n):
                a, b = job % buffers, (job + 1) % buffers
                yield usable(2 * value + 1)
                if buffers == 2 and i + 1 < n:
                    yield keys()
                yield p_ready[a], weights[a]
                weights[a] += 1
                if i + 1 == n:
                    pipe.append(o_full[0])
                if i + 1 < n and (buffers == 2 or two):
                    pipe.append(s_full[a])  # A's next scores, or B's (three buffers)
                more = buffers == 3 and i + 2 < n
                if more:
                    yield keys()
                if two:
                    yield p_ready[b], weights[b]
                    weights[b] += 1
                    if i + 1 == n:
                        pipe.append(o_full[1])
                if more or (buffers == 2 and two and i + 1 < n):
                    pipe.append(s_full[b])
                pipe.append(step[steps % 16])
                if i + 2 == n:
                    pipe.append(q_empty)
                value += 1
                job = (job + 2) % buffers
                steps += 1

    def softmax(x):
        steps, c, job, scores, ends, idles = 0, 0, 0, [0] * 3, 0, 0
        for seg, (n, two, longest) in enumerate(segments):
            for _ in pause(longest):
                yield None
            if q8:
                yield q_raw, seg
                q_full.arrive()
            for i in range(n):
                a, b = job, (job + 1) % buffers
                mine = b if x else a
                phase = scores[mine]
                scores[a] += 1
                scores[b] += two
                job = (job + 2) % buffers
                if x and not two:
                    continue
                yield s_full[mine], phase
                if q8:
                    yield usable(c + 2 * i + 1)
                if buffers == 3 and i and rng.random() < 0.3:  # O rescaled
                    yield step[(steps + i) % 16], (steps + i) // 16
                yield None
                p_ready[mine].arrive()
            if x and not two:
                yield o_full[0], seg
                idle.arrive()
            else:
                yield o_full[x], ends
                ends += 1
                if not two:
                    yield idle, idles
                    idles += 1
            steps += n + 1
            c += 2 * n

    roles = {"load": load(), "mma": mma(), **{f"helper{w}": helper() for w in range(helpers)},
             **{f"softmax{'AB'[x]}{w}": softmax(x) for x in range(2) for w in range(warps)}}
    waits, stalled = {}, 0
    while roles:
        who = rng.choices([*roles, "land", "pipe"],
                          [*(0.02 if r == slow else 1.0 for r in roles), bool(landing), bool(pipe)])[0]
        if who == "land":
            landing.pop(rng.randrange(len(landing))).arrive()
        elif who == "pipe":
            pipe.pop(0).arrive()
        elif who in waits and not waits[who][0].passed(waits[who][1], who):
            stalled += 1
            if stalled > 100000:
                raise Missed("nobody gets on: " + str({w: b.name for w, (b, _) in waits.items()}))
            continue
        else:
            waits.pop(who, None)
            try:
                wait = next(roles[who])
                if wait:
                    waits[who] = wait
            except StopIteration:
                del roles[who]
        stalled = 0


def games(count):
    for seed in range(count):
        rng = random.Random(seed)
        yield ([(rng.choice([1, 1, 1, 2, 2, 3, 5, 9]), rng.random() < 0.5, rng.choice([0, 0, 30]))
                for _ in range(rng.randint(1, 14))], rng, rng.choice([None, "load", "mma", "helper0", "softmaxA0", "softmaxB1"]))


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("dim", [64, 128])
def test_every_wait_finds_its_phase(q8, dim):
    for segments, rng, slow in games(40):
        play(q8, dim, segments, rng, slow)


@pytest.mark.parametrize("dim", [64, 128])
def test_the_model_sees_a_shared_landing(dim):
    def missed(segments, rng, slow):
        try:
            play(False, dim, segments, rng, slow, shared=True)
        except Missed as e:
            return "missed its phase of full" in str(e)
        return False
    assert any(missed(*game) for game in games(40))
