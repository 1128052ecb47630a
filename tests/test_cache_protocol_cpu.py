"""The barrier protocol of the tree-attention kernel in tensor memory, run as a
discrete-event model under many random timings: a parity wait must pass only on
the phase it means, no phase may overtake its waiter, and every schedule must
end. Roles and waits follow cache_attn_tc.cu: the producer of K and V, the MMA
warp with its in-order tensor pipe, the loader of the query rows, and one softmax
group per row block. The one-barrier form of P (`shared_p`) with two score
buffers is the version that could miss a phase: the model has to find that."""
import random

import pytest


class Overtaken(Exception):
    pass


class Bar:
    def __init__(self, count):
        self.count, self.pending, self.done = count, count, 0

    def arrive(self):
        self.pending -= 1
        if self.pending == 0:
            self.done += 1
            self.pending = self.count

    def passes(self, phase):
        """The parity wait of `phase`: true when the last completed phase has its parity."""
        if self.done > phase + 1:
            raise Overtaken(f"phase {phase} awaited, {self.done} complete")
        if self.done == 0 or (self.done - 1) % 2 != phase % 2:
            return False
        if self.done != phase + 1:
            raise Overtaken(f"phase {phase} awaited, passed on {self.done - 1}")
        return True


class Model:
    def __init__(self, NT, KS, VS, pieces, rng, shared_p=False, rows=False):
        self.NT, self.KS, self.VS, self.pieces, self.rng = NT, KS, VS, pieces, rng
        self.SB = 2 if NT == 1 else 1
        self.PB = 1 if shared_p else self.SB
        b = self.b = {}
        for s in range(KS):
            b["kfull", s], b["kempty", s] = Bar(1), Bar(1)
        for s in range(VS):
            b["vfull", s], b["vempty", s] = Bar(1), Bar(1)
        for t in range(NT):
            b["odone", t], b["ofree", t], b["qfull", t] = Bar(1), Bar(1), Bar(1)
            for sb in range(self.SB):
                b["s", t, sb] = Bar(1)
            for sb in range(self.PB):
                b["p", t, sb] = Bar(1)
        b["qfree"] = Bar(1)
        for i in range(4):
            b["pready", i] = Bar(1)
        self.pipe, self.copies = [], []  # tensor pipe (in order), copies (any order)
        self.rows, self.landed = rows, set()
        self.state = {"k": {}, "v": {}, "q": None, "s": {}, "o": {}}

    def wait(self, name, phase):
        while not self.b[name].passes(phase):
            yield

    def producer(self, full, empty, n):
        for it in range(sum(self.pieces)):
            st, use = it % n, it // n
            if use:
                yield from self.wait((empty, st), use - 1)
            self.copies.append(((full, st), full[0], st, it))
            yield

    def producer_rows(self, full, empty, n):
        """Row by row: a tile is told by its warp, when the next one has been started or ahead of a wait."""
        told = 0

        def tell(upto):
            nonlocal told
            while any((full[0], i) not in self.landed for i in range(told, upto)):
                yield
            for i in range(told, upto):
                self.b[full, i % n].arrive()
            told = max(told, upto)

        for it in range(sum(self.pieces)):
            st, use = it % n, it // n
            if use and not self.b[empty, st].passes(use - 1):
                yield from tell(it)
                yield from self.wait((empty, st), use - 1)
            self.copies.append((None, full[0], st, it))
            yield
            yield from tell(it)
        yield from tell(sum(self.pieces))

    def loader(self):
        for k in range(len(self.pieces) + 1):
            if k:
                yield from self.wait("qfree", k - 1)
            self.b["pready", k % 4].arrive()
            if k < len(self.pieces):
                for t in range(self.NT):
                    self.copies.append((("qfull", t), "q", t, k))
            yield

    def issue_s(self, t, at, piece, last):
        self.pipe.append(("s", t, at % self.SB, at, piece))
        self.pipe.append(("commit", ("s", t, at % self.SB)))
        if t == self.NT - 1:
            self.pipe.append(("commit", ("kempty", at % self.KS)))
            if last:
                self.pipe.append(("commit", "qfree"))

    def issue_pv(self, t, at, last):
        self.pipe.append(("pv", t, at % self.SB, at))
        if t == self.NT - 1:
            self.pipe.append(("commit", ("vempty", at % self.VS)))
        if last:
            self.pipe.append(("commit", ("odone", t)))

    def mma(self):
        it, NT = 0, self.NT
        w = self.wait
        for piece, nk in enumerate(self.pieces):
            yield from w(("kfull", it % self.KS), it // self.KS)
            for t in range(NT):
                yield from w(("qfull", t), piece)
                self.issue_s(t, it, piece, nk == 1)
            yield from w(("vfull", it % self.VS), it // self.VS)
            for n in range(nk):
                at, more = it + n, n + 1 < nk
                nxt = at + 1
                if NT == 1:
                    if more:
                        yield from w(("kfull", nxt % self.KS), nxt // self.KS)
                        self.issue_s(0, nxt, piece, n + 2 == nk)
                        yield
                    pb = at % self.PB
                    yield from w(("p", 0, pb), at // self.PB)
                    if n == 0 and piece:
                        yield from w(("ofree", 0), piece - 1)
                    self.issue_pv(0, at, not more)
                    yield
                    if more:
                        yield from w(("vfull", nxt % self.VS), nxt // self.VS)
                else:
                    for t in range(NT):
                        yield from w(("p", t, 0), at)
                        if n == 0 and piece:
                            yield from w(("ofree", t), piece - 1)
                        if more and t == 0:
                            yield from w(("kfull", nxt % self.KS), nxt // self.KS)
                        if more and t == NT - 1:
                            yield from w(("vfull", nxt % self.VS), nxt // self.VS)
                        self.issue_pv(t, at, not more)
                        yield
                        if more:
                            self.issue_s(t, nxt, piece, n + 2 == nk)
                            yield
            it += nk

    def softmax(self, t):
        it = 0
        for piece in range(len(self.pieces) + 1):
            yield from self.wait(("pready", piece % 4), piece // 4)
            if piece == len(self.pieces):
                return
            for n in range(self.pieces[piece]):
                sb = it % self.SB
                yield from self.wait(("s", t, sb), it // self.SB)
                assert self.state["s"][t, sb] == ("s", it), "scores of another tile"
                if n and self.rng.random() < 0.3:  # a rescale of O
                    if self.SB == 2:
                        yield from self.wait(("vempty", (it - 1) % self.VS), (it - 1) // self.VS)
                    assert self.state["o"][t] == it - 1, "O still lacks a tile"
                yield
                self.state["s"][t, sb] = ("p", it)
                self.b["p", t, it % self.PB].arrive()
                it += 1
            yield from self.wait(("odone", t), piece)
            assert self.state["o"][t] == it - 1
            yield
            self.b["ofree", t].arrive()

    def step_async(self):
        todo = []
        if self.pipe:
            todo.append("pipe")
        if self.copies:
            todo.append("copy")
        if not todo:
            return False
        if self.rng.choice(todo) == "copy":
            name, what, st, tag = self.copies.pop(self.rng.randrange(len(self.copies)))
            self.state[what][st] = tag if what != "q" else None
            if what == "q":
                self.state["q"] = dict(self.state["q"] or {}, **{str(st): tag})
            if name is None:
                self.landed.add((what, tag))
            else:
                self.b[name].arrive()
            return True
        op = self.pipe.pop(0)
        if op[0] == "commit":
            self.b[op[1]].arrive()
        elif op[0] == "s":
            _, t, sb, at, piece = op
            assert self.state["k"][at % self.KS] == at and self.state["q"][str(t)] == piece
            assert self.state["s"].get((t, sb), ("used",))[0] == "used", "scores overwritten"
            self.state["s"][t, sb] = ("s", at)
        else:
            _, t, sb, at = op
            assert self.state["v"][at % self.VS] == at
            assert self.state["s"][t, sb] == ("p", at)
            self.state["s"][t, sb] = ("used",)
            self.state["o"][t] = at
        return True

    def run(self):
        self.state["q"] = {}
        feed = self.producer_rows if self.rows else self.producer
        roles = {"k": feed("kfull", "kempty", self.KS), "v": feed("vfull", "vempty", self.VS),
                 "mma": self.mma(), "q": self.loader()}
        roles.update({f"soft{t}": self.softmax(t) for t in range(self.NT)})
        speed = {r: self.rng.choice([0.05, 0.3, 1.0]) for r in [*roles, "async"]}
        idle = 0
        while roles:
            names = [*roles, "async"]
            r = self.rng.choices(names, [speed[n] for n in names])[0]
            before = (len(self.pipe), len(self.copies), tuple(b.done * 99 + b.pending for b in self.b.values()), len(roles))
            if r == "async":
                self.step_async()
            else:
                try:
                    next(roles[r])
                except StopIteration:
                    del roles[r]
            after = (len(self.pipe), len(self.copies), tuple(b.done * 99 + b.pending for b in self.b.values()), len(roles))
            idle = idle + 1 if before == after else 0
            if idle > 3000:
                raise Overtaken("nothing moves any more: " + ", ".join(roles))
        while self.step_async():
            pass


def pieces_of(rng):
    return [rng.choice([1, 1, 2, 3, 7]) for _ in range(rng.randint(1, 7))]


@pytest.mark.parametrize("rows", [False, True])
@pytest.mark.parametrize("NT,KS,VS", [(1, 2, 3), (1, 4, 4), (2, 2, 2), (2, 4, 4)])
def test_every_schedule_is_sound(NT, KS, VS, rows):
    for seed in range(150):
        rng = random.Random(seed * 31 + NT * 7 + KS)
        Model(NT, KS, VS, pieces_of(rng), rng, rows=rows).run()


def test_one_barrier_for_two_score_buffers_is_found():
    found = 0
    for seed in range(300):
        rng = random.Random(seed)
        try:
            Model(1, 2, 3, pieces_of(rng), rng, shared_p=True).run()
        except Overtaken:
            found += 1
    assert found
