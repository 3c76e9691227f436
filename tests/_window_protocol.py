"""The barriers of window_attn's kernel on pairs of SMs, played on the host in random orders.

Each role of the two CTAs is a generator that yields its waits and steps; what a role does between them is what it
announces to the others.  The arrivals that a barrier's phase takes are read from the source, and so are the three places
where a role's part depended on the data.  A wait knows a phase by its parity only, as on the GPU, so that a run fails
where a wait passes before its phase has completed, comes when the next has too, or where every role waits."""

from __future__ import annotations

import os
import re

from sparse_latent_attention_gb300 import build


class Fault(Exception):
    pass


class Barrier:
    def __init__(self, count, name):
        self.count, self.name = count, name
        self.arrived = self.tx = self.complete = 0

    def arrive(self, tx=0):
        if self.arrived == self.count:
            raise Fault(f"{self.name}: more arrivals than a phase takes")
        self.tx += tx
        self.arrived += 1
        self._check()

    def landed(self):
        """One of the copies that an arrival expected."""
        self.tx -= 1
        self._check()

    def _check(self):
        if self.arrived == self.count and self.tx == 0:
            self.arrived = 0
            self.complete += 1


class Source:
    """What the kernel's source says of its barriers."""

    def __init__(self):
        with open(os.path.join(build.CSRC, "sa_window_tc.cu")) as f:
            self.text = f.read()
        found = re.findall(r"mbar_init\(smem_addr\(&M\.(\w+)(?:\[\w+\])*\), ([^;]+)\);", self.text)
        self.counts = {name: count for name, count in found}
        assert len(self.counts) >= 20
        # rank 1's loading warp arrives at K's barriers
        self.rank1_arrives = bool(re.search(r"if \(!is_v && rank != 0\) arrive_at\(at_leader\(bar\)\);", self.text))
        start = re.search(r"const int n0 = ([^;]+);", self.text)   # a widening warp's first stage of a task
        self.first_stage = compile(start[1].replace("(int)", "") if start else "turn", "n0", "eval")

    def count(self, name, codes, rank):
        expr = self.counts[name]
        expr = re.sub(r"\(?kCodes \? (\d+) : (\d+)\)?", lambda m: m[1] if codes else m[2], expr)
        expr = re.sub(r"\(rank == 0 \? (\d+) : (\d+)\)", lambda m: m[1] if rank == 0 else m[2], expr)
        return eval(expr, {"kEpilogues": 1 if codes else 2, "kFmt": 0, "warps_of": lambda _: 32 if codes else 22})


SIZES = dict(k_full=4, k_empty=4, v_full=4, v_empty=4, q_full=4, q_empty=4, info_full=8, info_empty=8, task_full=4,
             task_empty=4, s_full=3, s_empty=3, p_full=2, p_empty=2, m_full=4, sum_full=2, sum_empty=2, o_full=1, o_empty=1,
             stats_full=1, stats_empty=1, pair_bar=4, mx_empty=4)


class Pair:
    """A pair of CTAs over a list of tasks, each given by its number of blocks."""

    def __init__(self, source, codes, tasks, rng):
        self.source, self.codes, self.tasks, self.rng = source, codes, tasks, rng
        self.bars = [{name: [Barrier(source.count(name, codes, rank), f"{name}[{i}] of rank {rank}") for i in range(n)]
                      for name, n in SIZES.items()} for rank in (0, 1)]
        self.products, self.copies = [], []      # committed, in order; under way, in any
        self.info = [[None] * 8, [None] * 8]     # the tile that each description is of
        self.stage = [[None] * 4, [None] * 4]    # codes: the stage that each place of V's ring holds
        self.roles = []
        for rank in (0, 1):
            add = lambda name, gen: self.roles.append([f"{name} of rank {rank}", gen, next(gen), rng.choice([.05, .3, 1, 1, 3])])
            add("tasks", self._tasks(rank))
            add("logits", self._logits(rank))
            add("P.V", self._pv(rank))
            if codes:
                add("descriptions", self._describe(rank))
                for is_v in (0, 1):
                    for turn in (0, 1):
                        for w in range(4):
                            add(f"{'KV'[is_v]}'s widening warp {turn} {w}", self._widen(rank, is_v, turn))
            else:
                add("K's loads", self._load(rank, False))
                add("V's loads", self._load(rank, True))
                add("Q's loads", self._load_q_of_tasks(rank))
            for grp in (0, 1):
                for w in range(4):
                    add(f"softmax {grp} {w}", self._softmax(rank, grp, w))
            for _ in range(1 if codes else 2):
                for w in range(4):
                    add(f"epilogue {w}", self._epilogue(rank, w))
        assert len(self.roles) == 2 * (32 if codes else 22)

    # -- the roles: ("wait" or "test", barrier, phase) and ("step",)

    def _fetch(self, rank, nth):
        yield "wait", self.bars[rank]["task_full"][nth % 4], nth // 4
        self.bars[rank]["task_empty"][nth % 4].arrive()
        yield ("step",)
        return self.tasks[nth] if nth < len(self.tasks) else None

    def _each_task(self, rank, body):
        nth = 0
        while (nb := (yield from self._fetch(rank, nth))) is not None:
            yield from body(nb)
            nth += 1

    def _both(self, name, i):
        return self.bars[0][name][i], self.bars[1][name][i]

    def _load_q(self, rank, nth):
        for q in range(4):
            yield "wait", self.bars[rank]["q_empty"][q], nth - 1
            full = self.bars[0]["q_full"][q]
            if rank == 0:
                full.arrive(2)
            self.copies.append(full.landed)
            yield ("step",)

    def _tasks(self, rank):
        loaded = 0
        for i in range(len(self.tasks) + 1):
            yield "wait", self.bars[rank]["task_empty"][i % 4], i // 4 - 1
            self.bars[rank]["task_full"][i % 4].arrive()
            yield ("step",)
            if self.codes and i < len(self.tasks) and self.tasks[i]:
                yield from self._load_q(rank, loaded)
                loaded += 1

    def _load_q_of_tasks(self, rank):
        loaded = 0

        def body(nb):
            nonlocal loaded
            if nb:
                yield from self._load_q(rank, loaded)
                loaded += 1
        yield from self._each_task(rank, body)

    def _logits(self, rank):
        m = g = c = 0

        def body(nb):
            nonlocal m, g, c
            if rank or nb == 0:
                return
            last = (nb + 3) // 4 - 1
            for i in range(last + 1):
                yield "wait", self.bars[0]["s_empty"][g % 3], g // 3 - 1
                for q in range(4):
                    if i == 0:
                        yield "wait", self.bars[0]["q_full"][q], c
                    yield "wait", self.bars[0]["k_full"][m % 4], m // 4
                    if i == last:
                        self.products.append(self._both("q_empty", q))
                    self.products.append(self._both("k_empty", m % 4))
                    m += 1
                    yield ("step",)
                self.products.append(self._both("s_full", g % 3))
                g += 1
            c += 1
        yield from self._each_task(rank, body)

    def _pv(self, rank):
        m = g = c = 0

        def body(nb):
            nonlocal m, g, c
            if nb == 0 or (self.codes and rank):
                return
            for i in range(0, nb, 4):
                if rank == 0:
                    yield "wait", self.bars[0]["p_full"][g & 1], g >> 1
                    if i == 0:
                        yield "wait", self.bars[0]["o_empty"][0], c - 1
                for _ in range(min(4, nb - i)):
                    yield "wait", self.bars[rank]["v_full"][m % 4], m // 4
                    if rank:
                        self.bars[0]["v_full"][m % 4].arrive()
                    else:
                        if self.codes and (self.stage[0][m % 4], self.stage[1][m % 4]) != (m, m):
                            raise Fault(f"V's stage {m} was written over")
                        self.products.append(self._both("v_empty", m % 4))
                    m += 1
                    yield ("step",)
                if rank == 0:
                    self.products.append(self._both("p_empty", g & 1))
                    if i + 4 >= nb:
                        self.products.append(self._both("o_full", 0))
                g += 1
            c += 1
        yield from self._each_task(rank, body)

    def _describe_tile(self, rank, g):
        yield ("step",)
        self.info[rank][g % 8] = g
        self.bars[rank]["info_full"][g % 8].arrive()
        yield ("step",)

    def _described(self, rank, g):
        if self.info[rank][g % 8] != g:
            raise Fault(f"the description of tile {g} is one of {self.info[rank][g % 8]}")

    def _load(self, rank, is_v):
        m = g = 0
        full, empty = ("v_full", "v_empty") if is_v else ("k_full", "k_empty")

        def body(nb):
            nonlocal m, g
            for i in range(0, nb, 4):
                blocks = min(4, nb - i)
                if not is_v:
                    yield from self._describe_tile(rank, g)
                for _ in range(blocks if is_v else 4):
                    yield "wait", self.bars[rank][empty][m % 4], m // 4 - 1
                    bar = self.bars[rank if is_v else 0][full][m % 4]
                    if is_v or rank == 0:
                        bar.arrive(1 if is_v else blocks)
                    elif self.source.rank1_arrives:
                        bar.arrive()
                    self.copies += [bar.landed] * (1 if is_v else (blocks - rank + 1) // 2)
                    m += 1
                    yield ("step",)
                g += 1
        yield from self._each_task(rank, body)

    def _describe(self, rank):
        g = 0

        def body(nb):
            nonlocal g
            for _ in range(0, nb, 4):
                yield "wait", self.bars[rank]["info_empty"][g % 8], g // 8 - 1
                yield from self._describe_tile(rank, g)
                g += 1
        yield from self._each_task(rank, body)

    def _widen(self, rank, is_v, turn):
        seq = g = 0
        bars = self.bars[rank]
        full, empty = ("v_full", "v_empty") if is_v else ("k_full", "k_empty")

        def body(nb):
            nonlocal seq, g
            tiles = (nb + 3) // 4
            stages = nb if is_v else 4 * tiles
            first = put = eval(self.source.first_stage, {"turn": turn, "seq": seq})
            for n in range(first, stages, 2):
                while put < stages and put <= n + 2:
                    m, tile = seq + put, g + (put >> 2)
                    if put > n and not (yield "test", bars[empty][m % 4], m // 4 - 1):
                        break
                    if (put & 2) == 0:
                        yield "wait", bars["info_full"][tile % 8], tile // 8
                    yield "wait", bars[empty][m % 4], m // 4 - 1
                    self._described(rank, tile)
                    if is_v:
                        self.stage[rank][m % 4] = m
                    if (put & 2) or put + 2 >= stages:
                        bars["info_empty"][tile % 8].arrive()
                    put += 2
                    yield ("step",)
                yield ("step",)
                if is_v and rank:
                    bars[full][(seq + n) % 4].arrive()
                self.bars[0][full][(seq + n) % 4].arrive()
            if is_v and first and (stages & 3) == 1:
                tile = g + tiles - 1
                yield "wait", bars["info_full"][tile % 8], tile // 8
                bars["info_empty"][tile % 8].arrive()
            seq += stages
            g += tiles
        yield from self._each_task(rank, body)

    def _softmax(self, rank, grp, w):
        g = c = v = 0
        bars = self.bars[rank]
        pair = 2 * grp + (w & 1)

        def body(nb):
            nonlocal g, c, v
            for i in range(0, nb, 4):
                v0, blocks, b = v, min(4, nb - i), g & 1
                v += blocks
                if b == grp:
                    yield "wait", bars["info_full"][g % 8], g // 8
                    yield "wait", bars["s_full"][g % 3], g // 3
                    self._described(rank, g)
                    yield ("step",)
                    self._described(rank, g)
                    if self.codes:
                        bars["info_empty"][g % 8].arrive()
                    yield "wait", bars["mx_empty"][pair], (g >> 1) - 1
                    bars["pair_bar"][pair].arrive()
                    yield "wait", bars["pair_bar"][pair], g >> 1
                    bars["mx_empty"][pair].arrive()
                    yield "wait", bars["p_empty"][b], (g >> 1) - 1
                    if g:
                        yield "wait", bars["m_full"][w], g - 1
                    bars["m_full"][w].arrive()
                    yield ("step",)
                    self.bars[0]["s_empty"][g % 3].arrive()
                    yield ("step",)
                    if self.rng.random() < 0.5:      # O is rescaled, and rows of V are cleared
                        if g:
                            yield "wait", bars["p_empty"][b ^ 1], (g - 1) >> 1
                        for j in ((w >> 1), (w >> 1) + 2):
                            if j < blocks:
                                yield "wait", bars["v_full"][(v0 + j) % 4], (v0 + j) // 4
                        yield ("step",)
                    self.bars[0]["p_full"][b].arrive()
                g += 1
            yield "wait", bars["stats_empty"][0], c - 1
            bars["stats_full"][0].arrive()
            c += 1
            yield ("step",)
        yield from self._each_task(rank, body)

    def _epilogue(self, rank, w):
        c = o = 0
        bars = self.bars[rank]

        def body(nb):
            nonlocal c, o
            yield "wait", bars["stats_full"][0], c
            if nb:
                yield "wait", bars["o_full"][0], o
            bars["stats_empty"][0].arrive()
            yield "wait", bars["sum_empty"][w & 1], c - 1
            bars["sum_full"][w & 1].arrive()
            yield "wait", bars["sum_full"][w & 1], c
            yield ("step",)
            bars["sum_empty"][w & 1].arrive()
            c += 1
            yield ("step",)
            if nb:
                self.bars[0]["o_empty"][0].arrive()
                o += 1
                yield ("step",)
        yield from self._each_task(rank, body)

    # -- a random order

    def _advance(self, role):
        name, gen, op, _ = role
        send = None
        if op[0] != "step":
            kind, bar, phase = op
            passes = bar.complete % 2 != phase % 2
            if passes and bar.complete <= phase:
                raise Fault(f"{name} passes {bar.name} before phase {phase}: {bar.complete} complete")
            if bar.complete > phase + 1:
                raise Fault(f"{name} comes too late for phase {phase} of {bar.name}: {bar.complete} complete")
            if kind == "wait" and not passes:
                return False
            send = passes if kind == "test" else None
        try:
            role[2] = gen.send(send)
        except StopIteration:
            role[2] = None
        return True

    def run(self):
        rng = self.rng
        tensor, memory = rng.choice([.02, .2, .6]), rng.choice([.02, .2, .6])
        idle = 0
        while live := [r for r in self.roles if r[2]]:
            moved = False
            for role in rng.choices(live, [r[3] for r in live], k=40):
                moved |= bool(role[2]) and self._advance(role)
                if self.products and rng.random() < tensor:
                    for bar in self.products.pop(0):
                        bar.arrive()
                    moved = True
                if self.copies and rng.random() < memory:
                    self.copies.pop(rng.randrange(len(self.copies)))()
                    moved = True
            idle = 0 if moved else idle + 1
            if idle > 50 and not (any(self._advance(r) for r in live) or self.products or self.copies):
                raise Fault("every role waits: " + ", ".join(f"{r[0]} for phase {r[2][2]} of {r[2][1].name}" for r in live))
