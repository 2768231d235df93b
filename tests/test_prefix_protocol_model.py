"""A randomised CPU model of the shared-prefix kernel's synchronisation
(csrc/prefix_decode_kernel.cu), checked under random interleavings: the TMA
producer, the e4m3 converters, the two MMA warps with their in-order tensor
pipes and the two softmax warpgroups run as step-wise processes over the same
random pieces; mbarriers have their hardware semantics (phases, arrival counts,
waits on a phase PARITY only).

With one new token per sequence the pieces of own tiles come last and run
differently: each softmax warp takes every 8th tile straight from the ring (after
the slot's issued word, as its phases go to different warps), leaves its state in
one of two buffers in the Q slots, and MMA warp g joins the pieces of parity g.

Checked: no wait passes on a stale phase, no buffer is overwritten before its
reader is done (Q slots, ring slots, S, P, O during a rescale and while the two
states are joined, the exchanged maxima), no MMA reads a Q slot before it is
filled (and converted), every state that leaves holds exactly the piece's tiles,
every role finishes. The model mirrors the kernel's waits one for one; a change
to either must keep them in step."""
import random

import pytest

WAIT = "wait"


class Barrier:
    def __init__(self, name, count):
        self.name, self.count, self.pending, self.completed = name, count, count, 0

    def arrive(self):
        self.pending -= 1
        assert self.pending >= 0, f"{self.name}: too many arrivals"
        if self.pending == 0:
            self.completed, self.pending = self.completed + 1, self.count

    def ready(self, phase):
        ok = (self.completed & 1) != (phase & 1)
        if ok:
            assert self.completed >= phase + 1, f"{self.name}: stale pass of phase {phase} at {self.completed}"
        return ok


class Model:
    def __init__(self, rng, fp8, pieces, stages, stages8, warp_pieces=()):
        self.rng, self.fp8, self.pieces, self.S, self.S8 = rng, fp8, pieces, stages, stages8
        self.warp_pieces = list(warp_pieces)
        B = Barrier
        two = lambda name, n: [B(f"{name}{i}", n) for i in range(2)]
        self.q_full, self.q_empty, self.q_ready = two("q_full", 1), two("q_empty", 2), two("q_ready", 1)
        self.kv_full = [B(f"kv_full{s}", 1) for s in range(stages)]
        self.kv_empty = [B(f"kv_empty{s}", 2) for s in range(stages)]
        self.kv8_full = [B(f"kv8_full{s}", 1) for s in range(stages8)]
        self.kv8_empty = [B(f"kv8_empty{s}", 1) for s in range(stages8)]
        self.x_full, self.x_free = B("x_full", 1), B("x_free", 1)
        self.dep_full, self.dep_free = two("dep_full", 8), two("dep_free", 1)
        self.q_done = B("q_done", 2)
        # warp pieces: the ring of BF16, or e4m3 slots over the space of both rings
        self.W = 2 * stages + stages8 if fp8 else stages
        self.w_full = [B(f"w_full{s}", 1) for s in range(self.W)] if fp8 else self.kv_full
        self.w_empty = [B(f"w_empty{s}", 1) for s in range(self.W)] if fp8 else self.kv_empty
        self.w_ring = [None] * self.W
        self.word = [None] * self.W      # tile issued into a slot
        self.dep = [{}, {}]              # warp -> (piece, its tiles) in a buffer
        self.joined = []                 # (piece, tiles) written out
        self.s_full = [two(f"s_full{g}.", 1) for g in range(2)]
        self.p_full = [two(f"p_full{g}.", 1) for g in range(2)]
        self.pv_done = [two(f"pv_done{g}.", 1) for g in range(2)]
        self.tma, self.pipe, self.tick = [], [[], []], 0
        self.q = [None, None]            # (piece, converted) in a Q slot
        self.scale = [[None, None], [None, None]]  # of a slot's last two fills
        self.q_readers = [set(), set()]  # S MMAs issued on a slot, not complete
        self.q_left = [set(), set()]     # pipelines that have not let go of a slot's fill
        self.ring, self.ring8 = [None] * stages, [None] * stages8
        self.ring_reads = {}             # tile -> readers outstanding
        self.s_buf, self.s_read = [[None, None], [None, None]], [[True, True], [True, True]]
        self.p_buf = [[None, None], [None, None]]
        self.pv_reads = [[None, None], [None, None]]
        self.o = [[], []]                # tiles accumulated in O of a pipeline
        self.pv_open = [0, 0]            # P V issued and not complete
        self.o_joining = False           # warpgroup 0 reads both O
        self.x = None
        self.out = []

    def tiles(self):
        kt = 0
        for i, (n, two) in enumerate(self.pieces):
            yield i, n, two, kt
            kt += n

    @staticmethod
    def mine(n, two, g):
        return list(range(n)) if two else list(range(g, n, 2))

    def slots(self):
        ones, uses = 0, [0, 0]
        for n, two in self.pieces:
            sl = [0, 1] if two else [ones & 1]
            yield sl, list(uses)
            for s in sl:
                uses[s] += 1
            ones += not two

    def until(self, bar, phase):
        while not bar.ready(phase):
            yield WAIT

    # ---------------------------------------------------------------- roles
    def producer(self):
        for (i, n, two, kt), (slots, uses) in zip(self.tiles(), self.slots()):
            for s in slots:
                if uses[s]:
                    yield from self.until(self.q_empty[s], uses[s] - 1)
                assert not self.q_readers[s] and not self.q_left[s], "Q slot overwritten while read"
                self.q[s] = None

                def land(s=s, i=i):
                    self.q[s], self.q_left[s] = (i, not self.fp8), {0, 1}
                    self.q_full[s].arrive()
                self.tma.append((self.tick + self.rng.randint(1, 25), land))
                yield
            for j in range(n):
                k = kt + j
                full, empty, S = (self.kv8_full, self.kv8_empty, self.S8) if self.fp8 else \
                    (self.kv_full, self.kv_empty, self.S)
                if k >= S:
                    yield from self.until(empty[k % S], k // S - 1)
                if not self.fp8:
                    self.fill(k, two)

                def land(k=k, full=full, S=S):
                    if self.fp8:
                        self.ring8[k % S] = k
                    else:
                        self.ring[k % S] = k
                    full[k % S].arrive()
                self.tma.append((self.tick + self.rng.randint(1, 30), land))
                yield
        kt = 0 if self.fp8 else sum(n for n, _ in self.pieces)
        full, empty, S = self.w_full, self.w_empty, self.W
        if self.fp8 and self.warp_pieces:
            yield from self.until(self.q_done, 0)
            assert not any(self.ring_reads.values()) and not any(self.pv_open), "rings in use"
            assert all(b.pending == b.count for b in self.kv8_empty), "a converter reads its ring"
        ring = self.w_ring if self.fp8 else self.ring
        for n in self.warp_pieces:
            for k in range(kt, kt + n):
                if k >= S:
                    yield from self.until(empty[k % S], k // S - 1)
                assert not self.ring_reads.get(ring[k % S]), "ring slot overwritten"
                ring[k % S], self.word[k % S], self.ring_reads[("w", k)] = None, k, 1

                def land(k=k):
                    ring[k % S] = ("w", k)
                    full[k % S].arrive()
                self.tma.append((self.tick + self.rng.randint(1, 30), land))
                yield
            kt += n

    def consumer(self, w):
        """Softmax warp w in the warp pieces."""
        joins = sum(1 for n, two in self.pieces if not two and n > 1)
        full, empty, S = self.w_full, self.w_empty, self.W
        kt = 0 if self.fp8 else sum(n for n, _ in self.pieces)
        for i, n in enumerate(self.warp_pieces):
            got = []
            for j in range((w - kt) % 8, n, 8):
                k = kt + j
                while self.word[k % S] != k:
                    yield WAIT
                yield from self.until(full[k % S], k // S)
                ring = self.w_ring if self.fp8 else self.ring
                assert ring[k % S] == ("w", k)
                for _ in range(self.rng.randint(0, 6)):
                    yield
                assert ring[k % S] == ("w", k)
                got.append(j)
                self.ring_reads[("w", k)] = 0
                for _ in range(empty[k % S].count):
                    empty[k % S].arrive()
            buf, use = i & 1, i >> 1
            if use:
                yield from self.until(self.dep_free[buf], use - 1)
            else:
                yield from self.until(self.q_done, 0)
                if joins:
                    yield from self.until(self.x_free, joins - 1)
                assert not self.q_readers[buf] and not self.q_left[buf], "state over a Q slot in use"
                assert not self.o_joining, "state over the join cells in use"
            assert w not in self.dep[buf], "state overwritten"
            self.dep[buf][w] = (i, got)
            yield
            self.dep_full[buf].arrive()
            kt += n

    def join_warps(self, g):
        """MMA warp g behind its last MMA: the pieces of parity g."""
        if self.warp_pieces:
            self.commit(g, self.q_done)
        for i, n in enumerate(self.warp_pieces):
            if i & 1 == g:
                yield from self.until(self.dep_full[g], i >> 1)
                tiles = []
                for w in range(8):
                    piece, got = self.dep[g][w]
                    assert piece == i
                    tiles += got
                    yield
                self.joined.append((i, sorted(tiles)))
                self.dep[g] = {}
                self.dep_free[g].arrive()

    def fill(self, k, two):
        old = self.ring[k % self.S]
        assert not self.ring_reads.get(old), f"ring slot of tile {old} overwritten"
        self.ring[k % self.S] = None
        self.ring_reads[k] = 4 if two else 2  # S and P V of each pipeline that takes it

    def converter(self):
        for i, n, two, kt in self.tiles():
            for j in range(n):
                k = kt + j
                yield from self.until(self.kv8_full[k % self.S8], k // self.S8)
                if k >= self.S:
                    yield from self.until(self.kv_empty[k % self.S], k // self.S - 1)
                assert self.ring8[k % self.S8] == k
                self.fill(k, two)
                for _ in range(self.rng.randint(0, 4)):
                    yield
                assert self.ring8[k % self.S8] == k
                self.ring[k % self.S] = k
                self.kv8_empty[k % self.S8].arrive()
                self.kv_full[k % self.S].arrive()

    def op(self, g, start, end):
        self.pipe[g].append([self.rng.randint(1, 8), start, end, False])

    def commit(self, g, bar):
        self.pipe[g].append([0, lambda: None, bar.arrive, False])

    def mma(self, g):
        c = 0
        for (i, n, two, kt), (slots, uses) in zip(self.tiles(), self.slots()):
            mine, my = self.mine(n, two, g), g if two else slots[0]

            def issue_s(q):
                k = kt + mine[q]
                self.q_readers[my].add((g, q))

                def start(k=k, i=i, my=my, b=(c + q) & 1):
                    assert self.q[my] == (i, True), "S on a Q slot that is not ready"
                    assert self.ring[k % self.S] == k and self.s_read[g][b]
                    assert self.pv_reads[g][b] is None, "S over a P in use"

                def end(k=k, q=q, i=i, my=my, b=(c + q) & 1):
                    self.ring_reads[k] -= 1
                    self.q_readers[my].discard((g, q))
                    self.s_buf[g][b], self.s_read[g][b] = (i, q), False
                self.op(g, start, end)
                self.commit(g, self.s_full[g][(c + q) & 1])
                if q + 1 == len(mine):
                    def let_go(my=my):
                        self.q_left[my].discard(g)
                        self.q_empty[my].arrive()
                    self.pipe[g].append([0, lambda: None, let_go, False])

            def issue_pv(q):
                k, x = kt + mine[q], c + q
                self.pv_reads[g][x & 1] = x
                self.pv_open[g] += 1

                def start(k=k, x=x, q=q, i=i):
                    assert self.p_buf[g][x & 1] == (i, q) and self.ring[k % self.S] == k
                    assert not self.o_joining or not (g == 1 and q == 0)
                    if q == 0:
                        self.o[g] = []

                def end(k=k, x=x, tile=(i, mine[q])):
                    self.o[g].append(tile)
                    self.ring_reads[k] -= 1
                    self.pv_reads[g][x & 1] = None
                    self.pv_open[g] -= 1
                self.op(g, start, end)
                self.commit(g, self.pv_done[g][x & 1])
                self.commit(g, self.kv_empty[k % self.S])

            for s in slots:
                yield from self.until((self.q_ready if self.fp8 else self.q_full)[s], uses[s])
                if s != my or not mine:
                    self.q_left[s].discard(g)
                    self.q_empty[s].arrive()
            s = v = j = 0
            while v < len(mine) or j < n:
                did, own = False, two or j % 2 == g
                if j < n and (not own or s < v + 2):
                    k = kt + j
                    if self.kv_full[k % self.S].ready(k // self.S):
                        if own:
                            issue_s(s)
                            s += 1
                        else:
                            self.kv_empty[k % self.S].arrive()
                        j, did = j + 1, True
                        yield
                if v < s and self.p_full[g][(c + v) & 1].ready((c + v) >> 1):
                    issue_pv(v)
                    v, did = v + 1, True
                    yield
                if not did:
                    yield WAIT
            c += len(mine)
        yield from self.join_warps(g)

    def softmax(self, g):
        count, joins = [0, 0], 0
        for (i, n, two, kt), (slots, uses) in zip(self.tiles(), self.slots()):
            mines = [self.mine(n, two, 0), self.mine(n, two, 1)]
            mine, c, my = mines[g], count[g], g if two else slots[0]
            if self.fp8 and my == g:
                yield from self.until(self.q_full[g], uses[g])
                assert self.q[g] == (i, False)
                yield
                self.q[g] = (i, True)
                self.scale[g][uses[g] & 1] = i
                self.q_ready[g].arrive()
            for q in range(len(mine)):
                x = c + q
                yield from self.until(self.s_full[g][x & 1], x >> 1)
                if self.fp8 and q == 0:
                    assert self.scale[my][uses[my] & 1] == i, "scale of another fill"
                if g == 1 and q == 0 and joins:
                    yield from self.until(self.x_free, joins - 1)
                assert self.s_buf[g][x & 1] == (i, q) and not self.s_read[g][x & 1]
                yield
                assert self.s_buf[g][x & 1] == (i, q)
                self.s_read[g][x & 1] = True
                for _ in range(self.rng.randint(0, 4)):
                    yield
                if q > 0 and self.rng.random() < 0.4:  # rescale O
                    yield from self.until(self.pv_done[g][(x - 1) & 1], (x - 1) >> 1)
                    assert self.pv_open[g] == 0, "O rescaled under a running P V"
                    yield
                    assert self.pv_open[g] == 0
                assert self.pv_reads[g][x & 1] is None, "P overwritten while read"
                self.p_buf[g][x & 1] = (i, q)
                self.p_full[g][x & 1].arrive()
            join = not two and n > 1
            if not (g == 1 and not two):
                last = c + len(mine) - 1
                yield from self.until(self.pv_done[g][last & 1], last >> 1)
                got = list(self.o[g])
                if join:
                    last1 = count[1] + len(mines[1]) - 1
                    yield from self.until(self.x_full, joins)
                    yield from self.until(self.pv_done[1][last1 & 1], last1 >> 1)
                    self.o_joining = True
                    assert self.x == i and self.o[1] == [(i, t) for t in mines[1]]
                    yield
                    assert self.x == i and self.o[1] == [(i, t) for t in mines[1]]
                    got += self.o[1]
                    self.o_joining = False
                    self.x_free.arrive()
                assert got == [(i, t) for t in mine] + ([(i, t) for t in mines[1]] if join else [])
                self.out.append((i, g))
            elif join:
                self.x = i
                self.x_full.arrive()
            joins += join
            count = [count[0] + len(mines[0]), count[1] + len(mines[1])]
        self.more += [self.consumer(w) for w in range(4 * g, 4 * g + 4)]

    def run(self):
        roles = [self.producer(), self.mma(0), self.mma(1), self.softmax(0), self.softmax(1)]
        if self.fp8:
            roles.append(self.converter())
        weights = [self.rng.choice([1, 1, 3, 10]) for _ in roles]  # some run ahead, some lag
        idle, self.more = 0, []
        while roles or self.more or self.tma or any(self.pipe):
            self.tick += 1
            moved = False
            for t in [t for t in self.tma if t[0] <= self.tick]:
                self.tma.remove(t)
                t[1]()
                moved = True
            for g in range(2):
                if self.pipe[g] and self.rng.random() < 0.5:
                    head = self.pipe[g][0]
                    if not head[3]:
                        head[1]()
                        head[3] = True
                    head[0] -= 1
                    moved = True
                    if head[0] <= 0:
                        self.pipe[g].pop(0)
                        head[2]()
            weights += [self.rng.choice([1, 1, 3, 10]) for _ in self.more]
            roles, self.more = roles + self.more, []
            if roles:
                r = self.rng.choices(range(len(roles)), weights)[0]
                try:
                    moved |= next(roles[r]) is not WAIT
                except StopIteration:
                    roles.pop(r)
                    weights.pop(r)
                    moved = True
            idle = 0 if moved or self.tma else idle + 1
            assert idle < 3000, "deadlock"
        assert sorted(self.out) == sorted((i, g) for i, (n, two) in enumerate(self.pieces)
                                          for g in ((0, 1) if two else (0,)))
        assert sorted(self.joined) == [(i, list(range(n))) for i, n in enumerate(self.warp_pieces)]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("seed", range(12))
def test_no_stale_wait_no_overwrite_no_deadlock(fp8, seed):
    rng = random.Random(seed * 2 + fp8)
    for _ in range(25):
        pieces = [(rng.choice([1, 1, 2, 3, 4, 5, 9]), rng.random() < 0.4) for _ in range(rng.randint(1, 8))]
        last = [rng.choice([1, 2, 5, 8, 9, 20]) for _ in range(rng.choice([0, 0, 1, 3, 7]))]
        Model(rng, fp8, pieces if rng.random() < 0.9 or not last else [], *((3, 4) if fp8 else (5, 0)), last).run()


def test_the_model_sees_a_missing_wait():
    """The checks bite: without warpgroup 1's wait for the joined state, or with
    one MMA warp's arrival on a ring slot taken as enough, some run fails."""
    class NoJoinWait(Model):
        def until(self, bar, phase):
            if bar is self.x_free:
                return
            yield from super().until(bar, phase)

    class OneArrival(Model):
        def __init__(self, *a):
            super().__init__(*a)
            for b in self.kv_empty:
                b.count = b.pending = 1

    class OneScale(Model):  # a slot's scales kept for one fill only
        def __init__(self, *a):
            super().__init__(*a)
            for s in range(2):
                class Cell(list):
                    def __getitem__(self, i):
                        return list.__getitem__(self, 0)

                    def __setitem__(self, i, v):
                        list.__setitem__(self, 0, v)
                self.scale[s] = Cell([None])

    class NoWord(Model):  # a warp trusts the parity alone
        def __init__(self, *a):
            super().__init__(*a)

            class Any(list):
                def __getitem__(self, i):
                    return Always()

            class Always:
                def __ne__(self, other):
                    return False
            self.word = Any(self.word)

    class NoSlotWait(Model):  # states go to the Q slots without asking for them
        def until(self, bar, phase):
            if bar is self.q_done:
                return
            yield from super().until(bar, phase)

    for broken in (NoJoinWait, OneArrival, OneScale, NoWord, NoSlotWait):
        failed = 0
        for seed in range(200):
            rng = random.Random(seed)
            pieces = [(rng.choice([1, 1, 2, 3, 4]), rng.random() < 0.3) for _ in range(12)]
            try:
                last = [rng.choice([1, 3, 9]) for _ in range(6)] if broken in (NoWord, NoSlotWait) else []
                broken(rng, broken is OneScale, pieces, *((3, 4) if broken is OneScale else (5, 0)), last).run()
            except AssertionError:
                failed += 1
        assert failed, broken.__name__
