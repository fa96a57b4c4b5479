"""The barriers of attn_fwd_varlen_kernel on the host: one CTA's roles as generators that yield
what they wait for, copies and products done at once.

A role's waits are all blocking ones, so whether the roles finish does not depend on their
speeds: one order of steps stands for all.  A wait names the phase that it means; as the
kernel's, it passes on that phase's parity alone, and the model checks that it was that phase.
"""

SLOTS, STAGES = 4, 4  # kVlSlots, kStagesWs


class Barrier:
    def __init__(self, count):
        self.count = self.left = count
        self.done = 0  # completed phases

    def arrive(self, n=1):
        self.left -= n
        assert self.left >= 0, "an arrival too many"
        if self.left == 0:
            self.done += 1
            self.left = self.count

    def passed(self, phase):
        """Wait for phase `phase` (-1: the one before the first) by its parity."""
        if (self.done & 1) == (phase & 1):
            return False
        assert self.done == phase + 1, "the wait saw another phase of the same parity"
        return True


def blocks_in_order(lens_q, lens_k, block, causal):
    """(sequence, block of rows) in the order of VlWalk: by level, the number of key blocks seen."""
    levels = {}
    for s, (nq, nk) in enumerate(zip(lens_q, lens_k)):
        nqb, high = -(-nq // block), -(-nk // block)
        for b in range(nqb):
            levels.setdefault(high - (nqb - 1 - b) if causal else high, []).append((s, b))
    return [x for level in sorted(levels, reverse=True) for x in levels[level]]


def units_of_ctas(lens_q, lens_k, Hq, Hkv, causal, ctas):
    """Each CTA's units (n0, n1, g0) in the scheduler's order, dealt in snake order."""
    pair = (Hq // Hkv) % 2 == 0
    block = 128 if pair else 256
    heads = Hq // 2 if pair else Hq
    order = blocks_in_order(lens_q, lens_k, block, causal)
    total = len(order) * heads

    def unit(t):
        s, b = order[t // heads]
        nk, rows = lens_k[s], lens_q[s] - b * block
        rel = nk - rows
        n = []
        for i in range(2):
            row0 = 0 if pair else 128 * i
            valid = max(0, min(128, rows - row0))
            seen = min(nk, rel + row0 + valid) if causal else nk
            n.append(-(-seen // 128) if valid > 0 and seen > 0 else 0)
        whole = min(nk, rel + 1) if causal else nk
        return (*n, max(0, whole) // 128)

    grid = min(ctas, total)
    lists = [[] for _ in range(grid)]
    for t in range(total):
        r, c = divmod(t, grid)
        lists[grid - 1 - c if r & 1 else c].append(unit(t))
    return lists


class Cta:
    """Units (n0, n1, g0): key tiles of the two query tiles, first guarded key tile.  With
    ``hand_out_all`` those without keys go through the slots, too."""

    def __init__(self, units, hand_out_all=False):
        self.blind = [] if hand_out_all else [u for u in units if max(u[:2]) == 0]  # stored by the scheduler
        self.units = [u for u in units if hand_out_all or max(u[:2]) > 0]
        two = range(2)
        self.q_full = [Barrier(1) for _ in two]
        self.kv_full = [Barrier(1) for _ in range(STAGES)]
        self.kv_empty = [Barrier(1 + (s & 1)) for s in range(STAGES)]
        self.s_full = [Barrier(1) for _ in two]
        self.p_full = [Barrier(4) for _ in two]
        self.o_full = [Barrier(1) for _ in two]
        self.o_empty = [Barrier(4) for _ in two]
        self.v_ok = [Barrier(1) for _ in two]
        self.unit_full = [Barrier(1) for _ in range(SLOTS)]
        self.unit_empty = [Barrier(11) for _ in range(SLOTS)]
        self.slot = [None] * SLOTS      # the descriptor in each slot (0: no more units)
        self.stage = [None] * STAGES    # the tile in each stage
        self.stored = []                # (tile, unit) in the order of their stores
        self.scores = [[], []]          # (unit, key tile) of each score product

    def scheduler(self):
        for t, u in enumerate(self.units + [0]):
            s = t % SLOTS
            yield self.unit_empty[s], t // SLOTS - 1
            self.slot[s] = 0 if u == 0 else (t, *u)
            self.unit_full[s].arrive()

    def fetch(self, at):
        """The next descriptor with keys behind the at-th one (0: none) and where it was."""
        while True:
            s = at % SLOTS
            yield self.unit_full[s], at // SLOTS
            u = self.slot[s]
            self.unit_empty[s].arrive()
            at += 1
            if u == 0 or max(u[1:3]) > 0:  # (always, where only units with keys are handed out)
                return u, at

    def producer(self):
        ring, at, scores = 0, 0, [0, 0]

        def load_q(u):
            for i in range(2):
                if u[1 + i] == 0:
                    continue
                if scores[i] > 0:
                    yield self.s_full[i], scores[i] - 1
                self.q_full[i].arrive()

        cur, at = yield from self.fetch(at)
        if cur:
            self.stage[0] = ("K", cur[0], 0)
            self.kv_full[0].arrive()
            ring = 1
            yield from load_q(cur)
        while cur:
            n = max(cur[1:3])
            for j in range(n):
                nxt, key = cur, j + 1
                if j + 1 == n:
                    nxt, at = yield from self.fetch(at)
                    key = 0
                vs, ks = ring % STAGES, (ring + 1) % STAGES
                yield self.kv_empty[vs], ring // STAGES - 1
                if nxt:
                    yield self.kv_empty[ks], (ring + 1) // STAGES - 1
                    self.stage[ks] = ("K", nxt[0], key)
                self.stage[vs] = ("V", cur[0], j)
                self.kv_full[vs].arrive()  # V_j and the K tile after it
                ring += 2 if nxt else 1
            scores = [scores[0] + cur[1], scores[1] + cur[2]]
            cur = nxt
            if cur:
                yield from load_q(cur)

    def issuer(self):
        ring, at, full = 0, 0, [0] * STAGES
        pn, qn, on, vn = [0, 0], [0, 0], [0, 0], [0, 0]
        cur, start = (-1, 0, 0, 1 << 30), True
        while cur:
            n = 1 if start else max(cur[1:3])
            for j in range(n):
                vs = ring % STAGES
                if not start:
                    ring += 1
                ks = ring % STAGES
                last, nxt = j + 1 == n, 0
                if last:
                    nxt, at = yield from self.fetch(at)
                if start and not nxt:
                    break
                yield self.kv_full[vs], full[vs]
                full[vs] += 1
                if j >= cur[3]:
                    yield self.v_ok[vs >> 1], vn[vs >> 1]
                    vn[vs >> 1] += 1
                for i in range(2):
                    n_i = cur[1 + i]
                    if j < n_i:
                        yield self.p_full[i], pn[i]
                        pn[i] += 1
                        if j == 0:
                            yield self.o_empty[i], on[i] - 1
                            on[i] += 1
                        assert self.stage[vs] == ("V", cur[0], j)
                        if j == n_i - 1:
                            self.o_full[i].arrive()
                    if i == 1 and not start:
                        self.kv_empty[vs].arrive()
                    first = last and bool(nxt) and nxt[1 + i] > 0
                    if j + 1 < n_i or first:
                        if first:
                            yield self.q_full[i], qn[i]
                            qn[i] += 1
                        at_tile = (nxt[0], 0) if first else (cur[0], j + 1)
                        assert self.stage[ks] == ("K", *at_tile)
                        self.scores[i].append(at_tile)
                        self.s_full[i].arrive()
                if not last or nxt:
                    self.kv_empty[ks].arrive()
                    ring += 1
                start = False
            cur = nxt

    def guard(self):
        at = tiles = 0
        while True:
            s = at % SLOTS
            yield self.unit_full[s], at // SLOTS
            u = self.slot[s]
            if u == 0:
                return
            for j in range(max(u[1:3])):
                vs = 1 + 2 * (tiles & 1)
                yield self.kv_full[vs], tiles >> 1
                assert self.stage[vs] == ("V", u[0], j)
                if j >= u[3]:
                    self.v_ok[tiles & 1].arrive()
                self.kv_empty[vs].arrive()
                tiles += 1
            self.unit_empty[s].arrive()
            at += 1

    def softmax(self, i):
        at, sn, on, j, n, cur, done = -1, 0, 0, 0, 0, None, None
        while True:
            if j == n:
                done, at = cur, at + 1
                yield self.unit_full[at % SLOTS], at // SLOTS
                cur = self.slot[at % SLOTS]
                j, n = 0, cur[1 + i] if cur else 0
            if j < n:
                yield self.s_full[i], sn
                sn += 1
                self.p_full[i].arrive(4)
                j += 1
            if done:
                if done[1 + i] > 0:
                    yield self.o_full[i], on
                    on += 1
                    self.o_empty[i].arrive(4)
                self.stored.append((i, done[0]))
                self.unit_empty[done[0] % SLOTS].arrive(4)
                done = None
            if cur == 0:
                return

    def run(self):
        """Whether every role comes to its end."""
        roles = [self.scheduler(), self.producer(), self.issuer(), self.guard(), self.softmax(0), self.softmax(1)]
        waits = [next(r, None) for r in roles]
        while any(w is not None for w in waits):
            moved = False
            for x, w in enumerate(waits):
                while w is not None and w[0].passed(w[1]):
                    w = waits[x] = next(roles[x], None)
                    moved = True
            if not moved:
                return False
        return True
