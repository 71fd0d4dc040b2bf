"""Barrier protocol of the cached-weights kernel (pieces of a line of products).

A piece has `steps` tiles of rows and two key tiles, key tile i being needed from
step begins[i] on (begins[i] == steps: not at all).  One warp loads the needed key
tiles into a ring for each i, one the tiles of rows, one their normalisers into a ring of the
same length and, a piece ahead, what the warpgroups need to know of each piece into a ring of
four.  Each warpgroup moves its key tile of the next piece from the ring to
one of its two places in TMEM right before it waits for its last product of this
piece (or at the piece's begin if it has none).  The products of a step alternate
between the key tiles; a tile of rows is released behind the step's products, its
normalisers by both warpgroups.  A piece that is not fresh works on the tile of rows
that the piece before ended on, which that one has not released.

mutation 1: the key tile goes to one and the same place.
mutation 2: the rows are released behind the first key tile's product.
mutation 3: the products' place is not waited for.
mutation 4: the normalisers are released by the first warpgroup alone.
mutation 5: a kept tile of rows is released all the same.
mutation 6: the key tile is moved without waiting for its place in the ring to fill.
mutation 7: one ring for the key tiles of both i.
mutation 8: a piece is noted behind the normalisers of the one before.
mutation 9: a piece's note is released as soon as the next one is there.
"""
from .engine import Engine


def run(pieces, seed, mutation=0, depth=1, rows=3):
    """pieces: (steps, begins0, begins1, same): same, with one step: the rows of the piece before."""
    work = []
    for k, (steps, b0, b1, same) in enumerate(pieces):
        kept = bool(same) and steps == 1 and k > 0 and pieces[k - 1][0] == 1
        work.append([steps, (b0, b1), not kept, True])
    for k in range(len(work) - 1):
        work[k][3] = work[k + 1][2]  # last: the next piece's rows are others
    e = Engine(seed)
    keys = 2 * depth

    def place_of(i, n, both):
        """(place, phase) of the n-th key tile of i, the both-th of all."""
        if mutation == 7:
            return both % keys, (both // keys) & 1
        return i * depth + n % depth, (n // depth) & 1

    for s in range(keys):
        e.bar(f"KFull{s}", 1)
        e.bar(f"KEmpty{s}", 1)
    for s in range(rows):
        e.bar(f"QFull{s}", 1)
        e.bar(f"QEmpty{s}", 1)
        e.bar(f"LFull{s}", 1)
        e.bar(f"LEmpty{s}", 1 if mutation == 4 else 2)
    for s in range(4):
        e.bar(f"PFull{s}", 1)
        e.bar(f"PEmpty{s}", 2)
    for i in range(2):
        e.bar(f"S{i}", 1)
        e.bar(f"SFree{i}", 1)
        for w in range(2):
            e.bar(f"A{i}{w}", 1)

    def fresh_steps():
        n = 0
        for k, (steps, _, fresh, _) in enumerate(work):
            for s in range(steps):
                if fresh:
                    yield n, k, s
                    n += 1

    def load_keys():
        n = [0, 0]
        for k, (steps, begins, _, _) in enumerate(work):
            for i in range(2):
                if begins[i] < steps:
                    s, phase = place_of(i, n[i], sum(n))
                    yield ("wait", f"KEmpty{s}", phase ^ 1)
                    e.bars[f"KFull{s}"].arrive(1, 1)
                    e.load(f"k{s}", ("K", k, i), f"KFull{s}")
                    n[i] += 1

    def load_rows():
        for n, k, s in fresh_steps():
            yield ("wait", f"QEmpty{n % rows}", ((n // rows) & 1) ^ 1)
            e.bars[f"QFull{n % rows}"].arrive(1, 1)
            e.load(f"q{n % rows}", ("Q", n), f"QFull{n % rows}")

    def normalisers():
        def note(k):
            if k == len(work):
                return
            yield ("wait", f"PEmpty{k % 4}", ((k // 4) & 1) ^ 1)
            e.mem[f"p{k % 4}"] = ("P", k)
            yield ("step",)
            e.bars[f"PFull{k % 4}"].arrive()

        n = 0
        yield from note(0)
        for k, (steps, _, fresh, _) in enumerate(work):
            if mutation != 8:
                yield from note(k + 1)
            for s in range(steps if fresh else 0):
                yield ("wait", f"LEmpty{n % rows}", ((n // rows) & 1) ^ 1)
                e.mem[f"l{n % rows}"] = ("L", n)
                yield ("step",)
                e.bars[f"LFull{n % rows}"].arrive()
                n += 1
            if mutation == 8:
                yield from note(k + 1)

    def mma():
        n, staged, used = 0, [0, 0], [0, 0]
        for k, (steps, begins, fresh, last) in enumerate(work):
            for s in range(steps):
                if fresh:
                    yield ("wait", f"QFull{n % rows}", (n // rows) & 1)
                    n += 1
                slot = (n - 1) % rows
                for i in range(2):
                    if s < begins[i]:
                        continue
                    if s == begins[i]:
                        yield ("wait", f"A{i}{staged[i] & 1}", (staged[i] >> 1) & 1)
                        staged[i] += 1
                    if mutation != 3:
                        yield ("wait", f"SFree{i}", (used[i] & 1) ^ 1)
                    used[i] += 1
                    place = 0 if mutation == 1 else (staged[i] - 1) & 1
                    e.mma([(f"q{slot}", ("Q", n - 1)), (f"a{i}{place}", ("K", k, i))], [(f"S{i}", ("S", k, i, s))])
                    e.commit(f"S{i}")
                    if mutation == 2 and i == 0 and (last or s + 1 < steps):
                        e.commit(f"QEmpty{slot}")
                if mutation == 2 and begins[0] <= s:
                    continue
                if last or s + 1 < steps or mutation == 5:
                    e.commit(f"QEmpty{slot}")

    def sums(i):
        state = dict(n=0, staged=0)

        def stage(k):
            steps, begins, _, _ = work[k]
            mine = state["n"] + (i == 1 and begins[0] < steps)
            state["n"] += sum(b < steps for b in begins)
            if begins[i] == steps:
                return
            s, phase = place_of(i, state["staged"], mine)
            if mutation != 6:
                yield ("wait", f"KFull{s}", phase)
            e.expect(f"k{s}", ("K", k, i))
            yield ("step",)
            e.expect(f"k{s}", ("K", k, i))
            place = state["staged"] & 1
            e.mem[f"a{i}{0 if mutation == 1 else place}"] = ("K", k, i)
            e.bars[f"KEmpty{s}"].arrive()
            e.bars[f"A{i}{place}"].arrive()
            state["staged"] += 1

        used = n = 0
        yield ("wait", "PFull0", 0)
        yield from stage(0)
        for k, (steps, begins, fresh, last) in enumerate(work):
            more = k + 1 < len(work)
            if more:
                yield ("wait", f"PFull{(k + 1) % 4}", ((k + 1) // 4) & 1)
            if mutation == 9:
                e.bars[f"PEmpty{k % 4}"].arrive()
            if begins[i] == steps and more:
                yield from stage(k + 1)
            for s in range(steps):
                n += fresh
                slot = (n - 1) % rows
                if s >= begins[i]:
                    if s + 1 == steps and more:
                        yield from stage(k + 1)
                    yield ("wait", f"LFull{slot}", ((n - 1) // rows) & 1)
                    yield ("wait", f"S{i}", used & 1)
                    used += 1
                    e.expect(f"S{i}", ("S", k, i, s))
                    yield ("step",)
                    e.expect(f"S{i}", ("S", k, i, s))
                    e.bars[f"SFree{i}"].arrive()
                    yield ("step",)
                    e.expect(f"l{slot}", ("L", n - 1))
                else:
                    yield ("wait", f"LFull{slot}", ((n - 1) // rows) & 1)
                if (last or s + 1 < steps) and not (mutation == 4 and i == 1):
                    e.bars[f"LEmpty{slot}"].arrive()
            e.expect(f"p{k % 4}", ("P", k))
            if mutation != 9:
                e.bars[f"PEmpty{k % 4}"].arrive()

    e.roles = {"keys": load_keys(), "rows": load_rows(), "l": normalisers(), "mma": mma(), "sum0": sums(0),
               "sum1": sums(1)}
    e.run()
