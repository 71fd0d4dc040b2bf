"""Barrier protocol of the cached-weights kernel (pieces of a line of products).

A piece has `steps` tiles of rows and two key tiles, key tile i being needed from
step begins[i] on (begins[i] == steps: not at all).  One warp loads the needed key
tiles into a ring for each i, and the tiles of rows (deep: a warp for each i); one their normalisers into a ring
of the same length and, a piece ahead, what the warpgroups need to know of each piece
into a ring of four.  A warp for each key tile issues its products, which take two places
by turns; the last of a piece frees the key tile, those of a step by both warps the rows.
Deep: a key tile has a warpgroup.
A piece that is not fresh works on the tile of rows that the piece before ended on,
which that one has not released.
Else the three warpgroups take the steps by turns, both key tiles of each.  A barrier for each
place and warpgroup tells of the products.  At the piece's end they hand their sums
of both key tiles to the first two, through one of two places.
The normalisers are released by the warpgroups that use them; their ring is longer than the
warpgroups are many.

mutation 1: one place for a key tile's products.
mutation 2: the rows are released by one of the warps alone.
mutation 3: the products' place is not waited for.
mutation 4: deep: the normalisers are released by one warpgroup alone.
mutation 5: a kept tile of rows is released all the same.
mutation 6: a product is issued without waiting for its key tile.
mutation 8: a piece is noted behind the normalisers of the one before.
mutation 9: a piece's note is released as soon as the next one is there.
mutation 10: the sums are written without waiting for their place.
mutation 11: a key tile is freed behind its first product.
mutation 7: a barrier for each key tile and warpgroup, whatever the place.
mutation 13: as many places for normalisers as for rows.
mutation 12: a barrier for each place, whoever reads it.
"""
from .engine import Engine


def run(pieces, seed, mutation=0, depth=2, rows=2, deep=False):
    """pieces: (steps, begins0, begins1, same): same, with one step: the rows of the piece before."""
    work = []
    for k, (steps, b0, b1, same) in enumerate(pieces):
        kept = deep and bool(same) and steps == 1 and k > 0 and pieces[k - 1][0] == 1
        work.append([steps, (b0, b1), not kept, True])
    for k in range(len(work) - 1):
        work[k][3] = work[k + 1][2]  # last: the next piece's rows are others
    groups = 2 if deep else 3
    norms = rows if mutation == 13 else max(rows, 4)
    e = Engine(seed)

    def place_of(i, n):
        """(place, phase) of the n-th key tile of i."""
        return i * depth + n % depth, (n // depth) & 1

    for s in range(2 * depth):
        e.bar(f"KFull{s}", 1)
        e.bar(f"KEmpty{s}", 1)
    for s in range(rows):
        e.bar(f"QFull{s}", 1)
        e.bar(f"QEmpty{s}", 1 if mutation == 2 else 2)
    for s in range(norms):
        e.bar(f"LFull{s}", 1)
        e.bar(f"LEmpty{s}", 1 if mutation == 4 or not deep else groups)
    for s in range(4):
        e.bar(f"PFull{s}", 1)
        e.bar(f"PEmpty{s}", groups)
    for w in range(4):
        e.bar(f"SFree{w}", 1)
        for g in range(3):
            e.bar(f"S{w}{g}", 1)

    def bar_of(place, group):
        return f"S{place // 2 * 2 if mutation == 7 else place}{0 if deep or mutation == 12 else group}"

    for i in range(2):
        e.bar(f"XFull{i}", groups)
        e.bar(f"XEmpty{i}", 2)

    def load(tiles, with_rows):
        n, q = [0, 0], 0
        for k, (steps, begins, fresh, _) in enumerate(work):
            for i in tiles:
                if begins[i] < steps:
                    s, phase = place_of(i, n[i])
                    yield ("wait", f"KEmpty{s}", phase ^ 1)
                    e.bars[f"KFull{s}"].arrive(1, 1)
                    e.load(f"k{s}", ("K", k, i), f"KFull{s}")
                    n[i] += 1
            for _ in range(steps if fresh and with_rows else 0):
                yield ("wait", f"QEmpty{q % rows}", ((q // rows) & 1) ^ 1)
                e.bars[f"QFull{q % rows}"].arrive(1, 1)
                e.load(f"q{q % rows}", ("Q", q), f"QFull{q % rows}")
                q += 1

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
                yield ("wait", f"LEmpty{n % norms}", ((n // norms) & 1) ^ 1)
                e.mem[f"l{n % norms}"] = ("L", n)
                yield ("step",)
                e.bars[f"LFull{n % norms}"].arrive()
                n += 1
            if mutation == 8:
                yield from note(k + 1)

    def mma(i):
        n, taken, used, group = 0, 0, 0, groups - 1
        for k, (steps, begins, fresh, last) in enumerate(work):
            for s in range(steps):
                n += fresh
                group = (group + 1) % groups
                slot = (n - 1) % rows
                yield ("wait", f"QFull{slot}", ((n - 1) // rows) & 1)
                if s >= begins[i]:
                    if s == begins[i]:
                        sl, phase = place_of(i, taken)
                        if mutation != 6:
                            yield ("wait", f"KFull{sl}", phase)
                        taken += 1
                    sl = place_of(i, taken - 1)[0]
                    w = 2 * i + (0 if mutation == 1 else used & 1)
                    if mutation != 3:
                        yield ("wait", f"SFree{2 * i + (used & 1)}", (used >> 1 & 1) ^ 1)
                    bar = bar_of(2 * i + (used & 1), group)
                    used += 1
                    e.mma([(f"q{slot}", ("Q", n - 1)), (f"k{sl}", ("K", k, i))], [(f"S{w}", ("S", k, i, s))])
                    e.commit(bar)
                    if s == begins[i] if mutation == 11 else s + 1 == steps:
                        e.commit(f"KEmpty{sl}")
                if (last or s + 1 < steps or mutation == 5) and not (mutation == 2 and i == 1):
                    e.commit(f"QEmpty{slot}")

    def sums(group):
        used, n, step, made = {}, 0, 0, [0, 0]
        yield ("wait", "PFull0", 0)
        for k, (steps, begins, fresh, last) in enumerate(work):
            more = k + 1 < len(work)
            if more:
                yield ("wait", f"PFull{(k + 1) % 4}", ((k + 1) // 4) & 1)
            if mutation == 9:
                e.bars[f"PEmpty{k % 4}"].arrive()
            for s in range(steps):
                n += fresh
                slot = (n - 1) % norms
                mine = deep or step % groups == group
                step += 1
                if mine:
                    yield ("wait", f"LFull{slot}", ((n - 1) // norms) & 1)
                for i in range(2):
                    if s < begins[i]:
                        continue
                    place = 2 * i + (made[i] & 1)
                    turns = made[i] >> 1
                    made[i] += 1
                    if not mine or deep and i != group:
                        continue
                    w = 2 * i if mutation == 1 else place
                    bar = bar_of(place, group)
                    phase = turns & 1 if mutation == 12 else used.get(bar, 0) & 1
                    yield ("wait", bar, phase)
                    used[bar] = used.get(bar, 0) + 1
                    e.expect(f"S{w}", ("S", k, i, s))
                    yield ("step",)
                    e.expect(f"S{w}", ("S", k, i, s))
                    e.bars[f"SFree{place}"].arrive()
                    yield ("step",)
                    e.expect(f"l{slot}", ("L", n - 1))
                if mine and (last or s + 1 < steps) and not (mutation == 4 and group != 0):
                    e.bars[f"LEmpty{slot}"].arrive()
            if not deep:
                h = k & 1
                if mutation != 10:
                    yield ("wait", f"XEmpty{h}", (k >> 1 & 1) ^ 1)
                e.mem[f"x{h}{group}"] = ("X", k)
                yield ("step",)
                e.bars[f"XFull{h}"].arrive()
                if group < 2:
                    yield ("wait", f"XFull{h}", k >> 1 & 1)
                    for _ in range(2):
                        for g in range(groups):
                            e.expect(f"x{h}{g}", ("X", k))
                        yield ("step",)
                    e.bars[f"XEmpty{h}"].arrive()
            e.expect(f"p{k % 4}", ("P", k))
            if mutation != 9:
                e.bars[f"PEmpty{k % 4}"].arrive()

    loads = {"load0": load([0], True), "load1": load([1], False)} if deep else {"load": load([0, 1], True)}
    e.roles = {**loads, "l": normalisers(), "mma0": mma(0), "mma1": mma(1)}
    for group in range(groups):
        e.roles[f"sum{group}"] = sums(group)
    e.run()
