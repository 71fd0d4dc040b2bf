"""Barrier protocol of the cached-keys kernel (pieces of a line of key tiles).

Per piece of nt key tiles one warp loads Q (QFull; QEmpty is committed behind
the piece's last scores), another K(x), V(x) in consecutive ring entries.  With
one row tile the two streams (softmax warpgroups) take the even and the odd key
tiles, each with its own S, P and O; with two row tiles (pair) both take every
key tile.  A slot is freed behind its last reader.  At the piece's end the
warpgroups write their statistics, meet, wait for both O, read them (one row
tile: both warpgroups both O; pair: each its own) and meet again before the next
piece's P.  The next piece's first scores are issued behind the piece's last
products.

mutation 1: no meeting behind the epilogue.
mutation 2: pair: a K slot freed behind the first stream's scores.
mutation 3: Q released behind the piece's first scores.
"""
from .engine import Engine


def run(pieces, seed, mutation=0, slots=6):
    """pieces: (key tiles, pair)."""
    e = Engine(seed)
    for name in ("QFull", "QEmpty"):
        e.bar(name, 1)
    for i in range(2):
        e.bar(f"S{i}", 1)
        e.bar(f"P{i}", 128)
        e.bar(f"O{i}", 1)
        e.bar(f"Meet{i}", 2)
    for s in range(slots):
        e.bar(f"Full{s}", 1)
        e.bar(f"Empty{s}", 1)

    def steps(piece, i):
        nt, pair = piece
        return nt if pair else (nt + 1 - i) // 2

    def tile(piece, i, s):
        return s if piece[1] else 2 * s + i

    def kv():
        seq = 0
        for k, (nt, _) in enumerate(pieces):
            for x in range(nt):
                for which in ("K", "V"):
                    s = seq % slots
                    yield ("wait", f"Empty{s}", ((seq // slots) & 1) ^ 1)
                    e.bars[f"Full{s}"].arrive(1, 1)
                    e.load(f"slot{s}", (which, k, x), f"Full{s}")
                    seq += 1

    def q():
        for k, (_, pair) in enumerate(pieces):
            yield ("wait", "QEmpty", (k & 1) ^ 1)
            n = 2 if pair else 1
            e.bars["QFull"].arrive(1, n)
            for i in range(n):
                e.load(f"sQ{i}", ("Q", k, i), "QFull")

    def mma():
        base, p_ph = 0, [0, 0]

        def scores(k, piece, base, i, s):
            x = tile(piece, i, s)
            n = base + 2 * x
            yield ("wait", f"Full{n % slots}", (n // slots) & 1)
            qi = i if piece[1] else 0
            e.mma([(f"sQ{qi}", ("Q", k, qi)), (f"slot{n % slots}", ("K", k, x))],
                  [(f"S{i}", ("S", k, i, x))])
            e.commit(f"S{i}")
            if not piece[1] or i == 1 or mutation == 2:
                if not (mutation == 2 and piece[1] and i == 1):
                    e.commit(f"Empty{n % slots}")
            last = (i == 1 and s + 1 == piece[0]) if piece[1] else 2 * s + i + 1 == piece[0]
            if last if mutation != 3 else (s == 0 and i == 0):
                e.commit("QEmpty")

        def values(k, piece, base, i, s):
            x = tile(piece, i, s)
            n = base + 2 * x + 1
            yield ("wait", f"Full{n % slots}", (n // slots) & 1)
            yield ("wait", f"P{i}", p_ph[i])
            p_ph[i] ^= 1
            clears = x + 1 == piece[0]
            reads = [(f"S{i}", ("P", k, i, x)),
                     (f"slot{n % slots}", ("Vc" if clears else "V", k, x))]
            if s:
                reads.append((f"O{i}", ("O", k, i, s)))
            e.mma(reads, [(f"O{i}", ("O", k, i, s + 1))])
            if not piece[1] or i == 1:
                e.commit(f"Empty{n % slots}")
            if s + 1 == steps(piece, i):
                e.commit(f"O{i}")

        for k, piece in enumerate(pieces):
            if k == 0:
                yield ("wait", "QFull", 0)
                for i in range(2):
                    if steps(piece, i):
                        yield from scores(0, piece, 0, i, 0)
            last = steps(piece, 0) - 1
            for s in range(last):
                yield from values(k, piece, base, 0, s)
                yield from scores(k, piece, base, 0, s + 1)
                yield from values(k, piece, base, 1, s)
                if s + 1 < steps(piece, 1):
                    yield from scores(k, piece, base, 1, s + 1)
            for i in range(2):
                if last < steps(piece, i):
                    yield from values(k, piece, base, i, last)
            base += 2 * piece[0]
            if k + 1 < len(pieces):
                nxt = pieces[k + 1]
                yield ("wait", "QFull", (k + 1) & 1)
                for i in range(2):
                    if steps(nxt, i):
                        yield from scores(k + 1, nxt, base, i, 0)

    def softmax(ti):
        s_ph, o_ph, base = 0, [0, 0], 0
        for k, piece in enumerate(pieces):
            nt, pair = piece
            for s in range(steps(piece, ti)):
                x = tile(piece, ti, s)
                yield ("wait", f"S{ti}", s_ph)
                s_ph ^= 1
                e.expect(f"S{ti}", ("S", k, ti, x))
                if s:  # rescale O
                    e.expect(f"O{ti}", ("O", k, ti, s))
                    yield ("step",)
                    e.expect(f"O{ti}", ("O", k, ti, s))
                if x + 1 == nt and (not pair or ti == 0):  # clears V rows
                    n = base + 2 * x + 1
                    yield ("wait", f"Full{n % slots}", (n // slots) & 1)
                    e.expect(f"slot{n % slots}", ("V", k, x))
                    e.mem[f"slot{n % slots}"] = ("Vc", k, x)
                yield ("step",)
                e.mem[f"S{ti}"] = ("P", k, ti, x)
                e.bars[f"P{ti}"].arrive(128)
            base += 2 * nt
            e.mem[f"ml{ti}"] = ("ml", k)
            e.bars["Meet0"].arrive()
            yield ("wait", "Meet0", k & 1)
            used = [i for i in range(2) if steps(piece, i)]
            for i in used:
                yield ("wait", f"O{i}", o_ph[i])
                o_ph[i] ^= 1
            mine = [ti] if pair else used
            for _ in range(2):
                for i in mine:
                    e.expect(f"O{i}", ("O", k, i, steps(piece, i)))
                if not pair:
                    e.expect("ml0", ("ml", k))
                    e.expect("ml1", ("ml", k))
                yield ("step",)
            if mutation != 1:
                e.bars["Meet1"].arrive()
                yield ("wait", "Meet1", k & 1)

    e.roles = {"kv": kv(), "q": q(), "mma": mma(), "sm0": softmax(0), "sm1": softmax(1)}
    e.run()
