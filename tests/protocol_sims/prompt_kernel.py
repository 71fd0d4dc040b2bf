"""Barrier protocol of the packed-prompt kernel (two query tiles per item).

A feeding warp hands the items out through two shared slots (FeedFull /
FeedEmpty, read by every role).  Per item the producer loads Q_i of each query
tile that sees keys (QFull_i; QEmpty_i is committed behind the tile's last
scores), then K(m), V(m) in consecutive entries of a ring.  The MMA issuer
runs, behind each product P V_i(m), the tile's next scores S_i -- at an item's
end the next item's first.  Softmax warpgroup i reads S_i, may rescale O_i,
clears the V rows behind the sequence's end (the first query tile that uses the
last V tile), writes P over S_i; at the item's end it waits for O_i and reads it.

buffers = 3 (64-wide heads): the scores of step n = 2 * (key tile) + (query
tile) go to buffer n % 3 and are issued before the product of the step before;
S_i, P_i and O_i have two barriers in turn, and O_i is committed with every
product, which a rescale waits for.

mutation 1: Q_i released before its last scores are issued.
mutation 2: P V_i issued without waiting for P_i.
mutation 3: an item's slot given back before it is read.
mutation 6: items without keys skipped when the next item is looked for (the
            roles that are still at this item hold their slots).
mutation 4: (buffers = 3) one barrier each for S_i and P_i.
mutation 5: (buffers = 3) a rescale that does not wait for the product.
mutation 7: (buffers = 3) one barrier for O_i: the last product but one, still
            under way, has the parity that passes for the last.
"""
from .engine import Engine

FEED = 2


def run(items, seed, mutation=0, buffers=2, slots=5):
    """items: (key tiles of query tile 0, of query tile 1)."""
    e = Engine(seed)
    turns = 2 if buffers == 3 and mutation != 4 else 1
    o_turns = 2 if buffers == 3 and mutation != 7 else 1
    for i in range(2):
        e.bar(f"QFull{i}", 1)
        e.bar(f"QEmpty{i}", 1)
        for t in range(o_turns):
            e.bar(f"O{i}{t}", 1)
        for t in range(turns):
            e.bar(f"S{i}{t}", 1)
            e.bar(f"P{i}{t}", 128)
    for s in range(slots):
        e.bar(f"Full{s}", 1)
        e.bar(f"Empty{s}", 1)
    for f in range(FEED):
        e.bar(f"FeedFull{f}", 1)
        e.bar(f"FeedEmpty{f}", 4)

    def turn(c):
        return (c & 1, c >> 1 & 1) if turns == 2 else (0, c & 1)

    def o_turn(c):
        return (c & 1, c >> 1 & 1) if o_turns == 2 else (0, c & 1)

    def buf(i, step):
        return f"S{i}" if buffers == 2 else f"S{(2 * step + i) % 3}"

    def feed():
        for k in range(len(items) + 1):
            f = k % FEED
            yield ("wait", f"FeedEmpty{f}", ((k // FEED) & 1) ^ 1)
            e.mem[f"feed{f}"] = ("item", k)
            e.bars[f"FeedFull{f}"].arrive()

    def fed(k):
        f = k % FEED
        yield ("wait", f"FeedFull{f}", (k // FEED) & 1)
        if mutation == 3:
            e.bars[f"FeedEmpty{f}"].arrive()
            yield ("step",)
            e.expect(f"feed{f}", ("item", k))
        else:
            e.expect(f"feed{f}", ("item", k))
            yield ("step",)
            e.expect(f"feed{f}", ("item", k))
            e.bars[f"FeedEmpty{f}"].arrive()
        return items[k] if k < len(items) else None

    def tma():
        seq, armed, k = 0, [0, 0], 0
        while True:
            it = yield from fed(k)
            if it is None:
                return
            for i in range(2):
                if it[i]:
                    yield ("wait", f"QEmpty{i}", (armed[i] & 1) ^ 1)
                    armed[i] += 1
                    e.bars[f"QFull{i}"].arrive(1, 1)
                    e.load(f"sQ{i}", ("Q", k, i), f"QFull{i}")
            for m in range(max(it)):
                for which in ("K", "V"):
                    s = seq % slots
                    yield ("wait", f"Empty{s}", ((seq // slots) & 1) ^ 1)
                    e.bars[f"Full{s}"].arrive(1, 1)
                    e.load(f"slot{s}", (which, k, m), f"Full{s}")
                    seq += 1
            k += 1

    def mma():
        st = {"kv": 0, "k": 0}
        s_n, p_n, q_n = [0, 0], [0, 0], [0, 0]

        def next_tiles():
            k = st["k"]
            it = yield from fed(k)
            st["k"] += 1
            while mutation == 6 and it is not None and not max(it):
                k = st["k"]
                it = yield from fed(k)
                st["k"] += 1
            return None if it is None else (k, it)

        def full(n):
            return ("wait", f"Full{n % slots}", (n // slots) & 1)

        def scores(k, it, i, m, step):
            n = 2 * step
            yield full(n)
            if mutation == 1 and m + 1 == it[i]:
                e.commit(f"QEmpty{i}")
            e.mma([(f"sQ{i}", ("Q", k, i)), (f"slot{n % slots}", ("K", k, m))],
                  [(buf(i, step), ("S", k, i, m))])
            e.commit(f"S{i}{turn(s_n[i])[0]}")
            s_n[i] += 1
            if mutation != 1 and m + 1 == it[i]:
                e.commit(f"QEmpty{i}")

        def first(k, it, i, step):
            yield ("wait", f"QFull{i}", q_n[i] & 1)
            q_n[i] += 1
            yield from scores(k, it, i, 0, step)

        def product(k, it, i, m, step):
            n = 2 * step + 1
            t, par = turn(p_n[i])
            if mutation != 2:
                yield ("wait", f"P{i}{t}", par)
            p_n[i] += 1
            tag = "Vc" if m + 1 == max(it) else "V"
            reads = [(buf(i, step), ("P", k, i, m)), (f"slot{n % slots}", (tag, k, m))]
            if m:
                reads.append((f"O{i}", ("O", k, i, m)))
            e.mma(reads, [(f"O{i}", ("O", k, i, m + 1))])
            if buffers == 3:
                e.commit(f"O{i}{o_turn(p_n[i] - 1)[0]}")
            elif m + 1 == it[i]:
                e.commit(f"O{i}0")

        cur = yield from next_tiles()
        started = False  # the item's first scores are issued
        while cur is not None:
            nxt = yield from next_tiles()
            k, it = cur
            if max(it) and not started:
                for i in range(2):
                    if it[i]:
                        yield from first(k, it, i, st["kv"])
                e.commit(f"Empty{(2 * st['kv']) % slots}")
            started = False
            for m in range(max(it)):
                step, last = st["kv"], m + 1 == max(it)
                yield full(2 * step + 1)
                for i in range(2):
                    if not last:
                        order = [product, scores] if buffers == 2 else [scores, product]
                        for f in order:
                            if f is product and m < it[i]:
                                yield from product(k, it, i, m, step)
                            if f is scores and m + 1 < it[i]:
                                yield from scores(k, it, i, m + 1, step + 1)
                    else:
                        if m < it[i]:
                            yield from product(k, it, i, m, step)
                        if nxt is not None and nxt[1][i]:
                            yield from first(nxt[0], nxt[1], i, step + 1)
                e.commit(f"Empty{(2 * step + 1) % slots}")
                if not last or (nxt is not None and max(nxt[1])):
                    e.commit(f"Empty{(2 * step + 2) % slots}")
                    started = last
                st["kv"] += 1
            cur = nxt

    def softmax(ti):
        c, o_n, kv, k = 0, 0, 0, 0
        while True:
            it = yield from fed(k)
            if it is None:
                return
            for m in range(it[ti]):
                b = buf(ti, kv + m)
                t, par = turn(c)
                yield ("wait", f"S{ti}{t}", par)
                e.expect(b, ("S", k, ti, m))
                yield ("step",)
                if m and e.rnd.random() < 0.5:  # rescale O: only where the maximum grew
                    if buffers == 3 and mutation != 5:
                        t, par = o_turn(c - 1)
                        yield ("wait", f"O{ti}{t}", par)
                    e.expect(f"O{ti}", ("O", k, ti, m))
                    yield ("step",)
                    e.expect(f"O{ti}", ("O", k, ti, m))
                if m + 1 == max(it) and (ti == 0 or it[0] < max(it)):  # clears V rows
                    n = 2 * (kv + m) + 1
                    yield ("wait", f"Full{n % slots}", (n // slots) & 1)
                    e.expect(f"slot{n % slots}", ("V", k, m))
                    e.mem[f"slot{n % slots}"] = ("Vc", k, m)
                e.expect(b, ("S", k, ti, m))
                e.mem[b] = ("P", k, ti, m)
                e.bars[f"P{ti}{turn(c)[0]}"].arrive(128)
                c += 1
            kv += max(it)
            if it[ti]:
                if buffers == 3:
                    t, par = o_turn(c - 1)
                    yield ("wait", f"O{ti}{t}", par)
                else:
                    yield ("wait", f"O{ti}0", o_n & 1)
                o_n += 1
                e.expect(f"O{ti}", ("O", k, ti, it[ti]))
                yield ("step",)
                e.expect(f"O{ti}", ("O", k, ti, it[ti]))
            k += 1

    e.roles = {"feed": feed(), "tma": tma(), "mma": mma(), "sm0": softmax(0), "sm1": softmax(1)}
    e.run()
