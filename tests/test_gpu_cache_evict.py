"""Eviction on the GPU against a plain implementation, position by position: all results are equal bit by bit."""
import math
import random

import pytest
import torch

import context_causal_attention_zigzag_gb300 as cpa

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def plan(scores, c, keep, first, recent):
    """Where the position at each place of one head was: scores [c]."""
    if keep >= c:
        return list(range(c))
    f = min(first, keep)
    t = min(recent, keep - f)
    cut = keep - t
    order = sorted(range(f, c - t), key=lambda j: (math.isnan(scores[j]), -scores[j] if scores[j] == scores[j] else 0, j))
    stay = set(order[:cut - f]) | set(range(f))
    late = iter(sorted(j for j in stay if j >= cut))
    return [j if j in stay else next(late) for j in range(cut)] + list(range(c - t, c))


def make(ctx, Hkv, D, P, dtype, seed=0, kind="plain", spare=2, extra=1):
    rng = random.Random(seed)
    need = [-(-x // P) for x in ctx]
    ids = list(range(sum(need) + spare))
    rng.shuffle(ids)
    width, rows, at = max(need + [0]) + extra, [], 0
    for n in need:
        rows.append(ids[at:at + n] + [-1] * (width - n))
        at += n
    pages = len(ids)
    g = torch.Generator().manual_seed(seed)
    cache = torch.randn(2, pages, P, Hkv, D, generator=g).to(TYPES[dtype]).to(DEV)
    weights = torch.randn(pages, Hkv, P, generator=g)
    if kind == "ties":
        weights = weights.round()
    elif kind == "equal":
        weights.fill_(0.25)
    elif kind == "zeros":
        weights[torch.rand(weights.shape, generator=g) < 0.7] = 0
        weights[torch.rand(weights.shape, generator=g) < 0.2] = -0.0
    elif kind == "wild":
        for value in (math.nan, math.inf, -math.inf, 0.0, -0.0, 1e-40, -1e-40, 3e38):
            weights[torch.rand(weights.shape, generator=g) < 0.1] = value
    elif kind == "small":
        weights = weights * 1e-41
    return cache[0], cache[1], weights.to(DEV), ints(rows).view(len(ctx), width)


def reference(weights, scores, k, v, table, ctx, keep, first, recent, most, room):
    k, v, w = k.clone(), v.clone(), weights.clone()
    P, Hkv = k.shape[1:3]
    kept = torch.full((len(ctx), Hkv, most), -1, dtype=torch.int32)
    freed = []
    t = table.cpu()
    sc = scores.cpu()
    new = [min(c, b) for c, b in zip(ctx, keep)]
    for r, (c, b) in enumerate(zip(ctx, keep)):
        pos = torch.arange(c)
        page = t[r].long()[pos // P]
        for g in range(Hkv):
            m = torch.tensor(plan(sc[page, g, pos % P].tolist(), c, b, first, recent), dtype=torch.long)
            kept[r, g, :len(m)] = m.int()
            to = torch.arange(len(m))
            src, dst = (page[m].to(DEV), (m % P).to(DEV)), (page[to].to(DEV), (to % P).to(DEV))
            k[dst[0], dst[1], g] = k[src[0], src[1], g]
            v[dst[0], dst[1], g] = v[src[0], src[1], g]
            w[dst[0], g, dst[1]] = w[src[0], g, src[1]]
        if b < c:
            freed += t[r, -(-b // P):-(-c // P)].tolist()
    listed = freed[:room]
    return k, v, w, ints(new), kept.to(DEV), ints(listed + [-1] * (room - len(listed))), ints([len(listed)])


def same(a, b):
    a, b = (x.view(torch.int32) if x.dtype == torch.float32 else x for x in (a, b))
    return torch.equal(a, b)


def run(ctx, keep, first, recent, Hkv, D, P, dtype, kind="plain", seed=0, scores=False, most=None, layout=None):
    k, v, w, table = make(ctx, Hkv, D, P, dtype, seed, kind)
    if layout == "heads first":
        k, v = (x.transpose(1, 2).contiguous().transpose(1, 2) for x in (k, v))
    sc = w.flip(2).contiguous() if scores else None
    most = max([min(c, b) for c, b in zip(ctx, keep)] + [1]) if most is None else most
    want = reference(w, w if sc is None else sc, k, v, table, ctx, keep, first, recent, most, table.numel())
    got = cpa.cache_evict(w, k, v, table, ints(ctx), ints(keep), most, first=first, recent=recent, scores=sc)
    assert cpa.device_status() == 0
    for name, x, y in zip(("k", "v", "weights", "new_lens", "kept", "freed", "count"), (k, v, w) + got, want):
        assert same(x, y), f"{name}: {int((x != y).sum())} differ"


CASES = [
    # ctx, keep, first, recent, Hkv, D, page
    ([1000], [600], 4, 64, 8, 128, 64),
    ([1], [0], 0, 0, 1, 64, 16),
    ([1, 0, 2], [1, 0, 1], 0, 0, 2, 64, 16),
    ([17, 16, 15], [16, 16, 16], 0, 1, 2, 128, 16),
    ([500, 300, 40, 999], [200, 300, 60, 1], 4, 32, 2, 64, 32),
    ([700], [100], 0, 0, 3, 128, 128),
    ([700], [100], 200, 50, 2, 64, 128),         # the first ones alone
    ([700], [100], 30, 500, 2, 64, 128),         # nothing between
    ([700], [400], 0, 390, 1, 128, 16),          # the last ones move within themselves
    ([3001], [3000], 4, 2900, 2, 128, 16),       # by one place
    ([2600], [2500], 0, 2400, 8, 64, 384),
    ([5000] * 3, [4999, 1, 2500], 4, 128, 8, 128, 256),
    ([40] * 100, [20] * 100, 1, 8, 2, 64, 16),
    ([20000, 7], [5000, 7], 16, 1000, 4, 128, 1024),
    ([100], [0], 4, 10, 2, 64, 16),
]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("ctx,keep,first,recent,Hkv,D,P", CASES)
def test_cache_evict(ctx, keep, first, recent, Hkv, D, P, dtype):
    run(ctx, keep, first, recent, Hkv, D, P, dtype)


@pytest.mark.parametrize("kind", ["ties", "equal", "zeros", "wild", "small"])
@pytest.mark.parametrize("ctx,keep", [([900, 33], [300, 32]), ([6000], [5000])])
def test_equal_and_special_scores(ctx, keep, kind):
    run(ctx, keep, 4, 30, 2, 64, 16, "bf16", kind=kind, seed=3)


def test_scores_of_their_own_and_room_to_spare():
    run([900, 100, 5], [400, 300, 5], 2, 20, 2, 128, 64, "bf16", scores=True, most=700, layout="heads first")


def test_a_request_longer_than_shared_memory_holds():
    run([140001], [70000], 4, 100, 1, 64, 64, "bf16")


def test_many_heads_share_the_sms():
    run([300] * 40, [150] * 40, 4, 16, 16, 64, 64, "bf16")


def test_attention_over_what_stays():
    """After an eviction attention over the cache is attention over the kept positions, and the pages
    that became free serve the next tokens."""
    H, Hkv, D, P, ctx, keep = 8, 2, 64, 16, [200, 90], [64, 70]
    k, v, w, table = make(ctx, Hkv, D, P, "bf16", seed=9, extra=0)
    k0, v0 = k.clone(), v.clone()
    new_lens, kept, freed, count = cpa.cache_evict(w, k, v, table, ints(ctx), ints(keep), 70, first=4, recent=8)
    assert new_lens.tolist() == [64, 70] and int(count) == 13 - 4 + 6 - 5
    one = ints([1, 1])
    slots, cu, used = cpa.page_tables(new_lens, one, table, freed[:int(count)].contiguous(), P, 2)
    assert int(used) == 1
    g = torch.Generator().manual_seed(1)
    q, kk, vv = (torch.randn(2, h, D, generator=g).bfloat16().to(DEV) for h in (H, Hkv, Hkv))
    cpa.cache_write(kk, vv, k, v, slots)
    out, lse = cpa.tree_attention(q, k, v, table, new_lens, cu)
    assert cpa.device_status() == 0
    table0 = make(ctx, Hkv, D, P, "bf16", seed=9, extra=0)[3]
    for r in range(2):
        for h in range(H):
            pos = kept[r, h * Hkv // H, :keep[r]].long()
            page = table0[r].long()[pos // P]
            keys = torch.cat([k0[page, pos % P, h * Hkv // H], kk[r, h * Hkv // H][None]]).double()
            vals = torch.cat([v0[page, pos % P, h * Hkv // H], vv[r, h * Hkv // H][None]]).double()
            p = torch.softmax(keys @ q[r, h].double() / math.sqrt(D), 0)
            assert float((p @ vals - out[r, h].double()).abs().max()) < 2.0 ** -7 * float(vals.abs().max())


def test_decoding_with_a_limited_cache():
    """Steps of a server, its calls one after another: tables, rotary and write, attention, weights, eviction."""
    H, Hkv, D, P, R, limit = 8, 2, 64, 16, 3, 48
    freqs, _ = cpa.rotary_frequencies(D)
    pages = 40
    cache = torch.zeros(2, pages, P, Hkv, D, device=DEV, dtype=torch.bfloat16)
    weights = torch.zeros(pages, Hkv, P, device=DEV)
    free = torch.arange(pages, device=DEV, dtype=torch.int32)
    table = torch.full((R, 8), -1, device=DEV, dtype=torch.int32)
    ctx, seen = ints([0] * R), ints([0] * R)
    g = torch.Generator().manual_seed(5)
    # What a plain program holds: each head's keys, values and weights.
    held = [[([], [], []) for _ in range(Hkv)] for _ in range(R)]
    for step in range(40):
        new = [(7, 3, 11)[r] if step == 0 else 1 + (step + r) % 3 for r in range(R)]
        fresh = ints(new)
        slots, cu, used = cpa.page_tables(ctx, fresh, table, free, P, sum(new))
        free = free[int(used):].contiguous()
        at = torch.cat([torch.arange(int(seen[r]), int(seen[r]) + n) for r, n in enumerate(new)]).int().to(DEV)
        q, k, v = (torch.randn(sum(new), h, D, generator=g).bfloat16().to(DEV) for h in (H, Hkv, Hkv))
        q, _, _ = cpa.rotary_cache_write(q, k, v, freqs, at, cache[0], cache[1], slots)
        out, lse = cpa.tree_attention(q, cache[0], cache[1], table, ctx, cu)
        cpa.cache_weights(q, cache[0], table, ctx, cu, lse, weights)
        turned = cpa.rotary(k, freqs, at)
        first = 0
        for r, n in enumerate(new):
            for hk in range(Hkv):
                ks, vs, ws = held[r][hk]
                x = len(ks)
                ks += list(turned[first:first + n, hk].double().cpu())
                vs += list(v[first:first + n, hk].double().cpu())
                ws += [0.0] * n
                K, V = torch.stack(ks), torch.stack(vs)
                for h in range(hk * H // Hkv, (hk + 1) * H // Hkv):
                    z = q[first:first + n, h].double().cpu() @ K.T / math.sqrt(D)
                    z[torch.arange(x + n)[None] > torch.arange(n)[:, None] + x] = -math.inf
                    p = torch.softmax(z, 1)
                    assert float((p @ V - out[first:first + n, h].double().cpu()).abs().max()) < 0.03
                    for j in range(x + n):
                        ws[j] += float(p[:, j].sum())
            first += n
        total = [int(c) + n for c, n in zip(ctx, new)]
        new_lens, kept, freed, count = cpa.cache_evict(
            weights, cache[0], cache[1], table, ints(total), ints([limit] * R), limit, first=2, recent=8)
        assert cpa.device_status() == 0
        free = torch.cat([free, freed[:int(count)]])
        for r in range(R):
            for hk in range(Hkv):
                m = kept[r, hk][kept[r, hk] >= 0].tolist()
                held[r][hk] = tuple([x[j] for j in m] for x in held[r][hk])
                pos = torch.arange(len(m), device=DEV)
                got = weights[table[r].long()[pos // P], hk, pos % P].double().cpu()
                assert torch.allclose(got, torch.tensor(held[r][hk][2], dtype=torch.float64), rtol=2e-3, atol=1e-4)
        ctx, seen = new_lens, seen + fresh
    assert free.numel() == pages - sum(-(-int(c) // P) for c in ctx)
    assert len(set(free.tolist())) == free.numel()


def test_broken_calls_are_reported_and_left():
    for what in ("page", "negative keep", "long", "most", "room"):
        ctx, keep = [100, 80], [50, 40]
        k, v, w, table = make(ctx, 2, 64, 16, "bf16")
        c, b, most = ints(ctx), ints(keep), 50
        outputs = cpa.cache_evict_outputs(k, table, c, most)
        if what == "page":
            table[1, 2] = -1
        elif what == "negative keep":
            b[1] = -1
        elif what == "long":
            c[1] = 100000
        elif what == "most":
            b[1] = 51
        else:
            outputs = outputs[:2] + (outputs[2][:1], outputs[3])
        before = k.clone(), v.clone(), w.clone()
        new_lens, kept, freed, count = cpa.cache_evict(w, k, v, table, c, b, most, outputs=outputs)
        assert cpa.device_status() == -1, what
        if what == "room":
            assert new_lens.tolist() == keep and int(count) == 1
            continue
        assert new_lens.tolist() == [50, int(c[1])], what
        mine = table[1].long()
        mine = mine[(mine >= 0) & (mine < k.shape[0])]
        for x, y in zip((k, v, w), before):
            assert torch.equal(x[mine], y[mine]), what
    assert cpa.device_status() == 0


def test_graph_replays_see_new_lengths():
    Hkv, D, P = 2, 64, 16
    k, v, w, table = make([300, 200], Hkv, D, P, "bf16", seed=2)
    state = [x.clone() for x in (k, v, w)]
    c, b = ints([300, 200]), ints([100, 150])
    outputs = cpa.cache_evict_outputs(k, table, c, 150)
    ws = cpa.cache_evict_workspace(k, table, 150)

    def call():
        cpa.cache_evict(w, k, v, table, c, b, 150, first=2, recent=10, outputs=outputs, workspace=ws)
    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for ctx, keep in (([300, 200], [100, 150]), ([250, 199], [30, 150]), ([120, 10], [119, 3])):
        for x, y in zip((k, v, w), state):
            x.copy_(y)
        c.copy_(ints(ctx))
        b.copy_(ints(keep))
        graph.replay()
        torch.cuda.synchronize()
        want = reference(state[2], state[2], state[0], state[1], table, ctx, keep, 2, 10, 150, table.numel())
        for x, y in zip((k, v, w) + tuple(outputs), want):
            assert same(x, y)


@pytest.mark.parametrize("R,Hkv,longest", [(20, 8, 3000), (70, 3, 2100)])
def test_wide_tables_in_one_launch_and_their_freed_pages(R, Hkv, longest):
    rng = random.Random(R)
    ctx = [longest] + [rng.randrange(longest) for _ in range(R - 1)]
    run(ctx, [rng.randrange(c + 20) for c in ctx], 4, 32, Hkv, 64, 16, "fp16", seed=R)


def test_two_calls_at_once():
    calls = []
    for i in range(2):
        ctx, keep = [5000 + i, 800, 20000], [2000, 100 + i, 700]
        k, v, w, table = make(ctx, 4, 64, 32, "bf16", seed=i)
        want = reference(w, w, k, v, table, ctx, keep, 4, 60, 2000, table.numel())
        calls.append((torch.cuda.Stream(), (w, k, v, table, ints(ctx), ints(keep), 2000), want))
    torch.cuda.synchronize()
    got = []
    for s, args, _ in calls:
        with torch.cuda.stream(s):
            got.append(cpa.cache_evict(*args, first=4, recent=60))
    torch.cuda.synchronize()
    assert cpa.device_status() == 0
    for (_, (w, k, v, *_), want), out in zip(calls, got):
        for x, y in zip((k, v, w) + out, want):
            assert same(x, y)


@pytest.mark.parametrize("ctx,keep,first,recent,Hkv", [
    ([9000], [4000], 4, 64, 8), ([40000, 33000], [20000, 5], 0, 1000, 1), ([140001], [70000], 4, 100, 1),
    ([140001], [139000], 0, 0, 1)])
@pytest.mark.parametrize("kind", ["ties", "equal", "wild"])
def test_equals_among_ctas_and_windows(ctx, keep, first, recent, Hkv, kind):
    run(ctx, keep, first, recent, Hkv, 64, 64, "bf16", kind)


def test_offsets_beyond_32_bits():
    """A cache of 5 GB whose requests lie at its end gives what a small one does, bit by bit."""
    H, Hkv, D, P, pages = 16, 8, 128, 64, 40000
    assert pages * P * Hkv * D > 1 << 31
    ctx, new = [500, 333], [3, 20]
    need = [-(-(c + n) // P) for c, n in zip(ctx, new)]
    table = torch.full((2, max(need)), -1, dtype=torch.int32, device=DEV)
    for r, n in enumerate(need):
        table[r, :n] = torch.arange(n, device=DEV) + sum(need[:r])
    g = torch.Generator().manual_seed(5)
    small = torch.randn(2, sum(need), P, Hkv, D, generator=g).to(torch.bfloat16).to(DEV)
    weights = torch.rand(sum(need), Hkv, P, generator=g).to(DEV)
    q, k, v = (torch.randn(sum(new), n, D, generator=g).to(torch.bfloat16).to(DEV) for n in (H, Hkv, Hkv))
    freqs, at = torch.rand(D // 2, generator=g, dtype=torch.float64).to(DEV), torch.arange(sum(new), device=DEV).int()
    slot = [int(table[r, p // P]) * P + p % P for r in range(2) for p in range(ctx[r], ctx[r] + new[r])]
    results = []
    for first in (0, pages - sum(need)):
        if first:
            cache = [torch.empty(pages, P, Hkv, D, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
            for x, y in zip(cache, small):
                x[first:] = y
            w = torch.empty(pages, Hkv, P, device=DEV)
            w[first:] = weights
        else:
            cache, w = [x.clone() for x in small], weights.clone()
        t = torch.where(table >= 0, table + first, table)
        slots = torch.tensor(slot, device=DEV) + first * P
        cu, total = ints([0, new[0], sum(new)]), ints([c + n for c, n in zip(ctx, new)])
        out, kc, vc = cpa.rotary_cache_write(q, k, v, freqs, at, cache[0], cache[1], slots)
        o, lse = cpa.tree_attention(out, kc, vc, t, ints(ctx), cu)
        cpa.cache_weights(out, kc, t, ints(ctx), cu, lse, w)
        moved = cpa.cache_evict(w, kc, vc, t, total, ints([200, 100]), 200, first=4, recent=30)
        assert cpa.device_status() == 0
        freed = torch.where(moved[2] >= 0, moved[2] - first, moved[2])
        results.append((out, o, kc[first:].clone(), vc[first:].clone(), w[first:].clone(), moved[0], moved[1], freed, moved[3]))
        del cache, kc, vc, w
    for x, y in zip(*results):
        assert same(x, y)


def test_first_or_recent_beyond_any_length():
    for first, recent in ((1 << 40, 3), (0, 1 << 32)):
        run([300, 90], [100, 80], first, recent, 2, 64, 16, "bf16")


@pytest.mark.parametrize("R,width", [(2500, 3), (3000, 3)])  # the freed pages listed by the one launch, by one of their own
def test_thousands_of_requests(R, width):
    rng = random.Random(R)
    ctx = [rng.randrange(16 * (width - 1) + 1) for _ in range(R)]
    run(ctx, [rng.randrange(c + 5) for c in ctx], 1, 3, 1, 64, 16, "bf16", seed=R)


def test_a_step_from_a_graph():
    """Turn and write, attend, weigh and evict, captured once and replayed with other lengths: the eager call's bits."""
    H, Hkv, D, P, most, N = 8, 2, 64, 16, 120, 40
    k0, v0, w0, table = make([300, 300, 300], Hkv, D, P, "bf16", seed=9, extra=0)
    w0.abs_()
    g = torch.Generator().manual_seed(9)
    q, k, v = (torch.randn(N, n, D, generator=g).to(torch.bfloat16).to(DEV) for n in (H, Hkv, Hkv))
    freqs = torch.rand(D // 2, generator=g, dtype=torch.float64).to(DEV)
    ctx, cu, total, at = ints([0] * 3), ints([0] * 4), ints([0] * 3), torch.zeros(N, dtype=torch.int32, device=DEV)
    slots, keep = torch.full((N,), -1, dtype=torch.int64, device=DEV), ints([most, 30, 0])
    kc, vc, w = k0.clone(), v0.clone(), w0.clone()
    turned, out, lse = torch.empty_like(q), torch.empty_like(q), torch.empty(H, N, device=DEV)
    moved = cpa.cache_evict_outputs(kc, table, ctx, most)
    spaces = (cpa.tree_attention_workspace(q, kc, cu), cpa.cache_weights_workspace(q, kc, cu),
              cpa.cache_evict_workspace(kc, table, most))

    def step():
        cpa.rotary_cache_write(q, k, v, freqs, at, kc, vc, slots, out=turned)
        cpa.tree_attention(turned, kc, vc, table, ctx, cu, out=out, lse=lse, workspace=spaces[0])
        cpa.cache_weights(turned, kc, table, ctx, cu, lse, w, decay=0.5, workspace=spaces[1])
        cpa.cache_evict(w, kc, vc, table, total, keep, most, first=2, recent=20, outputs=moved, workspace=spaces[2])

    def set_lens(lens, new):
        for x, y in zip((kc, vc, w), (k0, v0, w0)):
            x.copy_(y)
        ctx.copy_(ints(lens))
        cu.copy_(ints([sum(new[:i]) for i in range(4)]))
        total.copy_(ints([a + b for a, b in zip(lens, new)]))
        places = [(r, p) for r in range(3) for p in range(lens[r], lens[r] + new[r])]
        at.zero_()
        slots.fill_(-1)
        at[:len(places)] = ints([p for _, p in places])
        slots[:len(places)] = torch.tensor([int(table[r, p // P]) * P + p % P for r, p in places], device=DEV)

    set_lens([10, 10, 10], [1, 1, 1])
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for lens, new in (([250, 0, 299], [30, 9, 1]), ([100, 17, 200], [1, 1, 1]), ([0, 280, 0], [40, 0, 0])):
        results = []
        for run_step in (step, graph.replay):
            set_lens(lens, new)
            run_step()
            torch.cuda.synchronize()
            assert cpa.device_status() == 0
            n = sum(new)
            results.append([x.clone() for x in (turned, out[:n], lse[:, :n], kc, vc, w) + tuple(moved)])
        for x, y in zip(*results):
            assert same(x.contiguous(), y.contiguous())
        assert results[0][6].tolist() == [min(a + b, c) for a, b, c in zip(lens, new, (most, 30, 0))]
