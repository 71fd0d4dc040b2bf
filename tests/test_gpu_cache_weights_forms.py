"""The weight of cached positions in each form of its tensor-core kernel: keys that stream past a
request's rows, rows that stream past two key tiles, and a step beside a longer prompt.

Tolerances.  A term exp(scale q.k - lse) is off by its exponent's error, the sum of D products by
D 2^-23 of their absolute sum S and the scaling and subtraction by 4 2^-23 (1 + S + |lse|), and by
2^-21 for the exponential.  A tile of 128 terms is added in four sums of at most 32 terms and those
in two steps: 34 2^-24.  Tiles are added with compensation, 2 2^-24; then the sums of three
warpgroups, of the CTAs that share an item, and the old value: one 2^-24 each.
"""
import math

import pytest
import torch

import context_causal_attention_zigzag_gb300 as cpa

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
CTAS = 160  # at most

# ctx, new, H, Hkv, D, page.  Calls of more than 32 rows (tokens x H / Hkv) go to the tensor cores; up to
# 128 rows a request on the average keys stream.
FORMS = {
    "keys": ([130, 20, 64, 700], [9, 0, 13, 1], 8, 2, 64, 32),
    "keys128": ([1000, 0, 255], [3, 12, 1], 32, 8, 128, 64),
    "rows": ([300, 20, 64], [150, 0, 170], 8, 2, 64, 16),
    "rows128": ([700, 0, 40], [300, 80, 1], 16, 2, 128, 256),
    "prompt beside steps": ([500] * 40, [1] * 17 + [300] + [0] * 2 + [1] * 20, 8, 2, 128, 128),
}


def normal(seed, *shape, dtype):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(dtype).to(DEV)


def ints(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device=DEV)


def offsets(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def table_of(need, seed=0, spare=3):
    g = torch.Generator().manual_seed(seed)
    ids = torch.randperm(sum(need) + spare, generator=g).tolist()
    width, rows, at = max(need), [], 0
    for n in need:
        rows.append(ids[at:at + n] + [-1] * (width - n))
        at += n
    return ints(rows), sum(need) + spare


def places(table, r, n, P):
    pos = torch.arange(n, device=DEV)
    return table[r].long()[pos // P], pos % P


def reference(q, k_cache, table, ctx, new, lse, weights, decay=1.0):
    """(weights, tolerance) in 64 bits; tokens see the old positions and those up to their own."""
    H, D = q.shape[1:]
    P, Hkv = k_cache.shape[1:3]
    w, tol = weights.double().clone(), torch.zeros_like(weights, dtype=torch.float64)
    first, G, u = offsets(new), H // Hkv, 2.0 ** -24
    items = sum(-(-(x + n) // 256) for x, n in zip(ctx, new) if n) * Hkv
    shared = CTAS // max(1, items) + 2  # CTAs that may share an item
    for r, (x, n) in enumerate(zip(ctx, new)):
        if n == 0:
            continue
        page, i = places(table, r, x + n, P)
        k, pos = k_cache[page, i].double(), torch.arange(x + n, device=DEV)
        seen = pos[None] <= torch.arange(n, device=DEV)[:, None] + x
        for g in range(Hkv):
            total = torch.where(pos < x, w[page, g, i] * decay, 0.0)
            off = total.abs() * u
            for h in range(g * G, g * G + G):
                qq, l = q[first[r]:first[r + 1], h].double(), lse[h, first[r]:first[r + 1]].double()[:, None]
                some = seen & ~(l == -math.inf)
                S = qq.abs() @ k[:, g].abs().T / math.sqrt(D)
                t = torch.where(some, (qq @ k[:, g].T / math.sqrt(D) - l).exp(), 0.0)
                total = total + t.sum(0)
                bound = t * (2 * u * (D * S + 4 * (1 + S + l.abs())) + 2.0 ** -21) + 2.0 ** -126
                off = off + torch.where(some, bound, 0.0).sum(0)
            off = off + total.abs() * (34 + 2 + 3 + shared + 1) * u
            w[page, g, i], tol[page, g, i] = total, off
    return w, tol


def check(got, want, tol):
    off = (got.double() - want).abs()
    assert not bool(torch.isnan(off).any()) and not bool((off > tol).any()), \
        f"off by {off.max().item():.3e}, {(off - tol).max().item():.3e} over its bound"


def make(ctx, new, H, Hkv, D, P, dtype="bf16", scale=1.0):
    assert sum(new) * H // Hkv > 32
    table, pages = table_of([-(-(x + n) // P) for x, n in zip(ctx, new)])
    q = normal(1, sum(new), H, D, dtype=TYPES[dtype]) * scale
    k = normal(2, pages, P, Hkv, D, dtype=TYPES[dtype]) * scale
    g = torch.Generator().manual_seed(3)
    lse = (torch.rand(H, sum(new), generator=g) * 2 - 1).to(DEV)
    weights = torch.rand(pages, Hkv, P, generator=g).mul(5).to(DEV)
    return q, k, table, ints(ctx), ints(offsets(new)), lse, weights


def live_places(k, table, ctx, new):
    live = torch.zeros(k.shape[:2], dtype=torch.bool, device=DEV)
    for r, (x, n) in enumerate(zip(ctx, new)):
        if n:
            live[places(table, r, x + n, k.shape[1])] = True
    return live


@pytest.mark.parametrize("form", list(FORMS))
def test_what_lies_outside_does_not_reach_a_request(form):
    ctx, new = FORMS[form][:2]
    q, k, table, c, cu, lse, weights = make(*FORMS[form])
    want, tol = reference(q, k, table, ctx, new, lse, weights, 0.9)
    live = live_places(k, table, ctx, new)
    k[~live] = math.nan
    old = weights.clone()
    got = cpa.cache_weights(q, k, table, c, cu, lse, weights, decay=0.9)
    assert cpa.device_status() == 0
    check(got, want, tol)
    assert torch.equal(got.transpose(1, 2)[~live], old.transpose(1, 2)[~live])


@pytest.mark.parametrize("form", list(FORMS))
def test_rows_with_broken_normalisers(form):
    """-inf: the row gives nothing; NaN and +inf: exp says what it gives, to what it sees and no more."""
    ctx, new = FORMS[form][:2]
    q, k, table, c, cu, lse, weights = make(*FORMS[form])
    last = sum(new) - 1
    for h, i, value in ((1, 0, -math.inf), (0, last, -math.inf), (2, last // 2, math.inf), (3, last // 3, math.nan)):
        lse[h, i] = value
    want, tol = reference(q, k, table, ctx, new, lse, weights)
    got = cpa.cache_weights(q, k, table, c, cu, lse, weights)
    assert torch.equal(torch.isnan(got), torch.isnan(want)) and bool(torch.isnan(want).any())
    keep = ~torch.isnan(want)
    assert not bool(((got.double() - want).abs() > tol)[keep].any())


@pytest.mark.parametrize("form", list(FORMS))
@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_rows_that_give_nothing_may_hold_anything(form, value):
    """Padding within a request, say: q as it was left, lse -inf."""
    ctx, new = FORMS[form][:2]
    q, k, table, c, cu, lse, weights = make(*FORMS[form])
    want_q = q.clone()
    for h in range(q.shape[1]):
        for i in (h % sum(new), (sum(new) - 1 - h) % sum(new), sum(new) // 2):
            lse[h, i] = -math.inf
            q[i, h, h % 7] = value
            want_q[i, h] = 0
    want, tol = reference(want_q, k, table, ctx, new, lse, weights)
    got = cpa.cache_weights(q, k, table, c, cu, lse, weights)
    assert cpa.device_status() == 0
    check(got, want, tol)


@pytest.mark.parametrize("form", list(FORMS))
def test_graphs_streams_and_changing_lengths(form):
    ctx, new = FORMS[form][:2]
    q, k, table, c, cu, lse, weights = make(*FORMS[form])
    start = weights.clone()
    ws = cpa.cache_weights_workspace(q, k, cu)
    cpa.cache_weights(q, k, table, c, cu, lse, weights, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cpa.cache_weights(q, k, table, c, cu, lse, weights, workspace=ws)
    for shorter, turn in ((0, 0), (100, 1), (57, 2)):
        lens = [max(0, x - shorter) for x in ctx]
        counts = [n if i % 2 else max(0, n - turn) for i, n in enumerate(new)]
        c.copy_(ints(lens))
        cu.copy_(ints(offsets(counts)))
        weights.copy_(start)
        graph.replay()
        want, tol = reference(q, k, table, lens, counts, lse, start)
        check(weights, want, tol)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        weights.copy_(start)
        cpa.cache_weights(q, k, table, c, cu, lse, weights)
    s.synchronize()
    check(weights, want, tol)
    assert cpa.device_status() == 0


@pytest.mark.parametrize("form", list(FORMS))
@pytest.mark.parametrize("what", ["page", "negative page", "negative", "long", "offsets", "falling offsets"])
def test_broken_lengths_and_tables_are_reported(form, what):
    """The error word says so, and nothing is written where no request has a page."""
    ctx, new = FORMS[form][:2]
    q, k, table, c, cu, lse, weights = make(*FORMS[form])
    used = torch.zeros(k.shape[0], dtype=torch.bool, device=DEV)
    used[table[table >= 0].long()] = True
    old = weights.clone()
    want, tol = reference(q, k, table, ctx, new, lse, weights)
    if what == "page":
        table[0, 0] = k.shape[0]
    elif what == "negative page":
        table[0, 0] = -7
    elif what == "negative":
        c[0] = -5
    elif what == "long":
        c[0] = 1 << 30
    elif what == "offsets":
        cu[-1] = sum(new) + 1
    else:
        cu[1] = sum(new)
        cu[2] = 0
    cpa.cache_weights(q, k, table, c, cu, lse, weights)
    assert cpa.device_status() == -1 and cpa.device_status() == 0
    assert torch.equal(weights[~used], old[~used])
    if what.endswith("page"):  # the other requests have their weights
        for r, (x, n) in enumerate(zip(ctx, new)):
            if r > 0 and n:
                page, i = places(table, r, x + n, k.shape[1])
                check(weights[page, :, i], want[page, :, i], tol[page, :, i])


@pytest.mark.parametrize("ctx,new,H,Hkv,D,P", [
    ([100, 7], [5000, 3], 14, 2, 64, 128),            # rows stream, cut items
    ([300] * 60, [1] * 59 + [900], 8, 2, 128, 64),    # keys stream past a prompt of 29 tiles
    ([3000] * 40, [30] * 40, 4, 1, 64, 16),
])
def test_every_row_counts_once(ctx, new, H, Hkv, D, P):
    """Scores of 0 and lse of 0: each row that sees a position gives it 1, and sums of ones are exact."""
    q, k, table, c, cu, lse, weights = make(ctx, new, H, Hkv, D, P)
    q.zero_()
    lse.zero_()
    want = weights.clone()
    for r, (x, n) in enumerate(zip(ctx, new)):
        page, i = places(table, r, x + n, P)
        rows = torch.clamp(x + n - torch.arange(x + n, device=DEV), max=n).float() * (H // Hkv)
        want[page, :, i] = rows[:, None].expand(-1, Hkv)
    got = cpa.cache_weights(q, k, table, c, cu, lse, weights, decay=0.0)
    assert cpa.device_status() == 0
    assert torch.equal(got, want)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("ctx,new,H,Hkv,D,P", [
    ([100, 7], [2500, 3], 14, 2, 64, 128), ([50], [2000], 8, 2, 128, 64), ([300] * 60, [1] * 59 + [900], 8, 2, 128, 64)])
def test_small_scores_to_a_part_of_a_row(ctx, new, H, Hkv, D, P, dtype):
    """With scores near 0 the bound is below what a single row gives (2 e^-1 of some 2500 x 7 x 1.2, 3e-5 of
    a sum): the bound's part is 5e-6."""
    q, k, table, c, cu, lse, weights = make(ctx, new, H, Hkv, D, P, dtype, scale=2.0 ** -4)
    want, tol = reference(q, k, table, ctx, new, lse, weights)
    assert float((tol / want).max()) < 6e-6
    check(cpa.cache_weights(q, k, table, c, cu, lse, weights), want, tol)


def test_tiles_are_added_with_compensation():
    """A first tile of 2^27 and 2047 of 6.4, each below half a step of it (8): one in three is added to that sum.
    Without the compensation 682 x 6.4 are lost, 3.2e-5 of the sum.  Bound: 4 2^-23 (1 + 16.7) + 2^-21 for the
    large terms, 45 2^-24 for the sums, 1.2e-5."""
    ctx, n, H, Hkv, D, P = 256, 32768, 32, 4, 64, 256
    table, pages = table_of([-(-(ctx + n) // P)])
    q = torch.zeros(n, H, D, device=DEV, dtype=torch.bfloat16)
    k = normal(2, pages, P, Hkv, D, dtype=torch.bfloat16)
    lse = torch.full((H, n), math.log(20), device=DEV)
    lse[:, 0] = -24 * math.log(2)
    weights = torch.zeros(pages, Hkv, P, device=DEV)
    cpa.cache_weights(q, k, table, ints([ctx]), ints([0, n]), lse, weights)
    assert cpa.device_status() == 0
    page, i = places(table, 0, ctx, P)
    want = 8 * ((-lse[0, 0].double()).exp() + (n - 1) * (-lse[0, 1].double()).exp())
    off = (weights[page, :, i].double() / want - 1).abs()
    assert float(off.max()) < 1.2e-5


def test_more_rows_than_stream_past():
    """Single tokens of so many requests that the form for a few rows each is not taken."""
    R, H, D, P = 140000, 128, 64, 16
    q = torch.zeros(R, H, D, device=DEV, dtype=torch.bfloat16)
    k = torch.ones(R, P, 1, D, device=DEV, dtype=torch.bfloat16)
    table = torch.arange(R, device=DEV, dtype=torch.int32).flip(0).contiguous()[:, None]
    ctx = torch.arange(R, device=DEV, dtype=torch.int32) % 12
    weights = torch.full((R, 1, P), 3.0, device=DEV)
    cpa.cache_weights(q, k, table, ctx, torch.arange(R + 1, device=DEV, dtype=torch.int32),
                      torch.zeros(H, R, device=DEV), weights, decay=0.5)
    assert cpa.device_status() == 0
    pos, x = torch.arange(P, device=DEV), ctx.flip(0)[:, None]
    want = torch.where(pos < x, 1.5 + H, torch.where(pos == x, float(H), 3.0))
    assert torch.equal(weights[:, 0], want)


def test_most_rows_of_one_request_where_keys_stream():
    """2^17 requests, all tokens one's: tiles of one token, 2^17 steps of 1.7 us to an item at most (0.2 s of the
    2 after which waits give up).  Each row gives 1, and sums up to 2^24 are exact."""
    R, H, D, P = 1 << 17, 128, 64, 1024
    N, at = R, 70001
    q = torch.zeros(N, H, D, device=DEV, dtype=torch.bfloat16)
    k = torch.ones(N // P, P, 1, D, device=DEV, dtype=torch.bfloat16)
    table = torch.full((R, N // P), -1, device=DEV, dtype=torch.int32)
    table[at] = torch.arange(N // P, device=DEV, dtype=torch.int32).flip(0)
    cu = torch.zeros(R + 1, device=DEV, dtype=torch.int32)
    cu[at + 1:] = N
    weights = torch.full((N // P, 1, P), 3.0, device=DEV)
    cpa.cache_weights(q, k, table, torch.zeros(R, device=DEV, dtype=torch.int32), cu, torch.zeros(H, N, device=DEV),
                      weights)
    assert cpa.device_status() == 0
    want = (N - torch.arange(N, device=DEV)).float() * H
    assert torch.equal(weights.flip(0).reshape(-1), want)
