"""The attention weight of cached positions on the GPU against the definition in 64 bits.

Tolerances.  A term exp(z), z = scale q.k - lse, is off by its exponent's error:
the sum of D products by D 2^-23 of their absolute sum S (an adder that
truncates), its scaling and the subtraction by 4 2^-23 (1 + S + |lse|); and by
2^-21 for the exponential.  A sum of n terms in float32 is off by n 2^-24 of
itself in whatever order, the decayed old value by 2^-23, and each term below 2^-126
may be taken as 0.
"""
import math

import pytest
import torch

import context_causal_attention_zigzag_gb300 as cpa

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


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


def table_of(need, seed=0, spare=3, extra=0):
    g = torch.Generator().manual_seed(seed)
    ids = torch.randperm(sum(need) + spare, generator=g).tolist()
    width, rows, at = max(need + [0]) + extra, [], 0
    for n in need:
        rows.append(ids[at:at + n] + [-1] * (width - n))
        at += n
    return ints(rows).view(len(need), width), sum(need) + spare


def random_tree(n, seed):
    g = torch.Generator().manual_seed(seed)
    words = []
    for i in range(n):
        parent = int(torch.randint(-1, i, (1,), generator=g)) if i else -1
        words.append((words[parent] if parent >= 0 else 0) | (1 << i))
    return [w - (1 << 64) if w >> 63 else w for w in words]


def reference(q, k_cache, table, ctx, new, lse, weights, tree, scale, decay):
    """(weights, tolerance) in 64 bits."""
    H, D = q.shape[1:]
    P, Hkv = k_cache.shape[1:3]
    w, tol = weights.double().clone(), torch.zeros_like(weights, dtype=torch.float64)
    first, G = offsets(new), H // Hkv
    scale = 1 / math.sqrt(D) if scale is None else scale
    u = 2.0 ** -23
    for r, (x, n) in enumerate(zip(ctx, new)):
        if n == 0:
            continue
        pos = torch.arange(x + n, device=DEV)
        page = table[r].long()[pos // P]
        k = k_cache[page, pos % P].double()
        if tree is None:
            seen = pos[None] <= torch.arange(n, device=DEV)[:, None] + x
        else:
            words = [b & (1 << 64) - 1 for b in tree[first[r]:first[r + 1]].tolist()]
            seen = torch.tensor([[j < x or bool(b >> (j - x) & 1) for j in range(x + n)] for b in words], device=DEV)
        for g in range(Hkv):
            total = torch.where(pos < x, w[page, g, pos % P] * decay, 0.0)
            off = total.abs() * u
            for h in range(g * G, g * G + G):
                qq, l = q[first[r]:first[r + 1], h].double(), lse[h, first[r]:first[r + 1]].double()[:, None]
                some = seen & ~(l == -math.inf)
                z = qq @ k[:, g].T * scale - l
                S = qq.abs() @ k[:, g].abs().T * scale
                t = torch.where(some, z.exp(), 0.0)
                total = total + t.sum(0)
                off = off + torch.where(some, t * (u * (D * S + 4 * (1 + S + l.abs())) + 2.0 ** -21) + 2.0 ** -126,
                                        0.0).sum(0)
            off = off + total.abs() * (n * G + 2) * u / 2
            w[page, g, pos % P], tol[page, g, pos % P] = total, off
    return w, tol


def check(got, want, tol):
    off = (got.double() - want).abs()
    assert not bool(torch.isnan(off).any()) and not bool((off > tol).any()), \
        f"off by {off.max().item():.3e}, {(off - tol).max().item():.3e} over its bound"


CASES = [
    # ctx, new, H, Hkv, D, page, tree
    ([1000], [1], 32, 8, 128, 64, False),
    ([0], [1], 4, 2, 64, 16, False),
    ([127, 128, 129, 0, 500], [1, 1, 1, 1, 1], 8, 2, 128, 16, False),
    ([100, 0, 37, 255], [3, 64, 0, 17], 14, 2, 64, 32, True),
    ([300, 5000], [64, 7], 32, 8, 128, 128, True),
    ([0, 0, 0], [300, 1, 129], 4, 4, 128, 256, False),
    ([0, 40], [1030, 200], 8, 1, 128, 64, False),
    ([70, 0, 3], [255, 257, 256], 6, 2, 64, 16, False),
    ([1] * 70, [1] * 70, 4, 1, 64, 32, False),
    ([9000], [130], 8, 2, 64, 1024, False),
    ([10, 20], [40, 3], 100, 1, 64, 384, False),     # many query heads, a page of three tiles
    ([200] * 3, [33, 65, 1], 128, 1, 128, 16, False),
    ([0], [2500], 14, 2, 64, 128, False),
    ([0] * 20, [100, 37, 0, 500, 1] * 4, 16, 8, 64, 16, False),
    ([40000, 3, 17], [1, 2, 1], 8, 8, 128, 64, False),
    ([600, 30], [1, 1500], 32, 8, 64, 64, False),     # one step beside a whole prompt
]


def make(ctx, new, H, Hkv, D, P, tree, dtype, seed=0, padded=0):
    table, pages = table_of([-(-(x + n) // P) for x, n in zip(ctx, new)], seed)
    N = sum(new) + padded
    q = normal(seed + 1, N, H, D, dtype=TYPES[dtype])
    k = normal(seed + 2, pages, P, Hkv, D, dtype=TYPES[dtype])
    v = normal(seed + 3, pages, P, Hkv, D, dtype=TYPES[dtype])
    words = ints([w for r, n in enumerate(new) for w in random_tree(n, r)] + [0] * padded, torch.int64) if tree else None
    cu = ints(offsets(new))
    out, lse = cpa.tree_attention(q, k, v, table, ints(ctx), cu, words)
    if padded:
        lse[:, -padded:] = math.nan
    g = torch.Generator().manual_seed(seed + 4)
    weights = torch.rand(pages, Hkv, P, generator=g).mul(5).to(DEV)
    return q, k, table, ints(ctx), cu, lse, weights, words


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("ctx,new,H,Hkv,D,P,tree", CASES)
def test_cache_weights(ctx, new, H, Hkv, D, P, tree, dtype):
    q, k, table, c, cu, lse, weights, words = make(ctx, new, H, Hkv, D, P, tree, dtype)
    want, tol = reference(q, k, table, ctx, new, lse, weights, words, None, 0.9)
    again = weights.clone()
    got = cpa.cache_weights(q, k, table, c, cu, lse, weights, tree=words, decay=0.9)
    assert cpa.device_status() == 0 and got.data_ptr() == weights.data_ptr()
    check(got, want, tol)
    assert torch.equal(got, cpa.cache_weights(q, k, table, c, cu, lse, again, tree=words, decay=0.9))
    # Each row gave 1 in all: with nothing there before, a head's weights add up to its rows.
    if sum(ctx) == 0:
        sums = torch.zeros_like(weights, dtype=torch.float64)
        for r, n in enumerate(new):
            pos = torch.arange(n, device=DEV)
            sums[table[r].long()[pos // P], :, pos % P] = got.double()[table[r].long()[pos // P], :, pos % P]
        assert torch.allclose(sums.sum((0, 2)), torch.full((Hkv,), float(sum(new) * H // Hkv), dtype=torch.float64,
                                                           device=DEV), rtol=1e-3)


def test_scale_strides_and_padded_rows():
    ctx, new, H, Hkv, D, P = [300, 70], [5, 9], 8, 2, 128, 16
    q, k, table, c, cu, lse, weights, _ = make(ctx, new, H, Hkv, D, P, False, "bf16", padded=4)
    wide = torch.full((18, H + 4, D), math.nan, device=DEV, dtype=torch.bfloat16)
    wide[:, 2:2 + H] = q
    heads_first = k.transpose(1, 2).contiguous().transpose(1, 2)
    lse = lse * 0.3
    want, tol = reference(q, k, table, ctx, new, lse, weights, None, 0.05, 1.0)
    check(cpa.cache_weights(wide[:, 2:2 + H], heads_first, table, c, cu, lse, weights, scale=0.05), want, tol)


def test_what_lies_outside_does_not_reach_a_request():
    ctx, new, H, Hkv, D, P = [130, 20, 64], [1, 0, 3], 4, 2, 64, 32
    q, k, table, c, cu, lse, weights, _ = make(ctx, new, H, Hkv, D, P, False, "bf16")
    want, tol = reference(q, k, table, ctx, new, lse, weights, None, None, 1.0)
    live = torch.zeros(k.shape[0], P, dtype=torch.bool, device=DEV)
    for r, (x, n) in enumerate(zip(ctx, new)):
        pos = torch.arange(x + n, device=DEV)
        live[table[r].long()[pos // P], pos % P] = n > 0
    k[~live] = math.nan
    old = weights.clone()
    got = cpa.cache_weights(q, k, table, c, cu, lse, weights)
    check(got, want, tol)
    assert torch.equal(got.transpose(1, 2)[~live], old.transpose(1, 2)[~live])
    # A row that saw nothing gives nothing; a NaN normaliser reaches what its row sees and no more.
    for value in (-math.inf, math.nan):
        lse[1, 0] = value
        want, tol = reference(q, k, table, ctx, new, lse, old, None, None, 1.0)
        weights.copy_(old)
        got = cpa.cache_weights(q, k, table, c, cu, lse, weights)
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        keep = ~torch.isnan(want)
        assert not bool(((got.double() - want).abs() > tol)[keep].any())
        if math.isnan(value):
            assert int(torch.isnan(want).sum()) == 131


def test_graphs_streams_and_changing_lengths():
    ctx, new, H, Hkv, D, P = [400, 90, 256], [1, 1, 1], 8, 2, 128, 64
    q, k, table, c, cu, lse, weights, _ = make(ctx, new, H, Hkv, D, P, False, "bf16")
    start = weights.clone()
    ws = cpa.cache_weights_workspace(q, k, cu)
    cpa.cache_weights(q, k, table, c, cu, lse, weights, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cpa.cache_weights(q, k, table, c, cu, lse, weights, workspace=ws)
    for shorter in (0, 100, 57):
        lens = [max(0, x - shorter) for x in ctx]
        c.copy_(ints(lens))
        weights.copy_(start)
        graph.replay()
        want, tol = reference(q, k, table, lens, new, lse, start, None, None, 1.0)
        check(weights, want, tol)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        weights.copy_(start)
        cpa.cache_weights(q, k, table, c, cu, lse, weights)
    s.synchronize()
    check(weights, want, tol)


def test_broken_lengths_and_tables_are_reported():
    ctx, new, H, Hkv, D, P = [100, 50], [2, 2], 4, 2, 64, 16
    for what in ("page", "negative", "long", "offsets", "tree"):
        q, k, table, c, cu, lse, weights, _ = make(ctx, new, H, Hkv, D, P, False, "bf16")
        tree = None
        if what == "page":
            table[0, 1] = k.shape[0]
        elif what == "negative":
            c[1] = -5
        elif what == "long":
            c[1] = 10000
        elif what == "offsets":
            cu[1] = 9
        else:
            q, k, table, c, cu, lse, weights, _ = make([3], [70], H, Hkv, D, P, False, "bf16")
            tree = torch.zeros(70, dtype=torch.int64, device=DEV)
        cpa.cache_weights(q, k, table, c, cu, lse, weights, tree=tree)
        assert cpa.device_status() == -1, what
    assert cpa.device_status() == 0


@pytest.mark.parametrize("R,most_ctx,most_new", [(1500, 60, 3), (1300, 5, 90)])
def test_thousands_of_requests(R, most_ctx, most_new):
    g = torch.Generator().manual_seed(R)
    ctx, new = (torch.randint(0, n + 1, (R,), generator=g).tolist() for n in (most_ctx, most_new))
    q, k, table, c, cu, lse, weights, _ = make(ctx, new, 4, 1, 64, 16, False, "bf16", seed=R)
    want, tol = reference(q, k, table, ctx, new, lse, weights, None, None, 1.0)
    got = cpa.cache_weights(q, k, table, c, cu, lse, weights)
    assert cpa.device_status() == 0
    check(got, want, tol)
