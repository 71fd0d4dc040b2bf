"""Answering calls on the GPU against a plain implementation in 64 bits.

Tolerances.  With p the normalised weights, A = sum_j p_j |v_j| and S the row's
largest sum_d |q_d k_d| * scale:
  - the output's rounding is off by eps/2 |o| at most, the weights' rounding to
    the input type for the second product by eps/2 A, and in float16, whose
    smallest step is 2^-24, by another 2^-25 per key and unit of v against a
    sum of weights of at least 1;
  - a float32 sum of D products is off by D 2^-23 S at most (an adder that
    truncates), and a weight by as much relative to itself; the sums over n
    keys by n 2^-23 relative; twice (weights and their sum).
  - lse is off by the scores' error, the sum's, and 2^-22 (1 + |lse|) for the
    logarithm and the last roundings.
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


def plain(q, k, v, seen, scale=None):
    """q [n, H, D], k, v [m, Hkv, D], seen [n, m] -> (o, lse, tol_o, tol_lse) in 64 bits."""
    n, H, D = q.shape
    m, Hkv = k.shape[:2]
    eps = torch.finfo(q.dtype).eps
    tiny = 2.0 ** -25 if q.dtype == torch.float16 else 0.0
    f = 2.0 ** -23
    q, k, v = q.double(), k.double(), v.double()
    o, to = torch.zeros(n, H, D, dtype=torch.float64, device=DEV), torch.zeros(n, H, D, dtype=torch.float64, device=DEV)
    lse, tl = (torch.full((H, n), -math.inf, dtype=torch.float64, device=DEV),
               torch.zeros(H, n, dtype=torch.float64, device=DEV))
    scale = 1 / math.sqrt(D) if scale is None else scale
    for h in range(H):
        if n == 0 or m == 0:
            break
        kk, vv = k[:, h // (H // Hkv)], v[:, h // (H // Hkv)]
        s = (q[:, h] @ kk.T * scale).masked_fill(~seen, -math.inf)
        S = (q[:, h].abs() @ kk.abs().T * scale).masked_fill(~seen, 0).amax(1, keepdim=True)
        top = s.amax(1, keepdim=True)
        p = torch.where(seen, (s - top.clamp_min(-1e300)).exp(), 0.0)
        z = p.sum(1, keepdim=True)
        some = z > 0
        p = torch.where(some, p / z, 0.0)
        o[:, h] = p @ vv
        A = p @ vv.abs()
        rel = 2 * f * (D * S + m)
        to[:, h] = eps / 2 * (o[:, h].abs() + A) * (1 + 2 * eps) + A * rel + m * tiny * vv.abs().max()
        l = torch.where(some, z.log() + top, -math.inf)
        lse[h] = l[:, 0]
        tl[h] = (f * (D * S + m) + 2 * f * (1 + l.abs()))[:, 0]
    return o, lse, to, tl


def check(got, want, tol, what):
    got = got.double()
    empty = torch.isinf(want)
    assert torch.equal(torch.isinf(got), empty), what
    off = torch.where(empty, torch.zeros_like(want), (got - want).abs())
    worst = off - torch.where(empty, torch.zeros_like(want), tol)
    assert not bool((worst > 0).any()) and not bool(torch.isnan(off).any()), \
        f"{what}: off by {off.max().item():.3e}, {worst.max().item():.3e} over its bound"


# ---------------------------------------------------------------------------
# packed prompts
# ---------------------------------------------------------------------------

def prompt_reference(q, k, v, nq, nk, causal, scale=None):
    parts = []
    fq, fk = offsets(nq), offsets(nk)
    for r, (n, m) in enumerate(zip(nq, nk)):
        i, j = torch.arange(n, device=DEV)[:, None], torch.arange(m, device=DEV)[None]
        seen = (j <= i + m - n) if causal else torch.ones(n, m, dtype=torch.bool, device=DEV)
        parts.append(plain(q[fq[r]:fq[r + 1]], k[fk[r]:fk[r + 1]], v[fk[r]:fk[r + 1]], seen, scale))
    o, lse, to, tl = zip(*parts)
    return torch.cat(o), torch.cat(lse, 1), torch.cat(to), torch.cat(tl, 1)


PROMPTS = [
    # nq, nk (None: nq), H, Hkv, D
    ([1], None, 4, 2, 128),
    ([128], None, 4, 4, 128),
    ([129], None, 2, 1, 64),
    ([77, 1, 0, 300, 128, 127], None, 4, 2, 128),
    ([255, 256, 257, 513], None, 3, 1, 64),
    ([5, 1, 64, 200], [300, 129, 64, 456], 8, 2, 128),
    ([5, 1, 64, 200], [300, 129, 64, 456], 14, 2, 64),
    ([40, 200, 3, 1], [39, 10, 0, 1], 4, 4, 128),     # rows that see nothing
    ([1] * 70, None, 4, 1, 64),
    ([1030], [2100], 2, 2, 128),
    ([5, 0, 33, 1], [3000, 700, 2000, 5], 8, 2, 64),        # few rows, many keys
    ([37, 2, 130] * 44, None, 16, 8, 64),                    # many sequences, sorted
    ([37, 0, 130] * 44, [20, 5, 140] * 44, 12, 12, 128),
    ([3700], None, 64, 32, 64),                              # one long one
    ([100] * 64, [0, 0, 0, 90] * 16, 16, 8, 64),             # runs of items without keys
    ([300] * 40, [40, 0, 0, 0] * 10, 16, 16, 128),
    ([5], [0], 4, 2, 128),
    ([1025, 33, 600, 700], [3300, 1500, 2900, 3100], 32, 8, 64),   # many key tiles an item
    ([900, 130], [1900, 2100], 32, 8, 128),
    ([70, 0, 3], [0, 0, 0], 4, 4, 64),
    ([0, 0, 7] + [0] * 3000 + [20, 1], None, 4, 2, 64),      # mostly empty sequences
]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("nq,nk,H,Hkv,D", PROMPTS)
def test_prompt_attention(nq, nk, H, Hkv, D, causal, dtype):
    nk = nq if nk is None else nk
    q = normal(1, sum(nq), H, D, dtype=TYPES[dtype])
    k, v = (normal(s, sum(nk), Hkv, D, dtype=TYPES[dtype]) for s in (2, 3))
    out, lse = cpa.prompt_attention(q, k, v, ints(offsets(nq)), ints(offsets(nk)), causal=causal)
    assert cpa.device_status() == 0
    o, l, to, tl = prompt_reference(q, k, v, nq, nk, causal)
    check(out, o, to, "out")
    check(lse, l, tl, "lse")


def test_prompt_attention_of_a_fused_projection_with_scale_and_large_scores():
    H, Hkv, D, nq = 4, 2, 128, [130, 70, 300]
    x = normal(5, sum(nq), H + 2 * Hkv, D, dtype=torch.bfloat16) * 3
    q, k, v = x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:]
    cu = ints(offsets(nq))
    out, lse = cpa.prompt_attention(q, k, v, cu, scale=0.3)
    o, l, to, tl = prompt_reference(q, k, v, nq, nq, True, 0.3)
    check(out, o, to, "out")
    check(lse, l, tl, "lse")


@pytest.mark.parametrize("nq,nk", [
    ([3, 5, 2, 4], None),                                    # a block a token
    ([100, 60, 140, 30], None),                              # an item a CTA
    ([2, 1, 3, 1], [600, 900, 700, 800]),                    # keys shared among CTAs
    ([100, 60, 140, 30] * 30, None),                         # sorted
    ([100, 60, 140, 30] * 30, [150, 70, 140, 200] * 30),
])
def test_prompt_attention_keeps_sequences_apart_and_rows_behind_the_last(nq, nk):
    # The rows of the second sequence, and those behind the last, are NaN or
    # infinite: no other sequence's result changes, and rows behind stay as they
    # were.
    H, Hkv, D = 4, 2, 128
    tail = 37
    nk = nq if nk is None else nk
    q = normal(1, sum(nq) + tail, H, D, dtype=torch.bfloat16)
    k, v = (normal(s, sum(nk) + tail, Hkv, D, dtype=torch.bfloat16) for s in (2, 3))
    cu_q, cu_k = ints(offsets(nq)), ints(offsets(nk))
    want, wlse = cpa.prompt_attention(q, k, v, cu_q, cu_k)
    bad, bad_k = slice(nq[0], nq[0] + nq[1]), slice(nk[0], nk[0] + nk[1])
    for t, x, b, n in ((q, math.nan, bad, nq), (k, math.inf, bad_k, nk), (v, math.nan, bad_k, nk)):
        t[b] = x
        t[sum(n):] = x
    out, lse = torch.full_like(want, 7.0), torch.full_like(wlse, 7.0)
    cpa.prompt_attention(q, k, v, cu_q, cu_k, out=out, lse=lse)
    good = torch.ones(sum(nq), dtype=torch.bool, device=DEV)
    good[bad] = False
    good = good.nonzero()[:, 0]
    assert torch.equal(out[good], want[good]) and torch.equal(lse[:, good], wlse[:, good])
    assert bool((out[sum(nq):] == 7).all()) and bool((lse[:, sum(nq):] == 7).all())
    assert bool(torch.isnan(out[bad]).all())
    assert cpa.device_status() == 0


def test_prompt_attention_reports_broken_offsets():
    q = normal(1, 300, 2, 64, dtype=torch.float16)
    for cu in ([0, 200, 100, 300], [0, 100, 301], [5, 100, 300], [0, -4, 300], [0, 300, 0, 300]):
        out, _ = cpa.prompt_attention(q, q, q, ints(cu))
        assert cpa.device_status() == -1, cu
        assert out.shape == q.shape
    assert cpa.device_status() == 0


# 4 rows a sequence on the average and many keys (the cut line), 262 (sorted blocks).
@pytest.mark.parametrize("H,nq,nk", [(1, 1 << 14, 1 << 21), (2, 1 << 20, 1 << 20)])
def test_offsets_that_name_the_same_rows_over_and_over(H, nq, nk):
    # Every other sequence claims all rows: far more work than the tensors hold.
    q = normal(1, nq, H, 64, dtype=torch.bfloat16)
    k = normal(2, nk, H, 64, dtype=torch.bfloat16)
    cu_q, cu_k = (ints([0, n] * 2000 + [0, n]) for n in (nq, nk))
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    begin.record()
    cpa.prompt_attention(q, k, k, cu_q, cu_k)
    end.record()
    assert cpa.device_status() == -1
    assert begin.elapsed_time(end) < 1000
    pages = normal(3, 8, 16, H, 64, dtype=torch.bfloat16)
    table = torch.zeros(4001, 2000, dtype=torch.int32, device=DEV)
    cpa.tree_attention(q, pages, pages, table, ints([100] * 4001), cu_q)
    assert cpa.device_status() == -1
    cpa.prompt_attention(q[:300], q[:300], q[:300], ints([0, 300]))
    assert cpa.device_status() == 0


# ---------------------------------------------------------------------------
# the cache
# ---------------------------------------------------------------------------

class Cache:
    """A paged cache with pages dealt at random, filled with `fill` elsewhere."""

    def __init__(self, ctx, new, Hkv, D, P, dtype, order="tokens", fill=math.nan, seed=11, wider=1):
        self.ctx, self.new, self.P = ctx, new, P
        need = [-(-(c + n) // P) for c, n in zip(ctx, new)]
        pages = sum(need) + 2
        g = torch.Generator().manual_seed(seed)
        ids = torch.randperm(pages, generator=g, dtype=torch.int32)
        width = max(need + [1]) + wider
        table = torch.full((len(ctx), width), -7, dtype=torch.int32)
        first = offsets(need)
        for r, n in enumerate(need):
            table[r, :n] = ids[first[r]:first[r] + n]
        self.table = table.to(DEV)

        def empty():
            if order == "heads":
                return torch.full((pages, Hkv, P, D), fill, dtype=dtype, device=DEV).transpose(1, 2)
            return torch.full((pages, P, Hkv, D), fill, dtype=dtype, device=DEV)
        if order == "interleaved":
            both = torch.full((pages, 2, P, Hkv, D), fill, dtype=dtype, device=DEV)
            self.k, self.v = both[:, 0], both[:, 1]
        else:
            self.k, self.v = empty(), empty()
        self.K = [normal(100 + r, c + n, Hkv, D, dtype=dtype) for r, (c, n) in enumerate(zip(ctx, new))]
        self.V = [normal(500 + r, c + n, Hkv, D, dtype=dtype) for r, (c, n) in enumerate(zip(ctx, new))]
        for r, (c, n) in enumerate(zip(ctx, new)):
            pos = torch.arange(c + n, device=DEV)
            page = self.table[r].long()[pos // P]
            self.k[page, pos % P] = self.K[r]
            self.v[page, pos % P] = self.V[r]


def random_tree(seed, n):
    g = torch.Generator().manual_seed(seed)
    rows = []
    for i in range(n):
        parent = int(torch.randint(-1, i, (1,), generator=g)) if i else -1
        rows.append((rows[parent] if parent >= 0 else 0) | 1 << i)
    return rows


def signed(words):
    return [w - (1 << 64) if w >> 63 else w for w in words]


def tree_reference(q, cache, words=None, scale=None):
    parts, first = [], offsets(cache.new)
    for r, (c, n) in enumerate(zip(cache.ctx, cache.new)):
        seen = torch.ones(n, c + n, dtype=torch.bool)
        for i in range(n):
            w = (1 << (i + 1)) - 1 if words is None else words[first[r] + i]
            for j in range(n):
                seen[i, c + j] = bool(w >> j & 1)
        parts.append(plain(q[first[r]:first[r + 1]], cache.K[r], cache.V[r], seen.to(DEV), scale))
    o, lse, to, tl = zip(*parts)
    return torch.cat(o), torch.cat(lse, 1), torch.cat(to), torch.cat(tl, 1)


def run_tree(q, cache, words=None, **kw):
    tree = None if words is None else ints(signed(words), torch.int64)
    return cpa.tree_attention(q, cache.k, cache.v, cache.table, ints(cache.ctx), ints(offsets(cache.new)),
                              tree, **kw)


TREES = [
    # ctx, new, H, Hkv, D, page, tree
    ([1000], [1], 8, 2, 128, 64, False),
    ([0], [1], 4, 2, 128, 16, False),
    ([0, 1, 127, 128, 129, 500], [1] * 6, 4, 1, 128, 32, False),
    ([0, 1, 127, 128, 129, 500], [1] * 6, 16, 16, 64, 16, False),
    ([300, 0, 55, 1000], [5, 0, 64, 31], 8, 2, 128, 16, True),
    ([300, 0, 55, 1000], [5, 7, 64, 31], 14, 2, 64, 64, True),
    ([129, 3000, 64], [33, 64, 64], 8, 1, 128, 256, True),    # up to 512 rows of one kv head
    ([1, 640], [63, 64], 96, 1, 64, 128, True),               # 96 heads share a kv head
    ([0, 100, 777], [300, 1, 200], 4, 2, 128, 32, False),      # parts of prompts
    ([20000], [3], 4, 2, 128, 128, True),
    ([5] * 200, [1] * 200, 2, 1, 64, 16, False),
    ([40000], [1], 2, 1, 64, 384, False),
    ([300, 7, 900, 0, 64], [1, 0, 2, 0, 5], 8, 2, 128, 32, True),   # requests without new tokens
    ([60] * 30, [0, 3] * 15, 4, 2, 64, 16, False),
    ([400] * 40, [64] * 40, 8, 2, 64, 64, True),
]


@pytest.mark.parametrize("wider", [1, 4000])  # a wide table is answered by the tensor cores
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("ctx,new,H,Hkv,D,P,tree", TREES)
def test_tree_attention(ctx, new, H, Hkv, D, P, tree, dtype, wider):
    cache = Cache(ctx, new, Hkv, D, P, TYPES[dtype], wider=wider)
    q = normal(9, sum(new), H, D, dtype=TYPES[dtype])
    words = [w for r, n in enumerate(new) for w in random_tree(r, n)] if tree else None
    out, lse = run_tree(q, cache, words)
    assert cpa.device_status() == 0
    o, l, to, tl = tree_reference(q, cache, words)
    check(out, o, to, "out")
    check(lse, l, tl, "lse")


@pytest.mark.parametrize("wider", [1, 300])
@pytest.mark.parametrize("order", ["heads", "interleaved"])
def test_tree_attention_other_cache_orders_strides_and_scale(order, wider):
    cache = Cache([200, 77], [9, 3], 2, 128, 32, torch.bfloat16, order, wider=wider)
    wide = normal(4, 12, 12, 128, dtype=torch.bfloat16)
    q = wide[:, 2:10]
    words = random_tree(1, 9) + random_tree(2, 3)
    out, lse = run_tree(q, cache, words, scale=0.21)
    o, l, to, tl = tree_reference(q, cache, words, 0.21)
    check(out, o, to, "out")
    check(lse, l, tl, "lse")


@pytest.mark.parametrize("wider", [1, 300])  # small: CUDA cores; wide: tensor cores
def test_tree_attention_rows_that_see_nothing_and_bits_behind_the_last_token(wider):
    cache = Cache([0, 0, 50], [3, 2, 4], 2, 64, 16, torch.float16, wider=wider)
    q = normal(4, 9, 4, 64, dtype=torch.float16)
    words = [0, 0b10, 0b111, 0, 0, 0b1 | 1 << 40, 0b10 | 1 << 63, 0b100, 0]
    out, lse = run_tree(q, cache, words)
    o, l, to, tl = tree_reference(q, cache, words)
    check(out, o, to, "out")
    check(lse, l, tl, "lse")
    assert bool((out[[0, 3, 4]] == 0).all()) and bool((lse[:, [0, 3, 4]] == -math.inf).all())
    assert cpa.device_status() == 0


@pytest.mark.parametrize("wider", [1, 300])  # small: CUDA cores; wide: tensor cores
def test_tree_attention_leaves_rows_behind_the_last_and_ignores_other_pages(wider):
    # Pages of other requests and unused parts of pages hold NaN (the cache's
    # fill) or infinities; q has padded rows.
    for fill in (math.nan, math.inf):
        cache = Cache([130, 20], [3, 2], 2, 128, 64, torch.bfloat16, fill=fill, wider=wider)
        q = normal(4, 12, 8, 128, dtype=torch.bfloat16)
        q[5:] = fill
        out, lse = torch.full_like(q, 7.0), torch.full((8, 12), 7.0, device=DEV)
        run_tree(q, cache, out=out, lse=lse)
        o, l, to, tl = tree_reference(q[:5], cache)
        check(out[:5], o, to, "out")
        check(lse[:, :5], l, tl, "lse")
        assert bool((out[5:] == 7).all()) and bool((lse[:, 5:] == 7).all())


@pytest.mark.parametrize("wider", [1, 300])  # small: CUDA cores; wide: tensor cores
def test_tree_attention_reports_bad_pages_and_lengths(wider):
    cache = Cache([130, 20], [3, 2], 2, 128, 64, torch.bfloat16, fill=0.0, wider=wider)
    q = normal(4, 5, 8, 128, dtype=torch.bfloat16)
    ctx, cu, good = ints([130, 20]), ints([0, 3, 5]), cache.table.clone()
    o, l, to, tl = tree_reference(q, cache)
    for page in (-1, 1000, 2 ** 31 - 1):
        table = good.clone()
        table[0, 1] = page
        out, lse = cpa.tree_attention(q, cache.k, cache.v, table, ctx, cu)
        assert cpa.device_status() == -1, page
        check(out[3:], o[3:], to[3:], "the other request")
    for ctx_, cu_ in (([-5, 20], [0, 3, 5]), ([100000, 20], [0, 3, 5]), ([130, 20], [0, 4, 3]),
                      ([130, 20], [0, 3, 6]), ([2 ** 31 - 1, 20], [0, 3, 5])):
        cpa.tree_attention(q, cache.k, cache.v, good, ints(ctx_), ints(cu_))
        assert cpa.device_status() == -1, (ctx_, cu_)
    wide = normal(4, 65, 8, 128, dtype=torch.bfloat16)
    big = Cache([10], [65], 2, 128, 64, torch.bfloat16, wider=wider)
    cpa.tree_attention(wide, big.k, big.v, big.table, ints([10]), ints([0, 65]),
                       torch.zeros(65, dtype=torch.int64, device=DEV))
    assert cpa.device_status() == -1
    assert cpa.device_status() == 0


@pytest.mark.parametrize("N", [1, 300])
def test_caches_of_one_head_or_page_with_meaningless_strides(N):
    kc, vc = (normal(s, 8, 64, 64, dtype=torch.float16) for s in (1, 2))
    k1 = kc.as_strided((8, 64, 1, 64), (4096, 64, 8, 1))
    v1 = vc.as_strided((8, 64, 1, 64), (4096, 64, 0, 1))
    q = normal(3, N, 4, 64, dtype=torch.float16)
    pages = [2, 0, 1, 7, 5, 3, 6, 4]
    out, lse = cpa.tree_attention(q, k1, v1, ints([pages]), ints([150]), ints([0, N]))
    K, V = (x[pages].reshape(-1, 1, 64)[:150 + N] for x in (kc, vc))
    at = torch.arange(150 + N, device=DEV)
    o, l, to, tl = plain(q, K, V, at[None] <= 150 + at[:N, None])
    check(out, o, to, "out")
    check(lse, l, tl, "lse")
    page = normal(5, 16, 2, 64, dtype=torch.float16)
    one = page.as_strided((1, 16, 2, 64), (3, 128, 64, 1))
    other = torch.zeros_like(page)
    x = normal(6, 2, 2, 64, dtype=torch.float16)
    cpa.cache_write(x, x, one, other.as_strided((1, 16, 2, 64), (0, 128, 64, 1)),
                    ints([3, 9], torch.int64))
    assert torch.equal(page[[3, 9]], x) and torch.equal(other[[3, 9]], x)
    assert cpa.device_status() == 0


@pytest.mark.parametrize("wider", [1, 300])
def test_requests_that_share_pages(wider):
    # Two requests with the same first pages (a common prompt), each with its own
    # behind them; the same request twice gives the same result twice.
    cache = Cache([100, 100, 100], [3, 3, 3], 2, 128, 16, torch.bfloat16, wider=wider)
    cache.table[1, :4] = cache.table[0, :4]
    cache.table[2] = cache.table[0]
    for own in (cache.K, cache.V):
        own[1][:64] = own[0][:64]
        own[2] = own[0]
    q = normal(4, 9, 8, 128, dtype=torch.bfloat16)
    q[6:] = q[:3]
    out, lse = run_tree(q, cache)
    o, l, to, tl = tree_reference(q, cache)
    check(out, o, to, "out")
    check(lse, l, tl, "lse")
    assert cpa.device_status() == 0


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("N,Hkv,D,P,order", [(1, 8, 128, 64, "tokens"), (37, 2, 64, 16, "heads"),
                                             (300, 3, 128, 384, "interleaved"), (1000, 1, 64, 128, "tokens")])
def test_cache_write(N, Hkv, D, P, order, dtype):
    pages = -(-N // P) + 2
    cache = Cache([pages * P - 2 * P], [0], Hkv, D, P, TYPES[dtype], order, fill=0.0)
    x = normal(3, N, 3 * Hkv, D, dtype=TYPES[dtype])
    k, v = x[:, :Hkv], x[:, Hkv:2 * Hkv]
    g = torch.Generator().manual_seed(N)
    slots = torch.randperm(cache.k.shape[0] * P, generator=g)[:N].to(DEV)
    skip = torch.arange(N, device=DEV) % 7 == 3
    want = [cache.k.clone(), cache.v.clone()]
    live = slots[~skip]
    for w, t in zip(want, (k, v)):
        w[live // P, live % P] = t[~skip]
    got = cpa.cache_write(k, v, cache.k, cache.v, torch.where(skip, -1 - slots, slots))
    assert got[0] is cache.k and got[1] is cache.v
    assert torch.equal(cache.k, want[0]) and torch.equal(cache.v, want[1])
    assert cpa.device_status() == 0


def test_cache_write_reports_slots_outside_the_cache():
    cache = Cache([100], [0], 2, 64, 16, torch.float16, fill=0.0)
    k = normal(3, 3, 2, 64, dtype=torch.float16)
    before, total = cache.k.clone(), cache.k.shape[0] * 16
    cpa.cache_write(k, k, cache.k, cache.v, ints([total, 2 ** 40, 5], torch.int64))
    assert cpa.device_status() == -1
    before[0, 5] = k[2]
    assert torch.equal(cache.k, before)


def tables_reference(ctx, new, table, free, P, num_slots):
    table, slots, at = table.clone(), [], 0
    for r, (c, n) in enumerate(zip(ctx, new)):
        have, need = -(-c // P), -(-(c + n) // P)
        for j in range(have, need):
            table[r, j] = free[at]
            at += 1
        slots += [int(table[r, p // P]) * P + p % P for p in range(c, c + n)]
    return table, slots + [-1] * (num_slots - len(slots)), offsets(new), at


@pytest.mark.parametrize("R,most,context,P,pad", [
    (1, 1, 0, 16, 0), (8, 1, 3000, 64, 8), (5, 700, 100, 16, 3), (1023, 3, 90, 32, 0),
    (1024, 5, 90, 16, 1), (2500, 9, 200, 16, 77), (3, 5000, 4000, 128, 0), (4, 0, 10, 16, 5),
    (60, 300, 500, 384, 0)])
def test_page_tables(R, most, context, P, pad):
    g = torch.Generator().manual_seed(R + most)
    ctx = torch.randint(0, context + 1, (R,), generator=g).tolist()
    new = torch.randint(0, most + 1, (R,), generator=g).tolist()
    have = [-(-c // P) for c in ctx]
    need = [-(-(c + n) // P) for c, n in zip(ctx, new)]
    width = max(need + [1]) + 1
    ids = torch.randperm(sum(need) + 9, generator=g, dtype=torch.int32)
    table = torch.full((R, width + 3), -5, dtype=torch.int32)
    first = offsets(have)
    for r, n in enumerate(have):
        table[r, :n] = ids[first[r]:first[r] + n]
    free = ids[sum(have):]
    total = sum(new) + pad
    want, wslots, wcu, wused = tables_reference(ctx, new, table, free.tolist(), P, total)
    dev_table = table.to(DEV)
    for _ in range(2):  # the same inputs give the same tables
        slots, cu, used = cpa.page_tables(ints(ctx), ints(new), dev_table[:, :width], free.to(DEV), P, total)
        assert slots.tolist() == wslots and cu.tolist() == wcu and used.item() == wused
        assert torch.equal(dev_table.cpu(), want)
    assert cpa.device_status() == 0


def test_page_tables_without_requests():
    none = ints([])
    slots, cu, used = cpa.page_tables(none, none, ints([]).reshape(0, 4), ints([1, 2]), 16, 5)
    assert slots.tolist() == [-1] * 5 and cu.tolist() == [0] and used.item() == 0
    assert cpa.device_status() == 0


def test_page_tables_reports_what_does_not_fit():
    def run(ctx, new, width, free, num_slots):
        table = torch.full((len(ctx), width + 1), -1, dtype=torch.int32, device=DEV)
        table[:, 0] = 40
        got = cpa.page_tables(ints(ctx), ints(new), table[:, :width], ints(free), 16, num_slots)
        assert cpa.device_status() == -1
        assert bool((table[:, width] == -1).all())
        return table, got
    # the pool runs out: the second request's second page is missing
    table, (slots, _, used) = run([16, 16], [16, 20], 3, [7, 8], 36)
    assert slots.tolist() == list(range(112, 128)) + list(range(128, 144)) + [-1] * 4
    assert used.item() == 3 and table[:, 1].tolist() == [7, 8]
    # the table is too narrow
    _, (slots, _, _) = run([16, 0], [20, 1], 2, [7, 8, 9], 21)
    assert slots.tolist() == list(range(112, 128)) + [-1] * 4 + [9 * 16]
    # more tokens than slots; a negative length; a missing old page
    run([0, 16], [5, 5], 3, [7, 8], 9)
    _, (slots, cu, _) = run([-3, 16], [5, 3], 3, [7, 8], 3)
    assert cu.tolist() == [0, 0, 3] and slots.tolist() == [112, 113, 114]
    run([20, 0], [3, 0], 3, [7, 8], 3)
    assert cpa.device_status() == 0


# ---------------------------------------------------------------------------
# used together
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", list(TYPES))
def test_prompt_then_cache_then_draft_then_next_token(dtype):
    """Prompts are answered, kept, extended by a drafted tree, of which one
    path is accepted, and by one more token: every step equals attention over
    the whole sequence."""
    H, Hkv, D, P, lens = 8, 2, 128, 16, [90, 5, 201]
    R, dt = len(lens), TYPES[dtype]
    drafts = 6
    table = torch.full((R, 40), -1, dtype=torch.int32, device=DEV)
    free = torch.arange(R * 20, dtype=torch.int32, device=DEV).flip(0).contiguous()
    kc, vc = (torch.full((R * 20, P, Hkv, D), math.nan, dtype=dt, device=DEV) for _ in range(2))
    x = normal(1, sum(lens), H + 2 * Hkv, D, dtype=dt)
    q, k, v = x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:]
    zero = ints([0] * R)
    slots, cu, used = cpa.page_tables(zero, ints(lens), table, free, P, sum(lens) + 4)
    cpa.cache_write(k, v, kc, vc, slots[:sum(lens)].contiguous())
    out, lse = cpa.prompt_attention(q, k, v, cu)
    o, l, to, tl = prompt_reference(q, k, v, lens, lens, True)
    check(out, o, to, "prompt")
    # a drafted tree: 0 - 1 - 2, 0 - 3, 4 - 5
    words = [0b1, 0b11, 0b111, 0b1001, 0b10000, 0b110000]
    free = free[used.item():].contiguous()
    y = normal(2, R * drafts, H + 2 * Hkv, D, dtype=dt)
    qd, kd, vd = y[:, :H], y[:, H:H + Hkv], y[:, H + Hkv:]
    slots, cu, used = cpa.page_tables(ints(lens), ints([drafts] * R), table, free, P, R * drafts)
    cpa.cache_write(kd, vd, kc, vc, slots)
    od, ld = cpa.tree_attention(qd, kc, vc, table, ints(lens), cu, ints(words * R, torch.int64))
    first = offsets(lens)
    keys, vals = [], []
    for r in range(R):
        a, b = slice(first[r], first[r + 1]), slice(r * drafts, (r + 1) * drafts)
        K, V = torch.cat([k[a], kd[b]]), torch.cat([v[a], vd[b]])
        seen = torch.ones(drafts, lens[r] + drafts, dtype=torch.bool, device=DEV)
        seen[:, lens[r]:] = torch.tensor([[bool(w >> j & 1) for j in range(drafts)] for w in words])
        o, l, to, tl = plain(qd[b], K, V, seen)
        check(od[b], o, to, "drafts")
        check(ld[:, b], l, tl, "drafts' lse")
        keys.append(K[:lens[r] + 3])  # the path 0 - 1 - 2 is accepted
        vals.append(V[:lens[r] + 3])
    # the next token overwrites a rejected draft's slot
    free = free[used.item():].contiguous()
    ctx = ints([n + 3 for n in lens])
    z = normal(3, R, H + 2 * Hkv, D, dtype=dt)
    slots, cu, _ = cpa.page_tables(ctx, ints([1] * R), table, free, P, R)
    cpa.cache_write(z[:, H:H + Hkv], z[:, H + Hkv:], kc, vc, slots)
    on, ln = cpa.tree_attention(z[:, :H], kc, vc, table, ctx, cu)
    for r in range(R):
        K = torch.cat([keys[r], z[r:r + 1, H:H + Hkv]])
        V = torch.cat([vals[r], z[r:r + 1, H + Hkv:]])
        o, l, to, tl = plain(z[r:r + 1, :H], K, V, torch.ones(1, K.shape[0], dtype=torch.bool, device=DEV))
        check(on[r:r + 1], o, to, "next token")
        check(ln[:, r:r + 1], l, tl, "next token's lse")
    assert cpa.device_status() == 0


def test_partials_of_two_caches_merge_as_ring_partials_do():
    """The lse of tree_attention joins with lse_merge: the cache split over two
    ranks gives the whole cache's result."""
    H, Hkv, D = 8, 2, 128
    whole = Cache([700], [1], Hkv, D, 64, torch.bfloat16)
    q = normal(9, 1, H, D, dtype=torch.bfloat16)
    parts = []
    for a, b in ((0, 300), (300, 701)):
        half = Cache([b - a - 1], [1], Hkv, D, 64, torch.bfloat16)
        pos = torch.arange(b - a, device=DEV)
        page = half.table[0].long()[pos // 64]
        half.k[page, pos % 64], half.v[page, pos % 64] = whole.K[0][a:b], whole.V[0][a:b]
        parts.append(run_tree(q, half))
    (oa, la), (ob, lb) = parts
    o, l = cpa.lse_merge(oa.float()[None], la[None].contiguous(), ob.float()[None], lb[None].contiguous())
    wo, wl, to, tl = tree_reference(q, whole)
    check(o[0], wo, 2 * to, "merged")
    check(l[0], wl, 2 * tl, "merged lse")


def test_two_captured_steps_replay_with_new_lengths():
    """A decoding step captured once replays on new lengths, tables and values;
    two graphs, each with its own workspace, replay at once on two streams."""
    H, Hkv, D, P, R = 8, 2, 128, 16, 3
    dt = torch.bfloat16

    class Step:
        def __init__(self, seed):
            self.table = torch.full((R, 40), -1, dtype=torch.int32, device=DEV)
            self.kc, self.vc = (normal(seed + i, 130, P, Hkv, D, dtype=dt) for i in range(2))
            self.ctx, self.new = ints([0] * R), ints([1] * R)
            self.free = torch.arange(130, dtype=torch.int32, device=DEV)
            self.x = normal(seed + 2, R, H + 2 * Hkv, D, dtype=dt)
            self.stream, self.graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
            with torch.cuda.stream(self.stream):
                self.run()
            self.stream.synchronize()
            with torch.cuda.graph(self.graph, stream=self.stream):
                self.run()

        def run(self):
            x = self.x
            slots, cu, _ = cpa.page_tables(self.ctx, self.new, self.table, self.free, P, R)
            cpa.cache_write(x[:, H:H + Hkv], x[:, H + Hkv:], self.kc, self.vc, slots)
            self.out, self.lse = cpa.tree_attention(x[:, :H], self.kc, self.vc, self.table, self.ctx, cu)
            self.po, _ = cpa.prompt_attention(x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:], cu)

        def set(self, seed, ctx):
            ids = torch.randperm(130, generator=torch.Generator().manual_seed(seed), dtype=torch.int32)
            self.table.copy_(ids[:120].reshape(R, 40))
            self.free.copy_(ids.flip(0))
            self.ctx.copy_(ints(ctx))
            self.x.copy_(normal(seed, *self.x.shape, dtype=dt))

        def check(self, ctx):
            for r, c in enumerate(ctx):
                pos = torch.arange(c + 1, device=DEV)
                page = self.table[r].long()[pos // P]
                o, l, to, tl = plain(self.x[r:r + 1, :H], self.kc[page, pos % P], self.vc[page, pos % P],
                                     torch.ones(1, c + 1, dtype=torch.bool, device=DEV))
                check(self.out[r:r + 1], o, to, "replayed out")
                check(self.lse[:, r:r + 1], l, tl, "replayed lse")
            v = self.x[:, H + Hkv:]
            assert torch.equal(self.po, v.repeat_interleave(H // Hkv, 1))  # one key: its value

    a, b = Step(1), Step(50)
    for seed, ca, cb in ((7, [5, 500, 33], [0, 1, 600]), (8, [600, 0, 128], [129, 16, 15])):
        a.set(seed, ca)
        b.set(seed + 100, cb)
        torch.cuda.synchronize()
        for _ in range(3):
            a.graph.replay()
            with torch.cuda.stream(b.stream):
                b.graph.replay()
        torch.cuda.synchronize()
        a.check(ca)
        b.check(cb)
    assert cpa.device_status() == 0


def test_a_planned_call_captured_once_replays_with_other_lengths():
    H, Hkv, D, R = 16, 8, 64, 130
    cu = ints([0] * (R + 1))
    q = normal(1, 4000, H, D, dtype=torch.float16)
    k, v = (normal(s, 4000, Hkv, D, dtype=torch.float16) for s in (2, 3))
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        cpa.prompt_attention(q, k, v, cu)
    stream.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        out, lse = cpa.prompt_attention(q, k, v, cu)
    for seed in range(3):
        g = torch.Generator().manual_seed(seed)
        lens = torch.randint(0, 31, (R,), generator=g).tolist()
        if seed == 1:
            lens = [0] * 100 + [133] * 30
        cu.copy_(ints(offsets(lens)))
        n = sum(lens)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        o, l, to, tl = prompt_reference(q[:n], k[:n], v[:n], lens, lens, True)
        check(out[:n], o, to, "out")
        check(lse[:, :n], l, tl, "lse")
    assert cpa.device_status() == 0


@pytest.mark.parametrize("wider", [1, 20000])  # small: CUDA cores; wide: tensor cores
def test_a_cache_whose_offsets_pass_32_bits(wider):
    # Pages 2^25 values apart: the last ones lie more than 2^32 bytes, and more
    # than 2^31 values, from the first.
    H, Hkv, D, P, pages, stride = 8, 2, 128, 16, 80, 1 << 25
    rows = P * Hkv * D
    buffers = [torch.empty((pages - 1) * stride + rows, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    kc, vc = (b.as_strided((pages, P, Hkv, D), (stride, Hkv * D, D, 1)) for b in buffers)
    ctx, new = [1200, 5], [1, 1]
    k, v = (normal(s, 1201 + 6, Hkv, D, dtype=torch.bfloat16) for s in (2, 3))
    ids = torch.randperm(pages, generator=torch.Generator().manual_seed(3), dtype=torch.int32)[:78].tolist()
    table = torch.full((2, 77 + wider), -1, dtype=torch.int32)
    table[0, :76], table[1, 0] = torch.tensor(ids[:76], dtype=torch.int32), ids[76]
    table = table.to(DEV)
    slots = torch.cat([table[r].long()[pos // P] * P + pos % P
                       for r, pos in enumerate((torch.arange(1201, device=DEV), torch.arange(6, device=DEV)))])
    cpa.cache_write(k, v, kc, vc, slots)
    q = normal(4, 2, H, D, dtype=torch.bfloat16)
    out, lse = cpa.tree_attention(q, kc, vc, table, ints(ctx), ints([0, 1, 2]))
    assert cpa.device_status() == 0
    for r, at in enumerate((slice(0, 1201), slice(1201, 1207))):
        n = at.stop - at.start
        o, l, to, tl = plain(q[r:r + 1], k[at], v[at], torch.ones(1, n, dtype=torch.bool, device=DEV))
        check(out[r:r + 1], o, to, "out")
        check(lse[:, r:r + 1], l, tl, "lse")


@pytest.mark.parametrize("ctx,new,H,Hkv,D,P", [([45000, 0, 30000], [16, 1, 3], 14, 2, 64, 256),
                                               ([87000], [1], 32, 8, 128, 16),
                                               ([2867] * 37, [1] * 37, 16, 16, 128, 64)])
def test_tree_results_do_not_depend_on_what_ran_before(ctx, new, H, Hkv, D, P):
    # Rows of a tile that no token fills hold whatever shared memory held.
    cache = Cache(ctx, new, Hkv, D, P, torch.bfloat16)
    q = normal(9, sum(new), H, D, dtype=torch.bfloat16)
    first = run_tree(q, cache)
    other = normal(8, 700, 8, 128, dtype=torch.bfloat16) * 50
    k = normal(4, 700, 2, 128, dtype=torch.bfloat16) * 50
    for n in range(6):
        cpa.prompt_attention(other[:700 - n], k[:700 - n], k[:700 - n], ints([0, 200, 700 - n]))
        big = Cache([300 + n] * 40, [30] * 40, 2, 128, 64, torch.bfloat16)
        run_tree(normal(n, 1200, 8, 128, dtype=torch.bfloat16) * 50, big)
        assert all(torch.equal(a, b) for a, b in zip(run_tree(q, cache), first))


def test_results_do_not_change_from_run_to_run():
    cache = Cache([5000, 33, 700], [7, 1, 12], 2, 128, 64, torch.bfloat16)
    q = normal(9, 20, 8, 128, dtype=torch.bfloat16)
    first = run_tree(q, cache)
    p = normal(3, 700, 8, 128, dtype=torch.bfloat16)
    k = normal(4, 700, 2, 128, dtype=torch.bfloat16)
    pfirst = cpa.prompt_attention(p, k, k, ints([0, 200, 700]))
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(run_tree(q, cache), first))
        assert all(torch.equal(a, b) for a, b in zip(cpa.prompt_attention(p, k, k, ints([0, 200, 700])), pfirst))
