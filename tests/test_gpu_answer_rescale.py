"""The running maximum of the answering calls on the GPU: rows whose best score
rises by more than the lazy maximum allows (8 in log2) at later key tiles, so that
the sum and O are corrected, next to rows whose scores fall, against the 64-bit
form.  Values shrink as the scores rise, so that what the early tiles gave still
counts in O."""
import pytest
import torch

import context_causal_attention_zigzag_gb300 as cpa
from test_gpu_answer import DEV, TYPES, check, ints, normal, offsets, signed, random_tree
from test_gpu_answer_weights import tight

pytestmark = pytest.mark.gpu

RISES = {"every tile": lambda t: t, "some tiles": lambda t: (t + 1) // 3, "late": lambda t: max(0, t - 4)}
STEP = 5.8  # 8.4 in log2


def stairs(seed, n, m, H, Hkv, D, dtype, rise):
    """q [n, H, D], k, v [m, Hkv, D]: scores (scale 1) that climb by STEP with the key
    tile for three rows of four, and fall for the fourth."""
    g = torch.Generator().manual_seed(seed)
    u = torch.zeros(D)
    u[[1, 17, 33, 60]] = 0.5
    sign = torch.where(torch.arange(n) % 4 == 3, -1.0, 1.0)[:, None, None]
    at = torch.tensor([float(rise(j // 128)) for j in range(m)])[:, None, None]
    q = torch.randn(n, H, D, generator=g) * 0.3 + sign * u
    k = torch.randn(m, Hkv, D, generator=g) * 0.3 + STEP * at * u
    v = torch.randn(m, Hkv, D, generator=g) * torch.exp(0.5 * (at.max() - at).clamp(max=12.0))
    return tuple(x.to(dtype).to(DEV) for x in (q, k, v))


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("rise", list(RISES))
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("nq,nk,H,Hkv,D", [
    ([300, 700], [1300, 1500], 64, 32, 128),          # two heads an item
    ([300, 700], [1300, 1500], 64, 32, 64),
    ([300, 700], [1300, 1500], 48, 16, 128),          # 256 rows an item
    ([300, 700], [1300, 1500], 48, 16, 64),
    ([1500], [1500], 64, 32, 64),                     # one sequence, unequal tile counts
    ([1500], [1500], 48, 16, 64),
    ([640], [640], 8, 4, 64),                         # an item a CTA
    ([640], [640], 8, 4, 128),
    ([3, 40], [1300, 1500], 4, 2, 64),                # the cached-keys kernel, items cut
    ([3, 40], [1300, 1500], 4, 2, 128),
    ([2] * 150, [1300] * 150, 4, 2, 128),             # and most of them whole
])
def test_rising_scores_in_prompts(nq, nk, H, Hkv, D, causal, rise, dtype):
    parts = [stairs(r % 2, n, m, H, Hkv, D, TYPES[dtype], RISES[rise]) for r, (n, m) in enumerate(zip(nq, nk))]
    q, k, v = (torch.cat(x) for x in zip(*parts))
    out, lse = cpa.prompt_attention(q, k, v, ints(offsets(nq)), ints(offsets(nk)), causal=causal, scale=1.0)
    assert cpa.device_status() == 0
    first, done = offsets(nq), {}
    for r, (n, m) in enumerate(zip(nq, nk)):
        if (r % 2, n, m) not in done:
            i, j = torch.arange(n, device=DEV)[:, None], torch.arange(m, device=DEV)[None]
            seen = (j <= i + m - n) if causal else torch.ones(n, m, dtype=torch.bool, device=DEV)
            done[r % 2, n, m] = tight(*parts[r], seen, 1.0)
        o, l, to, tl = done[r % 2, n, m]
        at = slice(first[r], first[r + 1])
        check(out[at], o, to, "out")
        check(lse[:, at], l, tl, "lse")


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("rise", list(RISES))
@pytest.mark.parametrize("ctx,new,H,Hkv,D,P,tree", [
    ([2000, 1200], [3, 9], 8, 2, 128, 16, True),      # one row tile, items cut
    ([2000, 1200], [3, 9], 8, 2, 64, 64, False),
    ([1900, 1200], [64, 40], 16, 2, 128, 32, True),   # two row tiles, items cut
    ([1900, 1200], [300, 200], 4, 2, 64, 128, False),
    ([1600, 900] * 50, [1, 6] * 50, 8, 4, 128, 64, True),   # whole items
    ([1600, 900] * 50, [64, 30] * 50, 16, 4, 64, 64, True),
    ([1600, 900] * 50, [70, 64] * 50, 16, 4, 128, 256, False),
])
def test_rising_scores_in_the_cache(ctx, new, H, Hkv, D, P, tree, rise, dtype):
    dt = TYPES[dtype]
    kinds = [stairs(r, new[r], ctx[r] + new[r], H, Hkv, D, dt, RISES[rise]) for r in range(2)]
    words = [random_tree(r, new[r]) for r in range(2)]
    need = [-(-(c + n) // P) for c, n in zip(ctx, new)]
    ids = torch.randperm(sum(need), generator=torch.Generator().manual_seed(2), dtype=torch.int32).to(DEV)
    kc, vc = (normal(s, sum(need), P, Hkv, D, dtype=dt) for s in (7, 8))
    table = torch.full((len(ctx), max(need) + 1), -7, dtype=torch.int32, device=DEV)
    first = offsets(need)
    for r, (c, n) in enumerate(zip(ctx, new)):
        table[r, :need[r]] = ids[first[r]:first[r + 1]]
        pos = torch.arange(c + n, device=DEV)
        page = table[r].long()[pos // P]
        kc[page, pos % P], vc[page, pos % P] = kinds[r % 2][1:]
    q = torch.cat([kinds[r % 2][0] for r in range(len(ctx))])
    bits = ints(signed(sum((words[r % 2] for r in range(len(ctx))), [])), torch.int64) if tree else None
    out, lse = cpa.tree_attention(q, kc, vc, table, ints(ctx), ints(offsets(new)), bits, scale=1.0)
    assert cpa.device_status() == 0
    want = []
    for r in range(2):
        c, n = ctx[r], new[r]
        seen = torch.ones(n, c + n, dtype=torch.bool)
        for i in range(n):
            w = words[r][i] if tree else (1 << (i + 1)) - 1
            seen[i, c:] = torch.tensor([bool(w >> j & 1) for j in range(n)])
        want.append(tight(*kinds[r], seen.to(DEV), 1.0))
    first = offsets(new)
    for r in range(len(ctx)):
        o, l, to, tl = want[r % 2]
        at = slice(first[r], first[r + 1])
        check(out[at], o, to, "out")
        check(lse[:, at], l, tl, "lse")
