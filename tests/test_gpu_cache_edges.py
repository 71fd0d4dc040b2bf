"""Weights and eviction of cached positions: tables far wider than their requests, empty calls, and rows
of q that belong to no request or to another one."""
import math

import pytest
import torch

import context_causal_attention_zigzag_gb300 as cpa
from test_gpu_cache_evict import TYPES, ints, make, reference, same
from test_gpu_cache_weights_forms import FORMS, check, live_places
from test_gpu_cache_weights_forms import make as make_weights
from test_gpu_cache_weights_forms import reference as weights_reference

pytestmark = pytest.mark.gpu
DEV = "cuda"


def wide(table, width):
    out = torch.full((table.shape[0], width), -1, device=DEV, dtype=torch.int32)
    out[:, :table.shape[1]] = table
    return out


# Positions that the table has room for: one launch, a CTA, a cluster of 4, of 8, runs longer than shared memory.
@pytest.mark.parametrize("room", [2032, 12000, 40000, 131072, 1 << 20, 1 << 26])
@pytest.mark.parametrize("kind", ["plain", "ties", "equal", "wild"])
@pytest.mark.parametrize("ctx,keep,Hkv", [([900, 33, 0, 1, 500], [300, 32, 5, 0, 480], 2), ([1999], [77], 8)])
def test_eviction_with_tables_wider_than_requests(ctx, keep, Hkv, kind, room):
    P, most = 16, 500
    k, v, w, table = make(ctx, Hkv, 64, P, "bf16", kind=kind, seed=room)
    table = wide(table, room // P)
    want = reference(w, w, k, v, table, ctx, keep, 4, 30, most, table.numel())
    got = cpa.cache_evict(w, k, v, table, ints(ctx), ints(keep), most, first=4, recent=30)
    assert cpa.device_status() == 0
    for name, x, y in zip(("k", "v", "weights", "new_lens", "kept", "freed", "count"), (k, v, w) + got, want):
        assert same(x, y), f"{name}: {int((x != y).sum())} differ"


@pytest.mark.parametrize("width", [1, 3])
def test_eviction_of_no_request(width):
    k, v, w, _ = make([100], 2, 64, 16, "fp16")
    before = w.clone()
    none = torch.empty(0, device=DEV, dtype=torch.int32)
    table, freed = torch.empty(0, width, device=DEV, dtype=torch.int32), torch.zeros(5000, device=DEV, dtype=torch.int32)
    new_lens, kept, _, count = cpa.cache_evict_outputs(k, table, none, 7)
    cpa.cache_evict(w, k, v, table, none, none, 7, outputs=(new_lens, kept, freed, count))
    assert cpa.device_status() == 0 and int(count) == 0 and bool((freed == -1).all()) and torch.equal(w, before)


@pytest.mark.parametrize("form", list(FORMS) + ["few"])
@pytest.mark.parametrize("pages", [100, 5000])
def test_weights_with_tables_wider_than_requests(form, pages):
    few = ([130, 0, 64], [1, 2, 3], 4, 2, 64, 32)
    args = make_weights(*FORMS[form]) if form != "few" else small(*few)
    ctx, new = (FORMS[form] if form != "few" else few)[:2]
    q, k, table, c, cu, lse, weights = args
    want, tol = weights_reference(q, k, table, ctx, new, lse, weights)
    got = cpa.cache_weights(q, k, wide(table, pages), c, cu, lse, weights)
    assert cpa.device_status() == 0
    check(got, want, tol)


def small(ctx, new, H, Hkv, D, P):
    """Few rows: requests of the others, the first tokens alone."""
    q, k, table, c, cu, lse, weights = make_weights(ctx, [n + 20 for n in new], H, Hkv, D, P)
    n = sum(new)
    return q[:n], k, table, c, ints([sum(new[:i]) for i in range(len(new) + 1)]), lse[:, :n].contiguous(), weights


def test_few_rows_that_give_nothing_may_hold_anything():
    ctx, new, H, Hkv, D, P = [130, 0, 64], [1, 2, 3], 4, 2, 64, 32
    q, k, table, c, cu, lse, weights = small(ctx, new, H, Hkv, D, P)
    q, clean = q.clone(), q.clone()
    for h, i, value in ((0, 0, math.nan), (1, 2, math.inf), (3, 5, -math.inf)):
        lse[h, i] = -math.inf
        q[i, h, 3], clean[i, h] = value, 0
    want, tol = weights_reference(clean, k, table, ctx, new, lse, weights)
    check(cpa.cache_weights(q, k, table, c, cu, lse, weights), want, tol)


@pytest.mark.parametrize("form", list(FORMS))
def test_rows_of_another_request_stay_its_own(form):
    """Tiles of rows are loaded in boxes that reach into the next request's."""
    ctx, new = FORMS[form][:2]
    q, k, table, c, cu, lse, weights = make_weights(*FORMS[form])
    want, tol = weights_reference(q, k, table, ctx, new, lse, weights)
    last = max(r for r, n in enumerate(new) if n)
    q[sum(new) - new[last]:] = math.nan
    got = cpa.cache_weights(q, k, table, c, cu, lse, weights)
    alone = live_places(k, table, ctx, [n if r == last else 0 for r, n in enumerate(new)])
    got, want, tol = (x.transpose(1, 2) for x in (got, want, tol))
    check(got[~alone], want[~alone], tol[~alone])
    assert bool(torch.isnan(got[alone]).all())


def test_calls_without_tokens():
    f = torch.ones(32, dtype=torch.float64, device=DEV)
    for dtype in TYPES.values():
        x = torch.zeros(0, 2, 64, device=DEV, dtype=dtype)
        at, slots = (torch.empty(0, device=DEV, dtype=t) for t in (torch.int32, torch.int64))
        cache = torch.ones(2, 3, 16, 2, 64, device=DEV, dtype=dtype)
        assert cpa.rotary(x, f, at).shape == (0, 2, 64) and cpa.rotary_bwd(x[None], f).shape == (1, 0, 2, 64)
        out, kc, vc = cpa.rotary_cache_write(x, x, x, f, at, cache[0], cache[1], slots)
        assert out.shape == (0, 2, 64) and bool((cache == 1).all())
        w = torch.ones(3, 2, 16, device=DEV)
        table = torch.zeros(2, 1, device=DEV, dtype=torch.int32)
        cpa.cache_weights(x, kc, table, ints([5, 0]), ints([0, 0, 0]), torch.empty(2, 0, device=DEV), w)
        assert bool((w == 1).all())
    assert cpa.device_status() == 0
