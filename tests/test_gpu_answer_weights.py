"""Softmax weights of the answering calls far below a row's best, on the GPU.

The tensor cores multiply weights rounded to the input type.  float16 has a
smallest step of 2^-24; the largest weight of a row is 2^7 at least, so a weight
is off by eps/2 of itself or 2^-25 / 2^7 = 2^-32 of the largest, and the sum of the
weights is no less than the largest: m keys are off by m 2^-32 max |v|.  The other
terms are those of test_gpu_answer; an output below 2^-14 is itself rounded to that
step, by 2^-25.
"""
import pytest
import torch

import context_causal_attention_zigzag_gb300 as cpa
from test_gpu_answer import DEV, TYPES, check, ints, normal, offsets, plain

pytestmark = pytest.mark.gpu


def tight(q, k, v, seen, scale=None):
    """plain() with the bound above for float16's step."""
    o, lse, to, tl = plain(q, k, v, seen, scale)
    if q.dtype == torch.float16:
        G, most = q.shape[1] // k.shape[1], v.double().abs().amax((0, 2))
        for h in range(q.shape[1]):
            to[:, h] += 2.0 ** -25 - k.shape[0] * (2.0 ** -25 - 2.0 ** -32) * most[h // G]
    return o, lse, to, tl


def weak_tail(m, Hkv, D, at, dtype):
    """Keys and values: one strong key whose value is 0, m - 1 keys 17 nats below it
    for the queries of strong_query (scale 1)."""
    k, v = torch.zeros(m, Hkv, D, dtype=dtype, device=DEV), normal(5, m, Hkv, D, dtype=dtype).abs() + 0.5
    k[at, :, 0], v[at] = 4.0, 0.0
    return k, v


def strong_query(n, H, D, dtype):
    q = torch.zeros(n, H, D, dtype=dtype, device=DEV)
    q[..., 0] = 4.25
    return q


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("at", [0, 7000])
@pytest.mark.parametrize("nq,nk,R,H,Hkv,D", [
    (600, 16384, 1, 64, 32, 128), (600, 16384, 1, 64, 32, 64), (300, 16384, 2, 30, 10, 64),  # two heads an item; one
    (1, 8192, 160, 4, 1, 64), (1, 8192, 160, 4, 1, 128)])                                  # cached-keys kernel
def test_many_weak_keys_behind_a_strong_one_in_a_prompt(nq, nk, R, H, Hkv, D, at, dtype):
    dt = TYPES[dtype]
    k, v = weak_tail(nk, Hkv, D, at, dt)
    q = strong_query(nq, H, D, dt)
    out, lse = cpa.prompt_attention(q.repeat(R, 1, 1), k.repeat(R, 1, 1), v.repeat(R, 1, 1),
                                    ints(offsets([nq] * R)), ints(offsets([nk] * R)), causal=False, scale=1.0)
    assert cpa.device_status() == 0
    o, l, to, tl = tight(q[:1], k, v, torch.ones(1, nk, dtype=torch.bool, device=DEV), 1.0)
    check(out, o.expand_as(out), to.expand_as(out), "out")
    check(lse, l.expand_as(lse), tl.expand_as(lse), "lse")


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("at", [0, 7000])
@pytest.mark.parametrize("new,R,H,Hkv,D", [(1, 300, 2, 1, 128), (1, 300, 2, 1, 64),
                                           (64, 160, 4, 1, 128), (64, 160, 4, 1, 64)])  # one row tile; two
def test_many_weak_keys_behind_a_strong_one_in_the_cache(new, R, H, Hkv, D, at, dtype):
    dt, P, m = TYPES[dtype], 64, 16384
    k, v = weak_tail(m, Hkv, D, at, dt)
    q = strong_query(new, H, D, dt)
    ids = torch.randperm(m // P, generator=torch.Generator().manual_seed(1)).to(DEV)
    kc, vc = (torch.empty(m // P, P, Hkv, D, dtype=dt, device=DEV) for _ in range(2))
    kc[ids], vc[ids] = k.view_as(kc), v.view_as(vc)
    table = ids.int()[None].repeat(R, 1)  # the same cache for every request
    out, lse = cpa.tree_attention(q.repeat(R, 1, 1), kc, vc, table, ints([m - new] * R),
                                  ints(offsets([new] * R)), scale=1.0)
    assert cpa.device_status() == 0
    i, j = torch.arange(new, device=DEV)[:, None], torch.arange(m, device=DEV)[None]
    o, l, to, tl = tight(q, k, v, j <= i + m - new, 1.0)
    check(out, o.repeat(R, 1, 1), to.repeat(R, 1, 1), "out")
    check(lse, l.repeat(1, R), tl.repeat(1, R), "lse")


@pytest.mark.parametrize("H,Hkv", [(64, 32), (48, 16)])
@pytest.mark.parametrize("D", [64, 128])
def test_scores_beyond_the_exact_integers_stay_finite(D, H, Hkv):
    # A score of 2^25 has a step of 4: a weight may come out far above its bound.
    dt = torch.float16
    q, k = normal(1, 600, H, D, dtype=dt) * 1000, normal(2, 600, Hkv, D, dtype=dt) * 1000
    v = normal(3, 600, Hkv, D, dtype=dt)
    out, lse = cpa.prompt_attention(q, k, v, ints([0, 600]), scale=4.0)
    assert bool(torch.isfinite(out).all()) and bool(torch.isfinite(lse).all())
    kc, vc = (x[:592].view(37, 16, Hkv, D) for x in (k, v))
    table = torch.arange(37, dtype=torch.int32, device=DEV)[None]
    out, lse = cpa.tree_attention(q[:100].contiguous(), kc, vc, table, ints([492]), ints([0, 100]), scale=4.0)
    assert bool(torch.isfinite(out).all()) and bool(torch.isfinite(lse).all())
    assert cpa.device_status() == 0
