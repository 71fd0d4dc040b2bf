"""Rotary positions on the GPU against the definition in 64 bits.

Tolerances.  With c and s the float32 cosine and sine, off by at most d from the
true ones, a result m (a c - b s) is off by m (|a| + |b|) (d + 4 2^-24) (two
products, their sum and the magnitude's), and by half a step of its type.  d:
  - the angle, at most pi/4 after the split, is rounded to float32 (2^-24 pi/4), the
    phase cut at 2^-32 of a turn (2^-29 rad): 2^-23 together;
  - float32: sincospif is off by 2 units of 2^-24 at most; d = 2^-22 in all;
  - 16 bits: __sinf and __cosf are off by 2^-21.41 and 2^-21.19; d = 2^-20;
  - the frequency in turns and the angle of the definition in 64 bits are off by a
    few 2^-53 of the angle itself: |angle| 2^-50.
"""
import math

import pytest
import torch

import context_causal_attention_zigzag_gb300 as cpa

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def normal(seed, *shape, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(dtype).to(DEV)


def frequencies(rot, base=500000.0):
    return torch.tensor([base ** (-2 * i / rot) for i in range(rot // 2)], dtype=torch.float64, device=DEV)


def turned(x, at, freqs, interleaved=False, magnitude=1.0, transposed=False):
    """(y, tolerance) in 64 bits: x [.., tokens, H, D] at positions [.., tokens]."""
    rot = 2 * freqs.numel()
    y = x.double().clone()
    angle = at.double()[..., None] * freqs
    c, s = angle.cos()[..., None, :] * magnitude, angle.sin()[..., None, :] * magnitude
    s = -s if transposed else s
    one, two = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    a, b = y[..., one].clone(), y[..., two].clone()
    y[..., one], y[..., two] = a * c - b * s, a * s + b * c
    eps = torch.finfo(x.dtype).eps
    d = (2.0 ** -22 if x.dtype == torch.float32 else 2.0 ** -20) + angle.abs()[..., None, :] * 2.0 ** -50
    off = abs(magnitude) * (a.abs() + b.abs()) * (d + 2.0 ** -22)
    tol = torch.zeros_like(y)
    tol[..., one], tol[..., two] = off, off
    tiny = 2.0 ** -25 if x.dtype == torch.float16 else 0.0
    tol[..., :rot] += (eps / 2 * (y.abs() + tol) + tiny)[..., :rot]
    return y, tol


def check(got, want, tol, what=""):
    off = (got.double() - want).abs()
    assert not bool(torch.isnan(off).any()) and not bool((off > tol).any()), \
        f"{what} off by {off.max().item():.3e}, {(off - tol).max().item():.3e} over its bound"


SHAPES = [
    # B, S, H, D, rot
    (1, 1, 1, 8, 2), (1, 1, 32, 128, 128), (2, 5, 3, 64, 64), (1, 777, 8, 128, 64),
    (3, 33, 14, 64, 20), (1, 129, 5, 80, 80), (1, 40, 2, 256, 2), (1, 40, 2, 256, 254), (1, 70, 1, 24, 6),
    (2, 1000, 32, 128, 128), (1, 3, 500, 64, 32), (1, 20001, 2, 128, 96),
]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("B,S,H,D,rot", SHAPES)
def test_rotary_and_its_gradient(B, S, H, D, rot, interleaved, dtype):
    x, f = normal(1, B, S, H, D, dtype=TYPES[dtype]), frequencies(rot)
    g = torch.Generator().manual_seed(3)
    at = torch.randint(-1000, 2000000, (B, S), generator=g).int().to(DEV)
    y = cpa.rotary(x, f, at, interleaved=interleaved, magnitude=1.25)
    check(y, *turned(x, at, f, interleaved, 1.25), "forward")
    assert torch.equal(y[..., rot:], x[..., rot:])
    dx = cpa.rotary_bwd(x, f, at, interleaved=interleaved, magnitude=1.25)
    check(dx, *turned(x, at, f, interleaved, 1.25, True), "gradient")
    assert cpa.device_status() == 0


def test_gradient_against_differences_and_autograd():
    x, w, f = normal(1, 1, 9, 2, 64), normal(2, 1, 9, 2, 64), frequencies(48)
    at = torch.arange(9, device=DEV, dtype=torch.int32) * 1000
    got = cpa.rotary_bwd(w, f, at, magnitude=1.5)
    leaf = x.double().requires_grad_()
    angle = (at.double()[:, None] * f)[:, None]
    a, b = leaf[..., :24], leaf[..., 24:48]
    y = torch.cat([a * angle.cos() - b * angle.sin(), a * angle.sin() + b * angle.cos()], -1) * 1.5
    torch.cat([y, leaf[..., 48:]], -1).mul(w.double()).sum().backward()
    check(got, leaf.grad, turned(w, at, f, False, 1.5, True)[1])
    # <w, (R(x + h e) - R(x - h e)) / 2 h> for some e: R is linear, so h = 1 gives it but for roundings.
    for k in range(8):
        e = torch.zeros_like(x)
        e.view(-1)[k * 131] = 1
        d = (cpa.rotary(x + e, f, at, magnitude=1.5).double() - cpa.rotary(x - e, f, at, magnitude=1.5).double()) / 2
        assert abs(float((d * w.double()).sum() - got.double().view(-1)[k * 131])) < 64 * 2.0 ** -20 * 8


@pytest.mark.parametrize("layout", [cpa.ZIGZAG, cpa.CONTIGUOUS])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("cp", [1, 2, 5])
def test_into_and_out_of_the_ring(cp, layout, dtype):
    B, S, H, D = 2, 20 * cp, 3, 64
    x, f = normal(4, B, S, H, D, dtype=TYPES[dtype]), frequencies(D)
    at = torch.randint(0, 5000, (B, S), device=DEV, dtype=torch.int32)
    plain = cpa.rotary(x, f, at)
    inside = cpa.rotary(x, f, at, cp=cp, layout=layout, to_sharded=True)
    assert torch.equal(inside, cpa.zigzag_permute(plain, cp, layout))
    sharded = cpa.zigzag_permute(x, cp, layout)
    assert torch.equal(cpa.rotary(sharded, f, at, cp=cp, layout=layout, from_sharded=True), plain)
    assert torch.equal(cpa.rotary(sharded, f, at, cp=cp, layout=layout, from_sharded=True, to_sharded=True), inside)
    # One row of positions for all sequences, and none: offset + the natural position.
    row = cpa.rotary(x, f, at[0].contiguous(), cp=cp, layout=layout, to_sharded=True)
    assert torch.equal(row[0], inside[0])
    some = cpa.rotary(x, f, offset=70000, cp=cp, layout=layout, to_sharded=True)
    count = torch.arange(70000, 70000 + S, device=DEV, dtype=torch.int32)
    assert torch.equal(some, cpa.rotary(x, f, count, cp=cp, layout=layout, to_sharded=True))


def test_padding_on_the_way_in_and_out():
    cp, n, H, D = 2, 1001, 2, 128
    S = cpa.padded_length(n, cp)
    x, f = normal(5, 1, n, H, D, dtype=torch.bfloat16), frequencies(D)
    inside = cpa.rotary(x, f, cp=cp, to_sharded=True, length=S)
    assert torch.equal(inside, cpa.zigzag_permute_pad(cpa.rotary(x, f), cp, S))
    back = cpa.rotary_bwd(inside, f, cp=cp, from_sharded=True, length=n)
    assert torch.equal(back, cpa.rotary_bwd(cpa.rotary(x, f), f))
    assert torch.equal(cpa.rotary(x[:, :0], f, cp=cp, to_sharded=True, length=8),
                       torch.zeros(1, 8, H, D, device=DEV, dtype=torch.bfloat16))


def test_far_positions_and_the_scalings():
    at = torch.tensor([2**31 - 1, -2**31, 2**30 + 7, 0], dtype=torch.int32, device=DEV)
    x = normal(6, 4, 2, 64)
    for kind in (cpa.ROTARY_PLAIN, cpa.ROTARY_LINEAR, cpa.ROTARY_BASE, cpa.ROTARY_PARTS):
        f, m = cpa.rotary_frequencies(64, 10000.0, kind, 8.0, 4096.0)
        check(cpa.rotary(x, f, at, magnitude=m), *turned(x, at, f, magnitude=m))
    # Beyond 32 bits only through the offset.
    far = 1 << 40
    check(cpa.rotary(x, f, offset=far), *turned(x, torch.arange(far, far + 4, device=DEV), f))


def test_views_in_place_and_what_is_not_finite():
    H, Hkv, D, n = 4, 2, 64, 50
    f, at = frequencies(32), torch.arange(n, device=DEV, dtype=torch.int32)
    x = normal(7, n, H + 2 * Hkv, D, dtype=torch.bfloat16)
    want = cpa.rotary(x[:, :H].contiguous(), f, at)
    assert torch.equal(cpa.rotary(x[:, :H], f, at), want)
    y = x.clone()
    assert cpa.rotary(y[:, :H], f, at, out=y[:, :H]).data_ptr() == y.data_ptr()
    assert torch.equal(y[:, :H], want) and torch.equal(y[:, H:], x[:, H:])
    z = torch.full_like(x, 7)
    cpa.rotary(x[:, :H], f, at, out=z[:, 2:2 + H])
    assert torch.equal(z[:, 2:2 + H], want) and bool((z[:, :2] == 7).all()) and bool((z[:, 2 + H:] == 7).all())
    x[3, 0, 1], x[4, 1, 40], x[5, 1, 33] = math.nan, math.inf, math.nan
    y = cpa.rotary(x[:, :H], f, at)
    bad = torch.isnan(y)
    assert bad[3, 0, [1, 17]].all() and bad[5, 1, 33] and int(bad.sum()) == 3
    assert y[4, 1, 40] == math.inf


def check_write(n, H, Hkv, D, P, rot, interleaved, dtype, padded, fused=False, in_place=False, order="thd"):
    f = frequencies(rot)
    g = torch.Generator().manual_seed(n)
    pages = -(-n // P) + 2
    slots = torch.randperm(pages * P, generator=g)[:n].to(DEV)
    slots = torch.cat([slots, torch.full((padded,), -1, device=DEV)])
    at = torch.randint(0, 1000000, (n + padded,), generator=g).int().to(DEV)
    x = normal(8, n + padded, H + 2 * Hkv, D, dtype=TYPES[dtype])
    q, k, v = x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    if order == "htd":  # [pages, heads, tokens, D]
        cache = normal(9, 2, pages, Hkv, P, D, dtype=TYPES[dtype]).transpose(2, 3)
    else:  # keys and values by turns
        cache = normal(9, pages, 2, P, Hkv, D, dtype=TYPES[dtype]).transpose(0, 1)
    kc, vc = cache[0].clone(memory_format=torch.preserve_format), cache[1].clone(memory_format=torch.preserve_format)
    if order != "plain":
        kc, vc = cache[0], cache[1]
    before = kc.clone(), vc.clone()
    x0 = x.clone()
    qq, kk, vv = x0[:, :H], x0[:, H:H + Hkv], x0[:, H + Hkv:]
    out, kr, vr = cpa.rotary_cache_write(q, k, v, f, at, kc, vc, slots, interleaved=interleaved, magnitude=0.75,
                                         out=q if in_place else None)
    assert cpa.device_status() == 0
    check(out, *turned(qq, at, f, interleaved, 0.75), "q")
    page, i = slots[:n] // P, slots[:n] % P
    y, tol = turned(kk, at, f, interleaved, 0.75)
    check(kr[page, i], y[:n], tol[:n], "k")
    assert torch.equal(vr[page, i], vv[:n])
    rest = torch.ones(pages, P, dtype=torch.bool, device=DEV)
    rest[page, i] = False
    assert torch.equal(kr[rest], before[0][rest]) and torch.equal(vr[rest], before[1][rest])
    if fused and in_place:
        assert torch.equal(x[:, H:], x0[:, H:])


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("n,H,Hkv,D,P,rot,interleaved,padded", [
    (1, 32, 8, 128, 64, 128, False, 0), (64, 32, 8, 128, 64, 128, True, 3), (37, 14, 2, 64, 16, 20, False, 5),
    (700, 8, 1, 128, 256, 64, False, 1), (5000, 2, 2, 64, 32, 64, True, 0), (3, 128, 1, 64, 16, 6, False, 2)])
def test_rotary_cache_write(n, H, Hkv, D, P, rot, interleaved, padded, dtype):
    check_write(n, H, Hkv, D, P, rot, interleaved, dtype, padded)


@pytest.mark.parametrize("order", ["htd", "by turns"])
def test_rotary_cache_write_of_a_fused_projection_in_place(order):
    check_write(100, 8, 2, 128, 16, 128, False, "bf16", 4, fused=True, in_place=True, order=order)
    check_write(100, 8, 2, 128, 16, 64, True, "bf16", 4, fused=True, in_place=True, order=order)


def test_rotary_cache_write_skips_and_reports_slots_outside():
    f, x = frequencies(64), normal(10, 3, 2, 64, dtype=torch.bfloat16)
    cache = torch.zeros(2, 2, 16, 2, 64, device=DEV, dtype=torch.bfloat16)
    at = torch.zeros(3, dtype=torch.int32, device=DEV)
    out, kc, vc = cpa.rotary_cache_write(x, x, x, f, at, cache[0], cache[1],
                                         torch.tensor([1 << 40, 5, 32], device=DEV))
    assert cpa.device_status() == -1 and cpa.device_status() == 0
    assert torch.equal(out, x) and torch.equal(kc[0, 5], x[1]) and int((vc != 0).any(-1).any(-1).sum()) == 1


def test_other_streams_and_graphs():
    x, f = normal(11, 300, 4, 128, dtype=torch.bfloat16), frequencies(128)
    at = torch.arange(300, device=DEV, dtype=torch.int32)
    want = cpa.rotary(x, f, at)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = cpa.rotary(x, f, at)
    s.synchronize()
    assert torch.equal(got, want)
    out, graph = torch.empty_like(x), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cpa.rotary(x, f, at, out=out)
    at += 5
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, cpa.rotary(x, f, at))


@pytest.mark.parametrize("B,S_nat,S,H,Hkv,D,rot,cp,own", [(2, 90, 96, 4, 2, 64, 64, 4, False), (1, 61, 64, 2, 1, 128, 96, 2, True)])
def test_training_through_the_ring(B, S_nat, S, H, Hkv, D, rot, cp, own):
    """q and k turned into the ring's order, attention and its gradient there, the gradients turned back out,
    against the formula in 64 bits.  The ring's float32 results are held to 1e-4; inputs off by 2^-21 |x| (above)
    move scores by 2^-21 |q| |k| / sqrt(D), about 2^-21 sqrt(D) = 6e-6, and results by a few times that."""
    q, k, v, do = (normal(20 + i, B, S_nat, n, D) for i, n in enumerate((H, Hkv, Hkv, H)))
    freqs = frequencies(rot)
    at = torch.arange(S_nat, device=DEV, dtype=torch.int32).repeat(B, 1)
    if own:  # a second document's positions begin anew
        at[:, S_nat // 2:] -= S_nat // 2
    into, back = dict(cp=cp, to_sharded=True, length=S), dict(cp=cp, from_sharded=True, length=S_nat)
    qs, ks = cpa.rotary(q, freqs, at, **into), cpa.rotary(k, freqs, at, **into)
    vs, dos = cpa.zigzag_permute_pad(v, cp, S), cpa.zigzag_permute_pad(do, cp, S)
    o, lse = cpa.ring_fwd(qs, ks, vs, cp)
    dq, dk, dv = cpa.ring_bwd(qs, ks, vs, o, dos, lse, cp)
    got = (cpa.zigzag_unpermute(o, cp)[:, :S_nat], cpa.rotary_bwd(dq, freqs, at, **back),
           cpa.rotary_bwd(dk, freqs, at, **back), cpa.zigzag_unpermute(dv, cp)[:, :S_nat])
    x = [t.double().requires_grad_() for t in (q, k, v)]
    angle = (at.double()[..., None] * freqs)[:, :, None]

    def turn(t):
        a, b, rest = t.split([rot // 2, rot // 2, D - rot], -1)
        c, s = angle.cos(), angle.sin()
        return torch.cat([a * c - b * s, a * s + b * c, rest], -1).transpose(1, 2)
    qt, kt, vt = turn(x[0]), turn(x[1]), x[2].transpose(1, 2)
    kt, vt = (t.repeat_interleave(H // Hkv, 1) for t in (kt, vt))
    z = qt @ kt.transpose(2, 3) / math.sqrt(D)
    z = z.masked_fill(torch.ones(S_nat, S_nat, device=DEV, dtype=torch.bool).triu(1), -math.inf)
    want = (z.softmax(-1) @ vt).transpose(1, 2)
    for name, a, b in zip(("o", "dq", "dk", "dv"), got, (want,) + torch.autograd.grad(want, x, do.double())):
        assert float((a.detach().double() - b.detach()).abs().max()) <= 1.5e-4, name


def test_offsets_beyond_32_bits():
    S, H, D, cp = 600000, 32, 128, 4
    x, f = torch.empty(1, S, H, D, dtype=torch.bfloat16, device=DEV), frequencies(D)
    x[0, -100:] = normal(30, 100, H, D, dtype=torch.bfloat16)
    want = cpa.rotary(x[0, -100:].clone(), f, offset=S - 100)
    out = cpa.rotary(x, f, cp=cp, to_sharded=True)
    # The last chunk of the zigzag order is the second of rank 0.
    c = S // (2 * cp)
    assert torch.equal(out[0, 2 * c - 100:2 * c], want)
    assert torch.equal(cpa.rotary(x, f)[0, -100:], want)
