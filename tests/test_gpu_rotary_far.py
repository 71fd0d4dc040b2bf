"""Rotary angles of far positions against decimal arithmetic.

Tolerances are those of the near positions: cosine and sine off by 2^-22 (float32) or 2^-20 (16 bits), and
the products, their sum and the magnitude by 2^-22 of |a| + |b|; then half a step of the type.  A frequency
is held to half a unit of 2^-64 of a turn, so a position p adds |p| 2^-65 of a turn, |p| 2^-62."""
import decimal
import math

import pytest
import torch

import context_causal_attention_zigzag_gb300 as cpa

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
TWO_PI = 2 * decimal.Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")


def angles(freqs, positions):
    """p f without its whole turns, float64 [positions, freqs]."""
    with decimal.localcontext(decimal.Context(prec=80)):
        return torch.tensor([[float((decimal.Decimal(f) * p).remainder_near(TWO_PI)) for f in freqs.tolist()]
                             for p in positions], dtype=torch.float64, device=DEV)


def check(y, x, freqs, positions):
    """x, y [tokens, H, D], all values of a head in pairs half a head apart."""
    a, b = x.double().chunk(2, -1)
    angle = angles(freqs, positions)[:, None]
    want = torch.cat([a * angle.cos() - b * angle.sin(), a * angle.sin() + b * angle.cos()], -1)
    far = torch.tensor([abs(p) * 2.0 ** -62 for p in positions], dtype=torch.float64, device=DEV)[:, None, None]
    d = (2.0 ** -22 if x.dtype == torch.float32 else 2.0 ** -20) + far + 2.0 ** -22
    tol = (d * (a.abs() + b.abs())).repeat(1, 1, 2)
    tol = tol + torch.finfo(x.dtype).eps / 2 * (want.abs() + tol) + (2.0 ** -25 if x.dtype == torch.float16 else 0.0)
    off = (y.double() - want).abs()
    assert not bool((off > tol).any()), f"off by {off.max().item():.3e}, {(off - tol).max().item():.3e} over its bound"


def inputs(n, dtype):
    g = torch.Generator().manual_seed(n)
    return torch.randn(n, 3, 64, generator=g).to(TYPES[dtype]).to(DEV)


def frequencies(kind):
    if kind == "wide":  # of either sign, from none to many turns a position
        return torch.tensor([0.0, 1.0, -1.0, 0.5, 3.0, -2.5, math.pi, 2 * math.pi, 100.25, -1000.0, 1e-6, -1e-9, 1e-15, 0.1]
                            + [0.7 ** i for i in range(18)], dtype=torch.float64, device=DEV)
    return cpa.rotary_frequencies(64, 500000.0, kind, 8.0, 4096.0)[0]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("kind", [cpa.ROTARY_PLAIN, cpa.ROTARY_PARTS, "wide"])
def test_positions_of_32_bits(kind, dtype):
    positions = [2**31 - 1, -2**31, 2**31 - 12345, 2**30 + 7, -2**29 - 1, 123456789, 10**6 + 1, 1, 0, -1]
    x, f = inputs(len(positions), dtype), frequencies(kind)
    at = torch.tensor(positions, dtype=torch.int32, device=DEV)
    check(cpa.rotary(x, f, at), x, f, positions)
    check(cpa.rotary_bwd(x, f, at), x, f, [-p for p in positions])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("offset", [2**32, 2**40 + 3, -2**40, 2**44 + 1])
def test_offsets_beyond_32_bits(offset, dtype):
    x, f = inputs(40, dtype), frequencies(cpa.ROTARY_PLAIN)
    check(cpa.rotary(x, f, offset=offset), x, f, range(offset, offset + 40))


def test_keys_on_their_way_into_the_cache():
    positions = [2**31 - 1, -2**31, 2**30 + 7, 10**6 + 1]
    x, f = inputs(4, "fp16"), frequencies(cpa.ROTARY_PLAIN)
    cache = torch.zeros(2, 1, 16, 3, 64, device=DEV, dtype=torch.float16)
    at, slots = torch.tensor(positions, dtype=torch.int32, device=DEV), torch.tensor([3, 0, 7, 9], device=DEV)
    out, kc, _ = cpa.rotary_cache_write(x, x.clone(), x, f, at, cache[0], cache[1], slots)
    check(out, x, f, positions)
    check(kc[0, slots], x, f, positions)
