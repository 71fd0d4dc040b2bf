"""Rotary and cache calls: what they refuse before any launch, and the frequencies (no GPU needed)."""
import ctypes
import math

import pytest
import torch

import context_causal_attention_zigzag_gb300 as cp_attn
from context_causal_attention_zigzag_gb300 import _binding

E, U, W = _binding.ERR_INVALID_ARG, _binding.ERR_UNSUPPORTED, _binding.ERR_WORKSPACE
null, fake, odd = ctypes.c_void_p(0), ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1004)


def at(x):
    return ctypes.c_void_p(x)


def call(name, args, **changes):
    assert not set(changes) - set(args)
    return getattr(cp_attn.lib(), name)(*dict(args, **changes).values())


ROTARY = dict(x=fake, xs=256, out=at(0x100000), os=256, B=2, S_nat=8, S=8, H=2, D=128, rot=128, inter=0,
              freqs=fake, m=1.0, tr=0, pos=null, ps=0, off=0, cp=2, layout=1, frm=0, to=1, dtype=1, stream=null)
CACHE = dict(pages=8, P=16, ps=16 * 2 * 64, ts=2 * 64, hs=64)
WRITE = dict(q=at(0x400000), qs=256, k=at(0x500000), ks=128, v=at(0x600000), vs=128, out=at(0x700000), os=256,
             pos=fake, slots=fake, N=4, rot=64, inter=0, freqs=fake, m=1.0, kc=at(0x800000), vc=at(0x900000),
             **CACHE, H=4, Hkv=2, D=64, dtype=1, stream=null)
WEIGHTS = dict(q=at(0x400000), qs=256, kc=at(0x800000), **CACHE, table=fake, width=4, stride=4, ctx=fake, cu=fake,
               tree=null, lse=at(0x2000), w=at(0x500000), decay=1.0, R=2, N=4, H=4, Hkv=2, D=64, dtype=1, scale=0.0,
               ws=fake, wb=1 << 30, stream=null)
EVICT = dict(w=at(0x500000), sc=null, kc=at(0x800000), vc=at(0x900000), **CACHE, table=fake, width=4, stride=4,
             ctx=at(0x1000), keep=at(0x2000), first=0, recent=0, most=10, new=at(0x3000), kept=at(0x4000),
             freed=at(0x5000), room=8, count=at(0x6000), R=2, Hkv=2, D=64, dtype=1, ws=fake, wb=1 << 30, stream=null)
BAD_CACHE = [dict(pages=0), dict(pages=1 << 28), dict(P=17), dict(ps=32), dict(ts=100), dict(hs=66), dict(kc=null),
             dict(kc=odd)]
BAD_HEADS = [dict(D=32), dict(D=96), dict(Hkv=0), dict(dtype=9), dict(dtype=0x11)]
BAD_TURN = [dict(rot=0), dict(rot=3), dict(rot=130), dict(inter=2), dict(freqs=null), dict(freqs=odd),
            dict(m=float("nan")), dict(m=float("inf"))]


@pytest.mark.parametrize("changes", BAD_TURN + [
    dict(x=null), dict(x=odd), dict(out=odd), dict(xs=255), dict(xs=252), dict(os=260), dict(xs=1 << 40), dict(B=-1),
    dict(B=65536), dict(S_nat=9), dict(S_nat=-1), dict(S=(1 << 30) + 4), dict(S=6), dict(H=0), dict(H=70000),
    dict(D=0), dict(D=12), dict(D=264), dict(cp=0), dict(layout=2), dict(frm=2), dict(to=-1), dict(tr=2), dict(dtype=3),
    dict(dtype=0x11), dict(pos=odd, ps=4), dict(pos=at(0x1002)), dict(out=fake), dict(out=at(0x1000 + 512 * 15)),
    dict(out=fake, frm=0, to=1)])
def test_rotary_refuses(changes):
    assert call("cpattn_rotary", ROTARY, **changes) == E


def test_empty_calls_do_nothing():
    assert call("cpattn_rotary", ROTARY, B=0, x=null, out=null) == 0
    assert call("cpattn_rotary", ROTARY, S=0, S_nat=0, x=null, out=null) == 0
    assert call("cpattn_rotary_cache_write", WRITE, N=0, q=null, k=null, v=null, out=null, slots=null, pos=null) == 0
    assert call("cpattn_cache_weights", WEIGHTS, N=0, q=null, lse=null) == 0
    assert call("cpattn_cache_weights", WEIGHTS, R=0) == 0


@pytest.mark.parametrize("changes", BAD_CACHE + BAD_HEADS + BAD_TURN + [
    dict(vc=odd), dict(N=-1), dict(N=1 << 31), dict(q=null), dict(k=odd), dict(v=null), dict(out=null), dict(slots=odd),
    dict(slots=null), dict(pos=null), dict(pos=at(0x1002)), dict(qs=250), dict(ks=100), dict(vs=129), dict(os=128),
    dict(H=3), dict(out=at(0x500000)), dict(out=at(0x600000 + 128)), dict(out=at(0x800000)), dict(out=at(0x900010)),
    dict(out=at(0x400010)), dict(out=at(0x400000), os=264)])
def test_rotary_cache_write_refuses(changes):
    assert call("cpattn_rotary_cache_write", WRITE, **changes) == E


@pytest.mark.parametrize("changes", BAD_CACHE + BAD_HEADS + [
    dict(H=3), dict(H=0), dict(H=258, qs=258 * 64), dict(R=-1), dict(R=(1 << 20) + 1), dict(N=-1), dict(N=1 << 30),
    dict(width=-1), dict(stride=2), dict(width=1 << 28, stride=1 << 28), dict(q=null), dict(qs=250), dict(lse=null),
    dict(lse=at(0x2002)), dict(w=null), dict(w=at(0x500002)), dict(table=null), dict(ctx=null), dict(cu=null),
    dict(tree=odd), dict(scale=float("nan")), dict(decay=float("nan")), dict(decay=float("inf")),
    dict(w=at(0x400000)), dict(w=at(0x800000)), dict(w=at(0x2010))])
def test_cache_weights_refuses(changes):
    assert call("cpattn_cache_weights", WEIGHTS, **changes) == E


@pytest.mark.parametrize("changes", BAD_CACHE + BAD_HEADS + [
    dict(vc=odd), dict(R=-1), dict(R=65536), dict(width=-1), dict(stride=3), dict(first=-1), dict(recent=-1), dict(most=0),
    dict(most=(1 << 26) + 1), dict(room=-1), dict(w=null), dict(w=at(0x500002)), dict(sc=at(0x500002)),
    dict(sc=at(0x500100)), dict(table=null), dict(ctx=null), dict(keep=null), dict(new=null), dict(kept=null),
    dict(freed=null), dict(count=null), dict(new=at(0x1000)), dict(new=at(0x2004)), dict(kept=at(0x4002))])
def test_cache_evict_refuses(changes):
    assert call("cpattn_cache_evict", EVICT, **changes) == E


def test_types_and_workspaces():
    for name, args in (("cpattn_rotary_cache_write", WRITE), ("cpattn_cache_weights", WEIGHTS), ("cpattn_cache_evict", EVICT)):
        assert call(name, args, dtype=0) == U
    lib = cp_attn.lib()
    need = lib.cpattn_cache_evict_workspace_bytes(2, 2, 4, 16, 10)
    assert need > 0 and lib.cpattn_cache_evict_workspace_bytes(-1, 2, 4, 16, 10) == 0
    for bad in (dict(ws=null), dict(ws=at(0x1010)), dict(wb=need - 1)):
        assert call("cpattn_cache_evict", EVICT, **bad) == W
    assert lib.cpattn_cache_weights_workspace_bytes(-1, 4, 2, 64) == 0
    for bad in (dict(ws=null), dict(ws=at(0x1010))):
        assert call("cpattn_cache_weights", WEIGHTS, **bad) == W


def test_binding_refuses_what_does_not_fit():
    x, i = torch.zeros(4, 2, 64, dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int32)
    f, cache = torch.ones(32, dtype=torch.float64), torch.zeros(2, 16, 2, 64, dtype=torch.bfloat16)
    for fn in (lambda: cp_attn.rotary(x, f, i), lambda: cp_attn.rotary_bwd(x, f, i),
               lambda: cp_attn.rotary_cache_write(x, x, x, f, i, cache, cache, i.long()),
               lambda: cp_attn.cache_weights(x, cache, i[None], i[:1], i[:2], torch.zeros(2, 4), torch.zeros(2, 2, 16)),
               lambda: cp_attn.cache_evict(torch.zeros(2, 2, 16), cache, cache, i[None], i[:1], i[:1], 4)):
        with pytest.raises(ValueError):
            fn()


def test_frequencies():
    plain, one = cp_attn.rotary_frequencies(64, 500000.0, device="cpu")
    want = torch.tensor([500000.0 ** (-2 * i / 64) for i in range(32)], dtype=torch.float64)
    assert one == 1.0 and torch.allclose(plain, want, rtol=1e-14)
    linear, _ = cp_attn.rotary_frequencies(64, 500000.0, cp_attn.ROTARY_LINEAR, 4.0, device="cpu")
    assert torch.allclose(linear, want / 4, rtol=1e-14)
    # The slowest pair is slowed by the factor, the fastest not at all.
    base, _ = cp_attn.rotary_frequencies(64, 500000.0, cp_attn.ROTARY_BASE, 4.0, device="cpu")
    assert math.isclose(float(base[0]), 1.0) and math.isclose(float(base[-1]), float(want[-1]) / 4, rel_tol=1e-12)
    parts, m = cp_attn.rotary_frequencies(64, 500000.0, cp_attn.ROTARY_PARTS, 4.0, 8192.0, 1.0, 32.0, device="cpu")
    assert math.isclose(m, 0.1 * math.log(4) + 1)
    turns = 8192 * want / (2 * math.pi)
    g = ((turns - 1) / 31).clamp(0, 1)
    assert torch.allclose(parts, want * (1 - g) / 4 + want * g, rtol=1e-12)
    assert parts[0] == want[0] and math.isclose(float(parts[-1]), float(want[-1]) / 4, rel_tol=1e-12)


@pytest.mark.parametrize("args", [
    (0, 1e4, 0, 1.0, 0, 1, 32), (7, 1e4, 0, 1.0, 0, 1, 32), (64, 1.0, 0, 1.0, 0, 1, 32), (64, math.nan, 0, 1.0, 0, 1, 32),
    (64, 1e4, 4, 1.0, 0, 1, 32), (64, 1e4, -1, 1.0, 0, 1, 32), (64, 1e4, 1, 0.5, 0, 1, 32), (64, 1e4, 1, math.inf, 0, 1, 32),
    (2, 1e4, 2, 2.0, 0, 1, 32), (64, 1e4, 3, 2.0, 0, 1, 32), (64, 1e4, 3, 2.0, 4096, 32, 1), (64, 1e4, 3, 2.0, 4096, -1, 32)])
def test_frequencies_refuse(args):
    with pytest.raises(cp_attn.CpattnError):
        cp_attn.rotary_frequencies(*args, device="cpu")


# What is written (weights 1024 bytes, a cache 32768, lists of tens of bytes) at the end of, within or around
# something else.
@pytest.mark.parametrize("changes", [
    dict(w=at(0x7ffffc)), dict(w=at(0x807ffc)), dict(w=at(0x400600)), dict(w=at(0x1000)), dict(w=at(0xffc)),
    dict(tree=at(0x500018)), dict(w=at(0x10f000), ws=at(0x100000)), dict(ws=at(0x800000)), dict(ws=at(0x400000))])
def test_cache_weights_refuses_overlaps(changes):
    apart = dict(table=at(0x1000), ctx=at(0x1100), cu=at(0x1200), tree=at(0x1300), ws=at(0x100000))
    assert call("cpattn_cache_weights", WEIGHTS, **dict(apart, **changes)) == E


@pytest.mark.parametrize("changes", [
    dict(new=at(0x4000)), dict(kept=at(0x1f9c)), dict(kept=at(0x5000)), dict(freed=at(0x1004)), dict(freed=at(0x7014)),
    dict(count=at(0x4010)), dict(count=at(0x701c)), dict(w=at(0x7000)), dict(w=at(0x800000)), dict(sc=at(0x4ffc04)),
    dict(kept=at(0x807fe0)), dict(new=at(0x900000)), dict(table=at(0x800100)), dict(keep=at(0x907ff8)),
    dict(ws=at(0x4000)), dict(ws=at(0x1000)), dict(ws=at(0x500300)), dict(ws=at(0x900000)), dict(sc=at(0x900000))])
def test_cache_evict_refuses_overlaps(changes):
    apart = dict(table=at(0x7000), ws=at(0x100000))
    assert call("cpattn_cache_evict", EVICT, **dict(apart, **changes)) == E
