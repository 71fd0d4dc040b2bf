"""Rotary and cache calls: limits and overlaps that they refuse before any launch, beside calls that
differ by little and pass the checks (no GPU needed: those answer anything but a refusal)."""
import ctypes

import pytest

import context_causal_attention_zigzag_gb300 as cp_attn
from context_causal_attention_zigzag_gb300 import _binding

E = _binding.ERR_INVALID_ARG
null = ctypes.c_void_p(0)
GB = 1 << 30


def at(x):
    return ctypes.c_void_p(x)


def call(name, args, **changes):
    assert not set(changes) - set(args)
    return getattr(cp_attn.lib(), name)(*dict(args, **changes).values())


CACHE = dict(pages=8, P=16, ps=16 * 2 * 64, ts=2 * 64, hs=64)
# N = 0 and R = 0 come back before a launch; other calls that pass the checks are not made where there is a GPU.
WEIGHTS = dict(q=at(1000 * GB), qs=128 * 64, kc=at(GB), **CACHE, table=at(2 * GB), width=4, stride=4, ctx=at(3 * GB),
               cu=at(4 * GB), tree=null, lse=at(2000 * GB), w=at(5 * GB), decay=1.0, R=2, N=4, H=4, Hkv=1, D=64, dtype=1,
               scale=0.0, ws=null, wb=0, stream=null)


@pytest.mark.parametrize("G", [1, 3, 4, 43, 64, 65, 128])
def test_rows_whose_tiles_outlast_the_waits(G):
    most = (128 // G) << 20
    args = dict(WEIGHTS, H=G)
    assert call("cpattn_cache_weights", args, N=most + 1) == E
    # (The workspace is looked at last: without one nothing is launched.)
    assert call("cpattn_cache_weights", args, N=most) == _binding.ERR_WORKSPACE


ROTARY = dict(x=at(GB), xs=256, out=at(2 * GB), os=384, B=2, S_nat=8, S=8, H=2, D=128, rot=128, inter=0,
              freqs=at(3 * GB), m=1.0, tr=0, pos=at(4 * GB), ps=8, off=0, cp=2, layout=1, frm=0, to=1, dtype=1, stream=null)
WRITE = dict(q=at(GB), qs=256, k=at(2 * GB), ks=128, v=at(3 * GB), vs=128, out=at(4 * GB), os=384, pos=at(5 * GB),
             slots=at(6 * GB), N=4, rot=64, inter=0, freqs=at(7 * GB), m=1.0, kc=at(8 * GB), vc=at(9 * GB), **CACHE, H=4,
             Hkv=2, D=64, dtype=1, stream=null)
CACHE_BYTES = 8 * 16 * 2 * 64 * 2


# out's rows are 512 bytes, 768 apart: 16 of them in the first, 4 in the second call.
@pytest.mark.parametrize("changes", [
    dict(pos=at(2 * GB)), dict(pos=at(2 * GB - 60)), dict(pos=at(2 * GB + 15 * 768 + 508)), dict(pos=at(2 * GB + 516), ps=100),
    dict(freqs=at(2 * GB + 768)), dict(freqs=at(2 * GB - 504)), dict(freqs=at(2 * GB + 700))])
def test_rotary_refuses_overlaps(changes):
    assert call("cpattn_rotary", ROTARY, **changes) == E


@pytest.mark.parametrize("changes", [
    dict(pos=at(4 * GB + 768)), dict(slots=at(4 * GB - 24)), dict(slots=at(4 * GB + 508 - 508 % 8)), dict(freqs=at(4 * GB)),
    dict(pos=at(8 * GB)), dict(pos=at(9 * GB + CACHE_BYTES - 4)), dict(slots=at(8 * GB - 8)), dict(freqs=at(9 * GB + 64)),
    dict(q=at(8 * GB)), dict(q=at(8 * GB - 16)), dict(k=at(9 * GB + CACHE_BYTES - 16)), dict(v=at(8 * GB + 4096)),
    dict(k=at(8 * GB)), dict(vc=at(8 * GB)), dict(vc=at(8 * GB + CACHE_BYTES // 8)), dict(vc=at(8 * GB - 128))])
def test_rotary_cache_write_refuses_overlaps(changes):
    assert call("cpattn_rotary_cache_write", WRITE, **changes) == E


EVICT = dict(w=at(GB), sc=null, kc=at(8 * GB), vc=at(9 * GB), **CACHE, table=at(2 * GB), width=4, stride=4, ctx=at(3 * GB),
             keep=at(3 * GB + 64), first=0, recent=0, most=10, new=at(4 * GB), kept=at(5 * GB), freed=at(6 * GB), room=8,
             count=at(7 * GB), R=2, Hkv=2, D=64, dtype=1, ws=null, wb=0, stream=null)
TOKEN, PAGE = 2 * 64, 16 * 2 * 64  # values


@pytest.mark.parametrize("strides,apart", [
    (dict(), 0), (dict(), 8), (dict(), PAGE - 8), (dict(), -PAGE), (dict(), 8 * PAGE - 8), (dict(), 56),
    (dict(ps=2 * PAGE), PAGE - 64), (dict(ps=2 * PAGE), 3 * PAGE + 8), (dict(ps=PAGE, hs=16 * 64, ts=64), 64),
    (dict(ps=2 * PAGE, ts=2 * TOKEN), TOKEN - 32), (dict(pages=1, ps=64), 3 * TOKEN), (dict(pages=1, ps=64, hs=16 * 64, ts=64), 64)])
def test_keys_and_values_that_share_elements(strides, apart):
    assert call("cpattn_cache_evict", EVICT, **strides, vc=at(8 * GB + 2 * apart)) == E


@pytest.mark.parametrize("strides,apart", [
    (dict(), 8 * PAGE), (dict(), -8 * PAGE), (dict(ps=2 * PAGE), PAGE), (dict(ps=2 * PAGE), -PAGE), (dict(ps=2 * PAGE), 5 * PAGE),
    (dict(ps=2 * PAGE, hs=16 * 64, ts=64), PAGE), (dict(ps=2 * PAGE, ts=2 * TOKEN), TOKEN),
    (dict(ps=2 * PAGE, ts=2 * TOKEN, hs=2 * 64), 64), (dict(ps=2 * PAGE, hs=2 * 16 * 64, ts=64), 16 * 64),
    (dict(hs=8 * PAGE, ps=16 * 64, ts=64), 8 * 16 * 64), (dict(pages=1, ps=64), 16 * TOKEN),
    (dict(ps=6 * PAGE), 5 * PAGE)])
def test_keys_and_values_side_by_side(strides, apart):
    assert call("cpattn_cache_evict", EVICT, **strides, vc=at(8 * GB + 2 * apart)) == _binding.ERR_WORKSPACE
