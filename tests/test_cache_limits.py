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
