"""What the binding of the rotary and cache calls hands on (no GPU needed: the launch is recorded instead)."""
import types

import numpy as np
import pytest
import torch

import context_causal_attention_zigzag_gb300 as cpa
from context_causal_attention_zigzag_gb300 import _binding

CPU = types.SimpleNamespace(index=-1)


@pytest.fixture
def launched(monkeypatch):
    calls = []
    monkeypatch.setattr(_binding, "_cuda_device", lambda t: CPU)
    monkeypatch.setattr(_binding, "_launch", lambda name, device, *args: calls.append((name, args)))
    monkeypatch.setattr(_binding, "_workspace", lambda given, device, need, *args: torch.empty(max(1, need(*args)), dtype=torch.uint8))
    return calls


def named(call):
    """The arguments by their names in include/cpattn.h."""
    names = {
        "cpattn_rotary": "x x_stride out out_stride B S_nat S H D rot interleaved freqs magnitude transposed positions "
                         "positions_stride offset cp_size layout from_sharded to_sharded dtype",
        "cpattn_cache_evict": "weights scores k_cache v_cache num_pages page_size page_stride token_stride head_stride "
                              "block_table table_width table_stride ctx_lens keep first recent most new_lens kept freed "
                              "num_freed_max num_freed R Hkv D dtype workspace workspace_bytes"}[call[0]].split()
    assert len(names) == len(call[1])
    return dict(zip(names, call[1]))


def turn(S=8, **kw):
    x = torch.zeros(2, S, 2, 64)
    return cpa.rotary(x, torch.ones(32, dtype=torch.float64), out=torch.zeros_like(x), **kw)


def evict(**kw):
    cache, i = torch.zeros(2, 2, 16, 2, 64, dtype=torch.bfloat16), torch.zeros(1, dtype=torch.int32)
    most = kw.pop("most", 4)
    outputs = tuple(torch.zeros(n, dtype=torch.int32) for n in (1, 8, 2, 1))
    return cpa.cache_evict(torch.zeros(2, 2, 16), cache[0], cache[1], torch.zeros(1, 2, dtype=torch.int32), i, i, most,
                           outputs=outputs, **kw)


@pytest.mark.parametrize("whole", [int, np.int32, np.int64, torch.tensor])
def test_integers_of_any_kind(launched, whole):
    turn(offset=whole(-70000), cp=whole(4), layout=whole(cpa.CONTIGUOUS), to_sharded=True)
    evict(first=whole(3), recent=whole(5), most=whole(4))
    one, two = (named(c) for c in launched)
    got = [one[n] for n in ("offset", "cp_size", "layout")] + [two[n] for n in ("first", "recent", "most")]
    assert got == [-70000, 4, 0, 3, 5, 4] and all(type(x) is int for x in got)


@pytest.mark.parametrize("bad", [None, "4", b"4", 4.0])
def test_what_is_no_integer_is_refused(launched, bad):
    for name in ("offset", "cp", "layout"):
        with pytest.raises(TypeError):
            turn(**{name: bad})
    for name in ("first", "recent"):
        with pytest.raises(TypeError):
            evict(**{name: bad})
    assert not launched


def test_integers_that_do_not_fit_are_refused(launched):
    for kw in (dict(offset=1 << 63), dict(offset=-(1 << 63) - 1), dict(cp=(1 << 32) + 1), dict(layout=1 << 32),
               dict(length=(1 << 32) + 8, to_sharded=True)):
        with pytest.raises(ValueError):
            turn(**kw)
    with pytest.raises(ValueError):
        evict(most=(1 << 32) + 4)
    assert not launched
    # Many first or recent positions mean all; fewer than none reach the library, which refuses them.
    evict(first=1 << 40, recent=1 << 31)
    evict(first=-(1 << 32), recent=-(1 << 40))
    assert [named(c)[n] for c in launched for n in ("first", "recent")] == [2**31 - 1] * 2 + [-1] * 2


@pytest.mark.parametrize("shape,stride", [((8,), 0), ((1, 8), 0), ((2, 8), 8)])
def test_positions_of_one_row_or_of_each_sequence(launched, shape, stride):
    turn(positions=torch.zeros(shape, dtype=torch.int32))
    assert named(launched[0])["positions_stride"] == stride


@pytest.mark.parametrize("shape", [(8, 1), (4, 2), (2, 4), (16,), (1, 16), (8, 2), (1, 1, 8), (2, 1, 8), (), (3, 8), (7,)])
def test_positions_of_another_shape_are_refused(launched, shape):
    with pytest.raises(ValueError):
        turn(positions=torch.zeros(shape, dtype=torch.int32))
    assert not launched
