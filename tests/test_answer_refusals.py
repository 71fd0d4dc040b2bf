"""Answering calls: what they refuse, before any launch (no GPU needed)."""
import ctypes

import pytest
import torch

import context_causal_attention_zigzag_gb300 as cp_attn
from context_causal_attention_zigzag_gb300 import _binding

E, U, W = _binding.ERR_INVALID_ARG, _binding.ERR_UNSUPPORTED, _binding.ERR_WORKSPACE
null, fake, odd = ctypes.c_void_p(0), ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1004)


def call(name, args, **changes):
    args = dict(args, **changes)
    return getattr(cp_attn.lib(), name)(*args.values())


TABLES = dict(ctx=fake, new=fake, R=2, P=16, free=fake, num_free=4, table=fake, width=4, stride=4,
              cu=fake, slots=fake, num_slots=8, used=fake, stream=null)
CACHE = dict(pages=8, P=16, ps=16 * 2 * 64, ts=2 * 64, hs=64)
WRITE = dict(k=fake, ks=128, v=fake, vs=128, slots=fake, N=4, kc=fake, vc=fake, **CACHE, Hkv=2, D=64,
             dtype=1, stream=null)
far = ctypes.c_void_p(0x10000)
TREE = dict(q=fake, qs=256, kc=fake, vc=fake, **CACHE, table=fake, width=4, stride=4, ctx=fake,
            cu=fake, tree=null, out=far, lse=fake, R=2, N=4, H=4, Hkv=2, D=64, dtype=1, scale=0.0,
            ws=fake, wb=1 << 30, stream=null)
PROMPT = dict(q=fake, qs=256, k=fake, ks=128, v=fake, vs=128, cu_q=fake, cu_k=fake, out=far,
              lse=fake, R=2, Nq=4, Nk=4, H=4, Hkv=2, D=64, causal=1, dtype=1, scale=0.0, ws=fake,
              wb=1 << 30, stream=null)


@pytest.mark.parametrize("changes", [
    dict(R=-1), dict(P=0), dict(P=24), dict(P=192), dict(P=2048), dict(num_free=-1), dict(width=-1),
    dict(stride=3), dict(num_slots=-1), dict(num_slots=1 << 31), dict(ctx=null), dict(new=null),
    dict(free=null), dict(table=null), dict(cu=null), dict(slots=null), dict(used=null),
    dict(slots=odd), dict(ctx=ctypes.c_void_p(0x1002))])
def test_page_tables_refuses(changes):
    assert call("cpattn_page_tables", TABLES, **changes) == E


BAD_CACHE = [dict(pages=0), dict(pages=1 << 28), dict(P=17), dict(ps=32), dict(ts=100), dict(hs=66),
             dict(hs=32), dict(ps=1 << 40), dict(kc=null), dict(vc=odd)]
BAD_HEADS = [dict(D=32), dict(D=96), dict(Hkv=0), dict(dtype=9), dict(dtype=0x11)]


@pytest.mark.parametrize("changes", BAD_CACHE + BAD_HEADS + [
    dict(N=-1), dict(N=1 << 31), dict(k=null), dict(v=odd), dict(slots=null), dict(slots=odd),
    dict(ks=127), dict(vs=120), dict(ks=1 << 40)])
def test_cache_write_refuses(changes):
    assert call("cpattn_cache_write", WRITE, **changes) == E


@pytest.mark.parametrize("changes", BAD_CACHE + BAD_HEADS + [
    dict(H=3), dict(H=0), dict(H=258, qs=258 * 64), dict(R=-1), dict(N=-1), dict(width=-1), dict(stride=2),
    dict(width=1 << 28, stride=1 << 28), dict(q=null), dict(qs=250), dict(out=odd), dict(lse=null),
    dict(table=null), dict(ctx=null), dict(cu=null), dict(tree=odd),
    dict(scale=float("nan")), dict(scale=float("inf"))])
def test_tree_attention_refuses(changes):
    assert call("cpattn_tree_attn", TREE, **changes) == E


@pytest.mark.parametrize("changes", BAD_HEADS + [
    dict(H=3), dict(R=-1), dict(Nq=-1), dict(Nk=-1), dict(causal=2), dict(q=null), dict(k=null),
    dict(v=odd), dict(qs=250), dict(ks=100), dict(vs=129), dict(cu_q=null), dict(cu_k=null),
    dict(out=null), dict(lse=null), dict(scale=float("nan"))])
def test_prompt_attention_refuses(changes):
    assert call("cpattn_prompt_attn", PROMPT, **changes) == E


def test_outputs_that_overlap_inputs_are_refused():
    big, end = ctypes.c_void_p(0x100000), ctypes.c_void_p(0x100000 + 2 * 3 * 256 + 2 * 4 * 64 - 16)
    assert call("cpattn_tree_attn", TREE, q=big, out=end) == E
    assert call("cpattn_tree_attn", TREE, q=big, out=big) == E
    for name, last in (("q", end), ("k", ctypes.c_void_p(0x100000 + 2 * 4 * 128 - 16)), ("v", big)):
        assert call("cpattn_prompt_attn", PROMPT, **{name: big, "out": last}) == E, name


def test_float32_is_unsupported():
    assert call("cpattn_cache_write", WRITE, dtype=0) == U
    assert call("cpattn_tree_attn", TREE, dtype=0) == U
    assert call("cpattn_prompt_attn", PROMPT, dtype=0) == U


def test_the_ring_calls_refuse_float16():
    fwd = cp_attn.lib().cpattn_ring_fwd
    assert fwd(*[fake] * 5, 1, 4, 2, 64, 64, 2, 1, 1, cp_attn.F16, 0.0, null) == E


def test_workspace_is_checked():
    lib = cp_attn.lib()
    need = lib.cpattn_tree_attn_workspace_bytes(4, 4, 2, 64)
    assert need > 0 and lib.cpattn_tree_attn_workspace_bytes(-1, 4, 2, 64) == 0
    for bad in (dict(ws=null), dict(ws=ctypes.c_void_p(0x1010)), dict(wb=need - 1)):
        assert call("cpattn_tree_attn", TREE, **bad) == W
    need = lib.cpattn_prompt_attn_workspace_bytes(2, 4, 4, 64)
    assert need > 0 and lib.cpattn_prompt_attn_workspace_bytes(-1, 4, 4, 64) == 0
    for bad in (dict(ws=null), dict(ws=ctypes.c_void_p(0x1010)), dict(wb=need - 1)):
        assert call("cpattn_prompt_attn", PROMPT, **bad) == W


def test_empty_calls_do_nothing():
    assert call("cpattn_cache_write", WRITE, N=0, k=null, v=null, slots=null) == 0
    assert call("cpattn_tree_attn", TREE, N=0, q=null, out=null, lse=null) == 0
    assert call("cpattn_tree_attn", TREE, R=0) == 0
    assert call("cpattn_prompt_attn", PROMPT, Nq=0, q=null, out=null, lse=null) == 0


def test_binding_refuses_host_tensors():
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        cp_attn.prompt_attention(x, x, x, i)
    with pytest.raises(ValueError):
        cp_attn.cache_write(x, x, x[None], x[None], i)
    with pytest.raises(ValueError):
        cp_attn.page_tables(i, i, i[None], i, 16, 8)
    with pytest.raises(ValueError):
        cp_attn.tree_attention(x, x[None], x[None], i[None], i, i)


@pytest.mark.parametrize("pages,heads", [(1, 2), (4, 1), (4, 2)])
def test_binding_refuses_caches_with_gaps_between_values(pages, heads):
    class Host:
        index = -1

    wide = torch.zeros(pages, 16, heads, 128, dtype=torch.float16)
    whole = torch.zeros(pages, 16, heads, 64, dtype=torch.float16)
    for k, v in ((wide[..., ::2], wide[..., ::2]), (whole, wide[..., ::2])):
        with pytest.raises(ValueError):
            _binding._cache_args(k, v, heads, 64, torch.float16, Host)
    assert _binding._cache_args(whole, whole, heads, 64, torch.float16, Host)[1] == 16


def test_sizes_whose_work_could_outlast_the_bounded_waits_are_refused():
    most = 1 << 20
    assert call("cpattn_tree_attn", TREE, R=most + 1) == E
    for P in (16, 128, 1024):
        width = (1 << 26) // P
        assert call("cpattn_tree_attn", TREE, P=P, width=width + 1, stride=width + 1) == E
        assert call("cpattn_tree_attn", TREE, P=P, width=width, stride=width, ws=null) == W
    assert call("cpattn_prompt_attn", PROMPT, R=most + 1) == E
    assert call("cpattn_prompt_attn", PROMPT, R=most, H=1024, Hkv=512, qs=1024 * 64, ks=512 * 64,
                vs=512 * 64) == E


def test_packed_rows_whose_items_could_outlast_the_bounded_waits_at_a_low_clock_are_refused():
    # 2^27 keys in one item take more than 2 s at 1.5 GHz.
    most, apart = 1 << 26, dict(out=ctypes.c_void_p(1 << 50), ws=null)
    for size in ("Nq", "Nk"):
        assert call("cpattn_prompt_attn", PROMPT, **{size: most + 1}, **apart) == E
    assert call("cpattn_prompt_attn", PROMPT, Nq=most, Nk=most, **apart) == W


def test_an_out_within_a_cache_is_refused():
    # 8 pages of 16 tokens, 2 heads of 64: 2 * 8 * 2048 bytes; out has 4 * 4 * 64 values.
    cache, size, out = 0x1000000, 2 * 8 * 2048, 2 * 4 * 4 * 64
    need = cp_attn.lib().cpattn_tree_attn_workspace_bytes(4, 4, 2, 64)
    for which in ("kc", "vc"):
        for at in (cache, cache + size - 16, cache + 4096, cache - out + 16):
            args = {which: ctypes.c_void_p(cache), "out": ctypes.c_void_p(at), "wb": need}
            assert call("cpattn_tree_attn", TREE, **args) == E, (which, at)


@pytest.mark.parametrize("out,lse", [((4, 6, 64), (4, 6)), ((24, 64), None), (None, (24,)), (None, (1, 6, 4))])
def test_binding_refuses_outputs_of_another_shape(out, lse):
    # lse is [H, N]: one of [N, H] would be filled in the other order.
    class Host:
        index = -1

    H, N, D = 6, 4, 64
    q = torch.zeros(N, H, D, dtype=torch.float16)
    right = torch.empty(N, H, D, dtype=torch.float16), torch.empty(H, N)
    assert all(a is b for a, b in zip(_binding._answer_outputs(q, N, H, D, *right, Host), right))
    wrong = (right[0] if out is None else torch.empty(out, dtype=torch.float16),
             right[1] if lse is None else torch.empty(lse))
    with pytest.raises(ValueError):
        _binding._answer_outputs(q, N, H, D, *wrong, Host)


def test_page_tables_of_more_requests_than_its_counters_hold_are_refused():
    # The kernel steps through the requests 1024 at a time in an int.
    for R in ((1 << 30) + 1, (1 << 31) - 1):
        assert call("cpattn_page_tables", TABLES, R=R) == E
