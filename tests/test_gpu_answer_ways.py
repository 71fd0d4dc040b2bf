"""Prompt attention on the GPU by the kernel that its sizes choose; test_answer_way
asserts without a GPU that these sizes choose it."""
import math

import pytest
import torch

import context_causal_attention_zigzag_gb300 as cpa
from test_gpu_answer import TYPES, check, ints, normal, offsets, prompt_reference

pytestmark = pytest.mark.gpu

# rows of q, sequences, H, Hkv, D: more items than SMs and more rows than a tile a sequence
PLANNED = [(4000, 20, 16, 8, 64), (4000, 20, 16, 8, 128), (5000, 30, 18, 6, 64)]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("N,R,H,Hkv,D", PLANNED)
def test_a_sorted_call_captured_once_replays_with_other_lengths(N, R, H, Hkv, D, dtype):
    cu = ints([0] * (R + 1))
    q = normal(1, N, H, D, dtype=TYPES[dtype])
    k, v = (normal(s, N, Hkv, D, dtype=TYPES[dtype]) for s in (2, 3))
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        cpa.prompt_attention(q, k, v, cu)
    stream.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        out, lse = cpa.prompt_attention(q, k, v, cu)
    g = torch.Generator().manual_seed(N)
    uneven = torch.randint(0, N // R, (R,), generator=g).tolist()
    for lens in (uneven, [0] * (R - 1) + [N], [N // R] * R, [0] * R, [1] * R, [0, N - 7] + [0] * (R - 3) + [7]):
        cu.copy_(ints(offsets(lens)))
        out.fill_(7.0)
        lse.fill_(7.0)
        n = sum(lens)
        torch.cuda.synchronize()
        graph.replay()
        graph.replay()  # the plan starts over
        torch.cuda.synchronize()
        o, l, to, tl = prompt_reference(q[:n], k[:n], v[:n], lens, lens, True)
        check(out[:n], o, to, "out")
        check(lse[:, :n], l, tl, "lse")
        assert bool((out[n:] == 7).all()) and bool((lse[:, n:] == 7).all())
    assert cpa.device_status() == 0


# nq, nk (None: nq), H, Hkv, D: the CUDA cores' kernel; sequences of SHARE keys and more
# are left to the cut line
SHARE = 32
SHARED = [
    ([400] + [1] * 63, None, 32, 8, 128),
    ([0] * 30 + [500] + [0] * 33, None, 32, 8, 64),
    ([3, 0, 1, 31, 32, 33, 2, 300, 1, 0] + [1] * 60, None, 32, 8, 128),
    ([1] * 256, [31, 32, 33, 0, 700] + [1] * 251, 32, 8, 128),
    ([5, 3] * 60 + [200, 40], [2, 3] * 60 + [20, 90], 12, 4, 128),    # some rows see nothing
    ([2, 1] * 60 + [200, 40], [2, 1] * 60 + [20, 300], 21, 3, 128),
    ([700] + [0] * 150, None, 32, 8, 64),
]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("nq,nk,H,Hkv,D", SHARED)
def test_uneven_batches_are_shared_between_two_kernels(nq, nk, H, Hkv, D, causal, dtype):
    nk, tail = nq if nk is None else nk, 3
    q = normal(1, sum(nq) + tail, H, D, dtype=TYPES[dtype])
    k, v = (normal(s, sum(nk), Hkv, D, dtype=TYPES[dtype]) for s in (2, 3))
    q[sum(nq):] = math.nan
    out, lse = torch.full_like(q, 7.0), torch.full((H, q.shape[0]), 7.0, device=q.device)
    cpa.prompt_attention(q, k, v, ints(offsets(nq)), ints(offsets(nk)), causal=causal, out=out, lse=lse)
    assert cpa.device_status() == 0
    n = sum(nq)
    o, l, to, tl = prompt_reference(q[:n], k, v, nq, nk, causal)
    check(out[:n], o, to, "out")
    check(lse[:, :n], l, tl, "lse")
    assert bool((out[n:] == 7).all()) and bool((lse[:, n:] == 7).all())


def test_shared_batches_replay_with_other_lengths_and_report_broken_offsets():
    H, Hkv, D, N, R = 32, 8, 128, 463, 64
    cu = ints(offsets([400] + [1] * 63))
    q = normal(1, N, H, D, dtype=torch.bfloat16)
    k, v = (normal(s, N, Hkv, D, dtype=torch.bfloat16) for s in (2, 3))
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        cpa.prompt_attention(q, k, v, cu)
    stream.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        out, lse = cpa.prompt_attention(q, k, v, cu)
    for lens in ([7] * 64, [0] * 63 + [463], [1] * 63 + [33], [31, 32] * 7 + [0] * 50, [0] * 64):
        cu.copy_(ints(offsets(lens)))
        out.fill_(7.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert cpa.device_status() == 0
        n = sum(lens)
        o, l, to, tl = prompt_reference(q[:n], k[:n], v[:n], lens, lens, True)
        check(out[:n], o, to, "out")
        check(lse[:, :n], l, tl, "lse")
        assert bool((out[n:] == 7).all())
    for broken in ([0, 400, 300] + [463] * 62, [0, 463, 0, 463] + [463] * 61, [2] + [463] * 64, [0] * 64 + [464]):
        cpa.prompt_attention(q, k, v, ints(broken))
        assert cpa.device_status() == -1, broken[:4]
    assert cpa.device_status() == 0
