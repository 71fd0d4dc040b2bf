"""Prompt attention on the GPU by the kernel that its sizes choose; test_answer_way
asserts without a GPU that these sizes choose it."""
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
