"""Runs one workload's forward (and backward) a few times: the program that
profiler captures (ncu) wrap.

    python -m context_causal_attention_zigzag_gb300.profile_case fwd_s32768
    python -m context_causal_attention_zigzag_gb300.profile_case bwd_s16384 [--onepass]
    python -m context_causal_attention_zigzag_gb300.profile_case bwd_s131072_g1
    python -m context_causal_attention_zigzag_gb300.profile_case docs_s16384 [--onepass]
    python -m context_causal_attention_zigzag_gb300.profile_case permute_s32768
    python -m context_causal_attention_zigzag_gb300.profile_case merge_s32768
    python -m context_causal_attention_zigzag_gb300.profile_case answer_step_batch [--time]

Cases are reduced versions of the named workloads (same heads, head dim and
layout; fewer tokens or batches) so that a full counter capture of one launch
stays small: a few hundred MB on the device and a few ms per launch.

The answer_* cases are calls on packed prompts and the paged cache at the sizes
that the documentation quotes; --time prints their device time, by CUDA events
around a graph of six calls on three inputs in turn, median of seven behind a
flush of L2.
"""
import argparse
import random

import torch

from . import _binding as cpa
from . import inputs

CASES = {
    # half of the S=32768 forward workload (one batch of two)
    "fwd_s32768": inputs.Workload("fwd_s32768", 1, 32, 8, 32768, 128, 8, cpa.ZIGZAG, True,
                                  torch.bfloat16, backward=False, seed=5),
    # the S=131072 forward+backward workload at S=16384 (1/64 of its tile pairs)
    "bwd_s16384": inputs.Workload("bwd_s16384", 1, 32, 8, 16384, 128, 4, cpa.ZIGZAG, True,
                                  torch.bfloat16, backward=True, seed=5),
    # one kv group of the S=131072 workload (4 query heads on 1 kv head): the
    # same per-head Q / dO working set as the full workload, 1/8 of its heads
    "bwd_s131072_g1": inputs.Workload("bwd_s131072_g1", 1, 4, 1, 131072, 128, 16, cpa.ZIGZAG,
                                      True, torch.bfloat16, backward=True, seed=5),
    # the packed-document workload reduced the same way (documents of mean
    # length 1024 instead of 8192)
    "docs_s16384": inputs.Workload("docs_s16384", 1, 32, 8, 16384, 128, 4, cpa.ZIGZAG, True,
                                   torch.bfloat16, backward=True, seed=5, doc_mean=1024,
                                   doc_seed=2006),
}


# The HBM-bound kernels on a query-sized tensor of the S=32768 shape (larger
# than L2): zigzag permute of a bf16 [1, 32768, 32, 128] tensor (256 MiB),
# LSE merge of two float32 partials of that shape (512 MiB each).
HBM_CASES = {"permute_s32768": (1, 32768, 32, 128, 8), "merge_s32768": (1, 32768, 32, 128, 8)}


def run_hbm(case: str, repeats: int) -> int:
    B, S, H, D, cp = HBM_CASES[case]
    dev = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device="cpu").manual_seed(6)
    if case.startswith("permute"):
        x = torch.randn((B, S, H, D), generator=g).to(torch.bfloat16).to(dev)
        y = torch.empty_like(x)
        for _ in range(repeats):
            cpa.zigzag_permute(x, cp, cpa.ZIGZAG, out=y)
    else:
        o_a = torch.randn((B, S, H, D), generator=g).to(dev)
        o_b = torch.randn((B, S, H, D), generator=g).to(dev)
        l_a = torch.randn((B, H, S), generator=g).to(dev)
        l_b = torch.randn((B, H, S), generator=g).to(dev)
        o_out, l_out = torch.empty_like(o_a), torch.empty_like(l_a)
        for _ in range(repeats):
            cpa.lse_merge(o_a, l_a, o_b, l_b, o_out, l_out)
    torch.cuda.synchronize()
    return cpa.device_status()


def _lens(seed, n, lo, hi):
    rng = random.Random(seed)
    return rng, [hi] + [rng.randint(lo, hi) for _ in range(n - 1)]


def _prompts(seed, n, lo, hi, prefix=0):
    """Rows of q and of k of n packed sequences."""
    rng, nq = _lens(seed, n, lo, hi)
    return nq, [x + (rng.randint(1, prefix) if prefix else 0) for x in nq]


def _cached(seed, n, lo, hi, few, most):
    """Cached positions and new tokens of n requests."""
    rng, ctx = _lens(seed, n, lo, hi)
    return ctx, [most] + [rng.randint(few, most) for _ in range(n - 1)]


_BF, _FP = torch.bfloat16, torch.float16
# name: (call, lengths, H, Hkv, D, dtype, more)
ANSWER_CASES = {
    "answer_prompt_short": ("prompt", _prompts(1, 1, 77, 77), 32, 8, 128, _BF, {}),
    "answer_prompts_packed": ("prompt", _prompts(2, 16, 100, 2000), 32, 8, 128, _BF, {}),
    "answer_prompts_packed_full": ("prompt", _prompts(2, 16, 100, 2000), 32, 8, 128, _BF,
                                   {"causal": False}),
    "answer_prompts_prefix": ("prompt", _prompts(3, 5, 33, 1025, 2500), 32, 8, 64, _FP, {}),
    "answer_prompt_long": ("prompt", _prompts(4, 1, 16384, 16384), 32, 8, 128, _BF, {}),
    "answer_prompt_long_d64": ("prompt", _prompts(4, 1, 16384, 16384), 32, 8, 64, _BF, {}),
    "answer_step_one": ("tree", _cached(5, 1, 1000, 1000, 1, 1), 32, 8, 128, _BF, {"page": 64}),
    "answer_step_batch": ("tree", _cached(6, 64, 100, 8192, 1, 1), 32, 8, 128, _BF, {"page": 64}),
    "answer_drafts": ("tree", _cached(7, 16, 500, 5000, 5, 31), 32, 8, 128, _FP,
                      {"page": 16, "tree": True}),
    "answer_long_cache": ("tree", _cached(8, 2, 100000, 131072, 6, 8), 32, 8, 128, _BF,
                          {"page": 128, "tree": True}),
    # the next 2048 tokens of a prompt, 8192 of it in the cache
    "answer_next_part": ("tree", ([8192], [2048]), 32, 8, 128, _BF, {"page": 64}),
    # a step of 63 single tokens and one part of a prompt
    "answer_mixed_step": ("tree", (_cached(9, 63, 100, 8192, 1, 1)[0] + [4096], [1] * 63 + [1024]),
                          32, 8, 128, _BF, {"page": 64}),
    "answer_write_step": ("write", 64, 32, 8, 128, _BF, {"page": 64}),
    "answer_write_prompt": ("write", 32001, 32, 8, 128, _BF, {"page": 64}),
    "answer_tables_step": ("tables", _cached(11, 8, 0, 3000, 1, 1), 0, 0, 0, None,
                           {"page": 64}),
    "answer_tables_queue": ("tables", _cached(12, 1000, 0, 500, 0, 700), 0, 0, 0, None, {"page": 16}),
}


def answer_call(case: str, seed: int):
    """One call of an answering case on inputs of its own, and what it has to move
    (bytes) and compute (flops)."""
    call, lens, H, Hkv, D, dtype, more = ANSWER_CASES[case]
    dev = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev).to(dtype)

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device=dev)

    def offsets(x):
        return ints([sum(x[:i]) for i in range(len(x) + 1)])

    def pages(n):
        return torch.randperm(n, generator=g, device=dev).int()

    P = more.get("page")
    if call == "prompt":
        nq, nk = lens
        causal = more.get("causal", True)
        q, k, v = normal(sum(nq), H, D), normal(sum(nk), Hkv, D), normal(sum(nk), Hkv, D)
        cq, ck, ws = offsets(nq), offsets(nk), cpa.prompt_attention_workspace(q, offsets(nq))
        out, lse = torch.empty_like(q), torch.empty(H, sum(nq), device=dev)
        pairs = sum(n * (m - n) + n * (n + 1) // 2 if causal else n * m for n, m in zip(nq, nk))
        return (lambda: cpa.prompt_attention(q, k, v, cq, ck, causal=causal, out=out, lse=lse, workspace=ws),
                2 * D * (2 * H * sum(nq) + 2 * Hkv * sum(nk)) + 4 * H * sum(nq), 4 * D * H * pairs)
    if call == "tree":
        ctx, new = lens
        need = [-(-(c + n) // P) for c, n in zip(ctx, new)]
        ids, table = pages(sum(need)), torch.full((len(ctx), max(need)), -1, dtype=torch.int32, device=dev)
        table[torch.arange(max(need), device=dev)[None] < ints(need)[:, None]] = ids
        q, k, v = normal(sum(new), H, D), normal(sum(need), P, Hkv, D), normal(sum(need), P, Hkv, D)
        cu, cl, ws = offsets(new), ints(ctx), cpa.tree_attention_workspace(q, k, offsets(new))
        out, lse, words = torch.empty_like(q), torch.empty(H, sum(new), device=dev), None
        if more.get("tree"):  # each drafted token's parent is the one half its number
            seen = {0: 1}
            for i in range(1, max(new)):
                seen[i] = seen[i // 2] | 1 << i
            words = torch.tensor([seen[i] for n in new for i in range(n)], device=dev)
        pairs = sum(n * c + n * (n + 1) // 2 for c, n in zip(ctx, new))
        return (lambda: cpa.tree_attention(q, k, v, table, cl, cu, words, out=out, lse=lse, workspace=ws),
                2 * D * (2 * H * sum(new) + 2 * Hkv * sum(ctx + new)) + 4 * H * sum(new), 4 * D * H * pairs)
    if call == "write":
        n = -(-lens // P) + 2
        k, v = normal(lens, Hkv, D), normal(lens, Hkv, D)
        kc, vc = normal(n, P, Hkv, D), normal(n, P, Hkv, D)
        slots = (pages(n).long()[:, None] * P + torch.arange(P, device=dev)).flatten()[:lens].contiguous()
        return lambda: cpa.cache_write(k, v, kc, vc, slots), 8 * lens * (Hkv * D + 1), 0
    ctx, new = lens
    have, need = [-(-c // P) for c in ctx], [-(-(c + n) // P) for c, n in zip(ctx, new)]
    ids, table = pages(sum(need)), torch.full((len(ctx), max(need)), -1, dtype=torch.int32, device=dev)
    table[torch.arange(max(need), device=dev)[None] < ints(have)[:, None]] = ids[:sum(have)]
    free, cl, nl, total = ids[sum(have):].contiguous(), ints(ctx), ints(new), sum(new)
    slots, cu, used = cpa.page_tables(cl, nl, table, free, P, total)
    return (lambda: cpa.page_tables(cl, nl, table, free, P, total, slots=slots, cu=cu, used=used),
            12 * len(ctx) + 8 * (sum(need) - sum(have)) + 8 * total, 0)


def run_answer(case: str, repeats: int, timed: bool) -> int:
    calls = [answer_call(case, seed) for seed in range(3)]
    for i in range(repeats):
        calls[i % 3][0]()
    torch.cuda.synchronize()
    if timed:
        for f, _, _ in calls:
            f()
        torch.cuda.synchronize()
        graph, n = torch.cuda.CUDAGraph(), 6
        with torch.cuda.graph(graph):
            for i in range(n):
                calls[i % 3][0]()
        flush = torch.empty(512 << 20, dtype=torch.uint8, device="cuda")
        for _ in range(3):
            graph.replay()
        us = []
        for _ in range(7):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            flush.zero_()
            a.record()
            graph.replay()
            b.record()
            torch.cuda.synchronize()
            us.append(a.elapsed_time(b) / n * 1e3)
        t = sorted(us)[3]
        print(f"{case}: {t:.1f} us, {calls[0][1] / t / 1e3:.0f} GB/s, {calls[0][2] / t / 1e6:.1f} TFLOP/s")
    return cpa.device_status()


def run(case: str, repeats: int = 3, onepass: bool = False, timed: bool = False) -> int:
    if case in HBM_CASES:
        return run_hbm(case, repeats)
    if case in ANSWER_CASES:
        return run_answer(case, repeats, timed)
    w = CASES[case]
    dev = torch.device("cuda", torch.cuda.current_device())
    q, k, v, do = (x.to(dev) if x is not None else None for x in inputs.generate(w))
    qs, ks, vs = (cpa.zigzag_permute(x, w.cp, w.layout) for x in (q, k, v))
    dos = cpa.zigzag_permute(do, w.cp, w.layout) if do is not None else None
    cu = w.doc_offsets()
    bounds = cpa.doc_bounds(cu, w.S) if cu is not None else None
    for _ in range(repeats):
        if bounds is None:
            o, lse = cpa.ring_fwd(qs, ks, vs, w.cp, w.layout, w.causal)
        else:
            o, lse = cpa.ring_fwd_docs(qs, ks, vs, w.cp, bounds, w.layout, w.causal)
        if dos is not None and bounds is None:
            cpa.ring_bwd(qs, ks, vs, o, dos, lse, w.cp, w.layout, w.causal,
                         grad_dtype=torch.float32, onepass=onepass)
        elif dos is not None:
            cpa.ring_bwd_docs(qs, ks, vs, o, dos, lse, w.cp, bounds, w.layout, w.causal,
                              grad_dtype=torch.float32, onepass=onepass)
    torch.cuda.synchronize()
    return cpa.device_status()


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("case", choices=sorted(CASES) + sorted(HBM_CASES) + sorted(ANSWER_CASES))
    ap.add_argument("--repeats", type=int, default=3)
    ap.add_argument("--onepass", action="store_true",
                    help="the one-pass backward (CPATTN_BWD_ONEPASS) instead of the two kernels")
    ap.add_argument("--time", action="store_true", help="print the device time (answer_* cases)")
    a = ap.parse_args()
    status = run(a.case, a.repeats, a.onepass, a.time)
    print(f"{a.case}: status {status}")
    raise SystemExit(0 if status == 0 else 1)


if __name__ == "__main__":
    main()
