"""Cases, plain forms and exact values of the operators around long-context
attention: rotary positions (alone, and with the write into the paged cache),
the attention weight that cached positions gather, and the eviction of the
lightest of them.

A case's lengths follow from the case alone (its "mix" number), its tensors
from the seed alone.
"""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
# (query heads, kv heads, head dim): the repository's grouped and plain layouts,
# and generic multi-query and odd-group ones.
HEADS = [(32, 8, 128), (16, 16, 128), (2, 2, 64), (8, 1, 128), (14, 2, 64), (32, 8, 64)]
PAGES = [16, 32, 64, 128, 256]


def listed():
    return [
        # The queries of a long training sequence on their way into the ring: rotated and
        # brought into the ranks' order in one pass.
        dict(name="rotary_train_into_ring", op="rotary", B=1, S=131072, H=32, D=128, rot=128,
             interleaved=False, cp=16, way="in", bwd=False, docs=0, far=0, dtype="bf16", mix=1),
        # Their float32 gradients on the way out, packed documents of uneven length.
        dict(name="rotary_grads_out_of_ring_fp32", op="rotary", B=2, S=16384, H=32, D=128, rot=128,
             interleaved=False, cp=4, way="out", bwd=True, docs=9, far=0, dtype="fp32", mix=2),
        # A short prompt behind a very long context, half of each head rotated, pairs side by side.
        dict(name="rotary_short_far_fp16", op="rotary", B=1, S=777, H=8, D=128, rot=64,
             interleaved=True, cp=1, way="keep", bwd=False, docs=0, far=1000000, dtype="fp16", mix=3),
        # One decoding step of a busy server: queries, keys and values of its tokens.
        dict(name="rotary_write_one_step", op="write", tokens=64, padded=3, rot=128, interleaved=False,
             page=64, H=32, Hkv=8, D=128, dtype="bf16", mix=4),
        # Those of a long packed prompt.
        dict(name="rotary_write_prompt", op="write", tokens=32001, padded=0, rot=128,
             interleaved=False, page=64, H=32, Hkv=8, D=128, dtype="bf16", mix=5),
        # What one user's new token looked at: latency.
        dict(name="weights_one_user", op="weights", reqs=1, shortest=1000, longest=1000, fewest=1,
             most=1, tree=False, decay=1.0, page=64, H=32, Hkv=8, D=128, dtype="bf16", mix=6),
        # The same for a busy server, contexts of all lengths.
        dict(name="weights_one_token_batch", op="weights", reqs=64, shortest=100, longest=8192,
             fewest=1, most=1, tree=False, decay=0.98, page=64, H=32, Hkv=8, D=128, dtype="bf16",
             mix=7),
        # A batch of prompts of uneven length just taken in; 64-wide heads.
        dict(name="weights_prompts_mixed_fp16", op="weights", reqs=16, shortest=0, longest=0,
             fewest=100, most=2000, tree=False, decay=1.0, page=16, H=32, Hkv=8, D=64, dtype="fp16",
             mix=8),
        # One long document just taken in.
        dict(name="weights_long_document", op="weights", reqs=1, shortest=0, longest=0, fewest=16384,
             most=16384, tree=False, decay=1.0, page=128, H=32, Hkv=8, D=128, dtype="bf16", mix=9),
        # One user's cache is brought back under its limit.
        dict(name="evict_one_user", op="evict", reqs=1, shortest=1100, longest=1100, share=0.9,
             first=4, recent=128, page=64, H=32, Hkv=8, D=128, dtype="bf16", mix=10),
        # Those of a busy server, half of each kept.
        dict(name="evict_batch", op="evict", reqs=16, shortest=1000, longest=8192, share=0.5, first=4,
             recent=256, page=64, H=32, Hkv=8, D=128, dtype="bf16", mix=11),
        # A long document after its prompt: an eighth stays.
        dict(name="evict_long_document", op="evict", reqs=1, shortest=131072, longest=131072,
             share=0.125, first=4, recent=1000, page=128, H=32, Hkv=8, D=128, dtype="bf16", mix=12),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)) - 1e-9)))))


def draw(rng):
    op = rng.choice(["rotary", "write", "weights", "weights", "evict"])
    H, Hkv, D = rng.choice(HEADS)
    mix, dtype = rng.randrange(1 << 30), rng.choice(["bf16", "fp16"])
    rot, interleaved = rng.choice([D, D, D // 2, D // 4, 20]), rng.choice([False, True])
    if op == "rotary":
        dtype = rng.choice(list(TYPES))
        B, cp, way = rng.choice([1, 1, 2, 3]), rng.choice([2, 4, 16]), rng.choice(["keep", "in", "out"])
        S = _log(rng, 1, (131072 * 32 * 128 // (H * D * B)) // (2 if dtype == "fp32" else 1) // 4)
        S = S if way == "keep" else -(-S // (2 * cp)) * 2 * cp
        return dict(op=op, B=B, S=S, H=H, D=D, rot=rot, interleaved=interleaved,
                    cp=1 if way == "keep" else cp, way=way, bwd=rng.choice([False, True]),
                    docs=rng.choice([0, 0, min(S, 7)]), far=rng.choice([0, 0, 1000000]), dtype=dtype,
                    mix=mix)
    if op == "write":
        return dict(op=op, tokens=_log(rng, 1, 32001), padded=rng.choice([0, 5]), rot=rot,
                    interleaved=interleaved, page=rng.choice(PAGES), H=H, Hkv=Hkv, D=D, dtype=dtype,
                    mix=mix)
    page = rng.choice(PAGES)
    if op == "weights" and rng.choice([False, True]):
        most = _log(rng, 1, 8192)
        return dict(op=op, reqs=_log(rng, 1, max(1, min(32, 12000 // most))),
                    shortest=0, longest=rng.choice([0, 0, _log(rng, 1, 4096)]),
                    fewest=rng.choice([1, most]), most=most, tree=False, decay=1.0, page=page, H=H,
                    Hkv=Hkv, D=D, dtype=dtype, mix=mix)
    longest = _log(rng, 1, 131072)
    reqs, shortest = _log(rng, 1, max(1, min(128, 262144 // longest))), rng.choice([0, 1, longest])
    if op == "weights":
        most = rng.choice([1, 1, _log(rng, 1, 64)])
        return dict(op=op, reqs=reqs, shortest=shortest, longest=longest, fewest=1, most=most,
                    tree=rng.choice([False, True]), decay=rng.choice([1.0, 0.9]), page=page, H=H,
                    Hkv=Hkv, D=D, dtype=dtype, mix=mix)
    return dict(op=op, reqs=max(1, reqs // 2), shortest=shortest, longest=longest,
                share=rng.choice([0.125, 0.5, 0.9]), first=rng.choice([0, 4]),
                recent=rng.choice([0, 32, 300]), page=page, H=H, Hkv=Hkv, D=D, dtype=dtype, mix=mix)


# ---------------------------------------------------------------------------
# lengths, from the case alone
# ---------------------------------------------------------------------------

def _between(rng, n, lo, hi):
    """n lengths of [lo, hi], the first of them hi."""
    lo = min(lo, hi)
    return [hi] + [rng.randint(lo, hi) for _ in range(n - 1)]


def _request_lens(c):
    """Tokens in the cache, and new ones, of each request."""
    rng = random.Random(c["mix"])
    ctx = _between(rng, c["reqs"], c["shortest"], c["longest"])
    return ctx, _between(rng, c["reqs"], c["fewest"], c["most"])


def _evict_lens(c):
    """Tokens in the cache, and how many stay; every fifth request is under its limit."""
    rng = random.Random(c["mix"])
    ctx = _between(rng, c["reqs"], c["shortest"], c["longest"])
    return ctx, [x + 3 if r % 5 == 4 else int(x * c["share"]) for r, x in enumerate(ctx)]


def _document_positions(c):
    """Positions of the S tokens that begin again at each document."""
    rng = random.Random(c["mix"])
    cuts = sorted(rng.sample(range(1, c["S"]), min(c["docs"] - 1, c["S"] - 1)))
    return [p for a, b in zip([0] + cuts, cuts + [c["S"]]) for p in range(b - a)]


def _offsets(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def work(c):
    D = c["D"]
    if c["op"] == "rotary":
        n = c["B"] * c["S"] * c["H"]
        elt = 4 if c["dtype"] == "fp32" else 2
        return {"bytes": 2 * elt * n * D + 4 * c["rot"] + (4 * c["S"] if c["docs"] or c["far"] else 0),
                "flops": 3 * n * c["rot"]}
    H, Hkv = c["H"], c["Hkv"]
    if c["op"] == "write":
        n = c["tokens"] + c["padded"]
        return {"bytes": 4 * D * H * n + 4 * D * Hkv * 2 * c["tokens"] + 12 * n + 4 * c["rot"],
                "flops": 3 * n * (H + Hkv) * c["rot"]}
    if c["op"] == "weights":
        ctx, new = _request_lens(c)
        rows, old = sum(new), sum(ctx)
        pairs = sum(n * x + n * (n + 1) // 2 for x, n in zip(ctx, new))
        return {"bytes": 2 * D * (H * rows + Hkv * (old + rows)) + 4 * H * rows
                + 4 * Hkv * (2 * old + rows), "flops": 2 * D * H * pairs}
    # A middle position stays with the same chance wherever it lies.
    total = 0.0
    for x, keep in zip(*_evict_lens(c)):
        if keep >= x:
            continue
        f = min(c["first"], keep)
        t = min(c["recent"], keep - f)
        middle = x - f - t
        moved = t + (x - keep) * (keep - t - f) / middle
        total += Hkv * (4 * middle + moved * (8 * D + 8) + 4 * keep)
    return {"bytes": max(1, int(total)), "flops": 0}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _ints(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device=DEV)


def _tree_masks(rng, new, tree):
    """A row's bits: itself and its ancestors in a random tree, as signed 64-bit words."""
    words = []
    for n in new:
        rows = []
        for i in range(n):
            parent = rng.randrange(-1, i) if tree else i - 1
            rows.append((rows[parent] if parent >= 0 else 0) | (1 << i))
        words += [w - (1 << 64) if w >> 63 else w for w in rows]
    return words


def _frequencies(rot):
    return torch.tensor([500000.0 ** (-2 * i / rot) for i in range(rot // 2)], dtype=torch.float64,
                        device=DEV)


def prepare(c, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    rng = random.Random(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32).to(TYPES[c["dtype"]])

    def pages(n):
        return torch.randperm(n, generator=gen, device=DEV, dtype=torch.int32)

    def block_table(need):
        """A table of `need` pages a request, and how many pages there are."""
        ids, width = pages(sum(need) + 3), max(need)
        table = torch.full((len(need), width), -1, dtype=torch.int32, device=DEV)
        table[torch.arange(width, device=DEV)[None] < _ints(need)[:, None]] = ids[:sum(need)]
        return table, sum(need) + 3

    s = dict(case=c)
    if c["op"] == "rotary":
        x = normal(c["B"], c["S"], c["H"], c["D"])
        at = None
        if c["docs"]:
            at = _ints(_document_positions(c))
        elif c["far"]:
            at = torch.arange(c["S"], device=DEV, dtype=torch.int32) + (c["far"] + rng.randrange(1000))
        s.update(x=x, at=at, freqs=_frequencies(c["rot"]))
        return s
    H, Hkv, D, P = c["H"], c["Hkv"], c["D"], c["page"]
    if c["op"] == "write":
        n = c["tokens"]
        npages = -(-n // P) + 2
        slots = (pages(npages).long()[:, None] * P + torch.arange(P, device=DEV)).flatten()[:n]
        # Decoding steps stand anywhere in their requests, a prompt's tokens one after another.
        first = torch.randint(0, 100000, (n + c["padded"],), generator=gen, device=DEV, dtype=torch.int32)
        at = first if n <= 256 else torch.arange(n + c["padded"], device=DEV, dtype=torch.int32)
        s.update(q=normal(n + c["padded"], H, D), k=normal(n + c["padded"], Hkv, D),
                 v=normal(n + c["padded"], Hkv, D), freqs=_frequencies(c["rot"]), at=at,
                 k_cache=normal(npages, P, Hkv, D), v_cache=normal(npages, P, Hkv, D),
                 slots=torch.cat([slots, torch.full((c["padded"],), -1, device=DEV)]))
        return s
    if c["op"] == "weights":
        ctx, new = _request_lens(c)
        table, npages = block_table([-(-(x + n) // P) for x, n in zip(ctx, new)])
        s.update(q=normal(sum(new), H, D), k_cache=normal(npages, P, Hkv, D), table=table,
                 ctx=_ints(ctx), cu=_ints(_offsets(new)), most=max(new),
                 masks=_ints(_tree_masks(rng, new, c["tree"]) if max(new) <= 64 else [0] * sum(new),
                             torch.int64),
                 weights=torch.rand(npages, Hkv, P, generator=gen, device=DEV).pow(4) * 9)
        s["lse"] = _over_heads(s, _normalisers)
        return s
    ctx, keep = _evict_lens(c)
    table, npages = block_table([max(1, -(-x // P)) for x in ctx])
    # A few positions draw much, many next to nothing; scores are pooled over neighbours.
    weights = torch.randn(npages, Hkv, P, generator=gen, device=DEV).mul_(2).exp_()
    weights[weights < 0.02] = 0
    s.update(k_cache=normal(npages, P, Hkv, D), v_cache=normal(npages, P, Hkv, D), table=table,
             ctx=_ints(ctx), keep=_ints(keep), most=max(max(min(x, k) for x, k in zip(ctx, keep)), 1),
             weights=weights,
             scores=torch.nn.functional.max_pool1d(weights, 3, stride=1, padding=1).contiguous())
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _into_ring(S, cp):
    """The natural position of each place of the ranks' order."""
    chunk = S // (2 * cp)
    rank = torch.arange(cp, device=DEV)
    starts = torch.stack([rank, 2 * cp - 1 - rank], 1).flatten() * chunk
    return (starts[:, None] + torch.arange(chunk, device=DEV)).flatten()


def _rotate(x, at, freqs, interleaved, sign):
    """x [.., tokens, heads, D] at positions [tokens], in 32 bits but for the angles."""
    rot = 2 * freqs.shape[0]
    angle = at.double()[:, None] * freqs
    cos, sin = angle.cos().float()[:, None], (angle.sin() * sign).float()[:, None]
    y = x.float()
    pair = y[..., :rot].unflatten(-1, (-1, 2)) if interleaved else y[..., :rot].unflatten(-1, (2, -1)).transpose(-1, -2)
    a, b = pair[..., 0], pair[..., 1]
    turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1)
    turned = turned.flatten(-2) if interleaved else turned.transpose(-1, -2).flatten(-2)
    return torch.cat([turned, y[..., rot:]], -1).to(x.dtype)


def _rotary(s):
    c, x = s["case"], s["x"]
    at = torch.arange(c["S"], device=DEV) if s["at"] is None else s["at"]
    if c["way"] != "keep":
        order = _into_ring(c["S"], c["cp"])
        if c["way"] == "in":
            x, at = x[:, order], at[order]
        else:
            back = torch.empty_like(order)
            back[order] = torch.arange(c["S"], device=DEV)
            x = x[:, back]
    return _rotate(x, at, s["freqs"], c["interleaved"], -1.0 if c["bwd"] else 1.0)


def _write(s):
    c = s["case"]
    n, turn = c["tokens"], (s["at"], s["freqs"], c["interleaved"], 1.0)
    s["k_cache"].flatten(0, 1)[s["slots"][:n]] = _rotate(s["k"], *turn)[:n]
    s["v_cache"].flatten(0, 1)[s["slots"][:n]] = s["v"][:n]
    return _rotate(s["q"], *turn), s["k_cache"], s["v_cache"]


def _rows(cu, total):
    """(sequence, position in it) of every packed row."""
    t = torch.arange(total, device=cu.device)
    r = torch.searchsorted(cu[1:].long(), t, right=True)
    return r, t - cu.long()[r]


def _over_heads(s, what):
    """what(scores [R, heads, G, n, m], seen [R, n, m], rows, heads) of some kv heads at a time, joined."""
    c, q, P = s["case"], s["q"], s["case"]["page"]
    R, n, Hkv, G, D = c["reqs"], s["most"], c["Hkv"], c["H"] // c["Hkv"], c["D"]
    cu, ctx = s["cu"].long(), s["ctx"].long()[:, None, None]
    i, j = torch.arange(n, device=DEV), torch.arange(s["table"].shape[1] * P, device=DEV)
    m = j.shape[0]
    rows = (cu[:-1, None] + i).clamp(max=q.shape[0] - 1)
    draft = j - ctx
    if c["tree"]:
        chosen = (s["masks"][rows][:, :, None] >> draft.clamp(0, 63)) & 1 == 1
    else:
        chosen = draft <= i[:, None]
    seen = ((draft < 0) | (chosen & (draft < cu.diff()[:, None, None]))) & (i[:, None] < cu.diff()[:, None, None])
    at, parts = s["table"].long().clamp(min=0), []
    # As many kv heads at a time as 8 GB of scores allow: all of them in most cases.
    step = max(1, min(Hkv, int(2e9 // max(1, R * G * n * m))))
    for g in range(0, Hkv, step):
        h = slice(g, g + step)
        k = s["k_cache"][:, :, h][at].flatten(1, 2).permute(0, 2, 3, 1).float()
        qq = q.view(-1, Hkv, G, D)[:, h][rows].permute(0, 2, 3, 1, 4).float()
        z = (qq.flatten(2, 3) @ k).mul_(1 / math.sqrt(D)).view(*qq.shape[:4], m)
        parts.append(what(s, z, seen, rows, h))
    return torch.cat(parts, 1 if what is _sums else 0)


def _normalisers(s, z, seen, rows, h):
    r, pos = _rows(s["cu"], s["q"].shape[0])
    lse = z.masked_fill_(~seen[:, None, None], -math.inf).logsumexp(-1)
    return lse.flatten(1, 2).permute(1, 0, 2)[:, r, pos].contiguous()


def _sums(s, z, seen, rows, h):
    lse = s["lse"].view(s["case"]["Hkv"], -1, s["q"].shape[0])[h][:, :, rows].permute(2, 0, 1, 3)
    return z.sub_(lse[..., None]).exp_().masked_fill_(~seen[:, None, None], 0).sum((2, 3))


def _weights(s):
    c, P, w = s["case"], s["case"]["page"], s["weights"]
    sums = _over_heads(s, _sums)
    ctx, new = s["ctx"].long()[:, None, None], s["cu"].long().diff()[:, None, None]
    j = torch.arange(sums.shape[-1], device=DEV)
    at = (s["table"].long()[:, None, j // P] * c["Hkv"] + torch.arange(c["Hkv"], device=DEV)[:, None]) * P + j % P
    live = ((j < ctx + new) & (new > 0)).expand_as(at)
    old = torch.where(j < ctx, w.flatten()[at.clamp(min=0)] * c["decay"], 0)
    w.view(-1)[at[live]] = (old + sums)[live]
    return w


def _evict(s):
    c, P, Hkv = s["case"], s["case"]["page"], s["case"]["Hkv"]
    ctx, keep = s["ctx"].long()[:, None, None], s["keep"].long()[:, None, None]
    keep = torch.minimum(ctx, keep)
    f = keep.clamp(max=c["first"])
    t = (keep - f).clamp(max=c["recent"])
    cut = torch.where(keep < ctx, keep - t, ctx)
    j = torch.arange(s["table"].shape[1] * P, device=DEV)
    g = torch.arange(Hkv, device=DEV)[:, None]
    page = s["table"].long().clamp(min=0)[:, None, j // P]
    at = (page * Hkv + g) * P + j % P
    score = torch.nan_to_num(s["scores"].flatten()[at], nan=-math.inf, posinf=math.inf, neginf=-math.inf)
    # The first and last of a request before its middle, its middle before what lies behind it.
    kind = ((j < f) | (j >= ctx - t)).long() + (j < ctx).long() * 2
    kind = torch.where(j < ctx, kind, 0).expand_as(at)
    order = score.argsort(dim=-1, descending=True, stable=True)
    order = order.gather(-1, kind.gather(-1, order).argsort(dim=-1, descending=True, stable=True))
    rank = torch.empty_like(order).scatter_(-1, order, j.expand_as(order))
    stays = (rank < keep) & (j < ctx)
    # Slot i gets position kept[i]: survivors below the cut stay, holes get those above it in order.
    hole, late = (j < cut) & ~stays, (j >= cut) & (j < ctx - t) & stays
    nth = late.long().cumsum(-1) - 1
    source = torch.zeros_like(order).scatter_(-1, torch.where(late, nth, j.numel() - 1), j.expand_as(order).where(late, 0))
    kept = torch.where(hole, source.gather(-1, (hole.long().cumsum(-1) - 1).clamp(min=0)), j)
    kept = torch.where((j >= cut) & (j < keep), j + (ctx - keep), kept)
    kept = torch.where(j < keep, kept, -1)[..., :s["most"]]
    kept = torch.nn.functional.pad(kept, (0, s["most"] - kept.shape[-1]), value=-1)
    # Only what changes its place is copied, all of it read before any is written.
    r, g, to = ((kept >= 0) & (kept != torch.arange(s["most"], device=DEV))).nonzero(as_tuple=True)
    frm = kept[r, g, to]
    src, dst = s["table"].long()[r, frm // P], s["table"].long()[r, to // P]
    for x in (s["k_cache"], s["v_cache"]):
        x[dst, to % P, g] = x[src, frm % P, g]
    s["weights"][dst, g, to % P] = s["weights"][src, g, frm % P]
    have, need = (ctx + P - 1) // P, (keep + P - 1) // P
    col = torch.arange(s["table"].shape[1], device=DEV)
    gone = ((col >= need[:, 0]) & (col < have[:, 0])).flatten()
    place = torch.where(gone, gone.long().cumsum(0) - 1, gone.numel())
    freed = torch.full((gone.numel() + 1,), -1, dtype=torch.int32, device=DEV)
    freed = freed.scatter_(0, place, s["table"].flatten())[:-1]
    freed = torch.where(torch.arange(gone.numel(), device=DEV) < gone.sum(), freed, -1)
    return (s["k_cache"], s["v_cache"], s["weights"], keep.flatten().int(), kept.int(), freed,
            gone.sum()[None].int())


def run(s):
    c = s["case"]
    if not own:
        return {"rotary": _rotary, "write": _write, "weights": _weights, "evict": _evict}[c["op"]](s)
    import context_causal_attention_zigzag_gb300 as cpa
    # Outputs and scratch are made on the first pass and kept, as a training or serving loop keeps them.
    if c["op"] == "rotary":
        call = cpa.rotary_bwd if c["bwd"] else cpa.rotary
        if "keep_out" not in s:
            s["keep_out"] = torch.empty_like(s["x"])
        return call(s["x"], s["freqs"], s["at"], interleaved=c["interleaved"], cp=c["cp"],
                    from_sharded=c["way"] == "out", to_sharded=c["way"] == "in", out=s["keep_out"])
    if c["op"] == "write":
        if "keep_out" not in s:
            s["keep_out"] = torch.empty_like(s["q"])
        return cpa.rotary_cache_write(s["q"], s["k"], s["v"], s["freqs"], s["at"], s["k_cache"],
                                      s["v_cache"], s["slots"], interleaved=c["interleaved"],
                                      out=s["keep_out"])
    if c["op"] == "weights":
        if "scratch" not in s:
            s["scratch"] = cpa.cache_weights_workspace(s["q"], s["k_cache"], s["cu"])
        return cpa.cache_weights(s["q"], s["k_cache"], s["table"], s["ctx"], s["cu"], s["lse"],
                                 s["weights"], tree=s["masks"] if c["tree"] else None,
                                 decay=c["decay"], workspace=s["scratch"])
    if "outputs" not in s:
        s["outputs"] = cpa.cache_evict_outputs(s["k_cache"], s["table"], s["ctx"], s["most"])
        s["scratch"] = cpa.cache_evict_workspace(s["k_cache"], s["table"], s["most"])
    new_lens, kept, freed, count = cpa.cache_evict(
        s["weights"], s["k_cache"], s["v_cache"], s["table"], s["ctx"], s["keep"], s["most"],
        first=c["first"], recent=c["recent"], scores=s["scores"], outputs=s["outputs"],
        workspace=s["scratch"])
    return s["k_cache"], s["v_cache"], s["weights"], new_lens, kept, freed, count


# ---------------------------------------------------------------------------
# the definition, in 64 bits
# ---------------------------------------------------------------------------

def _turned(x, at, freqs, interleaved, sign):
    """x [tokens, heads, D] in 64 bits: every pair as a complex number times e^(i angle)."""
    rot = 2 * freqs.shape[0]
    y = x.double().clone()
    one, two = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    z = torch.complex(y[..., one].contiguous(), y[..., two].contiguous())
    z = z * torch.polar(torch.ones_like(freqs), sign * freqs * at.double()[:, None])[:, None]
    y[..., one], y[..., two] = z.real, z.imag
    return y


def exact(c, seed):
    if c["op"] == "evict" or (c["op"] == "weights" and work(c)["flops"] > 2.5e12):
        return None
    s = prepare(c, seed)
    if c["op"] == "rotary":
        S, cp = c["S"], c["cp"]
        at = torch.arange(S, device=DEV) if s["at"] is None else s["at"]
        ranks = [p for r in range(cp) for p in (r, 2 * cp - 1 - r)]
        out = []
        for x in s["x"]:
            if c["way"] == "out":  # the chunks as they stand, back to their places
                x = torch.cat([x.chunk(2 * cp)[ranks.index(p)] for p in range(2 * cp)])
            y = _turned(x, at, s["freqs"], c["interleaved"], -1 if c["bwd"] else 1)
            out.append(torch.cat([y.chunk(2 * cp)[p] for p in ranks]) if c["way"] == "in" else y)
        return torch.stack(out)
    if c["op"] == "write":
        n, P = c["tokens"], c["page"]
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        turn = (s["at"], s["freqs"], c["interleaved"], 1)
        kc[s["slots"][:n] // P, s["slots"][:n] % P] = _turned(s["k"], *turn)[:n]
        vc[s["slots"][:n] // P, s["slots"][:n] % P] = s["v"][:n].double()
        return _turned(s["q"], *turn), kc, vc
    w, q, P = s["weights"].double(), s["q"].double(), c["page"]
    ctx, new = _request_lens(c)
    first, G = _offsets(new), c["H"] // c["Hkv"]
    for r, (x, n) in enumerate(zip(ctx, new)):
        pos = torch.arange(x + n, device=DEV)
        page = s["table"][r].long()[pos // P]
        k = s["k_cache"][page, pos % P].double()
        hide = torch.zeros(n, x + n, dtype=torch.bool, device=DEV)
        if c["tree"]:
            words = s["masks"][first[r]:first[r + 1]].tolist()
            hide[:, x:] = torch.tensor([[not (b >> j) & 1 for j in range(n)] for b in words], device=DEV)
        else:
            hide = torch.ones(n, x + n, dtype=torch.bool, device=DEV).triu(x + 1)
        for g in range(c["Hkv"]):
            total = torch.where(pos < x, w[page, g, pos % P] * c["decay"], 0.0)
            for h in range(g * G, g * G + G):
                for a in range(0, n, 4096):
                    b = min(n, a + 4096)
                    i = slice(first[r] + a, first[r] + b)
                    z = (q[i, h] @ k[:, g].T) / math.sqrt(c["D"]) - s["lse"][h, i, None].double()
                    total = total + z.exp().masked_fill_(hide[a:b], 0.0).sum(0)
            w[page, g, pos % P] = total
    return w
