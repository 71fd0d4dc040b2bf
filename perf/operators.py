"""Cases, plain forms and exact values of the answering operators: the paged
cache's tables, the write into it, attention of drafted tokens over it, and
attention over packed prompts.

A case's sequence lengths follow from the case alone (its "mix" number), its
tensors from the seed alone.
"""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
# (query heads, kv heads, head dim): the repository's grouped and plain layouts,
# and generic multi-query and odd-group ones.
HEADS = [(32, 8, 128), (16, 16, 128), (2, 2, 64), (8, 1, 128), (14, 2, 64), (32, 8, 64)]
PAGES = [16, 32, 64, 128, 256]


def listed():
    return [
        # One short question to an idle server: latency.
        dict(name="prompt_one_short", op="prompt", seqs=1, shortest=77, longest=77, prefix=0,
             H=32, Hkv=8, D=128, dtype="bf16", mix=1),
        # An ordinary batch of questions of uneven length.
        dict(name="prompt_packed_mixed", op="prompt", seqs=16, shortest=100, longest=2000, prefix=0,
             H=32, Hkv=8, D=128, dtype="bf16", mix=2),
        # Follow-up turns: new tokens behind a context whose keys are at hand; 64-wide heads.
        dict(name="prompt_behind_prefix_fp16", op="prompt", seqs=5, shortest=33, longest=1025,
             prefix=2500, H=32, Hkv=8, D=64, dtype="fp16", mix=3),
        # One long document, no grouping.
        dict(name="prompt_long_document", op="prompt", seqs=1, shortest=16384, longest=16384,
             prefix=0, H=32, Hkv=8, D=128, dtype="bf16", mix=4),
        # One user, next token: latency.
        dict(name="tree_one_token_one_user", op="tree", reqs=1, shortest=1000, longest=1000,
             fewest=1, most=1, tree=False, page=64, H=32, Hkv=8, D=128, dtype="bf16", mix=5),
        # Next tokens of a busy server, contexts of all lengths.
        dict(name="tree_one_token_batch", op="tree", reqs=64, shortest=100, longest=8192, fewest=1,
             most=1, tree=False, page=64, H=32, Hkv=8, D=128, dtype="bf16", mix=6),
        # Verification of drafted trees of uneven size.
        dict(name="tree_drafts_fp16", op="tree", reqs=16, shortest=500, longest=5000, fewest=5,
             most=31, tree=True, page=16, H=32, Hkv=8, D=128, dtype="fp16", mix=7),
        # Two whole books in the cache, a small tree each.
        dict(name="tree_long_cache", op="tree", reqs=2, shortest=100000, longest=131072, fewest=6,
             most=8, tree=True, page=128, H=32, Hkv=8, D=128, dtype="bf16", mix=8),
        # The keys and values of one decoding step's tokens.
        dict(name="write_one_step", op="write", tokens=64, padded=3, page=64, Hkv=8, D=128,
             dtype="bf16", mix=9),
        # The keys and values of a long packed prompt.
        dict(name="write_prompt", op="write", tokens=32001, padded=0, page=64, Hkv=8, D=128,
             dtype="bf16", mix=10),
        # One decoding step of a small batch, slots padded to a fixed length.
        dict(name="tables_one_step", op="tables", reqs=8, context=3000, fewest=1, most=1, padded=8,
             page=64, mix=11),
        # Prompts of a whole queue admitted at once.
        dict(name="tables_admit_queue", op="tables", reqs=1000, context=500, fewest=0, most=700,
             padded=100, page=16, mix=12),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)) - 1e-9)))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "tree", "tree", "write", "tables"])
    H, Hkv, D = rng.choice(HEADS)
    mix, dtype = rng.randrange(1 << 30), rng.choice(list(TYPES))
    if op == "prompt":
        longest = _log(rng, 1, 8192)
        return dict(op=op, seqs=_log(rng, 1, max(1, min(64, 16384 // longest))),
                    shortest=rng.choice([0, 1, longest]), longest=longest,
                    prefix=rng.choice([0, 0, _log(rng, 1, 4096)]), H=H, Hkv=Hkv, D=D, dtype=dtype,
                    mix=mix)
    if op == "tree":
        longest = _log(rng, 1, 131072)
        most = rng.choice([1, 1, _log(rng, 1, 64)])
        return dict(op=op, reqs=_log(rng, 1, max(1, min(256, 262144 // longest))),
                    shortest=rng.choice([0, 1, longest]), longest=longest, fewest=1, most=most,
                    tree=rng.choice([False, True]), page=rng.choice(PAGES), H=H, Hkv=Hkv, D=D,
                    dtype=dtype, mix=mix)
    if op == "write":
        return dict(op=op, tokens=_log(rng, 1, 32001), padded=rng.choice([0, 5]),
                    page=rng.choice(PAGES), Hkv=Hkv, D=D, dtype=dtype, mix=mix)
    most = _log(rng, 1, 2000)
    return dict(op=op, reqs=_log(rng, 1, max(1, min(1000, 350000 // most))),
                context=_log(rng, 1, 4000), fewest=rng.choice([0, 1, most]), most=most,
                padded=rng.choice([0, 64]), page=rng.choice(PAGES), mix=mix)


# ---------------------------------------------------------------------------
# lengths, from the case alone
# ---------------------------------------------------------------------------

def _between(rng, n, lo, hi):
    """n lengths of [lo, hi], the first of them hi."""
    lo = min(lo, hi)
    return [hi] + [rng.randint(lo, hi) for _ in range(n - 1)]


def _prompt_lens(c):
    rng = random.Random(c["mix"])
    nq = _between(rng, c["seqs"], c["shortest"], c["longest"])
    return nq, [n + (rng.randint(1, c["prefix"]) if c["prefix"] else 0) for n in nq]


def _tree_lens(c):
    rng = random.Random(c["mix"])
    return (_between(rng, c["reqs"], c["shortest"], c["longest"]),
            _between(rng, c["reqs"], c["fewest"], c["most"]))


def _table_lens(c):
    rng = random.Random(c["mix"])
    return ([rng.randint(0, c["context"]) for _ in range(c["reqs"])],
            _between(rng, c["reqs"], c["fewest"], c["most"]))


def _offsets(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def work(c):
    if c["op"] == "prompt":
        nq, nk = _prompt_lens(c)
        pairs = sum(q * (k - q) + q * (q + 1) // 2 for q, k in zip(nq, nk))
        return {"bytes": 2 * c["D"] * (2 * c["H"] * sum(nq) + 2 * c["Hkv"] * sum(nk))
                + 4 * c["H"] * sum(nq), "flops": 4 * c["D"] * c["H"] * pairs}
    if c["op"] == "tree":
        ctx, new = _tree_lens(c)
        rows = sum(new)
        pairs = sum(n * x + n * (n + 1) // 2 for x, n in zip(ctx, new))
        return {"bytes": 2 * c["D"] * (2 * c["H"] * rows + 2 * c["Hkv"] * (sum(ctx) + rows))
                + 4 * c["H"] * rows, "flops": 4 * c["D"] * c["H"] * pairs}
    if c["op"] == "write":
        return {"bytes": 8 * c["tokens"] * c["Hkv"] * c["D"] + 8 * (c["tokens"] + c["padded"]),
                "flops": 0}
    ctx, new = _table_lens(c)
    P = c["page"]
    used = sum(-(-(x + n) // P) + -x // P for x, n in zip(ctx, new))
    return {"bytes": 12 * c["reqs"] + 8 * used + 8 * (sum(new) + c["padded"]), "flops": 0}


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


def prepare(c, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    rng = random.Random(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32).to(TYPES[c["dtype"]])

    def pages(n):
        return torch.randperm(n, generator=gen, device=DEV, dtype=torch.int32)

    s = dict(case=c)
    if c["op"] == "prompt":
        nq, nk = _prompt_lens(c)
        s.update(q=normal(sum(nq), c["H"], c["D"]), k=normal(sum(nk), c["Hkv"], c["D"]),
                 v=normal(sum(nk), c["Hkv"], c["D"]), cu_q=_ints(_offsets(nq)),
                 cu_k=_ints(_offsets(nk)), most_q=max(nq), most_k=max(nk))
    elif c["op"] == "tree":
        ctx, new = _tree_lens(c)
        need = [-(-(x + n) // c["page"]) for x, n in zip(ctx, new)]
        ids, width, cu = pages(sum(need) + 3), max(need), _offsets(need)
        table = torch.full((c["reqs"], width), -1, dtype=torch.int32, device=DEV)
        at = torch.arange(width, device=DEV)[None] < _ints(need)[:, None]
        table[at] = ids[:cu[-1]]
        s.update(q=normal(sum(new), c["H"], c["D"]),
                 k_cache=normal(sum(need) + 3, c["page"], c["Hkv"], c["D"]),
                 v_cache=normal(sum(need) + 3, c["page"], c["Hkv"], c["D"]), table=table,
                 ctx=_ints(ctx), cu=_ints(_offsets(new)), most=max(new),
                 masks=_ints(_tree_masks(rng, new, c["tree"]), torch.int64))
    elif c["op"] == "write":
        n, P = c["tokens"], c["page"]
        npages = -(-n // P) + 2
        slots = (pages(npages).long()[:, None] * P + torch.arange(P, device=DEV)).flatten()[:n]
        s.update(k=normal(n + c["padded"], c["Hkv"], c["D"]), v=normal(n + c["padded"], c["Hkv"], c["D"]),
                 k_cache=normal(npages, P, c["Hkv"], c["D"]), v_cache=normal(npages, P, c["Hkv"], c["D"]),
                 slots=torch.cat([slots, torch.full((c["padded"],), -1, device=DEV)]))
    else:
        ctx, new = _table_lens(c)
        P = c["page"]
        have = [-(-x // P) for x in ctx]
        need = [-(-(x + n) // P) for x, n in zip(ctx, new)]
        ids, width = pages(sum(need) + 5), max(1, max(need))
        table = torch.full((c["reqs"], width), -1, dtype=torch.int32, device=DEV)
        at = torch.arange(width, device=DEV)[None] < _ints(have)[:, None]
        table[at] = ids[:sum(have)]
        s.update(table=table, free=ids[sum(have):].clone(), ctx=_ints(ctx), new=_ints(new),
                 tokens=sum(new) + c["padded"])
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _attend(q, k, v, seen, D):
    """q [R, n, Hkv, G, D], k, v [R, m, Hkv, D], seen [R, n, m] -> (o [R, n, Hkv, G, D], lse [R, Hkv, G, n])."""
    R, n, Hkv, G, _ = q.shape
    m = k.shape[1]
    o = torch.empty((R, n, Hkv, G, D), dtype=torch.float32, device=q.device)
    lse = torch.empty((R, Hkv, G, n), dtype=torch.float32, device=q.device)
    # As many kv heads at a time as 16 GB of scores allow: all of them in most cases.
    step = max(1, min(Hkv, int(4e9 // max(1, R * G * n * m))))
    for g in range(0, Hkv, step):
        h = slice(g, g + step)
        w = q[:, :, h].shape[2]
        qq = q[:, :, h].permute(0, 2, 3, 1, 4).reshape(R, w, G * n, D).float()
        s = (qq @ k[:, :, h].permute(0, 2, 3, 1).float()).mul_(1.0 / math.sqrt(D)).view(R, w, G, n, m)
        s.masked_fill_(~seen[:, None, None], -math.inf)
        top = s.amax(-1, keepdim=True).clamp_min(-1e30)
        p = s.sub_(top).exp_()
        total = p.sum(-1, keepdim=True)
        vv = v[:, :, h].permute(0, 2, 1, 3).float()
        oo = (p.view(R, w, G * n, m) @ vv).view(R, w, G, n, D) / total.clamp_min(1e-30)
        o[:, :, h] = oo.permute(0, 3, 1, 2, 4)
        lse[:, h] = (total.log() + top).squeeze(-1)
    return o, lse


def _rows(cu, total):
    """(sequence, position in it) of every packed row."""
    t = torch.arange(total, device=cu.device)
    r = torch.searchsorted(cu[1:].long(), t, right=True)
    return r, t - cu.long()[r]


def _prompt(s):
    c, q, k, v = s["case"], s["q"], s["k"], s["v"]
    G = c["H"] // c["Hkv"]
    cq, ck = s["cu_q"].long(), s["cu_k"].long()
    i, j = torch.arange(s["most_q"], device=q.device), torch.arange(s["most_k"], device=q.device)
    nq, nk = cq.diff()[:, None, None], ck.diff()[:, None, None]
    seen = (j[None, None] <= i[None, :, None] + nk - nq) & (j < nk)
    qp = q[(cq[:-1, None] + i).clamp(max=q.shape[0] - 1)]
    at = (ck[:-1, None] + j).clamp(max=k.shape[0] - 1)
    o, lse = _attend(qp.view(*qp.shape[:2], c["Hkv"], G, c["D"]), k[at], v[at], seen, c["D"])
    r, pos = _rows(s["cu_q"], q.shape[0])
    return (o[r, pos].reshape(q.shape).to(q.dtype),
            lse.flatten(1, 2).permute(1, 0, 2)[:, r, pos].contiguous())


def _tree(s):
    c, q, P = s["case"], s["q"], s["case"]["page"]
    G, cu, ctx = c["H"] // c["Hkv"], s["cu"].long(), s["ctx"].long()[:, None, None]
    i, j = torch.arange(s["most"], device=q.device), torch.arange(s["table"].shape[1] * P, device=q.device)
    rows = (cu[:-1, None] + i).clamp(max=q.shape[0] - 1)
    at = s["table"].long().clamp(min=0)
    k, v = (x[at].flatten(1, 2) for x in (s["k_cache"], s["v_cache"]))
    draft = j - ctx
    bit = (s["masks"][rows][:, :, None] >> draft.clamp(0, 63)) & 1
    seen = (draft < 0) | ((bit == 1) & (draft < cu.diff()[:, None, None]))
    qp = q[rows]
    o, lse = _attend(qp.view(*qp.shape[:2], c["Hkv"], G, c["D"]), k, v, seen, c["D"])
    r, pos = _rows(s["cu"], q.shape[0])
    return (o[r, pos].reshape(q.shape).to(q.dtype),
            lse.flatten(1, 2).permute(1, 0, 2)[:, r, pos].contiguous())


def _write(s):
    n = s["case"]["tokens"]
    at = s["slots"][:n]
    s["k_cache"].flatten(0, 1)[at] = s["k"][:n]
    s["v_cache"].flatten(0, 1)[at] = s["v"][:n]
    return s["k_cache"], s["v_cache"]


def _tables(s):
    P, ctx, new, table = s["case"]["page"], s["ctx"].long(), s["new"].long(), s["table"]
    have, need = (ctx + P - 1) // P, (ctx + new + P - 1) // P
    ends = (need - have).cumsum(0)
    col = torch.arange(table.shape[1], device=table.device)[None]
    fresh = (col >= have[:, None]) & (col < need[:, None])
    pick = (ends - need)[:, None] + col
    table.copy_(torch.where(fresh, s["free"][pick.clamp(0, s["free"].shape[0] - 1)], table))
    cu = torch.cat([new.new_zeros(1), new.cumsum(0)])
    r, i = _rows(cu, s["tokens"])
    live = r < ctx.shape[0]
    r = r.clamp(max=ctx.shape[0] - 1)
    pos = torch.where(live, ctx[r] + i, 0)
    slots = torch.where(live, table[r, pos // P].long() * P + pos % P, -1)
    return table, slots, cu.int(), ends[-1:].int()


def run(s):
    op = s["case"]["op"]
    if not own:
        return {"prompt": _prompt, "tree": _tree, "write": _write, "tables": _tables}[op](s)
    import context_causal_attention_zigzag_gb300 as cpa
    # Outputs and scratch are made on the first pass and kept, as a serving loop keeps them.
    if op == "prompt":
        if "keep" not in s:
            out, lse = cpa.prompt_attention(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"])
            s["keep"] = dict(out=out, lse=lse, workspace=cpa.prompt_attention_workspace(s["q"], s["cu_q"]))
        return cpa.prompt_attention(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], **s["keep"])
    if op == "tree":
        args = (s["q"], s["k_cache"], s["v_cache"], s["table"], s["ctx"], s["cu"])
        tree = s["masks"] if s["case"]["tree"] else None
        if "keep" not in s:
            out, lse = cpa.tree_attention(*args, tree)
            s["keep"] = dict(out=out, lse=lse, workspace=cpa.tree_attention_workspace(s["q"], s["k_cache"], s["cu"]))
        return cpa.tree_attention(*args, tree, **s["keep"])
    if op == "write":
        return cpa.cache_write(s["k"], s["v"], s["k_cache"], s["v_cache"], s["slots"])
    if "keep" not in s:
        s["keep"] = dict(zip(("slots", "cu", "used"),
                             cpa.page_tables(s["ctx"], s["new"], s["table"], s["free"],
                                             s["case"]["page"], s["tokens"])))
    return (s["table"], *cpa.page_tables(s["ctx"], s["new"], s["table"], s["free"],
                                         s["case"]["page"], s["tokens"], **s["keep"]))


# ---------------------------------------------------------------------------
# the definition, in 64 bits: one sequence and one kv head at a time
# ---------------------------------------------------------------------------

def _softmax_rows(q, k, v, hide, out, lse, rows):
    """q [n, H, D], k, v [m, Hkv, D] in 64 bits; hide [n, m]."""
    n, H, D = q.shape
    G = H // k.shape[1]
    for h in range(H):
        for a in range(0, n, 4096):
            z = q[a:a + 4096, h] @ k[:, h // G].T / math.sqrt(D)
            z[hide[a:a + 4096]] = -math.inf
            l = torch.logsumexp(z, -1)
            w = torch.where(hide[a:a + 4096], 0.0, (z - l[:, None]).exp())
            out[rows[a:a + 4096], h] = w @ v[:, h // G]
            lse[h, rows[a:a + 4096]] = l


def exact(c, seed):
    if c["op"] not in ("prompt", "tree"):
        return None
    # 64-bit products run at about a thousandth of the tensor cores' rate.
    if work(c)["flops"] > 5e12:
        return None
    s = prepare(c, seed)
    q = s["q"].double()
    out, lse = torch.zeros_like(q), torch.zeros(q.shape[1], q.shape[0], dtype=torch.float64, device=DEV)
    if c["op"] == "prompt":
        nq, nk = _prompt_lens(c)
        fq, fk = _offsets(nq), _offsets(nk)
        for r, (n, m) in enumerate(zip(nq, nk)):
            hide = torch.ones(n, m, dtype=torch.bool, device=DEV).triu(m - n + 1)
            at = slice(fk[r], fk[r + 1])
            _softmax_rows(q[fq[r]:fq[r + 1]], s["k"][at].double(), s["v"][at].double(), hide, out, lse,
                          torch.arange(fq[r], fq[r + 1], device=DEV))
        return out, lse
    ctx, new = _tree_lens(c)
    first = _offsets(new)
    for r, (x, n) in enumerate(zip(ctx, new)):
        pos = torch.arange(x + n, device=DEV)
        page = s["table"][r].long()[pos // c["page"]]
        k, v = (t[page, pos % c["page"]].double() for t in (s["k_cache"], s["v_cache"]))
        words = s["masks"][first[r]:first[r + 1]].tolist()
        hide = torch.zeros(n, x + n, dtype=torch.bool, device=DEV)
        hide[:, x:] = torch.tensor([[not (w >> j) & 1 for j in range(n)] for w in words], device=DEV)
        _softmax_rows(q[first[r]:first[r + 1]], k, v, hide, out, lse,
                      torch.arange(first[r], first[r + 1], device=DEV))
    return out, lse
