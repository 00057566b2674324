"""Cases of the operators that the attention layers of a hybrid stack need beside the Gated DeltaNet layer, and of
speculation over a tree of drafts:

  plan     block tables and slot maps of a paged KV cache, built on the GPU from the requests' lengths;
  write    the K and V rows of new tokens into their cache slots;
  prefill  causal attention over packed prompts, each after a prefix that is in the cache already (or none);
  tree     attention of a tree of drafted tokens over the cache (one node: the decode step);
  vtree    the gated delta rule over a tree of drafts, a pool slot written per node.

With ``own`` false ``run`` computes them from elementary torch operations in 32 bits; with it true it makes the calls of
gated_deltanet_delta_amd.  ``exact`` computes the same results in 64 bits, from the definitions.
"""
import math

import torch

own = False

BF16, F32 = torch.bfloat16, torch.float32


# ----------------------------------------------------------------------------
# the cases
# ----------------------------------------------------------------------------

def listed():
    return [
        # four requests decode one token each: the plan and the write of every decode step
        dict(name="plan decode step, 4 requests", op="plan", batch=4, page=16, ctx_hi=8192, new_hi=1, leave=0, pad=0),
        # a full server's step: prompts, decodes, idle rows and leaving requests in one batch, slot map padded to a capture size
        dict(name="plan mixed step, 512 requests", op="plan", batch=512, page=16, ctx_hi=16384, new_hi=1000, leave=9, pad=4097),
        dict(name="write decode step, 4 tokens", op="write", tokens=4, heads=4, d=256, page=16, dtype="bf16", fused=True),
        # a prompt's K and V, pages of the 528 tokens that hybrid cache managers use
        dict(name="write prompt, 32771 tokens", op="write", tokens=32771, heads=4, d=256, page=528, dtype="bf16", fused=False),
        # one prompt of the prefill benchmark's length, 24 query heads on 4 KV heads
        dict(name="prefill one prompt, 8192", op="prefill", new="8192", ctx="0", heads=4, group=6, d=256, page=528, dtype="bf16", fused=False),
        # ragged prompts, some after a cached prefix, one a single token, read out of fused projection rows
        dict(name="prefill ragged, prefixes", op="prefill", new="1,63,4099,1500,2047,700", ctx="8191,0,0,20011,528,130", heads=8, group=4, d=128,
             page=528, dtype="bf16", fused=True),
        dict(name="prefill fp32, short prompts", op="prefill", new="301,1,777", ctx="0,64,0", heads=2, group=4, d=64, page=16, dtype="f32", fused=False),
        # the decode step of four requests at 8K
        dict(name="tree decode step, 4 x 8K", op="tree", batch=4, nodes=1, ctx_lo=8100, ctx_hi=8192, heads=4, group=6, d=256, page=16, dtype="bf16", fused=True),
        # 16-node trees over long contexts
        dict(name="tree 16 nodes, 4 x 100K", op="tree", batch=4, nodes=16, ctx_lo=80000, ctx_hi=120000, heads=4, group=6, d=256, page=528, dtype="bf16", fused=False),
        # many requests of ragged lengths, 8 nodes each
        dict(name="tree 8 nodes, 64 ragged", op="tree", batch=64, nodes=8, ctx_lo=33, ctx_hi=16384, heads=8, group=4, d=128, page=16, dtype="bf16", fused=False),
        # the verify benchmark's four slots with a tree of 4 nodes
        dict(name="vtree 4 slots x 4 nodes", op="vtree", batch=4, nodes=4, kheads=16, group=3, d=128, dtype="bf16"),
        # sixteen slots with trees of 15 nodes
        dict(name="vtree 16 slots x 15 nodes", op="vtree", batch=16, nodes=15, kheads=16, group=3, d=128, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(("plan", "write", "prefill", "prefill", "tree", "tree", "vtree"))
    page = rng.choice((16, 16, 32, 64, 528))
    dtype = rng.choice(("bf16", "bf16", "bf16", "f32"))
    d = rng.choice((64, 128, 256))
    if op == "plan":
        return dict(op=op, batch=_log(rng, 1, 512), page=page, ctx_hi=_log(rng, 16, 16384), new_hi=_log(rng, 1, 1000),
                    leave=rng.choice((0, 2, 5, 9)), pad=_log(rng, 1, 5000) - 1)
    if op == "write":
        return dict(op=op, tokens=_log(rng, 1, 20000), heads=rng.choice((1, 2, 4, 8)), d=d, page=page, dtype=dtype, fused=rng.random() < 0.5)
    if op == "prefill":
        heads, group = rng.choice((1, 2, 4, 8)), rng.choice((1, 2, 3, 4, 6, 8))
        seqs = rng.randint(1, 6)
        budget = (1.5e11 if dtype == "bf16" else 2e10) / (4 * heads * group * d) / seqs  # query-key pairs of one sequence
        new, ctx = [], []
        for _ in range(seqs):
            n = _log(rng, 1, max(1, min(8192, int(math.sqrt(budget)))))
            new.append(n)
            ctx.append(0 if rng.random() < 0.5 else _log(rng, 1, max(1, min(30000, int(budget / n)))))
        return dict(op=op, new=",".join(map(str, new)), ctx=",".join(map(str, ctx)), heads=heads, group=group, d=d, page=page, dtype=dtype,
                    fused=rng.random() < 0.5)
    if op == "tree":
        heads, group, batch = rng.choice((1, 2, 4, 8)), rng.choice((1, 2, 3, 4, 6, 8)), _log(rng, 1, 64)
        most = max(64, int(3e8 / (batch * heads * d)))  # cached tokens of a request
        lo, hi = sorted((_log(rng, 1, min(100000, most)), _log(rng, 1, min(100000, most))))
        return dict(op=op, batch=batch, nodes=_log(rng, 1, 32), ctx_lo=lo, ctx_hi=hi, heads=heads, group=group, d=d, page=page, dtype=dtype,
                    fused=rng.random() < 0.5)
    return dict(op=op, batch=_log(rng, 1, 16), nodes=rng.randint(1, 15), kheads=rng.choice((1, 2, 4, 8, 16)), group=rng.choice((1, 2, 3, 4)),
                d=rng.choice((32, 64, 128)), dtype=dtype)


def _type(case):
    return BF16 if case["dtype"] == "bf16" else F32


def _spread(lo, hi, n):
    """n lengths between lo and hi, spread over their logarithm, the same for every seed."""
    return [max(lo, min(hi, int(round(lo * (hi / lo) ** ((0.35 + 0.6180339887 * i) % 1.0))))) for i in range(n)]


def _plan_lengths(case):
    """(cached, new) tokens of every row; new = -1 where a request leaves, 0 where it idles."""
    kv = _spread(1, case["ctx_hi"], case["batch"])
    prompts = _spread(1, case["new_hi"], case["batch"])
    new = []
    for i in range(case["batch"]):
        if case["leave"] and i % case["leave"] == case["leave"] - 1:
            new.append(-1)
        elif i % 3 == 1:
            new.append(prompts[i])
        else:
            new.append(0 if i % 16 == 15 else 1)
        if case["new_hi"] > 1 and i % 7 == 3:
            kv[i] = 0  # a request that has just come
            new[i] = prompts[i]
    return kv, new


def _pages(tokens, page):
    return -(-tokens // page)


def _two(case):
    return [int(t) for t in case["new"].split(",")], [int(t) for t in case["ctx"].split(",")]


def work(case):
    op = case["op"]
    if op == "plan":
        kv, new = _plan_lengths(case)
        n = sum(max(t, 0) for t in new)
        fresh = sum(_pages(c + t, case["page"]) - _pages(c, case["page"]) for c, t in zip(kv, new) if t > 0)
        gone = sum(_pages(c, case["page"]) for c, t in zip(kv, new) if t < 0)
        return {"bytes": 16 * len(kv) + 8 * fresh + 8 * gone + 8 * (n + case["pad"]), "flops": 0}
    size = 2 if case["dtype"] == "bf16" else 4
    if op == "write":
        return {"bytes": case["tokens"] * (4 * case["heads"] * case["d"] * size + 4), "flops": 0}
    if op == "prefill":
        new, ctx = _two(case)
        hq = case["heads"] * case["group"]
        pairs = sum(n * c + n * (n + 1) // 2 for n, c in zip(new, ctx))
        return {"bytes": case["d"] * size * (2 * hq * sum(new) + 2 * case["heads"] * (sum(new) + sum(ctx))), "flops": 4 * hq * case["d"] * pairs}
    if op == "tree":
        ctx = _spread(case["ctx_lo"], case["ctx_hi"], case["batch"])
        hq, rows = case["heads"] * case["group"], case["batch"] * case["nodes"]
        return {"bytes": case["d"] * size * (2 * hq * rows + 2 * case["heads"] * (rows + sum(ctx))),
                "flops": 4 * hq * case["d"] * case["nodes"] * (sum(ctx) + case["batch"])}
    hv, d, b, k = case["kheads"] * case["group"], case["d"], case["batch"], case["nodes"]
    chan = 2 * case["kheads"] * d + hv * d
    return {"bytes": 4 * b * (1 + k) * hv * d * d + b * k * (size * (chan + 2 * hv + hv * d) + 12 * chan) + 12 * b * chan + 16 * chan,
            "flops": 7 * b * k * hv * d * d}


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape, std=1.0, dtype=F32):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _cache(case, g, ctx, spare):
    """K and V pages and the block tables of rows with ctx tokens each: pages in no order, each row's own."""
    page = case["page"]
    need = [_pages(c, page) for c in ctx]
    width, total = max(need + [1]) + spare, sum(need) + 1
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(ctx), width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    shape = (total, case["heads"], page, case["d"])
    # keys have channels that stand out, as trained ones do
    k = _randn(g, *shape) + 0.5 * _randn(g, 1, case["heads"], 1, case["d"])
    return k.to(_type(case)), _randn(g, *shape, dtype=_type(case)), table


def _qkv(case, g, rows):
    """q, k and v rows: tensors of their own, or the three parts of one fused projection row."""
    hk, hq, d, dt = case["heads"], case["heads"] * case["group"], case["d"], _type(case)
    if not case["fused"]:
        return _randn(g, rows, hq, d, dtype=dt), _randn(g, rows, hk, d, dtype=dt), _randn(g, rows, hk, d, dtype=dt)
    both = _randn(g, rows, hq + 2 * hk, d, dtype=dt)
    return both[:, :hq], both[:, hq:hq + hk], both[:, hq + hk:]


def _attn_geometry(case, pages, width):
    import gated_deltanet_delta_amd as gdn
    return gdn.AttnGeometry(n_q_heads=case["heads"] * case.get("group", 1), n_kv_heads=case["heads"], d_head=case["d"], page_tokens=case["page"],
                            n_pages=pages, max_pages=width, max_tree=max(1, case.get("nodes", 1)), dtype=_type(case))


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = {"op": op, "case": case}
    if op == "plan":
        kv, new = _plan_lengths(case)
        page = case["page"]
        have = [_pages(c, page) for c in kv]
        fresh = sum(_pages(c + max(n, 0), page) - h for c, n, h in zip(kv, new, have))
        total = sum(have) + fresh + 17
        width = max(_pages(c + max(n, 0), page) for c, n in zip(kv, new)) + 2
        order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
        table = torch.full((len(kv), width), -1, dtype=torch.int32, device="cuda")
        at = torch.cumsum(torch.tensor([0] + have[:-1], device="cuda"), 0)
        col = torch.arange(width, device="cuda")[None]
        mine = col < torch.tensor(have, device="cuda")[:, None]
        table[mine] = order[(at[:, None] + col)[mine]]
        free = torch.full((total,), -1, dtype=torch.int32, device="cuda")
        n_free = total - sum(have)
        free[:n_free] = order[sum(have):]
        cap = sum(max(n, 0) for n in new) + case["pad"]
        out = lambda n: torch.empty(n, dtype=torch.int32, device="cuda")  # noqa: E731
        s.update(kv_len=_ints(kv), new_len=_ints(new), free=free, n_free=_ints([n_free]), table=table, cu=out(len(kv) + 1), slot_map=out(cap),
                 position=out(cap), kv_out=out(len(kv)), n_free_out=out(1))
        if own:
            s["geom"] = _attn_geometry(dict(heads=1, d=64, page=page, dtype="bf16"), total, width)
    elif op == "write":
        n, page = case["tokens"], case["page"]
        pages = _pages(n, page) + 3
        where = torch.randperm(pages, generator=g, device="cuda")
        t = torch.arange(n, device="cuda") + page // 2  # the first token comes into a page that is half full
        shape = (pages, case["heads"], page, case["d"])
        _, k, v = _qkv(dict(case, group=2), g, n)
        s.update(slot_map=(where[t // page] * page + t % page).to(torch.int32), k=k, v=v, k_cache=_randn(g, *shape, dtype=_type(case)),
                 v_cache=_randn(g, *shape, dtype=_type(case)))
        if own:
            import gated_deltanet_delta_amd as gdn
            s["geom"] = _attn_geometry(case, pages, pages)
            s["cache"] = gdn.KVCache(s["k_cache"], s["v_cache"])
    elif op == "prefill":
        new, ctx = _two(case)
        q, k, v = _qkv(case, g, sum(new))
        kc, vc, table = _cache(case, g, ctx, 1)
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        s.update(q=q, k=k, v=v, k_cache=kc, v_cache=vc, table=table, cu=_ints(cu), ctx=_ints(ctx), o=torch.empty(q.shape, dtype=q.dtype, device="cuda"))
        if own:
            import gated_deltanet_delta_amd as gdn
            s["geom"] = _attn_geometry(case, kc.shape[0], table.shape[1])
            s["cache"] = gdn.KVCache(kc, vc) if any(ctx) else None
            s["workspace"] = gdn.alloc_attn_prefill_workspace(s["geom"], sum(new), len(new))
    elif op == "tree":
        b, n = case["batch"], case["nodes"]
        ctx = _spread(case["ctx_lo"], case["ctx_hi"], b)
        q, k, v = _qkv(case, g, b * n)
        kc, vc, table = _cache(case, g, ctx, 2)
        s.update(q=q.unflatten(0, (b, n)), k=k.unflatten(0, (b, n)), v=v.unflatten(0, (b, n)), k_cache=kc, v_cache=vc, table=table, ctx=_ints(ctx),
                 parent=_parents(g, b, n), o=torch.empty((b, n) + tuple(q.shape[1:]), dtype=q.dtype, device="cuda"))
        if own:
            import gated_deltanet_delta_amd as gdn
            s["geom"] = _attn_geometry(case, kc.shape[0], table.shape[1])
            s["cache"] = gdn.KVCache(kc, vc)
            s["workspace"] = gdn.alloc_attn_tree_workspace(s["geom"], b, n)
    else:
        b, n, hk, d, dt = case["batch"], case["nodes"], case["kheads"], case["d"], _type(case)
        hv = hk * case["group"]
        chan, slots = 2 * hk * d + hv * d, b * (n + 1)
        ring = 1 << (n + 2).bit_length()
        perm = torch.randperm(slots, generator=g, device="cuda").to(torch.int32)
        pos = torch.zeros(slots, 32, dtype=torch.int32, device="cuda")
        pos[:, 0] = torch.randint(0, 4096, (slots,), generator=g, device="cuda", dtype=torch.int32) * 65536
        s.update(state=_randn(g, slots, hv, d, d, std=0.02), conv_state=_randn(g, slots, ring, chan, std=0.1), conv_pos=pos,
                 conv_w=_randn(g, chan, 4, std=0.5), x=_randn(g, b, n, chan, dtype=dt), a=_randn(g, b, n, hv, dtype=dt), b=_randn(g, b, n, hv, dtype=dt),
                 slot=perm[:b].contiguous(), snap=perm[b:].view(b, n).contiguous(), parent=_parents(g, b, n),
                 o=torch.empty(b, n, hv, d, dtype=dt, device="cuda"))
        if own:
            import gated_deltanet_delta_amd as gdn
            s["geom"] = gdn.Geometry(n_k_heads=hk, n_v_heads=hv, d_k=d, d_v=d, conv_ring=ring, max_draft=n, n_slots=slots, dtype=dt)
            s["pool"] = gdn.SlotPool(s["state"], s["conv_state"], pos)
    return s


def _parents(g, b, n):
    """A tree of n nodes a row: every node hangs from an earlier one or (-1) from the committed tokens."""
    j = torch.arange(n, device="cuda")
    return (torch.floor(torch.rand(b, n, generator=g, device="cuda") * (j + 1)) - 1).to(torch.int32).clamp(max=n - 2).contiguous()


# ----------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------

def run(state):
    op, s = state["op"], state
    if own:
        import gated_deltanet_delta_amd as gdn
        if op == "plan":
            gdn.kv_plan(s["geom"], s["kv_len"], s["new_len"], s["free"], s["n_free"], s["table"], s["cu"], s["slot_map"], s["position"], s["kv_out"],
                        s["n_free_out"])
            return [s[n] for n in ("table", "free", "cu", "slot_map", "position", "kv_out", "n_free_out")]
        if op == "write":
            gdn.kv_write(s["geom"], s["cache"], s["k"], s["v"], s["slot_map"])
            return [s["k_cache"], s["v_cache"]]
        if op == "prefill":
            paged = {} if s["cache"] is None else dict(cache=s["cache"], block_table=s["table"], ctx_len=s["ctx"])
            gdn.attn_prefill(s["geom"], s["q"], s["k"], s["v"], s["cu"], s["o"], s["workspace"], **paged)
            return s["o"]
        if op == "tree":
            gdn.attn_tree(s["geom"], s["cache"], s["table"], s["ctx"], s["q"], s["k"], s["v"], s["parent"], s["o"], s["workspace"])
            return s["o"]
        gdn.verify_tree_slots(s["geom"], s["pool"], s["x"], s["a"], s["b"], s["conv_w"], s["slot"], s["parent"], s["snap"], s["o"])
        return [s["o"], s["state"], s["conv_state"], s["conv_pos"]]
    return {"plan": _plan, "write": _write, "prefill": _prefill, "tree": _tree, "vtree": _vtree}[op](s)


def _plan(s):
    page = s["case"]["page"]
    kv, new, f0 = s["kv_len"].long(), s["new_len"].long(), s["n_free"].long()
    n = new.clamp(min=0)
    have = (kv + page - 1) // page
    need = torch.where(new < 0, 0, (kv + n + page - 1) // page - have)
    gone = torch.where(new < 0, have, 0)
    cum_need, cum_gone, cum_n = need.cumsum(0), gone.cumsum(0), n.cumsum(0)
    last = kv.numel() - 1
    # the free stack, with the leaving rows' pages on top
    r = torch.arange(s["free"].numel(), device="cuda") - f0
    row = torch.searchsorted(cum_gone, r, right=True).clamp(max=last)
    at = (r - (cum_gone - gone)[row]).clamp(0, s["table"].shape[1] - 1)
    free = torch.where((r >= 0) & (r < cum_gone[-1:]), s["table"][row, at], s["free"])
    top = f0 + cum_gone[-1:]
    # new pages from the top of the stack down, rows in order
    j = torch.arange(s["table"].shape[1], device="cuda")[None] - have[:, None]
    m = (cum_need - need)[:, None] + j
    table = torch.where((j >= 0) & (j < need[:, None]), free[(top - 1 - m).clamp(0, free.numel() - 1)], s["table"])
    t = torch.arange(s["slot_map"].numel(), device="cuda")
    row = torch.searchsorted(cum_n, t, right=True).clamp(max=last)
    fits = t < cum_n[-1:]
    pos = torch.where(fits, kv[row] + t - (cum_n - n)[row], 0)
    slots = torch.where(fits, table[row, pos // page].long() * page + pos % page, -1)
    cu = torch.cat([torch.zeros_like(f0), cum_n])
    out = (table, free, cu, slots, pos, torch.where(new < 0, 0, kv + n), top - cum_need[-1:])
    return [v.to(torch.int32) for v in out]


def _write(s):
    page = s["case"]["page"]
    at = s["slot_map"].long()
    s["k_cache"][at // page, :, at % page] = s["k"]
    s["v_cache"][at // page, :, at % page] = s["v"]
    return [s["k_cache"], s["v_cache"]]


def _softmax_product(logits, v):
    p = torch.exp(logits - logits.amax(-1, keepdim=True))
    return (p @ v) / p.sum(-1, keepdim=True)


def _rows_of(cache, table, count):
    """The first `count` cached rows of one request: [heads][count][d], in 32 bits."""
    page = cache.shape[2]
    got = cache[table[:_pages(count, page)].long()].transpose(0, 1)
    return got.flatten(1, 2)[:, :count].float()


def _prefill(s):
    case = s["case"]
    new, ctx = _two(case)
    hk, group, d = case["heads"], case["group"], case["d"]
    scale, at, block = 1.0 / math.sqrt(d), 0, 1024
    for i, (n, c) in enumerate(zip(new, ctx)):
        k = torch.cat([_rows_of(s["k_cache"], s["table"][i], c), s["k"][at:at + n].transpose(0, 1).float()], 1)
        v = torch.cat([_rows_of(s["v_cache"], s["table"][i], c), s["v"][at:at + n].transpose(0, 1).float()], 1)
        for lo in range(0, n, block):
            hi = min(n, lo + block)
            q = s["q"][at + lo:at + hi].float().unflatten(1, (hk, group)).permute(1, 2, 0, 3).flatten(1, 2)
            logits = (q @ k[:, :c + hi].transpose(1, 2)) * scale
            ahead = torch.arange(c + hi, device="cuda")[None] > c + torch.arange(lo, hi, device="cuda")[:, None]
            logits = logits.unflatten(1, (group, hi - lo)).masked_fill(ahead, -math.inf).flatten(1, 2)
            o = _softmax_product(logits, v[:, :c + hi]).unflatten(1, (group, hi - lo))
            s["o"][at + lo:at + hi] = o.permute(2, 0, 1, 3).flatten(1, 2).to(s["o"].dtype)
        at += n
    return s["o"]


def _tree(s):
    case = s["case"]
    b, n, hk, group, d, page = (case[x] for x in ("batch", "nodes", "heads", "group", "d", "page"))
    wide = _pages(case["ctx_hi"], page)
    table = s["table"][:, :wide].long().clamp(min=0)
    cached = [c[table].permute(0, 2, 1, 3, 4).flatten(2, 3).float() for c in (s["k_cache"], s["v_cache"])]
    q = s["q"].float().unflatten(2, (hk, group)).permute(0, 2, 3, 1, 4).flatten(2, 3)  # [b][hk][group n][d]
    scale = 1.0 / math.sqrt(d)
    outside = torch.arange(table.shape[1] * page, device="cuda")[None] >= s["ctx"][:, None]
    logits = ((q @ cached[0].transpose(2, 3)) * scale).masked_fill(outside[:, None, None], -math.inf)
    k, v = (s[x].float().transpose(1, 2) for x in ("k", "v"))
    # the nodes on each node's path: powers of (identity + parent matrix)
    path = torch.eye(n, device="cuda") + (s["parent"][:, :, None] == torch.arange(n, device="cuda")).float()
    for _ in range(max(1, (n - 1).bit_length())):
        path = ((path @ path) > 0).float()
    drafts = ((q @ k.transpose(2, 3)) * scale).unflatten(2, (group, n)).masked_fill(path[:, None, None] == 0, -math.inf).flatten(2, 3)
    o = _softmax_product(torch.cat([logits, drafts], -1), torch.cat([cached[1], v], 2))
    return o.unflatten(2, (group, n)).permute(0, 3, 1, 2, 4).flatten(2, 3).to(s["o"].dtype)


def _vtree(s):
    case = s["case"]
    b, n, hk, group, d = (case[x] for x in ("batch", "nodes", "kheads", "group", "d"))
    ring, hv = s["conv_state"].shape[1], hk * group
    rows, slot, snap = torch.arange(b, device="cuda"), s["slot"].long(), s["snap"].long()
    pos = (s["conv_pos"][slot, 0].long() & 0xFFFFFFFF) >> 16
    back = torch.arange(-3, 0, device="cuda")
    hist = [s["conv_state"][slot[:, None], (pos[:, None] + back) % ring]]  # window before each node's children: first the committed one
    states, depths = [s["state"][slot]], [torch.zeros_like(pos)]
    out = []
    for j in range(n):
        up = s["parent"][:, j].long() + 1
        h = torch.stack(hist, 1)[rows, up]
        S = torch.stack(states, 1)[rows, up]
        depth = torch.stack(depths, 1)[rows, up] + 1
        window = torch.cat([h, s["x"][:, j, None].float()], 1)  # [b][4][chan]
        y = (window * s["conv_w"].t()).sum(1)
        y = y / (1 + torch.exp(-y))
        q, k = (y[:, i * hk * d:(i + 1) * hk * d].view(b, hk, d) for i in (0, 1))
        q, k = (t / torch.sqrt((t * t).sum(-1, keepdim=True) + 1e-6) for t in (q, k))
        q, k = (t.repeat_interleave(group, 1) for t in (q, k))
        v = y[:, 2 * hk * d:].view(b, hv, d)
        alpha = 1 / (1 + torch.exp(s["a"][:, j].float()))[..., None]
        beta = 1 / (1 + torch.exp(-s["b"][:, j].float()))[..., None]
        u = beta * (v - alpha * (S * k[:, :, None]).sum(-1))
        S = alpha[..., None] * S + u[..., None] * k[:, :, None]
        out.append((S * q[:, :, None]).sum(-1))
        hist.append(window[:, 1:])
        states.append(S)
        depths.append(depth)
        s["state"][snap[:, j]] = S
        s["conv_state"][snap[:, j][:, None], (pos + depth)[:, None].add(back) % ring] = window[:, 1:]
        s["conv_pos"][snap[:, j], 0] = ((pos + depth) << 16).to(torch.int32)
    return [torch.stack(out, 1).to(s["o"].dtype), s["state"], s["conv_state"], s["conv_pos"]]


# ----------------------------------------------------------------------------
# the definitions in 64 bits
# ----------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "plan":
        return None  # whole numbers only
    if op == "write":
        out = []
        for rows, cache in ((s["k"], s["k_cache"]), (s["v"], s["v_cache"])):
            flat = cache.double().transpose(1, 2).flatten(0, 1)  # [cache slot][head][d]
            flat.index_copy_(0, s["slot_map"].long(), rows.double())
            out.append(flat.unflatten(0, (cache.shape[0], cache.shape[2])).transpose(1, 2).contiguous())
        return out
    if op == "vtree":
        return _exact_vtree(case, s)
    hk, group, d = case["heads"], case["group"], case["d"]
    o = torch.empty(s["o"].shape, dtype=torch.float64, device="cuda")
    if op == "prefill":
        new, ctx = _two(case)
        at = 0
        for i, (n, c) in enumerate(zip(new, ctx)):
            for h in range(hk * group):
                k = torch.cat([_exact_rows(s["k_cache"], s["table"][i], c, h // group), s["k"][at:at + n, h // group].double()])
                v = torch.cat([_exact_rows(s["v_cache"], s["table"][i], c, h // group), s["v"][at:at + n, h // group].double()])
                for lo in range(0, n, 4096):
                    hi = min(n, lo + 4096)
                    seen = torch.ones(hi - lo, c + n, dtype=torch.bool, device="cuda").tril(c + lo)
                    o[at + lo:at + hi, h] = _exact_attention(s["q"][at + lo:at + hi, h].double(), k, v, seen)
            at += n
        return o
    parent, ctx = s["parent"].tolist(), s["ctx"].tolist()
    n = case["nodes"]
    for i in range(case["batch"]):
        seen = torch.zeros(n, ctx[i] + n, dtype=torch.bool)
        seen[:, :ctx[i]] = True
        for j in range(n):
            at = j
            while at >= 0:
                seen[j, ctx[i] + at] = True
                at = parent[i][at]
        seen = seen.cuda()
        for h in range(hk):
            k = torch.cat([_exact_rows(s["k_cache"], s["table"][i], ctx[i], h), s["k"][i, :, h].double()])
            v = torch.cat([_exact_rows(s["v_cache"], s["table"][i], ctx[i], h), s["v"][i, :, h].double()])
            for e in range(h * group, (h + 1) * group):
                o[i, :, e] = _exact_attention(s["q"][i, :, e].double(), k, v, seen)
    return o


def _exact_rows(cache, table, count, head):
    page = cache.shape[2]
    t = torch.arange(count, device="cuda")
    return cache[table.long()[t // page], head, t % page].double()


def _exact_attention(q, k, v, seen):
    logits = (q @ k.t()) / math.sqrt(q.shape[1])
    logits = torch.where(seen, logits, torch.full_like(logits, -math.inf))
    return torch.exp(logits - torch.logsumexp(logits, 1, keepdim=True)) @ v


def _exact_vtree(case, s):
    """S = alpha S' (I - beta k k^T) + beta v k^T with the matrix formed, one row of the batch at a time."""
    b, n, hk, group, d = (case[x] for x in ("batch", "nodes", "kheads", "group", "d"))
    ring, hv = s["conv_state"].shape[1], hk * group
    state, conv, pos = s["state"].double(), s["conv_state"].double(), s["conv_pos"].clone()
    o = torch.empty(b, n, hv, d, dtype=torch.float64, device="cuda")
    slot, snap, parent, word = s["slot"].tolist(), s["snap"].tolist(), s["parent"].tolist(), s["conv_pos"][:, 0].tolist()
    w, eye = s["conv_w"].double(), torch.eye(d, dtype=torch.float64, device="cuda")
    for i in range(b):
        p = (word[slot[i]] & 0xFFFFFFFF) >> 16
        start = [conv[slot[i], (p + e) % ring] for e in (-3, -2, -1)]
        S0 = state[slot[i]].clone()
        for j in range(n):
            path, at = [], j
            while at >= 0:
                path.insert(0, at)
                at = parent[i][at]
            inputs = start + [s["x"][i, e].double() for e in path]
            y = sum(w[:, t] * inputs[len(inputs) - 4 + t] for t in range(4))
            y = y * torch.sigmoid(y)
            q, k, v = y[:hk * d].view(hk, d), y[hk * d:2 * hk * d].view(hk, d), y[2 * hk * d:].view(hv, d)
            q, k = ((t * torch.rsqrt((t * t).sum(1, keepdim=True) + 1e-6)).repeat_interleave(group, 0) for t in (q, k))
            alpha = torch.exp(-torch.nn.functional.softplus(s["a"][i, j].double(), threshold=1e9))[:, None, None]
            beta = torch.sigmoid(s["b"][i, j].double())[:, None, None]
            S = S0 if parent[i][j] < 0 else state[snap[i][parent[i][j]]]
            S = alpha * torch.bmm(S, eye - beta * (k[:, :, None] * k[:, None, :])) + beta * (v[:, :, None] * k[:, None, :])
            o[i, j] = torch.bmm(S, q[:, :, None])[:, :, 0]
            state[snap[i][j]] = S
            for t in range(3):
                conv[snap[i][j], (p + len(path) - 3 + t) % ring] = inputs[len(inputs) - 3 + t]
            pos[snap[i][j], 0] = ((p + len(path)) << 16) if (p + len(path)) < 32768 else ((p + len(path)) << 16) - (1 << 32)
    return [o, state, conv, pos]
