"""Cases of the operators around the paged KV cache of a hybrid stack's attention layers: what q and k go through before
they enter it, and what keeps it within a budget of tokens:

  rope     rotary positions of q and k, the rotated k and the v going into their cache slots in the same pass;
  weights  the attention weight that the newest queries of a request give to each of its cached tokens, added up;
  evict    which cached tokens stay within a row's budget, by that weight, and the moves that close the gaps;
  move     the K and V rows of those moves.

With ``own`` false ``run`` computes them from elementary torch operations in 32 bits (angles in 64); with it true it makes the
calls of gated_deltanet_delta_amd.  ``exact`` computes the same results in 64 bits, from the definitions.
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
        # one token of each of four requests far into their contexts: a quarter of the head rotates, k and v go to the cache
        dict(name="rope decode step, 4 tokens", op="rope", tokens=4, heads=4, group=6, d=256, rot=64, layout="half", scaling="none", far=262144,
             page=16, dtype="bf16", fused=True, cache=True, inverse=False),
        # a long prompt beyond the trained context, frequencies scaled by parts, pages of the 528 tokens that hybrid cache managers use
        dict(name="rope prompt, 32771 tokens", op="rope", tokens=32771, heads=4, group=6, d=256, rot=64, layout="half", scaling="parts", far=100000,
             page=528, dtype="bf16", fused=True, cache=True, inverse=False),
        # whole heads in the interleaved layout, no cache behind them (a prompt that is attended and not kept)
        dict(name="rope whole heads, 5003 tokens", op="rope", tokens=5003, heads=8, group=4, d=128, rot=128, layout="pairs", scaling="base", far=30000,
             page=16, dtype="bf16", fused=False, cache=False, inverse=False),
        # the transposed rotation of a gradient, fp32
        dict(name="rope transposed, fp32, 777 tokens", op="rope", tokens=777, heads=2, group=4, d=64, rot=48, layout="half", scaling="linear", far=5000,
             page=16, dtype="f32", fused=False, cache=False, inverse=True),
        # the decode step of four requests at 8K: every step adds its weights
        dict(name="weights decode step, 4 x 8K", op="weights", batch=4, n=1, ctx_lo=8100, ctx_hi=8192, heads=4, group=6, d=256, page=16, dtype="bf16"),
        # the last 32 tokens of long prompts judge what is kept of them
        dict(name="weights of 32 tokens, 4 x 100K", op="weights", batch=4, n=32, ctx_lo=80000, ctx_hi=120000, heads=4, group=6, d=256, page=528, dtype="bf16"),
        # many requests of ragged lengths, four tokens accepted in each
        dict(name="weights of 4 tokens, 64 ragged", op="weights", batch=64, n=4, ctx_lo=33, ctx_hi=16384, heads=8, group=4, d=128, page=16, dtype="bf16"),
        # four requests that have outgrown their budget by a few pages
        dict(name="evict 4 rows, 8K by 128", op="evict", batch=4, ctx_lo=8192, ctx_hi=8192, budget=8064, page=16, sink=4, recent=512, before=True),
        # a batch of prompts cut to a common budget after their prefill
        dict(name="evict 64 ragged prompts", op="evict", batch=64, ctx_lo=500, ctx_hi=16384, budget=2048, page=16, sink=4, recent=256, before=False),
        # long contexts kept at a fixed size
        dict(name="evict 3 rows, 120K to 16K", op="evict", batch=3, ctx_lo=110000, ctx_hi=120000, budget=16384, page=528, sink=64, recent=4096, before=True),
        # the rows that the first of these moves, in one layer
        dict(name="move 4 rows, 117 tokens", op="move", batch=4, moves_lo=100, moves_hi=117, heads=4, d=256, page=16, dtype="bf16"),
        # those of the ragged prompts
        dict(name="move 64 rows, up to 2048 tokens", op="move", batch=64, moves_lo=300, moves_hi=2048, heads=8, d=128, page=16, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(("rope", "rope", "weights", "weights", "evict", "move"))
    page = rng.choice((16, 16, 32, 64, 528))
    dtype = rng.choice(("bf16", "bf16", "bf16", "f32"))
    heads, group, d = rng.choice((1, 2, 4, 8)), rng.choice((1, 2, 3, 4, 6, 8)), rng.choice((64, 128, 256))
    if op == "rope":
        row = heads * (group + 2) * d * (2 if dtype == "bf16" else 4)
        return dict(op=op, tokens=_log(rng, 1, min(32000, int(5e8 / row))), heads=heads, group=group, d=d, rot=16 * rng.randint(1, d // 16),
                    layout=rng.choice(("half", "pairs")), scaling=rng.choice(("none", "linear", "base", "parts")), far=_log(rng, 64, 1000000), page=page,
                    dtype=dtype, fused=rng.random() < 0.5, cache=rng.random() < 0.6, inverse=rng.random() < 0.2)
    if op == "weights":
        batch = _log(rng, 1, 64)
        n = _log(rng, 1, 64)
        most = max(128, int(min(3e8 / (batch * heads * d), (1.5e11 if dtype == "bf16" else 1.5e10) / (2 * batch * n * heads * group * d))))
        lo, hi = sorted((_log(rng, n, max(n, min(120000, most))), _log(rng, n, max(n, min(120000, most)))))
        return dict(op=op, batch=batch, n=n, ctx_lo=lo, ctx_hi=hi, heads=heads, group=group, d=d, page=page, dtype=dtype)
    if op == "evict":
        batch = _log(rng, 1, 64)
        most = min(120000, 1000000 // batch)
        lo, hi = sorted((_log(rng, 16, most), _log(rng, 16, most)))
        budget = _log(rng, 8, hi)
        sink = rng.choice((0, 1, 4, 64))
        return dict(op=op, batch=batch, ctx_lo=lo, ctx_hi=hi, budget=budget, page=page, sink=min(sink, budget // 4),
                    recent=int(budget * rng.choice((0.0, 0.1, 0.4))), before=rng.random() < 0.5)
    batch = _log(rng, 1, 64)
    lo, hi = sorted((_log(rng, 1, 2048), _log(rng, 1, min(2048, max(1, int(2.5e8 / (batch * heads * d)))))))
    return dict(op=op, batch=batch, moves_lo=lo, moves_hi=hi, heads=heads, d=d, page=page, dtype=dtype)


def _type(case):
    return BF16 if case["dtype"] == "bf16" else F32


def _size(case):
    return 2 if case["dtype"] == "bf16" else 4


def _spread(lo, hi, n):
    """n lengths between lo and hi, spread over their logarithm, the same for every seed."""
    return [max(lo, min(hi, int(round(lo * (hi / lo) ** ((0.35 + 0.6180339887 * i) % 1.0))))) for i in range(n)]


def _pages(tokens, page):
    return -(-tokens // page)


def _evicts(case):
    """(cached tokens, budget) of every row; every fifth row's budget is its own length: nothing to do."""
    ctx = _spread(case["ctx_lo"], case["ctx_hi"], case["batch"])
    return ctx, [c if i % 5 == 4 else case["budget"] for i, c in enumerate(ctx)]


def work(case):
    op = case["op"]
    if op == "rope":
        rows = case["heads"] * (2 * case["group"] + 2) + (case["heads"] * 3 if case["cache"] else 0)
        return {"bytes": case["tokens"] * (rows * case["d"] * _size(case) + 8),
                "flops": case["tokens"] * case["heads"] * (case["group"] + 1) * case["rot"] * 3}
    if op == "weights":
        keys = sum(_spread(case["ctx_lo"], case["ctx_hi"], case["batch"]))
        q = case["batch"] * case["n"] * case["heads"] * case["group"] * case["d"] * _size(case)
        return {"bytes": keys * (case["heads"] * case["d"] * _size(case) + 8) + q,
                "flops": 2 * case["n"] * case["heads"] * case["group"] * case["d"] * keys}
    if op == "evict":
        ctx, budget = _evicts(case)
        moves = sum(min(b, c - b) for c, b in zip(ctx, budget) if b < c)
        return {"bytes": sum(8 * c + 8 * min(b, c) for c, b in zip(ctx, budget)) + 8 * moves + 28 * case["batch"], "flops": 0}
    moves = sum(_spread(case["moves_lo"], case["moves_hi"], case["batch"]))
    return {"bytes": moves * (4 * case["heads"] * case["d"] * _size(case) + 8), "flops": 0}


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape, std=1.0, dtype=F32):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _tables(g, need, width, spare):
    """Block tables of rows that hold need[i] pages each: pages in no order, each row's own; the pages left over."""
    total = sum(need) + spare
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(need), width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    return table, order[at:], total


def _attn_geometry(case, pages, width):
    import gated_deltanet_delta_amd as gdn
    heads = case.get("heads", 1)
    return gdn.AttnGeometry(n_q_heads=heads * case.get("group", 1), n_kv_heads=heads, d_head=case.get("d", 64), page_tokens=case["page"],
                            n_pages=pages, max_pages=width, max_tree=max(1, case.get("n", 1)), dtype=_type(case) if "dtype" in case else BF16)


# frequencies of the scaled forms: eight times the context, of 32768 tokens where a form asks for it
_BASE, _FACTOR, _CONTEXT, _LOW, _HIGH = 1e6, 8.0, 32768, 1.0, 32.0


def _frequencies(case):
    """Radians per position of every pair, as 64-bit floats on the host."""
    half, scaling, base = case["rot"] // 2, case["scaling"], _BASE
    if scaling == "base" and half > 1:
        base *= _FACTOR ** (half / (half - 1))
    f = [base ** (-i / half) for i in range(half)]
    if scaling == "linear":
        f = [x / _FACTOR for x in f]
    if scaling == "parts":
        ramp = [min(1.0, max(0.0, (_CONTEXT * x / (2 * math.pi) - _LOW) / (_HIGH - _LOW))) for x in f]
        f = [x * ((1 - r) / _FACTOR + r) for x, r in zip(f, ramp)]
    return f


def _amplitude(case):
    return 0.1 * math.log(_FACTOR) + 1.0 if case["scaling"] == "parts" else 1.0


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = {"op": op, "case": case}
    if op == "rope":
        n, page, hk, hq, d, dt = case["tokens"], case["page"], case["heads"], case["heads"] * case["group"], case["d"], _type(case)
        if case["fused"]:
            both = _randn(g, n, hq + 2 * hk, d, dtype=dt)
            q, k, v = both[:, :hq], both[:, hq:hq + hk], both[:, hq + hk:]
        else:
            q, k, v = (_randn(g, n, h, d, dtype=dt) for h in (hq, hk, hk))
        # a prompt's positions follow one another; the tokens of a decode step are each somewhere
        first = torch.randint(0, case["far"], (n if n < 64 else 1,), generator=g, device="cuda")
        position = (first if n < 64 else first + torch.arange(n, device="cuda")).to(torch.int32)
        s.update(q=q, k=k, v=v, position=position, q_out=torch.empty(n, hq, d, dtype=dt, device="cuda"),
                 k_out=torch.empty(n, hk, d, dtype=dt, device="cuda"), freq=torch.tensor(_frequencies(case), dtype=torch.float64, device="cuda"))
        pages = _pages(n, page) + 3
        if case["cache"]:
            where = torch.randperm(pages, generator=g, device="cuda")
            t = torch.arange(n, device="cuda") + page // 2  # the first token comes into a page that is half full
            shape = (pages, hk, page, d)
            s.update(slot_map=(where[t // page] * page + t % page).to(torch.int32), k_cache=_randn(g, *shape, dtype=dt), v_cache=_randn(g, *shape, dtype=dt))
        if own:
            import gated_deltanet_delta_amd as gdn
            s["geom"] = _attn_geometry(case, pages, pages)
            s["rope"] = gdn.Rope(rot_dims=case["rot"], layout=case["layout"], base=_BASE, scaling=case["scaling"], factor=_FACTOR, context=_CONTEXT,
                                 low=_LOW, high=_HIGH, amplitude=_amplitude(case), inverse=case["inverse"])
            s["turns"] = gdn.rope_turns(s["rope"])
            s["kv"] = gdn.KVCache(s["k_cache"], s["v_cache"]) if case["cache"] else None
    elif op == "weights":
        b, n, page, hk, hq, d, dt = case["batch"], case["n"], case["page"], case["heads"], case["heads"] * case["group"], case["d"], _type(case)
        ctx = _spread(case["ctx_lo"], case["ctx_hi"], b)
        need = [_pages(c, page) for c in ctx]
        table, _, total = _tables(g, need, max(need) + 1, 1)
        # keys have channels that stand out, as trained ones do
        k = (_randn(g, total, hk, page, d) + 0.5 * _randn(g, 1, hk, 1, d)).to(dt)
        width = max(ctx) + 5
        score = torch.rand(b, width, generator=g, device="cuda") ** 8
        s.update(q=_randn(g, b, n, hq, d, std=1.5, dtype=dt), k_cache=k, table=table, kv_len=_ints(ctx), have=_ints([c - n for c in ctx]), score=score,
                 score_out=torch.zeros_like(score))
        if own:
            import gated_deltanet_delta_amd as gdn
            s["geom"] = _attn_geometry(case, total, table.shape[1])
            s["workspace"] = gdn.alloc_attn_weights_workspace(s["geom"], b, n, width)
    elif op == "evict":
        b, page = case["batch"], case["page"]
        ctx, budget = _evicts(case)
        need = [_pages(c, page) for c in ctx]
        table, rest, total = _tables(g, need, max(need) + 1, 7)
        free = torch.full((total,), -1, dtype=torch.int32, device="cuda")
        free[:7] = rest
        width = max(ctx) + 3
        # few tokens hold most of the weight, many hold none at all
        score = (torch.rand(b, width, generator=g, device="cuda") - 0.3).clamp(min=0) ** 6
        settled = [c * 7 // 8 if case["before"] else 0 for c in ctx]
        gone = [c // 3 if case["before"] else 0 for c in ctx]
        # the positions that earlier evictions left, each once, in no order
        pos = torch.full((b, width), -1, dtype=torch.int32, device="cuda")
        for i in range(b):
            pos[i, :settled[i]] = torch.randperm(settled[i] + gone[i], generator=g, device="cuda")[:settled[i]].to(torch.int32)
        moves = max([min(x, c - x) for c, x in zip(ctx, budget) if x < c] + [1])
        out = lambda *shape: torch.zeros(*shape, dtype=torch.int32, device="cuda")  # noqa: E731
        s.update(kv_len=_ints(ctx), budget=_ints(budget), score=score, token_pos=pos, row_state=_ints([[x, y] for x, y in zip(settled, gone)]), table=table,
                 free=free, n_free=_ints([7]), score_out=torch.zeros_like(score), token_pos_out=out(b, width), kv_len_out=out(b), row_state_out=out(b, 2),
                 n_free_out=out(1), move_src=out(b, moves), move_dst=out(b, moves), n_moves=out(b))
        if own:
            s["geom"] = _attn_geometry(case, total, table.shape[1])
    else:
        b, page, hk, d, dt = case["batch"], case["page"], case["heads"], case["d"], _type(case)
        moves = _spread(case["moves_lo"], case["moves_hi"], b)
        width = max(moves) + 3
        pages = _pages(2 * sum(moves), page) + 5
        # sources lie page by page behind one another, the gaps anywhere
        slots = torch.arange(pages * page, device="cuda")
        src, dst = slots[sum(moves):2 * sum(moves)], torch.randperm(sum(moves), generator=g, device="cuda")
        lists = torch.full((2, b, width), -1, dtype=torch.int32, device="cuda")
        at = 0
        for i, m in enumerate(moves):
            lists[0, i, :m], lists[1, i, :m] = src[at:at + m].to(torch.int32), dst[at:at + m].to(torch.int32)
            at += m
        shape = (pages, hk, page, d)
        s.update(move_src=lists[0].contiguous(), move_dst=lists[1].contiguous(), n_moves=_ints(moves), k_cache=_randn(g, *shape, dtype=dt),
                 v_cache=_randn(g, *shape, dtype=dt))
        if own:
            import gated_deltanet_delta_amd as gdn
            s["geom"] = _attn_geometry(case, pages, pages)
            s["kv"] = gdn.KVCache(s["k_cache"], s["v_cache"])
    return s


# ----------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------

_EVICT_OUT = ("score_out", "token_pos_out", "kv_len_out", "row_state_out", "n_free_out", "free", "move_src", "move_dst", "n_moves")


def run(state):
    op, s = state["op"], state
    if own:
        import gated_deltanet_delta_amd as gdn
        if op == "rope":
            paged = dict(v=s["v"], cache=s["kv"], slot_map=s["slot_map"]) if s["kv"] is not None else {}
            gdn.rope_rotate(s["geom"], s["rope"], s["turns"], s["position"], q=s["q"], k=s["k"], q_out=s["q_out"], k_out=s["k_out"], **paged)
            return [s["q_out"], s["k_out"]] + ([s["k_cache"], s["v_cache"]] if s["kv"] is not None else [])
        if op == "weights":
            gdn.attn_weights(s["geom"], s["k_cache"], s["table"], s["kv_len"], s["q"], s["score_out"], s["workspace"], score_in=s["score"],
                             have_len=s["have"])
            return s["score_out"]
        if op == "evict":
            gdn.evict_plan(s["geom"], s["kv_len"], s["budget"], s["score"], s["token_pos"], s["row_state"], s["table"], s["free"], s["n_free"],
                           s["score_out"], s["token_pos_out"], s["kv_len_out"], s["row_state_out"], s["n_free_out"], s["move_src"], s["move_dst"],
                           s["n_moves"], sink=s["case"]["sink"], recent=s["case"]["recent"])
            return [s[x] for x in _EVICT_OUT]
        gdn.kv_move(s["geom"], s["kv"], s["move_src"], s["move_dst"], s["n_moves"])
        return [s["k_cache"], s["v_cache"]]
    return {"rope": _rope, "weights": _weights, "evict": _evict, "move": _move}[op](s)


def _rope(s):
    case = s["case"]
    half, page = case["rot"] // 2, case["page"]
    angle = s["position"].double()[:, None] * s["freq"]
    if case["inverse"]:
        angle = -angle
    c, n = ((_amplitude(case) * f(angle)).float()[:, None] for f in (torch.cos, torch.sin))
    for x, out in ((s["q"], s["q_out"]), (s["k"], s["k_out"])):
        if case["layout"] == "half":
            a, b = x[..., :half].float(), x[..., half:2 * half].float()
            turned = torch.cat([a * c - b * n, a * n + b * c], -1)
        else:
            a, b = x[..., 0:2 * half:2].float(), x[..., 1:2 * half:2].float()
            turned = torch.stack([a * c - b * n, a * n + b * c], -1).flatten(-2)
        out[..., :2 * half] = turned.to(out.dtype)
        out[..., 2 * half:] = x[..., 2 * half:]
    if not case["cache"]:
        return [s["q_out"], s["k_out"]]
    at = s["slot_map"].long()
    s["k_cache"][at // page, :, at % page] = s["k_out"]
    s["v_cache"][at // page, :, at % page] = s["v"]
    return [s["q_out"], s["k_out"], s["k_cache"], s["v_cache"]]


def _weights(s):
    case = s["case"]
    n, hk, group, d, page = (case[x] for x in ("n", "heads", "group", "d", "page"))
    wide = s["table"].shape[1] - 1
    keys = s["k_cache"][s["table"][:, :wide].long().clamp(min=0)].permute(0, 2, 1, 3, 4).flatten(2, 3).float()  # [b][hk][key][d]
    q = s["q"].float().unflatten(2, (hk, group)).permute(0, 2, 1, 3, 4).flatten(2, 3)  # [b][hk][n group][d]
    logits = (q @ keys.transpose(2, 3)) * (1.0 / math.sqrt(d))
    j = torch.arange(wide * page, device="cuda")
    last = s["kv_len"][:, None] - n + torch.arange(n, device="cuda")  # the last key of each query
    outside = (j > last[:, :, None]).repeat_interleave(group, 1)[:, None]
    logits = logits.masked_fill_(outside, -math.inf)
    p = torch.exp(logits - logits.amax(-1, keepdim=True))
    total = (p / p.sum(-1, keepdim=True)).sum((1, 2))
    width = s["score"].shape[1]
    j = torch.arange(width, device="cuda")[None]
    total = torch.nn.functional.pad(total, (0, max(0, width - total.shape[1])))[:, :width]
    old = torch.where(j < s["have"][:, None], s["score"], 0.0)
    s["score_out"].copy_(torch.where(j < s["kv_len"][:, None], old + total, s["score_out"]))
    return s["score_out"]


def _evict(s):
    case = s["case"]
    page, width = case["page"], s["score"].shape[1]
    c, b = s["kv_len"].long()[:, None], s["budget"].long()[:, None]
    settled, gone = s["row_state"].long()[:, :1], s["row_state"].long()[:, 1:]
    b = torch.where((b >= 0) & (b < c), b, c)
    j = torch.arange(width, device="cuda")[None].expand(c.shape[0], -1)
    pos = torch.where(j < settled, s["token_pos"].long(), j + gone)
    first = (pos < case["sink"]) | (pos >= c + gone - case["recent"])
    order = torch.where(j < c, torch.where(first, math.inf, s["score"]), -math.inf).sort(dim=1, descending=True, stable=True).indices
    keep = torch.zeros_like(j, dtype=torch.bool).scatter_(1, order, j < b)
    hole, mover = (j < b) & ~keep, (j >= b) & keep
    count = hole.sum(1)
    lists = []
    for mark in (mover, hole):  # the indexes of each, in order, to the front
        lists.append(torch.where(mark, j, width).sort(1).values[:, :s["move_src"].shape[1]])
    m = torch.arange(s["move_src"].shape[1], device="cuda")[None]
    live = m < count[:, None]
    src, dst = (torch.where(live, x, 0) for x in lists)
    for value, out in ((s["score"], s["score_out"]), (pos.to(torch.int32), s["token_pos_out"])):
        moved = torch.where(j < b, value, out)
        at = torch.where(live, dst, width)
        out.copy_(torch.nn.functional.pad(moved, (0, 1)).scatter_(1, at, value.gather(1, src))[:, :width])
    for x, out in ((src, s["move_src"]), (dst, s["move_dst"])):
        out.copy_(torch.where(live, s["table"].long().gather(1, x // page) * page + x % page, -1).to(torch.int32))
    s["n_moves"].copy_(count)
    s["kv_len_out"].copy_(b[:, 0])
    s["row_state_out"].copy_(torch.cat([torch.where(b < c, b, settled), gone + c - b], 1))
    # pages behind the budget, rows in order, on top of the stack
    e = torch.arange(s["table"].shape[1], device="cuda")[None]
    left = (e >= (b + page - 1) // page) & (e < (c + page - 1) // page)
    at = torch.where(left, s["n_free"].long() + left.flatten().cumsum(0).view_as(left) - 1, s["free"].numel())
    s["free"].copy_(torch.nn.functional.pad(s["free"], (0, 1)).scatter_(0, at.flatten(), s["table"].flatten())[:-1])
    s["n_free_out"].copy_(s["n_free"] + left.sum())
    return [s[x] for x in _EVICT_OUT]


def _move(s):
    page = s["case"]["page"]
    live = torch.arange(s["move_src"].shape[1], device="cuda")[None] < s["n_moves"][:, None]
    src, dst = s["move_src"][live].long(), s["move_dst"][live].long()
    for cache in (s["k_cache"], s["v_cache"]):
        cache[dst // page, :, dst % page] = cache[src // page, :, src % page]
    return [s["k_cache"], s["v_cache"]]


# ----------------------------------------------------------------------------
# the definitions in 64 bits
# ----------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "weights": _exact_weights, "evict": _exact_evict, "move": _exact_move}[case["op"]](case, s)


def _exact_rope(case, s):
    """Every pair as a complex number, times A exp(i position f)."""
    rot, sign = case["rot"], -1.0 if case["inverse"] else 1.0
    turn = torch.polar(torch.full_like(s["freq"], _amplitude(case))[None].expand(case["tokens"], -1).contiguous(),
                       sign * torch.outer(s["position"].double(), s["freq"]))[:, None]
    out = []
    for x in (s["q"].double(), s["k"].double()):
        head = x[..., :rot]
        pairs = head.unflatten(-1, (2, rot // 2)).transpose(-1, -2) if case["layout"] == "half" else head.unflatten(-1, (rot // 2, 2))
        turned = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
        turned = turned.transpose(-1, -2).flatten(-2) if case["layout"] == "half" else turned.flatten(-2)
        out.append(torch.cat([turned, x[..., rot:]], -1))
    if case["cache"]:
        for rows, cache in ((out[1], s["k_cache"]), (s["v"].double(), s["v_cache"])):
            flat = cache.double().transpose(1, 2).flatten(0, 1)  # [cache slot][head][d]
            flat.index_copy_(0, s["slot_map"].long(), rows)
            out.append(flat.unflatten(0, (cache.shape[0], cache.shape[2])).transpose(1, 2).contiguous())
    return out


def _exact_weights(case, s):
    n, hk, group, d, page = (case[x] for x in ("n", "heads", "group", "d", "page"))
    out = s["score_out"].double()
    for i, c in enumerate(s["kv_len"].tolist()):
        t = torch.arange(c, device="cuda")
        total = torch.zeros(c, dtype=torch.float64, device="cuda")
        total[:c - n] = s["score"][i, :c - n].double()
        seen = torch.ones(n, c, dtype=torch.bool, device="cuda").tril(c - n)
        for h in range(hk):
            k = s["k_cache"][s["table"][i].long()[t // page], h, t % page].double()
            for e in range(group):
                logits = (s["q"][i, :, h * group + e].double() @ k.t()) / math.sqrt(d)
                logits = torch.where(seen, logits, torch.full_like(logits, -math.inf))
                total += torch.exp(logits - torch.logsumexp(logits, 1, keepdim=True)).sum(0)
        out[i, :c] = total
    return out


def _exact_evict(case, s):
    """Row by row on the host."""
    page, sink, recent = case["page"], case["sink"], case["recent"]
    score, pos, table, state = (s[x].tolist() for x in ("score", "token_pos", "table", "row_state"))
    out = {x: s[x].tolist() for x in _EVICT_OUT}
    stack = out["free"][:int(s["n_free"])]
    for i, (c, b) in enumerate(zip(s["kv_len"].tolist(), s["budget"].tolist())):
        settled, gone = state[i]
        where = [pos[i][j] if j < settled else j + gone for j in range(c)]
        left = list(range(c))
        if 0 <= b < c:
            order = sorted(range(c), key=lambda j: (0 if where[j] < sink or where[j] >= c + gone - recent else 1, -score[i][j], j))
            kept = set(order[:b])
            movers = [j for j in range(b, c) if j in kept]
            holes = [j for j in range(b) if j not in kept]
            left = list(range(b))
            for src, dst in zip(movers, holes):
                left[dst] = src
            stack += table[i][_pages(b, page):_pages(c, page)]
            state[i] = [b, gone + c - b]
        else:
            movers, holes = [], []
        out["score_out"][i][:len(left)] = [score[i][j] for j in left]
        out["token_pos_out"][i][:len(left)] = [where[j] for j in left]
        for name, at in (("move_src", movers), ("move_dst", holes)):
            slots = [table[i][j // page] * page + j % page for j in at]
            out[name][i] = slots + [-1] * (len(out[name][i]) - len(slots))
        out["n_moves"][i], out["kv_len_out"][i], out["row_state_out"][i] = len(movers), len(left), state[i]
    out["free"][:len(stack)] = stack
    out["n_free_out"] = [len(stack)]
    return [torch.tensor(out[x], dtype=torch.float64 if x == "score_out" else torch.int32, device="cuda") for x in _EVICT_OUT]


def _exact_move(case, s):
    slots = [s[x][i, :m].tolist() for i, m in enumerate(s["n_moves"].tolist()) for x in ("move_src", "move_dst")]
    src, dst = (torch.tensor([x for one in slots[at::2] for x in one], device="cuda") for at in (0, 1))
    out = []
    for cache in (s["k_cache"], s["v_cache"]):
        flat = cache.double().transpose(1, 2).flatten(0, 1)  # [cache slot][head][d]
        flat[dst] = flat[src]
        out.append(flat.unflatten(0, (cache.shape[0], cache.shape[2])).transpose(1, 2).contiguous())
    return out
