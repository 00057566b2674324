"""A cache within a budget on the GPU: attention weights of cached tokens against the fp64 oracle, eviction plans against
plain loops, the moves bit for bit, and all of them run together with the rest of the attention layer's operators."""
import numpy as np
import pytest
import torch

import attn_harness as AH
from oracle import attn_oracle as ao
from oracle import cache_oracle as co

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


def _i32(a):
    return torch.as_tensor(np.ascontiguousarray(a)).to(torch.int32).cuda()


# ---------------------------------------------------------------- weights

def _weights_bound(w, old, q, keys, scale):
    """Elementwise bound of |got - (old + w)| for n queries of Hq heads over c keys, as attn_harness.tolerance has it: a
    logit is off by (D + 2) U A, A the largest scale sum |q_d k_d|, the exponential's argument and the maximum that is taken
    off by (2 + A) U: 2 (D + 5) U (A + 1) in a weight and its normaliser, whose sum over c keys adds c U and its logarithm
    4 U (A + 1) (an argument of the size of the logit, in two roundings each way); the sum over the n Hq queries
    (n Hq + 1) U; the addition to old U (old + w)."""
    c, D = keys.shape[0], keys.shape[-1]
    g = q.shape[1] // keys.shape[1]
    A = scale * float(np.max(np.sum(np.abs(q).max(axis=0) * np.repeat(np.abs(keys).max(axis=0), g, axis=0), axis=-1)))
    rel = (2 * (D + 5) + 4) * U * (A + 1) + c * U + (q.shape[0] * q.shape[1] + 1) * U
    return 1.02 * (rel * w + U * (old + w)) + 1e-30


def _weights_case(seed, ctx, n, n_row, Hq, Hk, D, page, dtype, width_extra=7, pad=0):
    m = AH.gdn()
    P = AH.Paged(seed, ctx, Hk, D, page, dtype)
    geom = m.AttnGeometry(n_q_heads=Hq, n_kv_heads=Hk, d_head=D, page_tokens=page, n_pages=P.n_pages, max_pages=P.width, max_tree=max(n, 1), dtype=dtype)
    g = torch.Generator().manual_seed(seed + 1)
    B = len(ctx)
    rows = (torch.randn(B * n, Hq * D + pad, generator=g) * 1.5).to(dtype)
    if n_row is not None:  # what lies behind a row's own queries is not read
        for i, r in enumerate(n_row):
            rows[i * n + r:(i + 1) * n] = float("nan")
    q = rows[:, :Hq * D].unflatten(1, (Hq, D)).unflatten(0, (B, n))
    qd = rows.cuda()[:, :Hq * D].unflatten(1, (Hq, D)).unflatten(0, (B, n))
    width = max(ctx) + width_extra
    score = torch.rand(B, width, generator=g)
    return P, geom, q, qd, score, width


def _weights_ref(P, geom, q, ctx, n_row, page):
    out = []
    for i, c in enumerate(ctx):
        n = q.shape[1] if n_row is None else n_row[i]
        keys = np.asarray(ao.cached_rows(AH.host(P.k), P.table[i].tolist(), c))
        q64 = AH.host(q[i, :n])
        w = co.weights(q64, keys, geom.c_struct().scale) if n else None
        out.append((w, q64, keys))
    return out


WEIGHTS = [
    # ctx, n, n_row, Hq, Hk, D, page, dtype
    ((1,), 1, None, 1, 1, 64, 16, BF16),
    ((1, 2, 31, 32, 33, 63, 64, 65, 127, 257), 1, None, 6, 2, 128, 16, BF16),
    ((700, 40), 1, None, 24, 4, 256, 528, BF16),
    ((300, 5, 64), 4, (4, 0, 3), 8, 1, 64, 32, BF16),            # a full row tile; an idle row; fewer queries
    ((130, 33, 12), 5, (5, 5, 1), 7, 1, 128, 16, BF16),           # 35 rows: two row tiles
    ((2100, 64), 64, None, 4, 2, 256, 16, BF16),                # more row tiles than a round, masks across key tiles
    ((515, 9), 9, None, 64, 1, 256, 16, BF16),                  # 576 rows: Q in three rounds
    ((90, 64), 64, None, 64, 1, 64, 16, BF16),                  # 4096 rows
    ((257, 3), 3, None, 6, 3, 64, 16, F32),
    ((100, 300), 1, None, 12, 4, 256, 48, F32),
    ((150, 40), 40, None, 8, 2, 128, 16, F32),
    ((70, 33), 33, None, 6, 2, 256, 16, F32),                   # 99 rows
    ((50, 48), 48, None, 10, 2, 256, 16, F32),                  # 240 rows: Q in two rounds
]


@pytest.mark.parametrize("case", WEIGHTS, ids=str)
def test_weights_against_the_oracle(case):
    """Added to old scores up to have_len, taken from zero behind it; entries behind kv_len and idle rows stay."""
    print("weights", case, flush=True)
    m = AH.gdn()
    ctx, n, n_row, Hq, Hk, D, page, dtype = case
    P, geom, q, qd, score, width = _weights_case(50, ctx, n, n_row, Hq, Hk, D, page, dtype, pad=16 if n > 1 else 0)
    have = [max(0, c - 2) for c in ctx]
    old = score.clone()
    for i, h in enumerate(have):
        old[i, h:] = float("nan")  # not read
    out = torch.full_like(score, -7.0).cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = m.alloc_attn_weights_workspace(geom, len(ctx), n, width)
    ws.fill_(255)
    nr = None if n_row is None else _i32(n_row)
    m.attn_weights(geom, P.k.cuda(), P.table.cuda(), _i32(ctx), qd, out, ws, score_in=old.cuda(), have_len=_i32(have), n_row=nr, dev_err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    got = AH.host(out)
    for i, (w, q64, keys) in enumerate(_weights_ref(P, geom, q, ctx, n_row, page)):
        if w is None:
            assert np.all(got[i] == -7.0)
            continue
        base = np.zeros(ctx[i])
        base[:have[i]] = AH.host(score[i, :have[i]])
        d = np.abs(got[i, :ctx[i]] - (base + w))
        assert np.all(d <= _weights_bound(w, base, q64, keys, geom.c_struct().scale)), (i, d.max())
        assert np.all(got[i, ctx[i]:] == -7.0)


def test_weights_without_old_scores_and_in_place():
    m = AH.gdn()
    ctx = (77, 300)
    P, geom, q, qd, score, width = _weights_case(60, ctx, 2, None, 4, 2, 128, 16, BF16)
    args = (geom, P.k.cuda(), P.table.cuda(), _i32(ctx), qd)
    ws = m.alloc_attn_weights_workspace(geom, 2, 2, width)
    alone, both = torch.zeros(2, width, device="cuda"), score.cuda()
    m.attn_weights(*args, alone, ws)
    added = torch.zeros_like(alone)
    m.attn_weights(*args, added, ws, score_in=both)
    m.attn_weights(*args, both, ws, score_in=both)
    torch.cuda.synchronize()
    for i, c in enumerate(ctx):
        assert torch.equal(added[i, :c], score.cuda()[i, :c] + alone[i, :c])
        assert torch.equal(both[i, :c], added[i, :c]) and torch.equal(both[i, c:], score.cuda()[i, c:])
        assert abs(float(alone[i].double().sum()) - 8) < 8 * 1e-4  # all the weight of 2 x 4 queries


@pytest.mark.parametrize("n,G", [(1, 6), (6, 8), (20, 8)])
def test_weights_masked_keys_do_not_enter(n, G):
    """Infinite and NaN keys: the queries that attend them give NaN to what they attend, no other query does, and keys
    behind the row's end (the page's tail holds NaN) never count."""
    m = AH.gdn()
    ctx = (45 + n,)
    P, geom, q, qd, score, width = _weights_case(70, ctx, n, None, G, 1, 64, 16, BF16)
    last = ctx[0] - 1
    for bad in (float("nan"), float("inf"), float("-inf")):
        k = P.k.clone()
        k[P.table[0, last // 16], :, last % 16] = bad  # the newest token: only its own queries attend it
        out = torch.zeros(1, width, device="cuda")
        m.attn_weights(geom, k.cuda(), P.table.cuda(), _i32(ctx), qd, out, m.alloc_attn_weights_workspace(geom, 1, n, width))
        torch.cuda.synchronize()
        got = out[0].cpu()
        assert torch.isnan(got[:last + 1]).all() and torch.all(got[last + 1:] == 0)
        if n > 1:  # without the newest query, all is finite and as the oracle has it
            out.zero_()
            nr = [n - 1]
            m.attn_weights(geom, k.cuda(), P.table.cuda(), _i32([last]), qd, out, m.alloc_attn_weights_workspace(geom, 1, n, width), n_row=_i32(nr))
            torch.cuda.synchronize()
            w, q64, keys = _weights_ref(P, geom, q, [last], nr, 16)[0]
            d = np.abs(AH.host(out[0, :last]) - w)
            assert np.all(d <= _weights_bound(w, 0 * w, q64, keys, geom.c_struct().scale))


@pytest.mark.parametrize("n,G", [(1, 6), (6, 8), (9, 40)])
def test_weights_of_a_key_with_logits_of_minus_infinity(n, G):
    """A key that holds an infinity which every query meets with the other sign: its logits are -inf, its weight is 0, and
    all others are as the oracle has them (rows that only fill a tile of 32 meet it too: 6, 48 and 360 rows)."""
    m = AH.gdn()
    ctx = (45 + n,)
    P, geom, q, _, _, width = _weights_case(75, ctx, n, None, G, 1, 64, 16, BF16)
    q = q.clone()
    q[..., 3] = -1.0
    P.k[P.table[0, 0], :, 5, 3] = float("inf")
    out = torch.zeros(1, width, device="cuda")
    m.attn_weights(geom, P.k.cuda(), P.table.cuda(), _i32(ctx), q.cuda(), out, m.alloc_attn_weights_workspace(geom, 1, n, width))
    torch.cuda.synchronize()
    w, q64, keys = _weights_ref(P, geom, q, ctx, None, 16)[0]
    assert w[5] == 0 and np.all(np.isfinite(w))
    finite = np.where(np.isinf(keys), 0.0, keys)
    d = np.abs(AH.host(out[0, :ctx[0]]) - w)
    assert np.all(d <= _weights_bound(w, 0 * w, q64, finite, geom.c_struct().scale)), d
    assert float(out[0, 5]) == 0.0


def test_weights_of_a_row_of_2_to_26_tokens():
    """Keys times heads past 2^31: 32 heads over 2^26 + 1000 tokens, whose pages are all the same one, so that key j has the
    weight of key j % 512 over the number of its copies.  Parts of 128 keys are joined in eight chains of 65544, four
    roundings to a join: 4 x 65544 U = 0.0157 of a weight; its own logit, exponential and the parts' own sums are below
    0.001 of it as _weights_bound has them over 512 keys."""
    m = AH.gdn()
    G, D, page, c = 32, 64, 512, 2 ** 26 + 1000
    pages = -(-c // page)
    geom = m.AttnGeometry(n_q_heads=G, n_kv_heads=1, d_head=D, page_tokens=page, n_pages=1, max_pages=pages, max_tree=1)
    g = torch.Generator().manual_seed(140)
    k, q = torch.randn(1, 1, page, D, generator=g).to(BF16), torch.randn(1, 1, G, D, generator=g).to(BF16)
    out = torch.full((1, c), float("nan"), device="cuda")
    ws = m.alloc_attn_weights_workspace(geom, 1, 1, c)
    m.attn_weights(geom, k.cuda(), torch.zeros(1, pages, dtype=torch.int32, device="cuda"), _i32([c]), q.cuda(), out, ws)
    torch.cuda.synchronize()
    del ws
    q64, keys = AH.host(q[0, 0]), AH.host(k[0, 0])
    scale = geom.c_struct().scale
    assert np.all(_weights_bound(np.ones(page), np.zeros(page), q64[None], keys[:, None], scale) < 0.001)
    e = np.exp(scale * keys @ q64.T)  # [page][G]
    copies = c // page + (np.arange(page) < c % page)
    want = torch.tensor((e / (copies[:, None] * e).sum(axis=0)).sum(axis=1)).cuda()
    for at in range(0, c, 2 ** 20 * page // 16):  # whole pages at a time, and the last part of one
        part = out[0, at:at + 2 ** 20 * page // 16].double()
        part = torch.nn.functional.pad(part, (0, -len(part) % page)).view(-1, page)
        rest = c - at
        off = (part / want - 1).abs().flatten()[:rest]
        assert float(off.max()) < 0.017
    del out
    torch.cuda.empty_cache()


def test_weights_refused_rows_stay():
    m = AH.gdn()
    ctx = (40, 50, 60, 70)
    P, geom, q, qd, score, width = _weights_case(80, ctx, 3, None, 4, 1, 64, 16, BF16)
    ws = m.alloc_attn_weights_workspace(geom, 4, 3, width)
    def run(kv=ctx, have=None, n_row=None, table=P.table):  # noqa: E306
        out = torch.full((4, width), -1.0, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        m.attn_weights(geom, P.k.cuda(), table.cuda(), _i32(kv), qd, out, ws, score_in=score.cuda(),
                       have_len=None if have is None else _i32(have), n_row=None if n_row is None else _i32(n_row), dev_err=err)
        torch.cuda.synchronize()
        return int(err.item()), out
    code, good = run()
    assert code == 0
    for bad in (2, 0, -1, width + 1, geom.max_pages * 16 + 1, 2 ** 31 - 1, -2 ** 31):
        code, out = run(kv=(40, bad, 60, 70))
        assert code == m.DEV_BAD_LENGTH and torch.all(out[1] == -1.0) and torch.equal(out[[0, 2, 3]], good[[0, 2, 3]]), bad
    for bad in (-1, 61):
        code, out = run(have=(40, 50, bad, 70))
        assert code == m.DEV_BAD_LENGTH and torch.all(out[2] == -1.0) and torch.equal(out[[0, 1, 3]], good[[0, 1, 3]])
    for bad in (-1, 4, 2 ** 31 - 1):
        code, out = run(n_row=(bad, 3, 3, 3))
        assert code == m.DEV_BAD_K and torch.all(out[0] == -1.0) and torch.equal(out[1:], good[1:])
    for bad in (-1, P.n_pages, 2 ** 31 - 1):
        table = P.table.clone()
        table[3, 2] = bad
        code, out = run(table=table)
        assert code == m.DEV_BAD_PAGE and torch.equal(out[:3], good[:3])


@pytest.mark.parametrize("n,G", [(1, 2), (40, 2)])
def test_weights_of_idle_rows_alone(n, G):
    m = AH.gdn()
    P, geom, q, qd, score, width = _weights_case(85, (70, 90), n, None, G, 1, 64, 16, BF16)
    out = score.cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    m.attn_weights(geom, P.k.cuda(), P.table.cuda(), _i32((0, 2 ** 31 - 1)), qd, out, m.alloc_attn_weights_workspace(geom, 2, n, width),
                   n_row=_i32((0, 0)), dev_err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and torch.equal(out, score.cuda())


@pytest.mark.parametrize("n", [1, 9])
def test_weights_many_rows_of_the_batch(n):
    """More rows than a wave has lanes, most of them short, every third idle; a workspace of a larger call."""
    m = AH.gdn()
    ctx = tuple(n + (i * 37) % 90 for i in range(150))
    n_row = tuple(0 if i % 3 == 2 else 1 + i % n for i in range(150))
    P, geom, q, qd, score, width = _weights_case(86, ctx, n, n_row, 4, 1, 64, 16, BF16)
    ws = m.alloc_attn_weights_workspace(geom, 170, geom.max_tree, width + 1000)
    out = torch.full_like(score, -7.0).cuda()
    m.attn_weights(geom, P.k.cuda(), P.table.cuda(), _i32(ctx), qd, out, ws, n_row=_i32(n_row))
    torch.cuda.synchronize()
    got = AH.host(out)
    for i, (w, q64, keys) in enumerate(_weights_ref(P, geom, q, ctx, n_row, 16)):
        if w is None:
            assert np.all(got[i] == -7.0)
            continue
        d = np.abs(got[i, :ctx[i]] - w)
        assert np.all(d <= _weights_bound(w, 0 * w, q64, keys, geom.c_struct().scale)), (i, d.max())
        assert np.all(got[i, ctx[i]:] == -7.0)


@pytest.mark.parametrize("case", [
    # where 256 workgroups have more to do than one step of keys (512, fp32 d 256: 256) of one round of row tiles each, they take
    # steps one after the other and go from one round, KV head and batch row to the next: 320 steps over all, 6 row tiles to
    # a round; 720 of 2 tiles, an idle row; 324 of two rounds of 7 tiles, of one round in a batch row of fewer queries; 1112 of
    # 2 tiles; 294 of two rounds of 2.  (The longer ones of the cases further up make at most 256 steps, a workgroup each: 64
    # heads of 9 queries eighteen rounds of one tile, 5 heads of 48 queries on each of 2 KV heads eight.)
    ((17000, 9001, 700, 12345, 40), 32, None, 24, 4, 256, 528, BF16),
    ((20000, 9001, 700, 40, 15000), 5, (5, 4, 5, 0, 3), 64, 8, 64, 16, BF16),
    ((25000, 700, 15001, 64), 64, (64, 10, 64, 64), 14, 2, 64, 16, BF16),
    ((40000, 50, 30000), 7, None, 40, 8, 64, 528, F32),
    ((9000, 30, 5001, 300), 30, (30, 30, 7, 29), 12, 3, 256, 48, F32)],
    ids=lambda c: f"{len(c[0])}x{c[0][0]}-{c[1]}-{c[3]}on{c[4]}-{c[5]}")
def test_weights_of_many_rows_and_several_steps_to_a_workgroup(case):
    test_weights_against_the_oracle(case)


@pytest.mark.parametrize("case", [
    # up to 320 parts of 128 keys times KV heads, and 4096 over all rows: the parts are joined where the weights are summed,
    # a wave taking KV heads 0, 4, .. one after the other; 3, 12 and 32 query rows of a head, fewer in some batch rows
    ((1000, 130, 5), 1, None, 24, 8, 64, 16, BF16),
    ((1000, 130, 6), 6, (6, 1, 5), 10, 5, 128, 16, BF16),
    ((999, 8, 257), 8, (8, 8, 3), 28, 7, 64, 16, F32),
    # more parts of a row, or of all rows: they are joined in a kernel of their own
    ((6000, 70, 129), 3, (3, 1, 2), 16, 8, 128, 16, BF16),
    ((8200, 40), 8, (8, 7), 20, 5, 64, 48, F32),
    (tuple(4 + (i * 37) % 590 for i in range(150)), 4, tuple((1 + i) % 5 for i in range(150)), 16, 8, 64, 16, BF16)],
    ids=lambda c: f"{len(c[0])}x{c[0][0]}-{c[1]}-{c[3]}on{c[4]}-{c[5]}")
def test_weights_of_few_rows_and_more_heads_than_waves(case):
    test_weights_against_the_oracle(case)


def test_two_calls_at_once():
    """On two streams, each with a workspace of its own: the results of calls one after the other."""
    m = AH.gdn()
    for n in (1, 20):
        cases = [_weights_case(87 + k, (3000 + 100 * k, 50), n, None, 6, 2, 128, 16, BF16) for k in range(2)]
        args = [(g, P.k.cuda(), P.table.cuda(), _i32((3000 + 100 * k, 50)), qd) for k, (P, g, _, qd, _, _) in enumerate(cases)]
        outs = [torch.zeros(2, c[5], device="cuda") for c in cases]
        ws = [m.alloc_attn_weights_workspace(c[1], 2, n, c[5]) for c in cases]
        for a, o, w in zip(args, outs, ws):
            m.attn_weights(*a, o, w)
        torch.cuda.synchronize()
        want = [o.clone() for o in outs]
        streams = [torch.cuda.Stream() for _ in range(2)]
        for _ in range(3):
            for o in outs:
                o.zero_()
            torch.cuda.synchronize()
            for _ in range(4):
                for a, o, w, s in zip(args, outs, ws, streams):
                    m.attn_weights(*a, o, w, stream=s)
            torch.cuda.synchronize()
            for o, t in zip(outs, want):
                assert torch.equal(o, t)


def test_offsets_past_32_bits():
    """A cache of more than 2^32 bytes: its last pages are written, weighed and moved."""
    m = AH.gdn()
    Hk, D, pages = 4, 256, 140000
    geom = m.AttnGeometry(n_q_heads=8, n_kv_heads=Hk, d_head=D, page_tokens=16, n_pages=pages, max_pages=2)
    assert pages * Hk * 16 * D * 2 > 2 ** 32
    cache = m.KVCache(torch.zeros(pages, Hk, 16, D, dtype=BF16, device="cuda"), torch.zeros(pages, Hk, 16, D, dtype=BF16, device="cuda"))
    g = torch.Generator().manual_seed(130)
    k, v = (torch.randn(32, Hk, D, generator=g).to(BF16).cuda() for _ in range(2))
    table = torch.tensor([[pages - 1, pages - 70001]], dtype=torch.int32)
    slots = torch.cat([table[0, e] * 16 + torch.arange(16, dtype=torch.int32) for e in range(2)]).cuda()
    rope = m.Rope(rot_dims=256)
    k_out = torch.empty_like(k)
    pos = torch.arange(32, dtype=torch.int32, device="cuda")
    m.rope_rotate(geom, rope, m.rope_turns(rope), pos, k=k, k_out=k_out, v=v, cache=cache, slot_map=slots)
    torch.cuda.synchronize()
    for e in range(2):
        assert torch.equal(cache.k[table[0, e]].transpose(0, 1), k_out[16 * e:16 * e + 16])
        assert torch.equal(cache.v[table[0, e]].transpose(0, 1), v[16 * e:16 * e + 16])
    q = torch.randn(1, 1, 8, D, generator=g).to(BF16)
    score = torch.zeros(1, 32, device="cuda")
    m.attn_weights(geom, cache.k, table.cuda(), _i32([32]), q.cuda(), score, m.alloc_attn_weights_workspace(geom, 1, 1, 32))
    keys, q64 = AH.host(k_out), AH.host(q[0])
    w = co.weights(q64, keys, geom.c_struct().scale)
    assert np.all(np.abs(AH.host(score[0]) - w) <= _weights_bound(w, 0 * w, q64, keys, geom.c_struct().scale))
    to = torch.tensor([[(pages - 2) * 16 + 3]], dtype=torch.int32, device="cuda")
    m.kv_move(geom, cache, slots[31:].view(1, 1), to, _i32([1]))
    torch.cuda.synchronize()
    assert torch.equal(cache.k[pages - 2, :, 3], k_out[31]) and torch.equal(cache.v[pages - 2, :, 3], v[31])
    del cache
    torch.cuda.empty_cache()


# ---------------------------------------------------------------- plans

def _plan_case(seed, ctx, budget, page, sink, recent, settled=None, gone=None, ties=False, width_extra=3, free_extra=0, moves_extra=0):
    rng = np.random.Generator(np.random.PCG64(seed))
    B, width = len(ctx), max(max(ctx), 1) + width_extra
    need = [-(-c // page) for c in ctx]
    n_free = 3
    n_pages = sum(need) + n_free + free_extra
    ids = rng.permutation(n_pages).astype(np.int32)
    tables = np.full((B, max(need) + 2), -9, np.int32)
    at = 0
    for i, h in enumerate(need):
        tables[i, :h] = ids[at:at + h]
        at += h
    free = np.full(n_pages, -5, np.int32)
    free[:n_free] = ids[at:at + n_free]
    score = rng.random((B, width)).astype(np.float32) ** 4
    if ties:
        score = rng.choice(np.array([0.0, -0.0, 0.25, 0.25, 1.0, -1.0, np.nan, np.inf, -np.inf, 1e-40], np.float32), size=(B, width))
    settled = [0] * B if settled is None else settled
    gone = [0] * B if gone is None else gone
    pos = np.full((B, width), -77, np.int32)
    for i in range(B):
        pos[i, :settled[i]] = rng.permutation(settled[i] + gone[i])[:settled[i]]
    moves = max([min(b, c - b) for c, b in zip(ctx, budget) if 0 <= b < c] + [1]) + moves_extra
    return dict(ctx=list(ctx), budget=list(budget), page=page, sink=sink, recent=recent, n_pages=n_pages, tables=tables, free=free, n_free=n_free,
                score=score, pos=pos, state=np.stack([settled, gone], 1).astype(np.int32), moves=moves)


def _plan(c, in_place=False, call_twice=False):
    """Runs a plan; returns the outputs on the host, and the device error."""
    m = AH.gdn()
    B, width = c["score"].shape
    geom = m.AttnGeometry(n_q_heads=1, n_kv_heads=1, d_head=64, page_tokens=c["page"], n_pages=c["n_pages"], max_pages=c["tables"].shape[1])
    score, pos = torch.from_numpy(c["score"]).cuda(), _i32(c["pos"])
    full = lambda *s: torch.full(s, -3, dtype=torch.int32, device="cuda")  # noqa: E731
    t = dict(score_out=score if in_place else torch.full_like(score, -3.0), token_pos_out=pos if in_place else full(B, width), kv_len_out=full(B),
             row_state_out=full(B, 2), n_free_out=full(1), move_src=full(B, c["moves"]), move_dst=full(B, c["moves"]), n_moves=full(B))
    free, tables = _i32(c["free"]), _i32(c["tables"])
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for _ in range(2 if call_twice else 1):
        m.evict_plan(geom, _i32(c["ctx"]), _i32(c["budget"]), score, pos, _i32(c["state"]), tables, free, _i32([c["n_free"]]), *t.values(),
                     sink=c["sink"], recent=c["recent"], dev_err=err)
    torch.cuda.synchronize()
    assert np.array_equal(tables.cpu().numpy(), c["tables"])
    out = {k: v.cpu().numpy() for k, v in t.items()}
    out["free"] = free.cpu().numpy()
    return out, int(err.item())


def _check_plan(c, out, in_place=False):
    rows, stack, bad = co.evict(c["page"], c["n_pages"], c["tables"].shape[1], c["ctx"], c["budget"], c["score"], c["pos"], c["state"], c["tables"],
                                c["free"], c["n_free"], c["sink"], c["recent"], c["moves"])
    for i, r in enumerate(rows):
        assert out["kv_len_out"][i] == r["kv_len"] and out["row_state_out"][i].tolist() == r["state"], i
        k, n = len(r["pos"]), len(r["src"])
        assert out["n_moves"][i] == n, (i, out["n_moves"][i], n)
        for name, want in (("move_src", r["src"]), ("move_dst", r["dst"])):
            assert out[name][i].tolist() == want + [-1] * (c["moves"] - n), (i, name)
        assert np.array_equal(out["score_out"][i, :k], np.array(r["score"], np.float32), equal_nan=True), i
        assert out["token_pos_out"][i, :k].tolist() == r["pos"], i
        rest = (c["score"][i, k:], c["pos"][i, k:]) if in_place else (-3.0, -3)
        # a row that keeps its tokens in place has written the positions of all of them
        assert np.array_equal(out["score_out"][i, k:], np.broadcast_to(rest[0], out["score_out"][i, k:].shape), equal_nan=True), i
        assert np.all(out["token_pos_out"][i, k:] == rest[1]), i
    want = c["free"].copy()
    if stack is not None:
        want[:len(stack)] = stack
    assert out["free"].tolist() == want.tolist()
    assert out["n_free_out"][0] == (len(stack) if stack is not None else c["n_free"])
    return bad, stack


PLANS = [
    dict(ctx=(1,), budget=(0,), page=16, sink=0, recent=0),
    dict(ctx=(1, 5, 16, 17), budget=(1, -1, 8, 16), page=16, sink=0, recent=0),
    dict(ctx=(0, 100, 64, 65), budget=(0, 40, 63, 1), page=16, sink=1, recent=0),
    dict(ctx=(1000, 1023, 1024, 1025, 2049), budget=(500, 1000, 32, 1024, 64), page=32, sink=4, recent=20),
    dict(ctx=(5000, 333), budget=(100, 332), page=528, sink=4, recent=64, settled=(4000, 100), gone=(123, 7)),
    dict(ctx=(300, 300, 300), budget=(150, 299, 20), page=16, sink=2, recent=10, ties=True),
    dict(ctx=(3000, 2000), budget=(1500, 700), page=16, sink=8, recent=100, ties=True, settled=(3000, 0), gone=(5000, 9)),
    dict(ctx=(32768, 32769, 40000), budget=(32767, 32768, 20000), page=16, sink=4, recent=1000),
    dict(ctx=(70001,), budget=(34000,), page=64, sink=64, recent=5000, settled=(60000,), gone=(100000,)),
    dict(ctx=(70001,), budget=(50000,), page=64, sink=0, recent=0, ties=True),
    dict(ctx=tuple(20 + 3 * i for i in range(300)), budget=tuple((i * 7) % 60 - 1 for i in range(300)), page=16, sink=0, recent=0),
]


@pytest.mark.parametrize("case", PLANS, ids=lambda c: f"{len(c['ctx'])}x{c['ctx'][0]}-{c['budget'][0]}" + ("-ties" if c.get("ties") else ""))
@pytest.mark.parametrize("in_place", [False, True])
def test_plan_against_plain_loops(case, in_place):
    print("plan", {k: v if not isinstance(v, tuple) or len(v) < 8 else len(v) for k, v in case.items()}, in_place, flush=True)
    c = _plan_case(90, **case, moves_extra=5)
    out, err = _plan(c, in_place)
    bad, stack = _check_plan(c, out, in_place)
    assert not bad and stack is not None and err == 0


@pytest.mark.parametrize("value", [0.0, -3.5, float("nan"), float("-inf"), float("inf"), 1e-42])
@pytest.mark.parametrize("ctx,budget", [((8192, 16384, 300), (4000, 16383, 1)), ((20011,), (12345,)), ((100000, 24576), (3, 9000))])
def test_plan_with_equal_scores(value, ctx, budget):
    """Rows of one score alone: the lowest indexes stay, whatever the number of equals."""
    c = _plan_case(96, ctx, budget, 16, 0, 0)
    c["score"][:] = value
    out, err = _plan(c)
    bad, _ = _check_plan(c, out)
    assert not bad and err == 0
    # nothing moves: what stays is in place
    assert out["n_moves"].tolist() == [0] * len(ctx)


def test_plan_of_the_widest_rows():
    m = AH.gdn()
    c = _plan_case(97, (2 ** 18, 200001), (100000, 200000), 16, 4, 1000, settled=(2 ** 18, 0), gone=(77, 0), width_extra=0)
    assert c["score"].shape[1] == 2 ** 18
    out, err = _plan(c)
    bad, _ = _check_plan(c, out)
    assert not bad and err == 0
    with pytest.raises(m.GdnError, match="width: 262145"):
        _plan(_plan_case(98, (2 ** 18 + 1,), (5,), 16, 0, 0, width_extra=0))


@pytest.mark.parametrize("page", [16, 48, 528, 4096, 2 ** 20])
def test_plan_page_sizes(page):
    c = _plan_case(99, (5000, 4097, 100), (2500, 4096, 31), page, 1, 7)
    out, err = _plan(c)
    bad, _ = _check_plan(c, out)
    assert not bad and err == 0


def test_plan_again_gives_the_same():
    c = _plan_case(91, **PLANS[4])
    out, err = _plan(c, call_twice=True)
    assert err == 0
    _check_plan(c, out)


def test_plan_largest_batch():
    ctx = [1 + (i * 13) % 50 for i in range(4096)]
    c = _plan_case(92, ctx, [x // 2 if i % 3 else -1 for i, x in enumerate(ctx)], 16, 0, 0)
    out, err = _plan(c)
    bad, _ = _check_plan(c, out)
    assert not bad and err == 0


def test_plan_refused_rows():
    m = AH.gdn()
    base = dict(ctx=(100, 200, 300), budget=(50, 150, 10), page=16, sink=2, recent=8)
    for change in (dict(ctx=(100, -1, 300)), dict(ctx=(100, 2 ** 31 - 1, 300)), dict(ctx=(100, 304, 300)), dict(state=[(0, 0), (201, 0), (0, 0)]),
                   dict(state=[(0, 0), (-1, 0), (0, 0)]), dict(state=[(0, 0), (0, -1), (0, 0)]), dict(state=[(0, 0), (0, 2 ** 31 - 200), (0, 0)]),
                   dict(budget=(50, 9, 10)), dict(budget=(50, 0, 10)), dict(sink=11), dict(sink=2 ** 31 - 1), dict(moves=49), dict(moves=1)):
        c = _plan_case(93, **base)
        c.update({k: list(v) if isinstance(v, tuple) else v for k, v in change.items() if k != "state"})
        if "state" in change:
            c["state"] = np.array(change["state"], np.int32)
        out, err = _plan(c)
        bad, _ = _check_plan(c, out)
        assert bad and err == m.DEV_BAD_LENGTH, change


def test_plan_refused_pages():
    m = AH.gdn()
    base = dict(ctx=(100, 200, 300), budget=(50, 150, 10), page=16, sink=2, recent=8)
    for n_free in (-1, -2 ** 31, 2 ** 31 - 1, 20):  # out of range, or 24 pages come free where there is no room
        c = _plan_case(94, **base)
        c["n_free"] = n_free
        out, err = _plan(c)
        _, stack = _check_plan(c, out)
        assert stack is None and err == m.DEV_BAD_PAGE, n_free
    # a page that does not exist: its tokens are not moved, it is reported
    for bad in (-1, 10 ** 6):
        c = _plan_case(95, **base)
        c["tables"][2, 18] = bad
        rows, _, _ = co.evict(16, c["n_pages"], c["tables"].shape[1], c["ctx"], c["budget"], c["score"], c["pos"], c["state"], c["tables"], c["free"],
                              c["n_free"], 2, 8, c["moves"])
        out, err = _plan(c)
        assert err == m.DEV_BAD_PAGE
        n = len(rows[2]["src"])
        want = [-1 if not 0 <= s < c["n_pages"] * 16 else s for s in rows[2]["src"]]
        assert -1 in want and out["move_src"][2, :n].tolist() == want and out["move_dst"][2, :n].tolist() == rows[2]["dst"]


@pytest.mark.parametrize("bad", [
    [(2, 18, -1)],                                                   # freed, and moved from
    [(1, 0, 2 ** 31 - 1)],                                           # moved to
    [(0, 2, -2 ** 31), (0, 6, -1)],                                  # in a row that loses few tokens
    [(2, e, 10 ** 6 + e) for e in range(19)],                        # no page of a row at all
    [(i, e, -1 - e) for i in range(3) for e in range(0, 19, 2)]],
    ids=["source", "destination", "short", "whole", "every second"])
@pytest.mark.parametrize("in_place", [False, True])
def test_plan_of_rows_with_pages_that_do_not_exist(bad, in_place):
    """What is on them is not moved: the gap of such a pair keeps its token, score and position; what does not exist does
    not get onto the stack of free pages, so that rows served from it have pages of the cache."""
    m = AH.gdn()
    c = _plan_case(101, (100, 200, 300), (50, 150, 10), 16, 2, 8, settled=(60, 200, 0), gone=(9, 70, 0), moves_extra=3)
    for i, e, page in bad:
        if e < -(-c["ctx"][i] // 16):
            c["tables"][i, e] = page
    out, err = _plan(c, in_place)
    refused, stack = _check_plan(c, out, in_place)
    assert not refused and stack is not None and err == m.DEV_BAD_PAGE
    freed = [(i, e) for i, (lo, hi) in enumerate(((4, 7), (10, 13), (1, 19))) for e in range(lo, hi)]
    assert all(0 <= p < c["n_pages"] for p in stack) and len(stack) == 3 + len(freed) - len(set(freed) & {x[:2] for x in bad})
    geom = m.AttnGeometry(n_q_heads=1, n_kv_heads=1, d_head=64, page_tokens=16, n_pages=c["n_pages"], max_pages=len(stack))
    z = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    table, cu, slots, pos, kv, n_free, code = z(1, len(stack)), z(2), z(16 * len(stack)), z(16 * len(stack)), z(1), z(1), z(1)
    m.kv_plan(geom, z(1), _i32([16 * len(stack)]), _i32(out["free"]), _i32(out["n_free_out"]), table, cu, slots, pos, kv, n_free, dev_err=code)
    torch.cuda.synchronize()
    assert int(code.item()) == 0 and sorted(table[0].tolist()) == sorted(stack) and int(n_free.item()) == 0


# ---------------------------------------------------------------- moves

@pytest.mark.parametrize("Hk,D,page,dtype,counts", [
    (1, 64, 16, BF16, (1,)), (4, 256, 16, BF16, (0, 3, 130)), (3, 128, 528, F32, (70, 1)), (8, 128, 32, BF16, (300, 17, 0, 64)), (2, 256, 16, F32, (33,) * 9)])
def test_moves(Hk, D, page, dtype, counts):
    """Bit for bit, NaN among them; slots -1 skipped, entries behind n_moves not read, nothing else touched."""
    m = AH.gdn()
    B, width, total = len(counts), max(counts) + 2, sum(counts)
    pages = -(-(2 * total + 4) // page)
    geom = m.AttnGeometry(n_q_heads=Hk, n_kv_heads=Hk, d_head=D, page_tokens=page, n_pages=pages, max_pages=pages, dtype=dtype)
    g = torch.Generator().manual_seed(100)
    slots = torch.randperm(pages * page, generator=g)[:2 * total].to(torch.int32)
    src, dst = torch.full((B, width), 2 ** 31 - 1, dtype=torch.int32), torch.full((B, width), -5, dtype=torch.int32)
    at = 0
    for i, n in enumerate(counts):
        src[i, :n], dst[i, :n] = slots[at:at + n], slots[total + at:total + at + n]
        at += n
    if counts[-1] > 2:
        src[-1, 1], dst[-1, 2] = -1, -1
    cache = m.KVCache(*(torch.randn(pages, Hk, page, D, generator=g).to(dtype).cuda() for _ in range(2)))
    cache.k[0, 0, 0, 0] = float("nan")
    want = [t.clone() for t in (cache.k, cache.v)]
    for i, n in enumerate(counts):
        for e in range(n):
            a, b = int(src[i, e]), int(dst[i, e])
            if a >= 0 and b >= 0:
                for w, t in zip(want, (cache.k, cache.v)):
                    w[b // page, :, b % page] = t[a // page, :, a % page]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    m.kv_move(geom, cache, src.cuda(), dst.cuda(), _i32(counts), dev_err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    bits = torch.int16 if dtype == BF16 else torch.int32
    assert torch.equal(cache.k.view(bits), want[0].view(bits)) and torch.equal(cache.v.view(bits), want[1].view(bits))


@pytest.mark.parametrize("Hk,D,page,dtype,counts", [
    (40, 64, 48, BF16, (5, 9)),                                  # a token's pieces are more than a workgroup's threads
    (3, 64, 80, BF16, (200, 31, 11)),                            # ten moves of 24 pieces to a workgroup
    (1, 64, 16, BF16, (1000,) + (0,) * 597 + (40, 999)),         # 600 rows: 13 workgroups to a row, which go round
    (7, 128, 4096, F32, (64,))])
def test_moves_of_many_heads_rows_and_page_sizes(Hk, D, page, dtype, counts):
    test_moves(Hk, D, page, dtype, counts)


def test_moves_refused():
    m = AH.gdn()
    geom = m.AttnGeometry(n_q_heads=1, n_kv_heads=1, d_head=64, page_tokens=16, n_pages=4, max_pages=4)
    for src, dst, n, code in (((3, 64), (7, 9), 2, m.DEV_BAD_PAGE), ((3, 5), (7, -2), 2, m.DEV_BAD_PAGE), ((-2 ** 31, 5), (7, 9), 2, m.DEV_BAD_PAGE),
                              ((3, 5), (2 ** 31 - 1, 9), 2, m.DEV_BAD_PAGE), ((3, 5), (7, 9), 3, m.DEV_BAD_LENGTH), ((3, 5), (7, 9), -1, m.DEV_BAD_LENGTH)):
        cache = m.KVCache.zeros(geom)
        cache.k += torch.arange(1, 65, device="cuda").view(4, 1, 16, 1)
        was = cache.k.clone()
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        m.kv_move(geom, cache, _i32([src]), _i32([dst]), _i32([n]), dev_err=err)
        torch.cuda.synchronize()
        assert int(err.item()) == code
        ok = [(a, b) for a, b in zip(src, dst) if 0 <= a < 64 and 0 <= b < 64] if code == m.DEV_BAD_PAGE else []
        for a, b in ok:
            was[b // 16, :, b % 16] = a + 1
        assert torch.equal(cache.k, was)


# ---------------------------------------------------------------- together

class _Stack:
    """Two attention layers over one set of block tables: every step plans its tokens, rotates and writes them, attends, adds
    the weights up, and cuts the rows back.  All state is on the GPU and the host reads nothing back."""

    BUDGET, SINK, RECENT = 40, 2, 6

    def __init__(self, seed, B, new_most):
        m = self.m = AH.gdn()
        self.B, self.most = B, new_most
        self.geom = m.AttnGeometry(n_q_heads=6, n_kv_heads=2, d_head=64, page_tokens=16, n_pages=B * 7 + 3, max_pages=7, max_tree=4)
        self.width = 7 * 16
        self.rope = m.Rope(rot_dims=32, base=1e3)
        self.turns = m.rope_turns(self.rope)
        z = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
        N = B * new_most
        self.kv, self.kv_mid, self.new, self.free = z(B), z(B), z(B), torch.arange(self.geom.n_pages, dtype=torch.int32, device="cuda")
        self.n_free, self.n_mid, self.table, self.cu = z(1) + self.geom.n_pages, z(1), z(B, 7) - 1, z(B + 1)
        self.slot, self.pos, self.state, self.state_out, self.token_pos = z(N), z(N), z(B, 2), z(B, 2), z(B, self.width)
        self.score, self.budget = torch.zeros(B, self.width, device="cuda"), z(B) + self.BUDGET
        self.src, self.dst, self.moves, self.err = z(B, 48), z(B, 48), z(B), z(1)
        self.cache = [m.KVCache.zeros(self.geom) for _ in range(2)]
        self.qkv = [torch.zeros(N, 10, 64, dtype=BF16, device="cuda") for _ in range(2)]
        self.o = [torch.zeros(N, 6, 64, dtype=BF16, device="cuda") for _ in range(2)]
        self.ws = m.alloc_attn_prefill_workspace(self.geom, N, B, up_to=True)
        self.ww = m.alloc_attn_weights_workspace(self.geom, B, 1, self.width)
        self.row = torch.zeros(N, dtype=torch.int64, device="cuda")  # each packed token's row
        self.last = torch.zeros(B, dtype=torch.int64, device="cuda")  # each row's newest token

    def step(self):
        m, g, e = self.m, self.geom, self.err
        m.kv_plan(g, self.kv, self.new, self.free, self.n_free, self.table, self.cu, self.slot, self.pos, self.kv_mid, self.n_mid, dev_err=e)
        at = self.pos + self.state[:, 1][self.row]  # the position, not the place in the cache
        for i, (cache, x, o) in enumerate(zip(self.cache, self.qkv, self.o)):
            q, k, v = x[:, :6], x[:, 6:8], x[:, 8:]
            m.rope_rotate(g, self.rope, self.turns, at, q=q, k=k, v=v, cache=cache, slot_map=self.slot, dev_err=e)
            m.attn_prefill(g, q, k, v, self.cu, o, self.ws, cache=cache, block_table=self.table, ctx_len=self.kv, dev_err=e)
            # every layer's weights of the newest token of each row; new tokens come in with nothing
            m.attn_weights(g, cache.k, self.table, self.kv_mid, q[self.last][:, None], self.score, self.ww, score_in=self.score,
                           have_len=self.kv if i == 0 else None, dev_err=e)
        m.evict_plan(g, self.kv_mid, self.budget, self.score, self.token_pos, self.state, self.table, self.free, self.n_mid, self.score,
                     self.token_pos, self.kv, self.state_out, self.n_free, self.src, self.dst, self.moves, sink=self.SINK, recent=self.RECENT, dev_err=e)
        for cache in self.cache:
            m.kv_move(g, cache, self.src, self.dst, self.moves, dev_err=e)
        self.state.copy_(self.state_out)

    def feed(self, seed, new):
        g = torch.Generator().manual_seed(seed)
        rows, cu = np.repeat(np.arange(self.B), new), np.cumsum([0] + list(new))
        self.new.copy_(_i32(new))
        self.row[:len(rows)] = torch.from_numpy(rows).cuda()
        self.last.copy_(torch.from_numpy(cu[1:] - 1).cuda())
        for x in self.qkv:
            x.copy_(torch.randn(x.shape, generator=g).to(BF16))


@pytest.mark.parametrize("captured", [False, True])
def test_the_operators_run_together(captured):
    """Steps of ragged prompts and of single tokens, each against a model that keeps every row's tokens as a list: outputs,
    scores, positions, what stays, page counts, and at last every cached row."""
    B, most = 3, 20
    st = _Stack(1, B, most)
    freq = co.frequencies(32, 1e3)
    kept = [[] for _ in range(B)]  # per row: (position, score, k of each layer, v of each layer)
    seen = [0] * B
    scale = 64 ** -0.5
    graph = None
    if captured:
        st.feed(1000, [1] * B)  # warm: every workspace and module is there before the capture
        saved = {k: v.clone() for k, v in st.__dict__.items() if isinstance(v, torch.Tensor)}
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            st.step()
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            st.step()
        for k, v in saved.items():
            getattr(st, k).copy_(v)
        for c in st.cache:
            c.k.zero_()
            c.v.zero_()
    rng = np.random.Generator(np.random.PCG64(3))
    for step in range(14):
        new = [int(rng.integers(1, most + 1)) if step % 3 == 0 else 1 for _ in range(B)]
        st.feed(step, new)
        raw = [AH.host(x) for x in st.qkv]
        if graph is None:
            st.step()
        else:
            graph.replay()
        torch.cuda.synchronize()
        assert int(st.err.item()) == 0
        at = 0
        for i, n in enumerate(new):
            pos = [seen[i] + t for t in range(n)]
            kept[i] += [[p, 0.0, [], []] for p in pos]
            for layer in range(2):
                # what the layer computed from: the rotated rows as they were rounded, checked against the oracle's
                x = AH.host(st.qkv[layer][at:at + n])
                want = raw[layer][at:at + n].copy()
                want[:, :8] = co.rotate(want[:, :8], pos, freq, "half")
                assert np.all(np.abs(x - want) <= 2.0 ** -8 * np.abs(want) + 22 * U * 6)
                for r, row in zip(kept[i][-n:], x):
                    r[2].append(row[6:8])
                    r[3].append(row[8:])
                k, v = (np.stack([r[c][layer] for r in kept[i]]) for c in (2, 3))
                c0 = len(kept[i]) - n
                mask = np.arange(c0 + n)[None] <= c0 + np.arange(n)[:, None]
                o, mag = ao.attend(x[:, :6], k, v, mask, scale)
                assert np.all(np.abs(AH.host(st.o[layer][at:at + n]) - o) <= AH.tolerance(o, mag, x[:, :6], k, scale, c0 + n, BF16))
                for r, w in zip(kept[i], co.weights(x[n - 1:n, :6], k, scale)):
                    r[1] += w
            seen[i] += n
            at += n
            # what the plan kept is among what the model would keep: the scores agree to their rounding
            c = len(kept[i])
            if c > st.BUDGET:
                by_pos = {r[0]: r for r in kept[i]}
                left = st.token_pos[i, :st.BUDGET].tolist()
                assert len(set(left)) == st.BUDGET and set(left) <= set(by_pos)
                assert set(p for p in by_pos if p < st.SINK or p >= seen[i] - st.RECENT) <= set(left)
                gone = [r[1] for p, r in by_pos.items() if p not in left]
                free = [by_pos[p][1] for p in left if st.SINK <= p < seen[i] - st.RECENT]
                assert max(gone) <= min(free) * (1 + 1e-3)
                kept[i] = [by_pos[p] for p in left]
            assert int(st.kv[i]) == len(kept[i]) and st.state[i].tolist()[1] == seen[i] - len(kept[i])
            got = AH.host(st.score[i, :len(kept[i])])
            assert np.allclose(got, [r[1] for r in kept[i]], rtol=1e-3, atol=1e-6)
        used = sum(-(-len(r) // 16) for r in kept)
        assert int(st.n_free) == st.geom.n_pages - used
        pages = [p for i in range(B) for p in st.table[i, :-(-len(kept[i]) // 16)].tolist()] + st.free[:int(st.n_free)].tolist()
        assert sorted(pages) == list(range(st.geom.n_pages))  # every page is in one place
    for i in range(B):
        for layer, cache in enumerate(st.cache):
            rows = ao.cached_rows(AH.host(cache.k), st.table[i].tolist(), len(kept[i]))
            vals = ao.cached_rows(AH.host(cache.v), st.table[i].tolist(), len(kept[i]))
            assert np.array_equal(rows, np.stack([r[2][layer] for r in kept[i]]))
            assert np.array_equal(vals, np.stack([r[3][layer] for r in kept[i]]))


def test_plan_weights_and_moves_captured():
    """On a stream of the call's own, captured: replays with new lengths and scores give the eager results."""
    m = AH.gdn()
    ctx = (400, 90, 700)
    P, geom, q, qd, score, width = _weights_case(110, ctx, 2, None, 4, 2, 128, 16, BF16)
    kv, budget, state = _i32(ctx), _i32((100, 90, 650)), _i32(np.zeros((3, 2)))
    k, table = P.k.nan_to_num().cuda(), P.table.cuda()
    cache = m.KVCache(k, P.v.nan_to_num().cuda())
    z = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    free, n_free = z(geom.n_pages), z(1)
    s_in, s1, s2 = score.cuda(), torch.zeros(3, width, device="cuda"), torch.zeros(3, width, device="cuda")
    out = dict(token_pos_out=z(3, width), kv_len_out=z(3), row_state_out=z(3, 2), n_free_out=z(1), move_src=z(3, 320), move_dst=z(3, 320), n_moves=z(3))
    pos, err, ws = z(3, width), z(1), m.alloc_attn_weights_workspace(geom, 3, 2, width)

    def call(**kw):
        m.attn_weights(geom, k, table, kv, qd, s1, ws, score_in=s_in, dev_err=err, **kw)
        m.evict_plan(geom, kv, budget, s1, pos, state, table, free, n_free, s2, *out.values(), sink=1, recent=9, dev_err=err, **kw)
        m.kv_move(geom, cache, out["move_src"], out["move_dst"], out["n_moves"], dev_err=err, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(stream=side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call()
    for step, lens in enumerate(((400, 90, 700), (101, 2, 699), (399, 91, 2))):
        kv.copy_(_i32(lens))
        s_in.copy_(torch.rand(3, width, generator=torch.Generator().manual_seed(step)))
        start = [t.clone() for t in (cache.k, cache.v, s2)]
        call()
        torch.cuda.synchronize()
        every = [s1, s2, free, cache.k, cache.v, *out.values()]
        want = [t.clone() for t in every]
        for t, was in zip((cache.k, cache.v, s2), start):
            t.copy_(was)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(every, want):
            assert torch.equal(a, b)
        assert int(err.item()) == 0


def test_runs_give_the_same_bits():
    m = AH.gdn()
    for n, G in ((1, 6), (12, 6)):
        P, geom, q, qd, score, width = _weights_case(120, (5000, 1200), n, None, 2 * G, 2, 128, 16, BF16)
        outs = []
        for _ in range(3):
            out = torch.zeros(2, width, device="cuda")
            m.attn_weights(geom, P.k.cuda(), P.table.cuda(), _i32((5000, 1200)), qd, out, m.alloc_attn_weights_workspace(geom, 2, n, width))
            outs.append(out)
        torch.cuda.synchronize()
        assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
