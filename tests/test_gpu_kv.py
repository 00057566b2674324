"""The paged cache's bookkeeping and writes on the GPU: block tables, slot maps and the free stack against plain loops,
rows that cannot be served, refused values; rows written to their slots and nowhere else; the operators run together."""
import numpy as np
import pytest
import torch

import attn_harness as AH
from oracle import attn_oracle as ao

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
OUT = ("block_table", "free_pages", "cu_new", "slot_map", "position", "kv_len_out", "n_free_out")


def _cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(torch.int32).cuda()


def _plan_inputs(seed, kv_len, new_len, page, spare):
    """Tables with the rows' pages in no order, the rest of the pages on the stack."""
    rng = np.random.Generator(np.random.PCG64(seed))
    have = [-(-c // page) for c in kv_len]
    need = sum(max(0, -(-(c + max(n, 0)) // page) - h) for c, n, h in zip(kv_len, new_len, have))
    n_free = max(0, need + spare)
    n_pages = sum(have) + n_free + 3
    width = max(-(-(c + max(n, 0)) // page) for c, n in zip(kv_len, new_len)) + 2
    ids = rng.permutation(n_pages).astype(np.int32)
    tables = np.full((len(kv_len), width), -9, np.int32)
    at = 0
    for i, h in enumerate(have):
        tables[i, :h] = ids[at:at + h]
        at += h
    free = np.full(n_pages, -5, np.int32)
    free[:n_free] = ids[at:at + n_free]
    return n_pages, width, tables, free, n_free


def _plan(geom, kv_len, new_len, free, n_free, tables, max_tokens, err):
    m = AH.gdn()
    B = len(kv_len)
    t = dict(kv_len=_cuda(kv_len), new_len=_cuda(new_len), free_pages=_cuda(free), n_free=_cuda([n_free]),
             block_table=_cuda(tables), cu_new=torch.full((B + 1,), -3, dtype=torch.int32, device="cuda"),
             slot_map=torch.full((max_tokens,), -3, dtype=torch.int32, device="cuda"),
             position=torch.full((max_tokens,), -3, dtype=torch.int32, device="cuda"),
             kv_len_out=torch.full((B,), -3, dtype=torch.int32, device="cuda"),
             n_free_out=torch.full((1,), -3, dtype=torch.int32, device="cuda"))
    call = lambda: m.kv_plan(geom, *t.values(), dev_err=err)  # noqa: E731
    call()
    return t, call


def _same(t, ref):
    for name in OUT:
        got = t[name].cpu().numpy()
        assert np.array_equal(got.reshape(-1), np.asarray(ref[name]).reshape(-1)), name


def _lengths(seed, B, ctx_hi, new_hi):
    rng = np.random.Generator(np.random.PCG64(seed))
    kv = rng.integers(0, ctx_hi + 1, size=B)
    new = rng.integers(0, new_hi + 1, size=B)
    new[rng.random(B) < 0.2] = 0
    new[rng.random(B) < 0.2] = -1
    return [int(c) for c in kv], [int(n) for n in new]


@pytest.mark.parametrize("B,ctx_hi,new_hi,page,pad", [
    (1, 0, 1, 16, 0), (1, 40, 50, 16, 3), (4, 100, 1, 16, 0), (7, 64, 33, 16, 5), (65, 300, 20, 32, 0),
    (256, 50, 4, 528, 100), (300, 1000, 70, 16, 1), (1000, 40, 3, 16, 0), (4096, 20, 2, 16, 7)])
def test_plan_against_plain_loops(B, ctx_hi, new_hi, page, pad):
    """Random batches with idle, new and leaving rows; a second call on the same inputs gives the same."""
    print(f"plan B {B} ctx <= {ctx_hi} new <= {new_hi} page {page}", flush=True)
    m = AH.gdn()
    kv, new = _lengths(100 + B, B, ctx_hi, new_hi)
    n_pages, width, tables, free, n_free = _plan_inputs(101 + B, kv, new, page, 1)
    geom = m.AttnGeometry(n_q_heads=1, n_kv_heads=1, d_head=64, page_tokens=page, n_pages=n_pages, max_pages=width)
    cap = sum(max(n, 0) for n in new) + pad
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    t, call = _plan(geom, kv, new, free, n_free, tables, cap, err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    ref = ao.kv_plan(page, n_pages, width, kv, new, free, n_free, tables, cap)
    _same(t, ref)
    call()
    torch.cuda.synchronize()
    _same(t, ref)


def test_plan_pages_of_leaving_rows_serve_the_same_call():
    """An empty stack: the leaving row's pages go to the rows that grow."""
    m = AH.gdn()
    kv, new = [32, 48, 0], [1, -1, 20]
    n_pages, width, tables, free, n_free = _plan_inputs(3, kv, new, 16, -3)
    assert n_free == 0
    geom = m.AttnGeometry(n_q_heads=1, n_kv_heads=1, d_head=64, page_tokens=16, n_pages=n_pages, max_pages=width)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    t, _ = _plan(geom, kv, new, free, n_free, tables, 21, err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    _same(t, ao.kv_plan(16, n_pages, width, kv, new, free, n_free, tables, 21))
    assert sorted(t["block_table"].cpu().numpy()[[0, 2, 2], [2, 0, 1]]) == sorted(tables[1, :3])


@pytest.mark.parametrize("short", [1, 3, 8])
def test_plan_too_few_pages(short):
    """Rows in order until one does not fit: reported; it and the later ones get none, unless they need none."""
    m = AH.gdn()
    kv, new = [15, 31, 3, 40, 16, 5], [2, 40, 1, 70, 1, 0]
    n_pages, width, tables, free, n_free = _plan_inputs(4, kv, new, 16, -short)
    geom = m.AttnGeometry(n_q_heads=1, n_kv_heads=1, d_head=64, page_tokens=16, n_pages=n_pages, max_pages=width)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    cap = sum(new)
    t, _ = _plan(geom, kv, new, free, n_free, tables, cap, err)
    torch.cuda.synchronize()
    assert int(err.item()) == m.DEV_NO_PAGES
    ref = ao.kv_plan(16, n_pages, width, kv, new, free, n_free, tables, cap)
    _same(t, ref)
    assert ref["kv_len_out"][2] == 4 and ref["kv_len_out"][5] == 5  # they need no page


def test_plan_refused_values():
    m = AH.gdn()
    kv, new = [10, 20, 30], [5, 7, 3]
    n_pages, width, tables, free, n_free = _plan_inputs(5, kv, new, 16, 4)
    geom = m.AttnGeometry(n_q_heads=1, n_kv_heads=1, d_head=64, page_tokens=16, n_pages=n_pages, max_pages=width)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run(kv=kv, new=new, tables=tables, free=free, n_free=n_free, cap=15):
        err.zero_()
        t, _ = _plan(geom, kv, new, free, n_free, tables, cap, err)
        torch.cuda.synchronize()
        return int(err.item()), {k: v.cpu().numpy() for k, v in t.items()}

    for bad_kv, bad_new in ((-1, 7), (20, -2), (width * 16 - 6, 7), (2 ** 31 - 1, 7), (20, 2 ** 31 - 1), (-2 ** 31, -1)):
        code, t = run(kv=[10, bad_kv, 30], new=[5, bad_new, 3])
        assert code == m.DEV_BAD_LENGTH, (bad_kv, bad_new)
        assert t["kv_len_out"].tolist() == [15, bad_kv, 33] and t["cu_new"][1] == 5
        assert np.all(t["slot_map"][5:5 + max(0, min(bad_new, 7))] == -1)
        assert t["slot_map"][0] == tables[0, 0] * 16 + 10
    code, t = run(cap=9)
    assert code == m.DEV_BAD_SEQLENS and t["cu_new"].tolist() == [0, 5, 9, 9]
    assert np.all(t["slot_map"] >= 0)
    for bad in (-1, n_pages + 1):
        code, t = run(n_free=bad)
        assert code == m.DEV_BAD_PAGE and np.all(t["slot_map"] == -1) and t["n_free_out"] == bad
        assert t["kv_len_out"].tolist() == kv and np.array_equal(t["block_table"], tables)
    broken = tables.copy()
    broken[1, 1] = n_pages
    code, t = run(tables=broken)
    assert code == m.DEV_BAD_PAGE and np.all(t["slot_map"][5:12] == -1) and np.all(t["slot_map"][:5] >= 0)


def test_plan_sums_past_31_bits():
    """Lengths that are refused still count as tokens: their sum stays at the slot map's size, the served rows before
    them get theirs, the ones behind none."""
    m = AH.gdn()
    kv, new = [10, 20, 20, 20, 30], [5, 2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1, 3]
    n_pages, width, tables, free, n_free = _plan_inputs(6, kv, [5, 7, 7, 7, 3], 16, 4)
    geom = m.AttnGeometry(n_q_heads=1, n_kv_heads=1, d_head=64, page_tokens=16, n_pages=n_pages, max_pages=width)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    t, _ = _plan(geom, kv, new, free, n_free, tables, 700, err)
    torch.cuda.synchronize()
    assert int(err.item()) in (m.DEV_BAD_LENGTH, m.DEV_BAD_SEQLENS)  # both hold; the first that lands is kept
    assert t["cu_new"].tolist() == [0, 5, 700, 700, 700, 700]
    assert t["kv_len_out"].tolist() == [15, 20, 20, 20, 33]
    slots = t["slot_map"].cpu().numpy()
    assert slots[0] == tables[0, 0] * 16 + 10 and np.all(slots[5:] == -1)


@pytest.mark.parametrize("N,Hk,D,page,dtype,fused", [
    (1, 1, 64, 16, BF16, False), (5, 4, 256, 16, BF16, True), (530, 2, 128, 528, BF16, False), (100, 8, 64, 32, F32, True),
    (3000, 1, 256, 48, F32, False)])
def test_write_places_every_row_once(N, Hk, D, page, dtype, fused):
    """Every row at its slot, bit for bit, rows of slot -1 nowhere, everything else untouched."""
    m = AH.gdn()
    n_pages = -(-N // page) + 2
    geom = m.AttnGeometry(n_q_heads=Hk, n_kv_heads=Hk, d_head=D, page_tokens=page, n_pages=n_pages, max_pages=n_pages,
                          dtype=dtype)
    rng = np.random.Generator(np.random.PCG64(N))
    slots = rng.permutation(n_pages * page)[:N].astype(np.int32)
    slots[rng.random(N) < 0.1] = -1
    rows, parts = AH.qkv(N, N, Hk, Hk, D, dtype, fused)
    _, k, v = AH.to_gpu(rows, parts, fused, Hk, Hk)
    cache = m.KVCache(*(torch.randn(n_pages, Hk, page, D, generator=torch.Generator().manual_seed(s)).to(dtype).cuda()
                        for s in (1, 2)))
    want = []
    for pages, part in ((cache.k, parts[1]), (cache.v, parts[2])):
        w = pages.cpu().clone()
        for t, s in enumerate(slots):
            if s >= 0:
                w[s // page, :, s % page] = part[t]
        want.append(w)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    m.kv_write(geom, cache, k, v, _cuda(slots), dev_err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    assert torch.equal(cache.k.cpu(), want[0]) and torch.equal(cache.v.cpu(), want[1])
    before = cache.k.clone()
    for bad in (-2, n_pages * page, 2 ** 31 - 1):
        err.zero_()
        m.kv_write(geom, cache, k[:1], v[:1], _cuda([bad]), dev_err=err)
        torch.cuda.synchronize()
        assert int(err.item()) == m.DEV_BAD_PAGE and torch.equal(cache.k, before)


def test_write_no_tokens():
    m = AH.gdn()
    geom = m.AttnGeometry(n_q_heads=1, n_kv_heads=1, d_head=64, n_pages=2, max_pages=2)
    cache = m.KVCache.zeros(geom)
    e = torch.empty(0, 1, 64, dtype=BF16, device="cuda")
    m.kv_write(geom, cache, e, e, torch.empty(0, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert not cache.k.any()


def test_operators_together():
    """A serving run of three requests: prompts planned, attended and written; a tree of drafts attended; the accepted
    path planned and written; then a decode step.  Every attention output equals the fp64 attention over the request's
    whole token sequence, so each operator's product is what the next one reads."""
    m = AH.gdn()
    Hk, G, D, page, dtype = 2, 3, 128, 16, BF16
    Hq, B, scale = Hk * G, 3, D ** -0.5
    geom = m.AttnGeometry(n_q_heads=Hq, n_kv_heads=Hk, d_head=D, page_tokens=page, n_pages=40, max_pages=12, max_tree=6)
    cache = m.KVCache.zeros(geom)
    cache.k.fill_(float("nan"))
    cache.v.fill_(float("nan"))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    table = torch.full((B, 12), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(40, generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda()
    n_free, kv_len = _cuda([40]), _cuda([0, 0, 0])
    held = [([], []) for _ in range(B)]  # every request's committed k and v

    def plan(new, cap):
        nonlocal n_free, kv_len
        i32 = lambda n: torch.empty(n, dtype=torch.int32, device="cuda")  # noqa: E731
        cu, slots, pos, out, nf = i32(B + 1), i32(cap), i32(cap), i32(B), i32(1)
        m.kv_plan(geom, kv_len, _cuda(new), free, n_free, table, cu, slots, pos, out, nf, dev_err=err)
        before, kv_len, n_free = kv_len, out, nf
        return before, cu, slots, pos

    def dense(i, q, k, v, seen_own):
        kk, vv = (np.concatenate([np.asarray(held[i][e]).reshape(-1, Hk, D), t]) for e, t in ((0, k), (1, v)))
        c = len(held[i][0])
        seen = np.concatenate([np.ones((len(q), c), bool), seen_own], axis=1)
        ref, mag = ao.attend(q, kk, vv, seen, scale)
        return ref, AH.tolerance(ref, mag, q, kk, scale, len(kk), dtype)

    # prompts in two chunks: the second attends the first through the cache
    for step, new in enumerate(([37, 5, 64], [20, 0, 3])):
        N = sum(new)
        rows, parts = AH.qkv(200 + step, N + 4, Hq, Hk, D, dtype, True)
        q, k, v = AH.to_gpu(rows, parts, True, Hq, Hk)
        ctx, cu, slots, pos = plan(new, N + 4)
        o = torch.empty(N + 4, Hq, D, dtype=dtype, device="cuda")
        m.attn_prefill(geom, q, k, v, cu, o, m.alloc_attn_prefill_workspace(geom, N + 4, B), cache=cache, block_table=table,
                       ctx_len=ctx, dev_err=err)
        m.kv_write(geom, cache, k, v, slots, dev_err=err)
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        at = 0
        qh, kh, vh = (AH.host(p) for p in parts)
        for i, n in enumerate(new):
            if n:
                ref, tol = dense(i, qh[at:at + n], kh[at:at + n], vh[at:at + n], np.tril(np.ones((n, n), bool)))
                assert (np.abs(AH.host(o[at:at + n]) - ref) <= tol).all(), (step, i)
                assert pos[at:at + n].cpu().tolist() == list(range(len(held[i][0]), len(held[i][0]) + n))
            held[i][0].extend(kh[at:at + n])
            held[i][1].extend(vh[at:at + n])
            at += n
    # a tree of drafts per request
    n = 6
    par = np.array([[-1, 0, 0, 1, 2, 4], [-1, -1, 1, 2, 3, 4], [-1, 0, 1, 2, 3, 4]], np.int32)
    accepted = [[0, 2, 4], [], [0, 1, 2, 3, 4, 5]]  # each request's accepted path
    rows, parts = AH.qkv(300, B * n, Hq, Hk, D, dtype, False)
    q, k, v = (p.cuda().unflatten(0, (B, n)) for p in parts)
    o = torch.empty(B, n, Hq, D, dtype=dtype, device="cuda")
    ws = m.alloc_attn_tree_workspace(geom, B, n)
    m.attn_tree(geom, cache, table, kv_len, q, k, v, _cuda(par), o, ws, dev_err=err)
    qh, kh, vh = (AH.host(p).reshape(B, n, -1, D) for p in parts)
    for i in range(B):
        ref, tol = dense(i, qh[i], kh[i], vh[i], ao.tree_paths(par[i]))
        assert (np.abs(AH.host(o[i]) - ref) <= tol).all(), i
    # the accepted nodes, in path order, become tokens
    _, _, slots, _ = plan([len(p) for p in accepted], B * n)
    where = torch.full((B * n,), -1, dtype=torch.int32, device="cuda")
    picks = torch.tensor([i * n + j for i, p in enumerate(accepted) for j in p], device="cuda")
    where[picks] = slots[:len(picks)]
    m.kv_write(geom, cache, k.flatten(0, 1), v.flatten(0, 1), where, dev_err=err)
    for i, p in enumerate(accepted):
        held[i][0].extend(kh[i, p])
        held[i][1].extend(vh[i, p])
    # one decode step; then request 0 leaves and its pages come back
    rows, parts = AH.qkv(400, B, Hq, Hk, D, dtype, True)
    q, k, v = (t.unflatten(0, (B, 1)) for t in AH.to_gpu(rows, parts, True, Hq, Hk))
    o = torch.empty(B, 1, Hq, D, dtype=dtype, device="cuda")
    m.attn_tree(geom, cache, table, kv_len, q, k, v, _cuda([[-1]] * B), o, ws, dev_err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    qh, kh, vh = (AH.host(p).reshape(B, 1, -1, D) for p in parts)
    for i in range(B):
        ref, tol = dense(i, qh[i], kh[i], vh[i], np.ones((1, 1), bool))
        assert (np.abs(AH.host(o[i]) - ref) <= tol).all(), i
    assert kv_len.cpu().tolist() == [len(h[0]) for h in held]
    before = int(n_free.item())
    plan([-1, 0, 0], 0)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    assert int(n_free.item()) == before + -(-len(held[0][0]) // page) and kv_len.cpu().tolist()[0] == 0


@pytest.mark.parametrize("bad_stack", [False, True])
def test_plan_with_the_longest_slot_map(bad_stack):
    """max_tokens of 2^31 - 1: every padding entry is written, up to the last, and none outside the tables."""
    m = AH.gdn()
    kv, new = [10, 0], [5, 3]
    n_pages, width, tables, free, n_free = _plan_inputs(8, kv, new, 16, 2)
    geom = m.AttnGeometry(n_q_heads=1, n_kv_heads=1, d_head=64, page_tokens=16, n_pages=n_pages, max_pages=width)
    N, edge = 2 ** 31 - 1, 64
    i32 = dict(dtype=torch.int32, device="cuda")
    both = torch.full((2, N + 2 * edge), -3, **i32)  # 17 GB
    slot_map, position = both[0, edge:edge + N], both[1, edge:edge + N]
    out = [torch.full((n,), -3, **i32) for n in (3, 2, 1)]
    err = torch.zeros(1, **i32)
    m.kv_plan(geom, _cuda(kv), _cuda(new), _cuda(free), _cuda([n_pages + 1 if bad_stack else n_free]), _cuda(tables), out[0],
              slot_map, position, out[1], out[2], dev_err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == (m.DEV_BAD_PAGE if bad_stack else 0)
    used = 0 if bad_stack else 8
    if not bad_stack:
        ref = ao.kv_plan(16, n_pages, width, kv, new, free, n_free, tables, 8)
        assert slot_map[:8].tolist() == ref["slot_map"].tolist() and position[:8].tolist() == ref["position"].tolist()
    assert bool((slot_map[used:] == -1).all()) and bool((position[used:] == 0).all())
    assert bool((both[:, :edge] == -3).all()) and bool((both[:, edge + N:] == -3).all())
