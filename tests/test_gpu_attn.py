"""Attention over packed prompts and over trees of drafts, on the GPU, against the fp64 oracle: head layouts, lengths
from none to several tiles, pages that end inside a tile, fused rows, splits of the key axis, poisoned memory, refused
rows, streams and graphs."""
import numpy as np
import pytest
import torch

import attn_harness as AH
from oracle import attn_oracle as ao

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def _err():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def _cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(torch.int32).cuda()


def _check(got, ref, mag, q, k, scale, n_keys, dtype, what):
    got = AH.host(got)
    tol = AH.tolerance(ref, mag, q, k, scale, n_keys, dtype)
    off = np.abs(got - ref)
    assert np.isfinite(got).all(), f"{what}: not finite"
    worst = np.max(off / tol)
    assert worst <= 1.0, f"{what}: {worst:.2f} times its bound"


def _prefill_case(seed, new, ctx, Hk, G, D, page, dtype, fused=False, pad=0, scale=None):
    m = AH.gdn()
    Hq, N = Hk * G, sum(new) + pad
    pg = AH.Paged(seed, ctx, Hk, D, page, dtype)
    rows, parts = AH.qkv(seed + 1, N, Hq, Hk, D, dtype, fused)
    if pad:
        rows[sum(new):] = float("nan")
        parts = (rows[:, :Hq], rows[:, Hq:Hq + Hk], rows[:, Hq + Hk:])
        parts = parts if fused else tuple(p.contiguous() for p in parts)
    geom = m.AttnGeometry(n_q_heads=Hq, n_kv_heads=Hk, d_head=D, page_tokens=page, n_pages=pg.n_pages, max_pages=pg.width,
                          dtype=dtype, scale=scale)
    q, k, v = AH.to_gpu(rows, parts, fused, Hq, Hk)
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    o = torch.full((N, Hq, D), 7.0, dtype=dtype, device="cuda")
    return m, geom, pg, parts, (q, k, v), cu, o


def _run_prefill(m, geom, pg, dev, cu, ctx, o, err, paged=True):
    ws = m.alloc_attn_prefill_workspace(geom, o.shape[0], len(cu) - 1)
    extra = dict(cache=pg.cache(), block_table=pg.table.cuda(), ctx_len=_cuda(ctx)) if paged else {}
    m.attn_prefill(geom, *dev, _cuda(cu), o, ws, dev_err=err, **extra)


PREFILL = [
    # new, cached tokens of each sequence; KV heads, group, D, page, dtype, fused rows, padding rows
    ([1], [0], 1, 1, 64, 16, BF16, False, 0),
    ([1, 0, 33, 130, 64], [0, 5, 100, 0, 17], 2, 3, 64, 16, BF16, True, 3),
    ([65, 2, 1], [15, 528, 529], 2, 4, 128, 528, BF16, False, 0),
    ([300], [0], 4, 6, 256, 16, BF16, True, 0),
    ([7, 129], [1000, 31], 1, 8, 256, 32, BF16, False, 1),
    ([513, 5], [0, 2], 2, 1, 128, 16, BF16, False, 0),
    ([1, 0, 33, 70], [3, 0, 64, 0], 2, 3, 64, 16, F32, True, 5),
    ([40, 1], [0, 77], 1, 2, 128, 48, F32, False, 0),
    ([35, 3], [20, 0], 2, 2, 256, 16, F32, False, 0),
    ([5, 41], [0, 33], 1, 64, 64, 16, BF16, True, 2),
    ([3, 9], [17, 0], 1, 64, 128, 16, F32, False, 0),
]


@pytest.mark.parametrize("new,ctx,Hk,G,D,page,dtype,fused,pad", PREFILL)
def test_prefill_against_the_oracle(new, ctx, Hk, G, D, page, dtype, fused, pad):
    """Packed prompts after cached prefixes; empty sequences; rows behind the last sequence stay as they were (and
    what they hold, NaN, reaches nothing)."""
    print(f"prefill new {new} ctx {ctx} Hk {Hk} G {G} D {D} page {page} {dtype}", flush=True)
    m, geom, pg, parts, dev, cu, o = _prefill_case(11 + D + len(new), new, ctx, Hk, G, D, page, dtype, fused, pad)
    err = _err()
    _run_prefill(m, geom, pg, dev, cu, ctx, o, err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    n = sum(new)
    q, k, v = (AH.host(p)[:n] for p in parts)
    scale = D ** -0.5
    ref, mag = ao.prefill(q, k, v, cu, AH.host(pg.k), AH.host(pg.v), pg.table.numpy(), ctx, scale)
    kk = np.concatenate([k, np.nan_to_num(AH.host(pg.k)).transpose(0, 2, 1, 3).reshape(-1, Hk, D)])
    _check(o[:n], ref, mag, q, kk, scale, max(a + b for a, b in zip(new, ctx)), dtype, "prefill")
    assert torch.all(o[n:] == 7.0), "rows behind the last sequence were written"


def test_prefill_without_a_cache_equals_empty_prefixes():
    """ctx_len None takes no cache at all and gives the result of lengths of zero, bit for bit."""
    new = [90, 1, 200]
    m, geom, pg, parts, dev, cu, o = _prefill_case(5, new, [0, 0, 0], 2, 4, 128, 16, BF16)
    o2, err = o.clone(), _err()
    _run_prefill(m, geom, pg, dev, cu, [0, 0, 0], o, err)
    _run_prefill(m, geom, pg, dev, cu, None, o2, err, paged=False)
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and torch.equal(o, o2)


@pytest.mark.parametrize("dtype,D", [(BF16, 64), (BF16, 128), (BF16, 256), (F32, 64)])
def test_prefill_later_tokens_reach_no_earlier_row(dtype, D):
    """Infinities and NaN in the K and V of later tokens leave the rows before them bit for bit as they were; the rows
    that attend them become NaN or infinite as the definition says."""
    new, ctx = [150], [37]
    m, geom, pg, parts, dev, cu, o = _prefill_case(6, new, ctx, 2, 3, D, 16, dtype)
    clean, err = o.clone(), _err()
    _run_prefill(m, geom, pg, dev, cu, ctx, clean, err)
    k, v = dev[1].clone(), dev[2].clone()
    v[70, 0, 3] = float("inf")
    v[70, 1, 5] = float("nan")
    k[100, 0, 1] = float("nan")
    v[131, :, :] = float("-inf")
    _run_prefill(m, geom, pg, (dev[0], k, v), cu, ctx, o, err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    assert torch.equal(o[:70], clean[:70])
    first = o[70:100].float()
    assert torch.isinf(first[:, :3, 3]).all() and torch.isnan(first[:, 3:, 5]).all()
    keep = torch.ones_like(first, dtype=torch.bool)
    keep[:, :3, 3] = keep[:, 3:, 5] = False
    ref = clean[70:100].float()
    # both results have the same weights; the sums differ in order (2 n u sum p |v| with |v| <= 6 here) and, for bf16,
    # in whether key 70's weight was rounded (h p |v|) and in the outputs' rounding (h |ref| each)
    assert float(clean.abs().max()) < 6 and float(parts[2][:, :].abs().max()) < 6
    tol = 2 * 187 * 2.0 ** -24 * 6 + (AH.half_step(dtype) * (2 * ref.abs() + 6) if dtype == BF16 else 0.0)
    assert ((first - ref).abs() <= tol)[keep].all()
    assert torch.isnan(o[100:, :3].float()).all()
    assert torch.isfinite(o[100:131, 3:].float())[:, :, :5].all() and not torch.isfinite(o[131:, 3:].float()).any()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_prefill_large_logits(dtype):
    """Logits of several thousand: the running maximum keeps the weights in range; one key takes (nearly) all of a row."""
    new, ctx, D = [80], [50], 64
    m, geom, pg, parts, dev, cu, o = _prefill_case(8, new, ctx, 1, 2, D, 16, dtype, scale=40.0)
    err = _err()
    _run_prefill(m, geom, pg, dev, cu, ctx, o, err)
    torch.cuda.synchronize()
    q, k, v = (AH.host(p) for p in parts)
    ref, mag = ao.prefill(q, k, v, cu, AH.host(pg.k), AH.host(pg.v), pg.table.numpy(), ctx, 40.0)
    kk = np.concatenate([k, np.nan_to_num(AH.host(pg.k)).transpose(0, 2, 1, 3).reshape(-1, 1, D)])
    _check(o, ref, mag, q, kk, 40.0, 130, dtype, "large logits")


def test_prefill_refused_sequences():
    """A cached length that does not fit the table, and bounds that are not a partition: reported, the sequence's rows
    stay as they were, the others are right; a page outside the cache is reported."""
    new, ctx = [20, 30, 10], [16, 40, 0]
    m, geom, pg, parts, dev, cu, o = _prefill_case(9, new, ctx, 1, 2, 64, 16, BF16)
    good, err = o.clone(), _err()
    _run_prefill(m, geom, pg, dev, cu, ctx, good, err)
    bad = [16, pg.width * 16 + 1, 0]
    _run_prefill(m, geom, pg, dev, cu, bad, o, err)
    torch.cuda.synchronize()
    assert int(err.item()) == m.DEV_BAD_LENGTH
    assert torch.all(o[20:50] == 7.0) and torch.equal(o[:20], good[:20]) and torch.equal(o[50:], good[50:])
    for broken in ([0, 20, 10, 60], [0, 20, 50, 61], [1, 20, 50, 60], [-5, 20, 50, 60]):
        err.zero_()
        o.fill_(7.0)
        _run_prefill(m, geom, pg, dev, np.array(broken, np.int32), ctx, o, err)
        torch.cuda.synchronize()
        assert int(err.item()) == m.DEV_BAD_SEQLENS, broken
    err.zero_()
    table = pg.table.clone()
    table[1, 0] = pg.n_pages
    m.attn_prefill(geom, *dev, _cuda(cu), o, m.alloc_attn_prefill_workspace(geom, 60, 3), cache=pg.cache(),
                   block_table=table.cuda(), ctx_len=_cuda(ctx), dev_err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == m.DEV_BAD_PAGE and torch.equal(o[:20], good[:20]) and torch.equal(o[50:], good[50:])


def _check_sequences(pg, parts, cu, ctx, o, scale, dtype, what):
    """Every sequence of a packed batch on its own (its keys alone set its bound)."""
    q, k, v = (AH.host(p) for p in parts)
    kc, vc = AH.host(pg.k), AH.host(pg.v)
    Hk, D = k.shape[1:]
    for i, c in enumerate(ctx):
        lo, hi = int(cu[i]), int(cu[i + 1])
        if lo == hi:
            continue
        ref, mag = ao.prefill(q[lo:hi], k[lo:hi], v[lo:hi], np.array([0, hi - lo]), kc, vc, pg.table[i:i + 1].numpy(), [c], scale)
        pages = np.nan_to_num(kc[pg.table[i, :-(-c // kc.shape[2])].numpy()]).transpose(0, 2, 1, 3).reshape(-1, Hk, D)
        _check(o[lo:hi], ref, mag, q[lo:hi], np.concatenate([k[lo:hi], pages]), scale, c + hi - lo, dtype, f"{what} {i}")


@pytest.mark.parametrize("S,Hk,G,D,dtype", [(64, 1, 3, 64, BF16), (65, 2, 2, 128, BF16), (150, 1, 4, 64, BF16), (70, 2, 3, 64, F32)])
def test_prefill_many_sequences(S, Hk, G, D, dtype):
    """Up to and past 64 sequences: empty ones, single tokens, several blocks of rows, prefixes of all lengths, two of
    each length so that blocks of equal lengths meet."""
    rng = np.random.Generator(np.random.PCG64(S))
    half = [int(n) for n in rng.integers(0, 120, size=S // 2)]
    new = (half + half + [300])[:S] if S % 2 == 0 else half + half + [300]
    ctx = [int(c) for c in rng.integers(0, 90, size=S // 2)]
    ctx = ctx + ctx + [0] * (S - 2 * (S // 2))
    new[1], new[2], ctx[2] = 0, 1, 0
    m, geom, pg, parts, dev, cu, o = _prefill_case(500 + S, new, ctx, Hk, G, D, 16, dtype)
    err = _err()
    _run_prefill(m, geom, pg, dev, cu, ctx, o, err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    _check_sequences(pg, parts, cu, ctx, o, D ** -0.5, dtype, "sequence")


@pytest.mark.parametrize("D,dtype", [(64, BF16), (128, BF16), (256, BF16), (128, F32)])
def test_prefill_few_rows_behind_long_prefixes(D, dtype):
    """Few rows, many keys: the key axis is split, with parts that hold no key of the shorter rows, and joined; a
    sequence of its own and the same one in a batch of three differ by their rounding only."""
    new, ctx = [3, 1, 20], [3000, 0, 517]
    m, geom, pg, parts, dev, cu, o = _prefill_case(520 + D, new, ctx, 1, 4, D, 16, dtype)
    assert m.attn_prefill_workspace_bytes(geom, sum(new), 3) > 0
    err = _err()
    _run_prefill(m, geom, pg, dev, cu, ctx, o, err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    _check_sequences(pg, parts, cu, ctx, o, D ** -0.5, dtype, "sequence")


@pytest.mark.parametrize("S,cut,D,dtype", [(60, 17, 64, F32), (20, 51, 64, F32), (31, 33, 128, F32), (19, 53, 128, F32),
                                           (31, 33, 256, F32), (5, 51, 128, BF16), (14, 19, 64, BF16), (7, 36, 256, BF16)])
def test_prefill_odd_numbers_of_parts(S, cut, D, dtype):
    """Single tokens, one behind a prefix that fills `cut` parts of the key axis, as many as a call of this many
    sequences makes, mostly no multiple of the parts that a turn of the join takes."""
    new, ctx = [1] * S, [128 * cut - 1] + [5] * (S - 1)
    m, geom, pg, parts, dev, cu, o = _prefill_case(540 + S + D, new, ctx, 1, 1, D, 16, dtype)
    err = _err()
    _run_prefill(m, geom, pg, dev, cu, ctx, o, err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    _check_sequences(pg, parts, cu, ctx, o, D ** -0.5, dtype, "sequence")


def test_prefill_refused_sequence_among_many():
    """Blocks are ordered by their keys across sequences: a refused one leaves the others right, wherever it stands."""
    new, ctx = [40, 90, 40, 7, 200], [0, 64, 0, 300, 16]
    m, geom, pg, parts, dev, cu, o = _prefill_case(530, new, ctx, 2, 4, 64, 16, BF16)
    err = _err()
    for at in range(5):
        bad = list(ctx)
        bad[at] = -1
        err.zero_()
        o.fill_(7.0)
        _run_prefill(m, geom, pg, dev, cu, bad, o, err)
        torch.cuda.synchronize()
        assert int(err.item()) == m.DEV_BAD_LENGTH
        assert torch.all(o[cu[at]:cu[at + 1]] == 7.0)
        for i in range(5):
            if i == at:
                continue
            one = slice(int(cu[i]), int(cu[i + 1]))
            alone = torch.full_like(o[one], 7.0)
            m.attn_prefill(geom, *(t[one] for t in dev), _cuda([0, new[i]]), alone,
                           m.alloc_attn_prefill_workspace(geom, new[i], 1), cache=pg.cache(),
                           block_table=pg.table[i:i + 1].cuda(), ctx_len=_cuda([ctx[i]]), dev_err=_err())
            torch.cuda.synchronize()
            # each result's weights are rounded, against its own running maximum (h sum p |v|, |v| < max |v| + 4
            # in the cache too), and each output (h |o|)
            off = (alone.float() - o[one].float()).abs()
            assert (off <= 2 * AH.half_step(BF16) * (alone.float().abs() + float(parts[2].abs().max()) + 4)).all()


# Row counts n G that end one block of 256 rows inside the heads of the last token: 0 < n G mod 256 < G.
STRADDLE = [(3, 86), (3, 171), (5, 52), (6, 43), (6, 86), (6, 171), (7, 37), (12, 22)]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G,n", STRADDLE)
def test_prefill_last_token_in_two_row_blocks(G, n, D):
    """The last two row blocks attend the same keys: alone and behind a prefix (few rows: the key axis is split), twice
    the same beside others, and in so many sequences that it is not split.  No row keeps what the output held."""
    assert 0 < n * G % 256 < G
    print(f"last token in two row blocks: G {G} n {n} D {D}", flush=True)
    for seed, (new, ctx, Hk) in enumerate((([n], [0], 1), ([n], [700], 2), ([n, 5, n, 33, n - 1], [64, 0, 64, 130, 0], 2),
                                           ([n] * 40, [0, 17] * 20, 4))):
        m, geom, pg, parts, dev, cu, o = _prefill_case(900 + seed + D + G, new, ctx, Hk, G, D, 16, BF16)
        split = m.attn_prefill_workspace_bytes(geom, sum(new), len(new)) > 0
        assert split == (len(new) < 40)
        o.fill_(float("nan"))
        err = _err()
        _run_prefill(m, geom, pg, dev, cu, ctx, o, err)
        torch.cuda.synchronize()
        assert int(err.item()) == 0 and torch.isfinite(o).all()
        _check_sequences(pg, parts, cu, ctx[:5], o, D ** -0.5, BF16, f"G {G} n {n} D {D} batch {seed} sequence")


@pytest.mark.parametrize("S,at,back,N,G,D,dtype", [
    (3, 1, 2, 150, 1, 64, F32), (5, 3, 40, 400, 3, 128, F32), (130, 70, 90, 3900, 2, 64, F32),
    (70, 65, 300, 2100, 3, 64, BF16), (150, 20, 5, 4500, 1, 128, BF16), (64, 40, 700, 6400, 4, 256, BF16), (4, 2, 60, 320, 6, 64, BF16)])
def test_prefill_a_sequence_that_ends_before_it_begins(S, at, back, N, G, D, dtype):
    """Bounds that go back: reported in every form of the call, the sequences before are right, that one and those
    behind it stay as they were."""
    new = [N // S] * S
    m, geom, pg, parts, dev, cu, o = _prefill_case(940 + S + at, new, [0] * S, 1, G, D, 16, dtype)
    cu = cu.copy()
    cu[at + 1:] -= new[at] + back  # sequence `at` ends `back` tokens before it begins, the others follow on
    assert cu[at + 1] == cu[at] - back
    err = _err()
    _run_prefill(m, geom, pg, dev, cu, None, o, err, paged=False)
    torch.cuda.synchronize()
    assert int(err.item()) == m.DEV_BAD_SEQLENS
    ok = int(cu[at])
    _check_sequences(pg, parts, cu, [0] * at, o, D ** -0.5, dtype, "sequence")
    assert torch.all(o[ok:] == 7.0)


# ---------------------------------------------------------------------------
# trees
# ---------------------------------------------------------------------------

def _tree_case(seed, ctx, n, Hk, G, D, page, dtype, fused=False, max_tree=None):
    m = AH.gdn()
    B, Hq = len(ctx), Hk * G
    pg = AH.Paged(seed, ctx, Hk, D, page, dtype)
    rows, parts = AH.qkv(seed + 1, B * n, Hq, Hk, D, dtype, fused)
    geom = m.AttnGeometry(n_q_heads=Hq, n_kv_heads=Hk, d_head=D, page_tokens=page, n_pages=pg.n_pages, max_pages=pg.width,
                          max_tree=max_tree or max(n, 1), dtype=dtype)
    dev = tuple(t.unflatten(0, (B, n)) for t in AH.to_gpu(rows, parts, fused, Hq, Hk))
    par = AH.parents(seed + 2, B, n)
    o = torch.full((B, n, Hq, D), 7.0, dtype=dtype, device="cuda")
    return m, geom, pg, parts, dev, par, o


def _run_tree(m, geom, pg, dev, par, ctx, o, err, n_row=None, ws=None, cache=None):
    B, n = o.shape[:2]
    if ws is None:
        ws = m.alloc_attn_tree_workspace(geom, B, n)
        ws.fill_(0x7f)  # what a workspace held before must not matter
    m.attn_tree(geom, cache or pg.cache(), pg.table.cuda(), _cuda(ctx), *dev, _cuda(par), o, ws, dev_err=err,
                n_row=None if n_row is None else _cuda(n_row))


def _check_tree(pg, parts, par, ctx, o, n_row, G, D, dtype, what):
    B, n = o.shape[:2]
    Hk = pg.k.shape[1]
    q, k, v = (AH.host(p).reshape(B, n, -1, D) for p in parts)
    kc, vc = AH.host(pg.k), AH.host(pg.v)
    kk = np.concatenate([k.reshape(-1, Hk, D), np.nan_to_num(kc).transpose(0, 2, 1, 3).reshape(-1, Hk, D)])
    for i in range(B):
        e = n if n_row is None else n_row[i]
        ref, mag = ao.tree(q[i, :e], k[i, :e], v[i, :e], par[i, :e], kc, vc, pg.table[i].numpy(), ctx[i], D ** -0.5)
        _check(o[i, :e], ref, mag, q[i], kk, D ** -0.5, ctx[i] + e, dtype, f"{what} row {i}")
        assert torch.all(o[i, e:] == 7.0), f"{what}: row {i}: nodes past its count were written"


TREE = [
    # cached tokens per row, nodes, KV heads, group, D, page, dtype, fused, per-row counts
    ([0], 1, 1, 1, 64, 16, BF16, False, None),
    ([1, 0, 700, 31], 1, 4, 6, 256, 16, BF16, True, None),
    ([64, 0, 333], 7, 2, 3, 128, 16, BF16, False, [7, 1, 4]),
    ([100, 1057], 16, 4, 6, 256, 528, BF16, False, None),
    ([5, 2000, 0], 33, 1, 4, 128, 32, BF16, True, [33, 32, 2]),
    ([40], 64, 2, 8, 64, 16, BF16, False, None),
    ([4000], 3, 1, 2, 128, 48, BF16, False, None),
    ([30, 600], 5, 2, 3, 64, 16, F32, True, [2, 5]),
    ([0, 65], 1, 1, 8, 128, 16, F32, False, None),
    ([129], 9, 1, 2, 256, 16, F32, False, None),
    ([20, 7], 64, 1, 64, 64, 16, BF16, False, [64, 33]),
    ([31], 17, 1, 64, 128, 16, F32, True, None),
]


@pytest.mark.parametrize("ctx,n,Hk,G,D,page,dtype,fused,n_row", TREE)
def test_tree_against_the_oracle(ctx, n, Hk, G, D, page, dtype, fused, n_row):
    """Random trees (single nodes: the decode step) over caches of 0 to 4000 tokens."""
    print(f"tree ctx {ctx} n {n} Hk {Hk} G {G} D {D} page {page} {dtype} n_row {n_row}", flush=True)
    m, geom, pg, parts, dev, par, o = _tree_case(40 + n + D, ctx, n, Hk, G, D, page, dtype, fused)
    err = _err()
    _run_tree(m, geom, pg, dev, par, ctx, o, err, n_row)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    _check_tree(pg, parts, par, ctx, o, n_row, G, D, dtype, "tree")


def test_tree_many_rows():
    """More rows than workgroups need splits for: 70 rows of ragged lengths, one of them empty."""
    rng = np.random.Generator(np.random.PCG64(77))
    ctx = [int(c) for c in rng.integers(0, 200, size=70)]
    ctx[3] = 0
    m, geom, pg, parts, dev, par, o = _tree_case(78, ctx, 4, 8, 2, 64, 16, BF16)
    err = _err()
    _run_tree(m, geom, pg, dev, par, ctx, o, err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    _check_tree(pg, parts, par, ctx, o, None, 2, 64, BF16, "many rows")


@pytest.mark.parametrize("dtype,D", [(BF16, 64), (BF16, 128), (BF16, 256), (F32, 64)])
def test_tree_siblings_do_not_reach_each_other(dtype, D):
    """NaN and infinities in one branch's K and V leave the other branches' rows bit for bit as they were."""
    ctx, n = [90], 12
    m, geom, pg, parts, dev, par, o = _tree_case(50, ctx, n, 2, 3, D, 16, dtype)
    par[0] = [-1, 0, 0, 1, 1, 2, 2, 3, -1, 8, 4, 5]
    clean, err = o.clone(), _err()
    _run_tree(m, geom, pg, dev, par, ctx, clean, err)
    k, v = dev[1].clone(), dev[2].clone()
    v[0, 1] = float("nan")
    v[0, 8] = float("inf")
    k[0, 8] = float("nan")
    _run_tree(m, geom, pg, (dev[0], k, v), par, ctx, o, err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    on = ao.tree_paths(par[0])
    for j in range(n):
        if on[j, 1] or on[j, 8]:
            assert torch.isnan(o[0, j].float()).all(), j
        else:
            assert torch.equal(o[0, j], clean[0, j]), j


def test_tree_refused_rows():
    """Counts, parents and lengths out of range: reported, those rows stay as they were, the others are right."""
    ctx, n = [33, 100, 64, 16], 3
    m, geom, pg, parts, dev, par, o = _tree_case(60, ctx, n, 1, 2, 64, 16, BF16)
    good, err = o.clone(), _err()
    _run_tree(m, geom, pg, dev, par, ctx, good, err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0

    def others(row):
        for i in range(4):
            if i == row:
                assert torch.all(o[i] == 7.0)
            else:
                assert torch.equal(o[i], good[i])

    for what, code in (("count0", m.DEV_BAD_K), ("count4", m.DEV_BAD_K), ("self", m.DEV_BAD_PARENT),
                       ("below", m.DEV_BAD_PARENT), ("length", m.DEV_BAD_LENGTH), ("negative", m.DEV_BAD_LENGTH)):
        err.zero_()
        o.fill_(7.0)
        p, c, nr = par.copy(), list(ctx), None
        if what.startswith("count"):
            nr = [n, int(what[-1]), n, n]
        elif what == "self":
            p[1, 2] = 2
        elif what == "below":
            p[1, 0] = -2
        else:
            c[1] = -1 if what == "negative" else pg.width * 16 + 1
        _run_tree(m, geom, pg, dev, p, c, o, err, nr)
        torch.cuda.synchronize()
        assert int(err.item()) == code, what
        others(1)


@pytest.mark.parametrize("D,dtype", [(64, BF16), (128, BF16), (256, BF16), (64, F32)])
def test_full_tables(D, dtype):
    """Rows whose cached tokens fill their tables to the last entry, the largest length that is accepted, at lengths
    where the page ids of 1024 keys end; one token more is refused."""
    m = AH.gdn()
    for c in (1024, 2048 + 16):
        pg = AH.Paged(95, [c, 5], 1, D, 16, dtype, width_extra=0)
        geom = m.AttnGeometry(n_q_heads=2, n_kv_heads=1, d_head=D, n_pages=pg.n_pages, max_pages=pg.width, max_tree=3,
                              dtype=dtype)
        rows, parts = AH.qkv(96, 6, 2, 1, D, dtype, False)
        dev = tuple(p.cuda() for p in parts)
        o, err = torch.full((6, 2, D), 7.0, dtype=dtype, device="cuda"), _err()
        cu = np.array([0, 3, 6], np.int32)
        _run_prefill(m, geom, pg, dev, cu, [c, 5], o, err)
        tree = torch.full((2, 3, 2, D), 7.0, dtype=dtype, device="cuda")
        par = AH.parents(97, 2, 3)
        _run_tree(m, geom, pg, tuple(t.unflatten(0, (2, 3)) for t in dev), par, [c, 5], tree, err)
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        _check_sequences(pg, parts, cu, [c, 5], o, D ** -0.5, dtype, "sequence")
        _check_tree(pg, parts, par, [c, 5], tree, None, 2, D, dtype, "full table")
        _run_prefill(m, geom, pg, dev, cu, [c + 1, 5], o, err)
        torch.cuda.synchronize()
        assert int(err.item()) == m.DEV_BAD_LENGTH


def test_tree_cache_beyond_32_bit_offsets():
    """Pages that lie more than 2^31 elements and 2^32 bytes into the cache."""
    m = AH.gdn()
    Hk, D, page, n_pages = 8, 256, 64, 18000  # 2.36e9 elements per cache
    geom = m.AttnGeometry(n_q_heads=16, n_kv_heads=Hk, d_head=D, page_tokens=page, n_pages=n_pages, max_pages=3, max_tree=2)
    shape = (n_pages, Hk, page, D)
    cache = m.KVCache(torch.empty(shape, dtype=BF16, device="cuda"), torch.empty(shape, dtype=BF16, device="cuda"))
    ids = [n_pages - 1, 16500, 17999 - 3]
    pg = AH.Paged(90, [150], Hk, D, page, BF16)
    for e, at in enumerate(pg.table[0, :3].tolist()):
        cache.k[ids[e]] = pg.k[at].cuda()
        cache.v[ids[e]] = pg.v[at].cuda()
    rows, parts = AH.qkv(91, 2, 16, Hk, D, BF16, False)
    dev = tuple(p.cuda().unflatten(0, (1, 2)) for p in parts)
    par = np.array([[-1, 0]], np.int32)
    o, err = torch.empty(1, 2, 16, D, dtype=BF16, device="cuda"), _err()
    ws = m.alloc_attn_tree_workspace(geom, 1, 2)
    m.attn_tree(geom, cache, _cuda([ids]), _cuda([150]), *dev, _cuda(par), o, ws, dev_err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    _check_tree(pg, parts, par, [150], o, None, 2, D, BF16, "far pages")


def test_streams_and_graph_replays():
    """Two calls at once on two streams, each with its own workspace, and a captured call replayed with eager work in
    between: every result equals the eager one, bit for bit."""
    ctx, n = [700, 33], 6
    m, geom, pg, parts, dev, par, o = _tree_case(70, ctx, n, 2, 4, 128, 16, BF16)
    err, cache = _err(), pg.cache()
    table, c, p = pg.table.cuda(), _cuda(ctx), _cuda(par)
    eager = o.clone()
    ws = [m.alloc_attn_tree_workspace(geom, 2, n) for _ in range(3)]
    call = lambda out, w: m.attn_tree(geom, cache, table, c, *dev, p, out, w, dev_err=err)  # noqa: E731
    call(eager, ws[0])
    torch.cuda.synchronize()
    outs, streams = [o.clone(), o.clone()], [torch.cuda.Stream(), torch.cuda.Stream()]
    for out, st, w in zip(outs, streams, ws):
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            call(out, w)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], eager) and torch.equal(outs[1], eager)
    new = [50, 90]
    m2, geom2, pg2, _, dev2, cu2, o2 = _prefill_case(71, new, ctx, 2, 4, 128, 16, BF16)
    cache2, table2, c2, cu2 = pg2.cache(), pg2.table.cuda(), _cuda(ctx), _cuda(cu2)
    ws2 = m.alloc_attn_prefill_workspace(geom2, sum(new), 2)
    pre = lambda out: m.attn_prefill(geom2, *dev2, cu2, out, ws2, cache=cache2, block_table=table2, ctx_len=c2,  # noqa: E731
                                     dev_err=err)
    eager2 = o2.clone()
    pre(eager2)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(o, ws[2])
        pre(o2)
    for _ in range(3):
        o.fill_(1.0)
        o2.fill_(1.0)
        call(outs[0], ws[0])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        assert torch.equal(o, eager) and torch.equal(o2, eager2) and torch.equal(outs[0], eager)


@pytest.mark.parametrize("dtype,D", [(BF16, 256), (F32, 64)])
def test_one_workspace_for_calls_of_many_sizes(dtype, D):
    """A workspace for up to 2048 tokens serves every shorter prompt, and one for up to 40 rows every smaller batch of
    trees: results as with a workspace of the call's own, bit for bit."""
    m = AH.gdn()
    ws = None
    for n in (2048, 700, 256, 43, 1):
        mm, geom, pg, parts, dev, cu, o = _prefill_case(980, [n], [0], 1, 6, D, 16, dtype)
        if ws is None:
            ws = m.alloc_attn_prefill_workspace(geom, 2048, 3, up_to=True)
        err, own = _err(), o.clone()
        m.attn_prefill(geom, *dev, _cuda(cu), o, ws, dev_err=err)
        m.attn_prefill(geom, *dev, _cuda(cu), own, m.alloc_attn_prefill_workspace(geom, n, 1), dev_err=err)
        torch.cuda.synchronize()
        assert int(err.item()) == 0 and torch.isfinite(o).all() and torch.equal(o, own)
    ws = None
    for b, n in ((40, 5), (8, 5), (3, 1), (1, 4)):
        mm, geom, pg, parts, dev, par, o = _tree_case(990, [100] * b, n, 1, 6, D, 16, dtype, max_tree=5)
        if ws is None:
            ws = m.alloc_attn_tree_workspace(geom, 40, 5, up_to=True)
        err, own = _err(), o.clone()
        _run_tree(m, geom, pg, dev, par, [100] * b, o, err, ws=ws)
        _run_tree(m, geom, pg, dev, par, [100] * b, own, err)
        torch.cuda.synchronize()
        assert int(err.item()) == 0 and torch.isfinite(o).all() and torch.equal(o, own)


def test_calls_on_a_stream_of_their_own():
    """Calls that name a stream run in its order: inputs that arrive on it late are those that they read, and results
    equal those of the current stream, bit for bit."""
    ctx, n, new = [70, 33], 3, [50, 90]
    m, geom, pg, _, dev, par, o = _tree_case(74, ctx, n, 2, 4, 128, 16, BF16)
    table, c, p = pg.table.cuda(), _cuda(ctx), _cuda(par)
    _, _, _, _, pdev, cu, po = _prefill_case(75, new, ctx, 2, 4, 128, 16, BF16)
    cu, slots = _cuda(cu), _cuda(np.arange(geom.n_pages * 16 - 140, geom.n_pages * 16))
    err, cache = _err(), pg.cache()
    ws = m.alloc_attn_tree_workspace(geom, 2, n), m.alloc_attn_prefill_workspace(geom, 140, 2)

    def calls(q, pq, out, pout, stream):
        written = m.KVCache(cache.k.clone(), cache.v.clone())
        torch.cuda.synchronize()
        if stream is not None:
            with torch.cuda.stream(stream):
                torch.cuda._sleep(20_000_000)
                q.copy_(dev[0], non_blocking=True)
                pq.copy_(pdev[0], non_blocking=True)
        m.attn_tree(geom, cache, table, c, q, *dev[1:], p, out, ws[0], dev_err=err, stream=stream)
        m.attn_prefill(geom, pq, *pdev[1:], cu, pout, ws[1], cache=cache, block_table=table, ctx_len=c, dev_err=err, stream=stream)
        m.kv_write(geom, written, pout[:, :2], pout[:, 2:4], slots, dev_err=err, stream=stream)
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        return out, pout, written.k.view(torch.int16), written.v.view(torch.int16)

    here = calls(dev[0], pdev[0], o.clone(), po.clone(), None)
    late = calls(torch.zeros_like(dev[0]), torch.zeros_like(pdev[0]), o.clone(), po.clone(), torch.cuda.Stream())
    for a, b in zip(here, late):
        assert torch.equal(a, b)
