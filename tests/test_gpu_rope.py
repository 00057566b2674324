"""Rotary positions on the GPU against the fp64 oracle: layouts, scalings, parts of the head, strides, in place, the write
into the cache, far positions, the transposed map as a gradient."""
import numpy as np
import pytest
import torch

import attn_harness as AH
from oracle import cache_oracle as co

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


def _bound(x, y, half, layout, amplitude, dtype):
    """Elementwise bound of |got - y|.  The reduced angle (at most pi / 4) is off by four roundings, 4 U pi / 4, and the
    polynomials' own roundings and rests by 3 U: cos and sin by 7 U; times the amplitude, and two products and a sum: 4 U
    more; so 11 U A (|x_a| + |x_b|), and the output's rounding."""
    h = AH.half_step(dtype)
    e = np.zeros_like(y)
    a, b = (slice(0, half), slice(half, 2 * half)) if layout == "half" else (slice(0, 2 * half, 2), slice(1, 2 * half, 2))
    size = 11 * U * amplitude * (np.abs(x[..., a]) + np.abs(x[..., b]))
    e[..., a], e[..., b] = size, size
    e[..., :2 * half] += h * np.abs(y[..., :2 * half])
    return 1.02 * e


def _rows(seed, n, heads, d, dtype, pad):
    """Rows on the GPU, `pad` more elements apart than they are long."""
    g = torch.Generator().manual_seed(seed)
    whole = torch.randn(n, heads * d + pad, generator=g).to(dtype).cuda()
    return whole[:, :heads * d].unflatten(1, (heads, d))


def _check(got, x, position, rope, freq, dtype):
    x64, half = AH.host(x), rope.rot_dims // 2
    y = co.rotate(x64, position.tolist(), freq, rope.layout, float(np.float32(rope.amplitude)), rope.inverse)
    d = np.abs(AH.host(got) - y)
    assert np.all(d <= _bound(x64, y, half, rope.layout, rope.amplitude, dtype)), d.max()
    assert torch.equal(got[..., 2 * half:], x[..., 2 * half:])


CASES = [
    # n, Hq, Hk, D, rot, layout, scaling, dtype, padding of the rows
    (1, 1, 1, 64, 16, "half", "none", BF16, 0),
    (1, 24, 4, 256, 64, "half", "none", BF16, 64),
    (5, 24, 4, 256, 64, "half", "parts", BF16, 8),
    (37, 6, 2, 128, 128, "pairs", "base", BF16, 0),
    (130, 3, 1, 64, 48, "pairs", "linear", BF16, 24),
    (17, 4, 4, 256, 256, "half", "parts", F32, 4),
    (300, 8, 2, 64, 64, "pairs", "none", F32, 0),
    (3, 5, 1, 128, 112, "half", "linear", F32, 12),
    (2, 64, 1, 256, 240, "pairs", "parts", BF16, 0),
    (1100, 2, 1, 64, 32, "half", "none", BF16, 0),
]


def _rope(m, case, **kw):
    _, _, _, _, rot, layout, scaling, _, _ = case
    kw = dict(dict(rot_dims=rot, layout=layout, scaling=scaling, base=1e5, factor=4.0, context=2048.0, low=1.0, high=16.0), **kw)
    r = m.Rope(**kw)
    return r, co.frequencies(rot, 1e5, scaling, 4.0, 2048.0, 1.0, 16.0)


def _geom(m, case, pages=9, width=4):
    _, Hq, Hk, D, _, _, _, dtype, _ = case
    return m.AttnGeometry(n_q_heads=Hq, n_kv_heads=Hk, d_head=D, page_tokens=16, n_pages=pages, max_pages=width, dtype=dtype)


def _positions(seed, n, far=500000):
    return torch.randint(0, far, (n,), generator=torch.Generator().manual_seed(seed), dtype=torch.int32).cuda()


@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("inverse", [False, True])
def test_against_the_oracle(case, inverse):
    """q and k out of place, from rows that are apart; the inputs and what lies between the rows stay."""
    print("rope", case, inverse, flush=True)
    m = AH.gdn()
    n, Hq, Hk, D, _, _, _, dtype, pad = case
    rope, freq = _rope(m, case, amplitude=1.25 if inverse else 1.0, inverse=inverse)
    q, k, pos = _rows(1, n, Hq, D, dtype, pad), _rows(2, n, Hk, D, dtype, pad), _positions(3, n)
    whole = [t._base.clone() if t._base is not None else t.clone() for t in (q, k)]
    q_out, k_out = torch.full((n, Hq, D), float("nan"), dtype=dtype, device="cuda"), torch.full((n, Hk, D), float("nan"), dtype=dtype, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    m.rope_rotate(_geom(m, case), rope, m.rope_turns(rope), pos, q=q, k=k, q_out=q_out, k_out=k_out, dev_err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    _check(q_out, q, pos, rope, freq, dtype)
    _check(k_out, k, pos, rope, freq, dtype)
    for t, was in zip((q, k), whole):
        assert torch.equal(t._base if t._base is not None else t, was)


@pytest.mark.parametrize("case", CASES, ids=str)
def test_in_place_and_alone(case):
    """In place the same bits as out of place, in the rotated dimensions alone; q or k alone the same as together."""
    m = AH.gdn()
    n, Hq, Hk, D, rot, _, _, dtype, pad = case
    rope, _ = _rope(m, case)
    turns, g, pos = m.rope_turns(rope), _geom(m, case), _positions(4, n)
    q, k = _rows(5, n, Hq, D, dtype, pad), _rows(6, n, Hk, D, dtype, pad)
    q_out, k_out = torch.empty(n, Hq, D, dtype=dtype, device="cuda"), torch.empty(n, Hk, D, dtype=dtype, device="cuda")
    m.rope_rotate(g, rope, turns, pos, q=q, k=k, q_out=q_out, k_out=k_out)
    one_q, one_k = torch.empty_like(q_out), torch.empty_like(k_out)
    m.rope_rotate(g, rope, turns, pos, q=q, q_out=one_q)
    m.rope_rotate(g, rope, turns, pos, k=k, k_out=one_k)
    between = [t._base.clone() for t in (q, k)] if pad else None
    m.rope_rotate(g, rope, turns, pos, q=q, k=k)
    torch.cuda.synchronize()
    for a, b in ((one_q, q_out), (one_k, k_out), (q, q_out), (k, k_out)):
        assert torch.equal(a, b)
    if pad:
        for t, was in zip((q, k), between):
            assert torch.equal(t._base[:, t.shape[1] * D:], was[:, t.shape[1] * D:])


@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("k_in_place", [False, True])
def test_write_into_the_cache(case, k_in_place):
    """Rotated k and v at their slots, slot -1 skipped, everything else as it was; k_out the same with and without."""
    m = AH.gdn()
    n, Hq, Hk, D, _, _, _, dtype, pad = case
    pages = -(-n // 16) + 2
    g = _geom(m, case, pages, pages)
    rope, _ = _rope(m, case)
    turns, pos = m.rope_turns(rope), _positions(7, n)
    k, v = _rows(8, n, Hk, D, dtype, pad), _rows(9, n, Hk, D, dtype, 0)
    v[0, 0, 0] = float("nan")  # goes as it is
    slots = torch.randperm(pages * 16, generator=torch.Generator().manual_seed(10))[:n].to(torch.int32)
    if n > 1:
        slots[n // 2] = -1
    cache = m.KVCache(*(torch.randn(pages, Hk, 16, D, generator=torch.Generator().manual_seed(11 + i)).to(dtype).cuda() for i in range(2)))
    want_k, want_v = cache.k.clone(), cache.v.clone()
    k_ref = torch.empty(n, Hk, D, dtype=dtype, device="cuda")
    m.rope_rotate(g, rope, turns, pos, k=k, k_out=k_ref)
    k_out = None if k_in_place else torch.empty_like(k_ref)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    m.rope_rotate(g, rope, turns, pos, k=k, k_out=k_out, v=v, cache=cache, slot_map=slots.cuda(), dev_err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    assert torch.equal(k if k_in_place else k_out, k_ref)
    for t, s in enumerate(slots.tolist()):
        if s >= 0:
            want_k[s // 16, :, s % 16], want_v[s // 16, :, s % 16] = k_ref[t], v[t]
    bits = torch.int16 if dtype == BF16 else torch.int32
    assert torch.equal(cache.k.view(bits), want_k.view(bits)) and torch.equal(cache.v.view(bits), want_v.view(bits))


@pytest.mark.parametrize("n,Hq,Hk,D,rot,dtype", [(17001, 2, 1, 64, 32, BF16), (5003, 5, 1, 128, 128, BF16), (20000, 1, 1, 64, 16, F32)])
def test_many_tokens_give_the_bits_of_few(n, Hq, Hk, D, rot, dtype):
    """Calls whose workgroups take several tokens, the last one fewer, against calls of at most 700 tokens, cache and
    in-place rotation included; the first tokens against the oracle."""
    m = AH.gdn()
    case = (n, Hq, Hk, D, rot, "half", "parts", dtype, 0)
    rope, freq = _rope(m, case)
    turns, pages = m.rope_turns(rope), -(-n // 16) + 3
    g = _geom(m, case, pages=pages)
    q, k, v, pos = _rows(20, n, Hq, D, dtype, 0), _rows(21, n, Hk, D, dtype, 0), _rows(22, n, Hk, D, dtype, 0), _positions(23, n)
    slots = torch.randperm(pages * 16, generator=torch.Generator().manual_seed(24))[:n].to(torch.int32)
    slots[5::11] = -1
    slots = slots.cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run(step):
        cache = m.KVCache(*(torch.zeros(pages, Hk, 16, D, dtype=dtype, device="cuda") for _ in range(2)))
        q_out, k_in = torch.empty_like(q), k.clone()
        for at in range(0, n, step):
            e = slice(at, min(n, at + step))
            m.rope_rotate(g, rope, turns, pos[e], q=q[e], q_out=q_out[e], k=k_in[e], v=v[e], cache=cache, slot_map=slots[e], dev_err=err)
        alone = k.clone()
        m.rope_rotate(g, rope, turns, pos, k=alone, dev_err=err)  # the rotated dimensions alone move
        return q_out, k_in, cache.k, cache.v, alone
    whole, parts = run(n), run(700)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    for a, b in zip(whole, parts):
        assert torch.equal(a, b)
    assert torch.equal(whole[4], whole[1])
    _check(whole[0][:200], q[:200], pos[:200], rope, freq, dtype)
    _check(whole[1][-200:], k[-200:], pos[-200:], rope, freq, dtype)


def test_slots_outside_the_cache():
    m = AH.gdn()
    case = (4, 2, 2, 64, 32, "half", "none", BF16, 0)
    g, (rope, _) = _geom(m, case, 3, 3), _rope(m, case)
    k, v = _rows(1, 4, 2, 64, BF16, 0), _rows(2, 4, 2, 64, BF16, 0)
    for bad in (48, -2, 2 ** 31 - 1, -2 ** 31):
        cache = m.KVCache.zeros(g)
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        k_out = torch.empty_like(k)
        m.rope_rotate(g, rope, m.rope_turns(rope), _positions(3, 4), k=k, k_out=k_out, v=v, cache=cache,
                      slot_map=torch.tensor([5, bad, 47, -1], dtype=torch.int32, device="cuda"), dev_err=err)
        torch.cuda.synchronize()
        assert int(err.item()) == m.DEV_BAD_PAGE
        assert torch.equal(cache.k[0, :, 5], k_out[0]) and torch.equal(cache.v[2, :, 15], v[2])
        assert int((cache.k != 0).any(-1).any(1).sum()) == 2  # two cache slots written


def test_far_positions():
    """Up to 2^31 - 1, and negative ones turn the other way; the oracle's angle is taken from exact products."""
    m = AH.gdn()
    from fractions import Fraction
    case = (1, 1, 1, 64, 64, "half", "none", F32, 0)
    g, (rope, freq) = _geom(m, case), _rope(m, case)
    pos = [0, 1, -1, 1 << 20, (1 << 24) + 1, 2 ** 31 - 1, -2 ** 31, 1000003]
    two_pi = 2 * Fraction("3.14159265358979323846264338327950288419716939937510")
    x = torch.zeros(len(pos), 1, 64, device="cuda")
    x[..., :32] = 1.0
    out = torch.empty_like(x)
    m.rope_rotate(g, rope, m.rope_turns(rope), torch.tensor(pos, dtype=torch.int32, device="cuda"), q=x, q_out=out)
    got = AH.host(out)[:, 0]
    for i, p in enumerate(pos):
        for e, f in enumerate(m.rope_frequencies(rope)):
            t = Fraction(f) / two_pi * p
            angle = float((t - round(t)) * two_pi)
            # cos and sin as in _bound, and the turns' rounding: p 2^-64 turns
            tol = 8 * U + abs(p) * 2.0 ** -64 * 7
            assert abs(got[i, e] - np.cos(angle)) <= tol and abs(got[i, e + 32] - np.sin(angle)) <= tol, (p, e)


@pytest.mark.parametrize("layout,rot,D", [("half", 48, 64), ("pairs", 128, 128)])
def test_inverse_is_the_gradient(layout, rot, D):
    """Of L = sum(g * y): the transposed map of g, and what differences of L in fp64 give."""
    m = AH.gdn()
    case = (3, 2, 1, D, rot, layout, "linear", F32, 0)
    geom = _geom(m, case)
    rope, freq = _rope(m, case, amplitude=1.5)
    back, _ = _rope(m, case, amplitude=1.5, inverse=True)
    pos = _positions(12, 3, 3000)
    gen = torch.Generator().manual_seed(13)
    x, g = (torch.randn(3, 2, D, generator=gen).cuda() for _ in range(2))
    dx = torch.empty_like(g)
    m.rope_rotate(geom, back, m.rope_turns(back), pos, q=g, q_out=dx)
    dx, x64, g64 = AH.host(dx), AH.host(x), AH.host(g)
    bound = _bound(g64, dx, rot // 2, layout, 1.5, F32)
    rng = np.random.Generator(np.random.PCG64(14))
    loss = lambda z: float(np.sum(g64 * co.rotate(z, pos.tolist(), freq, layout, 1.5)))  # noqa: E731
    for _ in range(40):
        at = tuple(int(rng.integers(0, s)) for s in x64.shape)
        step = np.zeros_like(x64)
        step[at] = 0.5  # the map is linear: a difference is exact up to fp64 roundings
        assert abs((loss(x64 + step) - loss(x64 - step)) - dx[at]) <= bound[at] + 1e-11
    # undone where the amplitude is 1
    one, two = (_rope(m, case, inverse=i)[0] for i in (False, True))
    y, z = torch.empty_like(x), torch.empty_like(x)
    m.rope_rotate(geom, one, m.rope_turns(one), pos, q=x, q_out=y)
    m.rope_rotate(geom, two, m.rope_turns(two), pos, q=y, q_out=z)
    once = _bound(x64, x64, rot // 2, layout, 1.0, F32)
    assert np.all(np.abs(AH.host(z) - x64)[..., :rot] <= 4 * once[..., :rot] + 22 * U * np.abs(x64).max())


def test_infinities_and_nan_stay_in_their_pair():
    m = AH.gdn()
    case = (2, 1, 1, 64, 32, "half", "none", BF16, 0)
    geom, (rope, _) = _geom(m, case), _rope(m, case)
    x = torch.ones(2, 1, 64, dtype=BF16, device="cuda")
    x[0, 0, 3], x[0, 0, 40], x[1, 0, 31] = float("inf"), float("nan"), float("nan")
    out = torch.empty_like(x)
    m.rope_rotate(geom, rope, m.rope_turns(rope), torch.tensor([7, 7], dtype=torch.int32, device="cuda"), q=x, q_out=out)
    bad = ~torch.isfinite(out)
    want = torch.zeros_like(bad)
    want[0, 0, [3, 19, 40]] = True
    want[1, 0, [15, 31]] = True
    assert torch.equal(bad, want)


def test_long_rows_of_many_heads():
    """More units in a token than a workgroup has threads, and more than a product divides exactly."""
    m = AH.gdn()
    case = (3, 3000, 300, 256, 256, "pairs", "none", BF16, 0)
    geom, (rope, freq) = _geom(m, case), _rope(m, case)
    q, k, pos = _rows(40, 3, 3000, 256, BF16, 0), _rows(41, 3, 300, 256, BF16, 0), _positions(42, 3)
    q_out, k_out = torch.empty_like(q), torch.empty_like(k)
    m.rope_rotate(geom, rope, m.rope_turns(rope), pos, q=q, k=k, q_out=q_out, k_out=k_out)
    torch.cuda.synchronize()
    for a, b in ((q, q_out), (k, k_out)):
        pick = [0, 1, 2, 149, a.shape[1] - 1]
        _check(b[:, pick], a[:, pick], pos, rope, freq, BF16)
    # every head turns by the same angles: heads with the same contents come out the same
    q[:, 1:] = q[:, :1]
    m.rope_rotate(geom, rope, m.rope_turns(rope), pos, q=q, q_out=q_out)
    torch.cuda.synchronize()
    assert torch.equal(q_out, q_out[:, :1].expand_as(q_out))


def test_more_tokens_than_a_launch_takes():
    """2^27 + 100 tokens of 64 dimensions of q, k and v in one row each, 16 tokens to a workgroup of 512 threads: past 2^32
    threads, so the call takes two launches, 116 tokens in the second.  Equal to calls of 2^20 tokens; the slots of the first
    tokens, of those on both sides of 2^27 - 16, where the second launch begins, and of the last are in the cache."""
    m = AH.gdn()
    step, n = 2 ** 20, 2 ** 27 + 100
    g = torch.Generator(device="cuda").manual_seed(9)
    geom = m.AttnGeometry(n_q_heads=1, n_kv_heads=1, d_head=64, page_tokens=16, n_pages=40, max_pages=40)
    rope = m.Rope(rot_dims=16)
    turns = m.rope_turns(rope)
    block = torch.randn(step, 3, 64, generator=g, device="cuda").to(BF16)
    rows = torch.empty(n, 3, 64, dtype=BF16, device="cuda")
    for at in range(0, n, step):
        rows[at:at + step] = block[:min(step, n - at)]
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    slots = torch.full((n,), -1, dtype=torch.int32, device="cuda")
    here = [0, 1, 511, 2 ** 27 - 18, 2 ** 27 - 17, 2 ** 27 - 16, 2 ** 27 - 15, n - 2, n - 1]
    slots[torch.tensor(here, device="cuda")] = torch.arange(len(here), dtype=torch.int32, device="cuda") * 17
    cache, err = m.KVCache.zeros(geom), torch.zeros(1, dtype=torch.int32, device="cuda")
    m.rope_rotate(geom, rope, turns, pos, q=rows[:, :1], k=rows[:, 1:2], v=rows[:, 2:], cache=cache, slot_map=slots, dev_err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    for i, t in enumerate(here):
        assert torch.equal(cache.k[i * 17 // 16, :, i * 17 % 16], rows[t, 1:2]) and torch.equal(cache.v[i * 17 // 16, :, i * 17 % 16], rows[t, 2:])
    for at in range(0, n, step):
        part = block[:min(step, n - at)].clone()
        m.rope_rotate(geom, rope, turns, pos[at:at + step], q=part[:, :1], k=part[:, 1:2], dev_err=err)
        assert torch.equal(rows[at:at + step], part), at
    assert int(err.item()) == 0
    del rows, pos, slots
    torch.cuda.empty_cache()


def test_nothing_to_do():
    m = AH.gdn()
    case = (0, 2, 1, 64, 32, "half", "none", BF16, 0)
    geom, (rope, _) = _geom(m, case), _rope(m, case)
    q = torch.empty(0, 2, 64, dtype=BF16, device="cuda")
    m.rope_rotate(geom, rope, m.rope_turns(rope), torch.empty(0, dtype=torch.int32, device="cuda"), q=q)
    torch.cuda.synchronize()


def test_on_a_stream_and_in_a_graph():
    """On a stream that the call names, and captured: every replay gives the eager bits, with new inputs too."""
    m = AH.gdn()
    case = (9, 24, 4, 256, 64, "half", "parts", BF16, 0)
    g, (rope, _) = _geom(m, case), _rope(m, case)
    turns = m.rope_turns(rope)
    q, k, v, pos = _rows(1, 9, 24, 256, BF16, 0), _rows(2, 9, 4, 256, BF16, 0), _rows(3, 9, 4, 256, BF16, 0), _positions(4, 9)
    slots = torch.arange(9, dtype=torch.int32, device="cuda") * 3
    cache = m.KVCache.zeros(g)
    q_out, k_out = torch.empty_like(q), torch.empty_like(k)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    call = lambda **kw: m.rope_rotate(g, rope, turns, pos, q=q, k=k, q_out=q_out, k_out=k_out, v=v, cache=cache, slot_map=slots, dev_err=err, **kw)  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(stream=side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call()
    for seed in range(3):
        q.copy_(_rows(20 + seed, 9, 24, 256, BF16, 0))
        pos.copy_(_positions(30 + seed, 9))
        call()
        torch.cuda.synchronize()
        want = [t.clone() for t in (q_out, k_out, cache.k, cache.v)]
        for t in (q_out, k_out, cache.k, cache.v):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((q_out, k_out, cache.k, cache.v), want):
            assert torch.equal(a, b)
