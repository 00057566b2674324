"""The gated delta rule over trees of drafts on the GPU: every node's slot (state, conv history, position) and output
against the oracle, chains bit for bit against the chain verify, per-row counts, refused rows, and the commit."""
import dataclasses

import numpy as np
import pytest
import torch

import attn_harness as AH
import gdn_inputs as gi
import harness as H
from oracle import attn_oracle as ao
from test_gpu_debug_checks import _debug_library

pytestmark = pytest.mark.gpu


def _snap_slots(g, slots, k):
    free = [s for s in range(g.n_slots) if s not in set(int(x) for x in slots)]
    return np.array(free[:len(slots) * k], np.int32).reshape(len(slots), k)


def _run(g, inp, parent, ss, k, err, k_row=None, pool=None, lib=None):
    m = AH.gdn()
    geom, dt, B = H.to_geom(g), H.in_dtype(g), len(inp["slots"])
    pool = pool or H.make_pool(g, inp["state"], inp["hist"], inp["pos"])
    o = torch.full((B, k, g.n_v_heads, g.d_v), float("nan"), dtype=dt, device="cuda")
    m.verify_tree_slots(geom, pool, *(H.dev(inp[n][:, :k], dt) for n in ("x", "a", "b")),
                        H.dev(inp["conv_w"]) if g.conv_width else None, H.dev(inp["slots"]), H.dev(parent), H.dev(ss), o,
                        dev_err=err, k_row=None if k_row is None else H.dev(np.asarray(k_row, np.int32)))
    torch.cuda.synchronize()
    return pool, o


@pytest.mark.parametrize("Hk,G,d,k,B,W,dtype", [
    (16, 3, 128, 4, 4, 4, gi.BF16), (2, 3, 128, 16, 3, 4, gi.BF16), (2, 2, 64, 7, 2, 4, gi.F32), (1, 4, 32, 5, 3, 0, gi.BF16),
    (3, 1, 16, 16, 1, 4, gi.F32), (1, 1, 16, 1, 2, 0, gi.F32)])
def test_tree_against_the_oracle(Hk, G, d, k, B, W, dtype):
    print(f"tree Hk {Hk} G {G} d {d} k {k} B {B} W {W} {dtype}", flush=True)
    g = dataclasses.replace(gi.GEOM_QWEN, n_k_heads=Hk, n_v_heads=Hk * G, d_k=d, d_v=d, n_slots=B * (k + 1) + 1, max_draft=k,
                            conv_ring=32, conv_width=W, l2norm_qk=W > 0, dtype_in=dtype, dtype_out=dtype)
    inp = gi.verify_inputs(seed=800 + k + d, geom=g, batch=B, k=k)
    parent = AH.parents(810 + k, B, k)
    ss = _snap_slots(g, inp["slots"], k)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pool, o = _run(g, inp, parent, ss, k, err)
    assert int(err.item()) == 0
    hist, pos = H.read_hist(g, pool), H.positions(pool)
    untouched = H.make_pool(g, inp["state"], inp["hist"], inp["pos"])
    used = set(int(s) for s in ss.reshape(-1))
    for i, s in enumerate(inp["slots"]):
        o_r, st_r, h_r, depth = ao.verify_tree(g, inp["state"][s], inp["hist"][s], inp["x"][i], inp["a"][i], inp["b"][i],
                                               inp["conv_w"], parent[i])
        assert H.relerr(H.f64(o[i]), o_r) <= H.tol_for(g)
        for j in range(k):
            sj = int(ss[i, j])
            assert H.relerr(pool.state[sj].cpu().numpy(), st_r[j]) <= H.tol_for(g), (i, j)
            if W:
                assert np.array_equal(hist[sj], h_r[j].astype(np.float32)), (i, j)
                assert pos[sj] == int(inp["pos"][s]) + depth[j]
    for s in range(g.n_slots):
        if s not in used:
            assert torch.equal(pool.state[s], untouched.state[s]) and torch.equal(pool.conv_state[s], untouched.conv_state[s])
            assert torch.equal(pool.conv_pos[s], untouched.conv_pos[s])


@pytest.mark.parametrize("d,W,dtype", [(128, 4, gi.BF16), (64, 4, gi.F32), (32, 0, gi.BF16)])
def test_chain_equals_the_chain_verify_bit_for_bit(d, W, dtype):
    m = AH.gdn()
    k, B = 5, 3
    g = dataclasses.replace(gi.GEOM_QWEN, n_k_heads=2, n_v_heads=6, d_k=d, d_v=d, n_slots=24, max_draft=k, conv_width=W,
                            l2norm_qk=W > 0, dtype_in=dtype, dtype_out=dtype)
    inp = gi.verify_inputs(seed=830, geom=g, batch=B, k=k)
    ss = _snap_slots(g, inp["slots"], k)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    chain = np.tile(np.arange(-1, k - 1, dtype=np.int32), (B, 1))
    pool, o = _run(g, inp, chain, ss, k, err, k_row=[5, 1, 4])
    ref = H.make_pool(g, inp["state"], inp["hist"], inp["pos"])
    o2 = torch.full_like(o, float("nan"))
    dt = H.in_dtype(g)
    m.verify_k_slots(H.to_geom(g), ref, *(H.dev(inp[n][:, :k], dt) for n in ("x", "a", "b")),
                     H.dev(inp["conv_w"]) if W else None, H.dev(inp["slots"]), H.dev(ss), o2, dev_err=err,
                     k_row=H.dev(np.array([5, 1, 4], np.int32)))
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    assert torch.equal(torch.nan_to_num(o.float(), 9.0), torch.nan_to_num(o2.float(), 9.0))
    assert torch.equal(pool.state, ref.state) and torch.equal(pool.conv_pos, ref.conv_pos)
    if W:
        for s in ss.reshape(-1):
            assert torch.equal(pool.conv_state[int(s)], ref.conv_state[int(s)])


def test_branches_equal_chains_of_their_own_and_commit():
    """Every path of a tree equals that path verified as a chain, bit for bit; the commit picks a node's slot and a
    decode step continues from it."""
    m = AH.gdn()
    k = 8
    g = dataclasses.replace(gi.GEOM_QWEN, n_k_heads=4, n_v_heads=12, n_slots=20, max_draft=k, conv_ring=16)
    geom, dt = H.to_geom(g), H.in_dtype(g)
    inp = gi.verify_inputs(seed=840, geom=g, batch=2, k=k)
    parent = np.array([[-1, 0, 0, 1, 2, 2, -1, 6], [-1, -1, -1, 2, 2, 1, 5, 4]], np.int32)
    ss = _snap_slots(g, inp["slots"], k)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pool, o = _run(g, inp, parent, ss, k, err)
    cw = H.dev(inp["conv_w"])
    for i in range(2):
        for j in range(k):
            path, at = [], j
            while at >= 0:
                path.insert(0, at)
                at = int(parent[i, at])
            alone = H.make_pool(g, inp["state"], inp["hist"], inp["pos"])
            oc = torch.empty(1, len(path), 12, 128, dtype=dt, device="cuda")
            m.verify_k_slots(geom, alone, *(H.dev(inp[n][i:i + 1, path], dt) for n in ("x", "a", "b")), cw,
                             H.dev(inp["slots"][i:i + 1]), H.dev(ss[i:i + 1, path]), oc, dev_err=err)
            torch.cuda.synchronize()
            assert torch.equal(oc[0, -1], o[i, j]), (i, j)
            assert torch.equal(alone.state[int(ss[i, j])], pool.state[int(ss[i, j])]), (i, j)
            assert np.array_equal(H.read_hist(g, alone)[int(ss[i, j])], H.read_hist(g, pool)[int(ss[i, j])])
    nxt = torch.empty(2, dtype=torch.int32, device="cuda")
    m.commit_slots(geom, H.dev(inp["slots"]), H.dev(ss), H.dev(np.array([4 + 1, 0], np.int32)), nxt, dev_err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    assert nxt.cpu().tolist() == [int(ss[0, 4]), int(inp["slots"][1])]


SHAPES = {
    "full binary": [-1] + [(j - 1) // 2 for j in range(1, 15)],           # states of three depths wait at once
    "full binary, two roots": [-1, -1] + [(j - 2) // 2 for j in range(2, 16)],
    "star": [-1] * 16,
    "one root, 15 leaves": [-1] + [0] * 15,
    "comb": [-1, 0, 0, 1, 1, 3, 3, 5, 5, 7, 7, 9, 9, 11, 11, 13],
    "comb, teeth first": [-1, 0, 0, 2, 2, 4, 4, 6, 6, 8, 8, 10, 10, 12, 12, 14],
    "chain": list(range(-1, 15)),
    "forest": [-1, 0, 1, -1, 3, 3, -1, 6, 7, 8, 8, 6, -1, 12, 2, 13],
}


@pytest.mark.parametrize("shape", list(SHAPES))
@pytest.mark.parametrize("d,W,dtype", [(128, 4, gi.BF16), (32, 0, gi.F32)])
def test_tree_shapes_against_the_oracle(shape, d, W, dtype):
    """Trees that branch at every node, at none, at the root only, to one side: each node starts from its own parent's
    state and window."""
    par = np.array([SHAPES[shape]], np.int32)
    k = par.shape[1]
    g = dataclasses.replace(gi.GEOM_QWEN, n_k_heads=1, n_v_heads=2, d_k=d, d_v=d, n_slots=k + 2, max_draft=k, conv_ring=32,
                            conv_width=W, l2norm_qk=W > 0, dtype_in=dtype, dtype_out=dtype)
    inp = gi.verify_inputs(seed=870 + d, geom=g, batch=1, k=k)
    ss = _snap_slots(g, inp["slots"], k)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pool, o = _run(g, inp, par, ss, k, err)
    assert int(err.item()) == 0
    s = inp["slots"][0]
    o_r, st_r, h_r, depth = ao.verify_tree(g, inp["state"][s], inp["hist"][s], inp["x"][0], inp["a"][0], inp["b"][0],
                                           inp["conv_w"], par[0])
    assert H.relerr(H.f64(o[0]), o_r) <= H.tol_for(g)
    hist, pos = H.read_hist(g, pool), H.positions(pool)
    for j in range(k):
        sj = int(ss[0, j])
        assert H.relerr(pool.state[sj].cpu().numpy(), st_r[j]) <= H.tol_for(g), j
        if W:
            assert np.array_equal(hist[sj], h_r[j].astype(np.float32)), j
            assert pos[sj] == int(inp["pos"][s]) + depth[j]


def test_missing_slots_in_a_branching_tree():
    """A node without a slot that has two subtrees: its own output comes, neither subtree is touched, the walk goes on
    with the others."""
    m = AH.gdn()
    par = np.array([[-1, 0, 0, 1, 1, 2, 2, 3, 4]], np.int32)
    k = par.shape[1]
    g = dataclasses.replace(gi.GEOM_QWEN, n_k_heads=1, n_v_heads=2, n_slots=k + 2, max_draft=k, conv_ring=16)
    inp = gi.verify_inputs(seed=880, geom=g, batch=1, k=k)
    ss = _snap_slots(g, inp["slots"], k)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    good, og = _run(g, inp, par, ss, k, err)
    bad = ss.copy()
    bad[0, 1] = -1
    pool, o = _run(g, inp, par, bad, k, err)
    before = H.make_pool(g, inp["state"], inp["hist"], inp["pos"])
    assert int(err.item()) == m.DEV_BAD_SLOT
    for j in range(k):
        s = int(ss[0, j])
        if j in (1, 3, 4, 7, 8):
            assert torch.equal(pool.state[s], before.state[s])
            assert torch.equal(o[0, j], og[0, j]) if j == 1 else torch.isnan(o[0, j].float()).all()
        else:
            assert torch.equal(pool.state[s], good.state[s]) and torch.equal(o[0, j], og[0, j])


def test_refused_rows_and_snapshots():
    m = AH.gdn()
    k, B = 4, 3
    g = dataclasses.replace(gi.GEOM_QWEN, n_k_heads=2, n_v_heads=6, d_k=64, d_v=64, n_slots=16)
    inp = gi.verify_inputs(seed=850, geom=g, batch=B, k=k)
    parent = np.array([[-1, 0, 1, 0]] * B, np.int32)
    ss = _snap_slots(g, inp["slots"], k)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    good, og = _run(g, inp, parent, ss, k, err)
    assert int(err.item()) == 0
    before = H.make_pool(g, inp["state"], inp["hist"], inp["pos"])

    def skipped(pool, o, nodes):
        for i in range(B):
            for j in range(k):
                s = int(ss[i, j])
                if (i, j) in nodes:
                    assert torch.equal(pool.state[s], before.state[s]) and torch.equal(pool.conv_pos[s], before.conv_pos[s])
                else:
                    assert torch.equal(pool.state[s], good.state[s])
                    assert torch.equal(o[i, j], og[i, j])

    row1 = {(1, j) for j in range(k)}
    for bad in (-2, 3, 7):
        p = parent.copy()
        p[1, 3] = bad
        err.zero_()
        pool, o = _run(g, inp, p, ss, k, err)
        assert int(err.item()) == m.DEV_BAD_PARENT
        skipped(pool, o, row1)
        assert torch.isnan(o[1].float()).all()
    for bad in (0, 5, -1):
        err.zero_()
        pool, o = _run(g, inp, parent, ss, k, err, k_row=[4, bad, 4])
        assert int(err.item()) == m.DEV_BAD_K
        skipped(pool, o, row1)
    for bad in (-1, g.n_slots):
        slots = inp["slots"].copy()
        slots[1] = bad
        err.zero_()
        pool, o = _run(g, dict(inp, slots=slots), parent, ss, k, err,
                       pool=H.make_pool(g, inp["state"], inp["hist"], inp["pos"]))
        assert int(err.item()) == m.DEV_BAD_SLOT
        skipped(pool, o, row1)
    # node 1 has no slot: its output comes, its child 2 is skipped, its sibling 3 is not
    bad = ss.copy()
    bad[1, 1] = g.n_slots
    err.zero_()
    pool, o = _run(g, inp, parent, bad, k, err)
    assert int(err.item()) == m.DEV_BAD_SLOT
    assert torch.equal(o[1, 1], og[1, 1]) and torch.isnan(o[1, 2].float()).all() and torch.equal(o[1, 3], og[1, 3])
    assert torch.equal(pool.state[int(ss[1, 2])], before.state[int(ss[1, 2])])
    assert torch.equal(pool.state[int(ss[1, 1])], before.state[int(ss[1, 1])])
    assert torch.equal(pool.state[int(ss[1, 3])], good.state[int(ss[1, 3])])


def test_debug_library_reports_slots_used_twice():
    """The debug build checks rows' and snapshots' slots before the kernel; entries past a row's count are not used."""
    m = AH.gdn()
    g = dataclasses.replace(gi.GEOM_QWEN, n_k_heads=1, n_v_heads=2, n_slots=8)
    geom, dt = H.to_geom(g), H.in_dtype(g)
    inp = gi.verify_inputs(seed=890, geom=g, batch=2, k=2)
    pool = m.SlotPool.zeros(geom)
    args = [H.dev(inp[n][:, :2], dt) for n in ("x", "a", "b")] + [H.dev(inp["conv_w"]), H.dev(np.array([0, 1], np.int32))]
    par = H.dev(np.array([[-1, -1], [-1, 0]], np.int32))
    o = torch.empty(2, 2, 2, 128, dtype=dt, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    with _debug_library(m):
        for ss, k_row, want in (([[2, 3], [4, 5]], None, 0), ([[2, 3], [4, 0]], None, 7), ([[2, 3], [4, 0]], [2, 1], 0),
                                ([[2, 3], [3, 5]], [2, 1], 7)):
            err.zero_()
            m.verify_tree_slots(geom, pool, *args, par, H.dev(np.array(ss, np.int32)), o, dev_err=err,
                                k_row=None if k_row is None else H.dev(np.array(k_row, np.int32)))
            torch.cuda.synchronize()
            assert int(err.item()) == want, (ss, k_row)


def test_graph_replays_match_eager():
    m = AH.gdn()
    k, B = 6, 2
    g = dataclasses.replace(gi.GEOM_QWEN, n_k_heads=2, n_v_heads=4, n_slots=14, max_draft=k, conv_ring=16)
    geom, dt = H.to_geom(g), H.in_dtype(g)
    inp = gi.verify_inputs(seed=860, geom=g, batch=B, k=k)
    parent, ss = H.dev(AH.parents(861, B, k)), H.dev(_snap_slots(g, inp["slots"], k))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pool, eager = _run(g, inp, parent.cpu().numpy(), ss.cpu().numpy(), k, err)
    args = [H.dev(inp[n][:, :k], dt) for n in ("x", "a", "b")] + [H.dev(inp["conv_w"]), H.dev(inp["slots"]), parent, ss]
    again = H.make_pool(g, inp["state"], inp["hist"], inp["pos"])
    o = torch.empty_like(eager)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.verify_tree_slots(geom, again, *args, o, dev_err=err)
    for _ in range(3):
        o.fill_(1.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        assert torch.equal(o, eager) and torch.equal(again.state, pool.state) and torch.equal(again.conv_pos, pool.conv_pos)
