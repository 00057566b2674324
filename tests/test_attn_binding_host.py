"""The binding of the paged-cache, attention and tree entry points on the host (no GPU): which device a call's tensors
and stream are on, copies of the geometry, workspaces for calls of many sizes, limits."""
import copy
import dataclasses
import os
import pickle

import pytest
import torch

F32, BF16, I32 = torch.float32, torch.bfloat16, torch.int32


@pytest.fixture(scope="module")
def gdn():
    import gated_deltanet_delta_amd as m
    from gated_deltanet_delta_amd import build
    if not os.path.exists(m.LIB_PATH):
        build.build()
    m.lib()
    return m


class _On:
    """A tensor's type and shape under a device of its own: for the binding's host checks alone."""

    is_cuda = True

    def __init__(self, shape, dtype, index=0):
        self.t, self.index = torch.empty(shape, dtype=dtype, device="meta"), index
        self.dtype, self.shape, self.device = dtype, self.t.shape, torch.device("cuda", index)

    def get_device(self):
        return self.index

    def is_contiguous(self):
        return True

    def stride(self):
        return self.t.stride()

    def numel(self):
        return 1 << 30

    def element_size(self):
        return 1

    def data_ptr(self):
        return 16


@pytest.fixture
def on_gpu_0(gdn, monkeypatch):
    """GPU 0 is current, and no call gets to the library."""
    def got_past():
        raise AssertionError("the call got past the binding's checks")
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(gdn, "_current_stream", lambda device: 0)
    monkeypatch.setattr(gdn, "lib", got_past)


class _Stream:
    cuda_stream = 0

    def __init__(self, index):
        self.device_index = index


def _calls(m):
    """Every entry point with tensors of one device: (function, leading arguments, tensors by name)."""
    g = m.AttnGeometry(n_q_heads=4, n_kv_heads=2, d_head=64, n_pages=9, max_pages=3, max_tree=4)
    d = m.Geometry(n_k_heads=1, n_v_heads=2, d_k=16, d_v=16, n_slots=8, max_draft=3)
    C = d.conv_channels
    i = lambda *s: _On(s, I32)  # noqa: E731
    b = lambda *s: _On(s, BF16)  # noqa: E731
    page = (9, 2, 16, 64)
    plan = dict(kv_len=i(5), new_len=i(5), free_pages=i(9), n_free=i(1), block_table=i(5, 3), cu_new=i(6), slot_map=i(7),
                position=i(7), kv_len_out=i(5), n_free_out=i(1), dev_err=i(1))
    write = {"cache.k": b(*page), "cache.v": b(*page), "k": b(7, 2, 64), "v": b(7, 2, 64), "slot_map": i(7), "dev_err": i(1)}
    prefill = {"q": b(7, 4, 64), "k": b(7, 2, 64), "v": b(7, 2, 64), "cu_seqlens": i(3), "o": b(7, 4, 64), "workspace": i(1),
               "cache.k": b(*page), "cache.v": b(*page), "block_table": i(2, 3), "ctx_len": i(2), "dev_err": i(1)}
    tree = {"cache.k": b(*page), "cache.v": b(*page), "block_table": i(2, 3), "ctx_len": i(2), "q": b(2, 4, 4, 64),
            "k": b(2, 4, 2, 64), "v": b(2, 4, 2, 64), "parent": i(2, 4), "o": b(2, 4, 4, 64), "workspace": i(1), "n_row": i(2),
            "dev_err": i(1)}
    vtree = {"state": _On((8, 2, 16, 16), F32), "conv_state": _On((8, 8, C), F32), "conv_pos": i(8, m.POS_STRIDE),
             "x": b(2, 3, C), "a": b(2, 3, 2), "b": b(2, 3, 2), "conv_w": _On((C, 4), F32), "slot": i(2), "parent": i(2, 3),
             "snap_slot": i(2, 3), "o": b(2, 3, 2, 16), "dev_err": i(1), "k_row": i(2)}
    return dict(kv_plan=(m.kv_plan, g, plan), kv_write=(m.kv_write, g, write), attn_prefill=(m.attn_prefill, g, prefill),
                attn_tree=(m.attn_tree, g, tree), verify_tree_slots=(m.verify_tree_slots, d, vtree))


def _call(m, name, tensors, stream=None):
    fn, geom, _ = _calls(m)[name]
    kw = {k: t for k, t in tensors.items() if "." not in k and k not in ("state", "conv_state", "conv_pos")}
    if "cache.k" in tensors:
        kw["cache"] = m.KVCache(tensors["cache.k"], tensors["cache.v"])
    if "state" in tensors:
        kw["pool"] = m.SlotPool(tensors["state"], tensors["conv_state"], tensors["conv_pos"])
    fn(geom, **kw, stream=stream)


NAMES = ["kv_plan", "kv_write", "attn_prefill", "attn_tree", "verify_tree_slots"]


@pytest.mark.parametrize("name", NAMES)
def test_every_tensor_is_on_the_current_device(gdn, on_gpu_0, name):
    """Each tensor of a call on another device than the rest, and all of them on another device than the current one,
    are refused before the library sees an address."""
    names = list(_calls(gdn)[name][2])
    for other in names:
        tensors = _calls(gdn)[name][2]
        tensors[other] = _On(tuple(tensors[other].shape), tensors[other].dtype, 1)
        # the call's device is that of its first tensor; where that is the odd one, some other tensor is named
        with pytest.raises(ValueError, match=r"on cuda:[01], required: cuda:[01]"):
            _call(gdn, name, tensors)
    with pytest.raises(AssertionError, match="got past"):  # all of them on GPU 0
        _call(gdn, name, _calls(gdn)[name][2])
    tensors = {k: _On(tuple(t.shape), t.dtype, 1) for k, t in _calls(gdn)[name][2].items()}
    with pytest.raises(ValueError, match="required: the current device cuda:0"):
        _call(gdn, name, tensors)


@pytest.mark.parametrize("name", NAMES)
def test_the_stream_is_of_the_current_device(gdn, on_gpu_0, name):
    with pytest.raises(ValueError, match="stream: of cuda:1, required: of the current device cuda:0"):
        _call(gdn, name, _calls(gdn)[name][2], _Stream(1))


def test_a_geometry_that_was_used_can_be_copied(gdn):
    """Copies and pickles of a geometry carry its fields; each has a C struct of its own."""
    g = gdn.AttnGeometry(n_q_heads=6, n_kv_heads=2, d_head=128, n_pages=7, scale=0.25)
    g.check()  # makes its C struct
    for c in (copy.copy(g), copy.deepcopy(g), pickle.loads(pickle.dumps(g)), dataclasses.replace(g)):
        assert c == g and c is not g and hash(c) == hash(g)
        assert "_c_ref" not in c.__dict__
        c.check()
        assert gdn.attn_prefill_workspace_bytes(c, 9, 1) == gdn.attn_prefill_workspace_bytes(g, 9, 1) > 0
    other = dataclasses.replace(g, n_q_heads=5)
    with pytest.raises(gdn.GdnError, match="n_q_heads: 5"):
        other.check()


@pytest.mark.parametrize("Hk,G,D,dtype", [(4, 6, 256, BF16), (1, 1, 64, BF16), (2, 7, 128, BF16), (4, 6, 256, F32), (1, 3, 64, F32)])
def test_a_workspace_for_all_sizes(gdn, Hk, G, D, dtype):
    """The size for calls of up to n is the largest of theirs: a shorter call may need more than a longer one."""
    g = gdn.AttnGeometry(n_q_heads=Hk * G, n_kv_heads=Hk, d_head=D, n_pages=64, max_pages=64, max_tree=20, dtype=dtype)
    for most in (1, 9, 43, 256, 2048, 5000):
        for seqs in (1, 5):
            each = [gdn.attn_prefill_workspace_bytes(g, n, s) for n in range(1, most + 1) for s in range(1, seqs + 1)]
            assert gdn.attn_prefill_workspace_bytes(g, most, seqs, up_to=True) == max(each)
    assert gdn.attn_prefill_workspace_bytes(g, 100000, 1) == 0  # and the largest among them need none
    assert gdn.attn_prefill_workspace_bytes(g, (1 << 30) - 1, 1, up_to=True) == \
        gdn.attn_prefill_workspace_bytes(g, 100000, 3, up_to=True) > 0
    for batch, n in ((1, 1), (7, 20), (300, 3), (1500, 20)):
        each = [gdn.attn_tree_workspace_bytes(g, b, k) for b in range(1, batch + 1) for k in range(1, n + 1)]
        assert gdn.attn_tree_workspace_bytes(g, batch, n, up_to=True) == max(each)
    assert gdn.attn_prefill_workspace_bytes(g, 0, 1, up_to=True) == 0
    for bad in ((-1, 1), (9, 0)):
        assert gdn.attn_prefill_workspace_bytes(g, *bad, up_to=True) == 0
    for bad in ((0, 1), (1, 0), (1, 21)):
        assert gdn.attn_tree_workspace_bytes(g, *bad, up_to=True) == 0


def _prefill_status(m, g, n_tokens):
    """The status of a packed call that is refused for its missing cu_seqlens if for nothing else."""
    p, row = 0x10000, g.n_kv_heads * g.d_head
    st = m.lib().gdn_attn_prefill(g._ref(), p, g.n_q_heads * g.d_head, p, row, p, row, None, 1, n_tokens, p, p, p, p, p, 1 << 50, p,
                                  None, None)
    return m.lib().gdn_status_string(st).decode(), m.lib().gdn_last_error().decode()


def test_lengths_leave_room_for_whole_tiles(gdn):
    """The most cached and new tokens together, rounded up to tiles with the ones requested ahead, fit 31 bits."""
    g = gdn.AttnGeometry(n_q_heads=1, n_kv_heads=1, d_head=64, max_pages=(1 << 26) - 1)
    g.check()
    most = (1 << 30) - 4096
    assert g.max_pages * g.page_tokens + most + 4 * 64 < 1 << 31
    name, message = _prefill_status(gdn, g, most)
    assert name == "GDN_ERR_NULL" and "cu_seqlens" in message
    for n in (most + 1, (1 << 30) - 1):
        name, message = _prefill_status(gdn, g, n)
        assert name == "GDN_ERR_RANGE" and f"n_tokens: {n}, required: 0..{most}" in message


def test_scales_whose_base_2_form_is_not_finite_are_refused(gdn):
    for scale in (2.0 ** 127, 1e-45):
        gdn.AttnGeometry(scale=scale).check()
    for scale in (2.0 ** 127 * (1 + 2.0 ** -23), 3.4e38):
        with pytest.raises(gdn.GdnError, match="scale: .*supported by this library: <= 2\\^127"):
            gdn.AttnGeometry(scale=scale).check()
    with pytest.raises(gdn.GdnError, match="scale: inf, required: finite and > 0"):
        gdn.AttnGeometry(scale=float("inf")).check()
