"""The rotary, weights, eviction and move entry points on the host (no GPU): every refusal, from C under the sanitizers and
through the Python binding; which device a call's tensors are on; frequencies; the oracle's own pins."""
import copy
import math
import os
import pickle
import shutil
import subprocess
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import cache_oracle as co

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "gated_deltanet_delta_amd", "csrc")
BUILD = os.path.join(ROOT, "_build")
SAN = ["-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-fno-omit-frame-pointer", "-g", "-O1"]
F32, BF16, I32, I64 = torch.float32, torch.bfloat16, torch.int32, torch.int64


@pytest.fixture(scope="module")
def gdn():
    import gated_deltanet_delta_amd as m
    from gated_deltanet_delta_amd import build
    if not os.path.exists(m.LIB_PATH):
        build.build()
    m.lib()
    return m


def test_refusals_clean_under_asan_and_ubsan(gdn, tmp_path):
    """Every refusal path of the C entry points, with the host code under AddressSanitizer and UBSan."""
    from gated_deltanet_delta_amd import build
    if shutil.which("g++") is None or shutil.which("gcc") is None:
        pytest.skip("no host compiler")
    objs = [os.path.join(BUILD, n + ".o") for n in build.HIP_SOURCES]
    if not all(os.path.exists(o) for o in objs):
        build.build()
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    inc = ["-I", os.path.join(ROOT, "include"), "-I", CSRC]
    host = []
    for src in build.HOST_SOURCES:
        host.append(str(tmp_path / (src + ".o")))
        subprocess.run(["g++", "-std=c++17", "-fPIC", *SAN, *inc, "-c", os.path.join(CSRC, src), "-o", host[-1]], check=True)
    drv, exe = str(tmp_path / "drv.o"), str(tmp_path / "cache_refusals")
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-Werror", *SAN, *inc, "-c",
                    os.path.join(ROOT, "tests", "cache_refusals.c"), "-o", drv], check=True)
    subprocess.run(["g++", *SAN, drv, *host, *objs, "-L", os.path.join(rocm, "lib"), "-lamdhip64",
                    "-Wl,-rpath," + os.path.join(rocm, "lib"), "-o", exe], check=True)
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0", UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=120)
    assert r.returncode == 0, (r.returncode, r.stdout, r.stderr[-4000:])
    assert "cache refusals ok" in r.stdout
    assert "runtime error" not in r.stderr and "AddressSanitizer" not in r.stderr, r.stderr[-4000:]


# ---------------------------------------------------------------- frequencies

@pytest.mark.parametrize("kw", [
    dict(rot_dims=64, base=1e4), dict(rot_dims=16, base=1.5), dict(rot_dims=256, base=1e7),
    dict(rot_dims=128, base=1e4, scaling="linear", factor=4.0), dict(rot_dims=64, base=1e4, scaling="base", factor=8.0),
    dict(rot_dims=128, base=5e5, scaling="parts", factor=8.0, context=8192.0, low=1.0, high=4.0),
    dict(rot_dims=64, base=1e6, scaling="parts", factor=1.0, context=32768.0)])
def test_frequencies(gdn, kw):
    """The scaled forms from their formulas, and as fractions of a turn."""
    rope = gdn.Rope(**kw)
    rope.check()
    names = dict(kw)
    ref = co.frequencies(names.pop("rot_dims"), names.pop("base"), **names)
    got = np.array(gdn.rope_frequencies(rope))
    assert got.shape == ref.shape and np.max(np.abs(got / ref - 1)) < 1e-13
    two_pi = 2 * Fraction("3.14159265358979323846264338327950288")
    for f, t in zip(got, gdn.rope_turns(rope, "cpu").tolist()):
        # half a unit of rounding, and the 64-bit quotient's: its value is below 2^62
        assert abs(t - Fraction(float(f)) / two_pi * 2 ** 64) <= Fraction(3, 4) and 0 <= t < 2 ** 62


def test_frequencies_by_parts_between_the_others():
    """Many turns within the trained context: as trained; few: stretched; the blend falls from one to the other."""
    kw = dict(factor=8.0, context=32768, low=1.0, high=32.0)
    plain, parts = co.frequencies(128, 1e6), co.frequencies(128, 1e6, "parts", **kw)
    turns = 32768 * plain / (2 * math.pi)
    assert np.array_equal(parts[turns >= 32], plain[turns >= 32]) and np.allclose(parts[turns <= 1], plain[turns <= 1] / 8)
    assert np.all(np.diff(parts / plain) <= 1e-15) and 0 < np.sum((turns > 1) & (turns < 32))


def test_a_scaled_base_past_the_largest_number_is_refused(gdn):
    """base s^(R/(R-2)), which as an infinity would make every frequency but the first 0; just below it is taken (the
    exponents of the reference are up to 710, a few roundings of which are below 710 x 8 x 2^-53 < 1e-12)."""
    for base, factor, rot in ((1e300, 1e8, 16), (1e300, 1e9, 256), (2.0, 1e300, 16), (1e308, 1.8, 64)):
        with pytest.raises(gdn.GdnError, match="base, factor: "):
            gdn.Rope(rot_dims=rot, base=base, scaling="base", factor=factor).check()
        with pytest.raises(gdn.GdnError, match="base, factor: "):
            gdn.rope_turns(gdn.Rope(rot_dims=rot, base=base, scaling="base", factor=factor), "cpu")
        gdn.Rope(rot_dims=rot, base=base, scaling="linear", factor=factor).check()
    rope = gdn.Rope(rot_dims=64, base=1e300, scaling="base", factor=1e7)
    rope.check()
    got, ref = np.array(gdn.rope_frequencies(rope)), co.frequencies(64, 1e300, "base", 1e7)
    assert np.all(got > 0) and np.max(np.abs(got / ref - 1)) < 1e-12


def test_rope_mirror(gdn):
    r = gdn.Rope(layout="pairs", inverse=True)
    s = r.c_struct()
    assert (s.rot_dims, s.layout, s.scaling, s.flags, s.base, s.amplitude) == (64, 1, 0, 1, 1e4, 1.0)
    r.check()
    for other in (copy.copy(r), copy.deepcopy(r), pickle.loads(pickle.dumps(r))):
        assert other == r and "_c_ref" not in other.__dict__
        other.check()
    with pytest.raises(ValueError, match="layout: 'halves', required: one of half, pairs"):
        gdn.Rope(layout="halves").check()
    with pytest.raises(ValueError, match="scaling: 'ntk'"):
        gdn.Rope(scaling="ntk").check()
    with pytest.raises(gdn.GdnError, match="rot_dims: 24"):
        gdn.rope_turns(gdn.Rope(rot_dims=24), "cpu")
    with pytest.raises(gdn.GdnError, match="rot_dims: -2"):
        gdn.rope_frequencies(gdn.Rope(rot_dims=-2))


# ---------------------------------------------------------------- the binding

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


PAGE = (9, 2, 16, 64)


def _calls(m):
    """Every entry point with tensors of one device: (function, tensors by name)."""
    i = lambda *s: _On(s, I32)  # noqa: E731
    b = lambda *s: _On(s, BF16)  # noqa: E731
    f = lambda *s: _On(s, F32)  # noqa: E731
    rotate = {"turns": _On((16,), I64), "position": i(7), "q": b(7, 4, 64), "k": b(7, 2, 64), "q_out": b(7, 4, 64),
              "k_out": b(7, 2, 64), "v": b(7, 2, 64), "cache.k": b(*PAGE), "cache.v": b(*PAGE), "slot_map": i(7), "dev_err": i(1)}
    weights = {"k_cache": b(*PAGE), "block_table": i(2, 3), "kv_len": i(2), "q": b(2, 4, 4, 64), "score_out": f(2, 40),
               "workspace": i(1), "score_in": f(2, 40), "have_len": i(2), "n_row": i(2), "dev_err": i(1)}
    plan = {"kv_len": i(5), "budget": i(5), "score": f(5, 40), "token_pos": i(5, 40), "row_state": i(5, 2), "block_table": i(5, 3),
            "free_pages": i(9), "n_free": i(1), "score_out": f(5, 40), "token_pos_out": i(5, 40), "kv_len_out": i(5),
            "row_state_out": i(5, 2), "n_free_out": i(1), "move_src": i(5, 6), "move_dst": i(5, 6), "n_moves": i(5), "dev_err": i(1)}
    move = {"cache.k": b(*PAGE), "cache.v": b(*PAGE), "move_src": i(5, 6), "move_dst": i(5, 6), "n_moves": i(5), "dev_err": i(1)}
    return dict(rope_rotate=rotate, attn_weights=weights, evict_plan=plan, kv_move=move)


def _call(m, name, tensors, stream=None):
    geom = m.AttnGeometry(n_q_heads=4, n_kv_heads=2, d_head=64, n_pages=9, max_pages=3, max_tree=4)
    kw = {k: t for k, t in tensors.items() if "." not in k}
    if "cache.k" in tensors:
        kw["cache"] = m.KVCache(tensors["cache.k"], tensors["cache.v"])
    if name == "rope_rotate":
        kw["rope"] = m.Rope(rot_dims=32)
    getattr(m, name)(geom, **kw, stream=stream)


NAMES = ["rope_rotate", "attn_weights", "evict_plan", "kv_move"]


@pytest.mark.parametrize("name", NAMES)
def test_every_tensor_is_on_the_current_device(gdn, on_gpu_0, name):
    """Each tensor of a call on another device than the rest, and all of them on another device than the current one,
    are refused before the library sees an address."""
    for other in _calls(gdn)[name]:
        tensors = _calls(gdn)[name]
        tensors[other].index = 1
        tensors[other].device = torch.device("cuda", 1)
        with pytest.raises(ValueError, match="required: cuda:|required: the current device"):
            _call(gdn, name, tensors)
    tensors = _calls(gdn)[name]
    for t in tensors.values():
        t.index, t.device = 1, torch.device("cuda", 1)
    with pytest.raises(ValueError, match="tensors on cuda:1, required: the current device cuda:0"):
        _call(gdn, name, tensors)
    with pytest.raises(ValueError, match="stream: of cuda:1"):
        _call(gdn, name, _calls(gdn)[name], stream=_Stream(1))


@pytest.mark.parametrize("name", NAMES)
def test_every_shape_and_type_is_checked(gdn, on_gpu_0, name):
    with pytest.raises(AssertionError, match="got past"):
        _call(gdn, name, _calls(gdn)[name])
    for other, t in _calls(gdn)[name].items():
        if other == "workspace":
            continue
        wrong = F32 if t.dtype != F32 else BF16
        tensors = _calls(gdn)[name]
        tensors[other] = _On(tuple(t.shape), wrong)
        with pytest.raises(ValueError, match="dtype"):
            _call(gdn, name, tensors)
        tensors = _calls(gdn)[name]
        tensors[other] = _On((*t.shape[:-1], t.shape[-1] + 1), t.dtype)
        with pytest.raises(ValueError, match="shape|strides"):
            _call(gdn, name, tensors)
        tensors = _calls(gdn)[name]
        tensors[other] = None
        if other in ("q_out", "k_out", "score_in", "have_len", "n_row", "dev_err", "q"):
            continue  # may be left out (q_out without q may not, below)
        with pytest.raises((ValueError, AttributeError)):
            _call(gdn, name, tensors)


def test_rotate_arguments_that_do_not_go_together(gdn, on_gpu_0):
    def call(**change):
        tensors = _calls(gdn)["rope_rotate"]
        tensors.update(change)
        for n in [n for n, t in tensors.items() if isinstance(t, str)]:
            del tensors[n]
        _call(gdn, "rope_rotate", tensors)
    drop = "drop"
    with pytest.raises(ValueError, match="q, k: both missing"):
        call(q=None, k=None)
    with pytest.raises(ValueError, match="q_out: given without q"):
        call(q=None)
    with pytest.raises(ValueError, match="k: missing"):
        call(k=None)
    with pytest.raises(ValueError, match="v: missing"):
        call(v=None)
    with pytest.raises(ValueError, match="cache: missing"):
        call(**{"cache.k": drop, "cache.v": drop})
    with pytest.raises(AssertionError, match="got past"):
        call(**{"cache.k": drop, "cache.v": drop, "v": drop, "slot_map": drop})
    with pytest.raises(AssertionError, match="got past"):
        call(q=None, q_out=None)


# ---------------------------------------------------------------- the oracle

def test_oracle_rotation():
    """Closed forms: position 0 is the amplitude alone, a quarter turn swaps, lengths stay, layouts are one map on
    permuted dimensions, and products of rotated vectors depend on the distance alone."""
    rng = np.random.Generator(np.random.PCG64(5))
    x = rng.standard_normal((3, 2, 24))
    f = co.frequencies(16, 1e4)
    assert np.array_equal(co.rotate(x, [0, 0, 0], f, "half", 1.5)[..., :16], 1.5 * x[..., :16])
    quarter = co.rotate(x, [1, 1, 1], [math.pi / 2] * 8, "half")
    assert np.allclose(quarter[..., :8], -x[..., 8:16]) and np.allclose(quarter[..., 8:16], x[..., :8])
    y = co.rotate(x, [3, 70000, -9], f, "half")
    assert np.allclose(np.sum(y * y, -1), np.sum(x * x, -1)) and np.array_equal(y[..., 16:], x[..., 16:])
    perm = [d for i in range(8) for d in (i, i + 8)]
    pairs = co.rotate(x[..., perm + list(range(16, 24))], [3, 70000, -9], f, "pairs")
    assert np.allclose(pairs[..., :16], y[..., perm])
    assert np.allclose(co.rotate(y, [3, 70000, -9], f, "half", inverse=True), x)
    a, b = (np.sum(co.rotate(x[:1], [p], f, "half") * co.rotate(x[1:2], [p + 11], f, "half")) for p in (0, 900))
    assert abs(a - b) < 1e-10


def test_oracle_weights():
    """Equal logits share a query's weight evenly; all of it is given out; the last key gets one query's alone."""
    rng = np.random.Generator(np.random.PCG64(6))
    k = rng.standard_normal((9, 2, 8))
    q = rng.standard_normal((3, 6, 8))
    w = co.weights(q, k, 0.3)
    assert abs(w.sum() - 18) < 1e-12 and np.all(w > 0) and w[8] < 6
    assert np.allclose(co.weights(np.zeros((2, 2, 8)), k, 1.0), [2 * (1 / 8 + 1 / 9)] * 8 + [2 / 9])
    assert np.allclose(co.weights(q[:1], k[:1], 1.0), [6.0])


def test_oracle_evict():
    """One row by hand: tokens 1 and 5 have equal scores, token 0 is protected, the newest is too; a budget of less than
    the protected tokens is refused."""
    tables = np.array([[4, 2, 7]], np.int32)
    score = np.array([[0.0, 0.5, 0.9, 0.1, 0.2, 0.5, 0.6, 0.3]], np.float32)
    call = lambda b: co.evict(4, 9, 3, [8], [b], score, np.zeros((1, 8), np.int32), [[0, 3]], tables, [1], 1, 4, 1, 9)  # noqa: E731
    # positions 3 .. 10: token 0 (3 < 4) and token 7 stay; then 2 and 6, then 1 before 5
    rows, stack, bad = call(5)
    assert not bad and rows[0]["kv_len"] == 5 and rows[0]["state"] == [5, 6]
    assert rows[0]["pos"] == [3, 4, 5, 9, 10] and np.allclose(rows[0]["score"], [0.0, 0.5, 0.9, 0.6, 0.3])
    assert rows[0]["src"] == [2 * 4 + 2, 2 * 4 + 3] and rows[0]["dst"] == [4 * 4 + 3, 2 * 4 + 0]
    assert stack == [1]  # 5 tokens still take two pages
    rows, stack, bad = call(4)
    assert bad and rows[0]["kv_len"] == 8 and rows[0]["state"] == [0, 3] and rows[0]["pos"] == list(range(3, 11)) and stack == [1]
