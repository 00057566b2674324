"""The paged-cache, attention and tree entry points on the host (no GPU): every refusal, from C under the sanitizers and
through the Python binding; the oracle's own pins."""
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

import gdn_inputs as gi
from oracle import attn_oracle as ao
from oracle import gdn_oracle as orc

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "gated_deltanet_delta_amd", "csrc")
BUILD = os.path.join(ROOT, "_build")
SAN = ["-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-fno-omit-frame-pointer", "-g", "-O1"]


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
    drv, exe = str(tmp_path / "drv.o"), str(tmp_path / "attn_refusals")
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-Werror", *SAN, *inc, "-c",
                    os.path.join(ROOT, "tests", "attn_refusals.c"), "-o", drv], check=True)
    subprocess.run(["g++", *SAN, drv, *host, *objs, "-L", os.path.join(rocm, "lib"), "-lamdhip64",
                    "-Wl,-rpath," + os.path.join(rocm, "lib"), "-o", exe], check=True)
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0", UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=120)
    assert r.returncode == 0, (r.returncode, r.stdout, r.stderr[-4000:])
    assert "attention refusals ok" in r.stdout
    assert "runtime error" not in r.stderr and "AddressSanitizer" not in r.stderr, r.stderr[-4000:]


def test_geometry_mirror(gdn):
    g = gdn.AttnGeometry()
    g.check()
    s = g.c_struct()
    assert (s.n_q_heads, s.n_kv_heads, s.d_head, s.dtype) == (24, 4, 256, gdn.GDN_BF16) and s.scale == 0.0625
    with pytest.raises(gdn.GdnError, match="n_q_heads: 23"):
        gdn.AttnGeometry(n_q_heads=23).check()
    with pytest.raises(gdn.GdnError, match="d_head: 96"):
        gdn.AttnGeometry(d_head=96).check()


def test_workspace_sizes(gdn):
    """Few row tiles split the key axis and need a workspace; many do not."""
    g = gdn.AttnGeometry(max_tree=64)
    assert gdn.attn_prefill_workspace_bytes(g, 100000, 4) == 0
    # fp32: a part (sums, maximum, sum of weights) per row and split
    per = 24 * (256 + 2) * 4
    g32 = gdn.AttnGeometry(max_tree=64, dtype=torch.float32)
    for n, b in ((1, 1), (16, 4), (64, 2)):
        w = gdn.attn_tree_workspace_bytes(g32, b, n)
        assert w % (per * b * n) == 0 and 2 <= w // (per * b * n) <= 1024
    # bf16: parts of at most two blocks of rows (32 at least) per workgroup, so
    # the batch adds no more than 8 bytes per block of rows
    one, many = (gdn.attn_tree_workspace_bytes(g, b, 1) for b in (1, 1000))
    assert one >= 2 * 32 * (256 + 2) * 4 and 0 < many - one <= 8 * 1000 * 4 + 256


def test_binding_refuses_host_tensors(gdn):
    """Tensors that are not on the GPU never reach the library."""
    g = gdn.AttnGeometry(n_q_heads=2, n_kv_heads=1, d_head=64, n_pages=2, max_pages=2)
    t = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="q: must be a device tensor"):
        gdn.attn_prefill(g, t, t[:, :1], t[:, :1], i, t)
    with pytest.raises(ValueError, match="kv_len: must be a device tensor"):
        gdn.kv_plan(g, i, i, i, i[:1], t, i, i, i, i, i)
    with pytest.raises(ValueError, match="cache.k: must be a device tensor"):
        gdn.kv_write(g, gdn.KVCache(t, t), t, t, i)
    with pytest.raises(ValueError, match="cache.k: must be a device tensor"):
        gdn.attn_tree(g, gdn.KVCache(t, t), i, i, t[None], t[None], t[None], i, t[None])


class _OnGpu:
    """A tensor's shape, strides and type under an is_cuda that says yes: for the binding's host checks alone."""

    def __init__(self, t):
        self.t, self.is_cuda, self.dtype, self.shape = t, True, t.dtype, t.shape

    def stride(self):
        return self.t.stride()

    def is_contiguous(self):
        return self.t.is_contiguous()


def test_row_strides_of_the_binding(gdn):
    """Parts of a fused row pass with their row's stride; transposed or scattered rows are refused."""
    need = lambda t, shape: gdn._need_rows(_OnGpu(t), "q", shape, torch.float32)  # noqa: E731
    rows = torch.zeros(6, 8, 64)
    assert need(rows, (6, 8, 64)) == 512
    assert need(rows[:, 2:5], (6, 3, 64)) == 512
    assert need(rows[::2], (3, 8, 64)) == 1024
    assert need(rows[:1], (1, 8, 64)) == 512
    assert need(rows[:, 2:5].unflatten(0, (2, 3)), (2, 3, 3, 64)) == 512
    assert need(rows[:, :1].unflatten(0, (6, 1)), (6, 1, 1, 64)) == 512
    for bad, shape in ((rows.transpose(0, 1), (8, 6, 64)), (rows[:, ::2], (6, 4, 64)), (rows[..., ::2], (6, 8, 32)),
                       (rows.unflatten(0, (2, 3))[:, :2], (2, 2, 8, 64))):
        with pytest.raises(ValueError, match="strides"):
            need(bad, shape)
    with pytest.raises(ValueError, match="shape"):
        need(rows, (6, 8, 32))


# ---- the oracle's own pins -------------------------------------------------

def test_oracle_attention_special_cases():
    rng = np.random.Generator(np.random.PCG64(1))
    q, k, v = rng.normal(size=(3, 4, 8)), rng.normal(size=(5, 2, 8)), rng.normal(size=(5, 2, 8))
    one = np.zeros((3, 5), bool)
    one[:, 2] = True
    o, mag = ao.attend(q, k, v, one, 0.3)  # a single key: its value
    assert np.allclose(o, np.repeat(v[2], 2, axis=0)[None], atol=1e-14) and np.allclose(mag, np.abs(o))
    o, _ = ao.attend(np.zeros_like(q), k, v, np.ones((3, 5), bool), 0.3)  # equal logits: the mean
    assert np.allclose(o, np.repeat(v.mean(0), 2, axis=0)[None], atol=1e-14)
    a, _ = ao.attend(q, k, v, np.ones((3, 5), bool), 0.3)  # a constant added to every logit changes nothing
    shift = np.concatenate([k, np.ones((5, 2, 1))], axis=2), np.concatenate([q, np.full((3, 4, 1), 7.0)], axis=2)
    b, _ = ao.attend(shift[1], shift[0], np.concatenate([v, v[..., :1]], axis=2), np.ones((3, 5), bool), 0.3)
    assert np.allclose(a, b[..., :8], atol=1e-12)


def test_oracle_tree_of_a_chain_is_causal_attention():
    rng = np.random.Generator(np.random.PCG64(2))
    n, c, page = 5, 21, 16
    q, k, v = rng.normal(size=(n, 4, 8)), rng.normal(size=(n, 2, 8)), rng.normal(size=(n, 2, 8))
    kc, vc = rng.normal(size=(4, 2, page, 8)), rng.normal(size=(4, 2, page, 8))
    table = np.array([3, 1, 0])
    a, _ = ao.tree(q, k, v, np.arange(-1, n - 1), kc, vc, table, c, 0.4)
    b, _ = ao.prefill(q, k, v, [0, n], kc, vc, table[None], [c], 0.4)
    assert np.allclose(a, b, atol=1e-13)
    assert ao.tree_paths([-1, 0, 0, 2]).tolist() == [[1, 0, 0, 0], [1, 1, 0, 0], [1, 0, 1, 0], [1, 0, 1, 1]]


def test_oracle_verify_tree_of_a_chain_is_the_chain_verify():
    g = gi.Geometry(n_k_heads=1, n_v_heads=2, d_k=16, d_v=16, n_slots=2)
    inp = gi.verify_inputs(seed=3, geom=g, batch=1, k=4)
    s = int(inp["slots"][0])
    args = (g, inp["state"][s], inp["hist"][s], inp["x"][0], inp["a"][0], inp["b"][0], inp["conv_w"])
    o, st, h, depth = ao.verify_tree(*args, np.arange(-1, 3))
    o2, st2, h2 = orc.verify(*args)
    assert np.allclose(o, o2, atol=1e-13) and np.allclose(st, st2, atol=1e-13) and np.array_equal(h, h2)
    assert depth.tolist() == [1, 2, 3, 4]


def test_oracle_plan_by_hand():
    """Two pages of 16: a row that grows over a page border takes the stack's top, a leaving row's page goes there first."""
    r = ao.kv_plan(16, 6, 3, [15, 10, 0], [2, -1, 3], np.array([5, 2, -1, -1, -1, -1]), 2,
                   np.array([[0, -1, -1], [4, -1, -1], [-1, -1, -1]]), 7)
    assert r["block_table"].tolist() == [[0, 4, -1], [4, -1, -1], [2, -1, -1]]
    assert r["free_pages"].tolist() == [5, 2, 4, -1, -1, -1] and r["n_free_out"] == 1
    assert r["cu_new"].tolist() == [0, 2, 2, 5] and r["kv_len_out"].tolist() == [17, 0, 3]
    assert r["slot_map"].tolist() == [15, 64, 32, 33, 34, -1, -1] and r["position"].tolist() == [15, 16, 0, 1, 2, 0, 0]
