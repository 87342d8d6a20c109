"""The calls of a step with drafted trees on the bounds-checked build (libmoe_debug.so).

Their tests run once more against it, in a child process, and positive controls show that the checks are live without
any access out of bounds: MOE_FLAG_TEST_BOUNDS halves the capacity that they see."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from moe_expert_layer_top_gb300 import abi, attention

import attention_cases as ac

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def built():
    import moe_expert_layer_top_gb300 as pkg
    pkg.build.build()
    assert os.path.exists(pkg.build.DEBUG_LIB_PATH)
    assert torch.cuda.is_available()


@pytest.fixture(params=["debug", "normal"])
def library(request, monkeypatch):
    """One of the two libraries for a test; whether its checks are live."""
    monkeypatch.setenv("MOE_DEBUG_BOUNDS", "1" if request.param == "debug" else "0")
    monkeypatch.setattr(abi, "_lib", None)
    abi.load()
    yield request.param == "debug"
    torch.cuda.synchronize()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rows", [4, 64])  # both kinds of kernel
@pytest.mark.parametrize("flags", [0, abi.MOE_FLAG_TEST_BOUNDS])
def test_tree_checks_are_live(library, flags, rows, D):
    H, K, n = 8, 8, 6000  # more than half of the blocks leave a part
    rng = np.random.default_rng(2)
    c = ac.Cache(rng, [n], K, D, 64)
    q = ac.dev(ac.rows16(rng, (rows, H, D), "bf16", 1.0), "bf16")
    parents, lens, cu = ac.i32(list(range(-1, rows - 1))), ac.i32([n]), ac.i32([0, rows])
    want, z = attention.attend_tree(q, c.cache, c.table, lens, cu, parents, max_rows=rows, return_lse=True)
    out, lse = torch.zeros_like(q), torch.zeros(rows, H, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    io = abi.MoeAttendTreeIO(
        abi.MoeAttendPagedIO(q.data_ptr(), H * D, out.data_ptr(), H * D, lse.data_ptr(), c.table.data_ptr(),
                             lens.data_ptr(), cu.data_ptr(), 1, rows, c.max_pages, rows, H, abi.MOE_DTYPE_BF16,
                             D ** -0.5, flags), parents.data_ptr())
    kv = c.cache.as_abi()
    size = abi.moe_attend_tree_workspace(io, kv)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    assert abi.moe_attend_tree(io, kv, ws, size, st, torch.cuda.current_stream()) == abi.MOE_OK
    torch.cuda.synchronize()
    trips = library and flags
    assert st.item() == (abi.MOE_ERR_DEVICE_BOUNDS if trips else abi.MOE_OK)
    if not trips:
        assert torch.equal(out, want) and torch.equal(lse, z)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("flags", [0, abi.MOE_FLAG_TEST_BOUNDS])
def test_commit_checks_are_live(library, flags, D):
    K, page = 2, 16
    rng = np.random.default_rng(3)
    parts = [rng.integers(0, 256, (2, K, page, w), dtype=np.uint8) for w in (D // 2, D // 32, D // 2, D // 32)]
    c = attention.KVCacheMXFP4(*(torch.from_numpy(p).cuda() for p in parts))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    path, accepted, new = ac.i32([0, 2]), ac.i32([1]), ac.i32([0])
    table, lens, cu = ac.i32([1]), ac.i32([10]), ac.i32([0, 3])  # the page past the checks' limit
    io = abi.MoeCommitDraftsIO(table.data_ptr(), lens.data_ptr(), cu.data_ptr(), path.data_ptr(), accepted.data_ptr(),
                               new.data_ptr(), 1, 1, 2, 1, flags)
    assert abi.moe_commit_drafts(io, [c.as_abi()], st, torch.cuda.current_stream()) == abi.MOE_OK
    torch.cuda.synchronize()
    trips = library and flags
    assert st.item() == (abi.MOE_ERR_DEVICE_BOUNDS if trips else abi.MOE_OK)
    for was, now in zip(parts, (c.k_codes, c.k_scales, c.v_codes, c.v_scales)):
        want = was.copy()
        if not trips:
            want[1, :, 8] = was[1, :, 9]
        assert np.array_equal(now.cpu().numpy(), want)


def test_speculative_tests_under_the_bounds_checked_build():
    env = dict(os.environ, MOE_DEBUG_BOUNDS="1")
    cmd = [sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider",
           "tests/test_gpu_tree_attention.py", "tests/test_gpu_speculative.py"]
    r = subprocess.run(cmd, cwd=ROOT, env=env, capture_output=True, text=True, timeout=900)
    tail = "\n".join((r.stdout + r.stderr).splitlines()[-30:])
    assert r.returncode == 0, tail
    assert " passed" in r.stdout and "failed" not in r.stdout, tail
