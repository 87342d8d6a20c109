"""The attention calls on the bounds-checked build (libmoe_debug.so): every derived index (cached rows, rows of the
output, places in the workspace, tiles) is checked there before its access.

The attention tests run once more against it, in a child process, and positive controls show that the checks are live
without any access out of bounds: MOE_FLAG_TEST_BOUNDS halves the capacity that they see."""
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


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def seeded(seed, *shape):
    return torch.randn(*shape, device="cuda", generator=torch.Generator("cuda").manual_seed(seed)).bfloat16()


@pytest.mark.parametrize("flags", [0, abi.MOE_FLAG_TEST_BOUNDS])
def test_append_checks_are_live(library, flags):
    T, H, K, D, page = 32, 4, 2, 64, 16
    x = seeded(1, T, H + 2 * K, D)
    c = attention.KVCacheMXFP4.empty(2, page, K, D)
    c.v_codes.zero_()
    c.v_scales.zero_()
    out, slots, st = torch.empty(T, H, D, device="cuda").bfloat16(), torch.arange(T, device="cuda"), status()
    stride = (H + 2 * K) * D
    io = abi.MoeQkvAppendIO(x.data_ptr(), x[:, H:].data_ptr(), x[:, H + K:].data_ptr(), stride, stride, stride, T, H, K, D,
                            abi.MOE_DTYPE_BF16, slots=slots.data_ptr(), q_out=out.data_ptr(), norm_eps=1e-6, flags=flags)
    assert abi.moe_qkv_append(io, c.as_abi(), st, torch.cuda.current_stream()) == abi.MOE_OK
    torch.cuda.synchronize()
    trips = library and flags
    assert st.item() == (abi.MOE_ERR_DEVICE_BOUNDS if trips else abi.MOE_OK)
    assert c.v_codes[0].any() and bool(c.v_codes[1].any()) == (not trips)  # the rows past the checks' limit
    assert torch.equal(out, x[:, :H])


@pytest.mark.parametrize("flags", [0, abi.MOE_FLAG_TEST_BOUNDS])
def test_paged_checks_are_live(library, flags):
    H, K, D, n = 8, 8, 128, 6000  # more than half of the blocks leave a part
    c = ac.Cache(np.random.default_rng(2), [n], K, D, 64)
    q, lens, cu = seeded(3, 1, H, D), ac.i32([n]), ac.i32([0, 1])
    want, z = attention.attend_paged(q, c.cache, c.table, lens, cu, return_lse=True)
    out, lse, st = torch.zeros_like(q), torch.zeros(1, H, device="cuda"), status()
    io = abi.MoeAttendPagedIO(q.data_ptr(), H * D, out.data_ptr(), H * D, lse.data_ptr(), c.table.data_ptr(),
                              lens.data_ptr(), cu.data_ptr(), 1, 1, c.max_pages, 1, H, abi.MOE_DTYPE_BF16, D ** -0.5,
                              flags)
    kv = c.cache.as_abi()
    size = abi.moe_attend_paged_workspace(io, kv)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    assert abi.moe_attend_paged(io, kv, ws, size, st, torch.cuda.current_stream()) == abi.MOE_OK
    torch.cuda.synchronize()
    trips = library and flags
    assert st.item() == (abi.MOE_ERR_DEVICE_BOUNDS if trips else abi.MOE_OK)
    if not trips:
        assert torch.equal(out, want) and torch.equal(lse, z)


@pytest.mark.parametrize("flags", [0, abi.MOE_FLAG_TEST_BOUNDS])
def test_prompt_checks_are_live(library, flags):
    H, K, D, n, m = 8, 2, 128, 40, 6000  # keys in parts
    q, k, v = seeded(4, n, H, D), seeded(5, m, K, D), seeded(6, m, K, D)
    cr, ck = ac.i32([0, n]), ac.i32([0, m])
    want, z = attention.attend_prompt(q, k, v, cr, ck, return_lse=True)
    out, lse, st = torch.zeros_like(q), torch.zeros(n, H, device="cuda"), status()
    io = abi.MoeAttendPromptIO(q.data_ptr(), k.data_ptr(), v.data_ptr(), H * D, K * D, K * D, out.data_ptr(), H * D,
                               lse.data_ptr(), cr.data_ptr(), ck.data_ptr(), 1, n, m, H, K, D, abi.MOE_DTYPE_BF16, 1,
                               D ** -0.5, flags=flags)
    io.workspace_bytes = abi.moe_attend_prompt_workspace(io)
    ws = torch.empty(io.workspace_bytes, dtype=torch.uint8, device="cuda")
    io.workspace = ws.data_ptr()
    assert abi.moe_attend_prompt(io, st, torch.cuda.current_stream()) == abi.MOE_OK
    torch.cuda.synchronize()
    trips = library and flags
    assert st.item() == (abi.MOE_ERR_DEVICE_BOUNDS if trips else abi.MOE_OK)
    if not trips:
        assert torch.equal(out, want) and torch.equal(lse, z)


def test_attention_tests_under_the_bounds_checked_build():
    env = dict(os.environ, MOE_DEBUG_BOUNDS="1")
    cmd = [sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider",
           "tests/test_gpu_attention.py", "tests/test_gpu_attention_edges.py"]
    r = subprocess.run(cmd, cwd=ROOT, env=env, capture_output=True, text=True, timeout=900)
    tail = "\n".join((r.stdout + r.stderr).splitlines()[-30:])
    assert r.returncode == 0, tail
    assert " passed" in r.stdout and "failed" not in r.stdout, tail
