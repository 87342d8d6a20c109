"""The attention's PyTorch module and the library that it calls. No GPU is needed."""
import ctypes
import types

import pytest
import torch

import moe_expert_layer_top_gb300 as pkg
from moe_expert_layer_top_gb300 import abi, attention

ENTRIES = ("moe_qkv_append", "moe_attend_paged_workspace", "moe_attend_paged", "moe_attend_prompt_workspace",
           "moe_attend_prompt")


@pytest.fixture(scope="module", autouse=True)
def built():
    pkg.build.build()


def addresses(lib):
    return tuple(ctypes.cast(getattr(lib, name), ctypes.c_void_p).value for name in ENTRIES)


def test_calls_follow_a_change_of_the_library(monkeypatch):
    """A process that goes on to the bounds-checked library, and back, does not stay with the first one's kernels."""
    bound = []
    fake = types.SimpleNamespace(bind=lambda *a: bound.append(a))
    monkeypatch.setattr(attention, "_module", fake)
    monkeypatch.setattr(attention, "_bound", None, raising=False)
    want = []
    for debug in ("0", "1", "0"):
        monkeypatch.setenv("MOE_DEBUG_BOUNDS", debug)
        monkeypatch.setattr(abi, "_lib", None)
        lib = abi.load()
        assert attention._native() is fake and attention._native() is fake
        want.append(addresses(lib))
    assert want[0] != want[1]
    assert bound == want  # once for each change


def test_the_module_loads_once():
    assert attention._native() is attention._native()


def test_prompt_flags():
    io = abi.MoeAttendPromptIO(num_heads=8, num_kv_heads=2, head_dim=64, causal=1, scale=0.1)  # no rows: nothing runs
    assert abi.moe_attend_prompt(io) == abi.MOE_OK
    io.flags = abi.MOE_FLAG_TEST_SKIP_READY
    assert abi.moe_attend_prompt(io) == abi.MOE_OK
    io.flags = 1
    assert abi.moe_attend_prompt(io) == abi.MOE_ERR_INVALID_ARG


def test_append_and_paged_flags():
    cache = abi.MoeKvCache(num_pages=0, page_size=16, num_kv_heads=2, head_dim=64)
    for io, call in ((abi.MoeQkvAppendIO(num_heads=8, num_kv_heads=2, head_dim=64), abi.moe_qkv_append),
                     (abi.MoeAttendPagedIO(num_heads=8, max_rows=1, scale=0.1),
                      lambda io, c: abi.moe_attend_paged(io, c, None, 0))):
        for flags, code in ((0, abi.MOE_OK), (abi.MOE_FLAG_TEST_BOUNDS, abi.MOE_OK), (1, abi.MOE_ERR_INVALID_ARG),
                            (abi.MOE_FLAG_TEST_SKIP_READY, abi.MOE_ERR_INVALID_ARG)):
            io.flags = flags
            assert call(io, cache) == code


def test_inputs_that_require_gradients_are_refused():
    x = lambda *shape: torch.zeros(*shape, dtype=torch.bfloat16)
    q, k, cu = x(4, 8, 64), x(4, 2, 64), torch.tensor([0, 4], dtype=torch.int32)
    rope, pos = torch.zeros(4, 64), torch.zeros(4, dtype=torch.int32)

    def wants(t):
        return t.clone().requires_grad_()

    calls = [lambda: attention.qkv_append(wants(q), k, k),
             lambda: attention.qkv_append(q, wants(k), k),
             lambda: attention.qkv_append(q, k, wants(k)),
             lambda: attention.qkv_append(q, k, k, rope=wants(rope), positions=pos),
             lambda: attention.qkv_append(q, k, k, q_norm=wants(x(64))),
             lambda: attention.qkv_append(q, k, k, k_norm=wants(x(64))),
             lambda: attention.qkv_append(q, k, k, q_out=wants(q)),
             lambda: attention.attend_paged(wants(q), None, cu[None], cu[:1], cu),
             lambda: attention.attend_paged(q, None, cu[None], cu[:1], cu, out=wants(q)),
             lambda: attention.attend_prompt(wants(q), k, k, cu, cu),
             lambda: attention.attend_prompt(q, wants(k), k, cu, cu),
             lambda: attention.attend_prompt(q, k, wants(k), cu, cu),
             lambda: attention.attend_prompt(q, k, k, cu, cu, out=wants(q))]
    for call in calls:
        with pytest.raises(ValueError, match="no backward pass"):
            call()
        with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):  # these are host tensors
            call()


def test_a_stream_of_another_device_is_refused():
    """The call would run on the tensors' device, and not on that stream."""
    stream = types.SimpleNamespace(device=torch.device("cuda:1"))
    with pytest.raises(ValueError, match="stream is on cuda:1"):
        attention._on(stream, torch.device("cuda:0"))
