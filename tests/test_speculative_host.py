"""Refusals of the calls of a step with drafted trees. Everything here is decided on the host: no GPU is needed."""
import ctypes
import types

import pytest
import torch

import moe_expert_layer_top_gb300 as pkg
from moe_expert_layer_top_gb300 import abi, attention, speculative

from test_attention_host import INVALID, UNSUPPORTED, P, cache, paged_io

ENTRIES = ("moe_attend_tree_workspace", "moe_attend_tree", "moe_verify_drafts", "moe_commit_drafts")


@pytest.fixture(scope="module")
def lib():
    pkg.build.build()
    return abi.load()


def tree_io(parents=P, **kw):
    return abi.MoeAttendTreeIO(paged_io(**kw), parents)


@pytest.mark.parametrize("kw,expect", [
    (dict(num_heads=12), INVALID),
    (dict(dtype=2), INVALID),                       # logits only
    (dict(num_seqs=-1), INVALID),
    (dict(num_seqs=5000), UNSUPPORTED),
    (dict(max_pages=1 << 26), UNSUPPORTED),
    (dict(num_rows=1 << 27), UNSUPPORTED),
    (dict(max_rows=0), INVALID),
    (dict(scale=float("nan")), INVALID),
    (dict(q=None), INVALID),
    (dict(out=P + 8), INVALID),
    (dict(out_stride=4097), INVALID),
    (dict(lengths=None), INVALID),
    (dict(cu_rows=P + 2), INVALID),
    (dict(page_table=None), INVALID),
    (dict(parents=None), INVALID),
    (dict(parents=P + 2), INVALID),
    (dict(lse=P + 2), INVALID),
    (dict(flags=abi.MOE_FLAG_TEST_SKIP_READY << 2), INVALID),
])
def test_tree_refuses(lib, kw, expect):
    assert abi.moe_attend_tree(tree_io(**kw), cache(), P, 1 << 40) == expect


def test_tree_null_and_empty(lib):
    assert lib.moe_attend_tree(None, None, None, 0, None, None) == INVALID
    assert abi.moe_attend_tree(tree_io(num_rows=0, q=None, parents=None), cache(), None, 0) == abi.MOE_OK
    assert abi.moe_attend_tree(tree_io(num_seqs=0, cu_rows=None), cache(), None, 0) == abi.MOE_OK
    assert abi.moe_attend_tree(tree_io(), cache(k_codes=None), P, 1 << 40) == INVALID
    n = ctypes.c_int64(5)
    assert lib.moe_attend_tree_workspace(None, None, ctypes.byref(n)) == INVALID and n.value == 5


def verify_io(**kw):
    base = dict(logits=P, logits_stride=1000, draft_probs=P, draft_stride=1000, tokens=P, parents=P, cu_rows=P, temperature=P,
                accept_u=P, sample_u=P, out_tokens=P, path=P, accepted=P, num_seqs=2, num_rows=12, max_rows=6, vocab=1000,
                dtype=abi.MOE_DTYPE_F32, flags=0)
    base.update(kw)
    return abi.MoeVerifyDraftsIO(**base)


@pytest.mark.parametrize("kw,expect", [
    (dict(dtype=3), INVALID),
    (dict(flags=1), INVALID),
    (dict(num_seqs=-1), INVALID),
    (dict(num_rows=-1), INVALID),
    (dict(max_rows=0), INVALID),
    (dict(vocab=0), INVALID),
    (dict(num_seqs=65536), UNSUPPORTED),
    (dict(max_rows=257), UNSUPPORTED),
    (dict(vocab=(1 << 24) + 1, logits_stride=1 << 25, draft_stride=1 << 25), UNSUPPORTED),
    (dict(logits=None), INVALID),
    (dict(logits=P + 2), INVALID),
    (dict(logits=P + 1, dtype=abi.MOE_DTYPE_BF16), INVALID),
    (dict(logits_stride=999), INVALID),
    (dict(draft_stride=999), INVALID),
    (dict(draft_probs=P + 2), INVALID),
    (dict(tokens=None), INVALID),
    (dict(parents=P + 1), INVALID),
    (dict(cu_rows=None), INVALID),
    (dict(temperature=P + 2), INVALID),
    (dict(accept_u=None), INVALID),
    (dict(sample_u=None), INVALID),
    (dict(out_tokens=None), INVALID),
    (dict(path=P + 2), INVALID),
    (dict(accepted=None), INVALID),
])
def test_verify_refuses(lib, kw, expect):
    assert abi.moe_verify_drafts(verify_io(**kw)) == expect


def test_verify_null_and_empty(lib):
    assert lib.moe_verify_drafts(None, None, None) == INVALID
    assert abi.moe_verify_drafts(verify_io(num_seqs=0, logits=None)) == abi.MOE_OK
    assert abi.moe_verify_drafts(verify_io(), d_status=P + 1) == INVALID


def commit_io(**kw):
    base = dict(page_table=P, lengths=P, cu_rows=P, path=P, accepted=P, new_lengths=P, num_seqs=2, max_pages=8, path_stride=6,
                num_caches=2, flags=0)
    base.update(kw)
    return abi.MoeCommitDraftsIO(**base)


@pytest.mark.parametrize("kw,expect", [
    (dict(num_seqs=-1), INVALID),
    (dict(num_seqs=65536), UNSUPPORTED),
    (dict(max_pages=-1), INVALID),
    (dict(max_pages=1 << 26), UNSUPPORTED),
    (dict(path_stride=0), INVALID),
    (dict(num_caches=0), INVALID),
    (dict(num_caches=4097), UNSUPPORTED),
    (dict(flags=1), INVALID),
    (dict(page_table=None), INVALID),
    (dict(lengths=None), INVALID),
    (dict(cu_rows=P + 1), INVALID),
    (dict(path=None), INVALID),
    (dict(accepted=P + 2), INVALID),
    (dict(new_lengths=None), INVALID),
])
def test_commit_refuses(lib, kw, expect):
    assert abi.moe_commit_drafts(commit_io(**kw), [cache(), cache()]) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(page_size=24), UNSUPPORTED),
    (dict(page_size=32), INVALID),                  # not the first one's
    (dict(num_kv_heads=4), INVALID),
    (dict(head_dim=64), INVALID),
    (dict(head_dim=80), UNSUPPORTED),
    (dict(k_scales=None), INVALID),
    (dict(v_codes=P + 8), INVALID),
])
def test_commit_refuses_caches(lib, kw, expect):
    assert abi.moe_commit_drafts(commit_io(), [cache(), cache(**kw)]) == expect


def test_commit_null_and_empty(lib):
    assert lib.moe_commit_drafts(None, None, None, None) == INVALID
    assert abi.moe_commit_drafts(commit_io(num_seqs=0, lengths=None), [cache(), cache()]) == abi.MOE_OK
    assert abi.moe_commit_drafts(commit_io(), [cache(), cache()], d_status=P + 1) == INVALID


def test_calls_follow_a_change_of_the_library(lib, monkeypatch):
    bound, trees = [], []
    fake = types.SimpleNamespace(bind=lambda *a: bound.append(a), bind_trees=lambda *a: trees.append(a))
    monkeypatch.setattr(attention, "_module", fake)
    monkeypatch.setattr(attention, "_bound", None)
    monkeypatch.setattr(attention, "_bound_trees", None)
    want = []
    for debug in ("0", "1", "0"):
        monkeypatch.setenv("MOE_DEBUG_BOUNDS", debug)
        monkeypatch.setattr(abi, "_lib", None)
        loaded = abi.load()
        assert attention._native_trees() is fake and attention._native_trees() is fake
        want.append(tuple(ctypes.cast(getattr(loaded, name), ctypes.c_void_p).value for name in ENTRIES))
    assert trees == want and len(bound) == 3


def test_wrappers_refuse_host_tensors_and_gradients(lib):
    x = torch.zeros(4, 8, 64, dtype=torch.bfloat16)
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        attention.attend_tree(x, None, i[None], i[:1], i[:2], i)
    with pytest.raises(ValueError, match="no backward pass"):
        attention.attend_tree(x.clone().requires_grad_(), None, i[None], i[:1], i[:2], i)
    logits, u = torch.zeros(4, 9), torch.zeros(4)
    with pytest.raises(ValueError, match="CUDA"):
        speculative.verify_drafts(logits, i, i[:2], u, u[:1], max_rows=4)
    for name in ("draft_probs", "temperature"):
        with pytest.raises(ValueError, match="no backward pass"):
            speculative.verify_drafts(logits, i, i[:2], u, u[:1], max_rows=4, **{name: torch.zeros(4, 9, requires_grad=True)})
    with pytest.raises(ValueError, match="no backward pass"):
        speculative.verify_drafts(logits.clone().requires_grad_(), i, i[:2], u, u[:1], max_rows=4)
    with pytest.raises(ValueError, match="CUDA"):
        speculative.commit_drafts([object()], i[None], i[:1], i[:2], i[None], i[:1])
    with pytest.raises(TypeError, match="list"):
        speculative.commit_drafts(None, i[None], i[:1], i[:2], i[None], i[:1])
