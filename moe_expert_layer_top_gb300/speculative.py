"""The end of a speculative step with trees (or chains) of drafted tokens, for PyTorch device memory and streams.

A step appends the rows of a tree (``attention.qkv_append``) at the end of each
sequence, in any order that puts a row behind its parent, runs the layers with
``attention.attend_tree``, and ends with

* ``verify_drafts``: which of the drafted tokens the target accepts, from given
  random numbers, and the token behind them;
* ``commit_drafts``: the accepted tokens' keys and values moved together in the
  caches of all layers, and the sequences' new lengths.

Streams, outputs, gradients, errors and ``d_status`` are as for the calls of ``attention``.
"""
from __future__ import annotations

import torch

from . import abi, attention
from .attention import KVCacheMXFP4


def verify_drafts(logits: torch.Tensor, tokens: torch.Tensor, cu_rows: torch.Tensor, accept_u: torch.Tensor,
                  sample_u: torch.Tensor, *, parents: torch.Tensor | None = None,
                  draft_probs: torch.Tensor | None = None, temperature: torch.Tensor | None = None, max_rows: int,
                  d_status: torch.Tensor | None = None, stream=None) -> dict:
    """The drafted tokens against the target's probabilities.

    logits [rows][vocab] (bf16, fp16 or fp32; rows may be strided): the target's behind each row; tokens int32 [rows];
    cu_rows int32 [sequences + 1]; parents int32 [rows] as for ``attention.attend_tree`` (None: chains). The first row of
    each sequence is the root, a token that is settled; its children are asked in their order, then those of the
    accepted one, and so on.
    draft_probs fp32 [rows][vocab]: the probabilities that the children of each row were drawn from (independently). A
    rejection leaves max(p - draft_probs, 0) of the target's p, normalised. None: the children were chosen without
    chance, and a rejected token leaves p without it.
    temperature fp32 [sequences]: of the target, 0 for greedy; None: 1.
    accept_u fp32 [rows], sample_u fp32 [sequences]: random numbers in [0, 1).
    max_rows: rows of a sequence at most (up to 256).

    Returns {"tokens": int32 [sequences][max_rows], the accepted tokens, then the new one, then -1; "accepted": int32
    [sequences], how many were accepted; "path": int32 [sequences][max_rows], the rows from the root (0) to the last
    accepted one, then -1}.
    """
    module = (attention._module if abi._lib is attention._bound is attention._bound_trees
              else attention._native_trees())
    return attention._call("moe_verify_drafts", module.verify, stream, logits, tokens, cu_rows, accept_u, sample_u,
                           parents, draft_probs, temperature, max_rows, d_status)


def commit_drafts(caches, page_table: torch.Tensor, lengths: torch.Tensor, cu_rows: torch.Tensor, path: torch.Tensor,
                  accepted: torch.Tensor, *, d_status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The accepted rows' keys and values moved to follow the context, in the caches of all layers.

    caches: a ``KVCacheMXFP4`` or a list of them, alike in page size, kv heads and head size, none twice; page_table int32
    [sequences][pages], shared by them; lengths int32 [sequences], the tree's rows included; path and accepted as
    ``verify_drafts`` returns them. Token base + path[j] goes to base + j, where base is the length without the tree.

    Returns the new lengths, base + 1 + accepted (int32 [sequences]).
    """
    module = (attention._module if abi._lib is attention._bound is attention._bound_trees
              else attention._native_trees())
    if isinstance(caches, KVCacheMXFP4):
        caches = (caches,)

    def call(lengths):
        return module.commit(caches, page_table, lengths, cu_rows, path, accepted, d_status)

    return attention._call("moe_commit_drafts", call, stream, lengths)
