"""The smoke step with drafted trees runs both kinds of attention kernel."""
import pytest
import torch

import __graft_entry__ as entry
from moe_expert_layer_top_gb300 import abi, attention

pytestmark = pytest.mark.gpu


def test_smoke_runs_both_kinds_of_tree_kernels(monkeypatch):
    entry.build()
    abi.load()
    sizes, call = [], attention.attend_tree

    def attend_tree(q, cache, table, lengths, cu_rows, parents, *, max_rows, **kw):
        io = abi.MoeAttendTreeIO()
        io.rows.num_seqs, io.rows.num_rows, io.rows.max_pages = len(lengths), len(q), table.shape[1]
        io.rows.max_rows, io.rows.num_heads, io.rows.dtype = max_rows, q.shape[1], abi.MOE_DTYPE_BF16
        sizes.append((abi.moe_attend_tree_workspace(io, cache.as_abi()), cache.head_dim))
        return call(q, cache, table, lengths, cu_rows, parents, max_rows=max_rows, **kw)

    monkeypatch.setattr(attention, "attend_tree", attend_tree)
    entry._smoke_drafts(torch.device("cuda", 0))
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    # large trees: a block on each SM, with two parts of 256 rows, a reference and a sum for each, and a record of 32 bytes
    large = [n == sms * (2 * 256 * (D + 2) * 4 + 32) for n, D in sizes]
    assert any(large) and not all(large)
