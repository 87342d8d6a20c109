"""The attention in front of the MoE step, for PyTorch device memory and streams.

Three calls over the C ABI, in the order a decoder layer makes them:

* ``qkv_append``: RMSNorm of each query and key head, rotary positions, and
  the MXFP4 append of keys and values to a paged cache;
* ``attend_paged``: attention of the newest rows of each sequence (single
  tokens, or the rows of a verify step) over that cache;
* ``attend_prompt``: causal attention over packed prompts in 16 bits. Given
  ``k_cached`` and ``v_cached`` of ``qkv_append`` it attends over the very
  values that later steps read from the cache.

PyTorch only supplies device memory and streams here; every step runs in
libmoe.so, and a failed call raises. Sizes that live on the device (lengths,
pages, slots, positions) are checked there: pass ``d_status``, an int32 tensor
set to MOE_OK, and look at it when convenient (MOE_ERR_DEVICE_BOUNDS: something
was out of range and was not accessed; MOE_ERR_TIMEOUT: a wait inside the prompt
kernel did not end within a second, and the results are unspecified).

The calls serve only: they have no backward pass, and refuse inputs that require
a gradient unless gradients are off (``torch.no_grad()``).

The calls run on the tensors' device and on its current stream unless ``stream``
is given. Outputs and workspaces come from PyTorch's allocator, on the stream
of the call, so calls on several streams and captured graphs do not share any
and none is handed out again before the call has run. A tensor that is used on
another stream than the one it was allocated on is kept alive by the caller
(``Tensor.record_stream``), as for any PyTorch operator.
"""
from __future__ import annotations

import importlib.util
import os

import torch

from . import abi, build

_module = None
_bound = object()  # the library (abi.load()) whose entry points the module calls; none yet


def _native():
    """The module that takes the tensors apart (csrc/attention_torch.cpp), bound to the library that abi has loaded:
    after a change to another one (the bounds-checked build) the next call goes there."""
    global _bound
    lib = abi._lib or abi.load()
    if lib is not _bound:
        import ctypes
        (_module or _load()).bind(*(ctypes.cast(getattr(lib, name), ctypes.c_void_p).value for name in (
            "moe_qkv_append", "moe_attend_paged_workspace", "moe_attend_paged", "moe_attend_prompt_workspace",
            "moe_attend_prompt")))
        _bound = lib
    return _module


def _load():
    global _module
    if not os.path.exists(build.TORCH_LIB_PATH):
        raise RuntimeError(f"not built: {build.TORCH_LIB_PATH} (run __graft_entry__.build())")
    spec = importlib.util.spec_from_file_location("attention_torch", build.TORCH_LIB_PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    _module = module
    return module


class KVCacheMXFP4:
    """A paged key/value cache in MXFP4 (uint8 tensors, contiguous, on one CUDA device; the four stay the same).

    k_codes, v_codes:   [pages][kv heads][page size][head_dim/2], two E2M1 codes per byte (element 2i low)
    k_scales, v_scales: [pages][kv heads][page size][head_dim/32], UE8M0
    """
    __slots__ = ("_parts",)

    def __init__(self, k_codes: torch.Tensor, k_scales: torch.Tensor, v_codes: torch.Tensor, v_scales: torch.Tensor):
        module = _module if abi._lib is _bound else _native()
        module.check_cache(k_codes, k_scales, v_codes, v_scales)
        self._parts = (k_codes, k_scales, v_codes, v_scales)

    k_codes = property(lambda self: self._parts[0])
    k_scales = property(lambda self: self._parts[1])
    v_codes = property(lambda self: self._parts[2])
    v_scales = property(lambda self: self._parts[3])
    num_kv_heads = property(lambda self: self._parts[0].shape[1])
    page_size = property(lambda self: self._parts[0].shape[2])
    head_dim = property(lambda self: 2 * self._parts[0].shape[3])

    @classmethod
    def empty(cls, num_pages: int, page_size: int, num_kv_heads: int, head_dim: int, device="cuda") -> "KVCacheMXFP4":
        def make(width):
            return torch.empty((num_pages, num_kv_heads, page_size, width), dtype=torch.uint8, device=device)
        return cls(make(head_dim // 2), make(head_dim // 32), make(head_dim // 2), make(head_dim // 32))

    def as_abi(self) -> abi.MoeKvCache:
        pages, heads, page, half = self._parts[0].shape
        return abi.MoeKvCache(*(t.data_ptr() for t in self._parts), pages, page, heads, 2 * half)


def rope_table(positions: int, rotary_dim: int, theta: float = 10000.0, device="cuda") -> torch.Tensor:
    """fp32 [positions][rotary_dim]: rotary_dim/2 cosines, then as many sines, of p * theta^(-2i/rotary_dim).
    The angles are computed in 64 bits: in 32, those of far positions would be off by whole radians."""
    freq = theta ** (-torch.arange(0, rotary_dim, 2, dtype=torch.float64) / rotary_dim)
    angle = torch.arange(positions, dtype=torch.float64)[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], dim=1).float().to(device)


def _on(stream, device: torch.device):
    """The stream of a call: its outputs and workspace belong to it."""
    if not isinstance(stream, int) and stream.device != device:
        raise ValueError(f"stream is on {stream.device}, the tensors are on {device}")
    return torch.cuda.stream(torch.cuda.ExternalStream(stream, device) if isinstance(stream, int) else stream)


def _call(name: str, fn, stream, q: torch.Tensor, *args):
    if stream is None:
        result = fn(q, *args)
    else:
        with _on(stream, q.device):
            result = fn(q, *args)
    if result.__class__ is int:
        abi.check(name, result)
    return result


def qkv_append(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, *, positions: torch.Tensor | None = None,
               rope: torch.Tensor | None = None, interleaved: bool = False, q_norm: torch.Tensor | None = None,
               k_norm: torch.Tensor | None = None, eps: float = 1e-6, cache: KVCacheMXFP4 | None = None,
               slots: torch.Tensor | None = None, q_out: torch.Tensor | None = None, rotated_keys: bool = False,
               cached_values: bool = False, d_status: torch.Tensor | None = None, stream=None) -> dict:
    """Norm, rotation and append of T tokens in one pass.

    q [T][heads][D], k and v [T][kv heads][D] (bf16 or fp16; views of one fused projection are fine).
    rope fp32 [positions][R] as from ``rope_table``, R <= D, with positions int32 [T]; None: no rotation.
    q_norm, k_norm [D]: RMSNorm weights; None: that part is not normalised.
    cache with slots int64 [T] (page * page size + offset; negative: the token is not cached).
    q_out: a contiguous output for q, which may be q itself; otherwise outputs must not overlap inputs.

    Returns {"q"}, plus "k" (rotated keys in 16 bits) with rotated_keys, plus "k_cached" and "v_cached" (the
    values that the 4-bit cache keeps) with cached_values.
    """
    module = _module if abi._lib is _bound else _native()
    return _call("moe_qkv_append", module.append, stream, q, k, v, positions, rope, interleaved, q_norm, k_norm, eps,
                 cache, slots, q_out, rotated_keys, cached_values, d_status)


def attend_paged(q: torch.Tensor, cache: KVCacheMXFP4, page_table: torch.Tensor, lengths: torch.Tensor,
                 cu_rows: torch.Tensor, *, max_rows: int = 1, scale: float | None = None,
                 out: torch.Tensor | None = None, return_lse: bool = False, d_status: torch.Tensor | None = None,
                 stream=None):
    """Attention of the newest rows of each sequence over the MXFP4 cache.

    q [rows][heads][D]; page_table int32 [sequences][pages]; lengths int32 [sequences], the tokens in the
    cache with the query rows among them; cu_rows int32 [sequences + 1]: sequence b has rows
    cu_rows[b] .. cu_rows[b + 1] - 1, its last tokens, each seeing the keys up to itself. max_rows: the rows a
    sequence usually has at most: it picks the kernel variant. Any value gives right results, but the order of the
    sums, and so their last bits, follow it and the other sequences of the batch.
    scale: of the scores, 1/sqrt(D) by default. Rows that see no key give 0 and lse -inf; rows with a NaN or +inf
    among their scores give NaN in both. out must not overlap q.

    Returns out [rows][heads][D], and with return_lse also lse fp32 [rows][heads].
    """
    module = _module if abi._lib is _bound else _native()
    return _call("moe_attend_paged", module.paged, stream, q, cache, page_table, lengths, cu_rows, max_rows, scale, out,
                 return_lse, d_status)


def attend_prompt(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_rows: torch.Tensor, cu_keys: torch.Tensor, *,
                  causal: bool = True, scale: float | None = None, out: torch.Tensor | None = None,
                  return_lse: bool = False, d_status: torch.Tensor | None = None, stream=None):
    """Attention over packed prompts, or over chunks of prompts with the keys before them.

    q [rows][heads][D], k and v [keys][kv heads][D]; cu_rows, cu_keys int32 [sequences + 1]. Row i of a sequence
    with n rows and m keys sees keys 0 .. m - n + i (causal), or all m. Rows that see no key give 0 and lse -inf; rows
    with a NaN or +inf among their scores give NaN in both. out must not overlap the inputs.
    Few rows over many keys are computed in parts (the sizes of the tensors decide, not their contents).

    Returns out [rows][heads][D], and with return_lse also lse fp32 [rows][heads].
    """
    module = _module if abi._lib is _bound else _native()
    return _call("moe_attend_prompt", module.prompt, stream, q, k, v, cu_rows, cu_keys, causal, scale, out, return_lse,
                 d_status)
